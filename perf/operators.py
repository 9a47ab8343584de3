"""Cases of the serving operators over a 4-bit paged key/value cache.

A serving step of block-sparse top-k attention runs four operators in a row:

* ``step``    block table, slot map and query chunks of a batch, from each
              request's cached length and its number of new tokens;
* ``append``  the new tokens' K and V rounded to 4 bits (e2m1 codes, one e4m3
              scale per 16 dims) and written to the cache's pages, and the
              pooled index key of every key block that became complete; the
              cache is then read back as the values it stands for;
* ``select``  top-k key blocks of every query chunk, scored against the pooled
              index keys of the request's pages;
* ``attend``  attention of the new tokens over the selected blocks.

A page holds one key block (64 or 128 tokens), 16 query heads share one KV
head, a query chunk is up to 8 new tokens of one request whose positions share
position // 8, and the head dimension is 128.
"""
import math

import numpy as np
import torch

own = False

DIM, GROUP, CHUNK, SCALE_GROUP = 128, 16, 8, 16
EMPTY = -1
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a mid-sized batch, with requests that idle or finish
        dict(name="step_decode", op="step", requests=64, context=8192, new=1, ragged=True, heads=4, block=64, topk=16),
        # a mixed batch of odd size whose prompts arrive in pieces
        dict(name="step_ragged", op="step", requests=37, context=5000, new=700, ragged=True, heads=4, block=128, topk=16),
        # a large batch that takes in 100k tokens of prompts at once
        dict(name="step_prefill", op="step", requests=512, context=4096, new=400, ragged=True, heads=8, block=64, topk=32),
        # the new token of every request of a decode step
        dict(name="append_decode", op="append", requests=64, context=2048, new=1, ragged=True, heads=4, block=64, topk=16),
        # prompt pieces of odd lengths that start and end inside a page
        dict(name="append_ragged", op="append", requests=13, context=1500, new=333, ragged=True, heads=3, block=128, topk=16),
        # four prompts of 8192 tokens
        dict(name="append_prefill", op="append", requests=4, context=64, new=8192, ragged=False, heads=8, block=64, topk=32),
        # one user's decode step: latency
        dict(name="select_one", op="select", requests=1, context=8192, new=1, ragged=False, heads=4, block=64, topk=16),
        # a decode batch over long contexts
        dict(name="select_batch", op="select", requests=64, context=65536, new=1, ragged=False, heads=8, block=64, topk=32),
        # pieces of two prompts behind long contexts
        dict(name="select_prefill", op="select", requests=2, context=32768, new=2048, ragged=True, heads=4, block=64, topk=16),
        # one user's decode step: latency
        dict(name="attend_one", op="attend", requests=1, context=8192, new=1, ragged=False, heads=4, block=64, topk=16),
        # a large decode batch: every request reads its own 2048 keys per head
        dict(name="attend_batch", op="attend", requests=256, context=8192, new=1, ragged=False, heads=8, block=64, topk=32),
        # prompt pieces over cached contexts, blocks of 128 keys
        dict(name="attend_prefill", op="attend", requests=3, context=16384, new=1365, ragged=True, heads=4, block=128, topk=16),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "append", "select", "attend", "attend"])
    c = dict(op=op, heads=rng.randint(1, 8), block=rng.choice([64, 128]), topk=rng.randint(2, 32),
             ragged=rng.random() < 0.75)
    kind = rng.choice(["decode", "few", "prompt"])
    if op == "step":
        c["requests"] = _between(rng, 1, 512)
        c["context"] = _between(rng, 16, 8192)
        c["new"] = {"decode": 1, "few": rng.randint(2, 9), "prompt": _between(rng, 10, 400)}[kind]
    elif op == "append":
        c["context"] = _between(rng, 1, 2048)
        c["new"] = {"decode": 1, "few": rng.randint(2, 9), "prompt": _between(rng, 10, 8192)}[kind]
        c["requests"] = _between(rng, 1, max(1, min(256, 32768 // max(c["new"], c["context"] // 4))))
    elif op == "select":
        c["context"] = _between(rng, 8 * c["block"], 65536)
        c["topk"] = max(4, c["topk"])
        c["new"] = {"decode": 1, "few": rng.randint(2, 9), "prompt": _between(rng, 10, 2048)}[kind]
        rows = 64 * 65536 // (c["context"] * (1 + c["new"] // CHUNK))
        c["requests"] = _between(rng, 1, max(1, min(256, rows)))
    else:
        c["context"] = _between(rng, 1, 16384)
        c["new"] = {"decode": 1, "few": rng.randint(2, 9), "prompt": _between(rng, 10, 2048)}[kind]
        keys = c["topk"] * c["block"]
        chunks = 256 * 2048 // (keys * (2 + c["new"] // CHUNK))
        c["requests"] = _between(rng, 1, max(1, min(256, chunks, (256 * 8192) // (c["context"] + c["new"]))))
    return c


# ---------------------------------------------------------------------------
# inputs, made from the seed alone
# ---------------------------------------------------------------------------

def _batch(case, seed):
    """Cached and new lengths of the requests, their pages and the step's tables (host arrays).  The lengths belong
    to the case, the pages to the seed."""
    R, ctx, new, B = case["requests"], case["context"], case["new"], case["block"]
    rng = np.random.default_rng([R, ctx, new, B])
    if case["ragged"]:
        past = np.floor(np.exp(rng.uniform(0.0, math.log(ctx + 1.0), R))).astype(np.int64)
        past[rng.random(R) < 0.05] = 0
        n = rng.integers(1, new + 1, R)
    else:
        past = np.full(R, ctx, np.int64) - rng.integers(0, min(B, ctx), R)
        n = np.full(R, new, np.int64)
    past[0], n[0] = ctx, new  # the batch reaches the case's size
    if case["op"] == "append":
        # a piece that reaches past the next block starts at a page, as a scheduler cuts prompts (the pass then
        # leaves its own inputs, the tail's rows, as they were, and can be made again)
        past = np.where((past + n) // B >= past // B + 2, past // B * B, past)
    if case["op"] == "step" and R > 2:
        idle = rng.random(R)
        n = np.where(idle < 0.06, 0, np.where(idle < 0.12, -1, n))  # -1: the request has finished
        n[0] = new
    past_blocks, blocks = -(-past // B), -(-(past + np.maximum(n, 0)) // B)
    M = int(blocks.max()) + 3
    P = int(blocks.sum()) + 5
    rng = np.random.default_rng([seed, 1])
    order = rng.permutation(P)
    held = past_blocks if case["op"] == "step" else blocks
    table = np.zeros((R, M), np.int32)
    first = np.concatenate([[0], np.cumsum(held)])
    for r in range(R):
        table[r, :held[r]] = order[first[r]:first[r + 1]]
    free = order[first[-1]:]
    # free pages in a ring that starts anywhere
    head = int(rng.integers(0, P))
    ring = np.zeros(P, np.int32)
    ring[(head + np.arange(len(free))) % P] = free
    b = dict(R=R, B=B, M=M, P=P, past=past, new=n, table=table, ring=ring, head=head, free=len(free))
    b.update(_tables(b))
    return b


def _tables(b):
    """Token rows, slots, positions and query chunks of the new tokens (op "step" computes the same on the device)."""
    past, n, B = b["past"], np.maximum(b["new"], 0), b["B"]
    cu = np.concatenate([[0], np.cumsum(n)])
    T = int(cu[-1])
    req = np.repeat(np.arange(b["R"]), n)
    pos = past[req] + np.arange(T) - cu[req]
    slots = b["table"][req, pos // B].astype(np.int64) * B + pos % B
    starts = np.flatnonzero((np.diff(req, prepend=-1) != 0) | (pos % CHUNK == 0))
    counts = np.diff(np.append(starts, T))
    chunks = np.stack([req[starts], starts, counts, pos[starts]], 1).astype(np.int32)
    return dict(cu=cu.astype(np.int32), T=T, req=req, pos=pos, slots=slots, chunks=chunks, NC=len(chunks))


def _gen(seed, what):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 64 + what)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _kv_slices(case, seed, b, rows, step=1 << 16):
    """K and V of `rows` cached tokens, bf16 [n, heads, 128], a slice at a time: (first row, K, V).  A few channels
    of K are larger than the others, as rotary-embedded keys have them; V differs by head."""
    H = case["heads"]
    g = _gen(seed, 2)
    kc = torch.exp(0.4 * _randn((H, DIM), g))
    kc[:, ::37] *= 4.0
    vc = torch.exp(0.5 * _randn((H, 1), g))
    for i in range(0, rows, step):
        m = min(step, rows - i)
        yield i, (_randn((m, H, DIM), g) * kc).bfloat16(), (_randn((m, H, DIM), g) * vc).bfloat16()


def _selection(case, seed, b):
    """A selection as the scorer makes it: each chunk's own block, then distinct earlier ones; -1 fills the rest."""
    rng = np.random.default_rng([seed, 3])
    H, K, NC = case["heads"], case["topk"], b["NC"]
    diag = b["chunks"][:, 3] // b["B"]
    sel = np.full((H, NC, K), EMPTY, np.int32)
    sel[:, :, 0] = diag
    for g in range(NC):
        d, k = int(diag[g]), min(K - 1, int(diag[g]))
        for h in range(H):
            sel[h, g, 1:1 + k] = rng.choice(d, k, replace=False) if k else 0
    return sel


def _put(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x), device=DEV).to(dtype)


# ---------------------------------------------------------------------------
# state
# ---------------------------------------------------------------------------

def prepare(case, seed):
    b = _batch(case, seed)
    s = dict(op=case["op"], case=case, b=b, own=own)
    H, T, NC, P, B = case["heads"], b["T"], b["NC"], b["P"], b["B"]
    if own:
        from block_sparse_top_attn_gb300 import binding
        s["B"] = binding
        s["c"] = binding.make_cache_problem(num_requests=b["R"], num_pages=P, max_blocks=b["M"], num_q_heads=H * GROUP,
                                            topk=case["topk"], block_size=B, token_cap=T, chunk_cap=NC, device=DEV)
        s["status"] = torch.zeros(4, dtype=torch.int32, device=DEV)
    s["table"] = _put(b["table"])
    if case["op"] == "step":
        s["new"], s["past"] = _put(b["new"]), _put(b["past"])
        s["ring"], s["ring_at"] = _put(b["ring"]), _put([b["head"], b["free"]])
        s["cu"] = torch.zeros(b["R"] + 1, dtype=torch.int32, device=DEV)
        s["slots"] = torch.zeros(T, dtype=torch.int64, device=DEV)
        s["pos"] = torch.zeros(T, dtype=torch.int32, device=DEV)
        s["chunks"] = torch.zeros((NC, 4), dtype=torch.int32, device=DEV)
        s["past_out"], s["ring_at_out"] = torch.zeros_like(s["past"]), torch.zeros_like(s["ring_at"])
        return s
    s["cu"], s["chunks"], s["slots"] = _put(b["cu"]), _put(b["chunks"]), _put(b["slots"], torch.int64)
    if case["op"] == "append":
        _, s["k"], s["v"] = next(_kv_slices(case, seed, b, T, T))
        g = _gen(seed, 4)
        s["k_index"] = _randn((T, H, DIM), g).bfloat16()
        # index keys of the blocks that the cached tokens left incomplete
        s["tail"] = _randn((b["R"], 2, B, H, DIM), g).bfloat16()
        s["pool"] = torch.zeros((P, H, DIM), dtype=torch.bfloat16, device=DEV)
        # rows that complete a block, and rows whose block stays incomplete
        s["done"] = _put(np.flatnonzero(b["pos"] % B == B - 1), torch.int64)
        end = (b["past"] + b["new"])[b["req"]]
        s["keep"] = _put(np.flatnonzero((b["pos"] // B + 1) * B > end), torch.int64)
    elif case["op"] == "select":
        g = _gen(seed, 5)
        s["pool"] = (_randn((P, H, DIM), g) / math.sqrt(B)).bfloat16()
        s["q_index"] = _randn((T, H, DIM), g).bfloat16()
        s["sel"] = torch.full((H, NC, case["topk"]), EMPTY, dtype=torch.int32, device=DEV)
    else:
        s["q"] = _randn((T, H * GROUP, DIM), _gen(seed, 6)).bfloat16()
        s["sel"] = _put(_selection(case, seed, b))
        of_chunk = np.repeat(np.arange(NC), b["chunks"][:, 2])
        nq = int(b["chunks"][:, 2].max())
        s["place"] = _put(of_chunk * nq + np.arange(T) - b["chunks"][of_chunk, 1], torch.int64)  # in [chunks, nq]
    if case["op"] in ("append", "attend"):
        if own:
            s["cache"] = s["B"].new_cache(s["c"], device=DEV)
        else:
            s["codes"] = torch.zeros((P * B, H, 2, DIM), dtype=torch.uint8, device=DEV)
            s["scales"] = torch.zeros((P * B, H, 2, DIM // SCALE_GROUP), dtype=torch.float32, device=DEV)
    if case["op"] == "attend":  # every token of every request is in the cache
        slots = _put(_all_slots(b), torch.int64)
        for i, k, v in _kv_slices(case, seed, b, len(slots)):
            at = slots[i:i + len(k)]
            if own:
                c = s["B"].make_cache_problem(num_requests=1, num_pages=P, max_blocks=1, num_q_heads=H * GROUP,
                                              topk=1, block_size=B, token_cap=len(k), chunk_cap=1, device=DEV)
                s["B"].msa_cache_append(c, k, v, None, at, None, None, s["cache"], None, None, s["status"])
            else:
                _write(s, at, k, v)
        if own:
            s["o"] = torch.zeros((T, H * GROUP, DIM), dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.zeros((T, H * GROUP), dtype=torch.float32, device=DEV)
    return s


def _all_slots(b):
    """Slots of every token of every request, request by request."""
    total = b["past"] + np.maximum(b["new"], 0)
    req = np.repeat(np.arange(b["R"]), total)
    pos = np.arange(int(total.sum())) - np.repeat(np.concatenate([[0], np.cumsum(total)])[:-1], total)
    return b["table"][req, pos // b["B"]].astype(np.int64) * b["B"] + pos % b["B"]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return {"step": _run_step, "append": _run_append, "select": _run_select, "attend": _run_attend}[s["op"]](s)


def _run_step(s):
    if own:
        s["B"].msa_cache_step(s["c"], s["new"], s["past"], s["ring_at"], s["ring"], s["table"], s["past_out"],
                              s["ring_at_out"], s["cu"], s["slots"], s["pos"], s["chunks"], s["status"])
        return [s[k] for k in ("cu", "slots", "pos", "chunks", "table", "past_out", "ring_at_out", "ring")]
    b = s["b"]
    B, P, R, M, T, NC = b["B"], b["P"], b["R"], b["M"], b["T"], b["NC"]
    past, n = s["past"].long(), s["new"].clamp(min=0).long()
    head, count = s["ring_at"][0].long(), s["ring_at"][1].long()
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    old_blocks, blocks = (past + B - 1) // B, (past + n + B - 1) // B
    alloc = torch.cat([zero, torch.cumsum(blocks - old_blocks, 0)])
    cu = torch.cat([zero, torch.cumsum(n, 0)])
    # tokens
    rows = torch.arange(T, device=DEV)
    req = torch.searchsorted(cu[1:].contiguous(), rows, right=True).clamp(max=R - 1)
    pos = past[req] + rows - cu[req]
    blk = pos // B
    fresh = s["ring"][(head + alloc[req] + (blk - old_blocks[req]).clamp(min=0)) % P].long()
    page = torch.where(blk < old_blocks[req], s["table"][req, blk.clamp(max=M - 1)].long(), fresh)
    live = rows < cu[-1]
    slots = torch.where(live, page * B + pos % B, EMPTY)
    # the table's new entries: the token that opens a page writes it
    at = torch.where(live & (pos % B == 0), req * M + blk, R * M)
    table = torch.cat([s["table"].reshape(-1), zero.int()]).index_put((at,), page.int())[:-1].view(R, M)
    # query chunks
    nch = torch.where(n > 0, (past + n - 1) // CHUNK - past // CHUNK + 1, 0)
    cch = torch.cat([zero, torch.cumsum(nch, 0)])
    g = torch.arange(NC, device=DEV)
    cr = torch.searchsorted(cch[1:].contiguous(), g, right=True).clamp(max=R - 1)
    slot = past[cr] // CHUNK + g - cch[cr]
    first = torch.maximum(past[cr], slot * CHUNK)
    last = torch.minimum(past[cr] + n[cr], slot * CHUNK + CHUNK)
    chunks = torch.stack([cr, cu[cr] + first - past[cr], last - first, first], 1)
    chunks = torch.where((g < cch[-1])[:, None], chunks, EMPTY).int()
    # pages of finished requests go to the ring's end
    given = torch.where(s["new"] < 0, old_blocks, 0)
    cg = torch.cat([zero, torch.cumsum(given, 0)])
    j = torch.arange(P, device=DEV)
    gr = torch.searchsorted(cg[1:].contiguous(), j, right=True).clamp(max=R - 1)
    back = s["table"][gr, (j - cg[gr]).clamp(0, M - 1)]
    at = torch.where(j < cg[-1], (head + count + j) % P, P)
    ring = torch.cat([s["ring"], zero.int()]).index_put((at,), back)[:-1]
    past_out = torch.where(s["new"] < 0, 0, past + n).int()
    ring_at = torch.stack([(head + alloc[-1]) % P, count - alloc[-1] + cg[-1]]).int()
    return [cu.int(), slots, torch.where(live, pos, EMPTY).int(), chunks, table, past_out, ring_at, ring]


def _round(x):
    """Codes (0..15, the sign on top) and scales of rows in groups of 16: the scale is max / 6 rounded to e4m3, a
    code the nearest multiple of it among e2m1's values, ties to the even code."""
    g = x.float().view(*x.shape[:-1], DIM // SCALE_GROUP, SCALE_GROUP)
    t = g.abs().amax(-1) / 6.0
    _, e = torch.frexp(t)
    step = torch.exp2((e - 1).clamp(min=-6).float() - 3.0)
    scale = (torch.round(t / step) * step).clamp(max=448.0)
    a, d = g.abs(), scale[..., None]
    code = ((a > 0.25 * d).byte() + (a >= 0.75 * d).byte() + (a > 1.25 * d).byte() + (a >= 1.75 * d).byte()
            + (a > 2.5 * d).byte() + (a >= 3.5 * d).byte() + (a > 5.0 * d).byte())
    code = torch.where(d > 0, code + 8 * (g < 0).byte(), 0)
    return code.view(x.shape).byte(), scale


def _write(s, slots, k, v):
    for i, x in enumerate((k, v)):
        s["codes"][slots, :, i], s["scales"][slots, :, i] = _round(x)


def _values(codes, scales):
    """fp32 values of codes [..., 128] and scales [..., 8]."""
    lut = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=DEV)
    x = lut[codes.int()]
    return (x.view(*x.shape[:-1], -1, SCALE_GROUP) * scales[..., None]).view(x.shape)


def _run_append(s):
    if own:
        B = s["B"]
        B.msa_cache_append(s["c"], s["k"], s["v"], s["k_index"], s["slots"], s["cu"], s["chunks"], s["cache"],
                           s["tail"], s["pool"], s["status"])
        k, v = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        B.msa_cache_read(s["c"], s["slots"], s["cache"], k, v, s["status"])
        return [k, v, s["tail"], s["pool"]]
    b = s["b"]
    B, T = b["B"], b["T"]
    _write(s, s["slots"], s["k"], s["v"])
    kv = _values(s["codes"][s["slots"]], s["scales"][s["slots"]]).bfloat16()
    # every new token's place in its block
    rows = torch.arange(T, device=DEV)
    req = torch.searchsorted(s["cu"][1:].contiguous(), rows.int(), right=True)
    of_chunk = torch.searchsorted(s["chunks"][:, 1].contiguous(), rows.int(), right=True) - 1
    pos = s["chunks"][of_chunk, 3] + rows - s["chunks"][of_chunk, 1]
    blk, off = pos // B, pos % B
    # block means: the tokens of the call, and of earlier calls from the tail, in order
    done, keep = s["done"], s["keep"]
    if len(done):
        r, at = req[done], done - (B - 1)
        acc = torch.zeros((len(done), *s["k_index"].shape[1:]), device=DEV)
        for i in range(B):
            now = (at + i >= s["cu"][r])[:, None, None]
            acc = acc + torch.where(now, s["k_index"][(at + i).clamp(min=0)], s["tail"][r, blk[done] & 1, i]).float()
        s["pool"][s["slots"][done] // B] = (acc / B).bfloat16()
    s["tail"][req[keep], blk[keep] & 1, off[keep]] = s["k_index"][keep]
    return [kv[:, :, 0].contiguous(), kv[:, :, 1].contiguous(), s["tail"], s["pool"]]


def _run_select(s):
    if own:
        s["B"].msa_cache_select(s["c"], s["q_index"], s["pool"], s["table"], s["chunks"], s["sel"], s["status"])
        return s["sel"]
    b, case = s["b"], s["case"]
    NC, K, M = b["NC"], case["topk"], b["M"]
    r, row, n, first = s["chunks"].long().unbind(1)
    acc = torch.zeros((NC, case["heads"], DIM), device=DEV)
    for i in range(CHUNK):
        x = s["q_index"][(row + i).clamp(max=b["T"] - 1)].float()
        acc = torch.where((i < n)[:, None, None], acc + x, acc)
    q = (acc / n[:, None, None]).bfloat16().float()  # the mean of the chunk's index queries
    diag = first // b["B"]
    for h in range(case["heads"]):
        for at in range(0, NC, max(1, (1 << 20) // M)):
            c = slice(at, at + max(1, (1 << 20) // M))
            k = s["pool"][s["table"][r[c]].long(), h].float().permute(2, 0, 1).contiguous()  # [128, chunks, blocks]
            score = torch.zeros(k.shape[1:], device=DEV)
            for d in range(DIM):  # in the order of the dims: a product of two bf16 values is exact in fp32
                score = score + q[c, h, d, None] * k[d]
            earlier = torch.arange(M, device=DEV) < diag[c, None]
            score = torch.where(earlier, score + 0.0, -math.inf)
            top = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :K - 1]
            pad = torch.full((len(top), K), EMPTY, device=DEV, dtype=torch.long)
            pad[:, 0] = diag[c]
            live = torch.arange(top.shape[1], device=DEV) < diag[c, None]
            pad[:, 1:1 + top.shape[1]] = torch.where(live, top, EMPTY)
            s["sel"][h, c] = pad.int()
    return s["sel"]


def _run_attend(s):
    if own:
        s["B"].msa_cache_fwd(s["c"], s["q"], s["cache"], s["table"], s["chunks"], s["sel"], s["o"], s["lse"],
                             s["status"])
        return [s["o"], s["lse"]]
    b, case = s["b"], s["case"]
    B, H, K, NC, T = b["B"], case["heads"], case["topk"], b["NC"], b["T"]
    nq = int(b["chunks"][:, 2].max())
    r, row, _, first = s["chunks"].long().unbind(1)
    o = torch.empty((T, H, GROUP, DIM), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((T, H, GROUP), device=DEV)
    q = s["q"].view(T, H, GROUP, DIM)
    tok = torch.arange(nq, device=DEV)
    step = max(1, (1 << 21) // (K * B))
    for h in range(H):
        for at in range(0, NC, step):
            c = slice(at, at + step)
            sel = s["sel"][h, c].long()
            page = s["table"][r[c, None], sel.clamp(min=0)].long()
            inside = torch.arange(B, device=DEV)
            slots = (page[:, :, None] * B + inside).flatten(1)
            pos = torch.where(sel[:, :, None] >= 0, sel[:, :, None] * B + inside, 1 << 40).flatten(1)
            k, v = (_values(s["codes"][slots, h, i], s["scales"][slots, h, i]) for i in (0, 1))
            rows = (row[c, None] + tok).clamp(max=T - 1)
            x = torch.matmul(q[rows, h].float().flatten(1, 2), k.transpose(1, 2)) * DIM ** -0.5
            x = x.view(len(sel), nq, GROUP, -1)
            seen = pos[:, None, None, :] <= (first[c, None] + tok)[:, :, None, None]
            x = torch.where(seen, x, -math.inf)
            m = x.amax(-1, keepdim=True).clamp(min=-3e38)
            p = torch.exp(x - m)
            l = p.sum(-1, keepdim=True)
            y = torch.matmul(p.flatten(1, 2), torch.where(seen.any(1)[:, 0, :, None], v, 0)).view(*x.shape[:3], DIM)
            y = torch.where(l > 0, y / l, 0).bfloat16()
            z = (m + torch.log(l))[..., 0]
            t = slice(int(b["chunks"][at, 1]), int(b["chunks"][at:at + step, 1:3].sum(1).max()))
            place = s["place"][t] - at * nq
            o[t, h], lse[t, h] = y.flatten(0, 1)[place], z.flatten(0, 1)[place]
    return [o.view(T, H * GROUP, DIM), lse.view(T, H * GROUP)]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    b = _batch(case, 0)
    R, H, B, K, T, NC = b["R"], case["heads"], b["B"], case["topk"], b["T"], b["NC"]
    total = b["past"] + np.maximum(b["new"], 0)
    past_blocks, blocks = -(-b["past"] // B), -(-total // B)
    kept = DIM // 2 + DIM // SCALE_GROUP  # bytes of one token's K (or V) of one head in the cache
    if case["op"] == "step":
        # lengths in and out, token offsets; slot and position of every token; chunks; pages taken and given back
        pages = int((blocks - past_blocks).sum() + past_blocks[b["new"] < 0].sum())
        return dict(bytes=16 * R + 12 * T + 16 * NC + 8 * pages, flops=8 * T)
    if case["op"] == "append":
        # K, V and index keys in; the cache's bytes out and in again, its values out; the pooled keys of the blocks
        # that become complete, or the tail's rows
        done = int((total // B - b["past"] // B).sum())
        tail = int((total - np.maximum(b["past"], total // B * B)).sum())
        back = int(np.where(total // B > b["past"] // B, b["past"] % B, 0).sum())
        rows = 3 * 2 * DIM + 2 * 2 * kept + 2 * 2 * DIM
        return dict(bytes=H * (T * rows + 2 * DIM * (done + tail + back)) + 8 * T, flops=T * H * DIM * 8)
    first = b["chunks"][:, 3].astype(np.int64)
    req, rows = b["chunks"][:, 0], b["chunks"][:, 2].astype(np.int64)
    if case["op"] == "select":
        most = np.zeros(R, np.int64)
        np.maximum.at(most, req, first // B)
        return dict(bytes=H * 2 * DIM * (T + int(most.sum())) + NC * (H * K * 4 + 16) + 4 * int(most.sum()),
                    flops=2 * DIM * H * int((first // B).sum()))
    # keys of a chunk: its own block up to its last query, and whole earlier blocks
    keys = np.minimum(K - 1, first // B) * B + (first + rows - 1) % B + 1
    per_request = np.zeros(R, np.int64)
    np.add.at(per_request, req, keys)
    read = int(np.minimum(per_request, total).sum())  # chunks of one request may share blocks: each is read once
    return dict(bytes=H * read * 2 * kept + T * H * GROUP * (4 * DIM + 4) + NC * (H * K * 4 + 16),
                flops=4 * DIM * H * GROUP * int((keys * rows).sum()))


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    b = _batch(case, seed)
    return {"step": _exact_step, "append": _exact_append, "select": _exact_select,
            "attend": _exact_attend}[case["op"]](case, seed, b)


def _exact_step(case, seed, b):
    table, ring = b["table"].copy(), b["ring"].copy()
    P, B = b["P"], b["B"]
    head, count = b["head"], b["free"]
    taken, after, cu, slots, pos, chunks = 0, [], [0], [], [], []
    for r in range(b["R"]):
        past, n = int(b["past"][r]), int(b["new"][r])
        after.append(past + n if n >= 0 else 0)
        for p in range(past, past + n):
            if p % B == 0:
                table[r, p // B] = ring[(head + taken) % P]
                taken += 1
            if p == past or p % CHUNK == 0:
                chunks.append([r, len(pos), 0, p])
            chunks[-1][2] += 1
            slots.append(int(table[r, p // B]) * B + p % B)
            pos.append(p)
        cu.append(len(pos))
    given = 0
    for r in range(b["R"]):
        if b["new"][r] < 0:
            for i in range(-(-int(b["past"][r]) // B)):
                ring[(head + count + given) % P] = table[r, i]
                given += 1
    i32 = lambda x: np.asarray(x, np.int32)
    return [i32(cu), np.asarray(slots, np.int64), i32(pos), i32(chunks).reshape(-1, 4), table, i32(after),
            i32([(head + taken) % P, count - taken + given]), ring]


def _e4m3_values():
    x = [m * 2.0 ** -9 for m in range(8)]
    for e in range(1, 16):
        x += [(8 + m) * 2.0 ** (e - 10) for m in range(8)]
    return x[:-1]  # the last pattern is no number


def _nearest(x, values):
    """Index of the nearest of ascending `values` to x >= 0, ties to the even index, the largest value beyond."""
    v = torch.tensor(values, dtype=torch.float64, device=x.device)
    up = torch.searchsorted(v, x.contiguous()).clamp(1, len(values) - 1)
    lo, hi = v[up - 1], v[up]
    pick_up = ((hi - x) < (x - lo)) | (((hi - x) == (x - lo)) & (up % 2 == 0))
    return torch.where(pick_up, up, up - 1)


def _rounded64(x):
    """fp64 values that 4 bits and a scale keep of bf16 rows [..., 128]."""
    g = x.double().unflatten(-1, (DIM // SCALE_GROUP, SCALE_GROUP))
    e4 = torch.tensor(_e4m3_values(), dtype=torch.float64, device=x.device)
    scale = e4[_nearest(g.abs().amax(-1) / 6.0, _e4m3_values())][..., None]
    # against the scaled levels, which are exact, so that no quotient is rounded
    best = torch.zeros_like(g)
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    for i in range(1, 8):
        mid = (levels[i - 1] + levels[i]) / 2 * scale
        above = (g.abs() > mid) if i % 2 else (g.abs() >= mid)
        best = torch.where(above, levels[i] * scale, best)
    return (best * torch.sign(g)).flatten(-2)


def _exact_append(case, seed, b):
    H, B, T, P = case["heads"], b["B"], b["T"], b["P"]
    _, k, v = next(_kv_slices(case, seed, b, T, T))
    g = _gen(seed, 4)
    ki = _randn((T, H, DIM), g).bfloat16()
    tail = _randn((b["R"], 2, B, H, DIM), g).bfloat16()
    old, new_tail = tail.double(), tail.double().clone()
    pool = torch.zeros((P, H, DIM), dtype=torch.float64, device=DEV)
    x = ki.double()
    for r in range(b["R"]):
        past, n, row = int(b["past"][r]), int(b["new"][r]), int(b["cu"][r])
        for blk in range(past // B, -(-(past + n) // B)):
            lo, hi = max(past, blk * B), min(past + n, (blk + 1) * B)
            fresh = x[row + lo - past:row + hi - past]
            if hi == (blk + 1) * B:
                pool[b["table"][r, blk]] = (old[r, blk % 2, :lo - blk * B].sum(0) + fresh.sum(0)) / B
            else:
                new_tail[r, blk % 2, lo - blk * B:hi - blk * B] = fresh
    return [_rounded64(k), _rounded64(v), new_tail, pool]


def _exact_select(case, seed, b):
    """The order of the blocks is decided by scores that are rounded to fp32 after each of 128 additions; here each
    addition is made in fp64 and rounded."""
    NC, H, K, T = b["NC"], case["heads"], case["topk"], b["T"]
    g = _gen(seed, 5)
    pool = (_randn((b["P"], H, DIM), g) / math.sqrt(b["B"])).bfloat16()
    qi = _randn((T, H, DIM), g).bfloat16()
    sel = np.full((H, NC, K), EMPTY, np.int32)
    row = torch.as_tensor(b["chunks"][:, 1].astype(np.int64), device=DEV)
    n = torch.as_tensor(b["chunks"][:, 2].astype(np.int64), device=DEV)[:, None, None]
    total = torch.zeros((NC, H, DIM), dtype=torch.float64, device=DEV)
    for i in range(CHUNK):
        x = qi[torch.clamp(row + i, max=T - 1)].double()
        total = torch.where(i < n, (total + x).float().double(), total)
    mean = (total / n).float().bfloat16().double()
    by_request = {}
    for c, (r, _, _, first) in enumerate(b["chunks"].tolist()):
        by_request.setdefault(r, []).append((c, first // b["B"]))
    for r, members in by_request.items():
        which = torch.as_tensor([c for c, _ in members], device=DEV)
        most = max(d for _, d in members)
        pages = torch.as_tensor(b["table"][r, :most].astype(np.int64), device=DEV)
        k = pool[pages].double()
        score = torch.zeros((len(members), H, most), dtype=torch.float64, device=DEV)
        for d in range(DIM):
            score = (score + mean[which][:, :, d, None] * k[:, :, d].T[None]).float().double()
        score = score.cpu().numpy()
        for i, (c, diag) in enumerate(members):
            for h in range(H):
                order = np.lexsort((np.arange(diag), -score[i, h, :diag]))[:K - 1]
                sel[h, c, 0] = diag
                sel[h, c, 1:1 + len(order)] = order
    return sel


def _exact_attend(case, seed, b):
    H, K, B, T, NC = case["heads"], case["topk"], b["B"], b["T"], b["NC"]
    q = _randn((T, H * GROUP, DIM), _gen(seed, 6)).bfloat16().view(T, H, GROUP, DIM)
    sel = _selection(case, seed, b)
    total = b["past"] + b["new"]
    start = np.concatenate([[0], np.cumsum(total)])[:-1]
    k = torch.empty((int(total.sum()), H, DIM), dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    for i, ks, vs in _kv_slices(case, seed, b, len(k)):
        k[i:i + len(ks)], v[i:i + len(ks)] = ks, vs
    nq = int(b["chunks"][:, 2].max())
    r, row, n, first = (b["chunks"][:, i].astype(np.int64) for i in range(4))
    o = torch.zeros((T, H, GROUP, DIM), dtype=torch.float64, device=DEV)
    lse = torch.zeros((T, H, GROUP), dtype=torch.float64, device=DEV)
    step = max(1, (1 << 20) // (K * B))
    dev = lambda x: torch.as_tensor(x, device=DEV)
    for h in range(H):
        for at in range(0, NC, step):
            c = slice(at, min(NC, at + step))
            s = sel[h, c].astype(np.int64)[:, :, None]
            pos = (s * B + np.arange(B)).reshape(len(s), -1)
            there = (np.broadcast_to(s >= 0, s.shape[:2] + (B,)).reshape(pos.shape)) & (pos < total[r[c]][:, None])
            idx = dev(np.where(there, start[r[c]][:, None] + pos, 0))
            kk, vv = _rounded64(k[:, h][idx]), _rounded64(v[:, h][idx])
            rows = dev(np.minimum(row[c][:, None] + np.arange(nq), T - 1))
            x = torch.einsum("cqgd,ckd->cqgk", q[:, h][rows].double(), kk) / math.sqrt(DIM)
            seen = dev(there[:, None, :] & (pos[:, None, :] <= (first[c][:, None] + np.arange(nq))[:, :, None]))
            x = x.masked_fill(~seen[:, :, None, :], -math.inf)
            z = torch.logsumexp(x, -1)
            y = torch.einsum("cqgk,ckd->cqgd", torch.exp(x - z[..., None]), vv)
            live = dev(np.arange(nq) < n[c][:, None])
            o[rows[live], h], lse[rows[live], h] = y[live], z[live]
    return [o.view(T, H * GROUP, DIM), lse.view(T, H * GROUP)]
