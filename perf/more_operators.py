"""Cases of the operators between the projections and the attention.

Block-sparse attention takes queries, keys and index vectors that are normed
and carry their positions:

* ``fwd``     RMS norm of every head of Q, K, index Q and index K with learned
              weights, and the rotary rotation of their positions;
* ``bwd``     its gradients to the inputs and to the weights;
* ``append``  the same in a serving step: Q and index Q normed and rotated, K
              normed, rotated and rounded to the 4 bits of the paged cache (e2m1
              codes, one e4m3 scale per 16 dims), V rounded, and the pooled
              index key of every key block that became complete; the cache is
              then read back as the values it stands for.

The inputs are views of one projection's output, a row per token: Q (16 heads
per KV head), K, V, index Q, index K, 128 dims each.  The first ``rotary`` dims
of a head rotate; pair p is dims (p, p + rotary / 2), or (2p, 2p + 1) where
``adjacent``.  A pair follows one of ``axes`` position columns (text: one; time,
height and width of images and video: three).
"""
import math

import numpy as np
import torch

own = False

DIM, GROUP, CHUNK, SCALE_GROUP = 128, 16, 8, 16
EPS = 1e-6
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DEV = "cuda"
ROLES = ("q", "k", "q_index", "k_index")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    text = dict(axes=1, rotary=128, adjacent=False, per_head=False, norm=True, index=True, wide_weights=False)
    return [
        # one new token of one user: latency
        dict(text, name="fwd_one", op="fwd", tokens=1, start=8191, doc=8192, heads=4),
        # a packed training batch, half of a head's dims rotated, no index vectors
        dict(text, name="fwd_varlen32k", op="fwd", tokens=32768, start=0, doc=8192, heads=4, rotary=64, index=False),
        # images and text, odd length, a weight per head, neighbouring dims paired
        dict(text, name="fwd_vision", op="fwd", tokens=5003, start=1200, doc=16384, heads=3, axes=3, adjacent=True,
             per_head=True, wide_weights=True),
        # one long training document
        dict(text, name="fwd_long128k", op="fwd", tokens=131072, start=0, doc=131072, heads=8),
        # the smallest training problem
        dict(text, name="bwd_tiny", op="bwd", tokens=512, start=0, doc=512, heads=1, wide_weights=True),
        dict(text, name="bwd_vision", op="bwd", tokens=5003, start=1200, doc=16384, heads=3, axes=3, adjacent=True,
             per_head=True, wide_weights=True),
        dict(text, name="bwd_varlen32k", op="bwd", tokens=32768, start=0, doc=8192, heads=4, rotary=64, index=False),
        dict(text, name="bwd_long128k", op="bwd", tokens=131072, start=0, doc=131072, heads=8),
        # one user's decode step: latency
        dict(text, name="append_one", op="append", requests=1, context=8192, new=1, ragged=False, heads=4, block=64),
        # the new token of every request of a large decode batch
        dict(text, name="append_decode", op="append", requests=256, context=8192, new=1, ragged=True, heads=8, block=64),
        # prompt pieces of odd lengths with images, over blocks of 128 keys
        dict(text, name="append_vision", op="append", requests=13, context=1500, new=333, ragged=True, heads=3,
             block=128, axes=3, rotary=96, per_head=True, wide_weights=True),
        # four prompts of 8192 tokens
        dict(text, name="append_prefill", op="append", requests=4, context=64, new=8192, ragged=False, heads=8, block=64),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "append"])
    c = dict(op=op, heads=rng.randint(1, 8), axes=rng.choice([1, 1, 2, 3]), rotary=rng.choice([32, 64, 96, 128, 128]),
             adjacent=rng.random() < 0.4, per_head=rng.random() < 0.4, norm=rng.random() < 0.85,
             index=rng.random() < 0.7, wide_weights=rng.random() < 0.5)
    if op == "append":
        c["block"], c["ragged"] = rng.choice([64, 128]), rng.random() < 0.75
        c["context"] = _between(rng, 1, 16384)
        kind = rng.choice(["decode", "few", "prompt"])
        c["new"] = {"decode": 1, "few": rng.randint(2, 9), "prompt": _between(rng, 10, 8192)}[kind]
        most = min(256, 32768 // c["new"], (1 << 20) // (c["context"] + c["new"]))
        c["requests"] = _between(rng, 1, max(1, most))
    else:
        c["tokens"], c["doc"] = _between(rng, 1, 131072), _between(rng, 1, 131072)
        c["start"] = rng.randrange(c["doc"])
    return c


# ---------------------------------------------------------------------------
# inputs, made from the seed alone
# ---------------------------------------------------------------------------

def _counts(case):
    """Heads of q, k, q_index, k_index and v, in this order (0: none)."""
    H = case["heads"]
    return dict(q=GROUP * H, k=H, q_index=H if case["index"] else 0, k_index=H if case["index"] else 0, v=H)


def _spans(pos, axes):
    """Position columns of running positions: text counts on in every column; of every 700 positions the last 560 are an
    image of 28 columns, which has one time and its rows and columns."""
    cols = np.repeat(pos[:, None], axes, 1)
    i = pos % 700 - 140
    image = i >= 0
    base = pos - i
    grid = np.stack([base, base + i // 28, base + i % 28], 1)[:, 3 - axes:]
    return np.where(image[:, None] & (axes > 1), grid, cols).astype(np.int32)


def _pair_axes(case):
    """Position column of each pair: the columns' pairs follow one another, the first column's are fewest."""
    n, A = case["rotary"] // 2, case["axes"]
    if A == 1:
        return np.zeros(n, np.int64)
    if A == 2:
        return np.repeat([0, 1], n // 2)
    return np.repeat([0, 1, 2], [n // 4, 3 * n // 8, 3 * n // 8])


def _inv_freq(case):
    """Radians per position of each pair, fp64."""
    n = case["rotary"] // 2
    return np.array([5e6 ** (-i / n) for i in range(n)])


def _documents(case):
    """Positions of packed documents; the first one starts at position `start`."""
    rng = np.random.default_rng([case["tokens"], case["doc"], case["start"]])
    pos, n, at = [], 0, case["start"]
    while n < case["tokens"]:
        length = int(math.exp(rng.uniform(math.log(max(1, case["doc"] // 16)), math.log(case["doc"] + 1)))) if n else \
            max(1, case["doc"] - at)
        pos.append(np.arange(at, at + length))
        n, at = n + length, 0
    return np.concatenate(pos)[:case["tokens"]]


def _batch(case, seed):
    """Cached and new lengths of a serving step's requests, their pages and tables (host arrays).  The lengths belong to
    the case, the pages to the seed."""
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
    # a piece that reaches past the next block starts at a page, as a scheduler cuts prompts (the pass then leaves its
    # own inputs, the tail's rows, as they were, and can be made again)
    past = np.where((past + n) // B >= past // B + 2, past // B * B, past)
    blocks = -(-(past + n) // B)
    M, P = int(blocks.max()) + 3, int(blocks.sum()) + 5
    order = np.random.default_rng([seed, 1]).permutation(P)
    table = np.zeros((R, M), np.int64)
    first = np.concatenate([[0], np.cumsum(blocks)])
    for r in range(R):
        table[r, :blocks[r]] = order[first[r]:first[r + 1]]
    cu = np.concatenate([[0], np.cumsum(n)])
    T = int(cu[-1])
    req = np.repeat(np.arange(R), n)
    pos = past[req] + np.arange(T) - cu[req]
    slots = table[req, pos // B] * B + pos % B
    starts = np.flatnonzero((np.diff(req, prepend=-1) != 0) | (pos % CHUNK == 0))
    counts = np.diff(np.append(starts, T))
    chunks = np.stack([req[starts], starts, counts, pos[starts]], 1)
    return dict(R=R, B=B, M=M, P=P, past=past, new=n, cu=cu, T=T, req=req, pos=pos, slots=slots, chunks=chunks)


def _gen(seed, what):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 64 + what)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _put(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x), device=DEV).to(dtype)


def _rows(case, seed, T):
    """A projection's output, bf16 [T, heads, 128]: a few channels are larger than the others, tokens differ in size.
    And the views of it."""
    counts = _counts(case)
    g = _gen(seed, 2)
    n = sum(counts.values())
    channel = torch.exp(0.5 * _randn((n, DIM), g))
    channel[:, ::29] *= 5.0
    x = torch.empty((T, n, DIM), dtype=torch.bfloat16, device=DEV)
    for at in range(0, T, 8192):
        m = min(8192, T - at)
        x[at:at + m] = _randn((m, n, DIM), g) * torch.exp(0.3 * _randn((m, 1, 1), g)) * channel
    return x, _views(case, x)


def _views(case, x):
    counts, at, out = _counts(case), 0, {}
    for name in ("q", "k", "v", "q_index", "k_index"):
        if counts[name]:
            out[name] = x[:, at:at + counts[name]]
        at += counts[name]
    return out


def _weights(case, seed):
    """Norm weights of every tensor: fp32 or bf16, one for all heads or one per head."""
    g = _gen(seed, 3)
    out = {}
    for name in ROLES:
        n = _counts(case)[name]
        w = 1.0 + 0.2 * _randn((n, DIM) if case["per_head"] else (DIM,), g)
        if n and case["norm"]:
            out[name] = w if case["wide_weights"] else w.bfloat16()
    return out


def _gradients(case, seed, T):
    """Gradients of the attention's inputs, bf16, contiguous."""
    g = _gen(seed, 4)
    out = {}
    for name in ROLES:
        n = _counts(case)[name]
        if n:
            out[name] = torch.empty((T, n, DIM), dtype=torch.bfloat16, device=DEV)
            for at in range(0, T, 8192):
                m = min(8192, T - at)
                out[name][at:at + m] = 0.01 * _randn((m, n, DIM), g)
    return out


# ---------------------------------------------------------------------------
# state
# ---------------------------------------------------------------------------

def prepare(case, seed):
    s = dict(case=case, own=own)
    if case["op"] == "append":
        b = s["b"] = _batch(case, seed)
        T, pos = b["T"], b["pos"]
    else:
        T, pos = case["tokens"], _documents(case)
    s["T"] = T
    s["pos"] = _put(_spans(pos, case["axes"]))
    s["axis"], s["inv_freq"] = _put(_pair_axes(case), torch.int64), _put(_inv_freq(case), torch.float64)
    s["rows"], s["x"] = _rows(case, seed, T)
    s["w"] = _weights(case, seed)
    names = s["names"] = [n for n in ROLES if n in s["x"]]
    if case["op"] == "bwd":
        s["dy"] = _gradients(case, seed, T)
        s["dx"] = _views(case, torch.zeros_like(s["rows"]))
        s["dw"] = {n: torch.zeros_like(w) for n, w in s["w"].items()}
    else:
        s["y"] = {n: torch.zeros((T, s["x"][n].shape[1], DIM), dtype=torch.bfloat16, device=DEV) for n in names
                  if case["op"] == "fwd" or n in ("q", "q_index")}
    if own:
        from block_sparse_top_attn_gb300 import binding as B
        s["B"] = B
        s["status"] = torch.zeros(4, dtype=torch.int32, device=DEV)
        pairs = B.rope_pairs(_inv_freq(case), _pair_axes(case), device=DEV)
        tensors = {n: B.RopeTensor(v.shape[1], norm=case["norm"] and n != "v", rotate=n != "v", weight=s["w"].get(n),
                                   x_strides=v.stride()[:2]) for n, v in s["x"].items()
                   if n != "v" or case["op"] == "append"}
        s["p"] = B.make_rope_problem(T, pairs, adjacent=case["adjacent"], eps=EPS, **tensors)
        if case["op"] == "bwd":
            s["ws"] = torch.empty(B.msa_norm_rope_bwd_bytes(s["p"]), dtype=torch.uint8, device=DEV)
    if case["op"] == "append":
        H, P, B_ = case["heads"], b["P"], b["B"]
        s["cu"], s["chunks"], s["slots"] = _put(b["cu"]), _put(b["chunks"]), _put(b["slots"], torch.int64)
        if case["index"]:
            # index keys (normed and rotated) of the blocks that the cached tokens left incomplete
            s["tail"] = _randn((b["R"], 2, B_, H, DIM), _gen(seed, 5)).bfloat16()
            s["pool"] = torch.zeros((P, H, DIM), dtype=torch.bfloat16, device=DEV)
        if own:
            s["c"] = B.make_cache_problem(num_requests=b["R"], num_pages=P, max_blocks=b["M"], num_q_heads=H * GROUP,
                                          topk=16, block_size=B_, token_cap=T, chunk_cap=len(b["chunks"]), device=DEV)
            s["cache"] = B.new_cache(s["c"], device=DEV)
        else:
            s["codes"] = torch.zeros((P * B_, H, 2, DIM), dtype=torch.uint8, device=DEV)
            s["scales"] = torch.zeros((P * B_, H, 2, DIM // SCALE_GROUP), dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return {"fwd": _run_fwd, "bwd": _run_bwd, "append": _run_append}[s["case"]["op"]](s)


def _of(d):
    """The entries of q, k, q_index and k_index, None where there is none."""
    return [d.get(n) for n in ROLES]


def _cos_sin(s):
    """fp64 cosines and sines [T, 1, rotary / 2]."""
    angle = s["pos"][:, s["axis"]].double() * s["inv_freq"]
    return torch.cos(angle)[:, None], torch.sin(angle)[:, None]


def _rotate(case, x, cos, sin):
    R = case["rotary"]
    if case["adjacent"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., R:]], -1)


def _forward(s, name, cos, sin):
    """One tensor, normed and rotated, in the type of cos and sin."""
    x = s["x"][name].to(cos.dtype)
    if name in s["w"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["w"][name].to(cos.dtype)
    return _rotate(s["case"], x, cos, sin)


def _run_fwd(s):
    if own:
        s["B"].msa_norm_rope(s["p"], _of(s["x"]), s["pos"], _of(s["y"]), s["status"])
        return [s["y"][n] for n in s["names"]]
    cos, sin = (t.float() for t in _cos_sin(s))
    return [_forward(s, n, cos, sin).bfloat16() for n in s["names"]]


def _backward(s, name, cos, sin):
    g = _rotate(s["case"], s["dy"][name].float(), cos, -sin)
    if name not in s["w"]:
        return g.bfloat16(), None
    x, w = s["x"][name].float(), s["w"][name]
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    x = x * r
    dw = torch.sum(g * x, 0 if s["case"]["per_head"] else (0, 1), dtype=torch.float64).to(w.dtype)
    g = g * w.float()
    return (r * (g - x * (g * x).mean(-1, keepdim=True))).bfloat16(), dw


def _run_bwd(s):
    if own:
        s["B"].msa_norm_rope_bwd(s["p"], _of(s["dy"]), _of(s["x"]), s["pos"], _of(s["dx"]), _of(s["dw"]), s["status"],
                                 s["ws"])
        return [s["dx"][n] for n in s["names"]] + [s["dw"][n] for n in s["names"] if n in s["dw"]]
    cos, sin = (t.float() for t in _cos_sin(s))
    both = [_backward(s, n, cos, sin) for n in s["names"]]
    return [dx for dx, _ in both] + [dw for _, dw in both if dw is not None]


def _round(x):
    """Codes (0..15, the sign on top) and scales of rows in groups of 16: the scale is max / 6 rounded to e4m3, a
    code the nearest multiple of it among e2m1's values, ties to the even code."""
    g = x.view(*x.shape[:-1], DIM // SCALE_GROUP, SCALE_GROUP)
    t = g.abs().amax(-1) / 6.0
    _, e = torch.frexp(t)
    step = torch.exp2((e - 1).clamp(min=-6).to(x.dtype) - 3.0)
    scale = (torch.round(t / step) * step).clamp(max=448.0)
    a, d = g.abs(), scale[..., None]
    code = ((a > 0.25 * d).byte() + (a >= 0.75 * d).byte() + (a > 1.25 * d).byte() + (a >= 1.75 * d).byte()
            + (a > 2.5 * d).byte() + (a >= 3.5 * d).byte() + (a > 5.0 * d).byte())
    code = torch.where(d > 0, code + 8 * (g < 0).byte(), 0)
    return code.view(x.shape).byte(), scale.float()


def _values(codes, scales):
    """bf16 values of codes [..., 128] and scales [..., 8]."""
    lut = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=DEV)
    x = lut[codes.int()]
    return (x.view(*x.shape[:-1], -1, SCALE_GROUP) * scales[..., None]).view(x.shape).bfloat16()


def _run_append(s):
    index = s["case"]["index"]
    if own:
        B, x, y = s["B"], s["x"], s["y"]
        B.msa_cache_append_rope(s["c"], s["p"], x["q"], x["k"], x["v"], x.get("q_index"), x.get("k_index"), s["pos"],
                                s["slots"], s["cu"], s["chunks"], y["q"], y.get("q_index"), s["cache"], s.get("tail"),
                                s.get("pool"), s["status"])
        k = torch.empty((s["T"], s["case"]["heads"], DIM), dtype=torch.bfloat16, device=DEV)
        v = torch.empty_like(k)
        B.msa_cache_read(s["c"], s["slots"], s["cache"], k, v, s["status"])
        return [y["q"], k, v] + ([y["q_index"], s["tail"], s["pool"]] if index else [])
    b = s["b"]
    cos, sin = _cos_sin(s)
    q = _forward(s, "q", cos.float(), sin.float()).bfloat16()
    # K in 64 bits: its codes turn on which side of a border a value lies
    kv = _forward(s, "k", cos, sin), s["x"]["v"].float().contiguous()
    codes, scales = zip(*(_round(x) for x in kv))
    s["codes"][s["slots"]], s["scales"][s["slots"]] = torch.stack(codes, 2), torch.stack(scales, 2)
    kv = _values(s["codes"][s["slots"]], s["scales"][s["slots"]])
    out = [q, kv[:, :, 0].contiguous(), kv[:, :, 1].contiguous()]
    if not index:
        return out
    qi, ki = (_forward(s, n, cos.float(), sin.float()).bfloat16() for n in ("q_index", "k_index"))
    # every new token's place in its block
    B, T, cu, chunks = b["B"], b["T"], s["cu"].long(), s["chunks"].long()
    rows = torch.arange(T, device=DEV)
    req = torch.searchsorted(cu[1:].contiguous(), rows, right=True)
    of_chunk = torch.searchsorted(chunks[:, 1].contiguous(), rows, right=True) - 1
    pos = chunks[of_chunk, 3] + rows - chunks[of_chunk, 1]
    end = pos + cu[req + 1] - rows  # behind the request's last token
    blk = pos // B
    # means of the blocks that are complete now: the tokens of the call, and of earlier calls from the tail
    done = rows[pos % B == B - 1]
    member = done[:, None] - (B - 1) + torch.arange(B, device=DEV)
    now = member >= cu[req[done], None]
    old = s["tail"][req[done], blk[done] % 2]
    x = torch.where(now[:, :, None, None], ki[member.clamp(min=0)], old)
    s["pool"][s["slots"][done] // B] = (x.float().sum(1) / B).bfloat16()
    keep = rows[(blk + 1) * B > end]
    s["tail"][req[keep], blk[keep] % 2, pos[keep] % B] = ki[keep]
    return out + [qi, s["tail"], s["pool"]]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    n = _counts(case)
    weights = (2 + 2 * case["wide_weights"]) * DIM * (sum(n[r] for r in ROLES) if case["per_head"] else 4) * case["norm"]
    table = 12 * case["rotary"] // 2
    moved = sum(n[r] for r in ROLES)
    if case["op"] != "append":
        T = case["tokens"]
        # the tensors in and out (and the gradients in), positions, weights (and their gradients)
        bwd = case["op"] == "bwd"
        return dict(bytes=T * (moved * 2 * DIM * (2 + bwd) + 4 * case["axes"]) + weights * (1 + bwd) + table,
                    flops=T * moved * DIM * (20 if bwd else 10))
    b = _batch(case, 0)
    T, B, H = b["T"], b["B"], case["heads"]
    total = b["past"] + b["new"]
    kept = DIM // 2 + DIM // SCALE_GROUP  # bytes of one token's K (or V) of one head in the cache
    # q, k, v and index vectors in; q and index q out; the cache's bytes out and in again, its values out
    rows = 2 * DIM * (moved + n["v"] + n["q"] + n["q_index"]) + H * (2 * 2 * kept + 2 * 2 * DIM)
    tails = 0
    if case["index"]:  # pooled keys of the blocks that become complete, the tail's rows in and out
        tails = int((total // B - b["past"] // B).sum() + (total - np.maximum(b["past"], total // B * B)).sum()
                    + np.where(total // B > b["past"] // B, b["past"] % B, 0).sum())
    return dict(bytes=T * (rows + 8 + 4 * case["axes"]) + 2 * DIM * H * tails + weights + table,
                flops=T * DIM * (10 * moved + 16 * H))


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "append":
        return _exact_append(case, seed)
    pos = _spans(_documents(case), case["axes"])
    turn = _turns(case, pos)
    _, x = _rows(case, seed, case["tokens"])
    w = _weights(case, seed)
    names = [n for n in ROLES if n in x]
    if case["op"] == "fwd":
        return [torch.cat([_head64(case, x[n][:, h], _weight64(w, n, h), turn)[:, None] for h in range(x[n].shape[1])], 1)
                for n in names]
    dy = _gradients(case, seed, case["tokens"])
    dxs, dws = [], []
    for n in names:
        dx = torch.empty(x[n].shape, dtype=torch.float64, device=DEV)
        dw = []
        for h in range(x[n].shape[1]):
            dx[:, h], d = _grad64(case, x[n][:, h], _weight64(w, n, h), dy[n][:, h], turn)
            dw.append(d)
        dxs.append(dx)
        if n in w:
            dws.append(torch.stack(dw) if case["per_head"] else torch.stack(dw).sum(0))
    return dxs + dws


def _turns(case, pos):
    """The rotation of every token and pair as a complex number of length 1."""
    angle = torch.as_tensor(pos[:, _pair_axes(case)].astype(np.float64) * _inv_freq(case), device=DEV)
    return torch.polar(torch.ones_like(angle), angle)


def _weight64(w, name, h):
    if name not in w:
        return None
    return (w[name][h] if w[name].dim() == 2 else w[name]).double()


def _turn64(case, x, turn):
    """Rows [T, 128] with their first dims turned."""
    R = case["rotary"]
    pairs = x[:, :R].unflatten(1, (R // 2, 2)) if case["adjacent"] else x[:, :R].unflatten(1, (2, R // 2)).mT
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    out = x.clone()
    out[:, :R] = z.flatten(1) if case["adjacent"] else z.mT.flatten(1)
    return out


def _head64(case, x, w, turn):
    """One head [T, 128]."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).sum(1, keepdim=True) / DIM + EPS) * w
    return _turn64(case, x, turn)


def _grad64(case, x, w, dy, turn):
    """Gradients of <dy, y> to one head's x and to its weight."""
    x, g = x.double(), _turn64(case, dy.double(), turn.conj())
    if w is None:
        return g, None
    # y = x w / n with n = sqrt(|x|^2 / 128 + eps): d n / d x = x / (128 n)
    n = torch.sqrt((x * x).sum(1, keepdim=True) / DIM + EPS)
    along = (g * w * x).sum(1, keepdim=True)
    return g * w / n - x * along / (DIM * n ** 3), (g * x / n).sum(0)


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
    """fp64 values that 4 bits and a scale keep of fp64 rows [..., 128]."""
    g = x.unflatten(-1, (DIM // SCALE_GROUP, SCALE_GROUP))
    e4 = torch.tensor(_e4m3_values(), dtype=torch.float64, device=x.device)
    scale = e4[_nearest(g.abs().amax(-1) / 6.0, _e4m3_values())][..., None]
    best = torch.zeros_like(g)
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    for i in range(1, 8):
        mid = (levels[i - 1] + levels[i]) / 2 * scale
        above = (g.abs() > mid) if i % 2 else (g.abs() >= mid)
        best = torch.where(above, levels[i] * scale, best)
    return (best * torch.sign(g)).flatten(-2)


def _exact_append(case, seed):
    b = _batch(case, seed)
    B, T, P, H = b["B"], b["T"], b["P"], case["heads"]
    turn = _turns(case, _spans(b["pos"], case["axes"]))
    _, x = _rows(case, seed, T)
    w = _weights(case, seed)
    y = {n: torch.stack([_head64(case, x[n][:, h], _weight64(w, n, h), turn) for h in range(x[n].shape[1])], 1)
         for n in ROLES if n in x}
    out = [y["q"], _rounded64(y["k"]), _rounded64(x["v"].double())]
    if not case["index"]:
        return out
    old = _randn((b["R"], 2, B, H, DIM), _gen(seed, 5)).bfloat16().double()
    tail, pool = old.clone(), torch.zeros((P, H, DIM), dtype=torch.float64, device=DEV)
    page = b["slots"] // B
    for r in range(b["R"]):
        past, n, row = int(b["past"][r]), int(b["new"][r]), int(b["cu"][r])
        for blk in range(past // B, -(-(past + n) // B)):
            lo, hi = max(past, blk * B), min(past + n, (blk + 1) * B)
            fresh = y["k_index"][row + lo - past:row + hi - past]
            if hi == (blk + 1) * B:
                pool[page[row + lo - past]] = (old[r, blk % 2, :lo - blk * B].sum(0) + fresh.sum(0)) / B
            else:
                tail[r, blk % 2, lo - blk * B:hi - blk * B] = fresh
    return out + [y["q_index"], tail, pool]
