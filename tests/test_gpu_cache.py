"""GPU: the serving operators over the 4-bit paged cache (msa_cache_*, through
the C ABI and the Cache class) against the CPU oracle.  Tables, cache bytes,
index means and selections are compared bit for bit; the attention within
bounds derived from its roundings (``_close``)."""
import numpy as np
import pytest

from oracle import cache_oracle as C
from oracle import msa_oracle as O
from tests._util import from_bf16_tensor, to_bf16_tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from block_sparse_top_attn_gb300 import binding
    return binding


def _bf16(rng, shape, scale=1.0):
    return O.f64_to_bf16(rng.standard_normal(shape) * scale)


def _dev(x, dtype=None):
    import torch
    return torch.as_tensor(np.ascontiguousarray(x), device="cuda").to(dtype or torch.int32)


class Setup:
    """A batch with cached and new tokens: host tables from the oracle, device tensors, K and V as the cache holds
    them, and the calls."""

    def __init__(self, B, past, new, H=1, block=64, topk=4, seed=0, token_pad=0, chunk_pad=0, extra_pages=3,
                 k_exp=0, v_exp=0, scale=128 ** -0.5, garbage=None, k_scale=1.0, v_scale=1.0, page_base=0, kv=True):
        import torch
        rng = self.rng = np.random.default_rng(seed)
        self.B, self.H, self.block, self.K, self.scale = B, H, block, topk, scale
        self.past, self.new = np.array(past), np.array(new)
        R = len(past)
        total = self.past + np.maximum(self.new, 0)
        held, need = -(-self.past // block), -(-total // block)
        M, P = int(max(need.max(), 1)) + 2, int(need.sum()) + extra_pages + page_base
        order = page_base + rng.permutation(P - page_base)
        table = np.zeros((R, M), np.int64)
        at = 0
        for r in range(R):
            table[r, :held[r]] = order[at:at + held[r]]
            at += held[r]
        ring = np.zeros(P, np.int64)
        head, free = int(rng.integers(0, P)), order[at:]
        ring[(head + np.arange(len(free))) % P] = free
        self.start = dict(table=table, ring=ring, head=head, count=len(free))
        self.want = C.step(self.new, self.past, head, len(free), ring, table, block)
        self.T, self.NC = len(self.want["slot_map"]) + token_pad, len(self.want["chunks"]) + chunk_pad
        self.c = B.make_cache_problem(num_requests=R, num_pages=P, max_blocks=M, num_q_heads=16 * H, topk=topk,
                                      token_cap=max(self.T, 1), chunk_cap=max(self.NC, 1), softmax_scale=scale,
                                      block_size=block, k_exp=k_exp, v_exp=v_exp)
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")
        # K and V of every token of every request
        n = int(total.sum()) if kv else 0
        self.k_bits = _bf16(rng, (n, H, 128), k_scale)
        self.v_bits = _bf16(rng, (n, H, 128), v_scale)
        self.first = np.concatenate([[0], np.cumsum(total)])
        self.kv_exp = (k_exp, v_exp)
        self.cache = None
        self.garbage = garbage
        self.full = self.want["block_table"]

    def code(self):
        import torch
        torch.cuda.synchronize()
        return int(self.status[0].item())

    def fill(self):
        """The cache with every token in it, by msa_cache_append; bytes that hold no token keep `garbage`."""
        import torch
        self.cache = self.B.new_cache(self.c)
        if self.garbage is not None:
            self.cache.fill_(self.garbage)
        slots = []
        for r in range(len(self.past)):
            p = np.arange(self.first[r + 1] - self.first[r])
            slots.append(self.full[r, p // self.block] * self.block + p % self.block)
        slots = np.concatenate(slots)
        c = self.B.make_cache_problem(num_requests=1, num_pages=self.c.num_pages, max_blocks=1,
                                      num_q_heads=16 * self.H, topk=1, token_cap=len(slots), chunk_cap=1,
                                      block_size=self.block, k_exp=self.kv_exp[0], v_exp=self.kv_exp[1])
        self.B.msa_cache_append(c, to_bf16_tensor(self.k_bits, "cuda"), to_bf16_tensor(self.v_bits, "cuda"), None,
                                _dev(slots, torch.int64), None, None, self.cache, None, None, self.status)
        return self.cache

    def values(self):
        kv = C.round_rows(self.k_bits, self.kv_exp[0])[2]
        vv = C.round_rows(self.v_bits, self.kv_exp[1])[2]
        cut = lambda x: [x[self.first[r]:self.first[r + 1]] for r in range(len(self.past))]
        return cut(kv), cut(vv)

    def chunk_table(self):
        x = np.full((self.c.chunk_cap, 4), -1)
        x[:len(self.want["chunks"])] = self.want["chunks"]
        return _dev(x)

    def selection(self, policy="random"):
        sel = np.full((self.H, self.c.chunk_cap, self.K), -1)
        for g, (r, row, n, first) in enumerate(self.want["chunks"]):
            diag = int(first) // self.block
            for h in range(self.H):
                pick = [diag] + list(self.rng.choice(diag, min(diag, self.K - 1), replace=False))
                if policy == "holes":       # -1 anywhere, blocks in any order, often without the chunk's own block
                    pick = [b for b in pick if self.rng.random() < 0.6]
                    pick = (pick + [-1] * self.K)[:self.K]
                    self.rng.shuffle(pick)
                sel[h, g, :len(pick)] = pick
        return sel

    def forward(self, q_bits, sel, chunks=None, table=None, fill=7.0):
        import torch
        T = self.c.token_cap
        o = torch.full((T, 16 * self.H, 128), fill, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T, 16 * self.H), fill, dtype=torch.float32, device="cuda")
        self.B.msa_cache_fwd(self.c, to_bf16_tensor(q_bits, "cuda"), self.cache,
                             _dev(self.full) if table is None else table,
                             self.chunk_table() if chunks is None else chunks, _dev(sel), o, lse, self.status)
        return o, lse

    def queries(self, scale=1.0):
        return _bf16(self.rng, (self.c.token_cap, 16 * self.H, 128), scale)


def _close(o, lse, want):
    """o is off by half a step of bf16, 2^-8 |o|; by the rounding of p to fp16, 2^-11 of the p-weighted mean of |v|,
    and for a p below fp16's normal range at most 2^-25 where the largest p is 2^7 or more, so 2^-32 |v| for each of
    up to 4096 keys (which counts where the keys of all the weight have v = 0); and by the error ds of a score, twice
    (numerator and denominator).  ds: fp32 sums of 128 exact products in 8 MMAs, each of which may cut its sum to 24 bits
    instead of rounding it (2^-23 of the running magnitude), and two fp32 products: 2^-19 of sum |q k| scale
    covers them; exp2's 2^-22 is added.  lse: ds, and fp32 operations on it and on log2 of the sum (2^-21)."""
    wo, wl, absv, mag, vmax = want
    live = ~np.isnan(wl)
    got, gl = O.bf16_to_f64(from_bf16_tensor(o)), lse.double().cpu().numpy()
    ds = 2.0 ** -19 * mag + 2.0 ** -20
    bound = 2.0 ** -8 * np.abs(wo) + (2.0 ** -11 + 2 * ds)[..., None] * absv + 2.0 ** -32 * 4096 * vmax
    err = np.abs(got - wo)
    assert np.all(err[live] <= bound[live]), float((err[live] / bound[live]).max())
    inf = np.isneginf(wl)
    assert np.array_equal(np.isneginf(gl) & live, inf & live)
    el = np.abs(gl - np.where(inf, 0, wl))
    assert np.all(el[live & ~inf] <= (ds + 2.0 ** -21 * (1 + np.abs(np.where(inf, 0, wl))))[live & ~inf])
    assert np.all(got[~live] == 7.0) and np.all(gl[~live] == 7.0)     # rows that no chunk covers


# ---------------------------------------------------------------------------
# step
# ---------------------------------------------------------------------------

def _run_step(B, s, in_place=False):
    import torch
    R, M = s.start["table"].shape
    i32 = lambda *shape: torch.full(shape, -7, dtype=torch.int32, device="cuda")
    d = dict(new=_dev(s.new), lens=_dev(s.past), ring_at=_dev([s.start["head"], s.start["count"]]),
             ring=_dev(s.start["ring"]), table=_dev(s.start["table"]), cu=i32(R + 1),
             slots=torch.full((s.c.token_cap,), -7, dtype=torch.int64, device="cuda"), pos=i32(s.c.token_cap),
             chunks=i32(s.c.chunk_cap, 4))
    d["lens_out"], d["ring_out"] = (d["lens"], d["ring_at"]) if in_place else (i32(R), i32(2))
    B.msa_cache_step(s.c, d["new"], d["lens"], d["ring_at"], d["ring"], d["table"], d["lens_out"], d["ring_out"],
                     d["cu"], d["slots"], d["pos"], d["chunks"], s.status)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in d.items()}


BATCHES = {
    "one": ([0], [1]), "one_long": ([130], [1]), "idle": ([5, 0, 64], [0, 0, 0]),
    "decode": ([0, 63, 64, 65, 127, 128, 7, 8], [1] * 8),
    "mixed": ([0, 63, 100, 64, 1000, 5, 8, 300], [200, 1, -1, -1, 3, 0, 130, 9]),
    "finish": ([100, 1, 64], [-1, -1, -1]),
    "prefill": ([0, 4096, 17], [3000, 5000, 1]),
}


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", list(BATCHES) + ["wide"])
def test_step_bit_exact(B, name, block, in_place):
    if name == "wide":
        rng = np.random.default_rng(5)
        past, new = rng.integers(0, 500, 2500), rng.integers(-1, 12, 2500)
    else:
        past, new = BATCHES[name]
    s = Setup(B, past, new, block=block, token_pad=5, chunk_pad=3, kv=False)
    got = _run_step(B, s, in_place)
    assert s.code() == 0
    w, n, nc = s.want, len(s.want["slot_map"]), len(s.want["chunks"])
    assert np.array_equal(got["cu"], w["cu_tokens"])
    assert np.array_equal(got["slots"][:n], w["slot_map"]) and np.all(got["slots"][n:] == -1)
    assert np.array_equal(got["pos"][:n], w["positions"]) and np.all(got["pos"][n:] == -1)
    assert np.array_equal(got["chunks"][:nc], w["chunks"]) and np.all(got["chunks"][nc:] == -1)
    assert np.array_equal(got["table"], w["block_table"])
    assert np.array_equal(got["lens_out"], w["seq_lens"])
    assert got["ring_out"].tolist() == [w["head"], w["count"]]
    assert np.array_equal(got["ring"], w["free_ring"])


@pytest.mark.parametrize("change, code", [
    (dict(token_cap=-1), 4), (dict(chunk_cap=-1), 4), (dict(count=0), 4), (dict(new=(1, 10 ** 6)), 4),
    (dict(new=(0, -2)), 10), (dict(past=(0, -1)), 10), (dict(past=(1, 10 ** 9)), 10), (dict(head=10 ** 6), 10),
    (dict(head=-1), 10), (dict(count=10 ** 6), 10), (dict(status=5), 5)])
def test_step_refuses_and_writes_nothing(B, change, code):
    """Capacities one short, no free page, lengths and ring out of range, an earlier error."""
    import torch
    s = Setup(B, [64, 60, 10], [5, 20, -1])
    s.c.token_cap += change.get("token_cap", 0)
    s.c.chunk_cap += change.get("chunk_cap", 0)
    for key in ("count", "head"):
        s.start[key] = change.get(key, s.start[key])
    for key in ("new", "past"):
        if key in change:
            getattr(s, key)[change[key][0]] = change[key][1]
    s.status[0] = change.get("status", 0)
    got = _run_step(B, s)
    assert s.code() == code
    for key in ("cu", "slots", "pos", "chunks", "lens_out", "ring_out"):
        assert np.all(got[key] == -7), key
    assert np.array_equal(got["table"], s.start["table"]) and np.array_equal(got["ring"], s.start["ring"])


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------

def _special_rows(rng, bits):
    """Zeros, infinities and NaN, saturation, tiny groups, ties of codes and of scales."""
    x = O.bf16_to_f64(bits).copy()
    x[0] = 0
    x[1] *= 2.0 ** -10
    x[2] *= 2.0 ** 12
    x[3, :, :16] = np.array([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5] * 2) * np.array([1, -1] * 8)
    x[3, :, 16:32] = 3 * x[3, :, :16]
    x[4, :, ::16] = 6 * 1.0625 * np.array([1, 2, 4, 8, 0.5, 0.25, 16, 32])
    x[5] *= 2.0 ** -130
    out = O.f64_to_bf16(x)
    out[6, :, 5], out[6, :, 77], out[6, :, 127] = 0x7F80, 0xFF80, 0x7FC0
    return out


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("exp", [(0, 0), (-6, 3), (32, -32)])
@pytest.mark.parametrize("H", [1, 3])
def test_append_bytes_and_read(B, block, exp, H):
    """Every byte of the cache, those that hold no token among them; rows of slot -1 are left out; read gives the
    exact values in any order and leaves rows of slot -1 as they were."""
    import torch
    rng = np.random.default_rng(7)
    P, T = 6, 77
    slots = rng.permutation(P * block)[:T].astype(np.int64)
    slots[[10, 40]] = -1
    k, v = (_special_rows(rng, _bf16(rng, (T, H, 128), 2.0 ** e)) for e in exp)
    c = B.make_cache_problem(num_requests=1, num_pages=P, max_blocks=P, num_q_heads=16 * H, topk=1, token_cap=T,
                             chunk_cap=1, block_size=block, k_exp=exp[0], v_exp=exp[1])
    cache = B.new_cache(c)
    cache.fill_(0xA5)
    want = cache.cpu().numpy()
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    ds = _dev(slots, torch.int64)
    B.msa_cache_append(c, to_bf16_tensor(k, "cuda"), to_bf16_tensor(v, "cuda"), None, ds, None, None, cache, None,
                       None, st)
    C.append(want, k, v, slots, block, *exp)
    got = cache.cpu().numpy()
    # the codes of a group whose scale is NaN mean nothing: compare those groups by their scale alone
    kc, ks, kv = C.round_rows(k, exp[0])
    vc, vs, vv = C.round_rows(v, exp[1])
    for t in np.flatnonzero((ks == 0x7F).any((1, 2)) | (vs == 0x7F).any((1, 2))):
        page, off = divmod(int(slots[t]), block)
        for x in (got, want):
            b, i = x[page, :, off // 64], off % 64
            b[:, i * 64:i * 64 + 64] = 0
            b[:, 4608 + ((i * 64 + np.arange(64)) ^ ((i & 12) << 3))] = 0
    assert np.array_equal(got, want)
    order = rng.permutation(T)
    rk = torch.full((T, H, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    rv = torch.full_like(rk, 9.0)
    B.msa_cache_read(c, ds[torch.as_tensor(order, device="cuda")].contiguous(), cache, rk, rv, st)
    torch.cuda.synchronize()
    assert int(st[0].item()) == 0
    for got_x, vals in ((rk, kv), (rv, vv)):
        x = vals[order].copy()
        x[slots[order] < 0] = 9.0
        bits, nan = from_bf16_tensor(got_x), np.isnan(x)
        assert np.array_equal(np.isnan(O.bf16_to_f64(bits)), nan)
        assert np.array_equal(O.bf16_to_f64(bits)[~nan], O.bf16_to_f64(O.f64_to_bf16(x[~nan])))


def test_slots_out_of_range_are_left_out(B):
    import torch
    rng = np.random.default_rng(8)
    c = B.make_cache_problem(num_requests=1, num_pages=2, max_blocks=2, num_q_heads=16, topk=1, token_cap=5,
                             chunk_cap=1)
    k = to_bf16_tensor(_bf16(rng, (5, 1, 128)), "cuda")
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    cache = B.new_cache(c)
    B.msa_cache_append(c, k, k, None, _dev([0, 128, -2, 1 << 40, 127], torch.int64), None, None, cache, None, None,
                       st)
    torch.cuda.synchronize()
    assert int(st[0].item()) == B.MSA_ERR_INVALID_CACHE
    st.zero_()
    out = torch.full((5, 1, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    B.msa_cache_read(c, _dev([127, 0, 128, -(1 << 40), 0], torch.int64), cache, out, out.clone(), st)
    torch.cuda.synchronize()
    assert int(st[0].item()) == B.MSA_ERR_INVALID_CACHE
    x = out.float().cpu().numpy()
    assert np.all(x[2:4] == 9.0) and np.array_equal(x[1], x[4]) and not np.any(x[:2] == 9.0)
    # an earlier error: nothing is written
    before = cache.clone()
    B.msa_cache_append(c, k + 1, k, None, _dev([0, 1, 2, 3, 4], torch.int64), None, None, cache, None, None, st)
    B.msa_cache_read(c, _dev([0, 1, 2, 3, 4], torch.int64), cache, out, out.clone(), st)
    torch.cuda.synchronize()
    assert torch.equal(cache, before) and np.array_equal(out.float().cpu().numpy(), x)


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("past, new", [([0], [1]), ([63], [1]), ([127], [1]), ([60], [10]), ([60], [150]),
                                       ([60], [250]), ([0, 5, 100, 31], [200, 0, 300, 33]), ([64, 128], [64, 128])])
def test_index_means(B, block, past, new):
    """Means of the blocks that a call completes and the tail's rows, bit for bit; nothing else changes."""
    import torch
    s = Setup(B, past, new, H=2, block=block, token_pad=2, chunk_pad=2)
    R, T = len(past), s.c.token_cap
    ki = _bf16(s.rng, (T, 2, 128))
    tail, pool = _bf16(s.rng, (R, 2, block, 2, 128)), _bf16(s.rng, (s.c.num_pages, 2, 128))
    k = to_bf16_tensor(_bf16(s.rng, (T, 2, 128)), "cuda")
    slots = np.full(T, -1)
    slots[:len(s.want["slot_map"])] = s.want["slot_map"]
    dt, dp = to_bf16_tensor(tail, "cuda"), to_bf16_tensor(pool, "cuda")
    B.msa_cache_append(s.c, k, k, to_bf16_tensor(ki, "cuda"), _dev(slots, torch.int64), _dev(s.want["cu_tokens"]),
                       s.chunk_table(), B.new_cache(s.c), dt, dp, s.status)
    assert s.code() == 0
    C.index_update(ki, s.want["cu_tokens"], past, s.full, tail, pool, block)
    assert np.array_equal(from_bf16_tensor(dt), tail)
    assert np.array_equal(from_bf16_tensor(dp), pool)


@pytest.mark.parametrize("col, value", [(0, 1), (1, -1), (1, 60), (2, 0), (2, 9), (3, -1), (3, 3)])
def test_append_and_select_report_bad_chunk_rows(B, col, value):
    """A chunk row that does not fit the batch is reported, not followed."""
    import torch
    s = Setup(B, [3], [5])
    ki = to_bf16_tensor(_bf16(s.rng, (5, 1, 128)), "cuda")
    chunks = s.chunk_table()
    chunks[0, col] = value
    tail = torch.zeros((1, 2, 64, 1, 128), dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros((s.c.num_pages, 1, 128), dtype=torch.bfloat16, device="cuda")
    B.msa_cache_append(s.c, ki, ki, ki, _dev(s.want["slot_map"], torch.int64), _dev(s.want["cu_tokens"]), chunks,
                       B.new_cache(s.c), tail, pool, s.status)
    if (col, value) != (3, 3):
        assert s.code() == B.MSA_ERR_INVALID_CACHE
    if (col, value) in ((0, 1), (1, -1), (1, 60), (2, 0), (2, 9), (3, -1)):
        s.status.zero_()
        sel = torch.full((1, s.c.chunk_cap, s.K), -5, dtype=torch.int32, device="cuda")
        B.msa_cache_select(s.c, ki, pool, _dev(s.full), chunks, sel, s.status)
        assert s.code() == B.MSA_ERR_INVALID_CACHE and bool((sel == -5).all())


# ---------------------------------------------------------------------------
# select
# ---------------------------------------------------------------------------

def _select(B, s, qi, pool):
    import torch
    sel = torch.full((s.H, s.c.chunk_cap, s.K), -5, dtype=torch.int32, device="cuda")
    B.msa_cache_select(s.c, to_bf16_tensor(qi, "cuda"), to_bf16_tensor(pool, "cuda"), _dev(s.full), s.chunk_table(),
                       sel, s.status)
    assert s.code() == 0
    return sel.cpu().numpy()


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("topk", [1, 2, 7, 32])
@pytest.mark.parametrize("past, new, H, block", [
    ([0], [1], 1, 64), ([63, 64, 65, 0], [1, 1, 1, 1], 2, 64), ([5000, 33, 128 * 40], [1, 7, 20], 3, 128),
    ([3000, 0], [300, 100], 2, 64), ([64 * 33], [8], 1, 64), ([20000], [2], 1, 64)])
def test_selection_bit_exact(B, past, new, H, block, topk, ties):
    s = Setup(B, past, new, H=H, block=block, topk=topk, token_pad=1, chunk_pad=2)
    qi, pool = _bf16(s.rng, (s.c.token_cap, H, 128)), _bf16(s.rng, (s.c.num_pages, H, 128), 0.125)
    if ties:   # few distinct vectors, zeros of either sign
        qi = O.f64_to_bf16(s.rng.integers(-1, 2, qi.shape) * 1.0)
        rows = O.f64_to_bf16(s.rng.integers(-1, 2, (3, H, 128)) * 0.5)
        rows[0] = 0x8000
        pool = rows[s.rng.integers(0, 3, len(pool))]
    got = _select(B, s, qi, pool)
    want = C.select(qi, pool, s.full, s.want["chunks"], block, topk)
    assert np.array_equal(got[:, :want.shape[1]], want)
    assert np.all(got[:, want.shape[1]:] == -5)


def test_selection_at_the_longest_table(B):
    """49152 blocks in the table, a request that fills most of them: exact against the oracle."""
    s = Setup(B, [64 * 49000 + 5], [1], topk=32, extra_pages=0, kv=False)
    s.c.max_blocks = 49152
    full = np.zeros((1, 49152), np.int64)
    full[:, :s.full.shape[1]] = s.full
    s.full = full
    qi, pool = _bf16(s.rng, (1, 1, 128)), _bf16(s.rng, (s.c.num_pages, 1, 128))
    assert np.array_equal(_select(B, s, qi, pool), C.select(qi, pool, s.full, s.want["chunks"], 64, 32))


def test_selection_with_scores_that_are_not_numbers(B):
    """NaN and infinities in the index vectors: some order, but a valid selection."""
    s = Setup(B, [4000], [3], topk=16)
    qi, pool = _bf16(s.rng, (3, 1, 128)), _bf16(s.rng, (s.c.num_pages, 1, 128))
    pool[::3, :, 5], pool[1::7, :, 9] = 0x7FC0, 0xFF80
    got = _select(B, s, qi, pool)
    for g, (r, row, n, first) in enumerate(s.want["chunks"]):
        row = got[0, g].tolist()
        assert row[0] == first // 64 and len(set(row)) == 16 and all(0 <= b < first // 64 for b in row[1:])


def test_select_reports_bad_pages(B):
    import torch
    s = Setup(B, [400], [1])
    pool = torch.zeros((s.c.num_pages, 1, 128), dtype=torch.bfloat16, device="cuda")
    for bad in (-1, s.c.num_pages, 1 << 30):
        s.status.zero_()
        table = _dev(s.full)
        table[0, 2] = bad
        sel = torch.zeros((1, s.c.chunk_cap, s.K), dtype=torch.int32, device="cuda")
        B.msa_cache_select(s.c, pool[:1].contiguous(), pool, table, s.chunk_table(), sel, s.status)
        assert s.code() == B.MSA_ERR_INVALID_CACHE


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _attend_case(B, policy="random", q_scale=1.0, **kw):
    s = Setup(B, **kw)
    s.fill()
    sel, q = s.selection(policy), s.queries(q_scale)
    o, lse = s.forward(q, sel)
    assert s.code() == 0
    _close(o, lse, C.attend(q, *s.values(), s.want["chunks"], sel, s.block, s.scale))
    return s, q, sel


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("topk", [1, 4, 32])
@pytest.mark.parametrize("past, new, H", [
    ([0], [1], 1), ([15], [1], 2), ([63, 64, 65, 127, 128, 129], [1] * 6, 2), ([2500], [1], 1),
    ([700, 0, 1, 90], [3, 9, 2, 40], 3), ([61], [6], 1), ([5, 3000], [0, 130], 2), ([0], [333], 1)])
def test_attention(B, past, new, H, block, topk):
    """Single tokens and pieces, requests of length 0 and 1, idle ones, positions around page and tile borders;
    bytes behind the last token are 0xFF: NaN scales."""
    _attend_case(B, past=past, new=new, H=H, block=block, topk=topk, garbage=0xFF, token_pad=3, chunk_pad=2)


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("past, new", [([900, 64, 300], [1, 1, 1]), ([640, 10], [20, 5])])
def test_attention_over_any_selection(B, past, new, block):
    """Empty slots anywhere, blocks in any order, chunks without their own block, chunks that select nothing."""
    s, _, sel = _attend_case(B, policy="holes", past=past, new=new, H=4, block=block, topk=3, garbage=0xFF, seed=4)
    assert any((sel[h, g] < 0).all() for h in range(4) for g in range(len(s.want["chunks"])))


@pytest.mark.parametrize("R", [1, 2, 5, 20, 80, 200])
def test_attention_over_batch_sizes(B, R):
    """Every way the tiles are split over CTAs, decode and a few tokens at a time."""
    rng = np.random.default_rng(R)
    past = rng.integers(0, 1500, R)
    _attend_case(B, past=past, new=[1] * R, H=2, topk=16)
    _attend_case(B, past=past[:40], new=rng.integers(1, 9, min(R, 40)), H=1, topk=16, block=128)


@pytest.mark.parametrize("kw", [dict(k_exp=-8, k_scale=2.0 ** -8), dict(v_exp=20, v_scale=2.0 ** 20),
                                dict(k_exp=32, k_scale=2.0 ** 30, scale=2.0 ** -34), dict(q_scale=2.0 ** 40, scale=2.0 ** -44),
                                dict(q_scale=2.0 ** -100), dict(q_scale=30.0), dict(q_scale=0.0, scale=2.0 ** -60), dict(v_exp=-32, v_scale=2.0 ** -34)])
def test_attention_over_magnitudes(B, kw):
    """Cache exponents, queries far from 1, and scores in the hundreds (one key takes all the weight)."""
    _attend_case(B, past=[300, 70], new=[1, 12], H=1, topk=6, **kw)


@pytest.mark.parametrize("kw", [dict(k_exp=-8, k_scale=2.0 ** -8), dict(v_exp=20, v_scale=2.0 ** 20),
                                dict(k_exp=32, k_scale=2.0 ** 30, scale=2.0 ** -34),
                                dict(q_scale=2.0 ** 40, scale=2.0 ** -44), dict(q_scale=2.0 ** -100),
                                dict(q_scale=30.0), dict(q_scale=0.0, scale=2.0 ** -60)])
def test_chunk_attention_over_magnitudes(B, kw):
    """The same for chunks of several tokens with many heads (the 128-row kernel), and twice with the same bits."""
    import torch
    s, q, sel = _attend_case(B, past=[300, 70, 0], new=[12, 9, 3], H=8, topk=6, garbage=0xFF, **kw)
    a, b = s.forward(q, sel), s.forward(q, sel)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attention_of_non_finite_values(B):
    """A NaN among the values of an attended key reaches the dims of its group, in the rows that attend it; a NaN key
    makes its rows NaN; rows that may not attend them stay exact."""
    import torch
    s = Setup(B, past=[100], new=[4], topk=4, garbage=0xFF)
    s.v_bits[102, 0, 37] = 0x7F80           # position 102: dims 32 .. 47
    s.k_bits[103, 0, 5] = 0x7FC0            # position 103
    s.fill()
    sel, q = s.selection(), s.queries()
    sel[0, :, :2] = [1, 0]
    o, lse = s.forward(q, sel)
    assert s.code() == 0
    x = o.float().cpu().numpy()
    assert np.isfinite(x[:2]).all() and np.isfinite(lse[:3].cpu().numpy()).all()
    assert np.isnan(x[2][:, 32:48]).all() and np.isfinite(np.delete(x[2], range(32, 48), 1)).all()
    assert np.isnan(x[3]).all() and np.isnan(lse[3].cpu().numpy()).all()
    q[0, 3, 7], q[1, 4, 9] = 0x7FC0, 0xFF80  # a query that is not finite spoils its own row only
    o, lse = s.forward(q, sel)
    x = o.float().cpu().numpy()
    assert np.isnan(x[0, 3]).all() and np.isnan(x[1, 4]).all()
    assert np.isfinite(np.delete(x[0], 3, 0)).all() and np.isfinite(np.delete(x[1], 4, 0)).all()


@pytest.mark.parametrize("H, past, new", [(1, [100, 61], [4, 30]), (8, [100, 61], [4, 30]),
                                          (16, [0, 56, 130], [60, 8, 3])])
@pytest.mark.parametrize("block", [64, 128])
def test_attention_of_nan_values_inside_chunks(B, H, past, new, block):
    """Values that are NaN at positions of the new tokens themselves and before them, every block selected: the rows at
    and behind such a position have NaN in the dims of its group, all else is as without it."""
    import torch
    s = Setup(B, past=past, new=new, H=H, block=block, topk=4, garbage=0xFF)
    clean = s.v_bits.copy()
    marks = [(r, past[r] + t, 16 * g) for r, t, g in ((0, 2, 1), (0, 3, 7), (1, 0, 0), (1, 5, 3), (1, 7, 7))]
    marks.append((1, 9, 5))                                     # a past token
    for r, pos, d in marks:
        s.v_bits[s.first[r] + pos, :, d + 3] = 0xFF80
    s.fill()
    sel, q = s.selection(), s.queries()
    for g, (r, row, n, first) in enumerate(s.want["chunks"]):
        sel[:, g] = -1
        sel[:, g, :first // block + 1] = np.arange(first // block + 1)
    o, lse = s.forward(q, sel)
    assert s.code() == 0
    s.v_bits = clean
    want = C.attend(q, *s.values(), s.want["chunks"], sel, block, s.scale)
    got = from_bf16_tensor(o)
    bad = np.zeros(got.shape, bool)
    for g, (r, row, n, first) in enumerate(s.want["chunks"]):
        for t in range(n):
            for rr, pos, d in marks:
                if rr == r and pos <= first + t:
                    d -= d % 16                             # of the group that holds the mark
                    bad[row + t, :, d:d + 16] = True
    x = o.float().cpu().numpy()
    assert np.array_equal(np.isnan(x), bad)
    got[bad] = O.f64_to_bf16(want[0])[bad]
    _close(to_bf16_tensor(got, "cuda"), lse, want)


def test_attention_far_into_a_large_cache(B):
    """Pages beyond 2^32 bytes of cache."""
    kw = dict(past=[500, 130], new=[1, 3], H=4, topk=5, page_base=150000)
    s = Setup(B, **kw)
    assert (s.full.max() * 4) * 9216 > 1 << 32
    s.fill()
    sel, q = s.selection(), s.queries()
    o, lse = s.forward(q, sel)
    assert s.code() == 0
    _close(o, lse, C.attend(q, *s.values(), s.want["chunks"], sel, 64, s.scale))


@pytest.mark.parametrize("new", [[1, 1, 1], [8, 1, 30]])
@pytest.mark.parametrize("kind, code", [("twice", 5), ("future", 5), ("page", 10), ("page_low", 10), ("request", 10),
                                        ("count", 10), ("row", 10), ("position", 10)])
def test_attention_refuses_bad_tables(B, kind, code, new):
    """A bad selection, page or chunk row is reported; its chunk's rows are left as they were."""
    import torch
    s = Setup(B, past=[200, 300, 64], new=new, H=2, topk=4)
    s.fill()
    sel, q, chunks, table = s.selection(), s.queries(), s.chunk_table(), _dev(s.full)
    bad = s.want["chunks"][0]
    if kind == "twice":
        sel[1, 0, :2] = 2
    elif kind == "future":
        sel[1, 0, 1] = int(bad[3]) // 64 + 1
    elif kind in ("page", "page_low"):
        sel[1, 0], sel[0, 0] = [3, 0, -1, -1], [3, -1, -1, -1]
        table[0, 0] = s.c.num_pages if kind == "page" else -1
    else:
        col = dict(request=0, row=1, count=2, position=3)[kind]
        chunks[0, col] = {0: 3, 1: s.T, 2: 9, 3: 64 * s.c.max_blocks}[col]
    o, lse = s.forward(q, sel, chunks, table)
    assert s.code() == code
    x = o.float().cpu().numpy()
    rows = slice(0, int(bad[2]))
    hs = slice(16, 32) if kind in ("twice", "future", "page", "page_low") else slice(0, 32)
    assert np.all(x[rows, hs] == 7.0)
    # with the error standing, a later call writes nothing
    o, lse = s.forward(q, s.selection())
    torch.cuda.synchronize()
    assert bool((o == 7.0).all()) and bool((lse == 7.0).all())


def test_attention_repeats_bit_for_bit(B):
    import torch
    s, q, sel = _attend_case(B, past=[3000, 10, 500], new=[1, 1, 1], H=1, topk=32)
    a = s.forward(q, sel)
    for _ in range(5):
        b = s.forward(q, sel)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------

class Follow:
    """The oracle's side of a Cache object, step by step."""

    def __init__(self, B, kv, H, block, topk):
        self.kv, self.H, self.block, self.K = kv, H, block, topk
        R, M = kv.block_table.shape
        P = kv.free_ring.shape[0]
        self.table, self.ring = np.zeros((R, M), np.int64), np.arange(P)
        self.head, self.count, self.lens = 0, P, np.zeros(R, np.int64)
        self.tail, self.pool = np.zeros((R, 2, block, H, 128), np.uint16), np.zeros((P, H, 128), np.uint16)
        self.k = [np.zeros((0, H, 128)) for _ in range(R)]
        self.v = [np.zeros((0, H, 128)) for _ in range(R)]

    def step(self, new, k, v, ki, qi, q):
        s = C.step(new, self.lens, self.head, self.count, self.ring, self.table, self.block)
        C.index_update(ki, s["cu_tokens"], self.lens, s["block_table"], self.tail, self.pool, self.block)
        kv, vv = C.round_rows(k, 0)[2], C.round_rows(v, 0)[2]
        for r, n in enumerate(new):
            rows = slice(s["cu_tokens"][r], s["cu_tokens"][r + 1])
            self.k[r] = np.concatenate([self.k[r], kv[rows]]) if n >= 0 else self.k[r][:0]
            self.v[r] = np.concatenate([self.v[r], vv[rows]]) if n >= 0 else self.v[r][:0]
        self.table, self.ring, self.head, self.count = s["block_table"], s["free_ring"], s["head"], s["count"]
        self.lens = s["seq_lens"]
        sel = C.select(qi, self.pool, self.table, s["chunks"], self.block, self.K)
        return s, sel, C.attend(q, self.k, self.v, s["chunks"], sel, self.block, 128 ** -0.5)


def _drive(B, kv, f, new, T, rng, graph=None):
    """One step of the object (or a replay of its captured step) against the oracle."""
    import torch
    H = f.H
    x = dict(k=_bf16(rng, (T, H, 128)), v=_bf16(rng, (T, H, 128)), ki=_bf16(rng, (T, H, 128)),
             qi=_bf16(rng, (T, H, 128)), q=_bf16(rng, (T, 16 * H, 128)))
    d = {n: to_bf16_tensor(b, "cuda") for n, b in x.items()}
    if graph is None:
        kv.step(_dev(new), T)
        kv.append(d["k"], d["v"], d["ki"])
        sel = kv.select(d["qi"])
        kv._tables(T)["o"].fill_(7.0)
        kv._tables(T)["lse"].fill_(7.0)
        o, lse = kv.forward(d["q"], sel)
    else:
        g, bufs, sel, o, lse = graph
        bufs["new"].copy_(_dev(new))
        for n in d:
            bufs[n].copy_(d[n])
        o.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
    torch.cuda.synchronize()
    kv.check_status()
    s, wsel, want = f.step(new, x["k"], x["v"], x["ki"], x["qi"], x["q"])
    assert np.array_equal(kv.seq_lens.cpu().numpy(), f.lens)
    assert kv.ring.cpu().tolist() == [f.head, f.count]
    assert np.array_equal(sel.cpu().numpy()[:, :wsel.shape[1]], wsel)
    _close(o, lse, want)


def test_serving_run(B):
    """Prompts in pieces, decode steps, requests that finish and whose pages others take, until the ring has gone
    round; at the end the cache reads back as the oracle's values."""
    import torch
    rng = np.random.default_rng(11)
    H, block, K, R = 2, 64, 3, 4
    kv = B.Cache(num_requests=R, num_pages=14, max_blocks=6, num_q_heads=16 * H, topk=K, block_size=block,
                 max_tokens=300)
    f = Follow(B, kv, H, block, K)
    for new in ([100, 0, 1, 60], [1, 130, 1, 4], [1, 1, 1, 1], [3, 5, 2, 1], [1, -1, 1, -1], [1, 70, 0, 0],
                [-1, 1, 1, 200], [150, 1, -1, 1], [1, -1, 90, -1], [1, 64, 1, 64], [1] * 4, [1] * 4):
        T = int(np.maximum(new, 0).sum())
        _drive(B, kv, f, new, T + (T % 3), rng)
    for r in range(R):
        n = int(f.lens[r])
        if n:
            p = np.arange(n)
            k, v = kv.read(_dev(f.table[r, p // block] * block + p % block, torch.int64))
            assert np.array_equal(O.bf16_to_f64(from_bf16_tensor(k)), f.k[r])
            assert np.array_equal(O.bf16_to_f64(from_bf16_tensor(v)), f.v[r])
    kv.check_status()


@pytest.mark.parametrize("block", [64, 128])
def test_captured_step_replays(B, block):
    """A whole step captured into a CUDA graph on a side stream and replayed with new inputs, lengths and idle
    requests; two objects with their own graphs replay in turn."""
    import torch
    H, K, R, T = 2, 4, 3, 6
    made = []
    for i in range(2):
        rng = np.random.default_rng(20 + i)
        kv = B.Cache(num_requests=R, num_pages=30, max_blocks=8, num_q_heads=16 * H, topk=K, block_size=block,
                     max_tokens=183)
        f = Follow(B, kv, H, block, K)
        _drive(B, kv, f, [120, 3, 60], 183, rng)
        _drive(B, kv, f, [1, 2, 1], T, rng)
        bufs = {n: torch.zeros((T, H, 128), dtype=torch.bfloat16, device="cuda") for n in ("k", "v", "ki", "qi")}
        bufs["q"] = torch.zeros((T, 16 * H, 128), dtype=torch.bfloat16, device="cuda")
        bufs["new"] = torch.zeros(R, dtype=torch.int32, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            kv.step(bufs["new"], T)
            kv.append(bufs["k"], bufs["v"], bufs["ki"])
            sel = kv.select(bufs["qi"])
            o, lse = kv.forward(bufs["q"], sel)
        made.append((kv, f, rng, (g, bufs, sel, o, lse)))
    for new in ([1, 1, 1], [2, 0, 1], [1, 3, 2], [0, 0, 0], [6, 0, 0], [1, -1, 1], [1, 5, 0]):
        for kv, f, rng, graph in made:
            _drive(B, kv, f, new, T, rng, graph)


def test_steps_on_two_streams(B):
    """Two objects on streams of their own, their calls interleaved."""
    import torch
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = []
    for i, st in enumerate(streams):
        rng = np.random.default_rng(30 + i)
        kv = B.Cache(num_requests=2, num_pages=20, max_blocks=8, num_q_heads=32, topk=4, max_tokens=300)
        f = Follow(B, kv, 2, 64, 4)
        x = [dict(k=_bf16(rng, (T, 2, 128)), v=_bf16(rng, (T, 2, 128)), ki=_bf16(rng, (T, 2, 128)),
                  qi=_bf16(rng, (T, 2, 128)), q=_bf16(rng, (T, 32, 128))) for T in (300, 2)]
        runs.append((kv, f, st, x, [{n: to_bf16_tensor(b, "cuda") for n, b in y.items()} for y in x],
                     [_dev([200, 100]), _dev([1, 1])]))
    torch.cuda.synchronize()
    outs = {}
    for j, T in enumerate((300, 2)):
        for i, (kv, f, st, x, d, new) in enumerate(runs):
            kv.step(new[j], T, stream=st)
            kv.append(d[j]["k"], d[j]["v"], d[j]["ki"], stream=st)
            o, lse = kv.forward(d[j]["q"], kv.select(d[j]["qi"], stream=st), stream=st)
            with torch.cuda.stream(st):
                outs[i, j] = o.clone(), lse.clone()     # the next step's calls write the same buffers
    torch.cuda.synchronize()
    for i, (kv, f, st, x, d, new) in enumerate(runs):
        kv.check_status()
        for j in range(2):
            s, sel, want = f.step([[200, 100], [1, 1]][j], *(x[j][n] for n in ("k", "v", "ki", "qi", "q")))
            _close(*outs[i, j], want)


def test_whole_prompt_matches_the_training_forward(B):
    """A prompt appended at once gives the selection of msa_select_topk and, over the values that the cache holds,
    msa_fwd's outputs within both calls' roundings."""
    import torch
    rng = np.random.default_rng(40)
    H, K, n = 2, 5, 700
    bits = {m: _bf16(rng, (n, h, 128)) for m, h in (("k", H), ("v", H), ("ki", H), ("qi", H), ("q", 16 * H))}
    d = {m: to_bf16_tensor(x, "cuda") for m, x in bits.items()}
    kv = B.Cache(num_requests=1, num_pages=20, max_blocks=12, num_q_heads=16 * H, topk=K, max_tokens=n)
    kv.step(_dev([n]), n)
    kv.append(d["k"], d["v"], d["ki"])
    sel = kv.select(d["qi"])
    o, lse = kv.forward(d["q"], sel)
    prob = B.make_problem([0, n], [0], n, 16 * H, K)
    want_sel, _ = B.select_topk(prob, d["qi"], d["ki"])
    nc = prob.num_chunks
    assert torch.equal(sel[:, :nc], want_sel)
    k, v = kv.read(kv.slot_map)
    fo, flse, st = B.forward(prob, want_sel, d["q"], k, v)
    torch.cuda.synchronize()
    kv.check_status()
    assert int(st[0].item()) == 0
    # msa_fwd rounds p to bf16 (2^-8 of the weighted |v|, at most max |v|); both round o
    vmax = v.float().abs().max().item()
    assert (o.float() - fo.float()).abs().max().item() <= 2 * 2.0 ** -8 * vmax + 1.125 * 2.0 ** -8 * vmax
    assert (lse - flse).abs().max().item() <= 1e-4


def test_repeated_append_of_a_step_keeps_the_index(B):
    """A step that is taken back (its lengths restored) and appended again leaves the same means and tail: the open
    block's rows have a buffer of their own."""
    import torch
    s = Setup(B, [60, 10], [10, 3], H=1)
    ki = to_bf16_tensor(_bf16(s.rng, (13, 1, 128)), "cuda")
    tail = to_bf16_tensor(_bf16(s.rng, (2, 2, 64, 1, 128)), "cuda")
    pool = torch.zeros((s.c.num_pages, 1, 128), dtype=torch.bfloat16, device="cuda")
    cache = B.new_cache(s.c)
    out = []
    for _ in range(2):
        B.msa_cache_append(s.c, ki, ki, ki, _dev(s.want["slot_map"], torch.int64), _dev(s.want["cu_tokens"]),
                           s.chunk_table(), cache, tail, pool, s.status)
        torch.cuda.synchronize()
        out.append((tail.clone(), pool.clone(), cache.clone()))
    assert s.code() == 0
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_largest_batch_of_requests(B):
    """8192 requests, the most that a step takes: tables of more than 48 KB of shared memory a CTA."""
    rng = np.random.default_rng(50)
    s = Setup(B, rng.integers(0, 200, 8192), rng.integers(-1, 3, 8192), kv=False)
    got = _run_step(B, s, in_place=True)
    assert s.code() == 0
    assert np.array_equal(got["slots"], s.want["slot_map"]) and np.array_equal(got["chunks"], s.want["chunks"])
    assert np.array_equal(got["table"], s.want["block_table"]) and np.array_equal(got["ring"], s.want["free_ring"])
    assert np.array_equal(got["lens_out"], s.want["seq_lens"])


@pytest.mark.parametrize("past, new, H, kernel", [([0] * 60, [25] * 60, 2, "chunks"), ([300] * 200, [1] * 200, 2, "batch"),
                                                  ([900, 3], [1, 1], 1, "cluster")])
def test_captured_attention_of_every_kernel(B, past, new, H, kernel):
    """Each of the three attention kernels captured on a side stream and replayed: the same bits as the eager call."""
    import torch
    s = Setup(B, past=past, new=new, H=H, topk=6)
    s.fill()
    sel, q = s.selection(), s.queries()
    want_o, want_lse = s.forward(q, sel)
    assert s.code() == 0
    _close(want_o, want_lse, C.attend(q, *s.values(), s.want["chunks"], sel, s.block, s.scale))
    d = dict(q=to_bf16_tensor(q, "cuda"), table=_dev(s.full), chunks=s.chunk_table(), sel=_dev(sel))
    o, lse = torch.zeros_like(want_o), torch.zeros_like(want_lse)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        B.msa_cache_fwd(s.c, d["q"], s.cache, d["table"], d["chunks"], d["sel"], o, lse, s.status)
    for _ in range(3):
        o.zero_()
        lse.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want_o) and torch.equal(lse, want_lse)


def test_cache_without_index_keys(B):
    """A cache whose caller brings the selection: no index buffers, and read of the step's slots with padding."""
    import torch
    rng = np.random.default_rng(70)
    kv = B.Cache(num_requests=2, num_pages=9, max_blocks=4, num_q_heads=32, topk=2, max_tokens=210, index_keys=False)
    bits = {m: _bf16(rng, (210, h, 128)) for m, h in (("k", 2), ("v", 2), ("q", 32))}
    d = {m: to_bf16_tensor(x, "cuda") for m, x in bits.items()}
    kv.step(_dev([70, 130]), 210)
    kv.append(d["k"], d["v"])
    want = C.step([70, 130], [0, 0], 0, 9, np.arange(9), np.zeros((2, 4), int), 64)
    sel = np.full((2, kv._tables(210)["c"].chunk_cap, 2), -1)
    for g, (r, row, n, first) in enumerate(want["chunks"]):
        sel[:, g, 0], sel[:, g, 1] = first // 64, (0 if first >= 64 else -1)
    kv._o.fill_(7.0)
    kv._lse.fill_(7.0)
    o, lse = kv.forward(d["q"], _dev(sel))
    k, v = kv.read(kv.slot_map)
    torch.cuda.synchronize()
    kv.check_status()
    kq, vq = C.round_rows(bits["k"][:200], 0)[2], C.round_rows(bits["v"][:200], 0)[2]
    _close(o, lse, C.attend(bits["q"], [kq[:70], kq[70:]], [vq[:70], vq[70:]], want["chunks"], sel, 64, 128 ** -0.5))
    for x, y in ((k, kq), (v, vq)):
        assert np.array_equal(O.bf16_to_f64(from_bf16_tensor(x))[:200], y) and not bool(x[200:].any())


def test_refused_step_can_be_repaired(B):
    """A step that finds no free page changes nothing; after reset_status the batch goes on as before it."""
    import torch
    rng = np.random.default_rng(60)
    kv = B.Cache(num_requests=2, num_pages=3, max_blocks=4, num_q_heads=16, topk=2, max_tokens=130)
    f = Follow(B, kv, 1, 64, 2)
    _drive(B, kv, f, [64, 1], 65, rng)
    kv.step(_dev([1, 128]), 129)
    torch.cuda.synchronize()
    with pytest.raises(B.MSAError) as e:
        kv.check_status()
    assert e.value.code == B.MSA_ERR_CAPACITY
    kv.reset_status()
    _drive(B, kv, f, [1, 63], 64, rng)
    _drive(B, kv, f, [-1, 0], 1, rng)
    _drive(B, kv, f, [0, 65], 65, rng)


def _off(t):
    """A copy of t that is aligned to 16 bytes and to no more."""
    import torch
    n = 16 // t.element_size()
    base = torch.zeros(t.numel() + 2 * n + 64, dtype=t.dtype, device=t.device)
    at = n if base.data_ptr() % 32 == 0 else 0
    x = base[at:at + t.numel()].view(t.shape)
    assert x.data_ptr() % 32 == 16
    x.copy_(t)
    return x


@pytest.mark.parametrize("past, new", [([300, 90, 1], [1, 1, 1]), ([3] * 40, [70] * 40), ([0], [5])])
def test_tensors_aligned_to_16_bytes_only(B, past, new):
    """Every call with every pointer 16 bytes off a 32-byte border gives the same bits."""
    import torch
    s = Setup(B, past, new, H=2, topk=3)
    T, R, P = s.c.token_cap, len(past), s.c.num_pages
    i32 = torch.int32

    def run(f):
        new_, lens, at = f(_dev(s.new)), f(_dev(s.past)), f(_dev([s.start["head"], s.start["count"]]))
        ring, table = f(_dev(s.start["ring"])), f(_dev(s.start["table"]))
        cu, slots = f(torch.zeros(R + 1, dtype=i32, device="cuda")), f(torch.zeros(T, dtype=torch.int64, device="cuda"))
        pos, chunks = f(torch.zeros(T, dtype=i32, device="cuda")), f(torch.zeros((s.c.chunk_cap, 4), dtype=i32, device="cuda"))
        st = f(torch.zeros(4, dtype=i32, device="cuda"))
        B.msa_cache_step(s.c, new_, lens, at, ring, table, lens, at, cu, slots, pos, chunks, st)
        g = torch.Generator(device="cuda")
        g.manual_seed(3)
        rnd = lambda *shape: f(torch.randn(shape, generator=g, device="cuda").bfloat16())
        k, v, ki, qi, q = rnd(T, 2, 128), rnd(T, 2, 128), rnd(T, 2, 128), rnd(T, 2, 128), rnd(T, 32, 128)
        tail, pool, cache = rnd(R, 2, 64, 2, 128), rnd(P, 2, 128), f(B.new_cache(s.c))
        B.msa_cache_append(s.c, k, v, ki, slots, cu, chunks, cache, tail, pool, st)
        sel = f(torch.full((2, s.c.chunk_cap, 3), -1, dtype=i32, device="cuda"))
        B.msa_cache_select(s.c, qi, pool, table, chunks, sel, st)
        o, lse = f(torch.zeros((T, 32, 128), dtype=torch.bfloat16, device="cuda")), f(torch.zeros((T, 32), device="cuda"))
        B.msa_cache_fwd(s.c, q, cache, table, chunks, sel, o, lse, st)
        rk, rv = f(torch.zeros_like(k)), f(torch.zeros_like(v))
        B.msa_cache_read(s.c, slots, cache, rk, rv, st)
        torch.cuda.synchronize()
        assert int(st[0].item()) == 0
        return [lens, at, ring, table, cu, slots, pos, chunks, cache, tail, pool, sel, o, lse, rk, rv]

    for a, b in zip(run(lambda t: t), run(_off)):
        assert torch.equal(a, b)


def test_captured_step_with_a_join(B):
    """Calls captured behind a fork and a join with another stream's work (copies, kernels of others): the launches'
    programmatic serialisation must not skip a dependency."""
    import torch
    rng = np.random.default_rng(80)
    H, T = 2, 64
    kv = B.Cache(num_requests=T, num_pages=300, max_blocks=4, num_q_heads=16 * H, topk=2, block_size=64,
                 max_tokens=64 * T)
    f = Follow(B, kv, H, 64, 2)
    _drive(B, kv, f, [40 + i % 30 for i in range(T)], 64 * T, rng)
    _drive(B, kv, f, [1] * T, T, rng)
    names = {"k": H, "v": H, "ki": H, "qi": H, "q": 16 * H}
    src = {n: torch.zeros((T, h, 128), dtype=torch.bfloat16, device="cuda") for n, h in names.items()}
    dst = {n: torch.zeros_like(x) for n, x in src.items()}
    new = torch.ones(T, dtype=torch.int32, device="cuda")
    big = torch.zeros(1 << 26, device="cuda")
    g, side, other = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        other.wait_stream(side)
        kv.step(new, T)
        with torch.cuda.stream(other):
            big.add_(1.0)                                   # keeps the other branch behind the step
            for n in ("k", "v", "ki"):
                dst[n].copy_(src[n])
        side.wait_stream(other)
        kv.append(dst["k"], dst["v"], dst["ki"])
        for n in ("qi", "q"):
            dst[n].copy_(src[n])
        sel = kv.select(dst["qi"])
        o, lse = kv.forward(dst["q"], sel)
        keep_o, keep_lse, keep_sel = o.clone(), lse.clone(), sel.clone()
    for _ in range(4):
        x = {n: _bf16(rng, (T, h, 128)) for n, h in names.items()}
        for n in names:
            src[n].copy_(to_bf16_tensor(x[n], "cuda"))
        g.replay()
        torch.cuda.synchronize()
        kv.check_status()
        s, wsel, want = f.step([1] * T, *(x[n] for n in ("k", "v", "ki", "qi", "q")))
        assert np.array_equal(keep_sel.cpu().numpy()[:, :wsel.shape[1]], wsel)
        _close(keep_o, keep_lse, want)


def _keep_busy():
    """Work of some 20 ms on the current stream: what is queued there next comes later than another stream's work."""
    import torch
    x = torch.zeros(1 << 28, device="cuda")
    torch.cuda.synchronize()
    for _ in range(60):
        x.add_(1.0)
    return x


def test_read_on_a_side_stream(B):
    """read(stream=s) while the current stream is busy: the rows' first values and the kernel's are both s's work, so the
    result is there once s is done, rows of slot -1 are zero, and memory that the current stream still reads is not
    handed to it."""
    import torch
    rng = np.random.default_rng(90)
    kv = B.Cache(num_requests=1, num_pages=4, max_blocks=4, num_q_heads=32, topk=2, max_tokens=130, index_keys=False)
    bits = [_bf16(rng, (130, 2, 128)) for _ in range(2)]
    kv.step(_dev([130]), 130)
    kv.append(*(to_bf16_tensor(x, "cuda") for x in bits))
    slots = kv.slot_map.clone()
    slots[5] = -1
    want = [C.round_rows(x, 0)[2] for x in bits]
    for x in want:
        x[5] = 0.0
    side = torch.cuda.Stream()
    kv.read(slots, stream=side)             # the kernel is loaded: its first launch may wait for the whole device
    old = [torch.full((130, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    busy = _keep_busy()
    seen = [x.clone() for x in old]         # queued behind the work; the memory goes back to the allocator at once
    del old
    got = kv.read(slots, stream=side)
    side.synchronize()
    first = [x.clone() for x in got]
    torch.cuda.synchronize()
    kv.check_status()
    del busy
    assert all(bool((x == 3.0).all()) for x in seen)
    for late, early, w in zip(got, first, want):
        assert np.array_equal(O.bf16_to_f64(from_bf16_tensor(late)), w)
        assert torch.equal(late, early)


@pytest.mark.parametrize("past, new, H", [([3000] * 200, [1] * 200, 4), ([900, 64, 4000], [900, 300, 500], 4)])
def test_selection_with_bad_rows_among_many(B, past, new, H):
    """Bad chunk rows and pages in a launch of many CTAs, for single tokens and for prompts: the error is reported, bad
    rows are left as they were, and a good row is either the oracle's or, where its CTA came up behind the error, left."""
    s = Setup(B, past, new, H=H, topk=8, kv=False)
    qi, pool = _bf16(s.rng, (s.c.token_cap, H, 128)), _bf16(s.rng, (s.c.num_pages, H, 128), 0.125)
    want = C.select(qi, pool, s.full, s.want["chunks"], 64, 8)
    import torch
    d = dict(qi=to_bf16_tensor(qi, "cuda"), pool=to_bf16_tensor(pool, "cuda"), table=_dev(s.full))
    for kind in ("row", "page"):
        chunks, table = s.chunk_table(), d["table"].clone()
        bad = np.zeros(s.c.chunk_cap, bool)
        if kind == "row":
            at = s.rng.permutation(len(s.want["chunks"]))[:12]
            for i, g in enumerate(at):
                col, value = [(0, len(past)), (1, -1), (1, s.T), (2, 0), (2, 9), (3, -1)][i % 6]
                chunks[int(g), col] = value
            bad[at] = True
        else:
            r = len(past) // 2
            table[r, 0] = s.c.num_pages
            bad[[g for g, c in enumerate(s.want["chunks"]) if c[0] == r]] = True
        for _ in range(5):
            s.status.zero_()
            sel = torch.full((H, s.c.chunk_cap, 8), -5, dtype=torch.int32, device="cuda")
            B.msa_cache_select(s.c, d["qi"], d["pool"], table, chunks, sel, s.status)
            assert s.code() == B.MSA_ERR_INVALID_CACHE
            got = sel.cpu().numpy()
            left = (got == -5).all(2)
            if kind == "row":
                assert left[:, bad].all()
            ok = ~left & ~bad[None]
            assert np.array_equal(got[ok], want[ok])


def _attention_kernel(s):
    """Which of the three attention kernels msa_cache_fwd picks for a case, from the sizes, as it does."""
    import torch
    c, sms = s.c, torch.cuda.get_device_properties(0).multi_processor_count
    slots = -(-c.token_cap // c.chunk_cap)
    slots = min(8, 2 * slots if slots > 1 else 1)
    ranks, tiles = 1, c.topk * (c.block_size // 64)
    while ranks < 8 and 2 * ranks <= tiles and c.chunk_cap * slots * c.num_kv_heads * 2 * ranks <= 2 * sms:
        ranks *= 2
    return "cluster" if ranks > 1 else "chunks" if 4 * c.token_cap >= 5 * c.chunk_cap else "batch"


# sizes that the persistent kernels take, more items than they have CTAs
PERSISTENT = {
    "batch": dict(past=[(37 * i) % 500 for i in range(200)], new=[1] * 200, H=2),
    "batch, some of several tokens": dict(past=[(37 * i) % 500 for i in range(200)],
                                          new=[{3: 3, 50: 2, 120: 8, 199: 5}.get(i, 1) for i in range(200)], H=2),
    "chunks": dict(past=[(61 * i) % 300 for i in range(24)], new=[20, 3, 8, 1] * 6, H=8),
}


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("case", list(PERSISTENT))
def test_persistent_attention_over_any_selection(B, case, block):
    """Empty slots anywhere, blocks in any order, chunks without their own block, and runs of chunks that select
    nothing, in the two persistent kernels."""
    s = Setup(B, topk=4, block=block, garbage=0xFF, seed=4, token_pad=3, chunk_pad=2, **PERSISTENT[case])
    assert _attention_kernel(s) == case.split(",")[0]
    s.fill()
    sel, q = s.selection("holes"), s.queries()
    nothing = s.rng.random(sel.shape[:2]) < 0.4
    sel[nothing] = -1
    assert (sel < 0).all(2).mean() > 0.3
    o, lse = s.forward(q, sel)
    assert s.code() == 0
    _close(o, lse, C.attend(q, *s.values(), s.want["chunks"], sel, block, s.scale))


@pytest.fixture(scope="module")
def persistent(B):
    """The sizes above with everything in the cache, a selection, queries and the oracle's result: made once a case."""
    made = {}

    def get(case):
        if case not in made:
            s = Setup(B, topk=4, **PERSISTENT[case])
            assert _attention_kernel(s) == case.split(",")[0]
            s.fill()
            sel, q = s.selection(), s.queries()
            made[case] = s, sel, q, C.attend(q, *s.values(), s.want["chunks"], sel, 64, s.scale)
        return made[case]

    yield get
    made.clear()


@pytest.mark.parametrize("kind, code", [("twice", 5), ("future", 5), ("page", 10), ("request", 10), ("count", 10),
                                        ("row", 10), ("position", 10), ("straddle", 10)])
@pytest.mark.parametrize("case", list(PERSISTENT))
def test_persistent_attention_refuses_bad_tables(persistent, case, kind, code):
    """Bad selections, pages and chunk rows among many, in the persistent kernels: reported, their rows left as they
    were.  Other rows are right, or left by a CTA that came up behind the error; with the error standing, a call writes
    nothing; without it the same tensors serve again."""
    import torch
    s, good, q, want = persistent(case)
    sel, chunks, table = good.copy(), s.chunk_table(), _dev(s.full)
    s.status.zero_()
    T, H = s.T, s.H
    bad = np.zeros((T, 16 * H), bool)
    for g in [0, 7, len(s.want["chunks"]) - 1] + s.rng.choice(len(s.want["chunks"]), 4).tolist():
        r, row, n, first = (int(x) for x in s.want["chunks"][g])
        hs = slice(0, 16 * H)
        if kind in ("twice", "future"):
            hs = slice(16, 32)
            sel[1, g, :2] = first // 64 if kind == "twice" else [first // 64 + 1, -1]
        elif kind == "page":
            sel[:, g, :] = [first // 64, -1, -1, -1]
            table[r, first // 64] = s.c.num_pages if g else -1
            for x, c in enumerate(s.want["chunks"]):    # other chunks of the request may select the page
                if c[0] == r:
                    bad[c[1]:c[1] + c[2]] = True
        else:
            col = dict(request=0, row=1, count=2, position=3, straddle=3)[kind]
            chunks[g, col] = {"request": len(s.past), "row": T, "count": 9, "position": 64 * s.c.max_blocks,
                              "straddle": first // 8 * 8 + 9 - n}[kind]
            if kind == "straddle" and n == 1:
                chunks[g, 2] = 2                        # position 8 k + 7 with two tokens
                chunks[g, 3] = first // 8 * 8 + 7
        bad[row:row + n, hs] = True
    o, lse = s.forward(q, sel, chunks, table)
    assert s.code() == code
    got = o.float().cpu().numpy()
    left = (got == 7.0).all(2) & (lse.cpu().numpy() == 7.0)
    if kind != "page":
        assert left[bad].all()
    live = want[1].copy()
    live[left] = np.nan                                 # as _close has them: not written
    rest = live.copy()
    rest[bad] = np.nan
    o2, lse2 = o.clone(), lse.clone()
    mask = torch.as_tensor(bad, device="cuda")
    o2[mask], lse2[mask] = 7.0, 7.0                     # bad rows are not compared
    _close(o2, lse2, (want[0], rest, *want[2:]))
    o, lse = s.forward(q, good)
    torch.cuda.synchronize()
    assert bool((o == 7.0).all()) and bool((lse == 7.0).all())
    s.status.zero_()
    o, lse = s.forward(q, good)
    assert s.code() == 0
    _close(o, lse, want)


def test_append_and_read_with_bad_slots_among_many(B):
    """Slots outside the cache in launches of many CTAs: reported and left out; the other rows are right, or left as
    they were by CTAs that came up behind the error."""
    import torch
    rng = np.random.default_rng(91)
    P, T, H = 100, 6000, 2
    slots = rng.permutation(P * 64)[:T].astype(np.int64)
    at = rng.permutation(T)[:9]
    broken = slots.copy()
    broken[at] = [P * 64, -2, 1 << 40] * 3
    c = B.make_cache_problem(num_requests=1, num_pages=P, max_blocks=1, num_q_heads=16 * H, topk=1, token_cap=T,
                             chunk_cap=1)
    bits = _bf16(rng, (T, H, 128))
    x = to_bf16_tensor(bits, "cuda")
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    want = C.round_rows(bits, 0)[2]
    cache = B.new_cache(c)
    B.msa_cache_append(c, x, x, None, _dev(broken, torch.int64), None, None, cache, None, None, st)
    torch.cuda.synchronize()
    assert int(st[0].item()) == B.MSA_ERR_INVALID_CACHE
    st.zero_()
    out = [torch.full((T, H, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    B.msa_cache_read(c, _dev(slots, torch.int64), cache, *out, st)
    torch.cuda.synchronize()
    assert int(st[0].item()) == 0
    for y in out:       # per token, head and 16 dims: what the row holds, or the zeros of before
        y = O.bf16_to_f64(from_bf16_tensor(y)).reshape(T, H, 8, 16)
        right, zero = (y == want.reshape(y.shape)).all(3), (y == 0).all(3)
        assert zero[at].all() and (right | zero).all()
    cache = B.new_cache(c)
    B.msa_cache_append(c, x, x, None, _dev(slots, torch.int64), None, None, cache, None, None, st)
    for y in out:
        y.fill_(9.0)
    B.msa_cache_read(c, _dev(broken, torch.int64), cache, *out, st)
    torch.cuda.synchronize()
    assert int(st[0].item()) == B.MSA_ERR_INVALID_CACHE
    for y in out:
        y = O.bf16_to_f64(from_bf16_tensor(y)).reshape(T, H, 8, 16)
        right, left = (y == want.reshape(y.shape)).all(3), (y == 9.0).all(3)
        assert left[at].all() and (right | left).all()


def test_calls_from_several_threads(B):
    """Host threads with caches of very different sizes on streams of their own: a call must not fail because another
    thread's launch of the same kernel needs less shared memory.  (The entry points are called without the binding's
    checks, which hold the interpreter's lock: the threads then meet inside the library.)"""
    import ctypes
    import threading
    import torch

    def made(R, M):
        c = B.make_cache_problem(num_requests=R, num_pages=4, max_blocks=M, num_q_heads=16, topk=1, token_cap=1,
                                 chunk_cap=1)
        i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")
        step = (i32(R), i32(R), _dev([0, 4]), _dev(np.arange(4)), i32(R, M), i32(R), i32(2), i32(R + 1),
                torch.zeros(1, dtype=torch.int64, device="cuda"), i32(1), i32(1, 4) - 1, i32(4))
        rows = torch.zeros((4, 1, 128), dtype=torch.bfloat16, device="cuda")
        select = (rows[:1], rows, step[4], step[10], i32(1, 1, 1), step[11])
        stream = torch.cuda.Stream()
        fix = lambda t: [ctypes.byref(c)] + [ctypes.c_void_p(x.data_ptr()) for x in t] + [ctypes.c_void_p(stream.cuda_stream)]
        return (c, step, select, stream), fix(step), fix(select)

    work = [made(*x) for x in [(8192, 40000), (2000, 12000), (8000, 30000), (1900, 9000)]]
    torch.cuda.synchronize()
    failed, start = [0] * len(work), threading.Barrier(len(work))

    def run(i):
        _, step, select = work[i]
        start.wait()
        for _ in range(15000):
            failed[i] += B.lib.msa_cache_step(*step) != 0
            failed[i] += B.lib.msa_cache_select(*select) != 0

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * len(work)
    assert all(int(keep[1][-1][0].item()) == 0 for keep, _, _ in work)


@pytest.mark.parametrize("position, count, append_ok, select_ok", [
    (3, 5, True, True), (62, 5, False, True), (60, 5, False, True), (59, 5, True, True), (1 << 30, 5, False, False),
    (64 * 3, 5, False, False), (64 * 3 - 5, 5, True, True), ((1 << 31) - 6, 5, False, False), (0, 5, True, True)])
def test_append_and_select_check_positions(B, position, count, append_ok, select_ok):
    """A chunk row whose position does not fit: one that leaves its block is refused by append, one behind the block
    table by both, the largest int among them; any other is followed, and its rows of the index tail are those of its
    position."""
    import torch
    s = Setup(B, [3], [5])
    assert s.c.max_blocks == 3
    ki = _bf16(s.rng, (5, 1, 128))
    di = to_bf16_tensor(ki, "cuda")
    chunks = s.chunk_table()
    chunks[0, 2:] = torch.tensor([count, position], dtype=torch.int32)
    tail = torch.zeros((1, 2, 64, 1, 128), dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros((s.c.num_pages, 1, 128), dtype=torch.bfloat16, device="cuda")
    B.msa_cache_append(s.c, di, di, di, _dev(s.want["slot_map"], torch.int64), _dev(s.want["cu_tokens"]), chunks,
                       B.new_cache(s.c), tail, pool, s.status)
    want = np.zeros((1, 2, 64, 1, 128), np.uint16)
    assert s.code() == (0 if append_ok else B.MSA_ERR_INVALID_CACHE)
    if append_ok and (position + 5) % 64:
        want[0, position // 64 & 1, position % 64:position % 64 + 5] = ki
    if not append_ok or (position + 5) % 64:
        assert np.array_equal(from_bf16_tensor(tail), want) and not bool(pool.any())
    s.status.zero_()
    sel = torch.full((1, s.c.chunk_cap, s.K), -5, dtype=torch.int32, device="cuda")
    B.msa_cache_select(s.c, di, pool, torch.zeros((1, 3), dtype=torch.int32, device="cuda"), chunks, sel, s.status)
    assert s.code() == (0 if select_ok else B.MSA_ERR_INVALID_CACHE)
    if select_ok:
        assert int(sel[0, 0, 0].item()) == position // 64
    else:
        assert bool((sel == -5).all())
