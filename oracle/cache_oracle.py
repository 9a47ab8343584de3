"""Plain CPU oracle of the serving operators over the 4-bit paged cache.

TEST INFRASTRUCTURE ONLY, as ``msa_oracle``: only ``tests/`` imports it, and it
shares no code with the CUDA library.  fp64 throughout; tables and cache bytes
are exact, outputs of the attention are fp64.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from oracle.msa_oracle import bf16_to_f64, block_scores, f64_to_bf16

TILE, TILE_BYTES = 64, 9216
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def e4m3_value(code: int) -> float:
    """Value of an unsigned e4m3 pattern (0x7F is NaN)."""
    if code == 0x7F:
        return math.nan
    e, m = code >> 3, code & 7
    return m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)


E4M3 = np.array([e4m3_value(c) for c in range(0x7F)])


# ---------------------------------------------------------------------------
# tables
# ---------------------------------------------------------------------------

def step(new_lens, seq_lens, head, count, free_ring, block_table, block, chunk=8):
    """One step's tables, token by token.  Returns a dict; the inputs are not changed."""
    table, ring = np.array(block_table, np.int64), np.array(free_ring, np.int64)
    P = len(ring)
    taken, lens, cu, slots, pos, chunks = 0, [], [0], [], [], []
    for r, (n, past) in enumerate(zip(new_lens, seq_lens)):
        n, past = int(n), int(past)
        for p in range(past, past + max(n, 0)):
            if p % block == 0:
                table[r, p // block] = ring[(head + taken) % P]
                taken += 1
            if p == past or p % chunk == 0:
                chunks.append([r, len(pos), 0, p])
            chunks[-1][2] += 1
            slots.append(int(table[r, p // block]) * block + p % block)
            pos.append(p)
        cu.append(len(pos))
        lens.append(0 if n < 0 else past + n)
    assert taken <= count
    back = 0
    for r, (n, past) in enumerate(zip(new_lens, seq_lens)):
        if n < 0:
            for b in range(-(-int(past) // block)):
                ring[(head + count + back) % P] = table[r, b]
                back += 1
    return dict(block_table=table, free_ring=ring, head=(head + taken) % P, count=count - taken + back,
                seq_lens=np.array(lens), cu_tokens=np.array(cu), slot_map=np.array(slots, np.int64),
                positions=np.array(pos, np.int64), chunks=np.array(chunks, np.int64).reshape(-1, 4))


# ---------------------------------------------------------------------------
# 4-bit rounding and the cache's bytes
# ---------------------------------------------------------------------------

def round_group(x, exp):
    """(codes [16], e4m3 pattern) of 16 numbers, in rational arithmetic."""
    if not np.all(np.isfinite(x)):
        return None, 0x7F
    y = [Fraction(float(v)) / Fraction(2) ** exp for v in x]
    t = max(abs(v) for v in y) / 6
    scale = _nearest(t, [Fraction(float(v)) for v in E4M3])
    s = Fraction(float(E4M3[scale]))
    if s == 0:
        return [0] * len(y), 0
    levels = [Fraction(v) for v in E2M1]
    codes = [_nearest(abs(v) / s, levels) for v in y]
    return [c + 8 if c and v < 0 else c for c, v in zip(codes, y)], scale


def _nearest(t, values):
    """Index of the nearest of ascending values, ties to the even index; the last beyond it."""
    if t >= values[-1]:
        return len(values) - 1
    hi = next(i for i, v in enumerate(values) if v > t)
    lo = hi - 1
    a, b = t - values[lo], values[hi] - t
    return lo if a < b or (a == b and lo % 2 == 0) else hi


def round_rows(bits, exp):
    """Codes uint8 [..., 128], e4m3 patterns uint8 [..., 8] and fp64 values of bf16 rows, vectorised:
    exact because every product below is exact in fp64."""
    x = bf16_to_f64(np.asarray(bits)) * 2.0 ** -exp
    g = x.reshape(*x.shape[:-1], 8, 16)
    finite = np.isfinite(g).all(-1)
    amax = np.where(finite, np.abs(np.where(np.isfinite(g), g, 0)).max(-1), 0.0)
    # nearest e4m3 of amax / 6: compare 6 * midpoint with amax
    mids = (E4M3[:-1] + E4M3[1:]) / 2 * 6
    idx = np.searchsorted(mids, amax, side="left")             # mids below amax
    tie = (idx < len(mids)) & (mids[np.minimum(idx, len(mids) - 1)] == amax)
    idx = np.where(tie & (idx % 2 == 1), idx + 1, idx)         # between idx and idx + 1: the even one
    s = E4M3[idx][..., None]
    a = np.where(np.isfinite(g), np.abs(g), 0.0)
    code = np.zeros(g.shape, np.int64)
    for i in range(1, 8):
        mid = (E2M1[i - 1] + E2M1[i]) / 2 * s
        code = np.where((a > mid) if i % 2 else (a >= mid), i, code)
    code = np.where(s > 0, code + 8 * ((g < 0) & (code > 0)), 0)    # a zero has no sign
    pattern = np.where(finite, idx, 0x7F)
    vals = np.where(finite[..., None], np.array(E2M1 + [-v for v in E2M1])[code] * s, np.nan) * 2.0 ** exp
    return (code.reshape(x.shape).astype(np.uint8), pattern.astype(np.uint8), vals.reshape(x.shape))


def write_row(cache, slot, head, block, kcode, kscale, vcode, vscale):
    """Puts one token's rows into the cache's bytes [P, H, block / 64, 9216]."""
    page, off = divmod(int(slot), block)
    tile, t = divmod(off, TILE)
    b = cache[page, head, tile]
    pack = lambda c: (c[0::2] | (c[1::2] << 4)).astype(np.uint8)
    b[t * 64:t * 64 + 64] = pack(kcode)
    b[4096 + t * 8:4096 + t * 8 + 8] = kscale
    at = (t * 64 + np.arange(64)) ^ ((t & 12) << 3)
    b[4608 + at] = pack(vcode)
    b[8704 + np.arange(8) * 64 + t] = vscale


def append(cache, k_bits, v_bits, slots, block, k_exp=0, v_exp=0):
    """Writes bf16 rows [T, H, 128] to their slots (-1: not)."""
    kc, ks, _ = round_rows(k_bits, k_exp)
    vc, vs, _ = round_rows(v_bits, v_exp)
    for t, slot in enumerate(slots):
        if slot >= 0:
            for h in range(k_bits.shape[1]):
                write_row(cache, slot, h, block, kc[t, h], ks[t, h], vc[t, h], vs[t, h])


def index_update(k_index, cu, past, table, tail, pool, block):
    """Pooled index keys (bf16 bits) of the blocks that the step completes, and the tail's rows; in place."""
    for r in range(len(past)):
        n, row, p0 = int(cu[r + 1] - cu[r]), int(cu[r]), int(past[r])
        old = tail[r].copy()
        for b in range(p0 // block, -(-(p0 + n) // block)):
            lo, hi = max(p0, b * block), min(p0 + n, (b + 1) * block)
            new = k_index[row + lo - p0:row + hi - p0]
            if hi == (b + 1) * block:
                acc = np.zeros(new.shape[1:], np.float32)
                for x in list(old[b & 1, :lo - b * block]) + list(new):
                    acc = acc + bf16_to_f64(x).astype(np.float32)
                pool[table[r, b]] = f64_to_bf16((acc / np.float32(block)).astype(np.float64))
            else:
                tail[r, b & 1, lo - b * block:hi - b * block] = new


# ---------------------------------------------------------------------------
# selection and attention
# ---------------------------------------------------------------------------

def select(q_index, pool, table, chunks, block, topk):
    """sel int32 [H, NC, topk] from index queries [T, H, 128] and pooled keys [P, H, 128] (bf16 bits)."""
    H = q_index.shape[1]
    sel = np.full((H, len(chunks), topk), -1, np.int32)
    for g, (r, row, n, first) in enumerate(chunks):
        diag = first // block
        acc = np.zeros(q_index.shape[1:], np.float32)
        for i in range(n):
            acc = acc + bf16_to_f64(q_index[row + i]).astype(np.float32)
        q = f64_to_bf16((acc / np.float32(n)).astype(np.float64))
        for h in range(H):
            s = block_scores(q[None, h], pool[table[r, :diag], h])[0]
            ranked = sorted(range(diag), key=lambda b: (-float(s[b]), b))[:topk - 1]
            sel[h, g, :1 + len(ranked)] = [diag] + ranked
    return sel


def attend(q_bits, values_k, values_v, chunks, sel, block, scale, group=16):
    """fp64 attention.  values_k / values_v: per request, fp64 [tokens, H, 128] as the cache holds them.
    Returns o, lse, the p-weighted mean of |v| per element and the largest sum |q_d k_jd| * scale of a row
    (the last two bound rounding errors), and the largest |v| of the requests; rows that no chunk covers are NaN in
    o and lse."""
    q = bf16_to_f64(q_bits)
    T, Hq, D = q.shape
    o, absv = np.full((T, Hq, D), np.nan), np.zeros((T, Hq, D))
    lse, mag = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    for g, (r, row, n, first) in enumerate(chunks):
        for h in range(Hq // group):
            blocks = [int(b) for b in sel[h, g] if b >= 0]
            for i in range(n):
                pos = np.array([p for b in blocks for p in range(b * block, (b + 1) * block) if p <= first + i], int)
                hs = slice(h * group, (h + 1) * group)
                if pos.size == 0:
                    o[row + i, hs], lse[row + i, hs] = 0.0, -np.inf
                    continue
                k, v = values_k[r][pos, h], values_v[r][pos, h]
                x = q[row + i, hs] @ k.T * scale
                m = x.max(1, keepdims=True)
                p = np.exp(x - m)
                l = p.sum(1, keepdims=True)
                o[row + i, hs], lse[row + i, hs] = p @ v / l, (m + np.log(l))[:, 0]
                absv[row + i, hs] = p @ np.abs(v) / l
                mag[row + i, hs] = (np.abs(q[row + i, hs]) @ np.abs(k).T).max(1) * scale
    return o, lse, absv, mag, max((np.abs(v).max() for v in values_v if v.size), default=0.0)
