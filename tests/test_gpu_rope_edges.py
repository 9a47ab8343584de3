"""GPU: norm and rotary positions at the ends of what the calls allow (the largest finite rows, inputs and outputs that
share memory, padding, streams, status words), against the fp64 oracle with the bounds of ``test_gpu_rope``."""
import numpy as np
import pytest

from oracle import msa_oracle as O
from oracle import rope_oracle as R
from tests._util import to_bf16_tensor
from tests.test_gpu_cache import _bf16, _dev
from tests.test_gpu_rope import B, Layer, _append_problem, _check_forward, _check_grad, _expected_cache, _f64  # noqa: F401

pytestmark = pytest.mark.gpu

MOST = 0x7F7F       # the largest finite bf16
LIMIT = 2.0 ** 128 - 2.0 ** 120


def _large_rows(rng, shape):
    """bf16 bits of rows (first axis) of every size whose squares leave fp32's range: all of the largest value, two large
    values among ordinary ones, small values beside one large one; every fifth row is ordinary."""
    T = shape[0]
    x = rng.standard_normal(shape)
    big = np.array([0, 100, 120, 123, 0, 124.5, 125, 126, 60, 64])
    x *= (2.0 ** big[np.arange(T) % 10])[:, None, None]
    i = np.arange(T) % 10
    x[i == 8] *= 2.0 ** -118        # 2^-58, beside one of 2^64
    x[i == 8, :, 77] = -2.0 ** 64
    bits = O.f64_to_bf16(np.clip(x, -LIMIT, LIMIT))
    sign = (rng.integers(0, 2, shape) << 15).astype(np.uint16)
    bits[i == 7] = (MOST | sign)[i == 7]
    two = np.flatnonzero(i == 5)
    bits[two] = O.f64_to_bf16(rng.standard_normal((len(two), *shape[1:])))
    bits[two, :, 3], bits[two, :, 90] = O.f64_to_bf16(np.float64(2.5e38)), MOST | 0x8000
    return bits


@pytest.mark.parametrize("kw", [dict(H=2), dict(adjacent=True, rotary=64, per_head=True, wide=False, offset=1.0, scale=1.2)])
def test_largest_rows(B, kw):
    """The definition's values for rows up to bf16's largest, forward and gradients; the ordinary rows beside them keep
    their bits."""
    import torch
    L = Layer(B, seed=50, **kw)
    T = 40
    pos = L.positions(T)
    x = [_large_rows(L.rng, (T, h, 128)) for h in L.heads]
    dy = [_bf16(L.rng, (T, h, 128)) for h in L.heads]
    put = lambda rows: [to_bf16_tensor(b, "cuda") for b in rows]
    ys = L.rope.forward(_dev(pos), *put(x))
    dxs, dws = L.rope.backward(_dev(pos), put(dy), put(x))
    for i in range(4):
        _check_forward(L, i, x[i], pos, ys[i])
        _check_grad(L, i, O.bf16_to_f64(x[i]), O.bf16_to_f64(dy[i]), pos, dxs[i], dws[i])
    plain = np.flatnonzero(np.isin(np.arange(T) % 10, (0, 4)))
    alone = L.rope.forward(_dev(pos[plain]), *put([b[plain] for b in x]))
    grads, _ = L.rope.backward(_dev(pos[plain]), put([b[plain] for b in dy]), put([b[plain] for b in x]))
    at = _dev(plain).long()
    for a, b in zip((*alone, *grads), (*ys, *dxs)):
        assert torch.equal(a, b[at])


@pytest.mark.parametrize("kw", [dict(H=4), dict(H=3, adjacent=True, per_head=True, rotary=96)])
def test_codes_of_the_largest_rows(B, kw):
    """Half a million values: groups that fp32 does not tell are those of the exact value there too."""
    import torch
    L = Layer(B, seed=51, **kw)
    T = 1200
    pos = L.positions(T, 1 << 17)
    k, v = _large_rows(L.rng, (T, L.H, 128)), np.zeros((T, L.H, 128), np.uint16)
    c = B.make_cache_problem(num_requests=1, num_pages=T // 64 + 1, max_blocks=T // 64 + 1, num_q_heads=16 * L.H, topk=1,
                             token_cap=T, chunk_cap=1)
    cache, st = B.new_cache(c), torch.zeros(4, dtype=torch.int32, device="cuda")
    slots = L.rng.permutation(T).astype(np.int64)
    B.msa_cache_append_rope(c, _append_problem(B, L, T, False, False), None, to_bf16_tensor(k, "cuda"),
                            to_bf16_tensor(v, "cuda"), None, None, _dev(pos), _dev(slots, torch.int64), None, None,
                            None, None, cache, None, None, st)
    want = np.zeros(tuple(cache.shape), np.uint8)
    _expected_cache(L, want, k, v, pos, slots, 64)
    assert np.array_equal(cache.cpu().numpy(), want) and int(st[0].item()) == 0


@pytest.mark.parametrize("kw", [dict(), dict(adjacent=True, rotary=64, H=2)])
@pytest.mark.parametrize("exp", [-32, -9])
def test_codes_beyond_fp32(B, kw, exp):
    """Rows without a norm whose values, in units of 2^exp, leave fp32's range: their groups saturate."""
    import torch
    L = Layer(B, seed=52, norm=False, **kw)
    T = 60
    pos = L.positions(T)
    size = 2.0 ** np.array([0, 60, 90, 96, 100, 117, 119, 120, 122, 124])[np.arange(T) % 10]
    k, v = _bf16(L.rng, (T, L.H, 128), size[:, None, None]), np.zeros((T, L.H, 128), np.uint16)
    c = B.make_cache_problem(num_requests=1, num_pages=1, max_blocks=1, num_q_heads=16 * L.H, topk=1, token_cap=T,
                             chunk_cap=1, k_exp=exp)
    cache, st = B.new_cache(c), torch.zeros(4, dtype=torch.int32, device="cuda")
    slots = L.rng.permutation(T)
    B.msa_cache_append_rope(c, _append_problem(B, L, T, False, False), None, to_bf16_tensor(k, "cuda"),
                            to_bf16_tensor(v, "cuda"), None, None, _dev(pos), _dev(slots, torch.int64), None, None,
                            None, None, cache, None, None, st)
    want = np.zeros(tuple(cache.shape), np.uint8)
    _expected_cache(L, want, k, v, pos, slots, 64, (exp, 0))
    assert np.array_equal(cache.cpu().numpy(), want) and int(st[0].item()) == 0


def test_weight_of_another_type_at_the_same_address(B):
    """A weight whose data becomes bf16, one per head and fp32 again in the same memory: calls read, and write gradients,
    by what it is now."""
    import torch
    L = Layer(B, seed=53)
    T = 9
    pos = L.positions(T)
    x, dy = _bf16(L.rng, (T, 16, 128)), _bf16(L.rng, (T, 16, 128))
    buf = torch.zeros(16 * 128 * 4, dtype=torch.uint8, device="cuda")
    w = L.dev[0]
    for dtype, shape in ((torch.float32, (128,)), (torch.bfloat16, (128,)), (torch.float32, (16, 128)),
                         (torch.bfloat16, (16, 128)), (torch.float32, (128,))):
        w.data = buf.view(dtype)[:int(np.prod(shape))].view(shape)
        w.copy_(torch.from_numpy(L.rng.standard_normal(shape)))
        L.w[0] = _f64(w)
        _check_forward(L, 0, x, pos, L.rope.forward(_dev(pos), to_bf16_tensor(x, "cuda"))[0])
        (dx,), (dw,) = L.rope.backward(_dev(pos), [to_bf16_tensor(dy, "cuda")], [to_bf16_tensor(x, "cuda")])
        _check_grad(L, 0, O.bf16_to_f64(x), O.bf16_to_f64(dy), pos, dx, dw)


def test_gradients_of_inputs_with_common_elements(B):
    """One tensor as two inputs, and inputs that are parts of others: the bits of contiguous copies."""
    import torch
    L = Layer(B, seed=54, H=2, rotary=64)
    T = 300
    pos = _dev(L.positions(T))
    rows = to_bf16_tensor(_bf16(L.rng, (T, 34, 128)), "cuda")
    q, k = rows[:, :32], rows[:, 32:]
    dys = [to_bf16_tensor(_bf16(L.rng, (T, h, 128)), "cuda") for h in L.heads]
    for xs in ((q, k, k, k), (q, k, q[:, 4:6], q[:, 5:7]), (q, q[:, :2], k, q[:, 30:])):
        want = L.rope.backward(pos, dys, [x.contiguous() for x in xs])
        got = L.rope.backward(pos, dys, xs)
        assert all(torch.equal(a, b) for a, b in zip((*got[0], *got[1]), (*want[0], *want[1])))


def test_first_call_on_another_stream(B, monkeypatch):
    """What the constructor makes is there for every stream, whatever its own has still to do."""
    import torch
    x = _bf16(np.random.default_rng(55), (30, 16, 128))
    dev, pos, side = to_bf16_tensor(x, "cuda"), _dev(np.zeros(30)), torch.cuda.Stream()
    B.Rope(B.rope_frequencies(128), norm=False).forward(pos, dev * 0, stream=side)     # a kernel's first launch may wait
    busy = torch.zeros(1 << 28, device="cuda")
    left = [torch.full((4,), 5, dtype=torch.int32, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    del left
    pairs = B.rope_pairs

    def pairs_and_work(*args):
        table = pairs(*args)
        for _ in range(60):
            busy.add_(1.0)
        return table

    monkeypatch.setattr(B, "rope_pairs", pairs_and_work)
    rope = B.Rope(B.rope_frequencies(128), norm=False)
    y, = rope.forward(pos, dev, stream=side)
    side.synchronize()
    assert torch.equal(y, dev) and not torch.any(rope.status)      # position 0 turns nothing


def _nan_blocks(*shapes):
    """Fills memory that new tensors of these shapes are likely to get with NaN."""
    import torch
    left = [torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda") for s in shapes for _ in range(4)]
    torch.cuda.synchronize()
    del left


@pytest.mark.parametrize("kw", [dict(H=2), dict(adjacent=True, rotary=96, axes=2, norm=False)])
@pytest.mark.parametrize("T, gone", [(40, (0, 1, 5, 17, 30, 31, 38, 39)), (40, range(40)), (1100, range(3, 1100, 7)),
                                     (1, [0])])
def test_padding_of_new_tensors_is_zeros(B, kw, T, gone):
    """Without `out`: rows of padding, whatever the inputs hold there, are zeros in results and gradients, and the
    gradient of a projection before them is what the other rows give."""
    import torch
    L = Layer(B, seed=56, **kw)
    pos, gone = L.positions(T), np.array(gone)
    pos.reshape(T, -1)[gone, 0] = -1 - np.arange(len(gone))
    live = np.setdiff1d(np.arange(T), gone)
    n = sum(L.heads)
    rows, dy = _bf16(L.rng, (T, n, 128)), [_bf16(L.rng, (T, h, 128)) for h in L.heads]
    for b in (rows, *dy):
        b[gone] = 0x7FC0
    dev, dys = to_bf16_tensor(rows, "cuda"), [to_bf16_tensor(b, "cuda") for b in dy]
    at = np.concatenate([[0], np.cumsum(L.heads)])
    cut = [slice(a, b) for a, b in zip(at, at[1:])]
    for xs in ([dev[:, c] for c in cut], [dev[:, c].contiguous() for c in cut]):
        _nan_blocks((T, n, 128), *((T, h, 128) for h in L.heads))
        ys = L.rope.forward(_dev(pos), *xs)
        _nan_blocks((T, n, 128), *((T, h, 128) for h in L.heads))
        dxs, dws = L.rope.backward(_dev(pos), dys, xs)
        for i in range(4):
            assert not np.any(_f64(ys[i])[gone]) and not np.any(_f64(dxs[i])[gone])
            if len(live):
                x, g = rows[live][:, cut[i]], dy[i][live]
                _check_forward(L, i, x, pos[live], ys[i][_dev(live).long()])
                _check_grad(L, i, O.bf16_to_f64(x), O.bf16_to_f64(g), pos[live], dxs[i][_dev(live).long()], dws[i])
        hidden = torch.ones((T, 8), dtype=torch.bfloat16, device="cuda")
        hidden[_dev(gone).long()] = 0
        assert bool(torch.isfinite(hidden.T @ dxs[0].reshape(T, -1)).all())


def test_padding_of_an_append(B):
    """Token rows behind a step's last: zeros in new outputs, as they were in given ones."""
    import torch
    L = Layer(B, seed=57, H=2)
    T, n = 12, 7
    kv = B.Cache(num_requests=1, num_pages=4, max_blocks=2, num_q_heads=32, topk=2, max_tokens=T)
    x = [to_bf16_tensor(_bf16(L.rng, (T, h, 128)), "cuda") for h in (32, 2, 2, 2, 2)]
    for t in x:
        t[n:] = float("nan")
    kv.step(_dev([n]), T)
    _nan_blocks((T, 32, 128), (T, 2, 128))
    new = kv.append_rope(L.rope, *x)
    given = kv.append_rope(L.rope, *x, out=[torch.full((T, h, 128), 7.0, dtype=torch.bfloat16, device="cuda")
                                            for h in (32, 2)])
    for a, b in zip(new, given):
        assert torch.equal(a[:n], b[:n]) and not torch.any(a[n:]) and bool((b[n:] == 7.0).all())
    kv.check_status()


@pytest.mark.parametrize("axes", [1, 3])
def test_positions_that_begin_anywhere(B, axes):
    """Parts of longer position tensors, which begin between two borders of 16 bytes: the bits of copies; captured, the
    positions of the replay."""
    import torch
    L = Layer(B, seed=58, H=1, axes=axes)
    T, n = 20, 13
    pos = _dev(L.positions(T))
    x = [to_bf16_tensor(_bf16(L.rng, (n, h, 128)), "cuda") for h in L.heads]

    def run(p):
        kv = B.Cache(num_requests=1, num_pages=4, max_blocks=2, num_q_heads=16, topk=2, max_tokens=n)
        kv.step(_dev([n]), n)
        out = kv.append_rope(L.rope, x[0], x[1], x[1], x[2], x[3], positions=p)
        kv.check_status()
        return (*L.rope.forward(p, *x), *sum(L.rope.backward(p, x, x), ()), *out, kv.cache, kv.index_tail)

    for at in range(1, 5):
        part = pos[at:at + n]
        assert all(torch.equal(a, b) for a, b in zip(run(part), run(part.clone())))
    g, part = torch.cuda.CUDAGraph(), pos[1:1 + n]
    with torch.cuda.graph(g):
        y = L.rope.forward(part, *x)
    pos.copy_(_dev(L.positions(T)))
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(y, L.rope.forward(part.clone(), *x)))


@pytest.mark.parametrize("T", [0, 5])
@pytest.mark.parametrize("heads", [(0, 0, 0, 0), (16, 0, 1, 0), (0, 2, 0, 0)])
def test_weights_of_tensors_without_heads(B, T, heads):
    """A tensor of no heads, and calls of no tokens: the gradient of its weight is zeros."""
    import torch
    L = Layer(B, seed=59)
    pos = L.positions(T)
    x, dy = ([_bf16(L.rng, (T, h, 128)) for h in heads] for _ in range(2))
    put = lambda rows: [to_bf16_tensor(b, "cuda") for b in rows]
    left = [torch.full((128,), float("nan"), device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    del left
    dxs, dws = L.rope.backward(_dev(pos), put(dy), put(x))
    assert [tuple(d.shape) for d in dxs] == [(T, h, 128) for h in heads]
    for i, h in enumerate(heads):
        if T and h:
            _check_grad(L, i, O.bf16_to_f64(x[i]), O.bf16_to_f64(dy[i]), pos, dxs[i], dws[i])
        else:
            assert not torch.any(dws[i] != 0), i


@pytest.mark.parametrize("T", [1, 5, 400])
def test_a_bad_axis(B, T):
    """A pair's axis behind the positions' columns counts as the first and is reported; parts of the call that come up
    behind the report leave their rows as they were."""
    import torch
    L = Layer(B, seed=60)
    x, pos = to_bf16_tensor(_bf16(L.rng, (T, 1, 128)), "cuda"), _dev(L.positions(T))
    y, st = torch.full_like(x, 2.0), torch.zeros(4, dtype=torch.int32, device="cuda")
    p = B.make_rope_problem(T, B.rope_pairs(L.freq, [0, 2] * 32), k=B.RopeTensor(1, weight=L.dev[1]), eps=1e-6, num_axes=1)
    B.msa_norm_rope(p, [None, x, None, None], pos, [None, y, None, None], st)
    assert int(st[0].item()) == B.MSA_ERR_INVALID_ARGUMENT
    want = L.rope.forward(pos, None, x)[0]
    done, left = (y == want).all(-1), (y == 2.0).all(-1)
    assert bool((done | left).all()) and bool(done.any()) and (T > 1 or bool(done.all()))
