"""GPU: norm and rotary positions (msa_norm_rope), their gradients, and the 4-bit cache's append with both
(msa_cache_append_rope, Cache.append_rope) against the fp64 oracle.  Cache bytes and tables are compared bit for bit,
bf16 results within bounds derived from their roundings (``_forward_bound``, ``_grad_bound``)."""
import math

import numpy as np
import pytest

from oracle import cache_oracle as C
from oracle import msa_oracle as O
from oracle import rope_oracle as R
from tests._util import assert_grad_close, from_bf16_tensor, to_bf16_tensor
from tests.test_gpu_cache import Follow, Setup, _bf16, _close, _dev, _special_rows

pytestmark = pytest.mark.gpu

U = 2.0 ** -24          # half a step of fp32, relative
HALF = 2.0 ** -8        # half a step of bf16, relative
LEAST = 2.0 ** -134     # half a step of bf16's smallest values
EPS = 1e-6


@pytest.fixture(scope="module")
def B():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from block_sparse_top_attn_gb300 import binding
    return binding


def _f64(t):
    return t.detach().double().cpu().numpy()


class Layer:
    """One layer's rotation and weights, on the host in fp64 and as a Rope."""

    def __init__(self, B, seed=0, rotary=128, axes=1, adjacent=False, norm=True, per_head=False, wide=True, H=1,
                 offset=0.0, scale=1.0, base=1e4, index_norm=None, weights=True):
        import torch
        rng = self.rng = np.random.default_rng(seed)
        self.B, self.H, self.n, self.adjacent, self.offset, self.scale = B, H, rotary // 2, adjacent, offset, scale
        self.freq = base ** (-np.arange(self.n) / self.n)
        self.axis = None if axes == 1 else rng.integers(0, axes, self.n)
        if axes > 1:
            self.axis[:axes] = np.arange(axes)
        self.axes = axes
        self.heads = (16 * H, H, H, H)
        norms = (norm, norm, norm if index_norm is None else index_norm, norm if index_norm is None else index_norm)
        self.w, dev = [], []
        for h, on in zip(self.heads, norms):
            t = None
            if on and weights:
                t = torch.from_numpy(rng.standard_normal((h, 128) if per_head else 128) * 0.3 + 1 - offset)
                t = t.to(torch.float32 if wide else torch.bfloat16).cuda()
            dev.append(t)
            self.w.append(None if not on else 1.0 if t is None else _f64(t) + offset)
        self.dev = dev
        self.rope = B.Rope(self.freq, self.axis, *dev, norm=norms[0], index_norm=norms[2], adjacent=adjacent, eps=EPS,
                           weight_offset=offset, cos_scale=scale)

    def positions(self, T, most=5000):
        p = self.rng.integers(0, most, (T, self.axes))
        return p if self.axes > 1 else p[:, 0]

    def turns(self, pos):
        return R.turns(pos, self.freq, np.zeros(self.n, int) if self.axis is None else self.axis)

    def want(self, i, x, pos):
        return R.norm_rope(x, self.w[i], self.turns(pos), self.adjacent, EPS, self.scale)


def _amp(layer, n, turn):
    """|a cos| + |b sin| of every dim of normed rows n: what the rounding errors of a rotation are relative to."""
    a = np.abs(n)
    z = R._pairs(a, layer.n, layer.adjacent)
    c, s = np.abs(turn.real)[:, None] * layer.scale, np.abs(turn.imag)[:, None] * layer.scale
    return R._dims(a, (z.real * c + z.imag * s) + 1j * (z.imag * c + z.real * s), layer.adjacent)


def _forward_bound(layer, i, x, pos, want):
    """Half a step of bf16, and fp32's errors: 13.5 U for a normed value (the sum of 128 squares in chains of 8 and four
    more additions, halved by the root, with the division by 128 exact; rsqrtf 2 ulp; two products, the weight's
    offset), 5 U for a cosine (1 ulp, its argument's rounding, the scale), 2 U for the rotation: 32 U covers them."""
    n = R.norm_rope(x, layer.w[i], None, False, EPS)
    return HALF * np.abs(want) + (1 + HALF) * 32 * U * _amp(layer, n, layer.turns(pos)) + LEAST


def _check_forward(layer, i, x_bits, pos, got):
    x = O.bf16_to_f64(x_bits)
    want = layer.want(i, x, pos)
    off = np.abs(_f64(got) - want)
    assert np.all(off <= _forward_bound(layer, i, x, pos, want)), np.nanmax(off)


def _grad_bound(layer, i, x, dy, pos, want):
    """dx = r (u - x r mean(u x r)), u = w g.  g is off by 8 U of its amplitude (two products, the sum, the cosine's 5 U),
    u by two more, r by 11 U, x r by 12 U; the mean of 128 products by 12 + 10 + 21 additions' worth; the rest are a few
    products: 128 U covers each term."""
    n = np.sqrt((x * x).mean(-1, keepdims=True) + EPS) if layer.w[i] is not None else 1.0
    w = np.abs(layer.w[i]) if layer.w[i] is not None else 1.0
    u = _amp(layer, dy, layer.turns(pos)) * w
    term = u
    if layer.w[i] is not None:
        term = u + np.abs(x / n) * (u * np.abs(x / n)).mean(-1, keepdims=True)
    return HALF * np.abs(want) + (1 + HALF) * 128 * U * term / n + LEAST


CASES = [dict(), dict(rotary=64), dict(rotary=32, adjacent=True), dict(rotary=96, per_head=True, wide=False),
         dict(adjacent=True, axes=3, H=2), dict(axes=4, rotary=64, per_head=True, H=3), dict(norm=False),
         dict(norm=False, adjacent=True, rotary=96, scale=0.75), dict(wide=False, offset=1.0, scale=1.2, H=2),
         dict(index_norm=False, H=5, axes=2, per_head=True), dict(weights=False, offset=1.0)]


@pytest.mark.parametrize("kw", CASES)
@pytest.mark.parametrize("T", [1, 2, 7, 50, 301])
def test_forward(B, kw, T):
    """Every layout, weight and axis choice, from one token on; the four tensors of a call together."""
    L = Layer(B, seed=T, **kw)
    pos = L.positions(T)
    x = [_bf16(L.rng, (T, h, 128), np.exp(L.rng.standard_normal((T, 1, 1)))) for h in L.heads]
    ys = L.rope.forward(_dev(pos), *(to_bf16_tensor(b, "cuda") for b in x))
    assert len(ys) == 4
    for i, y in enumerate(ys):
        _check_forward(L, i, x[i], pos, y)


@pytest.mark.parametrize("kw", CASES)
@pytest.mark.parametrize("T", [1, 2, 7, 50, 301])
def test_backward(B, kw, T):
    L = Layer(B, seed=100 + T, **kw)
    pos = L.positions(T)
    x = [_bf16(L.rng, (T, h, 128), np.exp(L.rng.standard_normal((T, 1, 1)))) for h in L.heads]
    dy = [_bf16(L.rng, (T, h, 128)) for h in L.heads]
    dxs, dws = L.rope.backward(_dev(pos), [to_bf16_tensor(b, "cuda") for b in dy],
                               [to_bf16_tensor(b, "cuda") for b in x])
    for i in range(4):
        _check_grad(L, i, O.bf16_to_f64(x[i]), O.bf16_to_f64(dy[i]), pos, dxs[i], dws[i])


def _check_grad(L, i, x, dy, pos, dx, dw):
    want, rows = R.norm_rope_grad(x, L.w[i], dy, L.turns(pos), L.adjacent, EPS, L.scale)
    off = np.abs(_f64(dx) - want)
    assert np.all(off <= _grad_bound(L, i, x, dy, pos, want)), off.max()
    assert (dw is None) == (L.dev[i] is None)
    if dw is None:
        return
    assert dw.dtype == L.dev[i].dtype and dw.shape == L.dev[i].shape
    # a sum of N products, each off by 24 U of its amplitude, in fp32: at most N additions' worth more
    xr = np.abs(x) / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
    size = _amp(L, dy, L.turns(pos)) * xr
    sum_over = 0 if dw.dim() == 2 else (0, 1)
    n = size.shape[0] * (1 if dw.dim() == 2 else size.shape[1])
    want = rows.sum(sum_over)
    bound = (24 + n) * U * size.sum(sum_over) * (1 + HALF)
    bound = bound + ((HALF * np.abs(want) + LEAST) if dw.dtype.itemsize == 2 else U * np.abs(want) + 2.0 ** -149)
    assert np.all(np.abs(_f64(dw) - want) <= bound), np.abs(_f64(dw) - want).max()


def test_gradient_against_differences(B):
    """The returned gradients against differences of the definition, along random directions."""
    L = Layer(B, seed=9, H=1, rotary=64, axes=2)
    T = 20
    pos = L.positions(T)
    x, dy = _bf16(L.rng, (T, 16, 128)), _bf16(L.rng, (T, 16, 128))
    (dx,), (dw,) = L.rope.backward(_dev(pos), [to_bf16_tensor(dy, "cuda")], [to_bf16_tensor(x, "cuda")])
    x, dy, dx, dw = O.bf16_to_f64(x), O.bf16_to_f64(dy), _f64(dx), _f64(dw)
    t = L.turns(pos)
    f = lambda x, w: float((dy * R.norm_rope(x, w, t, False, EPS)).sum())
    h = 1e-5
    for _ in range(4):
        v = L.rng.standard_normal(x.shape)
        diff = (f(x + h * v, L.w[0]) - f(x - h * v, L.w[0])) / (2 * h)
        bound = (_grad_bound(L, 0, x, dy, pos, dx) * 1.01 * np.abs(v)).sum()
        assert abs((dx * v).sum() - diff) <= bound + 1e-5
        v = L.rng.standard_normal(128)
        diff = (f(x, L.w[0] + h * v) - f(x, L.w[0] - h * v)) / (2 * h)
        size = (_amp(L, dy, t) * np.abs(x) / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)).sum((0, 1))
        assert abs((dw * v).sum() - diff) <= (345 * U * size * np.abs(v)).sum() + 1e-5


@pytest.mark.parametrize("heads", [(1, 0, 0, 0), (0, 3, 0, 0), (0, 0, 5, 1), (40, 1, 0, 2), (7, 9, 2, 30), (133, 1, 1, 1)])
@pytest.mark.parametrize("per_head", [False, True])
def test_any_heads(B, heads, per_head):
    """Head counts that straddle warps and CTAs, tensors that are not there; the gradients' partial sums with them."""
    import torch
    rng = np.random.default_rng(sum(heads))
    T = 70
    L = Layer(B, seed=3, H=1)
    L.w, L.dev = [], []
    for h in heads:
        w = torch.from_numpy(rng.standard_normal((h, 128) if per_head else 128)).float().cuda()
        L.dev.append(w)
        L.w.append(_f64(w))
    L.rope = B.Rope(L.freq, None, *L.dev, eps=EPS)
    pos = L.positions(T)
    x = [_bf16(rng, (T, h, 128)) for h in heads]
    dy = [_bf16(rng, (T, h, 128)) for h in heads]
    put = lambda bits: [to_bf16_tensor(b, "cuda") if b.shape[1] else None for b in bits]
    ys = iter(L.rope.forward(_dev(pos), *put(x)))
    dxs, dws = L.rope.backward(_dev(pos), put(dy), put(x))
    for i in range(4):
        if heads[i]:
            _check_forward(L, i, x[i], pos, next(ys))
            _check_grad(L, i, O.bf16_to_f64(x[i]), O.bf16_to_f64(dy[i]), pos, dxs[i], dws[i])
        else:
            assert dxs[i] is None and dws[i] is None


def test_far_positions(B):
    """Angles at positions up to 2^31 - 1, where a 32-bit product would have lost them, and negative ones in columns
    behind the first."""
    L = Layer(B, seed=4, axes=2, rotary=64, base=3.0)
    pos = np.array([[2 ** 31 - 1, -2 ** 31], [2 ** 31 - 1, 2 ** 31 - 1], [1234567891, -987654321], [0, -1],
                    [16777217, 16777219], [2 ** 30, -2 ** 30]])
    x = _bf16(L.rng, (6, 1, 128))
    (y,) = L.rope.forward(_dev(pos), None, to_bf16_tensor(x, "cuda"))
    # the oracle's angle, an fp64 product of up to 2^31, is off by 2^-22 of a radian: as many U of the amplitude as 4
    xs = O.bf16_to_f64(x)
    want = L.want(1, xs, pos)
    bound = _forward_bound(L, 1, xs, pos, want) + 8 * U * np.abs(R.norm_rope(xs, L.w[1], None, False, EPS)).max()
    assert np.all(np.abs(_f64(y) - want) <= bound)


def test_magnitudes(B):
    """Rows of zeros, of values whose squares leave fp32's range above and below, and their gradients."""
    L = Layer(B, seed=5)
    T = 9
    scale = 2.0 ** np.array([0, -140, -100, -70, -40, 40, 64, 100, 120])[:, None, None]
    x = O.f64_to_bf16(L.rng.standard_normal((T, 16, 128)) * scale)
    x[0] = 0
    dy = O.f64_to_bf16(L.rng.standard_normal((T, 16, 128)))
    pos = L.positions(T)
    (y,) = L.rope.forward(_dev(pos), to_bf16_tensor(x, "cuda"))
    _check_forward(L, 0, x, pos, y)
    assert not np.any(_f64(y)[0])
    (dx,), (dw,) = L.rope.backward(_dev(pos), [to_bf16_tensor(dy, "cuda")], [to_bf16_tensor(x, "cuda")])
    _check_grad(L, 0, O.bf16_to_f64(x), O.bf16_to_f64(dy), pos, dx, dw)


def test_values_that_are_not_finite_stay_in_their_rows(B):
    import torch
    L = Layer(B, seed=6, H=1)
    T = 12
    x = _bf16(L.rng, (T, 16, 128))
    dirty = x.copy()
    dirty[3, 5, 7], dirty[4, 2, 100], dirty[5, 9, 64] = 0x7F80, 0x7FC0, 0xFF80
    pos = _dev(L.positions(T))
    a, = L.rope.forward(pos, to_bf16_tensor(x, "cuda"))
    b, = L.rope.forward(pos, to_bf16_tensor(dirty, "cuda"))
    same = torch.ones((T, 16), dtype=torch.bool, device="cuda")
    for t, h in ((3, 5), (4, 2), (5, 9)):
        assert torch.isnan(b[t, h].float()).any()
        same[t, h] = False
    assert torch.equal(a[same], b[same]) and torch.isnan(b[4, 2].float()).all()


def test_padding_is_left_as_it_was(B):
    """Rows with a negative first position, whatever they hold: outputs keep what was there, the weights' gradients do
    not see them."""
    import torch
    L = Layer(B, seed=7, H=2, axes=2, per_head=True)
    T = 40
    pos = L.positions(T)
    gone = np.array([0, 1, 5, 17, 30, 31, 38, 39])
    pos[gone, 0] = -1 - np.arange(len(gone))
    live = np.setdiff1d(np.arange(T), gone)
    x = [_bf16(L.rng, (T, h, 128)) for h in L.heads]
    dy = [_bf16(L.rng, (T, h, 128)) for h in L.heads]
    for b in (*x, *dy):
        b[gone] = 0x7FC0
    put = lambda bits: [to_bf16_tensor(b, "cuda") for b in bits]
    fill = lambda: [torch.full((T, h, 128), 7.0, dtype=torch.bfloat16, device="cuda") for h in L.heads]
    ys = L.rope.forward(_dev(pos), *put(x), out=fill())
    dxs, dws = L.rope.backward(_dev(pos), put(dy), put(x), out=fill())
    for i in range(4):
        assert np.all(_f64(ys[i])[gone] == 7.0) and np.all(_f64(dxs[i])[gone] == 7.0)
        _check_forward(L, i, x[i][live], pos[live], ys[i][_dev(live).long()])
        _check_grad(L, i, O.bf16_to_f64(x[i][live]), O.bf16_to_f64(dy[i][live]), pos[live], dxs[i][_dev(live).long()],
                    dws[i])
    # nothing but padding
    pos[:, 0] = -1
    _, dws = L.rope.backward(_dev(pos), put(dy), put(x))
    assert all(not torch.any(dw) for dw in dws)


def test_views_in_place_and_order_of_dims(B):
    """Inputs as parts of one projection's output, outputs in place, and head-major rows: the same bits as contiguous
    tensors; nothing around the rows is touched.  The gradients likewise, into the projection's gradient."""
    import torch
    L = Layer(B, seed=8, H=2, rotary=96)
    T, n = 33, sum((32, 2, 2, 2, 2))
    pos = _dev(L.positions(T))
    rows = to_bf16_tensor(_bf16(L.rng, (T, n, 128)), "cuda")
    cut = lambda x: (x[:, :32], x[:, 32:34], x[:, 36:38], x[:, 38:40])      # V lies between
    xs = cut(rows)
    want = L.rope.forward(pos, *(x.contiguous() for x in xs))
    for a, b in zip(L.rope.forward(pos, *xs), want):
        assert torch.equal(a, b)
    by_head = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in xs]
    for a, b in zip(L.rope.forward(pos, *by_head, out=[x.transpose(0, 1).contiguous().transpose(0, 1) for x in want]), want):
        assert torch.equal(a, b)
    dys = [to_bf16_tensor(_bf16(L.rng, (T, h, 128)), "cuda") for h in L.heads]
    dxw, dww = L.rope.backward(pos, dys, [x.contiguous() for x in xs])
    grad = torch.full_like(rows, 5.0)
    dxs, dws = L.rope.backward(pos, dys, xs, out=cut(grad))
    for a, b in zip((*dxs, *dws), (*dxw, *dww)):
        assert torch.equal(a, b)
    assert bool((grad[:, 34:36] == 5.0).all())
    dxs, _ = L.rope.backward(pos, dys, xs)      # new tensors, laid out as the inputs are, of one buffer
    assert all(torch.equal(a, b) and a.stride() == x.stride() for a, b, x in zip(dxs, dxw, xs))
    assert len({d.untyped_storage().data_ptr() for d in dxs}) == 1
    # in place: dx over dy, y over x
    over = [d.clone() for d in dys]
    dxs, dws = L.rope.backward(pos, over, [x.contiguous() for x in xs], out=over)
    for a, b in zip((*over, *dws), (*dxw, *dww)):
        assert torch.equal(a, b)
    # dx over x itself
    over = [x.contiguous() for x in xs]
    dxs, dws = L.rope.backward(pos, dys, over, out=over)
    for a, b in zip((*over, *dws), (*dxw, *dww)):
        assert torch.equal(a, b)
    v = rows[:, 34:36].clone()
    ys = L.rope.forward(pos, *xs, out=xs)
    for a, b, c in zip(ys, cut(rows), want):
        assert torch.equal(a, c) and torch.equal(b, c)
    assert torch.equal(rows[:, 34:36], v)


def test_rows_do_not_depend_on_the_call(B):
    """A row's result is the same bits alone, in any batch, with any other tensors; sums of gradients repeat bit for
    bit."""
    import torch
    L = Layer(B, seed=10, H=2)
    T = 600
    pos = L.positions(T)
    x = [to_bf16_tensor(_bf16(L.rng, (T, h, 128)), "cuda") for h in L.heads]
    dy = [to_bf16_tensor(_bf16(L.rng, (T, h, 128)), "cuda") for h in L.heads]
    ys = L.rope.forward(_dev(pos), *x)
    dxs, dws = L.rope.backward(_dev(pos), dy, x)
    for lo, hi in ((0, 1), (13, 14), (100, 107), (590, 600)):
        part = L.rope.forward(_dev(pos[lo:hi]), *(t[lo:hi] for t in x))
        grad, _ = L.rope.backward(_dev(pos[lo:hi]), [t[lo:hi] for t in dy], [t[lo:hi] for t in x])
        for a, b, c, d in zip(part, ys, grad, dxs):
            assert torch.equal(a, b[lo:hi]) and torch.equal(c, d[lo:hi])
    assert torch.equal(L.rope.forward(_dev(pos), None, x[1])[0], ys[1])
    for _ in range(3):
        again = L.rope.backward(_dev(pos), dy, x)
        assert all(torch.equal(a, b) for a, b in zip((*again[0], *again[1]), (*dxs, *dws)))


def test_rows_far_apart(B):
    """Rows whose offsets pass 32 bits, in elements and in bytes."""
    import torch
    L = Layer(B, seed=29)
    T, far = 4, (1 << 30) + 8
    buf = torch.empty((T - 1) * far + 16 * 128, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((T, 16, 128), (far, 128, 1))
    bits = _bf16(L.rng, (T, 16, 128))
    x.copy_(to_bf16_tensor(bits, "cuda"))
    pos = L.positions(T)
    want, = L.rope.forward(_dev(pos), to_bf16_tensor(bits, "cuda"))
    dy = to_bf16_tensor(_bf16(L.rng, (T, 16, 128)), "cuda")
    (dxw,), (dww,) = L.rope.backward(_dev(pos), [dy], [to_bf16_tensor(bits, "cuda")])
    (dx,), (dw,) = L.rope.backward(_dev(pos), [dy], [x], out=[x])
    assert torch.equal(dx, dxw) and torch.equal(dw, dww)
    x.copy_(to_bf16_tensor(bits, "cuda"))
    got, = L.rope.forward(_dev(pos), x, out=[x])
    _check_forward(L, 0, bits, pos, want)
    assert torch.equal(got, want)


def test_replaced_weights(B):
    """A weight whose storage was replaced, and one that was changed in place: calls use what is there now."""
    import torch
    L = Layer(B, seed=28)
    pos = L.positions(9)
    x = _bf16(L.rng, (9, 16, 128))
    for change in (lambda w: w.copy_(w * 2 + 1), lambda w: setattr(w, "data", w.clone() * 0.5)):
        L.rope.forward(_dev(pos), to_bf16_tensor(x, "cuda"))
        change(L.dev[0])
        L.w[0] = _f64(L.dev[0])
        _check_forward(L, 0, x, pos, L.rope.forward(_dev(pos), to_bf16_tensor(x, "cuda"))[0])


def test_no_tokens(B):
    import torch
    L = Layer(B, seed=11, H=1, wide=False)
    z = [torch.zeros((0, h, 128), dtype=torch.bfloat16, device="cuda") for h in L.heads]
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert [y.shape[0] for y in L.rope.forward(pos, *z)] == [0] * 4
    dxs, dws = L.rope.backward(pos, z, z)
    assert [d.shape[0] for d in dxs] == [0] * 4 and all(not torch.any(w) for w in dws)
    # and through the C call
    p = B.make_rope_problem(0, L.rope.pairs, k=B.RopeTensor(1, weight=L.dev[1]))
    dw = torch.full((128,), 3.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    none = [None, z[1], None, None]
    B.msa_norm_rope(p, none, pos, none, st)
    B.msa_norm_rope_bwd(p, none, none, pos, none, [None, dw, None, None], st,
                        torch.empty(B.msa_norm_rope_bwd_bytes(p), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert not torch.any(dw) and int(st[0].item()) == 0


def test_an_earlier_error_and_a_bad_axis(B):
    """A status that is set: nothing is written.  A pair's axis behind the positions' columns is reported and counts
    as the first."""
    import torch
    L = Layer(B, seed=12)
    x = to_bf16_tensor(_bf16(L.rng, (5, 1, 128)), "cuda")
    pos = _dev(L.positions(5))
    p = B.make_rope_problem(5, L.rope.pairs, k=B.RopeTensor(1, weight=L.dev[1]), eps=EPS)
    four = lambda t: [None, t, None, None]
    ws = torch.empty(B.msa_norm_rope_bwd_bytes(p), dtype=torch.uint8, device="cuda")
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    st[0] = 7
    y, dw = torch.full_like(x, 2.0), torch.full((128,), 2.0, device="cuda")
    B.msa_norm_rope(p, four(x), pos, four(y), st)
    B.msa_norm_rope_bwd(p, four(x), four(x), pos, four(y), four(dw), st, ws)
    torch.cuda.synchronize()
    assert int(st[0].item()) == 7 and bool((y == 2.0).all()) and bool((dw == 2.0).all())
    st.zero_()
    bad = B.rope_pairs(L.freq, [0, 2] * 32)
    p = B.make_rope_problem(5, bad, k=B.RopeTensor(1, weight=L.dev[1]), eps=EPS, num_axes=1)
    B.msa_norm_rope(p, four(x), pos, four(y), st)
    torch.cuda.synchronize()
    assert int(st[0].item()) == B.MSA_ERR_INVALID_ARGUMENT
    assert torch.equal(y, L.rope.forward(pos, None, x)[0])


def test_more_columns_than_the_pairs_use(B):
    import torch
    L = Layer(B, seed=13)
    x = to_bf16_tensor(_bf16(L.rng, (6, 1, 128)), "cuda")
    pos = L.positions(6)
    wide = np.stack([pos, pos + 5, pos * 0 - 3], 1)
    p = B.make_rope_problem(6, L.rope.pairs, k=B.RopeTensor(1, weight=L.dev[1]), eps=EPS, num_axes=3)
    y, st = torch.empty_like(x), torch.zeros(4, dtype=torch.int32, device="cuda")
    B.msa_norm_rope(p, [None, x, None, None], _dev(wide), [None, y, None, None], st)
    assert torch.equal(y, L.rope.forward(_dev(pos), None, x)[0]) and int(st[0].item()) == 0


def test_norm_alone(B):
    """Tensors that are only normed beside ones that are rotated, and a call that rotates nothing."""
    import torch
    L = Layer(B, seed=14, H=1, rotary=64)
    T = 21
    pos = _dev(L.positions(T))
    x = [_bf16(L.rng, (T, h, 128)) for h in L.heads]
    xs = [to_bf16_tensor(b, "cuda") for b in x]
    ts = [B.RopeTensor(h, rotate=i % 2 == 0, weight=w) for i, (h, w) in enumerate(zip(L.heads, L.dev))]
    still = [B.RopeTensor(h, rotate=False, weight=w) for h, w in zip(L.heads, L.dev)]
    turned = L.rope.forward(pos, *xs)
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    for pairs, tensors in ((L.rope.pairs, ts), (None, still)):
        p = B.make_rope_problem(T, pairs, *tensors, eps=EPS)
        ys = [torch.empty_like(t) for t in xs]
        B.msa_norm_rope(p, xs, pos, ys, st)
        dxs, dws = [torch.empty_like(t) for t in xs], [torch.empty_like(w) for w in L.dev]
        B.msa_norm_rope_bwd(p, xs, xs, pos, dxs, dws, st,
                            torch.empty(B.msa_norm_rope_bwd_bytes(p), dtype=torch.uint8, device="cuda"))
        for i, t in enumerate(tensors):
            if t.flags & B.MSA_ROPE_ROTATE:
                assert torch.equal(ys[i], turned[i])
                continue
            v = O.bf16_to_f64(x[i])
            want = R.norm_rope(v, L.w[i], None, False, EPS)
            assert np.all(np.abs(_f64(ys[i]) - want) <= (HALF + 32 * U) * np.abs(want) + LEAST)
            gx, gw = R.norm_rope_grad(v, L.w[i], v, None, False, EPS)
            n = np.sqrt((v * v).mean(-1, keepdims=True) + EPS)
            u = np.abs(v) * np.abs(L.w[i])
            term = (u + np.abs(v / n) * (u * np.abs(v / n)).mean(-1, keepdims=True)) / n
            assert np.all(np.abs(_f64(dxs[i]) - gx) <= HALF * np.abs(gx) + 129 * U * term + LEAST)
            rows = np.abs(v * v / n).sum((0, 1))
            assert np.all(np.abs(_f64(dws[i]) - gw.sum((0, 1))) <= (25 + T * L.heads[i]) * U * rows)
    assert int(st[0].item()) == 0


# ---------------------------------------------------------------------------
# streams, graphs
# ---------------------------------------------------------------------------

def test_captured_and_replayed(B):
    """Forward and backward captured into two graphs of one Rope, replayed in turn and side by side on two streams with
    new inputs."""
    import torch
    L = Layer(B, seed=15, H=2, per_head=True)
    made = []
    for T in (64, 150):
        bufs = dict(x=[torch.zeros((T, h, 128), dtype=torch.bfloat16, device="cuda") for h in L.heads],
                    dy=[torch.zeros((T, h, 128), dtype=torch.bfloat16, device="cuda") for h in L.heads],
                    pos=torch.zeros(T, dtype=torch.int32, device="cuda"))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            L.rope.forward(bufs["pos"], *bufs["x"])
            L.rope.backward(bufs["pos"], bufs["dy"], bufs["x"])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = (*L.rope.forward(bufs["pos"], *bufs["x"]), *sum(L.rope.backward(bufs["pos"], bufs["dy"], bufs["x"]), ()))
        made.append((T, bufs, side, g, out))
    for turn in range(3):
        want = []
        for T, bufs, side, g, out in made:
            bufs["pos"].copy_(_dev(L.positions(T)))
            for name in ("x", "dy"):
                for t, h in zip(bufs[name], L.heads):
                    t.copy_(to_bf16_tensor(_bf16(L.rng, (T, h, 128)), "cuda"))
            want.append((*L.rope.forward(bufs["pos"], *bufs["x"]),
                         *sum(L.rope.backward(bufs["pos"], bufs["dy"], bufs["x"]), ())))
        torch.cuda.synchronize()
        for _ in range(3):
            for T, bufs, side, g, out in made:
                with torch.cuda.stream(side):
                    g.replay()
        torch.cuda.synchronize()
        for (T, bufs, side, g, out), w in zip(made, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))


@pytest.mark.parametrize("call", ["forward", "backward"])
def test_on_a_side_stream(B, call):
    """A call given a stream is that stream's alone, its outputs and workspace among it."""
    import torch
    L = Layer(B, seed=16, H=2)
    T = 500
    pos = _dev(L.positions(T))
    x = [to_bf16_tensor(_bf16(L.rng, (T, h, 128)), "cuda") for h in L.heads]
    run = {"forward": lambda s: L.rope.forward(pos, *x, stream=s),
           "backward": lambda s: sum(L.rope.backward(pos, x, x, stream=s), ())}[call]
    want = run(None)
    side = torch.cuda.Stream()
    run(side)
    torch.cuda.synchronize()
    left = [torch.full((4,), 5, dtype=torch.int32, device="cuda") for _ in range(64)]
    busy = torch.zeros(1 << 28, device="cuda")
    torch.cuda.synchronize()
    del left
    for _ in range(60):
        busy.add_(1.0)
    got = run(side)
    side.synchronize()
    with torch.cuda.stream(side):
        early = [t.clone() for t in got]
    torch.cuda.synchronize()
    for a, b, c in zip(got, early, want):
        assert torch.equal(a, c) and torch.equal(b, c)


def test_from_several_threads(B):
    """One Rope, four host threads with streams and sizes of their own."""
    import threading

    import torch
    L = Layer(B, seed=17, H=1)
    jobs = []
    for T in (3, 40, 200, 1000):
        pos = _dev(L.positions(T))
        x = [to_bf16_tensor(_bf16(L.rng, (T, h, 128)), "cuda") for h in L.heads]
        jobs.append((pos, x, (*L.rope.forward(pos, *x), *sum(L.rope.backward(pos, x, x), ()))))
    torch.cuda.synchronize()
    bad = []

    def work(pos, x, want):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                got = (*L.rope.forward(pos, *x, stream=s), *sum(L.rope.backward(pos, x, x, stream=s), ()))
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want)):
                bad.append("differs")
        except Exception as e:  # a thread's exception would be lost
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


# ---------------------------------------------------------------------------
# the cache's append
# ---------------------------------------------------------------------------

def _expected_cache(L, cache, k_bits, v_bits, pos, slots, block, exps=(0, 0)):
    """The cache's bytes after the rows, from the definition in fp64."""
    k = O.bf16_to_f64(k_bits)
    with np.errstate(all="ignore"):
        kc, ks = R.round_values(L.want(1, k, pos), exps[0])
    vc, vs, _ = C.round_rows(v_bits, exps[1])
    for t, slot in enumerate(slots):
        if slot >= 0:
            for h in range(k.shape[1]):
                C.write_row(cache, slot, h, block, kc[t, h], ks[t, h], vc[t, h], vs[t, h])
    return ks, vs


def _without_codes_of_nan(caches, ks, vs, slots, block):
    """The codes of a group whose scale is NaN mean nothing."""
    for t in np.flatnonzero((ks == 0x7F).any((1, 2)) | (vs == 0x7F).any((1, 2))):
        if slots[t] < 0:
            continue
        page, off = divmod(int(slots[t]), block)
        for x in caches:
            b, i = x[page, :, off // 64], off % 64
            b[:, i * 64:i * 64 + 64] = 0
            b[:, 4608 + ((i * 64 + np.arange(64)) ^ ((i & 12) << 3))] = 0


def _append_problem(B, L, T, index=True, q=True, strides=None, **kw):
    dev = L.dev
    strides = strides or [None] * 5
    norms = [w is not None for w in L.w]
    t = [B.RopeTensor(h, norm=n, weight=w, x_strides=s) for h, n, w, s in zip(L.heads, norms, dev, strides)]
    v = B.RopeTensor(L.H, norm=False, rotate=False, x_strides=strides[4])
    return B.make_rope_problem(T, L.rope.pairs, t[0] if q else None, t[1], t[2] if q and index else None,
                               t[3] if index else None, v, adjacent=L.adjacent, eps=EPS, weight_offset=L.offset,
                               cos_scale=L.scale, **kw)


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("exp", [(0, 0), (-6, 3), (32, -32)])
@pytest.mark.parametrize("kw", [dict(), dict(adjacent=True, rotary=64, H=3, per_head=True, wide=False),
                                dict(norm=False, axes=3, rotary=96), dict(norm=False, adjacent=True, H=2),
                                dict(offset=1.0, scale=1.3, H=9, rotary=32), dict(weights=False, axes=2, H=2)])
def test_append_bytes(B, kw, exp, block):
    """Every byte of the cache, with special rows, rows of slot -1 and of negative positions; without index keys."""
    import torch
    L = Layer(B, seed=18, **kw)
    H, P, T = L.H, 6, 77
    rng = L.rng
    slots = rng.permutation(P * block)[:T].astype(np.int64)
    slots[[10, 40]] = -1
    pos = L.positions(T)
    pos[::9] = 0            # nothing turned: exact ties where there is no norm
    k, v = (_special_rows(rng, _bf16(rng, (T, H, 128), 2.0 ** e)) for e in exp)
    c = B.make_cache_problem(num_requests=1, num_pages=P, max_blocks=P, num_q_heads=16 * H, topk=1, token_cap=T,
                             chunk_cap=1, block_size=block, k_exp=exp[0], v_exp=exp[1])
    cache = B.new_cache(c)
    cache.fill_(0xA5)
    want = cache.cpu().numpy()
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    B.msa_cache_append_rope(c, _append_problem(B, L, T, False, False), None, to_bf16_tensor(k, "cuda"),
                            to_bf16_tensor(v, "cuda"), None, None, _dev(pos), _dev(slots, torch.int64), None, None,
                            None, None, cache, None, None, st)
    ks, vs = _expected_cache(L, want, k, v, pos, slots, block, exp)
    got = cache.cpu().numpy()
    assert int(st[0].item()) == 0
    _without_codes_of_nan((got, want), ks, vs, slots, block)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("block", [64, 128])
def test_append_of_rows_as_they_are(B, block):
    """K that is neither normed nor rotated: msa_cache_append's bytes, special rows and exact ties among them."""
    import torch
    L = Layer(B, seed=27, H=3)
    rng, P, T = L.rng, 4, 90
    k, v = (_special_rows(rng, _bf16(rng, (T, 3, 128))) for _ in range(2))
    k, v = to_bf16_tensor(k, "cuda"), to_bf16_tensor(v, "cuda")
    slots = _dev(rng.permutation(P * block)[:T], torch.int64)
    c = B.make_cache_problem(num_requests=1, num_pages=P, max_blocks=P, num_q_heads=48, topk=1, token_cap=T, chunk_cap=1,
                             block_size=block)
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    want, got = B.new_cache(c), B.new_cache(c)
    B.msa_cache_append(c, k, v, None, slots, None, None, want, None, None, st)
    still = B.RopeTensor(3, norm=False, rotate=False)
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    for pairs in (None, L.rope.pairs):
        got.zero_()
        p = B.make_rope_problem(T, pairs, k=still, v=still)
        B.msa_cache_append_rope(c, p, None, k, v, None, None, pos, slots, None, None, None, None, got, None, None, st)
        assert torch.equal(got, want) and int(st[0].item()) == 0


@pytest.mark.parametrize("kw", [dict(H=4), dict(H=4, adjacent=True, norm=False, axes=3)])
def test_codes_of_many_values(B, kw):
    """Two million values: dozens of them lie closer to a border than fp32 tells."""
    import torch
    L = Layer(B, seed=19, base=5e6, **kw)
    T = 4096
    pos = L.positions(T, 1 << 20)
    k, v = (_bf16(L.rng, (T, L.H, 128), np.exp(0.5 * L.rng.standard_normal((1, L.H, 128)))) for _ in range(2))
    c = B.make_cache_problem(num_requests=1, num_pages=T // 64, max_blocks=T // 64, num_q_heads=16 * L.H, topk=1,
                             token_cap=T, chunk_cap=1)
    cache, st = B.new_cache(c), torch.zeros(4, dtype=torch.int32, device="cuda")
    slots = L.rng.permutation(T).astype(np.int64)
    B.msa_cache_append_rope(c, _append_problem(B, L, T, False, False), None, to_bf16_tensor(k, "cuda"),
                            to_bf16_tensor(v, "cuda"), None, None, _dev(pos), _dev(slots, torch.int64), None, None,
                            None, None, cache, None, None, st)
    want = np.zeros(tuple(cache.shape), np.uint8)
    _expected_cache(L, want, k, v, pos, slots, 64)
    assert np.array_equal(cache.cpu().numpy(), want) and int(st[0].item()) == 0


@pytest.mark.parametrize("kw", [dict(H=4), dict(H=3, adjacent=True, per_head=True, rotary=96)])
@pytest.mark.parametrize("exp", [-32, 0, 9])
def test_codes_of_rows_of_all_sizes(B, kw, exp):
    """A million values of rows from 2^-12 to 2^119, whose squares leave fp32's range in a third of them: groups that
    fp32 does not tell are those of the exact value there too."""
    import torch
    L = Layer(B, seed=44, base=1e4, **kw)
    T = 3000
    pos = L.positions(T, 1 << 17)
    size = 2.0 ** np.array([-12, -3, 0, 40, 59, 61, 64, 90, 119])[np.arange(T) % 9]
    k, v = (_bf16(L.rng, (T, L.H, 128), size[:, None, None]) for _ in range(2))
    v = np.where(size[:, None, None] < 1e9, v, 0).astype(v.dtype)
    c = B.make_cache_problem(num_requests=1, num_pages=T // 64 + 1, max_blocks=T // 64 + 1, num_q_heads=16 * L.H, topk=1,
                             token_cap=T, chunk_cap=1, k_exp=exp, v_exp=0)
    cache, st = B.new_cache(c), torch.zeros(4, dtype=torch.int32, device="cuda")
    slots = L.rng.permutation(T).astype(np.int64)
    B.msa_cache_append_rope(c, _append_problem(B, L, T, False, False), None, to_bf16_tensor(k, "cuda"),
                            to_bf16_tensor(v, "cuda"), None, None, _dev(pos), _dev(slots, torch.int64), None, None,
                            None, None, cache, None, None, st)
    want = np.zeros(tuple(cache.shape), np.uint8)
    _expected_cache(L, want, k, v, pos, slots, 64, (exp, 0))
    assert np.array_equal(cache.cpu().numpy(), want) and int(st[0].item()) == 0


def test_scales_next_to_their_borders(B):
    """Groups whose largest value is steered next to a border between two scales, on either side of it, by the weight:
    the scale is that of the exact value."""
    import torch
    L = Layer(B, seed=20, H=8, per_head=True)
    T = 64
    pos = L.positions(T)
    k, v = _bf16(L.rng, (T, 8, 128)), _bf16(L.rng, (T, 8, 128))
    # one token's rows, and weights that bring each head's first group's largest value within 2^-22 of a border
    x = O.bf16_to_f64(k)
    y = L.want(1, x, pos)
    w = L.w[1].copy()
    for h in range(8):
        top = np.abs(y[h, h, :16]).max()
        mids = (C.E4M3[:-1] + C.E4M3[1:]) / 2 * 6
        mid = mids[np.searchsorted(mids, top)]
        w[h] *= mid / top * (1 + (h - 4) * 2.0 ** -23)
    dev = torch.from_numpy(w).float().cuda()
    L.dev[1], L.w[1] = dev, _f64(dev)
    c = B.make_cache_problem(num_requests=1, num_pages=1, max_blocks=1, num_q_heads=128, topk=1, token_cap=T,
                             chunk_cap=1)
    cache, st = B.new_cache(c), torch.zeros(4, dtype=torch.int32, device="cuda")
    slots = np.arange(T)
    B.msa_cache_append_rope(c, _append_problem(B, L, T, False, False), None, to_bf16_tensor(k, "cuda"),
                            to_bf16_tensor(v, "cuda"), None, None, _dev(pos), _dev(slots, torch.int64), None, None,
                            None, None, cache, None, None, st)
    want = np.zeros(tuple(cache.shape), np.uint8)
    _expected_cache(L, want, k, v, pos, slots, 64)
    assert np.array_equal(cache.cpu().numpy(), want)


def test_append_far_into_a_large_cache(B):
    """Slots whose bytes lie beyond 4 GB, and their groups that are done again."""
    import torch
    L = Layer(B, seed=30, H=2)
    P, T = 260_000, 300
    c = B.make_cache_problem(num_requests=1, num_pages=P, max_blocks=8, num_q_heads=32, topk=1, token_cap=T, chunk_cap=1)
    cache, st = B.new_cache(c), torch.zeros(4, dtype=torch.int32, device="cuda")
    pos = L.positions(T)
    k, v = _bf16(L.rng, (T, 2, 128)), _bf16(L.rng, (T, 2, 128))
    slots = P * 64 - 1 - np.arange(T)
    B.msa_cache_append_rope(c, _append_problem(B, L, T, False, False), None, to_bf16_tensor(k, "cuda"),
                            to_bf16_tensor(v, "cuda"), None, None, _dev(pos), _dev(slots, torch.int64), None, None,
                            None, None, cache, None, None, st)
    want = np.zeros((5, 2, 1, 9216), np.uint8)
    _expected_cache(L, want, k, v, pos, slots - (P - 5) * 64, 64)
    assert np.array_equal(cache[-5:].cpu().numpy(), want) and int(st[0].item()) == 0
    assert not torch.any(cache[:-5])


@pytest.mark.parametrize("kw", [dict(H=2), dict(H=1, adjacent=True, rotary=64), dict(H=3, axes=3, per_head=True, wide=False),
                                dict(H=11, index_norm=False)])
@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("past, new", [([0], [1]), ([63], [1]), ([127], [1]), ([60], [10]), ([60], [150]),
                                       ([60], [250]), ([0, 5, 100, 31], [200, 0, 300, 33]), ([64, 128], [64, 128])])
def test_append_equals_the_calls_apart(B, kw, block, past, new):
    """q, q_index, the tail and the pooled keys are, bit for bit, those of msa_norm_rope and msa_cache_append one after
    the other; the cache's bytes those of the definition; padding rows stay as they were."""
    import torch
    L = Layer(B, seed=21, **kw)
    s = Setup(B, past, new, H=L.H, block=block, token_pad=3, chunk_pad=2)
    T, n = s.c.token_cap, len(s.want["slot_map"])
    pos = np.full((T, L.axes), -1)
    pos[:n] = s.want["positions"][:, None] + np.arange(L.axes) * 3
    pos = pos if L.axes > 1 else pos[:, 0]
    slots = np.full(T, -1)
    slots[:n] = s.want["slot_map"]
    rows = to_bf16_tensor(_bf16(s.rng, (T, 20 * L.H, 128)), "cuda")     # q, k, v, q_index, k_index
    H = L.H
    q, k, v, qi, ki = (rows[:, a * H:b * H] for a, b in ((0, 16), (16, 17), (17, 18), (18, 19), (19, 20)))
    dp, ds, cu, ch = _dev(pos), _dev(slots, torch.int64), _dev(s.want["cu_tokens"]), s.chunk_table()
    tail = to_bf16_tensor(_bf16(s.rng, (len(past), 2, block, H, 128)), "cuda")
    pool = to_bf16_tensor(_bf16(s.rng, (s.c.num_pages, H, 128)), "cuda")
    fill = lambda t: torch.full(t.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    # apart
    wq, wk, wqi, wki = L.rope.forward(dp, q, k, qi, ki, out=[fill(q), fill(k), fill(qi), fill(ki)])
    wtail, wpool = tail.clone(), pool.clone()
    B.msa_cache_append(s.c, wk, v.contiguous(), wki, ds, cu, ch, B.new_cache(s.c), wtail, wpool, s.status)
    # in one call
    p = _append_problem(B, L, T, strides=[t.stride()[:2] for t in (q, k, qi, ki, v)])
    cache, gq, gqi = B.new_cache(s.c), fill(q), fill(qi)
    B.msa_cache_append_rope(s.c, p, q, k, v, qi, ki, dp, ds, cu, ch, gq, gqi, cache, tail, pool, s.status)
    assert s.code() == 0
    for a, b in ((gq, wq), (gqi, wqi), (tail, wtail), (pool, wpool)):
        assert torch.equal(a, b)
    want = np.zeros(tuple(cache.shape), np.uint8)
    _expected_cache(L, want, from_bf16_tensor(k), from_bf16_tensor(v), pos, slots, block)
    assert np.array_equal(cache.cpu().numpy(), want)


def test_bad_slots_positions_and_chunks(B):
    """Slots outside the cache, slots beside a negative position and chunk rows that do not fit: left out and reported;
    an earlier error: nothing is written."""
    import torch
    L = Layer(B, seed=22, H=2)
    T = 6
    c = B.make_cache_problem(num_requests=1, num_pages=2, max_blocks=2, num_q_heads=32, topk=1, token_cap=T, chunk_cap=1)
    k = to_bf16_tensor(_bf16(L.rng, (T, 2, 128)), "cuda")
    p, st = _append_problem(B, L, T, False, False), torch.zeros(4, dtype=torch.int32, device="cuda")

    def call(slots, pos, cache, p=p, **kw):
        a = dict(q=None, q_index=None, k_index=None, cu=None, chunks=None, q_out=None, q_index_out=None, tail=None, pool=None)
        a.update(kw)
        B.msa_cache_append_rope(c, p, a["q"], k, k, a["q_index"], a["k_index"], _dev(pos), _dev(slots, torch.int64),
                                a["cu"], a["chunks"], a["q_out"], a["q_index_out"], cache, a["tail"], a["pool"], st)
        torch.cuda.synchronize()
        return int(st[0].item())

    good = B.new_cache(c)
    assert call([0, 1, 2, 3, 4, 127], [0, 1, 2, 3, 4, 5], good) == 0
    for slots, pos in (([0, 128, 2, 3, 4, 127], [0] + [1, 2, 3, 4, 5]), ([0, -2, 2, 3, 4, 127], [0, 1, 2, 3, 4, 5]),
                       ([0, 1 << 40, 2, 3, 4, 127], [0, 1, 2, 3, 4, 5]), ([0, 1, 2, 3, 4, 127], [0, -1, 2, 3, 4, 5])):
        cache = B.new_cache(c)
        assert call(slots, pos, cache) == B.MSA_ERR_INVALID_CACHE
        for slot in (1,):
            b = cache[slot // 64, :, 0]
            assert not torch.any(b[:, slot * 64:slot * 64 + 64])
        # an earlier error: nothing is written
        before = cache.clone()
        call([0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5], cache)
        assert torch.equal(cache, before)
        st.zero_()
    # chunk rows
    full = _append_problem(B, L, T)
    q = to_bf16_tensor(_bf16(L.rng, (T, 32, 128)), "cuda")
    tail = torch.zeros((1, 2, 64, 2, 128), dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros((2, 2, 128), dtype=torch.bfloat16, device="cuda")
    for row, cu in (((1, 0, 6, 0), (0, 6)), ((0, -1, 6, 0), (0, 6)), ((0, 1, 6, 0), (0, 6)), ((0, 0, 9, 0), (0, 6)),
                    ((0, 0, 0, 0), (0, 6)), ((0, 0, 6, -1), (0, 6)), ((0, 0, 6, 1 << 20), (0, 6)), ((0, 0, 6, 60), (0, 6)),
                    ((0, 0, 6, 0), (1, 6)), ((0, 0, 6, 0), (0, 7)), ((0, 0, 6, 0), (0, 5))):
        code = call([0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5], B.new_cache(c), p=full, q=q, q_out=torch.empty_like(q),
                    q_index=k, q_index_out=torch.empty_like(k), k_index=k, cu=_dev(cu), chunks=_dev([row]), tail=tail,
                    pool=pool)
        assert code == B.MSA_ERR_INVALID_CACHE, row
        assert not torch.any(tail) and not torch.any(pool)
        st.zero_()
    assert call([0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5], B.new_cache(c), p=full, q=q, q_out=torch.empty_like(q),
                q_index=k, q_index_out=torch.empty_like(k), k_index=k, cu=_dev([0, 6]), chunks=_dev([[0, 0, 6, 0]]),
                tail=tail, pool=pool) == 0 and torch.any(tail)


class FollowRope(Follow):
    """Follow for steps through append_rope: the rows' positions are the step's own."""

    def __init__(self, B, kv, L, block, topk):
        super().__init__(B, kv, L.H, block, topk)
        self.L = L

    def step_rope(self, new, x, pos):
        """x: bits of q, k, v, q_index, k_index as the projections give them; pos: fp64 positions of the new tokens."""
        L, n = self.L, len(pos)
        rope = L.rope
        y = rope.forward(_dev(pos), *(to_bf16_tensor(x[m][:n], "cuda") for m in ("q", "k", "qi", "ki")))
        for i, m in enumerate(("q", "k", "qi", "ki")):
            _check_forward(L, i, x[m][:n], pos, y[i])
        q, _, qi, ki = (from_bf16_tensor(t) for t in y)
        q = np.concatenate([q, x["q"][n:]])     # padding rows, which no chunk covers
        codes, scales = R.round_values(L.want(1, O.bf16_to_f64(x["k"][:n]), pos), 0)
        k = np.array(C.E2M1 + [-v for v in C.E2M1])[codes] * np.repeat(C.E4M3[scales], 16, -1)
        # the oracle's step rounds K again: values of the cache stay what they are
        return self.step(new, O.f64_to_bf16(k), x["v"][:n], ki, qi, q)


def _drive_rope(B, kv, f, new, T, rng, graph=None):
    import torch
    H, L = f.H, f.L
    x = {m: _bf16(rng, (T, h, 128)) for m, h in (("q", 16 * H), ("k", H), ("v", H), ("qi", H), ("ki", H))}
    rows = torch.cat([to_bf16_tensor(x[m], "cuda") for m in ("q", "k", "v", "qi", "ki")], 1)
    n = int(np.maximum(new, 0).sum())
    seq = np.concatenate([f.lens[r] + np.arange(max(m, 0)) for r, m in enumerate(new)]) if n else np.zeros(0, int)
    pos = seq if L.axes == 1 else np.stack([seq, seq // 3, seq % 3 + 5], 1)
    full = np.full((T,) + pos.shape[1:], -1)
    full[:n] = pos
    if graph is None:
        kv.step(_dev(new), T)
        cut = [rows[:, a * H:b * H] for a, b in ((0, 16), (16, 17), (17, 18), (18, 19), (19, 20))]
        q, qi = kv.append_rope(L.rope, *cut, positions=None if L.axes == 1 else _dev(full))
        sel = kv.select(qi)
        kv._tables(T)["o"].fill_(7.0)
        kv._tables(T)["lse"].fill_(7.0)
        o, lse = kv.forward(q, sel)
    else:
        g, bufs, sel, o, lse = graph
        bufs["new"].copy_(_dev(new))
        bufs["rows"].copy_(rows)
        o.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
    torch.cuda.synchronize()
    kv.check_status()
    s, wsel, want = f.step_rope(new, x, pos)
    assert np.array_equal(kv.seq_lens.cpu().numpy(), f.lens)
    assert np.array_equal(sel.cpu().numpy()[:, :wsel.shape[1]], wsel)
    if n:
        _close(o, lse, want)


@pytest.mark.parametrize("kw", [dict(H=2), dict(H=1, axes=3, adjacent=True, rotary=64, per_head=True)])
def test_serving_run(B, kw):
    """Steps of prompts in pieces and single tokens through step, append_rope, select and forward, with requests that
    finish; at the end the cache reads back as the oracle's values."""
    import torch
    L = Layer(B, seed=23, **kw)
    H, block, K, R_ = L.H, 64, 3, 4
    kv = B.Cache(num_requests=R_, num_pages=14, max_blocks=6, num_q_heads=16 * H, topk=K, block_size=block,
                 max_tokens=300)
    f = FollowRope(B, kv, L, block, K)
    for new in ([100, 0, 1, 60], [1, 130, 1, 4], [1, 1, 1, 1], [1, -1, 1, -1], [1, 70, 0, 0], [-1, 1, 1, 200],
                [150, 1, -1, 1], [1, -1, 90, -1], [1] * 4):
        T = int(np.maximum(new, 0).sum())
        _drive_rope(B, kv, f, new, T + (T % 3), L.rng)
    for r in range(R_):
        n = int(f.lens[r])
        if n:
            p = np.arange(n)
            k, v = kv.read(_dev(f.table[r, p // block] * block + p % block, torch.int64))
            assert np.array_equal(O.bf16_to_f64(from_bf16_tensor(k)), f.k[r])
            assert np.array_equal(O.bf16_to_f64(from_bf16_tensor(v)), f.v[r])
    kv.check_status()


def test_captured_serving_step(B):
    """A step with append_rope captured and replayed; two caches share one Rope, their graphs replay in turn."""
    import torch
    L = Layer(B, seed=24, H=2)
    H, K, R_, T = 2, 4, 3, 6
    made = []
    for i in range(2):
        kv = B.Cache(num_requests=R_, num_pages=30, max_blocks=8, num_q_heads=16 * H, topk=K, max_tokens=183)
        f = FollowRope(B, kv, L, 64, K)
        _drive_rope(B, kv, f, [120, 3, 60], 183, L.rng)
        _drive_rope(B, kv, f, [1, 2, 1], T, L.rng)
        bufs = dict(rows=torch.zeros((T, 20 * H, 128), dtype=torch.bfloat16, device="cuda"),
                    new=torch.zeros(R_, dtype=torch.int32, device="cuda"))
        cut = [bufs["rows"][:, a * H:b * H] for a, b in ((0, 16), (16, 17), (17, 18), (18, 19), (19, 20))]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            kv.step(bufs["new"], T)
            q, qi = kv.append_rope(L.rope, *cut)
            sel = kv.select(qi)
            o, lse = kv.forward(q, sel)
        made.append((kv, f, (g, bufs, sel, o, lse)))
    for new in ([1, 1, 1], [2, 0, 1], [1, 3, 2], [0, 0, 0], [6, 0, 0], [1, -1, 1], [1, 5, 0]):
        for kv, f, graph in made:
            _drive_rope(B, kv, f, new, T, L.rng, graph)


def test_cache_without_index_keys_and_given_outputs(B):
    """append_rope of a cache without index keys; outputs in place of the inputs."""
    import torch
    L = Layer(B, seed=25, H=2)
    n = 70
    kv = B.Cache(num_requests=1, num_pages=4, max_blocks=3, num_q_heads=32, topk=2, max_tokens=n, index_keys=False)
    x = [to_bf16_tensor(_bf16(L.rng, (n, h, 128)), "cuda") for h in (32, 2, 2)]
    kv.step(_dev([n]), n)
    want = L.rope.forward(kv.positions, x[0])[0]
    q, qi = kv.append_rope(L.rope, *x)
    assert qi is None and torch.equal(q, want)
    first = kv.cache.clone()
    q, _ = kv.append_rope(L.rope, *x, out=[x[0]])
    assert q is x[0] and torch.equal(q, want) and torch.equal(first, kv.cache)
    kv.check_status()


# ---------------------------------------------------------------------------
# in training
# ---------------------------------------------------------------------------

def test_training_run(B):
    """Projections -> norm and rotation -> selection -> forward -> backward -> gradients of the projections and weights,
    over packed documents: each against the oracle of what it was given."""
    import torch
    L = Layer(B, seed=26, H=2, rotary=64, per_head=True)
    lengths = [200, 77, 130]
    cu = np.concatenate([[0], np.cumsum(lengths)])
    T = int(cu[-1])
    pos = np.concatenate([np.arange(n) for n in lengths])
    rows = _bf16(L.rng, (T, 40, 128))
    dev = to_bf16_tensor(rows, "cuda")
    cut = lambda x: (x[:, :32], x[:, 32:34], x[:, 34:36], x[:, 36:38], x[:, 38:40])
    q, k, v, qi, ki = cut(dev)
    yq, yk, yqi, yki = L.rope.forward(_dev(pos), q, k, qi, ki)
    for i, (y, at) in enumerate(((yq, 0), (yk, 1), (yqi, 3), (yki, 4))):
        _check_forward(L, i, cut(rows)[at], pos, y)
    prob = B.make_problem(cu, cu[:-1], T, 32, 3)
    sel, st = B.select_topk(prob, yqi, yki)
    v = v.contiguous()
    o, lse, st2 = B.forward(prob, sel, yq, yk, v)
    do = _bf16(L.rng, (T, 32, 128))
    bw = B.Backward(prob)
    dq, dk, dv = bw.run(sel, yq, yk, v, o, to_bf16_tensor(do, "cuda"), lse)
    torch.cuda.synchronize()
    bw.check_status()
    assert int(st[0].item()) == 0 and int(st2[0].item()) == 0
    bits = [from_bf16_tensor(t) for t in (yq, yk, v, o)]
    ref = O.backward_blocked(*bits[:3], bits[3], do, lse.double().cpu().numpy(), cu, cu[:-1], sel.cpu().numpy(), 64, 8,
                             128 ** -0.5)
    for name, got, want in zip(("dq", "dk", "dv"), (dq, dk, dv), ref):
        assert_grad_close(name, from_bf16_tensor(got), want)
    grad = torch.zeros_like(dev)
    gq, gk = cut(grad)[:2]
    (dxq, dxk), (dwq, dwk) = L.rope.backward(_dev(pos), (dq, dk), (q, k), out=(gq, gk))
    for i, (x, g, dx, dw) in enumerate(((q, dq, dxq, dwq), (k, dk, dxk, dwk))):
        _check_grad(L, i, _f64(x), _f64(g), pos, dx, dw)
    assert not torch.any(grad[:, 34:])
