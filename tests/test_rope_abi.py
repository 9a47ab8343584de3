"""Host-side argument checks of the norm and rotary entry points (CPU; the addresses are never dereferenced), the table
of pairs, and the Python classes' checks."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest


@pytest.fixture(scope="module")
def B():
    from block_sparse_top_attn_gb300 import build_lib
    build_lib.build()
    from block_sparse_top_attn_gb300 import binding
    return binding


class Pairs:  # what make_rope_problem looks at
    rotary_dim, num_axes = 128, 1

    class table:
        data_ptr = staticmethod(lambda: 1 << 20)


def _tensor(B, heads, **kw):
    return B.RopeTensor(heads, **kw)


def _problem(B, tokens=10, H=2, v=True, **kw):
    ts = dict(q=_tensor(B, 16 * H), k=_tensor(B, H), q_index=_tensor(B, H), k_index=_tensor(B, H))
    if v:
        ts["v"] = _tensor(B, H, norm=False, rotate=False)
    return B.make_rope_problem(tokens, Pairs, **ts, **kw)


def _cache_problem(B, **kw):
    return B.make_cache_problem(**{**dict(num_requests=4, num_pages=100, max_blocks=16, num_q_heads=32, topk=8,
                                          token_cap=10), **kw})


def _four(values):
    return (ctypes.c_void_p * 4)(*values)


GOOD = [(i + 1) << 20 for i in range(4)]
STATUS, POSITIONS, WS = 9 << 20, 10 << 20, 11 << 20


def _forward(B, p, x=GOOD, y=GOOD, positions=POSITIONS, status=STATUS):
    return B.lib.msa_norm_rope(p, None if x is None else _four(x), positions, None if y is None else _four(y), status,
                               None)


def _backward(B, p, dy=GOOD, x=GOOD, positions=POSITIONS, dx=GOOD, dw=(None,) * 4, status=STATUS, ws=WS, size=1 << 30):
    arr = lambda v: None if v is None else _four(v)
    return B.lib.msa_norm_rope_bwd(p, arr(dy), arr(x), positions, arr(dx), arr(dw), status, ws, size, None)


APPEND = ("q", "k", "v", "q_index", "k_index", "positions", "slot_map", "cu_tokens", "chunks", "q_out", "q_index_out",
          "cache", "index_tail", "index_pool", "status")


def _append(B, c, p, **kw):
    ptrs = {n: (i + 1) << 20 for i, n in enumerate(APPEND)}
    ptrs.update(kw)
    return B.lib.msa_cache_append_rope(None if c is None else ctypes.byref(c), None if p is None else ctypes.byref(p),
                                       *[ptrs[n] for n in APPEND], None)


def _passes(B, code):
    """Good arguments: on a machine with no GPU the call gets as far as the device check."""
    import torch
    if not torch.cuda.is_available():
        assert code in (B.MSA_ERR_CUDA, B.MSA_ERR_UNSUPPORTED_DEVICE)


def test_binding_has_the_headers_values(B):
    import pathlib
    import re
    text = (pathlib.Path(__file__).parent.parent / "include" / "msa.h").read_text()
    names = re.findall(r"\b(MSA_ROPE_\w+) = (\d+)", text)
    assert len(names) == 10
    for name, value in names:
        assert getattr(B, name) == int(value)


def test_struct_layout(B):
    """The last field that the library looks at is where the binding puts it."""
    p = _problem(B)
    assert B.msa_norm_rope_bwd_bytes(p) > 0
    p.tensor[4].y_head = 129
    assert B.msa_norm_rope_bwd_bytes(p) == 0
    assert ctypes.sizeof(B.msa_rope_pair) == 16


def test_pairs_are_turns_in_64_bits(B):
    f = [1.0, 0.5, 2 * math.pi, 7.25, 1e-9, 1e-18, 0.0, -0.3, 100.0, 5e6 ** -0.99, -1e-9, 3.0, 1e3, 1e-6, 0.1, -6.0]
    table = B.rope_pairs(f, [0, 1, 2, 3] * 4, device="cpu").table.numpy()
    two_pi = Fraction(6283185307179586476925286766559005768394, 10 ** 39)
    for w, (turns, axis), i in zip(f, table, range(16)):
        got = Fraction(int(turns) % 2 ** 64, 2 ** 64)
        want = Fraction(w) / two_pi
        off = (got - want) % 1
        off = min(off, 1 - off)
        # 2 pi and the quotient are rounded in fp64, the turns to 2^-64
        assert off <= abs(want) * Fraction(3, 2 ** 53) + Fraction(1, 2 ** 64), w
        assert axis == i % 4
    assert B.rope_pairs(B.rope_frequencies(64), device="cpu").num_axes == 1


@pytest.mark.parametrize("f, axes", [([math.nan] * 16, None), ([math.inf] * 16, None), ([1.0] * 16, [4] * 16),
                                     ([1.0] * 16, [-1] * 16)])
def test_bad_pairs(B, f, axes):
    with pytest.raises(B.MSAError):
        B.rope_pairs(f, axes, device="cpu")


def test_bad_pair_counts(B):
    for n in (0, 8, 17, 65):
        with pytest.raises(ValueError):
            B.rope_pairs([1.0] * n, device="cpu")
    with pytest.raises(ValueError):
        B.rope_pairs([1.0] * 16, [0] * 15, device="cpu")
    out = (B.msa_rope_pair * 65)()
    f = np.ones(65)
    assert B.lib.msa_rope_pairs(f.ctypes.data, None, 65, out) == 1
    assert B.lib.msa_rope_pairs(None, None, 4, out) == 1 and B.lib.msa_rope_pairs(f.ctypes.data, None, -1, out) == 1
    assert B.lib.msa_rope_pairs(f.ctypes.data, None, 64, out) == 0 and out[63].axis == 0


BAD = [("tokens", -1, 1), ("tokens", (1 << 24) + 1, 3), ("head_dim", 64, 3), ("rotary_dim", 16, 3),
       ("rotary_dim", 160, 3), ("rotary_dim", -32, 3), ("rotary_dim", 0, 1), ("num_axes", 0, 3), ("num_axes", 5, 3),
       ("eps", 0.0, 1), ("eps", -1.0, 1), ("eps", math.nan, 1), ("eps", math.inf, 1), ("weight_offset", math.nan, 1),
       ("weight_offset", math.inf, 1), ("cos_scale", 0.0, 1), ("cos_scale", math.inf, 1), ("cos_scale", math.nan, 1),
       ("pairs", None, 1), ("pairs", 8, 1)]


@pytest.mark.parametrize("field, value, code", BAD)
def test_bad_problems(B, field, value, code):
    p = _problem(B)
    setattr(p, field, value)
    assert _forward(B, p) == code and _backward(B, p) == code and B.msa_norm_rope_bwd_bytes(p) == 0
    assert _append(B, _cache_problem(B), p) == code


@pytest.mark.parametrize("field, value, code", [
    ("heads", -1, 1), ("heads", 16385, 3), ("flags", 16, 1), ("weight", 8, 1), ("x_token", 4, 1), ("x_token", -256, 1),
    ("x_token", 260, 1), ("x_token", 128, 1), ("x_head", 120, 1), ("x_head", 132, 1), ("y_token", 0, 1), ("y_head", 64, 1),
    ("y_token", 1 << 41, 1), ("x_head", 1 << 41, 1)])
def test_bad_tensors(B, field, value, code):
    for i in range(4):
        p = _problem(B)
        setattr(p.tensor[i], field, value)
        assert _forward(B, p) == code and _backward(B, p) == code and B.msa_norm_rope_bwd_bytes(p) == 0
        assert _append(B, _cache_problem(B), p) == code


def test_rows_by_head_and_by_token(B):
    """Token-major and head-major rows pass, rows that overlap do not."""
    for x_token, x_head, ok in ((256, 128, True), (128, 1280, True), (128, 1272, False), (248, 128, False),
                                (2048, 136, True), (128, 128, False)):
        p = _problem(B)
        p.tensor[1].x_token, p.tensor[1].x_head = x_token, x_head
        assert (B.msa_norm_rope_bwd_bytes(p) > 0) == ok, (x_token, x_head)


def test_null_and_misaligned_pointers(B):
    p = _problem(B)
    assert _forward(B, None) == 1 and _backward(B, None) == 1
    _passes(B, _forward(B, p))
    _passes(B, _backward(B, p))
    for bad in (None, (1 << 20) + 8):
        for kw in (dict(positions=bad), dict(status=bad)):
            assert _forward(B, p, **kw) == 1 and _backward(B, p, **kw) == 1
        assert _backward(B, p, ws=bad) == 1
        for i in range(4):
            rows = [bad if j == i else GOOD[j] for j in range(4)]
            assert _forward(B, p, x=rows) == 1 and _forward(B, p, y=rows) == 1
            for name in ("dy", "x", "dx"):
                assert _backward(B, p, **{name: rows}) == 1
            # a tensor that the call does not have needs no rows
            q = _problem(B)
            q.tensor[i].heads = 0
            _passes(B, _forward(B, q, x=rows, y=rows))
            _passes(B, _backward(B, q, x=rows, dy=rows, dx=rows))
    for name in ("x", "y"):
        assert _forward(B, p, **{name: None}) == 1
    for name in ("dy", "x", "dx", "dw"):
        assert _backward(B, p, **{name: None}) == 1
    assert _backward(B, p, size=B.msa_norm_rope_bwd_bytes(p) - 1) == 1
    # a weight's gradient without a weight, or without a norm
    assert _backward(B, p, dw=GOOD) == 1
    for t in p.tensor:
        t.weight = 1 << 20
    _passes(B, _backward(B, p, dw=GOOD))
    assert _backward(B, p, dw=[g + 8 for g in GOOD]) == 1
    for t in p.tensor:
        t.flags &= ~B.MSA_ROPE_NORM
    assert _backward(B, p, dw=GOOD) == 1


def test_no_tokens_need_no_rows(B):
    p = _problem(B, tokens=0)
    _passes(B, _forward(B, p, x=[None] * 4, y=[None] * 4, positions=None))
    _passes(B, _backward(B, p, dy=[None] * 4, x=[None] * 4, dx=[None] * 4, positions=None))


def test_append_arguments(B):
    c, p = _cache_problem(B), _problem(B)
    assert _append(B, None, p) == 1 and _append(B, c, None) == 1
    _passes(B, _append(B, c, p))
    for name in APPEND:
        for bad in (None, (1 << 20) + 8):
            assert _append(B, c, p, **{name: bad}) == 1, name
    for i, heads, code in ((0, 16, 1), (1, 1, 1), (1, 0, 1), (2, 1, 1), (3, 4, 1), (4, 0, 1), (4, 3, 1)):
        bad = _problem(B)
        bad.tensor[i].heads = heads
        if heads:
            bad.tensor[i].x_token = bad.tensor[i].y_token = 128 * heads
        assert _append(B, c, bad) == code, (i, heads)
    bad = _problem(B)
    bad.tensor[4].flags = B.MSA_ROPE_ROTATE
    assert _append(B, c, bad) == 1
    assert _append(B, c, _problem(B, tokens=9)) == 1
    for field, value, code in (("num_pages", 0, 1), ("block_size", 96, 3), ("topk", 33, 3), ("k_exp", 33, 1)):
        bad = _cache_problem(B)
        setattr(bad, field, value)
        assert _append(B, bad, p) == code
    # what a call leaves out it does not look at
    some = _problem(B)
    some.tensor[0].heads = some.tensor[2].heads = some.tensor[3].heads = 0
    _passes(B, _append(B, c, some, q=None, q_index=None, k_index=None, q_out=None, q_index_out=None, cu_tokens=None,
                       chunks=None, index_tail=None, index_pool=None))


def test_workspace_is_the_problems_alone(B):
    """The same on every machine; it grows with the weights' rows, not with the tokens beyond a bound."""
    sizes = [B.msa_norm_rope_bwd_bytes(_problem(B, tokens=n)) for n in (0, 1, 100, 10 ** 4, 10 ** 5, 10 ** 7)]
    assert sizes[0] >= 256 and sizes == sorted(sizes) and sizes[-1] == sizes[-2] < 1 << 21


def test_rope_object_checks_its_arguments(B):
    import torch
    bf = torch.bfloat16
    z = lambda *s: torch.zeros(s, dtype=bf)
    f = B.rope_frequencies(128)
    rope = B.Rope(f, device="cpu")
    pos = torch.zeros(5, dtype=torch.int32)
    q, k = z(5, 32, 128), z(5, 2, 128)
    for bad in (pos.long(), pos[:, None], pos.tolist(), torch.zeros(10, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="positions"):
            rope.forward(bad, q, k)
    for bad in (q.float(), z(4, 32, 128), z(5, 32, 64), z(5, 4096), z(5, 128, 32).transpose(1, 2)):
        with pytest.raises(ValueError, match="q:"):
            rope.forward(pos, bad, k)
    with pytest.raises(ValueError, match="k:"):
        rope.forward(pos, q, k.half())
    with pytest.raises(ValueError, match="grads"):
        rope.backward(pos, (q,), (q, k))
    with pytest.raises(ValueError, match="grads"):
        rope.backward(pos, (q, None), (q, k))
    with pytest.raises(ValueError, match="gradient of k"):
        rope.backward(pos, (q, z(5, 3, 128)), (q, k))
    many = B.Rope(f, axes=[0, 1, 2, 2] * 16, device="cpu")
    with pytest.raises(ValueError, match="positions"):
        many.forward(pos, q, k)
    with pytest.raises(ValueError, match="positions"):
        many.forward(torch.zeros((5, 2), dtype=torch.int32), q, k)
    for w in (torch.zeros(64), torch.zeros(128, dtype=torch.float16), torch.zeros((3, 128)), torch.zeros(256)[::2]):
        with pytest.raises(ValueError, match="weight"):
            B.RopeTensor(2, weight=w)
    with pytest.raises(ValueError, match="norm"):
        B.RopeTensor(2, norm=False, weight=torch.zeros(128))


def test_cache_object_checks_append_rope(B):
    import torch
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    kv = B.Cache(num_requests=2, num_pages=4, max_blocks=2, num_q_heads=16, topk=2, max_tokens=4, device="cpu")
    rope = B.Rope(B.rope_frequencies(64), device="cpu")
    q, k = z(3, 16, 128), z(3, 1, 128)
    with pytest.raises(RuntimeError):
        kv.append_rope(rope, q, k, k, k, k)
    kv._now = t = kv._tables(3)
    kv.slot_map, kv.positions, kv.chunks = t["slot_map"], t["positions"], t["chunks"]
    for args, what in (((k, k, k, k, k), "q:"), ((q, q, k, k, k), "k:"), ((q, k, k.float(), k, k), "v:"),
                       ((q, k, k, q, k), "q_index"), ((q, k, k, k, None), "k_index"), ((q[:2], k, k, k, k), "q:")):
        with pytest.raises(ValueError, match=what):
            kv.append_rope(rope, *args)
    many = B.Rope(B.rope_frequencies(64), axes=[0, 1] * 16, device="cpu")
    for pos in (None, torch.zeros((2, 2), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)):
        with pytest.raises(ValueError, match="positions"):
            kv.append_rope(many, q, k, k, k, k, positions=pos)
    bare = B.Cache(num_requests=2, num_pages=4, max_blocks=2, num_q_heads=16, topk=2, max_tokens=3, index_keys=False,
                   device="cpu")
    bare._now = bare._tables(3)
    bare.positions = bare._now["positions"]
    with pytest.raises(ValueError, match="k_index"):
        bare.append_rope(rope, q, k, k, None, k)


def test_rope_keeps_one_description_per_shape(B):
    """Strides of single rows do not matter; contiguous and strided inputs have descriptions of their own."""
    import torch
    rope = B.Rope(B.rope_frequencies(64), device="cpu")
    rows = torch.zeros((4, 20, 128), dtype=torch.bfloat16)
    q, k = rows[:, :16], rows[:, 16:17]
    p = rope._problem(4, (q, k, None, None), (q, k, None, None))
    assert (p.tensor[0].x_token, p.tensor[0].x_head, p.tensor[1].x_token, p.tensor[1].x_head) == (2560, 128, 2560, 128)
    assert rope._problem(4, (q, k, None, None), (q, k, None, None)) is p
    assert rope._problem(4, (q.contiguous(), k, None, None), (q, k, None, None)) is not p
    one = rope._problem(1, (q[:1], k[:1], None, None), (q[:1], k[:1], None, None))
    assert (one.tensor[0].x_token, one.tensor[1].x_token) == (2048, 128)
    for n in range(5, 200):
        rope._problem(n, (q, k, None, None), (q, k, None, None))
    assert len(rope._problems) <= 64


def test_descriptions_follow_a_weights_type(B):
    """A weight whose data is replaced by another type, shape or layout at the same address gets a description of its
    own, with its checks."""
    import torch
    buf = torch.zeros(4096, dtype=torch.uint8)
    w = torch.nn.Parameter(buf.view(torch.float32)[:256].view(2, 128), requires_grad=False)
    rope = B.Rope(B.rope_frequencies(64), k_weight=w, device="cpu")
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    flags = lambda: rope._problem(4, (None, x, None, None), (None, x, None, None)).tensor[1].flags
    fp32, per_head = B.MSA_ROPE_WEIGHT_FP32, B.MSA_ROPE_PER_HEAD
    base = B.MSA_ROPE_NORM | B.MSA_ROPE_ROTATE
    assert flags() == base | fp32 | per_head
    w.data = buf.view(torch.bfloat16)[:256].view(2, 128)
    assert flags() == base | per_head
    w.data = buf.view(torch.bfloat16)[:128]
    assert flags() == base
    w.data = buf.view(torch.float32)[:128]
    assert flags() == base | fp32
    assert {p.tensor[1].weight for p in rope._problems.values()} == {buf.data_ptr()}
    for bad in (buf.view(torch.float32)[:256:2], buf.view(torch.float16)[:128], buf.view(torch.float32)[:64]):
        w.data = bad
        with pytest.raises(ValueError, match="weight"):
            flags()
    w.data = torch.zeros(128)
    rope.device = torch.device("cuda", 0)       # as a weight that was moved away looks
    with pytest.raises(ValueError, match="k_weight"):
        flags()


def test_new_gradients_share_no_memory(B):
    """New tensors laid out as the inputs are: views of one buffer for views of one projection's output, tensors of their
    own where two inputs have elements in common."""
    import torch
    rows = torch.zeros((5, 12, 128), dtype=torch.bfloat16)
    place = lambda xs: [None if x is None else (x.data_ptr() - xs[0].data_ptr(), x.shape, x.stride()) for x in xs]
    for xs in ((rows[:, :6], rows[:, 6:8], rows[:, 9:11], rows[:, 11:]), (rows[:, 0::2], rows[:, 1::2]),
               (rows[:, 0:7:3], rows[:, 1:8:3], rows[:, 2:9:3])):
        made = B.Rope._like(xs)
        assert place(made) == place(xs) and len({x.untyped_storage().data_ptr() for x in made}) == 1
    q, k = rows[:, :8], rows[:, 8:9]
    for xs in ((q, k, q[:, :1], k), (None, k, None, k), (q, k, q, k), (q, rows[:, 7:9], rows[:, 8:10], rows[:, 9:11]),
               (q[:1], q[:1], k[:1], q[:1]), (rows[:4], rows[1:], None, rows[:4])):
        made = B.Rope._like(xs)
        for i, (x, d) in enumerate(zip(xs, made)):
            assert (x is None) == (d is None)
            if x is None:
                continue
            assert d.shape == x.shape and d.stride() == x.stride() and d.dtype == x.dtype
            d.fill_(i + 1)
        assert all(d is None or bool((d == i + 1).all()) for i, d in enumerate(made))


def test_outputs_that_share_memory_are_refused(B, monkeypatch):
    """Outputs that have elements in common with one another or with an input that is not theirs."""
    import contextlib

    import torch
    for name in ("device", "stream"):
        monkeypatch.setattr(torch.cuda, name, lambda *a: contextlib.nullcontext())
    calls = []
    for name in ("msa_norm_rope", "msa_norm_rope_bwd", "msa_cache_append_rope"):
        monkeypatch.setattr(B, name, lambda *a, name=name: calls.append(name))
    rope = B.Rope(B.rope_frequencies(64), device="cpu")
    T = 3
    pos = torch.zeros(T, dtype=torch.int32)
    new = lambda h: torch.zeros((T, h, 128), dtype=torch.bfloat16)
    rows = new(24)
    q, k, qi, ki = rows[:, :16], rows[:, 16:18], rows[:, 18:20], rows[:, 20:22]
    free = rows[:, 22:]
    for xs, out in (((q, k), (q, k)), ((q, k), (q, free)), ((q, k), (new(16), k)), ((q, k, k), (q, free, new(2))),
                    ((q, k, qi, ki), (q, k, qi, ki)), ((new(16), k), (q, free))):
        rope.forward(pos, *xs, out=out)
        rope.backward(pos, [new(x.shape[1]) for x in xs], [x.contiguous() for x in xs],
                      out=[new(x.shape[1]) for x in xs])
        assert calls == ["msa_norm_rope", "msa_norm_rope_bwd"], (xs, out)
        calls.clear()
    bad = (((q, k), (q, q[:, :2])), ((q, k), (new(16), q[:, 3:5])), ((q, k), (rows[:, 1:17], new(2))),
           ((q, k, qi, ki), (q, k, ki, qi)), ((q, k, k), (q, k, free)), ((q, k, q[:, :2]), (q, new(2), new(2))),
           ((q, k, qi), (new(16), free, free)), ((q, k, qi), (new(16), rows[:, 17:19], new(2))))
    for xs, out in bad:
        for _ in range(2):
            with pytest.raises(ValueError, match="out of .*: has elements in common"):
                rope.forward(pos, *xs, out=out)
            with pytest.raises(ValueError, match="out of .*: has elements in common|strides"):
                rope.backward(pos, [new(x.shape[1]) for x in xs], xs, out=out)
    # gradients over their inputs or incoming gradients, but not over another's
    x, g = (new(16), new(2)), (new(16), new(2))
    for out in (x, g, (x[0], g[1]), (g[0], new(2))):
        rope.backward(pos, g, x, out=out)
    with pytest.raises(ValueError, match="out of k: has elements in common"):
        rope.backward(pos, (new(16), g[1], new(2)), (new(16), new(2), x[1]), out=(new(16), x[1], new(2)))
    # the cache's append
    kv = B.Cache(num_requests=1, num_pages=4, max_blocks=2, num_q_heads=32, topk=2, max_tokens=T, device="cpu")
    kv._now = t = kv._tables(T)
    kv.slot_map, kv.positions, kv.chunks = t["slot_map"], t["positions"], t["chunks"]
    wide = new(40)
    q, k, v, qi, ki = wide[:, :32], wide[:, 32:34], wide[:, 34:36], wide[:, 36:38], wide[:, 38:]
    calls.clear()
    for out in ((q, qi), (new(32), qi), (q, new(2))):
        kv.append_rope(rope, q, k, v, qi, ki, out=out)
    assert len(calls) == 3
    for out in ((q, k), (q, v), (q, ki), (wide[:, 2:34], new(2)), (q, q[:, :2])):
        with pytest.raises(ValueError, match="out of .*: has elements in common"):
            kv.append_rope(rope, q, k, v, qi, ki, out=out)
    assert len(calls) == 3


def test_padding_of_new_outputs(B):
    """zero_padding is 0 or 1; a Rope's descriptions have it where the outputs are new."""
    import torch
    for value, code in ((2, 1), (-1, 1), (1, 0), (0, 0)):
        p = _problem(B)
        p.zero_padding = value
        if code:
            assert _forward(B, p) == code and _backward(B, p) == code and B.msa_norm_rope_bwd_bytes(p) == 0
            assert _append(B, _cache_problem(B), p) == code
        else:
            assert B.msa_norm_rope_bwd_bytes(p) > 0
    assert [_problem(B, zero_padding=z).zero_padding for z in (False, True)] == [0, 1] and _problem(B).zero_padding == 0
    rope = B.Rope(B.rope_frequencies(64), device="cpu")
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    xs = (None, x, None, None)
    new, given = rope._problem(4, xs, xs, zero=True), rope._problem(4, xs, xs)
    assert new is not given and new.zero_padding == 1 and given.zero_padding == 0


def test_positions_reach_the_library_aligned(B, monkeypatch):
    """Positions on a border of 16 bytes are passed on as they are, others as a copy."""
    import contextlib

    import torch
    for name in ("device", "stream"):
        monkeypatch.setattr(torch.cuda, name, lambda *a: contextlib.nullcontext())
    seen = []
    monkeypatch.setattr(B, "msa_norm_rope", lambda p, xs, positions, *a: seen.append(positions))
    monkeypatch.setattr(B, "msa_norm_rope_bwd", lambda p, dys, xs, positions, *a: seen.append(positions))
    rope = B.Rope(B.rope_frequencies(64), device="cpu")
    pos = torch.arange(40, dtype=torch.int32)
    x = torch.zeros((5, 2, 128), dtype=torch.bfloat16)
    first = (-pos.data_ptr() // 4) % 4      # a border
    for at in range(8):
        part = pos[first + at:first + at + 5]
        rope.forward(part, x)
        rope.backward(part, (x,), (x,))
        for got in seen:
            assert torch.equal(got, part) and got.data_ptr() % 16 == 0
            assert (got.data_ptr() == part.data_ptr()) == (at % 4 == 0)
        assert len(seen) == 2
        seen.clear()


def test_status_words_are_checked(B):
    """A status word that the device cannot write is refused before the launch."""
    import torch
    rope = B.Rope(B.rope_frequencies(64), device="cpu")
    pos, x = torch.zeros(4, dtype=torch.int32), torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    for bad in (torch.zeros(4, dtype=torch.int64), torch.zeros(0, dtype=torch.int32), 0, [0],
                torch.zeros(4, dtype=torch.int32, device="meta")):
        with pytest.raises(ValueError, match="status"):
            rope.forward(pos, x, status=bad)
        with pytest.raises(ValueError, match="status"):
            rope.backward(pos, (x,), (x,), status=bad)


def test_streams_of_other_devices_are_refused(B):
    """A launch there would read this device's memory from another."""
    import torch

    class Stream:
        device = torch.device("cuda", 1)

    rope = B.Rope(B.rope_frequencies(64), device="cpu")
    pos, x = torch.zeros(4, dtype=torch.int32), torch.zeros((4, 1, 128), dtype=torch.bfloat16)
    kv = B.Cache(num_requests=2, num_pages=4, max_blocks=2, num_q_heads=16, topk=2, max_tokens=4, device="cpu")
    kv._now = t = kv._tables(4)
    kv.slot_map, kv.positions, kv.chunks = t["slot_map"], t["positions"], t["chunks"]
    q = torch.zeros((4, 16, 128), dtype=torch.bfloat16)
    for call in (lambda s: rope.forward(pos, x, stream=s), lambda s: rope.backward(pos, (x,), (x,), stream=s),
                 lambda s: kv.append_rope(rope, q, x, x, x, x, stream=s)):
        with pytest.raises(ValueError, match="stream"):
            call(Stream)


def test_pairs_are_rounded_once(B):
    """The quotient by 2 pi is exact to the table's last bit: half of it, and 2^-3 of that for the arithmetic."""
    rng = np.random.default_rng(0)
    f = [B.rope_frequencies(128, 5e6), B.rope_frequencies(128), B.rope_frequencies(128, 1e9)]
    f += [np.exp(rng.uniform(-60, 26, 64)) for _ in range(20)] + [rng.uniform(-7, 7, 64)]
    f += [2.0 ** np.arange(-70, 38)[:64], 2.0 ** np.arange(-70, 38)[44:], 2 * math.pi * np.arange(1.0, 65),
          np.nextafter(2 * math.pi * np.arange(1.0, 65), 0), 2.0 ** -np.arange(1060.0, 1074)]
    # 2 pi to 75 digits
    two_pi = Fraction(6283185307179586476925286766559005768394338798750211641949889184615632812572, 10 ** 75)

    def off(w, turns):
        x = (Fraction(int(turns) % 2 ** 64, 2 ** 64) - Fraction(float(w)) / two_pi) % 1
        return min(x, 1 - x)

    def table(part):
        part = np.concatenate([part, np.ones(-len(part) % 64)])
        return zip(part, B.rope_pairs(part, device="cpu").table.numpy()[:, 0])

    for part in f:
        for w, turns in table(part):
            assert off(w, turns) <= Fraction(9, 8 * 2 ** 65), w
    for w, turns in table(2.0 ** rng.uniform(38, 110, 64)):
        assert off(w, turns) <= Fraction(9, 8 * 2 ** 65) + Fraction(float(w)) / two_pi / 2 ** 100, w


def test_new_gradients_of_views_far_apart(B):
    """Views far apart in one large buffer get memory of their own, not the distance between them."""
    import torch
    layers = torch.zeros((40, 6, 2, 128), dtype=torch.bfloat16)
    size = lambda made: sum({x.untyped_storage().data_ptr(): x.untyped_storage().nbytes() for x in made}.values())
    for xs in ((layers[0], layers[39]), (layers[3], layers[20], layers[21], layers[39]), (layers[5], layers[6])):
        made = B.Rope._like(xs)
        assert size(made) == len(xs) * layers[0].numel() * 2
        assert all(d.shape == x.shape and d.stride() == x.stride() for d, x in zip(made, xs))
    row = layers.view(1, -1, 128)       # one token: parts of its row, with a gap
    made = B.Rope._like((row[:, :16], row[:, 16:17], row[:, 18:19]))
    assert len({x.untyped_storage().data_ptr() for x in made}) == 1
    none = layers[:, :0]
    assert [d.shape for d in B.Rope._like((none[0], none[1]))] == [(0, 2, 128)] * 2
