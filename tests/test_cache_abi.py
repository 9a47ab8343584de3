"""Host-side argument checks of the serving entry points (CPU; the addresses are
never dereferenced) and the Python class's checks."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def B():
    from block_sparse_top_attn_gb300 import build_lib
    build_lib.build()
    from block_sparse_top_attn_gb300 import binding
    return binding


CALLS = {"msa_cache_step": 12, "msa_cache_append": 10, "msa_cache_read": 5, "msa_cache_select": 6, "msa_cache_fwd": 8}


def _problem(B, **kw):
    args = dict(num_requests=4, num_pages=100, max_blocks=16, num_q_heads=32, topk=8, token_cap=64)
    return B.make_cache_problem(**{**args, **kw})


def _call(B, name, c, ptrs):
    return getattr(B.lib, name)(None if c is None else ctypes.byref(c), *ptrs, None)


def test_sizes(B):
    c = _problem(B)
    assert c.chunk_cap == 16 and B.msa_cache_bytes(c) == 100 * 2 * 9216     # 64 / 8 + 2 * 4
    assert B.msa_cache_bytes(_problem(B, block_size=128)) == 2 * 100 * 2 * 9216
    assert B.msa_cache_chunk_bound(5, 5) == 5 and B.msa_cache_chunk_bound(0, 3) == 0
    assert B.msa_cache_chunk_bound(-1, 3) == 0
    big = _problem(B, num_pages=1 << 20, num_q_heads=16 * 8)
    assert B.msa_cache_bytes(big) == (1 << 20) * 8 * 9216


def test_binding_has_the_headers_values(B):
    import pathlib
    import re
    text = (pathlib.Path(__file__).parent.parent / "include" / "msa.h").read_text()
    for name in ("MSA_ERR_INVALID_CACHE", "MSA_CACHE_TILE_BYTES", "MSA_CHUNK_COLS"):
        assert getattr(B, name) == int(re.search(rf"\b{name} = (\d+)", text).group(1))


def test_chunk_bound_holds_every_step():
    """No lengths need more chunks than the bound (brute force over small batches)."""
    import itertools
    from block_sparse_top_attn_gb300 import binding as B
    need = lambda past, n: 0 if n == 0 else (past + n - 1) // 8 - past // 8 + 1
    worst = {n: max(need(p, n) for p in range(8)) for n in range(0, 40)}
    for R in (1, 2, 3):
        for ns in itertools.product(range(0, 40, 1 if R < 3 else 3), repeat=R):
            assert sum(worst[n] for n in ns) <= B.msa_cache_chunk_bound(sum(ns), R), ns


@pytest.mark.parametrize("name", list(CALLS))
def test_null_and_misaligned_pointers(B, name):
    good = [(i + 1) << 20 for i in range(CALLS[name])]
    assert _call(B, name, None, good) == B.MSA_ERR_INVALID_ARGUMENT
    for i in range(len(good)):
        if name == "msa_cache_append" and i == 2:
            continue   # k_index may be NULL: see below
        for bad in (None, good[i] + 8):
            ptrs = list(good)
            ptrs[i] = bad
            assert _call(B, name, _problem(B), ptrs) == B.MSA_ERR_INVALID_ARGUMENT, (i, bad)


def test_append_without_index_keys_needs_no_index_buffers(B):
    """The pointers behind k_index are not looked at without it; on a machine with no GPU the call then
    gets as far as the device check."""
    ptrs = [1 << 20, 2 << 20, None, 3 << 20, None, None, 4 << 20, None, None, 5 << 20]
    import torch
    if not torch.cuda.is_available():
        assert _call(B, "msa_cache_append", _problem(B), ptrs) in (B.MSA_ERR_CUDA, B.MSA_ERR_UNSUPPORTED_DEVICE)
    ptrs[2] = 6 << 20
    assert _call(B, "msa_cache_append", _problem(B), ptrs) == B.MSA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("field, value, code", [
    ("num_requests", 0, 1), ("num_requests", 8193, 3), ("num_pages", 0, 1), ("num_pages", (1 << 24) + 1, 3),
    ("max_blocks", 0, 1), ("max_blocks", 49153, 3), ("num_kv_heads", 0, 1), ("num_q_heads", 33, 3),
    ("head_dim", 64, 3), ("block_size", 32, 3), ("block_size", 96, 3), ("query_chunk", 16, 3), ("topk", 0, 3),
    ("topk", 33, 3), ("token_cap", 0, 1), ("token_cap", (1 << 24) + 1, 3), ("chunk_cap", 0, 1), ("k_exp", 33, 1),
    ("v_exp", -33, 1), ("softmax_scale", 0.0, 1), ("softmax_scale", -1.0, 1), ("softmax_scale", float("nan"), 1),
    ("softmax_scale", float("inf"), 1)])
def test_bad_problems(B, name, field, value, code):
    c = _problem(B)
    setattr(c, field, value)
    assert _call(B, name, c, [(i + 1) << 20 for i in range(CALLS[name])]) == code
    assert B.lib.msa_cache_bytes(ctypes.byref(c)) == 0


def test_heads_limit(B):
    c = _problem(B, num_q_heads=16 * 1025)
    assert B.msa_cache_bytes(c) == 0
    with pytest.raises(B.MSAError):
        B.new_cache(c, device="cpu")


def test_status_string(B):
    assert "cache" in B.status_string(B.MSA_ERR_INVALID_CACHE)


def test_cache_object_checks_its_arguments(B):
    """Wrong types, shapes, strides and order of calls raise before anything is launched (buffers on the CPU)."""
    import torch
    kv = B.Cache(num_requests=2, num_pages=4, max_blocks=2, num_q_heads=16, topk=2, max_tokens=4, device="cpu")
    with pytest.raises(RuntimeError):
        kv.append(torch.zeros(1), torch.zeros(1))
    with pytest.raises(RuntimeError):
        kv.forward(torch.zeros(1), torch.zeros(1))
    with pytest.raises(ValueError):
        kv.step(torch.zeros(3, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        kv.step(torch.zeros(2, dtype=torch.int64), 2)
    with pytest.raises(ValueError):
        kv.step([1, 1], 2)
    for tokens in (0, -1, 5):
        with pytest.raises(ValueError, match="tokens"):
            kv.step(torch.zeros(2, dtype=torch.int32), tokens)
    kv._now = t = kv._tables(3)
    kv.slot_map, kv.positions, kv.chunks = t["slot_map"], t["positions"], t["chunks"]
    x = torch.zeros((3, 1, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_index"):
        kv.append(x, x)
    with pytest.raises(ValueError, match="v"):
        kv.append(x, x.float(), x)
    with pytest.raises(ValueError, match="k"):
        kv.append(torch.zeros((3, 2, 128), dtype=torch.bfloat16)[:, :1], x, x)      # strided
    with pytest.raises(ValueError, match="q_index"):
        kv.select(x[:2])
    with pytest.raises(ValueError, match="q"):
        kv.forward(torch.zeros((3, 15, 128), dtype=torch.bfloat16), t["sel"])
    with pytest.raises(ValueError, match="sel"):
        kv.forward(torch.zeros((3, 16, 128), dtype=torch.bfloat16), t["sel"].long())
    with pytest.raises(ValueError, match="slots"):
        kv.read(torch.zeros(3, dtype=torch.int32))
    bare = B.Cache(num_requests=2, num_pages=4, max_blocks=2, num_q_heads=16, topk=2, max_tokens=3, index_keys=False,
                   device="cpu")
    bare._now = bare._tables(3)
    with pytest.raises(ValueError, match="k_index"):
        bare.append(x, x, x)
    with pytest.raises(RuntimeError):
        bare.select(x)


def test_cache_object_views_share_their_buffers(B):
    """Steps of any number of rows use prefixes of buffers made once; a bad description is refused at once."""
    import torch
    kv = B.Cache(num_requests=2, num_pages=4, max_blocks=2, num_q_heads=32, topk=3, max_tokens=200, device="cpu")
    for tokens in list(range(1, 201)) + [1, 200]:
        t = kv._tables(tokens)
        assert t["c"].token_cap == tokens and t["c"].chunk_cap == min(tokens, tokens // 8 + 4)
        assert t["o"].shape == (tokens, 32, 128) and t["sel"].shape == (2, t["c"].chunk_cap, 3)
        for name in ("slot_map", "positions", "chunks", "o", "lse", "sel"):
            assert t[name].is_contiguous() and t[name].data_ptr() == getattr(kv, "_" + name).data_ptr()
    for bad in (dict(topk=33), dict(num_q_heads=24), dict(block_size=96), dict(max_tokens=0), dict(k_exp=40)):
        with pytest.raises(B.MSAError):
            B.Cache(**{**dict(num_requests=2, num_pages=4, max_blocks=2, num_q_heads=32, topk=3, max_tokens=8,
                              device="cpu"), **bad})
