"""CPU model check of the hand-offs of the two persistent cached-attention
kernels (no GPU): `msa_cache_batch.cuh` (a service warp that feeds a ring, two
pairs of attending warps, joins through shared memory) and `msa_cache_chunk.cuh`
(list warp, decoders, two MMA issuers, softmax warps).

The model replays the kernels' order of waits, arrivals, copies and MMAs under
random interleavings.  A parity wait is correct only while the barrier is on
the awaited phase or has just completed it; copies land in any order, MMAs in
the order of their issuing thread; a buffer may be overwritten only once its
readers are done, and every reader must find its own tile, item or part.  Odd
rings, one phase of the query barrier for items without tiles, and scores
written over weights that are still read fail it."""
import random

import pytest


class _Bar:
    def __init__(self, name, count=1):
        self.name, self.done, self.count, self.arr = name, 0, count, 0

    def arrive(self):
        self.arr += 1
        assert self.arr <= self.count, f"surplus arrival on {self.name}"
        if self.arr == self.count:
            self.arr, self.done = 0, self.done + 1

    def ready(self, k):
        assert self.done in (k, k + 1), f"parity alias on {self.name}: phase {k}, completed {self.done}"
        return self.done == k + 1


class _Slot:
    """A buffer with its content and the number of readers still to come."""

    def __init__(self, name):
        self.name, self.tag, self.readers = name, None, 0

    def write(self, tag, readers):
        assert self.readers == 0, f"{self.name} overwritten before {self.readers} reads of {self.tag}"
        self.tag, self.readers = tag, readers

    def read(self, tag):
        assert self.tag == tag, f"{self.name} holds {self.tag}, wanted {tag}"
        self.readers -= 1


def _run(threads, rng, pending=(), bias=None):
    """Steps generators in random order until all end; pending: callables that make asynchronous work progress.
    bias: names of threads that run ten times as often."""
    live = dict(threads)
    idle = 0
    while live:
        names = list(live)
        weights = [10 if bias and n in bias else 1 for n in names]
        progress = False
        if pending and rng.random() < 0.4:
            progress = any([p(rng) for p in pending])
        name = rng.choices(names, weights)[0]
        try:
            progress = next(live[name]) is not None or progress
        except StopIteration:
            del live[name]
            progress = True
        idle = 0 if progress else idle + 1
        assert idle < 200000, f"deadlock: {list(live)}"


def _wait(bar, k):
    while not bar.ready(k):
        yield None
    yield 1


# ---------------------------------------------------------------------------
# batch kernel
# ---------------------------------------------------------------------------

def _batch(items, seed, ring=8, bias=None):
    rng = random.Random(seed)
    full = [_Bar(f"full{i}") for i in range(ring)]
    empty = [_Bar(f"empty{i}", 2) for i in range(ring)]
    item_full = [_Bar(f"item_full{i}") for i in range(2)]
    item_free = [_Bar(f"item_free{i}", 4) for i in range(2)]
    part_full = [_Bar(f"part_full{i}") for i in range(2)]
    part_free = [_Bar(f"part_free{i}") for i in range(2)]
    pair_full = _Bar("pair_full")
    stage = [_Slot(f"stage{i}") for i in range(ring)]
    item = [_Slot(f"item{i}") for i in range(2)]
    part = [_Slot(f"part{i}") for i in range(2)]
    flying, seen, written = [], {}, []

    def service():
        n = 0
        for i, nt in enumerate(items + [-1]):
            if i >= 2:
                yield from _wait(item_free[i & 1], (i >> 1) - 1)
            item[i & 1].write(i, 4)
            item_full[i & 1].arrive()
            yield 1
            for _ in range(max(nt, 0)):
                st, lap = n % ring, n // ring
                if lap > 0:
                    yield from _wait(empty[st], lap - 1)
                flying.append(n)
                n += 1
                yield 1

    def land(r):
        if not flying:
            return False
        n = flying.pop(r.randrange(len(flying)))
        stage[n % ring].write(n, 2)
        full[n % ring].arrive()
        return True

    def attend(w):
        pair, base = w >> 1, 0
        for i, nt in enumerate(items + [-1]):
            yield from _wait(item_full[i & 1], i >> 1)
            assert item[i & 1].tag == i
            if nt < 0:
                return
            n = base + ((base ^ pair) & 1)
            while n < base + nt:
                yield from _wait(full[n % ring], n // ring)
                stage[n % ring].read(n)
                seen.setdefault(n, []).append(w & 1)
                yield 1
                empty[n % ring].arrive()
                n += 2
            base += nt
            if w & 1:
                if i >= 1:
                    yield from _wait(part_free[pair], i - 1)
                part[pair].write(("odd", i), 1)
                part_full[pair].arrive()
            else:
                yield from _wait(part_full[pair], i)
                part[pair].read(("odd", i))
                yield 1
                if w == 2:
                    part[1].write(("pair", i), 1)
                    pair_full.arrive()
                else:
                    part_free[0].arrive()
                    yield from _wait(pair_full, i)
                    part[1].read(("pair", i))
                    yield 1
                    part_free[1].arrive()
                    assert item[i & 1].tag == i
                    written.append(i)
            item[i & 1].read(i)
            item_free[i & 1].arrive()
            yield 1

    threads = {"service": service(), **{f"w{w}": attend(w) for w in range(4)}}
    _run(threads, rng, [land], bias)
    assert not flying and written == list(range(len(items)))
    assert all(sorted(seen[n]) == [0, 1] for n in range(sum(items)))


ITEMS = [[32] * 3, [1, 2, 3, 4, 5, 6, 7], [0, 0, 5, 0, 1, 0, 0, 2], [], [0], [64, 1, 64], [3, 3, 3, 3, 3]]


@pytest.mark.parametrize("items", ITEMS)
@pytest.mark.parametrize("bias", [None, ["w0", "w1"], ["w2", "w3"], ["service"], ["w1"]])
def test_batch_hand_offs(items, bias):
    for seed in range(12):
        _batch(items, seed, bias=bias)


def test_batch_model_rejects_an_odd_ring():
    """A pair that skips every other phase of a stage takes the phase before it for its own."""
    with pytest.raises(AssertionError, match="parity alias|holds|surplus|overwritten"):
        for seed in range(300):
            _batch([40], seed, ring=5, bias=["w0", "w1", "service"])


# ---------------------------------------------------------------------------
# chunk kernel
# ---------------------------------------------------------------------------

def _chunk(items, seed, warps=2, q_phase_per_item=False, early_scores=False, bias=None):
    rng = random.Random(seed)
    q_full = _Bar("q_full", warps)
    k_full = [_Bar(f"k_full{i}", warps) for i in range(2)]
    v_full = [_Bar(f"v_full{i}", warps) for i in range(2)]
    s_full = [_Bar(f"s_full{i}") for i in range(2)]
    p_full = [_Bar(f"p_full{i}", warps) for i in range(2)]
    pv_done = [_Bar(f"pv_done{i}") for i in range(2)]
    list_full = [_Bar(f"list_full{i}") for i in range(2)]
    list_free = [_Bar(f"list_free{i}", 2 * warps + 2) for i in range(2)]
    lists = [_Slot(f"list{i}") for i in range(2)]
    K = [[_Slot(f"K{b}.{w}") for w in range(warps)] for b in range(2)]
    V = [[_Slot(f"V{b}.{w}") for w in range(warps)] for b in range(2)]
    SP = [[_Slot(f"SP{b}.{w}") for w in range(warps)] for b in range(2)]   # a warp's rows of S, then of P
    Q = [None] * warps
    O, stored = {"tag": None}, []
    mma = {"S": [], "PV": []}   # in order within an issuing thread, in any order between the two

    def run_mma(r):
        kind = r.choice(["S", "PV"])
        if not mma[kind]:
            return False
        n, i, first = mma[kind].pop(0)
        if kind == "S":
            assert Q == [i] * warps, (Q, i)
            for x in K[n & 1]:
                x.read(n)
            for x in SP[n & 1]:
                x.write(("S", n), 1)
            s_full[n & 1].arrive()
        else:
            for x in V[n & 1]:
                x.read(n)
            for x in SP[n & 1]:
                x.read(("P", n))
            if first:
                assert O["tag"] is None or O["tag"][0] in stored, "O overwritten before it was stored"
            else:
                assert O["tag"] == (i, n - 1)
            O["tag"] = (i, n)
            pv_done[n & 1].arrive()
        return True

    def list_warp():
        for i, nt in enumerate(items + [-1]):
            if i >= 2:
                yield from _wait(list_free[i & 1], (i >> 1) - 1)
            lists[i & 1].write(i, 2 * warps + 2)
            list_full[i & 1].arrive()
            yield 1

    def score_issuer():
        n = nq = 0
        for i, nt in enumerate(items + [-1]):
            yield from _wait(list_full[i & 1], i >> 1)
            if nt < 0:
                return
            lists[i & 1].read(i)
            list_free[i & 1].arrive()
            if nt > 0 or q_phase_per_item:
                yield from _wait(q_full, nq)
                nq += 1
            for _ in range(nt):
                yield from _wait(k_full[n & 1], n >> 1)
                if n >= 2 and not early_scores:
                    yield from _wait(pv_done[n & 1], (n >> 1) - 1)
                mma["S"].append((n, i, None))
                n += 1
                yield 1

    def out_issuer():
        n = 0
        for i, nt in enumerate(items + [-1]):
            yield from _wait(list_full[i & 1], i >> 1)
            if nt < 0:
                return
            lists[i & 1].read(i)
            list_free[i & 1].arrive()
            for j in range(nt):
                yield from _wait(p_full[n & 1], n >> 1)
                yield from _wait(v_full[n & 1], n >> 1)
                mma["PV"].append((n, i, j == 0))
                n += 1
                yield 1

    def decoder(w):
        n = 0
        for i, nt in enumerate(items + [-1]):
            yield from _wait(list_full[i & 1], i >> 1)
            if nt < 0:
                return
            for _ in range(nt):
                if n >= 2:
                    yield from _wait(s_full[n & 1], (n >> 1) - 1)
                K[n & 1][w].write(n, 1)
                k_full[n & 1].arrive()
                yield 1
                if n >= 2:
                    yield from _wait(pv_done[n & 1], (n >> 1) - 1)
                assert lists[i & 1].tag == i
                V[n & 1][w].write(n, 1)
                v_full[n & 1].arrive()
                n += 1
                yield 1
            lists[i & 1].read(i)
            list_free[i & 1].arrive()

    def softmax(w):
        seq = 0
        for i, nt in enumerate(items + [-1]):
            yield from _wait(list_full[i & 1], i >> 1)
            if nt < 0:
                return
            if nt > 0 or q_phase_per_item:
                Q[w] = i
                q_full.arrive()
                yield 1
            for j in range(nt):
                n = seq + j
                yield from _wait(s_full[n & 1], n >> 1)
                SP[n & 1][w].read(("S", n))
                yield 1
                SP[n & 1][w].write(("P", n), 1)
                if j > 0 and rng.random() < 0.3:        # this warp rescales its rows of O
                    yield from _wait(pv_done[(n - 1) & 1], (n - 1) >> 1)
                    assert O["tag"] == (i, n - 1)
                    yield 1
                    assert O["tag"] == (i, n - 1)
                p_full[n & 1].arrive()
                yield 1
            if nt > 0:
                n = seq + nt - 1
                yield from _wait(pv_done[n & 1], n >> 1)
                assert O["tag"] == (i, n)
                done.setdefault(i, set()).add(w)
                if len(done[i]) == warps:
                    stored.append(i)
            yield 1
            assert lists[i & 1].tag == i
            lists[i & 1].read(i)
            list_free[i & 1].arrive()
            seq += nt

    done = {}
    threads = {"list": list_warp(), "s_issuer": score_issuer(), "o_issuer": out_issuer(),
               **{f"d{w}": decoder(w) for w in range(warps)},
               **{f"s{w}": softmax(w) for w in range(warps)}}
    _run(threads, rng, [run_mma], bias)
    assert stored == [i for i, nt in enumerate(items) if nt > 0] and not mma["S"] and not mma["PV"]


@pytest.mark.parametrize("items", ITEMS)
@pytest.mark.parametrize("bias", [None, ["s0", "s1"], ["d0", "d1"], ["s_issuer"], ["o_issuer"], ["list", "d0"], ["s0"]])
def test_chunk_hand_offs(items, bias):
    for seed in range(8):
        _chunk(items, seed, bias=bias)


def test_chunk_model_rejects_a_query_phase_for_items_without_tiles():
    with pytest.raises(AssertionError, match="parity alias|deadlock"):
        for seed in range(200):
            _chunk([0, 0, 0, 0, 2, 0, 0, 0], seed, q_phase_per_item=True, bias=["s0", "s1", "list", "d0", "d1"])


def test_chunk_model_rejects_scores_over_weights_in_use():
    with pytest.raises(AssertionError, match="SP|parity alias|holds"):
        for seed in range(200):
            _chunk([9], seed, early_scores=True, bias=["d0", "d1", "s_issuer"])


# ---------------------------------------------------------------------------
# the status word, which other CTAs of a launch may set while a CTA starts
# ---------------------------------------------------------------------------

def _start(seed, voted, warps=4):
    """A CTA of select_kernel: every warp reads the status once, at a time of its own, and another CTA sets it at some
    time.  voted: the CTA leaves as a whole if any warp saw it set.  Warp 0 writes the row's length and the list's
    counters, every warp uses them behind a barrier (which a warp that has left does not hold up)."""
    rng = random.Random(seed)
    order = [f"w{w}" for w in range(warps)] + ["other CTA"]
    rng.shuffle(order)
    saw = {w: order.index(f"w{w}") > order.index("other CTA") for w in range(warps)}
    if voted:
        saw = dict.fromkeys(saw, any(saw.values()))
    stay = [w for w in saw if not saw[w]]
    written = 0 in stay
    for w in stay:
        assert written, f"warp {w} goes on with what warp 0 has not written"


def test_a_voted_status_keeps_a_cta_together():
    for seed in range(500):
        _start(seed, voted=True)


def test_status_model_rejects_a_decision_by_warp():
    with pytest.raises(AssertionError, match="has not written"):
        for seed in range(500):
            _start(seed, voted=False)


def _kernel_source(file, name):
    import pathlib
    import re
    text = (pathlib.Path(__file__).parent.parent / "block_sparse_top_attn_gb300" / "csrc" / file).read_text()
    body = re.search(rf"\b{name}\(\w+ a\) {{\n(.*?)\n}}\n", text, re.S).group(1)
    return re.sub(r"//[^\n]*", "", body)


def test_select_decides_on_the_status_by_a_vote():
    """What the model above stands for: the kernel's one look at the status is a vote of the CTA."""
    body = _kernel_source("msa_cache.cu", "select_kernel")
    assert body.count("status_bad(") == 1 and body.count("__syncthreads_or(status_bad(a.status))") == 1


@pytest.mark.parametrize("file, name", [("msa_cache_fwd.cu", "fwd_cache_kernel"),
                                        ("msa_cache_batch.cuh", "fwd_batch_kernel"),
                                        ("msa_cache_chunk.cuh", "fwd_chunk_kernel")])
def test_attention_decides_on_the_status_by_a_vote(file, name):
    """In the attention kernels one warp looks at the status, and what it does next needs all of its lanes or none:
    every look is a vote of the warp, in place or, where the read has to be early, of the value read."""
    import re
    body = _kernel_source(file, name)
    looks = re.findall(r"[^;]*status_bad\(a\.status\)[^;]*;", body)
    assert len(looks) == 1
    if "__any_sync(0xffffffffu, status_bad(a.status))" not in looks[0]:
        assert re.search(r"\bstale = status_bad\(a\.status\)", looks[0])
        uses = re.findall(r"[^;]*\bstale\b[^;]*;", body.replace(looks[0], ""))
        assert uses and all("__any_sync(0xffffffffu, stale)" in u or "bool stale = false" in u for u in uses)


def test_serving_kernels_read_by_plain_loads():
    """The serving kernels may come up while the kernel before them still writes, so none of them reads through the path
    for memory that is constant for a kernel's life (nor lets the compiler choose it)."""
    import pathlib
    import re
    csrc = pathlib.Path(__file__).parent.parent / "block_sparse_top_attn_gb300" / "csrc"
    files = sorted(csrc.glob("msa_cache*"))
    assert len(files) >= 5
    for f in files:
        code = re.sub(r"//[^\n]*", "", f.read_text())
        for word in ("__ldg", "ld.global.nc", "__restrict__"):
            assert word not in code, (f.name, word)
