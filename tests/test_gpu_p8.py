"""The paged 8-bit KV cache's operators (hy_op_kv_append_p8, hy_op_attention_p8,
hy_op_attention_p8_prompt) against the plain form of tests/p8_util.py."""
import ctypes

import numpy as np
import pytest

from bandwidth_bound_hybrid_gb300 import capi
from tests.p8_util import BLOCK, World

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L(gpu):
    from bandwidth_bound_hybrid_gb300 import build
    build.build()
    return capi.lib()


@pytest.fixture(autouse=True)
def clean_guard(L):
    L.hy_op_check_device(None, None)
    yield


def guard(L):
    bits = ctypes.c_uint32()
    L.hy_op_check_device(None, ctypes.byref(bits))
    return bits.value


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("nq,nkv,hd", [(4, 2, 64), (16, 4, 128), (16, 2, 256), (1, 1, 64), (8, 8, 128)])
@pytest.mark.parametrize("lens,n,page", [
    ([0], [1], 128), ([15], [1], 16), ([16], [15], 16), ([5], [26], 48), ([0, 31, 7, 130], [3, 1, 0, 64], 32),
    ([100, 0, 48, 17, 2], [90, 37, 16, 15, 14], 64)])
def test_append(L, nq, nkv, hd, lens, n, page):
    w = World(nq, nkv, hd, lens, n, page).fill()
    before = w.snapshot()
    assert w.append(L) == capi.HY_OK, L.hy_last_error()
    w.check_append(before)
    assert guard(L) == 0


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_append_unaligned_rows_and_no_values(L, hd):
    """Rows of y of an odd pitch at an odd address, kv_new null, rows behind the last sequence's."""
    w = World(4, 2, hd, [9, 40], [30, 8], 32, pad_y=1, gap_rows=3).fill()
    t = w.t
    odd = t.empty(w.d["y"].numel() + 1, device="cuda")[1:].view_as(w.d["y"]).copy_(w.d["y"])
    rope = t.empty(w.d["rope"].numel() + 2, device="cuda")[2:].view_as(w.d["rope"]).copy_(w.d["rope"])
    before = w.snapshot()
    assert w.append(L, new=False, y=odd.data_ptr(), rope=rope.data_ptr()) == capi.HY_OK
    w.check_append(before, new=False)


def test_append_however_it_is_cut(L):
    """One call, calls of a row each and calls of uneven pieces leave the same pages and tails."""
    nq, nkv, hd, T, n = 8, 2, 128, 21, 75
    got = []
    for cuts in ([n], [1] * n, [3, 16, 1, 30, 25], [11, 64]):
        w = World(nq, nkv, hd, [T], [n], 32, seed=5).fill()
        at = 0
        for k in cuts:
            start = w.t.tensor([0, k], dtype=w.t.int32, device="cuda")
            ln = w.t.tensor([T + at], dtype=w.t.int32, device="cuda")
            assert w.append(L, n=k, y=w.d["y"][at:].data_ptr(), start=start.data_ptr(), len=ln.data_ptr(), new=None) == capi.HY_OK
            at += k
            w.t.cuda.synchronize()
        # the tail's rows past the open ones may differ: those that earlier blocks have left there
        s = w.snapshot()
        s["tail"] = s["tail"][:2 * nkv * BLOCK * hd].view(2, nkv, BLOCK, hd)[:, :, :(T + n) % BLOCK].clone()
        got.append(s)
    for s in got[1:]:
        for k in s:
            assert w.t.equal(s[k], got[0][k]), k


def test_append_special_values(L):
    """NaN and infinities (also of the rounding to bf16) make their block NaN, tiny blocks are zero, neighbours stay exact."""
    nq, nkv, hd = 4, 2, 64
    w = World(nq, nkv, hd, [0, 8], [64, 3], 32)
    y = w.y[:, :(nq + 2 * nkv) * hd].reshape(w.rows, -1, hd)
    y[3, nq + nkv, 5] = np.nan          # V head 0, block 0
    y[17, nq + nkv + 1, 60] = np.inf    # V head 1, block 1
    y[40, nq + 1, 0] = 3.4e38           # K head 1, block 2: past bf16 after the rounding or the rotation
    y[32:48, nq + nkv] = 0              # V head 0, block 2
    y[48:64, nq + nkv + 1] *= np.float32(2.0 ** -105)  # V head 1, block 3: below 2^-100
    y[65, nq + nkv, 1] = -np.inf        # an open row
    y[66, nq, 2] = np.nan
    w.fill()
    before = w.snapshot()
    assert w.append(L) == capi.HY_OK
    w.check_append(before)


def test_append_refused_sequences(L):
    """Bad positions and rows are refused one by one; the others run."""
    nq, nkv, hd = 4, 2, 64
    w = World(nq, nkv, hd, [3, 20, 5, 16], [10, 7, 4, 20], 16, spare=0).fill()
    for lens in ([-1, 20, 5, 16], [3, w.cap - 6, 5, 16], [3, 20, 5, 2 ** 31 - 1]):
        v = World(nq, nkv, hd, [3, 20, 5, 16], [10, 7, 4, 20], 16, spare=0).fill()
        bad = [b for b in range(4) if lens[b] != v.lens[b]]
        ln = v.t.tensor(lens, dtype=v.t.int32, device="cuda")
        before = v.snapshot()
        assert v.append(L, len=ln.data_ptr()) == capi.HY_OK
        v.check_append(before, refused=bad)
        assert guard(L) == capi.HY_GUARD_BAD_POSITION
    for start, bad in (([0, 10, 17, 21, 42], [3]), ([-1, 10, 17, 21, 41], [0]), ([0, 10, 17, 16, 36], [2])):
        v = World(nq, nkv, hd, [3, 20, 5, 16], [10, 7, 4, 20], 16, spare=0)
        v.start = np.array(start, dtype=np.int32)
        for b in range(4):
            v.n[b] = start[b + 1] - start[b] if b not in bad else 0
        v.fill()
        before = v.snapshot()
        assert v.append(L, n=41, new=False) == capi.HY_OK
        v.check_append(before, refused=bad, new=False)
        assert guard(L) == capi.HY_GUARD_BAD_POSITION


def test_append_without_a_page(L):
    """A block whose page the table does not have is not written; its rows' values and everything else are."""
    w = World(4, 2, 64, [10, 0], [60, 33], 16).fill()
    w.table[0, 2] = w.pool
    w.d["table"].copy_(w.t.from_numpy(w.table))
    before = w.snapshot()
    assert w.append(L) == capi.HY_OK
    w.check_append(before, lost={(0, 2)})
    assert guard(L) == capi.HY_GUARD_BAD_INDEX


# ------------------------------------------------------------------ decode
SHAPES = [(4, 2, 64), (8, 1, 64), (2, 2, 64), (16, 4, 128), (8, 8, 128), (16, 2, 128), (8, 4, 128), (16, 2, 256), (4, 1, 256),
          (2, 2, 256), (4, 2, 256)]


@pytest.mark.parametrize("nq,nkv,hd", SHAPES)
@pytest.mark.parametrize("lens", [[0], [15], [16, 0, 31], [37, 1000, 255, 14], [4095], [700, 33, 47, 1, 0, 15, 16, 2047, 5]])
def test_decode(L, nq, nkv, hd, lens):
    w = World(nq, nkv, hd, lens, page=64).fill()
    before = w.snapshot()
    ws = w.workspace(L)
    assert w.decode(L, ws) == capi.HY_OK, L.hy_last_error()
    w.check_append(before)
    w.check_attention()
    assert guard(L) == 0


@pytest.mark.parametrize("nq,nkv,hd", [(4, 2, 64), (16, 4, 128), (16, 2, 256)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 0), (16, 4), (17, 16), (100, 33), (64, 2000), (700, 5), (5000, 3),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
def test_decode_window(L, nq, nkv, hd, window, sinks):
    """Pages out of view are not looked up (their table entries are bad ones), and what they hold does not matter."""
    w = World(nq, nkv, hd, [0, 3, 15, 31, 64, 115, 500, 1023, 1500], page=16, window=window, sinks=sinks, pad_o=3).fill()
    before = w.snapshot()
    ws = w.workspace(L)
    assert w.decode(L, ws) == capi.HY_OK
    w.check_append(before)
    w.check_attention()
    assert guard(L) == 0


@pytest.mark.parametrize("nq,nkv,hd,lens", [(16, 4, 128, [300 + 61 * i for i in range(70)]), (2, 1, 64, list(range(256))),
                                            (16, 2, 256, [3000, 40, 2000] * 7), (4, 4, 128, [9000, 17000, 12])])
@pytest.mark.parametrize("window", [0, 333])
def test_decode_many_sequences(L, nq, nkv, hd, lens, window):
    w = World(nq, nkv, hd, lens, page=128, window=window, sinks=4).fill()
    before = w.snapshot()
    ws = w.workspace(L)
    assert w.decode(L, ws) == capi.HY_OK
    w.check_append(before)
    w.check_attention()


def test_decode_steps_of_one_cache(L):
    """40 steps of ragged sequences with one workspace, on a stream of its own: across blocks' ends."""
    t = pytest.importorskip("torch")
    nq, nkv, hd = 8, 2, 128
    w = World(nq, nkv, hd, [3, 60, 470], page=32, spare=4, far_page=8).fill()
    ws = w.workspace(L)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    for step in range(40):
        before = w.snapshot()
        w.y[:] = w.rng.standard_normal(w.y.shape).astype(np.float32)
        for b in range(3):  # pages as they fill up
            for i in range(w.max_pages):
                if w.needs(b, i) and not 0 <= w.table[b, i] < w.pool:
                    free = sorted(set(range(w.pool)) - set(w.table[(w.table >= 0) & (w.table < w.pool)].tolist()))
                    w.table[b, i] = free[0]
        w.d["y"].copy_(t.from_numpy(w.y))
        w.d["table"].copy_(t.from_numpy(w.table))
        w.d["len"].copy_(t.tensor(w.lens, dtype=t.int32))
        t.cuda.synchronize()
        assert w.decode(L, ws, stream=side.cuda_stream) == capi.HY_OK
        side.synchronize()
        w.check_append(before)
        if step % 5 == 0 or any(x % BLOCK == BLOCK - 1 for x in w.lens):
            w.check_attention()
        for b in range(3):
            w.hist[b] = w.all_rows(b)
            w.lens[b] += 1


def test_decode_captured_and_replayed(L):
    """A captured call replays with new lengths, inputs and pages; two graphs with a workspace each overlap."""
    t = pytest.importorskip("torch")
    w = [World(16, 4, 128, [900, 100], page=64, seed=s).fill() for s in (1, 2)]
    ws = [x.workspace(L) for x in w]
    graphs = []
    for x, s in zip(w, ws):
        assert x.decode(L, s) == capi.HY_OK
        t.cuda.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            assert x.decode(L, s) == capi.HY_OK
        graphs.append(g)
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    for lens in ([900, 100], [17, 800], [0, 15]):
        for i, x in enumerate(w):
            v = World(16, 4, 128, lens, page=64, seed=10 + i)
            v.max_pages = x.max_pages
            v.pool = x.pool
            v.table = np.full_like(x.table, -1)
            ids = v.rng.permutation(x.pool)
            at = 0
            for b in range(2):
                for k in range(v.max_pages):
                    if v.needs(b, k):
                        v.table[b, k] = ids[at]
                        at += 1
            v.rope, v.cap = x.rope, x.cap
            old = x.d
            v.fill()
            for k in old:
                old[k].view(-1)[:v.d[k].numel()].copy_(v.d[k].view(-1))
            v.d, v.o, v.new = old, x.o, x.new
            x.now = v
        t.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with t.cuda.stream(s):
                g.replay()
        t.cuda.synchronize()
        for x in w:
            x.now.check_attention()


def test_decode_refused_positions(L):
    w = World(8, 2, 128, [40, 7, 300, 90], page=16, spare=0).fill()
    ws = w.workspace(L)
    for lens, bad in (([40, -1, 300, 90], [1]), ([40, 7, w.cap, 90], [2]), ([-5, -1, 2 ** 31 - 1, -9], [0, 1, 2, 3])):
        v = World(8, 2, 128, [40, 7, 300, 90], page=16, spare=0).fill()
        ln = v.t.tensor(lens, dtype=v.t.int32, device="cuda")
        before = v.snapshot()
        assert v.decode(L, ws, len=ln.data_ptr()) == capi.HY_OK
        v.check_append(before, refused=bad)
        v.check_attention(refused=bad)
        assert guard(L) == capi.HY_GUARD_BAD_POSITION
    before = w.snapshot()
    assert w.decode(L, ws) == capi.HY_OK
    w.check_append(before)
    w.check_attention()


def test_decode_without_a_page(L):
    """Rows of a page that the table does not have are left out; with none at all in view the output is 0."""
    nq, nkv, hd = 8, 2, 64
    w = World(nq, nkv, hd, [70, 100], page=16).fill()
    w.table[0, 2] = -3
    w.d["table"].copy_(w.t.from_numpy(w.table))
    ws = w.workspace(L)
    assert w.decode(L, ws) == capi.HY_OK
    assert guard(L) == capi.HY_GUARD_BAD_INDEX
    from tests.gpu_util import assert_elementwise
    from tests.p8_util import attend
    got = w.o.cpu().numpy()
    for b in range(2):
        held, u = w.held(b), np.arange(w.lens[b] + 1)
        keep = (u // 16 != 2) if b == 0 else u >= 0
        for g in range(nkv):
            yq = w.y[b, g * 4 * hd:(g + 1) * 4 * hd].reshape(4, hd)
            o, tol = attend(yq, w.rope[w.lens[b]][None], held[0, g][keep], held[1, g][keep], u[keep], w.lens[b], 0, 0)
            assert_elementwise(got[b, g * 4 * hd:(g + 1) * 4 * hd].reshape(4, hd), o, tol)


def test_decode_nan_out_of_view_and_in_view(L):
    """A NaN row reaches exactly the outputs whose view has it (K: the whole head, V: its element)."""
    nq, nkv, hd = 4, 2, 64
    for T, at in ((100, 40), (100, 98), (111, 105)):
        for window in (8, 64, 0):
            w = World(nq, nkv, hd, [T], page=32, window=window)
            w.hist[0][0, 0, at, 3] = np.nan
            w.hist[0][1, 1, at, 5] = np.nan
            w.fill()
            ws = w.workspace(L)
            assert w.decode(L, ws) == capi.HY_OK
            got = w.o.cpu().numpy().reshape(nq, hd)
            end = T + 1
            # a closed block is NaN as a whole, an open row alone
            first = at // BLOCK * BLOCK if at // BLOCK < end // BLOCK else at
            last = first + BLOCK - 1 if at // BLOCK < end // BLOCK else at
            seen = window == 0 or last > T - window
            assert np.isnan(got[:2]).all() == seen and np.isnan(got[:2]).any() == seen
            if at // BLOCK < end // BLOCK:
                assert np.isnan(got[2:]).all() == seen
            else:
                assert np.isnan(got[2:, 5]).all() == seen
                assert not np.isnan(np.delete(got[2:], 5, 1)).any()
            if not seen:
                assert not np.isnan(got).any()


@pytest.mark.parametrize("kmul,vmul", [(1e-3, 1e4), (30.0, 1e-20), (1.0, 1e30), (1e-12, 1.0)])
def test_decode_scales(L, kmul, vmul):
    w = World(8, 2, 128, [333, 46, 31], page=32, kmul=kmul, vmul=vmul).fill()
    ws = w.workspace(L)
    assert w.decode(L, ws) == capi.HY_OK
    w.check_attention()


def test_decode_pages_past_32_bits(L):
    """A pool whose last pages begin past 2^32 bytes."""
    nq, nkv, hd, page = 4, 2, 64, 128
    w = World(nq, nkv, hd, [1000, 300], page=page, far_page=0)
    far = (1 << 32) // (nkv * page * hd + 48) + 5
    w = World(nq, nkv, hd, [1000, 300], page=page, far_page=far).fill()
    assert int(w.table[0, 0]) * w.ps > 2 ** 32
    ws = w.workspace(L)
    assert w.decode(L, ws) == capi.HY_OK
    w.check_attention()


# ------------------------------------------------------------------ prompt
@pytest.mark.parametrize("nq,nkv,hd", SHAPES)
@pytest.mark.parametrize("lens,n", [([0], [1]), ([0], [37]), ([15], [1]), ([40, 0, 7], [16, 130, 0]), ([300], [257]),
                                    ([1000, 16, 129, 5], [3, 1, 31, 200])])
def test_prompt(L, nq, nkv, hd, lens, n):
    w = World(nq, nkv, hd, lens, n, page=64, gap_rows=2).fill()
    before = w.snapshot()
    ws = w.workspace(L, prompt=True)
    assert w.append(L) == capi.HY_OK
    assert w.prompt(L, ws) == capi.HY_OK, L.hy_last_error()
    w.check_append(before)
    w.check_attention(sample=12)
    assert guard(L) == 0


@pytest.mark.parametrize("nq,nkv,hd", [(4, 2, 64), (16, 4, 128), (16, 2, 256), (2, 2, 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 16), (100, 33), (64, 2000), (200, 5), (5000, 3),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
def test_prompt_window(L, nq, nkv, hd, window, sinks):
    w = World(nq, nkv, hd, [0, 115, 500, 1500], [33, 150, 9, 64], page=16, window=window, sinks=sinks, pad_o=3, pad_y=1).fill()
    ws = w.workspace(L, prompt=True)
    assert w.append(L) == capi.HY_OK
    assert w.prompt(L, ws) == capi.HY_OK
    w.check_attention(sample=8)
    assert guard(L) == 0


@pytest.mark.parametrize("nq,nkv,hd,lens,n,window", [(16, 4, 128, [3000], [700], 0), (4, 1, 64, [9000], [5], 0),
                                                     (16, 2, 256, [2000, 4000], [130, 1], 0), (8, 4, 128, [600] * 40, [7] * 40, 300),
                                                     (8, 8, 128, [40], [1500], 0)])
def test_prompt_large(L, nq, nkv, hd, lens, n, window):
    w = World(nq, nkv, hd, lens, n, page=128, window=window, sinks=4).fill()
    ws = w.workspace(L, prompt=True)
    assert w.append(L) == capi.HY_OK
    for _ in range(2):  # the workspace is as the last call left it
        w.o.fill_(-77.0)
        assert w.prompt(L, ws) == capi.HY_OK
        w.check_attention(sample=6)


def test_prompt_refused_sequences(L):
    nq, nkv, hd = 8, 2, 64
    args = (nq, nkv, hd, [40, 7, 300, 90], [20, 5, 33, 17])
    for lens, bad in (([40, -1, 300, 90], [1]), ([40, 7, 2 ** 31 - 1, 90], [2]), ([-1, -1, -1, -1], [0, 1, 2, 3])):
        w = World(*args, page=16, spare=0).fill()
        ws = w.workspace(L, prompt=True)
        assert w.append(L) == capi.HY_OK
        ln = w.t.tensor(lens, dtype=w.t.int32, device="cuda")
        assert w.prompt(L, ws, len=ln.data_ptr()) == capi.HY_OK
        w.check_attention(refused=bad)
        assert guard(L) == capi.HY_GUARD_BAD_POSITION
    w = World(*args, page=16, spare=0).fill()
    ws = w.workspace(L, prompt=True)
    assert w.append(L) == capi.HY_OK
    start = w.t.tensor([0, 20, 25, 24, 76], dtype=w.t.int32, device="cuda")  # out of order, past the rows
    assert w.prompt(L, ws, start=start.data_ptr()) == capi.HY_OK
    assert guard(L) == capi.HY_GUARD_BAD_POSITION
    w.check_attention(refused=[2, 3])


def test_prompt_without_a_page(L):
    """Rows of a page that the table does not have are left out; a query that sees no other rows gives 0."""
    nq, nkv, hd = 4, 2, 64
    w = World(nq, nkv, hd, [32], [40], page=16).fill()
    ws = w.workspace(L, prompt=True)
    assert w.append(L) == capi.HY_OK
    w.t.cuda.synchronize()
    w.table[0, 2] = -1  # positions 32 .. 47
    w.d["table"].copy_(w.t.from_numpy(w.table))
    w.window = 8
    assert w.prompt(L, ws) == capi.HY_OK
    assert guard(L) == capi.HY_GUARD_BAD_INDEX
    from tests.gpu_util import assert_elementwise
    from tests.p8_util import attend
    got, held, u = w.o.cpu().numpy(), w.held(0), np.arange(72)
    keep = u // 16 != 2
    for i in range(40):
        t = 32 + i
        if 39 <= t <= 47:
            assert (got[i] == 0).all()
            continue
        for g in range(nkv):
            yq = w.y[i, g * 2 * hd:(g + 1) * 2 * hd].reshape(2, hd)
            o, tol = attend(yq, w.rope[t][None], held[0, g][keep], held[1, g][keep], u[keep], t, 8, 0)
            assert_elementwise(got[i, g * 2 * hd:(g + 1) * 2 * hd].reshape(2, hd), o, tol)


def test_prompt_nan_rows(L):
    """A NaN in a block or an open row reaches the queries that see it and no other."""
    nq, nkv, hd = 4, 2, 64
    w = World(nq, nkv, hd, [20], [60], page=16, window=24)
    y = w.y.reshape(60, -1, hd)
    y[20, nq, 3] = np.nan       # K head 0 at position 40: block 2, positions 32 .. 47
    y[59, nq + nkv + 1, 5] = np.nan  # V head 1 at 79, the last row, which closes the block 64 .. 79
    w.fill()
    ws = w.workspace(L, prompt=True)
    assert w.append(L) == capi.HY_OK
    assert w.prompt(L, ws) == capi.HY_OK
    got = w.o.cpu().numpy().reshape(60, nq, hd)
    for i in range(60):
        t = 20 + i
        k = t >= 32 and t - 24 < 47   # sees a row of 32 .. 47
        assert np.isnan(got[i, :2]).all() == k and np.isnan(got[i, :2]).any() == k, t
        v = t >= 64
        assert np.isnan(got[i, 2:]).all() == v and np.isnan(got[i, 2:]).any() == v, t
    w = World(nq, nkv, hd, [20], [50], page=16)
    y = w.y.reshape(50, -1, hd)
    y[47, nq + nkv, 5] = np.nan  # V head 0 at 67, an open row
    w.fill()
    ws = w.workspace(L, prompt=True)
    assert w.append(L) == capi.HY_OK
    assert w.prompt(L, ws) == capi.HY_OK
    got = w.o.cpu().numpy().reshape(50, nq, hd)
    assert np.isnan(got[47:, :2, 5]).all()
    got[47:, :2, 5] = 0
    assert not np.isnan(got).any()


def test_prompt_and_steps_together(L):
    """Prompts in chunks, then decode steps, of two sequences on one set of pages: each against the plain form."""
    nq, nkv, hd, window, sinks = 8, 2, 64, 40, 3
    t = pytest.importorskip("torch")
    w = World(nq, nkv, hd, [0, 0], [50, 21], page=16, window=window, sinks=sinks, spare=8).fill()
    w.pool_all = list(range(w.pool))
    big = World(nq, nkv, hd, [130, 100], [0, 0], page=16, seed=3, spare=4).fill()  # its pool and tails, filled with noise
    w.d |= {k: big.d[k] for k in ("K", "V", "Ks", "Vs", "tail")}
    w.pool, w.ps, w.ss, w.ts = big.pool, big.ps, big.ss, big.ts
    w.max_pages, w.cap, w.rope = big.max_pages, big.cap, big.rope
    w.d["rope"] = big.d["rope"]
    ids = w.rng.permutation(w.pool)
    w.table = np.full((2, w.max_pages), -1, dtype=np.int32)
    at = 0
    for n in ([50, 21], [0, 40], [30, 3]):
        w.n = n
        w.start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        w.rows = sum(n)
        for b in range(2):
            for i in range((w.lens[b] + n[b]) // 16):
                if w.table[b, i] < 0:
                    w.table[b, i] = ids[at]
                    at += 1
        w.y = w.rng.standard_normal((w.rows, w.ldy)).astype(np.float32)
        w.d |= dict(y=t.from_numpy(w.y).cuda(), start=t.from_numpy(w.start).cuda(), table=t.from_numpy(w.table).cuda(),
                    len=t.tensor(w.lens, dtype=t.int32, device="cuda"))
        w.o = t.full((w.rows, w.ldo), -77.0, device="cuda")
        w.new = t.full((w.rows, 2, nkv, hd), -77.0, device="cuda")
        before = w.snapshot()
        ws = w.workspace(L, prompt=True)
        assert w.append(L) == capi.HY_OK and w.prompt(L, ws) == capi.HY_OK
        w.check_append(before)
        w.check_attention()
        for b in range(2):
            w.hist[b] = w.all_rows(b)
            w.lens[b] += n[b]
    w.n, w.rows, w.start = [1, 1], 2, np.array([0, 1, 2], dtype=np.int32)
    ws = w.workspace(L)
    w.o = t.full((2, w.ldo), -77.0, device="cuda")
    w.new = t.full((2, 2, nkv, hd), -77.0, device="cuda")
    for _ in range(20):
        for b in range(2):
            for i in range((w.lens[b] + 1) // 16):
                if w.table[b, i] < 0:
                    w.table[b, i] = ids[at]
                    at += 1
        w.y = w.rng.standard_normal((2, w.ldy)).astype(np.float32)
        w.d |= dict(y=t.from_numpy(w.y).cuda(), table=t.from_numpy(w.table).cuda(), len=t.tensor(w.lens, dtype=t.int32, device="cuda"))
        before = w.snapshot()
        assert w.decode(L, ws) == capi.HY_OK
        w.check_append(before)
        w.check_attention()
        for b in range(2):
            w.hist[b] = w.all_rows(b)
            w.lens[b] += 1
    assert guard(L) == 0


# ------------------------------------------------------------------ every row once
def equal_weights(nq, nkv, hd, lens, n=None, **kw):
    """q = 0 and V of +-127: all rows in view weigh the same, V's codes and sums are exact, and the output is their mean."""
    w = World(nq, nkv, hd, lens, n, **kw)
    rng = w.rng
    for b, T in enumerate(w.lens):
        w.hist[b][1] = 127 * (2 * rng.integers(0, 2, w.hist[b][1].shape) - 1)
    w.y[:, :nq * hd] = 0
    v = w.y[:, (nq + nkv) * hd:(nq + 2 * nkv) * hd]
    v[:] = 127 * (2 * rng.integers(0, 2, v.shape) - 1)
    return w.fill()


def check_means(w):
    """sum / n with the reciprocal and the product rounded once each (2^-24 of the value each): below 2^-22."""
    w.t.cuda.synchronize()
    nq, nkv, hd = w.nq, w.nkv, w.hd
    got = w.o.cpu().numpy()[:, :nq * hd].reshape(-1, nkv, nq // nkv, hd)
    for b in range(w.B):
        v = w.all_rows(b)[1].astype(np.float64)  # [nkv, T + n, hd]
        csum = np.concatenate([np.zeros((nkv, 1, hd)), v.cumsum(1)], 1)
        for i in range(w.n[b]):
            t = w.lens[b] + i
            lo = max(0, t - w.window + 1) if w.window else 0
            s = min(w.sinks, lo) if w.window else 0
            mean = (csum[:, t + 1] - csum[:, lo] + csum[:, s]) / (t + 1 - lo + s)
            err = np.abs(got[w.start[b] + i] - mean[:, None])
            assert (err <= 2.0 ** -22 * np.abs(mean[:, None])).all(), (b, i, err.max())


@pytest.mark.parametrize("nq,nkv,hd", [(4, 2, 64), (16, 4, 128), (8, 1, 128), (16, 2, 256), (4, 2, 256), (8, 8, 128)])
@pytest.mark.parametrize("lens,window,sinks", [([0], 0, 0), ([40000], 0, 0), ([9000, 17, 3333, 128, 2047], 0, 0),
                                               ([9000, 17, 3333, 128, 2047, 700], 500, 20), ([20000] * 3, 12345, 100)])
def test_decode_takes_every_row_once(L, nq, nkv, hd, lens, window, sinks):
    w = equal_weights(nq, nkv, hd, lens, page=64, window=window, sinks=sinks)
    ws = w.workspace(L)
    assert w.decode(L, ws) == capi.HY_OK
    check_means(w)


@pytest.mark.parametrize("nq,nkv,hd", [(4, 2, 64), (16, 4, 128), (8, 1, 128), (16, 2, 256), (4, 2, 256), (8, 8, 128)])
@pytest.mark.parametrize("lens,n,window,sinks", [([0], [300], 0, 0), ([5000], [3], 0, 0), ([1000, 17, 133, 128], [70, 200, 1, 33], 0, 0),
                                                 ([3000, 17, 133, 128], [70, 200, 1, 33], 500, 20), ([2000], [700], 129, 17)])
def test_prompt_takes_every_row_once(L, nq, nkv, hd, lens, n, window, sinks):
    w = equal_weights(nq, nkv, hd, lens, n, page=64, window=window, sinks=sinks)
    ws = w.workspace(L, prompt=True)
    assert w.append(L) == capi.HY_OK
    assert w.prompt(L, ws) == capi.HY_OK
    check_means(w)


# ------------------------------------------------------------------ as programs call them
def test_same_bits_again(L):
    """Nothing depends on the order in which CTAs arrive."""
    t = pytest.importorskip("torch")
    w = World(16, 4, 128, [5000, 300, 47], page=64).fill()
    ws = w.workspace(L)
    assert w.decode(L, ws) == capi.HY_OK
    t.cuda.synchronize()
    first = w.o.clone()
    for _ in range(10):
        assert w.decode(L, ws) == capi.HY_OK
        t.cuda.synchronize()
        assert t.equal(first, w.o)
    w = World(16, 4, 128, [900, 300], [500, 40], page=64).fill()
    ws = w.workspace(L, prompt=True)
    assert w.append(L) == capi.HY_OK and w.prompt(L, ws) == capi.HY_OK
    t.cuda.synchronize()
    first = w.o.clone()
    for _ in range(10):
        assert w.prompt(L, ws) == capi.HY_OK
        t.cuda.synchronize()
        assert t.equal(first, w.o)


@pytest.mark.parametrize("nq,nkv,hd", [(4, 2, 64), (16, 4, 128), (16, 2, 256)])
def test_decode_without_values_unaligned(L, nq, nkv, hd):
    """kv_new null; y and o at addresses of no alignment of their own."""
    w = World(nq, nkv, hd, [33, 15, 500], page=32, pad_y=1, pad_o=1).fill()
    t = w.t
    y = t.empty(w.d["y"].numel() + 1, device="cuda")[1:].view_as(w.d["y"]).copy_(w.d["y"])
    o = t.full((w.o.numel() + 1,), -77.0, device="cuda")[1:].view_as(w.o)
    before = w.snapshot()
    ws = w.workspace(L)
    assert w.decode(L, ws, new=False, y=y.data_ptr(), o=o.data_ptr()) == capi.HY_OK
    w.check_append(before, new=False)
    w.o = o
    w.check_attention()


def test_prompt_captured_and_on_two_streams(L):
    """Append and prompt attention in one graph each, replayed on two streams at once with new rows."""
    t = pytest.importorskip("torch")
    worlds = [World(8, 2, 128, [40, 0], [200, 33], page=32, seed=s).fill() for s in (1, 2)]
    graphs = []
    for w in worlds:
        w.ws = w.workspace(L, prompt=True)
        assert w.append(L) == capi.HY_OK and w.prompt(L, w.ws) == capi.HY_OK
        t.cuda.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            assert w.append(L) == capi.HY_OK and w.prompt(L, w.ws) == capi.HY_OK
        graphs.append(g)
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    for _ in range(3):
        for w in worlds:
            w.y[:] = w.rng.standard_normal(w.y.shape).astype(np.float32)
            w.d["y"].copy_(t.from_numpy(w.y))
            # the tail's old rows again: the last replay's open block has taken their place
            for b, T in enumerate(w.lens):
                rest = w.hist[b][:, :, T // BLOCK * BLOCK:]
                tl = w.d["tail"][b * w.ts:b * w.ts + 2 * w.nkv * BLOCK * w.hd].view(2, w.nkv, BLOCK, w.hd)
                tl[:, :, :T % BLOCK] = t.from_numpy(rest.copy()).cuda().bfloat16()
            w.o.fill_(-77.0)
        t.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with t.cuda.stream(s):
                g.replay()
        t.cuda.synchronize()
        for w in worlds:
            w.check_attention(sample=8)


def test_prompt_of_many_sequences(L):
    """256 sequences of up to three rows, some with none."""
    n = [i % 4 for i in range(256)]
    w = World(4, 2, 64, [(37 * i) % 300 for i in range(256)], n, page=16).fill()
    before = w.snapshot()
    ws = w.workspace(L, prompt=True)
    assert w.append(L) == capi.HY_OK
    w.check_append(before)
    assert w.prompt(L, ws) == capi.HY_OK
    w.check_attention()
    assert guard(L) == 0


def test_prompt_pages_past_32_bits(L):
    nq, nkv, hd, page = 4, 2, 64, 128
    far = (1 << 32) // (nkv * page * hd + 48) + 5
    w = World(nq, nkv, hd, [300, 100], [40, 200], page=page, far_page=far).fill()
    assert int(w.table[0, 0]) * w.ps > 2 ** 32
    before = w.snapshot()
    ws = w.workspace(L, prompt=True)
    assert w.append(L) == capi.HY_OK and w.prompt(L, ws) == capi.HY_OK
    w.check_append(before)
    w.check_attention(sample=8)


def test_decode_closes_a_block_without_a_page(L):
    """The block that closes has no page: nothing is written, its rows are attended to all the same."""
    w = World(8, 2, 64, [47, 31], page=16).fill()
    w.table[0, 2] = w.pool + 5
    w.d["table"].copy_(w.t.from_numpy(w.table))
    before = w.snapshot()
    ws = w.workspace(L)
    assert w.decode(L, ws) == capi.HY_OK
    assert guard(L) == capi.HY_GUARD_BAD_INDEX
    w.check_append(before, lost={(0, 2)})
    w.check_attention()
