"""The paged 8-bit cache's decode attention is limited by the blocks in view, not by the capacity that a window never shows."""
import ctypes

import numpy as np
import pytest

from bandwidth_bound_hybrid_gb300 import capi
from tests.p8_util import World
from tests.test_op_refusals import without_a_gpu


@pytest.fixture(scope="module")
def L():
    from bandwidth_bound_hybrid_gb300 import build
    build.build()
    return capi.lib()


CALL = """
import ctypes
def call(max_pages, window, sinks, batch=256):
    kv = capi.hy_kv_p8(A, A, A, A, 2 * 128 * 64, 2 * 8, 128, 9, A, 64 * 2 * 64, A, max_pages)
    return L.hy_op_attention_p8(A, 12 * 64, batch, ctypes.byref(kv), 8, 2, 64, window, sinks, A, A, A, 8 * 64, None, A, None)
"""


def test_a_window_bounds_the_list_of_tiles(L):
    """2^24 pages of 128 rows: 256 x 2 heads x 2^27 blocks are past 2^30, those of a window of 4096 are not (the calls that pass
    end at the missing GPU)."""
    views = [(0, 0), (4096, 4), (1 << 26, 0), (4096, 1 << 26), (2 ** 31 - 1, 2 ** 31 - 1), ((1 << 25) - 16, 0), ((1 << 25) - 32, 0)]
    r = without_a_gpu(CALL + f"print(*[call(1 << 23, w, s) for w, s in {views}])")
    assert r.returncode == 0, r.stderr[-2000:]
    no, ok = str(capi.HY_ERR_UNSUPPORTED), str(capi.HY_ERR_CUDA)
    # 2^30 / 512 = 2^21 blocks: window / 16 + 2
    assert r.stdout.split() == [no, ok, no, no, no, no, ok]


@pytest.mark.gpu
def test_windowed_decode_over_a_large_capacity(gpu, L):
    """256 sequences x 8 heads x 129 pages of 65536 rows (past 2^34 rows) under a window of 100: as over a small capacity."""
    lens = [i % 16 for i in range(252)] + [47, 300, 701, 95]
    w = World(8, 8, 64, lens, page=65536, window=100, sinks=4, spare=0).fill()
    t, pages = w.t, 129
    assert 256 * 8 * pages * 65536 > 1 << 34
    table = np.full((256, pages), -5, dtype=np.int32)
    table[:, :w.max_pages] = w.table
    table = t.from_numpy(table).cuda()
    rope = t.empty((pages * 65536, 32, 2), device="cuda")
    rope[:w.cap] = w.d["rope"]
    kv = w.kv(table=table.data_ptr(), max_pages=pages)
    before = w.snapshot()
    ws = w.workspace(L)
    assert w.decode(L, ws, kv=ctypes.byref(kv), rope=rope.data_ptr()) == capi.HY_OK, L.hy_last_error()
    w.check_append(before)
    w.check_attention()
    assert np.isfinite(w.o.cpu().numpy()).all()
    assert w.decode(L, ws, kv=ctypes.byref(kv), rope=rope.data_ptr(), window=0) == capi.HY_ERR_UNSUPPORTED
