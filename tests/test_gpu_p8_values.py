"""The paged 8-bit KV cache's attention over keys and values of unlike sizes: zero, tiny and
large ones.

Against the plain form of tests/p8_util.py with its tolerances; every output is first checked to be finite, as a comparison
with a bound does not fail for NaN."""
import numpy as np
import pytest

from bandwidth_bound_hybrid_gb300 import capi
from tests.p8_util import BLOCK, World, to_bf16

pytestmark = pytest.mark.gpu
K, V = 0, 1


@pytest.fixture(scope="module")
def L(gpu):
    from bandwidth_bound_hybrid_gb300 import build
    build.build()
    return capi.lib()


def scale_rows(w, b, which, lo, hi, mul):
    """K or V of sequence b's positions lo .. hi - 1, old and new, times mul (a power of two or 0: exact)."""
    T, at = w.lens[b], (w.nq + which * w.nkv) * w.hd
    h = w.hist[b][which, :, lo:min(hi, T)]
    h[...] = to_bf16(h * np.float32(mul))
    first = w.start[b] - T
    w.y[first + max(lo, T):first + min(hi, T + w.n[b]), at:at + w.nkv * w.hd] *= np.float32(mul)


def finite(w):
    w.t.cuda.synchronize()
    got = w.o.cpu().numpy()[:, :w.nq * w.hd]
    assert np.isfinite(got).all(), np.argwhere(~np.isfinite(got))[:4].tolist()


def decode(L, w):
    w.fill()
    ws = w.workspace(L)
    assert w.decode(L, ws) == capi.HY_OK, L.hy_last_error()
    finite(w)
    w.check_attention()


def prompt(L, w, sample=None):
    w.fill()
    ws = w.workspace(L, prompt=True)
    assert w.append(L) == capi.HY_OK
    assert w.prompt(L, ws) == capi.HY_OK, L.hy_last_error()
    finite(w)
    w.check_attention(sample=sample)


SHAPES = [(2, 2, 64), (8, 1, 64), (16, 4, 128), (16, 2, 256)]
# windows and sinks that end inside blocks, and a view of everything
VIEWS = [(8, 0), (24, 0), (24, 4), (1, 20), (40, 33), (0, 0)]


def zero_keys(w, mul):
    """Sequences in turn: all of K, or every other block of it, times mul."""
    for b, T in enumerate(w.lens):
        for j in range(0, T + w.n[b], BLOCK * (1 + b % 2)):
            scale_rows(w, b, K, j, j + BLOCK, mul)


@pytest.mark.parametrize("nq,nkv,hd", SHAPES)
@pytest.mark.parametrize("window,sinks", VIEWS)
@pytest.mark.parametrize("mul", [0.0, 2.0 ** -105])
def test_decode_blocks_of_scale_zero(L, nq, nkv, hd, window, sinks, mul):
    """Blocks of K whose scale is 0 (closed before, by the call, or still open), cut by the window and by the sinks."""
    w = World(nq, nkv, hd, [100, 100, 111, 127, 95, 40, 15, 47, 0], page=16, window=window, sinks=sinks)
    zero_keys(w, mul)
    decode(L, w)


@pytest.mark.parametrize("nq,nkv,hd", SHAPES)
@pytest.mark.parametrize("window,sinks", VIEWS)
@pytest.mark.parametrize("mul", [0.0, 2.0 ** -105])
def test_prompt_blocks_of_scale_zero(L, nq, nkv, hd, window, sinks, mul):
    w = World(nq, nkv, hd, [100, 90, 0, 31], [37, 38, 21, 1], page=16, window=window, sinks=sinks)
    zero_keys(w, mul)
    prompt(L, w)


@pytest.mark.parametrize("nq,nkv,hd", SHAPES)
@pytest.mark.parametrize("qmul,kmul,vmul", [(0.0, 0.0, 1.0), (2.0 ** -60, 0.0, 1.0), (2.0 ** -60, 2.0 ** -110, 1.0), (0.0, 2.0 ** -110, 1.0),
                                            (0.0, 0.0, 0.0)])
def test_zero_queries_over_zero_keys(L, nq, nkv, hd, qmul, kmul, vmul):
    """Queries and keys of zero or nearly: the mean of V in view (an idle slot, a first call on zeroed inputs)."""
    decode(L, World(nq, nkv, hd, [0, 5, 15, 16, 20, 100], page=16, qmul=qmul, kmul=kmul, vmul=vmul))
    prompt(L, World(nq, nkv, hd, [0, 5, 16, 100], [1, 7, 30, 12], page=16, qmul=qmul, kmul=kmul, vmul=vmul))


def one_hot(nq, nkv, hd, T, n, size):
    """Scores of up to 2^size, all far apart: no rotation, q and K along one axis, K's values a permutation of 0 .. 100
    and their multiples."""
    w = World(nq, nkv, hd, [T], n and [n], page=16)
    w.rope[..., 0], w.rope[..., 1] = 1, 0
    w.y[:, :(nq + nkv) * hd] = 0
    a = 2.0 ** ((size - 7) // 2)
    w.y[:, :nq * hd:hd] = a * np.where(np.arange(nq) % 2, -1, 1)
    val = (np.arange(T + (n or 1)) * 37 % 101 * a).astype(np.float32)
    w.hist[0][K] = 0
    w.hist[0][K, :, :, 0] = val[:T]
    w.y[:, nq * hd:(nq + nkv) * hd:hd] = val[T:, None]
    return w


@pytest.mark.parametrize("nq,nkv,hd", SHAPES)
@pytest.mark.parametrize("size", [21, 27, 31, 41, 61, 101])
def test_large_scores(L, nq, nkv, hd, size):
    """One row has all of the weight (largest or smallest K, by the query's sign): no overflow on the way there.

    The values of K are 1/100 of the largest apart and a block's codes move them by at most 1/254 of it, so two never meet.  The
    largest score is at least 2^(size - 4), so scores differ by 2^(size - 4) (0.01 - 2/254) > 2^(size - 13), and FP32 errs by
    at most 2 gamma(2 hd + 16) of the largest, 2^(size - 14) / 2^4."""
    decode(L, one_hot(nq, nkv, hd, 99, None, size))
    prompt(L, one_hot(nq, nkv, hd, 60, 40, size))
