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
    new = w.y[w.start[b]:w.start[b + 1]]
    new[max(lo - T, 0):max(hi - T, 0), at:at + w.nkv * w.hd] *= np.float32(mul)


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


# ------------------------------------------------------------------ V far apart
FAR = [2.0 ** 30, 2.0 ** 60, 2.0 ** 100]


def sizes(w, b):
    """Largest |V| [nkv, rows] of each row's closed block, or of the open row itself."""
    a = np.abs(w.all_rows(b)[1].astype(np.float64)).max(-1)
    nb = a.shape[1] // BLOCK * BLOCK
    a[:, :nb] = np.repeat(a[:, :nb].reshape(w.nkv, -1, BLOCK).max(-1), BLOCK, 1)
    return a


def check_apart(w, sample=40):
    """check_attention with the bound that holds where V's sizes A_t (of a block; an open row) are far apart: instead of n 2^-37
    max |V| for the weights' two fp16 parts, for each row in view 2^-34 (max p |V_td| + max_u p_u A_u).

    A weight p_t s_t (s_t = A_t / 127) is rounded twice at half of fp16's spacing below its normal range, 2^-25, where 2^E
    counts 2^14: 2^-38 2^E.  In a step whose scales are within 2^4, 2^E <= 2^5 s_t, times |c_td| <= 127: below 2^-33 |V_td| of
    the largest weight; the exponents' difference of at most 3 makes 2^E / s_t at most 2^4, so 2^-34.  In other steps 2^E <= 4
    max_u p_u s_u, times 127: 2^-36 max_u p_u A_u; an open row's power of two may be twice A / 127: 2^-35."""
    from tests.gpu_util import U32, assert_elementwise, gamma, rope_pair_abs
    from tests.p8_util import rotate32
    got, G, hd = w.o.cpu().numpy(), w.nq // w.nkv, w.hd
    for b in range(w.B):
        held, size, T, n = w.held(b), sizes(w, b), w.lens[b], w.n[b]
        for i in sorted(set(range(n)) if n <= sample else set(w.rng.choice(n, sample, replace=False).tolist()) | {n - 1}):
            t, u = T + i, np.arange(T + n)
            seen = (u <= t) & ((u < w.sinks) | (u > t - w.window) if w.window else True)
            for g in range(w.nkv):
                yq = w.y[w.start[b] + i, g * G * hd:(g + 1) * G * hd].reshape(G, hd).astype(np.float64)
                k, v, a = held[0, g][seen], held[1, g][seen], size[g][seen]
                q, scale = rotate32(yq, w.rope[t][None].astype(np.float64)), 1 / np.sqrt(hd)
                s = (q @ k.T) * scale
                top = s.max(-1, keepdims=True)
                p = np.exp(s - top)
                p /= p.sum(-1, keepdims=True)
                o, ak, aq = p @ v, np.abs(k), np.abs(q)
                delta = (2 * gamma(2 * hd + 16) + 2.0 ** -21) * scale * (aq @ ak.T)
                delta += 6 * U32 * scale * (np.stack([rope_pair_abs(y) for y in yq]) @ ak.T)
                delta += 2.0 ** -33 * scale * aq.max(-1, keepdims=True) * ak.sum(-1)
                e = (delta + 2.0 ** -20 + 4 * U32 * (np.abs(s) + np.abs(top) + 32)) * p
                tol = np.einsum("gt,gtd->gd", e, np.abs(v[None] - o[:, None]))
                tol += 2 * gamma(len(u) // 8 + 64) * (p @ np.abs(v)) + 16 * U32 * np.abs(o) + 1e-30
                tol += 2.0 ** -34 * (p.max(-1, keepdims=True) * np.abs(v).sum(0) + len(v) * (p * a).max(-1, keepdims=True))
                at = got[w.start[b] + i, g * G * hd:(g + 1) * G * hd].reshape(G, hd)
                assert_elementwise(at, o, tol, f"sequence {b}, row {i}, kv head {g}")


def run_apart(L, w, sample=40):
    w.fill()
    ws = w.workspace(L, prompt=True)
    assert w.append(L) == capi.HY_OK
    assert w.prompt(L, ws) == capi.HY_OK, L.hy_last_error()
    finite(w)
    check_apart(w, sample)


@pytest.mark.parametrize("nq,nkv,hd", SHAPES)
@pytest.mark.parametrize("mul", FAR)
def test_prompt_values_out_of_view(L, nq, nkv, hd, mul):
    """Large rows of V in a later block, or in one that the window has left, take no bits from rows that do not see them.

    A row that sees part of a closed block sees it with the block's scale, which the large rows have set (its codes say so too:
    those of the small rows are 0), so such a row's bound has the block's size even where the large rows are out of view, by
    the arithmetic of check_apart.  Rows that see none of the block have no such term."""
    w = World(nq, nkv, hd, [0, 90], [200, 70], page=16)
    scale_rows(w, 0, V, 115, 117, mul)
    scale_rows(w, 1, V, 131, 132, mul)
    run_apart(L, w, sample=300)
    w = World(nq, nkv, hd, [0, 200], [200, 24], page=16, window=40)
    scale_rows(w, 0, V, 35, 37, mul)
    scale_rows(w, 1, V, 170, 171, mul)
    run_apart(L, w, sample=300)
    w = World(nq, nkv, hd, [0], [150], page=16, window=20, sinks=5)
    scale_rows(w, 0, V, 9, 10, mul)  # a row of a sinks' block that is no sink itself: its block's codes are
    scale_rows(w, 0, V, 64, 65, mul)
    run_apart(L, w, sample=300)


@pytest.mark.parametrize("nq,nkv,hd", SHAPES)
@pytest.mark.parametrize("mul", [2.0 ** -60, 2.0 ** 10, *FAR])
def test_prompt_values_of_no_weight(L, nq, nkv, hd, mul):
    """A block in view whose V is far larger or smaller, with weights of about 2^-60: the others keep their bits."""
    w = World(nq, nkv, hd, [0, 70], [128, 60], page=16)
    w.rope[..., 0], w.rope[..., 1] = 1, 0
    w.y[:, :nq * hd] = 0
    w.y[:, :nq * hd:hd] = 4 * np.sqrt(hd)
    for b, lo in ((0, 32), (1, 48)):
        scale_rows(w, b, K, lo, lo + BLOCK, 0)
        scale_rows(w, b, V, lo, lo + BLOCK, mul)
    w.hist[1][K, :, 48:64, 0] = -10
    w.y[32:48, nq * hd:(nq + nkv) * hd:hd] = -10
    run_apart(L, w)


@pytest.mark.parametrize("nq,nkv,hd", SHAPES)
@pytest.mark.parametrize("span", [2, 6, 20, 90])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 20)])
def test_prompt_values_far_apart(L, nq, nkv, hd, span, window, sinks):
    """Every block of V of a size of its own, 2^-span to 2^span, some of them zero."""
    w = World(nq, nkv, hd, [0, 300], [256, 52], page=16, window=window, sinks=sinks)
    for b in range(2):
        for lo in range(0, w.lens[b] + w.n[b], BLOCK):
            scale_rows(w, b, V, lo, lo + BLOCK, 0.0 if w.rng.random() < 0.1 else 2.0 ** int(w.rng.integers(-span, span + 1)))
    run_apart(L, w)


def test_prompt_wide_steps_twice_and_nan(L):
    """Wide steps give the same bits again; a NaN block among far apart ones reaches the rows that see it and no others."""
    nq, nkv, hd = 16, 4, 128
    w = World(nq, nkv, hd, [0], [400], page=16, window=150)
    scale_rows(w, 0, V, 64, 80, 2.0 ** 50)
    scale_rows(w, 0, V, 200, 216, 2.0 ** 50)
    w.y.reshape(400, -1, hd)[130, nq + nkv:, 7] = np.nan  # V of all heads: block 128 .. 143
    w.fill()
    ws = w.workspace(L, prompt=True)
    assert w.append(L) == capi.HY_OK
    first = None
    for _ in range(3):
        assert w.prompt(L, ws) == capi.HY_OK
        w.t.cuda.synchronize()
        bits = w.o.view(w.t.int32).clone()
        assert first is None or w.t.equal(first, bits)
        first = bits
    got = w.o.cpu().numpy()
    t = np.arange(400)
    sees = (t >= 128) & (t - 150 < 143)
    assert np.isnan(got[sees]).all() and np.isfinite(got[~sees]).all()


@pytest.mark.parametrize("nq,nkv,hd", SHAPES)
@pytest.mark.parametrize("which", [K, V])
@pytest.mark.parametrize("mul", [2.0 ** -60, *FAR])
def test_prompt_open_rows_out_of_view(L, nq, nkv, hd, which, mul):
    """Rows of the open block, which are bf16 each for itself: later ones, or ones that the window has left, are of no matter."""
    w = World(nq, nkv, hd, [0, 37, 100], [200, 9, 13], page=16)
    for b, at in ((0, 198), (1, 45), (2, 112)):
        scale_rows(w, b, which, at, at + 1, mul)
    run_apart(L, w, sample=300)
    w = World(nq, nkv, hd, [180, 5], [27, 10], page=16, window=5, sinks=1)
    for b, at in ((0, 193), (1, 2), (1, 9)):
        scale_rows(w, b, which, at, at + 1, mul)
    run_apart(L, w, sample=300)


@pytest.mark.parametrize("nq,nkv,hd", SHAPES)
@pytest.mark.parametrize("span", [2, 20, 90])
def test_prompt_open_rows_far_apart(L, nq, nkv, hd, span):
    """V of every open row of a size of its own, beside closed blocks of one size; rows of zeros among them."""
    w = World(nq, nkv, hd, [0, 37, 160], [95, 9, 15], page=16)
    for b in range(3):
        end = w.lens[b] + w.n[b]
        for t in range(end // BLOCK * BLOCK, end):
            scale_rows(w, b, V, t, t + 1, 0.0 if w.rng.random() < 0.1 else 2.0 ** int(w.rng.integers(-span, span + 1)))
    run_apart(L, w)
