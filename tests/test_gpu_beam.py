"""Beam selection (hy_op_beam_select) and state reordering (hy_op_beam_reorder)
against plain FP64 / numpy forms.

Scores: |error| <= 2^-19 + 2^-24 |score|.  The last is the rounding of the FP32
output; lse errs by the relative error of the FP32 sum of exponentials: at
most 2^-21 of each ex2.approx and its argument's rounding (an argument below 8
in the terms that matter: 2^-22), and gamma(16 + 16) of the sums in a lane,
across the CTA and its carries (the chunks are added in FP64); the constant
log2 e of FP32 moves lse by 2^-26 times the distance of the mean logit from
the largest, 2^-22 below a distance of 16.
Picks have to be equal: wherever the reference has two candidates of
different beams closer than twice that bound the case would be ambiguous, so
every case asserts that it has none (within a beam the logits' order is
exact, and equal beams have equal sums)."""
import numpy as np
import pytest

from bandwidth_bound_hybrid_gb300 import capi
from tests.gpu_util import to_np

pytestmark = pytest.mark.gpu

LSE = 2.0 ** -19


@pytest.fixture(scope="module")
def L(gpu):
    from bandwidth_bound_hybrid_gb300 import build
    build.build()
    return capi.lib()


def _torch():
    import torch
    return torch


def select_ref(logits, score, done, eos, groups, beams, picks):
    """score, parent, token, done of the picks, and the smallest gap between neighbours of different beams."""
    V = logits.shape[1]
    x = logits.astype(np.float64).reshape(groups, beams, V)
    x = np.where(np.isnan(x), -np.inf, x)
    sc = score.astype(np.float64).reshape(groups, beams)
    dn = np.zeros((groups, beams), dtype=bool) if done is None else done.reshape(groups, beams) != 0
    out = [np.zeros((groups, picks)), *(np.zeros((groups, picks), dtype=np.int64) for _ in range(3))]
    gap = np.inf
    with np.errstate(all="ignore"):
        for g in range(groups):
            s = np.full((beams, V), -np.inf)
            for w in range(beams):
                if dn[g, w]:
                    if np.isfinite(sc[g, w]):
                        s[w, eos] = sc[g, w]
                    continue
                m = x[g, w].max()
                off = sc[g, w] - (m + np.log(np.exp(x[g, w] - m).sum()))
                if np.isfinite(off):
                    s[w] = off + x[g, w]
            f = s.ravel()
            order = np.lexsort((np.arange(f.size), -f))[:picks + 1]
            for a, b in zip(order, order[1:]):
                if a // V != b // V and np.isfinite(f[b]) and f[a] != f[b]:
                    gap = min(gap, f[a] - f[b])
            order = order[:picks]
            out[0][g], out[1][g], out[2][g] = f[order], order // V, order % V
            out[3][g] = dn[g][order // V] | (order % V == eos)
    return out, gap


def run_select(L, logits, score, done, eos, groups, beams, picks, ld=None, ws=None, inplace=False):
    torch = _torch()
    V = logits.shape[1]
    ld = ld or V
    buf = np.full((groups * beams, ld), 1e30, dtype=np.float32)
    buf[:, :V] = logits
    d = torch.from_numpy(buf).cuda()
    s = torch.from_numpy(score.astype(np.float32)).cuda()
    dn = None if done is None else torch.from_numpy(done.astype(np.int32)).cuda()
    if ws is None:
        n = L.hy_op_beam_select_workspace(groups, beams, V)
        assert n > 0
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    so = s if inplace else torch.full((groups, picks), 77.0, device="cuda")
    po, to, do = (torch.full((groups, picks), -7, dtype=torch.int32, device="cuda") for _ in range(3))
    if inplace and dn is not None:
        do = dn
    st = torch.cuda.current_stream().cuda_stream
    rc = L.hy_op_beam_select(d.data_ptr(), ld, groups, beams, V, picks, s.data_ptr(), None if dn is None else dn.data_ptr(),
                             eos, so.data_ptr(), po.data_ptr(), to.data_ptr(), do.data_ptr(), ws.data_ptr(), st)
    assert rc == 0, L.hy_last_error()
    torch.cuda.synchronize()
    return [to_np(t).reshape(groups, picks) for t in (so, po, to, do)]


def check(got, logits, score, done, eos, groups, beams, picks):
    ref, gap = select_ref(logits, score, done, eos, groups, beams, picks)
    with np.errstate(all="ignore"):
        big = 2 * (LSE + 2.0 ** -24 * np.nanmax(np.abs(np.where(np.isfinite(ref[0]), ref[0], 0))))
    assert gap > big, f"ambiguous case: two beams' candidates {gap:.3g} apart"
    for a, b, name in zip(got[1:], ref[1:], ("parent", "token", "done")):
        np.testing.assert_array_equal(a, b, err_msg=name)
    fin = np.isfinite(ref[0])
    np.testing.assert_array_equal(np.isneginf(got[0]), ~fin)
    err = np.abs(got[0][fin] - ref[0][fin])
    assert (err <= LSE + 2.0 ** -24 * np.abs(ref[0][fin])).all(), err.max()


def inputs(groups, beams, V, seed, spread=2.5):
    rng = np.random.default_rng(seed)
    logits = (rng.standard_normal((groups * beams, V)) * spread).astype(np.float32)
    score = (-20 * rng.random(groups * beams) - 1).astype(np.float32)
    return rng, logits, score


@pytest.mark.parametrize("groups,beams,V,picks", [
    (1, 1, 1, 1), (1, 1, 2, 2), (1, 2, 3, 6), (3, 2, 31, 4), (1, 4, 1024, 4), (2, 8, 4096, 8), (2, 8, 4097, 16),
    (1, 16, 5000, 32), (5, 3, 12289, 6), (1, 1, 151936, 32), (70, 1, 700, 2), (1, 7, 33000, 9),
    (8, 16, 60000, 8), (130, 2, 40001, 3), (1000, 1, 4500, 2)])
def test_select(L, groups, beams, V, picks):
    _, logits, score = inputs(groups, beams, V, V + picks)
    got = run_select(L, logits, score, None, -1, groups, beams, picks, ld=V + (V % 3))
    check(got, logits, score, None, -1, groups, beams, picks)


def test_select_first_step(L):
    """Only the first beam counts (the others start at -infinity)."""
    _, logits, score = inputs(2, 4, 9000, 1)
    score.reshape(2, 4)[:, 1:] = -np.inf
    check(run_select(L, logits, score, None, 5, 2, 4, 4), logits, score, None, 5, 2, 4, 4)


def test_select_ended_beams(L):
    rng, logits, score = inputs(6, 8, 5000, 2)
    done = (rng.random(48) < 0.4).astype(np.int32)
    done[:8] = 1  # a group whose beams have all ended: 8 picks go on, the rest have no probability
    logits[:, 2] += 12  # ending is likely
    score *= 0.2
    for picks in (8, 16):
        got = run_select(L, logits, score, done, 2, 6, 8, picks)
        check(got, logits, score, done, 2, 6, 8, picks)
    got = run_select(L, logits, score, done, 2, 6, 8, 8, inplace=True)
    check(got, logits, score, done, 2, 6, 8, 8)
    # an ended beam's logits are not read
    logits.reshape(6, 8, -1)[done.reshape(6, 8) != 0] = np.nan
    check(run_select(L, logits, score, done, 2, 6, 8, 8), logits, score, done, 2, 6, 8, 8)


def test_select_masked_tokens(L):
    """Most tokens masked with -infinity, the type's lowest value or NaN; rows with fewer finite tokens than picks, with none, with +infinity."""
    rng, logits, score = inputs(4, 3, 8200, 3)
    keep = rng.random(logits.shape) < 0.002
    masked = np.where(keep, logits, -np.inf).astype(np.float32)
    masked[3:6] = np.where(keep[3:6], logits[3:6], np.finfo(np.float32).min)
    masked[6:9] = np.where(keep[6:9], logits[6:9], np.nan)
    masked[9] = -np.inf
    masked[10] = -np.inf
    masked[10, [4, 8000]] = [1.0, 2.0]
    masked[11, 17] = np.inf
    for picks in (1, 6, 20):
        got = run_select(L, masked, score, None, 4, 4, 3, picks)
        check(got, masked, score, None, 4, 4, 3, picks)
    lowest = np.full_like(masked, np.finfo(np.float32).min)  # every token alike, at the lowest value
    check(run_select(L, lowest, score, None, 4, 4, 3, 6), lowest, score, None, 4, 4, 3, 6)
    masked[9:] = np.nan  # nothing at all: the first candidates in index order, with score -infinity
    got = run_select(L, masked, score, None, 4, 4, 3, 5)
    check(got, masked, score, None, 4, 4, 3, 5)
    assert got[2][3].tolist() == [0, 1, 2, 3, 4] and (got[1][3] == 0).all()


@pytest.mark.parametrize("beams,V,picks", [(1, 4096, 16), (4, 40000, 8), (16, 20000, 32), (2, 3, 5)])
def test_select_ties(L, beams, V, picks):
    """Equal logits everywhere, equal beams, and logits of few distinct values: the lowest index wins."""
    score = np.full(beams, -3.25, dtype=np.float32)
    flat = np.full((beams, V), 0.5, dtype=np.float32)
    check(run_select(L, flat, score, None, -1, 1, beams, picks), flat, score, None, -1, 1, beams, picks)
    rng, logits, _ = inputs(1, 1, V, 4)
    same = np.repeat(np.round(logits * 2) / 2, beams, 0)
    check(run_select(L, same, score, None, -1, 1, beams, picks), same, score, None, -1, 1, beams, picks)


def test_select_again_and_concurrently(L):
    """The same workspace call after call (its counters return to zero), in a graph, and two streams with one each."""
    torch = _torch()
    _, logits, score = inputs(3, 4, 20000, 5)
    ws = torch.zeros(L.hy_op_beam_select_workspace(3, 4, 20000), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        check(run_select(L, logits, score, None, 1, 3, 4, 4, ws=ws), logits, score, None, 1, 3, 4, 4)
    assert not ws[:256].any().item()
    d, s = torch.from_numpy(logits).cuda(), torch.from_numpy(score).cuda()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for st in streams:
        w = torch.zeros_like(ws)
        o = torch.empty((3, 4), device="cuda"), *(torch.empty((3, 4), dtype=torch.int32, device="cuda") for _ in range(3))
        outs.append((w, o))
    torch.cuda.synchronize()
    call = lambda st, w, o: L.hy_op_beam_select(d.data_ptr(), 20000, 3, 4, 20000, 4, s.data_ptr(), None, 1, o[0].data_ptr(),  # noqa: E731
                                                o[1].data_ptr(), o[2].data_ptr(), o[3].data_ptr(), w.data_ptr(), st.cuda_stream)
    for _ in range(3):
        for st, (w, o) in zip(streams, outs):
            assert call(st, w, o) == 0
    torch.cuda.synchronize()
    for w, o in outs:
        check([to_np(t) for t in o], logits, score, None, 1, 3, 4, 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[0]):
        assert call(streams[0], *outs[0]) == 0
    score2 = score[::-1].copy()
    s.copy_(torch.from_numpy(score2))
    g.replay()
    torch.cuda.synchronize()
    check([to_np(t) for t in outs[0][1]], logits, score2, None, 1, 3, 4, 4)


@pytest.mark.parametrize("groups,beams,V", [(6, 1, 151936), (640, 1, 262144), (6, 1, 1000003), (2, 3, 151936)])
def test_select_score_error(L, groups, beams, V):
    """The bound that include/hybrid.h states for the log-sum-exp, 2^-17 + 2^-21 ceil(V / 4096): logits of a lane that grow
    step after step (every step a new maximum), fall, are flat, a peak over a flat tail, normal, or far below zero.

    Per step of 4096 logits a lane's sum takes two roundings (2 2^-24) and an ex2.approx (2^-22) whose rounded argument
    counts 2^-24 ln 2 d 2^-d at most, d octaves apart: below 2^-21.  Apart from that 16 terms are summed (15 2^-24), each
    an ex2.approx (2^-22) of a rounded argument (2^-24 ln 2 times its octaves, whose mean weighted by the terms is at most
    log2 V <= 27: 19 2^-24), then the lanes (ex2, 6 2^-24), the warps (ex2, 9 2^-24) and the chunks (ex2, 2^-24); FP32's
    log2 e is 2^-26 off, times as many octaves (5 2^-24), and the logarithm errs by 2^-25: 73 2^-24 < 2^-17.  (One
    beam a group: every row's log-sum-exp shows.)"""
    torch = _torch()
    rows, dev = groups * beams, dict(device="cuda")
    g = torch.Generator(**dev)
    g.manual_seed(V)
    up = torch.arange(V, **dev).float() * (24.0 / V)
    kinds = [up, up.flip(0), torch.full((V,), 3.75, **dev), torch.where(torch.arange(V, **dev) == V // 3, 12.0, 0.25), up * 4 - 70]
    x = torch.empty((rows, V), **dev)
    for r in range(rows):
        x[r] = torch.randn(V, generator=g, **dev) * 2.5 if r % 6 == 5 else kinds[r % 6]
    score = torch.full((rows,), -2.0, **dev)
    ws = torch.zeros(L.hy_op_beam_select_workspace(groups, beams, V), dtype=torch.uint8, device="cuda")
    so = torch.empty((groups, beams), **dev)
    po, to = (torch.empty((groups, beams), dtype=torch.int32, **dev) for _ in range(2))
    assert L.hy_op_beam_select(x.data_ptr(), V, groups, beams, V, beams, score.data_ptr(), None, -1, so.data_ptr(), po.data_ptr(),
                               to.data_ptr(), None, ws.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    row = (po.long() + torch.arange(groups, **dev)[:, None] * beams).view(-1)
    lse = torch.cat([torch.logsumexp(x[i:i + 32].double(), -1) for i in range(0, rows, 32)])
    want = -2.0 + x[row, to.long().view(-1)].double() - lse[row]
    err = (so.double().view(-1) - want).abs() - 2.0 ** -24 * want.abs()
    assert (err <= 2.0 ** -17 + 2.0 ** -21 * -(-V // 4096)).all()


def test_select_offsets_past_32_bits(L):
    """2.2e9 logits: the last groups' rows lie past 2^31 elements."""
    torch = _torch()
    groups, beams, V = 900, 16, 151936
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    x = torch.empty((groups * beams, V), device="cuda")
    assert x.numel() > 2 ** 31
    x.normal_(0, 2.5, generator=g)
    score = -20 * torch.rand(groups * beams, generator=g, device="cuda") - 1
    ws = torch.zeros(L.hy_op_beam_select_workspace(groups, beams, V), dtype=torch.uint8, device="cuda")
    out = torch.empty((groups, 4), device="cuda"), *(torch.empty((groups, 4), dtype=torch.int32, device="cuda") for _ in range(3))
    assert L.hy_op_beam_select(x.data_ptr(), V, groups, beams, V, 4, score.data_ptr(), None, 2, out[0].data_ptr(), out[1].data_ptr(),
                               out[2].data_ptr(), out[3].data_ptr(), ws.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    for q in (0, 1, 700, groups - 2, groups - 1):
        rows = slice(q * beams, (q + 1) * beams)
        one = to_np(x[rows]), to_np(score[rows])
        check([to_np(t[q:q + 1]) for t in out], one[0], one[1], None, 2, 1, beams, 4)


# ------------------------------------------------------------------ reordering
@pytest.mark.parametrize("groups,beams,n_seg,seg,pitch,pad", [
    (1, 1, 1, 16, 16, 0), (1, 2, 1, 65536, 65536, 0), (3, 4, 5, 48, 80, 32), (2, 8, 7, 4112, 4112, 16), (1, 16, 3, 100000, 100016, 0),
    (5, 5, 1, 16, 0, 16), (1, 3, 2, 0, 16, 64), (2, 9, 64, 1024, 4096, 0)])
def test_reorder(L, groups, beams, n_seg, seg, pitch, pad):
    torch = _torch()
    rng = np.random.default_rng(beams * 100 + n_seg)
    stride = (n_seg - 1) * pitch + seg + pad
    total = groups * beams * stride
    st = torch.cuda.current_stream().cuda_stream
    for trial in range(4):
        a = rng.integers(0, 256, total).astype(np.uint8)
        parent = rng.integers(0, beams, (groups, beams)).astype(np.int32)
        if trial == 1:
            parent[:] = np.arange(beams)
        if trial == 2:
            parent = np.roll(np.tile(np.arange(beams, dtype=np.int32), (groups, 1)), 1, axis=1)  # a cycle
        want = a.copy()
        for g in range(groups):
            for i in range(beams):
                for s in range(n_seg):
                    to, fr = ((g * beams + k) * stride + s * pitch for k in (i, parent[g, i]))
                    want[to:to + seg] = a[fr:fr + seg]
        d = torch.from_numpy(a).cuda()
        p = torch.from_numpy(parent).cuda()
        assert L.hy_op_beam_reorder(d.data_ptr(), stride, n_seg, pitch, seg, groups, beams, p.data_ptr(), st) == 0, L.hy_last_error()
        np.testing.assert_array_equal(to_np(d), want)


def test_reorder_refuses_bad_parents(L):
    torch = _torch()
    a = np.arange(4 * 64, dtype=np.uint8).reshape(4, 64)
    d = torch.from_numpy(a.copy()).cuda()
    p = torch.tensor([1, -1, 4, 0], dtype=torch.int32, device="cuda")
    L.hy_op_check_device(None, None)
    assert L.hy_op_beam_reorder(d.data_ptr(), 64, 1, 64, 64, 1, 4, p.data_ptr(), None) == 0
    assert L.hy_op_check_device(None, None) == capi.HY_ERR_DEVICE_GUARD
    np.testing.assert_array_equal(to_np(d), a[[1, 1, 2, 0]])
    assert L.hy_op_check_device(None, None) == 0


@pytest.mark.parametrize("groups,beams,n_seg,seg,gap", [(1, 4, 3, 1040, 0), (3, 5, 7, 48, 32), (2, 16, 2, 65536, 16), (1, 2, 70, 16, 0)])
def test_reorder_interleaved(L, groups, beams, n_seg, seg, gap):
    """Layout [n_seg][groups * beams][seg (+ gap)], as [layer][beam][...] caches have it."""
    torch = _torch()
    rng = np.random.default_rng(beams * 10 + n_seg)
    a = rng.integers(0, 256, (n_seg, groups, beams, seg + gap)).astype(np.uint8)
    parent = rng.integers(0, beams, (groups, beams)).astype(np.int32)
    want = a.copy()
    for g in range(groups):
        want[:, g, :, :seg] = a[:, g, parent[g], :seg]
    d = torch.from_numpy(a).cuda()
    p = torch.from_numpy(parent).cuda()
    stride = seg + gap
    # the last segment of the last state ends with the tensor, or `gap` before
    assert L.hy_op_beam_reorder(d.data_ptr(), stride, n_seg, groups * beams * stride, seg, groups, beams, p.data_ptr(),
                                torch.cuda.current_stream().cuda_stream) == 0, L.hy_last_error()
    np.testing.assert_array_equal(to_np(d), want)


def test_reorder_offsets_past_32_bits(L):
    """States of 4.3 GB each, exchanged, in one segment and in segments far apart."""
    torch = _torch()
    n = 2 ** 29 + 2 ** 20 + 4  # values of 8 bytes
    a = torch.arange(2 * n, dtype=torch.int64, device="cuda").view(2, n)
    p = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert L.hy_op_beam_reorder(a.data_ptr(), n * 8, 1, n * 8, n * 8, 1, 2, p.data_ptr(), st) == 0, L.hy_last_error()
    want = torch.arange(n, dtype=torch.int64, device="cuda")
    assert torch.equal(a[0], want + n) and torch.equal(a[1], want)
    # two segments of two states, [segment][beam][...]
    b = a.view(2, 2, n // 2)
    assert L.hy_op_beam_reorder(b.data_ptr(), n // 2 * 8, 2, n * 8, n // 2 * 8, 1, 2, p.data_ptr(), st) == 0, L.hy_last_error()
    h = n // 2
    assert torch.equal(a[0, :h], want[h:] + n) and torch.equal(a[0, h:], want[:h] + n)
    assert torch.equal(a[1, :h], want[h:]) and torch.equal(a[1, h:], want[:h])
