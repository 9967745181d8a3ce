"""The 4-bit KV cache operators against a plain FP64 form: the decode attention
(hy_op_attention_q4) and the quantising append (hy_op_kv_append_q4).

Codes and scales of appended rows are compared exactly: the format's rule is
a fixed sequence of FP32 operations, and numpy's float32 rounds each of them
as the kernel does.

Attention tolerance, per (query head j, output dim d), derived as in
gpu_util.attention_tolerance: with score errors delta_t and relative errors
eps_t of the probabilities, |err| <= sum_t p_t (delta_t + eps_t) |V_t - o| +
rel_sum sum_t p_t |V_t| + 16 u |o|.  Here (u = 2^-24; a tensor-core sum of n
exact products is taken to err by at most 2 gamma(n), truncation included)
  delta_t = scale sum_b s_tb sum_{i in b} |q_i| (8 * 2 gamma(40))    the block sums of |code| <= 8
          + (2^-21 + gamma(NB + 8)) scale sum_i |q_i K_ti|           q as two fp16 parts (2^-22 each way), FP32 over blocks
          + 6 u scale sum_i (|a_i| + |b_i|) |K_ti|                   RoPE and the score factor
          + 2^-33 scale max|q| sum_i |K_ti|                          fp16 spacing below the head's normalised range
  eps_t   = 2^-20 + 4 u (|s_t| + max |s| + 32)                       ex2.approx, its FP32 argument, p s_V as two fp16 parts
          + npos 2^-35 max_t(s_V) in all                              p s_V below fp16's normal range: its two parts each err by
            half the subnormal spacing, 2^-25, where the largest s_V counts 2^14 or more, so a row's term by at most
            2 2^-25 / 2^14 max(s_V) |code| <= 2^-38 8 max(s_V); all npos rows may be such rows
  rel_sum = 2 gamma(36 (npos / 256 + 2) + 64)                        the per-warp tile sums and the joins."""
import ctypes

import numpy as np
import pytest

from bandwidth_bound_hybrid_gb300 import capi
from tests.gpu_util import U32, assert_elementwise, gamma, rope_pair_abs, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L(gpu):
    from bandwidth_bound_hybrid_gb300 import build
    build.build()
    return capi.lib()


def _torch():
    import torch
    return torch


# ------------------------------------------------------------------ plain form
def quant(x):
    """FP32 vectors [..., hd] -> codes int [..., hd], scales fp16 [..., hd / 32]."""
    x = np.asarray(x, dtype=np.float32)
    b = x.reshape(*x.shape[:-1], -1, 32)
    a = np.abs(b).max(-1)
    with np.errstate(over="ignore", invalid="ignore"):
        s = np.where(np.isfinite(a), np.minimum(a * (np.float32(1) / np.float32(7)), np.float32(65504)), np.float32(np.nan)).astype(np.float16)
        sf = s.astype(np.float32)
        inv = np.where(sf > 0, np.float32(1) / np.where(sf > 0, sf, np.float32(1)), np.float32(0)).astype(np.float32)
        c = np.rint(b * inv[..., None])
    return np.clip(c, -7, 7).reshape(x.shape), s


def pack(codes):
    n = (np.asarray(codes).astype(np.int64) + 8).astype(np.uint8)
    n = n.reshape(*n.shape[:-1], -1, 2, 16)
    return (n[..., 0, :] | (n[..., 1, :] << 4)).reshape(*codes.shape[:-1], -1)


def unpack(p):
    p = p.reshape(*p.shape[:-1], -1, 16)
    c = np.concatenate([p & 15, p >> 4], -1).astype(np.float64) - 8
    return c.reshape(*c.shape[:-2], -1)


def values(packed, scales):
    c = unpack(packed)
    return (c.reshape(*c.shape[:-1], -1, 32) * scales.astype(np.float64)[..., None]).reshape(c.shape)


def rope_np(cap, hd, theta=1e4):
    ang = np.arange(cap)[:, None] * theta ** (-2.0 * np.arange(hd // 2) / hd)
    return np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)


def rotate32(x, cs):
    """RoPE in FP32, each operation rounded on its own."""
    h = x.shape[-1] // 2
    c, s = cs[..., 0], cs[..., 1]
    return np.concatenate([x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s], -1)


def attend(q, K, V, Ks_blocks, yq):
    """o and its bound for the heads q [G][hd] (FP64, rotated) of one kv head."""
    G, hd = q.shape
    NB, npos = hd // 32, K.shape[0]
    scale = 1 / np.sqrt(hd)
    o, tol = np.zeros_like(q), np.zeros_like(q)
    aK = np.abs(K)
    vs = np.abs(V).max() / 7 + 1e-300
    for j in range(G):
        s = K @ q[j] * scale
        M = s.max()
        p = np.exp(s - M)
        p /= p.sum()
        o[j] = p @ V
        aq = np.abs(q[j])
        delta = scale * (np.abs(Ks_blocks) @ aq.reshape(NB, 32).sum(-1)) * 8 * 2 * gamma(40)
        delta += (2.0 ** -21 + gamma(NB + 8)) * scale * (aK @ aq) + 6 * U32 * scale * (aK @ rope_pair_abs(yq[j]))
        delta += 2.0 ** -33 * scale * aq.max() * aK.sum(-1)
        eps = 2.0 ** -20 + 4 * U32 * (np.abs(s) + np.abs(s).max() + 32)
        rel = 2 * gamma(36 * (npos // 256 + 2) + 64)
        tol[j] = ((delta + eps) * p) @ np.abs(V - o[j]) + rel * (p @ np.abs(V)) + 16 * U32 * np.abs(o[j])
        tol[j] += npos * 2.0 ** -35 * vs + 1e-30
    return o, tol


class Case:
    """A filled cache of `batch` sequences and the projections of one step."""

    def __init__(self, nq, nkv, hd, lens, seed=0, spare=3, qmul=1.5, kmul=1.0, vmul=1.0, pad_y=0, pad_o=0):
        torch = _torch()
        rng = np.random.default_rng(seed * 1009 + hd + nq + sum(lens))
        self.nq, self.nkv, self.hd, self.lens = nq, nkv, hd, list(lens)
        B = self.B = len(lens)
        cap = self.cap = max(max(lens) + 1, 1) + spare
        self.cap4 = (cap + 3) // 4 * 4
        NB = hd // 32
        self.K, self.Ks, self.V, self.Vs = [], [], [], []
        shape = (B, nkv, cap, hd)
        kc, ks = quant(rng.standard_normal(shape).astype(np.float32) * np.float32(kmul))
        vc, vs = quant(rng.standard_normal(shape).astype(np.float32) * np.float32(vmul))
        self.Kq, self.Vq = pack(kc), pack(vc)
        self.Ks = np.full((B, nkv, self.cap4, NB), np.nan, dtype=np.float16)
        self.Vs = self.Ks.copy()
        for b, T in enumerate(lens):  # whatever lies past a sequence's rows is never read: NaN scales there
            T = min(max(T, 0), cap)
            self.Ks[b, :, :T], self.Vs[b, :, :T] = ks[b, :, :T], vs[b, :, :T]
        self.ldy, self.ldo = (nq + 2 * nkv) * hd + pad_y, nq * hd + pad_o
        self.y = rng.standard_normal((B, self.ldy)).astype(np.float32)
        self.y[:, :nq * hd] *= qmul
        self.y[:, nq * hd:(nq + nkv) * hd] *= kmul
        self.y[:, (nq + nkv) * hd:(nq + 2 * nkv) * hd] *= vmul
        self.rope = rope_np(cap, hd)
        self.torch = torch

    def upload(self):
        t = self.torch
        f = lambda a: t.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.d = dict(y=f(self.y), Kq=f(self.Kq), Ks=f(self.Ks), Vq=f(self.Vq), Vs=f(self.Vs), rope=f(self.rope),
                      len=t.tensor(self.lens, dtype=t.int32, device="cuda"))
        self.o = t.full((self.B, self.ldo), -77.0, device="cuda")
        self.new = t.full((self.B, 2, self.nkv, self.hd), -77.0, device="cuda")
        return self

    def workspace(self, L):
        n = L.hy_op_attention_q4_workspace(self.B, self.nq, self.nkv, self.hd)
        assert n > 0
        return self.torch.zeros(n, dtype=self.torch.uint8, device="cuda")

    def call(self, L, ws, stream=None, **over):
        d = self.d
        st = self.torch.cuda.current_stream().cuda_stream if stream is None else stream
        a = dict(y=d["y"].data_ptr(), ldy=self.ldy, batch=self.B, Kq=d["Kq"].data_ptr(), Ks=d["Ks"].data_ptr(),
                 Vq=d["Vq"].data_ptr(), Vs=d["Vs"].data_ptr(), cap=self.cap, nq=self.nq, nkv=self.nkv, hd=self.hd,
                 len=d["len"].data_ptr(), rope=d["rope"].data_ptr(), o=self.o.data_ptr(), ldo=self.ldo,
                 new=self.new.data_ptr(), ws=ws.data_ptr(), stream=st)
        a.update(over)
        return L.hy_op_attention_q4(*a.values())

    def new_rows(self, b):
        """Packed codes, scales, values of sequence b's new k and v rows [2][nkv][...]."""
        hd, nq, nkv = self.hd, self.nq, self.nkv
        y = self.y[b, :(nq + 2 * nkv) * hd].reshape(-1, hd)
        k = rotate32(y[nq:nq + nkv], self.rope[self.lens[b]][None])
        c, s = quant(np.stack([k, y[nq + nkv:]]))
        return pack(c), s, values(pack(c), s)

    def check(self, refused=()):
        t, hd, nq, nkv = self.torch, self.hd, self.nq, self.nkv
        t.cuda.synchronize()
        G = nq // nkv
        got, new = to_np(self.o), to_np(self.new)
        gKq, gKs, gVq, gVs = (to_np(self.d[n]) for n in ("Kq", "Ks", "Vq", "Vs"))
        eKq, eKs, eVq, eVs = self.Kq.copy(), self.Ks.copy(), self.Vq.copy(), self.Vs.copy()
        for b, T in enumerate(self.lens):
            if b in refused:
                assert (got[b] == -77).all() and (new[b] == -77).all()
                continue
            pk, sc, val = self.new_rows(b)
            eKq[b, :, T], eVq[b, :, T], eKs[b, :, T], eVs[b, :, T] = pk[0], pk[1], sc[0], sc[1]
            np.testing.assert_array_equal(new[b], val.astype(np.float32))
            np.testing.assert_array_equal(got[b, nq * hd:], -77.0)
            y = self.y[b].astype(np.float64)
            for g in range(nkv):
                K, V = (values(q[b, g, :T + 1], s[b, g, :T + 1]) for q, s in ((eKq, eKs), (eVq, eVs)))
                yq = y[g * G * hd:(g + 1) * G * hd].reshape(G, hd)
                q = rotate32(yq, self.rope[T].astype(np.float64)[None])
                o, tol = attend(q, K, V, eKs[b, g, :T + 1].astype(np.float64), yq)
                assert_elementwise(got[b, g * G * hd:(g + 1) * G * hd].reshape(G, hd), o, tol,
                                   f"sequence {b} (T={T}), kv head {g}")
        # the appended rows, and every other byte as it was
        for g_, e_ in ((gKq, eKq), (gVq, eVq), (gKs.view(np.uint16), eKs.view(np.uint16)),
                       (gVs.view(np.uint16), eVs.view(np.uint16))):
            np.testing.assert_array_equal(g_, e_)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("T", [0, 1, 31, 32, 33, 63, 64, 255, 256, 257, 1000])
@pytest.mark.parametrize("nq,nkv,hd", [(4, 2, 64), (16, 4, 128), (16, 2, 256)])
def test_attention_one_sequence(L, nq, nkv, hd, T):
    c = Case(nq, nkv, hd, [T]).upload()
    ws = c.workspace(L)
    assert c.call(L, ws) == 0, L.hy_last_error()
    c.check()
    assert not ws[:256].any().item()


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_attention_group_sizes(L, G, hd):
    c = Case(3 * G, 3, hd, [517, 90], seed=G, pad_y=5, pad_o=7).upload()
    assert c.call(L, c.workspace(L)) == 0, L.hy_last_error()
    c.check()


@pytest.mark.parametrize("nq,nkv,hd,lens", [
    (16, 4, 128, [0, 4095, 1, 700, 33, 2048, 31, 64]),
    (16, 2, 256, [3000, 0, 5001]),
    (8, 8, 64, [9000, 12, 8999, 100]),
    (2, 1, 128, [20011]),
    (8, 1, 256, [7, 16384]),
])
def test_attention_ragged_batches(L, nq, nkv, hd, lens):
    c = Case(nq, nkv, hd, lens, seed=3).upload()
    ws = c.workspace(L)
    assert c.call(L, ws) == 0, L.hy_last_error()
    c.check()
    first = c.o.clone()
    for _ in range(3):  # the same workspace again: same bits (the split and its joins are fixed by the lengths)
        assert c.call(L, ws) == 0
    c.check()
    assert c.torch.equal(first, c.o)


@pytest.mark.parametrize("nkv,hd,lens", [(64, 64, [300, 0, 299, 31, 310, 64, 5, 290]),  # more heads than CTAs
                                          (13, 256, [2600, 2590, 2555, 2601])])  # 52 heads of equal length on 152 CTAs
def test_attention_in_spans(L, nkv, hd, lens):
    """Ranges of several heads in one CTA: spans of the tile list."""
    c = Case(nkv, nkv, hd, lens, seed=4).upload()
    ws = c.workspace(L)
    for _ in range(2):
        assert c.call(L, ws) == 0, L.hy_last_error()
    c.check()
    assert not ws[:8 * nkv * 32 * 4].any().item()


def test_attention_workspace_serves_every_batch(L):
    """One workspace, calls of different batches in turn."""
    a = Case(16, 4, 128, [1500, 40, 900, 2000, 3, 77, 1200, 600], seed=20).upload()
    b = Case(16, 4, 128, [5000], seed=21).upload()
    ws = a.workspace(L)
    assert ws.numel() == b.workspace(L).numel()
    for c in (a, b, a, b):
        assert c.call(L, ws) == 0
        c.check()


@pytest.mark.parametrize("qmul,kmul,vmul", [(40.0, 1.0, 1.0), (1e-3, 1.0, 1e4), (1.0, 30.0, 1e-5), (1e20, 1e-20, 1.0),
                                            (1.5, 1.0, 2e5), (0.0, 1.0, 1.0)])
def test_attention_magnitudes(L, qmul, kmul, vmul):
    """Peaked and flat softmaxes, values near both ends of the fp16 scales (2e5 saturates none: 65504 * 7 = 458k),
    zero queries (uniform weights)."""
    c = Case(8, 2, 128, [1500, 77], seed=5, qmul=qmul, kmul=kmul, vmul=vmul).upload()
    assert c.call(L, c.workspace(L)) == 0, L.hy_last_error()
    c.check()


def test_attention_large_values_after_small_ones(L):
    """V scales that grow by 2^30 along the rows: the products' fp16 range follows."""
    c = Case(8, 2, 64, [2000], seed=6)
    ramp = np.exp2(np.linspace(-14, 15, c.cap4))[None, None, :, None]
    c.Vs = (np.where(np.isnan(c.Vs), np.nan, ramp)).astype(np.float16)
    c.upload()
    assert c.call(L, c.workspace(L)) == 0, L.hy_last_error()
    c.check()


def test_attention_zero_blocks(L):
    c = Case(4, 2, 128, [300], seed=7)
    c.Ks[:, :, 10:40] = 0
    c.Vs[:, :, 100:200, 1] = 0
    c.y[:, 4 * 128:] = 0  # a new row of zeros: scales 0, codes 0
    c.upload()
    assert c.call(L, c.workspace(L)) == 0, L.hy_last_error()
    c.check()


def test_attention_nan_rows_show(L):
    """A NaN or an infinity in the projections reaches the outputs of its kv head, and no other."""
    c = Case(4, 2, 64, [40], seed=8).upload()
    yd = c.d["y"]
    yd[0, (4 + 2) * 64 + 3] = float("nan")  # v of kv head 0, first block
    assert c.call(L, c.workspace(L)) == 0
    o = to_np(c.o)[0].reshape(4, 64)
    assert np.isnan(o[:2, :32]).all() and np.isfinite(o[:2, 32:]).all() and np.isfinite(o[2:]).all()
    yd[0, (4 + 2) * 64 + 3] = 0.0
    yd[0, (4 + 1) * 64 + 5] = float("inf")  # k of kv head 1
    assert c.call(L, c.workspace(L)) == 0
    o = to_np(c.o)[0].reshape(4, 64)
    assert np.isfinite(o[:2]).all() and np.isnan(o[2:]).all()


def test_attention_refused_positions(L):
    """A position outside the cache refuses its sequence only, and shows in the guard word."""
    c = Case(16, 4, 128, [100, 103, 64], seed=9)
    c.lens = [100, c.cap, 64]
    c.upload()
    bits = ctypes.c_uint32(0)
    assert L.hy_op_check_device(None, ctypes.byref(bits)) == 0
    assert c.call(L, c.workspace(L)) == 0
    c.check(refused=(1,))
    assert L.hy_op_check_device(None, ctypes.byref(bits)) == capi.HY_ERR_DEVICE_GUARD
    assert bits.value == capi.HY_GUARD_BAD_POSITION
    c.lens = [-1, -5, c.cap + 9]
    c.upload()
    assert c.call(L, c.workspace(L)) == 0
    c.check(refused=(0, 1, 2))
    assert L.hy_op_check_device(None, None) == capi.HY_ERR_DEVICE_GUARD
    assert L.hy_op_check_device(None, None) == 0


def test_attention_on_streams_and_in_graphs(L):
    """Two calls at once on streams and workspaces of their own, and a captured call replayed as the cache grows."""
    torch = _torch()
    a = Case(16, 4, 128, [3000], seed=10).upload()
    b = Case(8, 2, 64, [777, 5], seed=11).upload()
    wa, wb = a.workspace(L), b.workspace(L)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        assert a.call(L, wa, stream=sa.cuda_stream) == 0 and b.call(L, wb, stream=sb.cuda_stream) == 0
    a.check()
    b.check()
    c = Case(16, 4, 128, [30], seed=12, spare=5).upload()
    ws = c.workspace(L)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        assert c.call(L, ws, stream=s.cuda_stream) == 0
    for T in (30, 31, 32):  # 32: the first row of another tile
        c.d["len"][0] = T
        torch.cuda.synchronize()
        g.replay()
        c.lens = [T]
        c.check()
        # what the call appended is part of the cache of the next one
        c.Kq, c.Ks, c.Vq, c.Vs = (to_np(c.d[n]) for n in ("Kq", "Ks", "Vq", "Vs"))


def test_attention_without_the_new_values(L):
    c = Case(4, 2, 64, [50], seed=13).upload()
    assert c.call(L, c.workspace(L), new=None) == 0
    c.torch.cuda.synchronize()
    assert (to_np(c.new) == -77).all()
    c.call(L, c.workspace(L))
    c.check()


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("nq,nkv,hd,T,n", [(4, 2, 64, 0, 1), (4, 2, 64, 5, 130), (16, 4, 128, 100, 77), (8, 8, 256, 31, 2),
                                           (16, 2, 256, 0, 300), (3, 3, 128, 9, 1)])
def test_append_rows(L, nq, nkv, hd, T, n):
    torch = _torch()
    c = Case(nq, nkv, hd, [T], spare=n + 2, pad_y=3 if n % 2 else 4)  # rows that are whole 16 bytes, or not
    rng = np.random.default_rng(n)
    y = (rng.standard_normal((n, c.ldy)) * np.exp(rng.uniform(-6, 6, (n, 1)))).astype(np.float32)
    y[n // 2, nq * hd:nq * hd + 40] = 0  # a block of zeros
    c.y[0] = y[0]
    c.upload()
    yd = torch.from_numpy(y).cuda()
    new = torch.full((n, 2, nkv, hd), -77.0, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    d = c.d
    args = lambda nn, val: (yd.data_ptr(), c.ldy, nn, d["Kq"].data_ptr(), d["Ks"].data_ptr(), d["Vq"].data_ptr(),  # noqa: E731
                            d["Vs"].data_ptr(), c.cap, nq, nkv, hd, d["len"].data_ptr(), d["rope"].data_ptr(), val, st)
    assert L.hy_op_kv_append_q4(*args(0, None)) == 0
    assert L.hy_op_kv_append_q4(*args(n, new.data_ptr())) == 0, L.hy_last_error()
    torch.cuda.synchronize()
    yy = y[:, :(nq + 2 * nkv) * hd].reshape(n, -1, hd)
    k = rotate32(yy[:, nq:nq + nkv], c.rope[T:T + n][:, None])
    codes, s = quant(np.stack([k, yy[:, nq + nkv:]], 1))
    pk = pack(codes)
    np.testing.assert_array_equal(to_np(new), values(pk, s).astype(np.float32))
    eKq, eKs, eVq, eVs = c.Kq.copy(), c.Ks.copy(), c.Vq.copy(), c.Vs.copy()
    for kv, (q, sc) in enumerate(((eKq, eKs), (eVq, eVs))):
        q[0, :, T:T + n] = pk[:, kv].transpose(1, 0, 2)
        sc[0, :, T:T + n] = s[:, kv].transpose(1, 0, 2)
    for name, e in (("Kq", eKq), ("Ks", eKs), ("Vq", eVq), ("Vs", eVs)):
        np.testing.assert_array_equal(to_np(d[name]).view(np.uint8), e.view(np.uint8))
    # rows past the capacity: nothing is written
    d["len"][0] = c.cap - n + 1
    assert L.hy_op_kv_append_q4(*args(n, None)) == 0
    assert L.hy_op_check_device(None, None) == capi.HY_ERR_DEVICE_GUARD
    d["len"][0] = -1
    assert L.hy_op_kv_append_q4(*args(n, None)) == 0
    assert L.hy_op_check_device(None, None) == capi.HY_ERR_DEVICE_GUARD
    for name, e in (("Kq", eKq), ("Ks", eKs), ("Vq", eVq), ("Vs", eVs)):
        np.testing.assert_array_equal(to_np(d[name]).view(np.uint8), e.view(np.uint8))


def test_append_special_values(L):
    """Blocks with huge, tiny, infinite and NaN values: the scale saturates, underflows, or is NaN."""
    torch = _torch()
    c = Case(1, 1, 64, [0], spare=8).upload()
    y = np.zeros((6, c.ldy), dtype=np.float32)
    y[0, 128:192] = 3e38                      # a / 7 past fp16: scale 65504, codes 7
    y[1, 128:192] = np.linspace(-1, 1, 64) * 2e-7  # a / 7 in fp16's subnormals
    y[2, 128:192] = 1e-12                     # scale 0
    y[3, 128:192] = 1
    y[3, 130] = np.inf
    y[4, 128:192] = 1
    y[4, 190] = np.nan
    y[5, 128:192] = -0.0
    d = c.d
    yd = torch.from_numpy(y).cuda()
    new = torch.empty((6, 2, 1, 64), device="cuda")
    assert L.hy_op_kv_append_q4(yd.data_ptr(), c.ldy, 6, d["Kq"].data_ptr(), d["Ks"].data_ptr(), d["Vq"].data_ptr(),
                                d["Vs"].data_ptr(), c.cap, 1, 1, 64, d["len"].data_ptr(), d["rope"].data_ptr(), new.data_ptr(),
                                torch.cuda.current_stream().cuda_stream) == 0
    v = to_np(new)[:, 1, 0]
    s = to_np(d["Vs"])[0, 0]
    for r in (0, 1, 2, 5):
        codes, sc = quant(y[r, 128:192])
        np.testing.assert_array_equal(s[r], sc)
        np.testing.assert_array_equal(v[r], values(pack(codes), sc).astype(np.float32))
    assert v[0].min() == 7 * 65504
    assert np.isnan(s[3, 0]) and np.isnan(v[3, :32]).all() and np.isfinite(v[3, 32:]).all()
    assert np.isnan(s[4, 1]) and np.isnan(v[4, 32:]).all() and np.isfinite(v[4, :32]).all()
