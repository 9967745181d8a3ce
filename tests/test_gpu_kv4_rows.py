"""The 4-bit attention at long contexts: every cached row counts once, with its own scales, wherever tiles, ranges, spans
and the joins of CTAs begin and end.

Three checks that a missing, doubled or exchanged row does not pass:

* Sums.  With zero queries every weight is 2^0, and with scales that are powers of two all products and partial sums are
  integers times 2^-1 below 2^23, so everything up to the last division is exact: o = S (1 / L) errs by the two
  roundings of FP32, 2 * 2^-24 |o| (1 + 2^-24).  A row more or less changes L, so o by 1 / L > 2^-18 of itself.
* Peaks.  A query that equals one row's key, scaled until every other row's score is at least 40 below it: o is that
  row's values.  Their product is exact (weight 1, two fp16 parts of a scale of 11 bits), the other rows add at most
  L e^-40 (1 + 2^-10) max |V|, the division 2^-23.
* Norms.  Normal keys, values and queries against FP64: 2-norm of a head's error at most 2^-19 of its outputs'.  Each row's
  weight errs by less than 2^-20 (ex2.approx, its FP32 argument, two fp16 parts), apart for each row, as the rows
  themselves are, so this is 2^-20 of the 2-norm; a warp adds up to 70 tiles in FP32, sqrt(70) 2^-24 < 2^-20."""
import math

import numpy as np
import pytest

from bandwidth_bound_hybrid_gb300 import capi
from tests.test_gpu_kv4 import pack, quant, rope_np

pytestmark = pytest.mark.gpu

# nkv, heads of a kv head, head dim, lengths: one range or many for each head, spans, two-level joins
SHAPES = [
    (1, 8, 256, [131071]),
    (2, 1, 128, [131070, 5]),
    (4, 4, 128, [131071, 120001, 125003, 130016, 121999, 128000, 127777, 120032]),
    (2, 8, 256, [16384, 1024, 1025, 9999, 15, 12345, 4097, 16000]),
    (13, 1, 256, [2600, 2590, 2555, 2601]),
    (8, 2, 64, [40000, 0, 39999, 31, 32, 33, 20480]),
    (64, 1, 64, [300, 0, 299, 31, 310, 64, 5, 290]),
]
IDS = ["%dx%dx%d-%d" % (k, g, h, len(n)) for k, g, h, n in SHAPES]


@pytest.fixture(scope="module")
def L(gpu):
    from bandwidth_bound_hybrid_gb300 import build
    build.build()
    return capi.lib()


class Cache:
    """A cache of random codes, and the calls on it.  Positions are not rotated (cos 1, sin 0)."""

    def __init__(self, L, nkv, G, hd, lens, seed, scales):
        import torch
        self.torch, self.L = torch, L
        self.nkv, self.G, self.hd, self.lens, self.B = nkv, G, hd, lens, len(lens)
        self.nq, self.cap = nkv * G, max(lens) + 1
        self.cap4 = (self.cap + 3) // 4 * 4
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.q = {}
        for n in "KV":
            half = [torch.randint(1, 16, (self.B, nkv, self.cap, hd // 2), generator=self.g, device="cuda", dtype=torch.uint8)
                    for _ in range(2)]
            self.q[n] = half[0] | (half[1] << 4)
            self.q[n + "s"] = scales(self, (self.B, nkv, self.cap4, hd // 32))
        self.rope = torch.zeros((self.cap, hd // 2, 2), device="cuda")
        self.rope[..., 0] = 1
        self.len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.ws = torch.zeros(L.hy_op_attention_q4_workspace(self.B, self.nq, nkv, hd), dtype=torch.uint8, device="cuda")
        self.y = torch.zeros((self.B, (self.nq + 2 * nkv) * hd), device="cuda")

    def new_row(self):
        """New k and v rows of whole numbers, 7 the largest of each block (scale 1)."""
        t, nkv, hd = self.torch, self.nkv, self.hd
        new = t.randint(-7, 8, (self.B, 2 * nkv, hd // 32, 32), generator=self.g, device="cuda").float()
        new[..., 3] = 7
        self.y.view(self.B, -1, hd)[:, self.nq:] = new.view(self.B, 2 * nkv, hd)

    def values(self, n, b, kv):
        """FP64 values [T + 1][hd] of the cached rows and the new one, as they stand after the call."""
        t, T = self.torch, self.lens[b] + 1
        p = self.q[n][b, kv, :T].view(T, self.hd // 32, 16)
        c = t.cat([p & 15, p >> 4], -1).double() - 8
        return (c * self.q[n + "s"][b, kv, :T].double()[..., None]).view(T, self.hd)

    def call(self):
        t = self.torch
        o = t.full((self.B, self.nq * self.hd), math.nan, device="cuda")
        rc = self.L.hy_op_attention_q4(self.y.data_ptr(), self.y.stride(0), self.B, self.q["K"].data_ptr(), self.q["Ks"].data_ptr(),
                                       self.q["V"].data_ptr(), self.q["Vs"].data_ptr(), self.cap, self.nq, self.nkv, self.hd,
                                       self.len.data_ptr(), self.rope.data_ptr(), o.data_ptr(), o.stride(0), None,
                                       self.ws.data_ptr(), t.cuda.current_stream().cuda_stream)
        assert rc == 0, self.L.hy_last_error()
        return o.view(self.B, self.nkv, self.G, self.hd).double()


def powers_of_two(c, shape):
    t = c.torch
    return t.exp2(t.randint(-1, 2, shape, generator=c.g, device="cuda").float()).half()


@pytest.mark.parametrize("nkv,G,hd,lens", SHAPES, ids=IDS)
def test_every_row_counts_once(L, nkv, G, hd, lens):
    c = Cache(L, nkv, G, hd, lens, 1, powers_of_two)
    c.new_row()
    o = c.call()
    for b, T in enumerate(lens):
        for kv in range(nkv):
            want = c.values("V", b, kv).sum(0) / (T + 1)
            err = (o[b, kv] - want).abs()
            assert (err <= 2.0 ** -23 * (1 + 2.0 ** -20) * want.abs()).all(), (b, T, kv, float((err / want.abs()).nan_to_num().max()))


def targets(c, rng, T, every):
    """G rows of one (sequence, kv head): around the borders of tiles, or any."""
    if every is not None:
        return [(every + j) % (T + 1) for j in range(c.G)]
    rows = [0, T, max(T - 1, 0)]
    while len(rows) < c.G + 3:
        tile = int(rng.integers(0, T // 16 + 1)) * 16
        rows.append(min(max(tile + int(rng.integers(-1, 2)), 0), T))
    rng.shuffle(rows)
    return rows[:c.G]


def peaked(c, rng, every=None):
    t, hd = c.torch, c.hd
    c.new_row()
    y = c.y.view(c.B, -1, hd)
    yk = c.y.view(c.B, -1, hd)[:, c.nq:c.nq + c.nkv]
    want, least = t.empty((c.B, c.nkv, c.G, hd), dtype=t.float64, device="cuda"), math.inf
    limit = t.empty((c.B, c.nkv, 1, 1), dtype=t.float64, device="cuda")
    for b, T in enumerate(c.lens):
        for kv in range(c.nkv):
            K, V = c.values("K", b, kv), c.values("V", b, kv)
            K[T], V[T] = yk[b, kv].double(), y[b, c.nq + c.nkv + kv].double()  # whole numbers under scale 1: held as they are
            rows = targets(c, rng, T, None if every is None else every + kv * c.G)
            q = K[rows]
            s = q @ K.T
            top = s.gather(1, t.tensor(rows, device="cuda")[:, None])
            rest = s.scatter(1, t.tensor(rows, device="cuda")[:, None], -math.inf).amax(1, keepdim=True)
            gap = (top - rest).clamp(max=1e6)
            factor = t.exp2(t.ceil(t.log2(60 * math.sqrt(hd) / gap)))  # a power of two: the query stays exact
            least = min(least, float((gap * factor).min()) / math.sqrt(hd))
            y[b, kv * c.G:(kv + 1) * c.G] = (q * factor).float()
            want[b, kv] = V[rows]
            limit[b, kv] = 2.0 ** -22 * V.abs().max() + (T + 1) * math.exp(-40) * 1.001 * V.abs().max()
    assert least >= 60  # scores of 60 apart: their own errors are far below the 20 between this and the 40 above
    o = c.call()
    err = (o - want).abs()
    bad = (err > limit).nonzero()
    assert bad.numel() == 0, (bad[:4].tolist(), float(err.max()))


@pytest.mark.parametrize("nkv,G,hd,lens", SHAPES, ids=IDS)
def test_peaks_at_the_borders(L, nkv, G, hd, lens):
    c = Cache(L, nkv, G, hd, lens, 2, lambda c, shape: c.torch.full(shape, 1.0, dtype=c.torch.float16, device="cuda"))
    rng = np.random.default_rng(nkv + hd)
    for _ in range(2 if sum(lens) * nkv > 10 ** 6 else 6):
        peaked(c, rng)


@pytest.mark.parametrize("nkv,G,hd,T", [(2, 8, 256, 700), (4, 4, 128, 1500), (8, 2, 64, 900)])
def test_a_peak_at_every_row(L, nkv, G, hd, T):
    """Each row of a context in turn, of one sequence and (the second call's plan) of eight."""
    for lens in ([T], [T - 3 * i for i in range(8)]):
        c = Cache(L, nkv, G, hd, lens, 3, lambda c, shape: c.torch.full(shape, 1.0, dtype=c.torch.float16, device="cuda"))
        for first in range(0, T + 1, nkv * G):
            peaked(c, None, first)


@pytest.mark.parametrize("nkv,G,hd,lens", SHAPES, ids=IDS)
def test_norms_against_64_bits(L, nkv, G, hd, lens):
    c = Cache(L, nkv, G, hd, lens, 4, powers_of_two)
    t = c.torch
    rng = np.random.default_rng(hd)
    for n in "KV":  # normal rows in the cache's own format, 4096 of them over and over with other signs of whole rows
        codes, s = quant(rng.standard_normal((4096, hd)).astype(np.float32))
        flip = 1 - 2 * (t.rand((c.B, nkv, c.cap), generator=c.g, device="cuda") < 0.5).int()
        at = t.randint(0, 4096, (c.B, nkv, c.cap), generator=c.g, device="cuda")
        both = t.from_numpy(np.stack([pack(codes), pack(-codes)])).cuda()
        c.q[n] = both[(flip < 0).long(), at].contiguous()
        c.q[n + "s"].zero_()
        c.q[n + "s"][:, :, :c.cap] = t.from_numpy(s).cuda()[at]
    c.rope = t.from_numpy(rope_np(c.cap, hd)).cuda()
    c.y = t.randn((c.B, (c.nq + 2 * nkv) * hd), generator=c.g, device="cuda")
    c.y[:, :c.nq * hd] *= 1.5
    o = c.call()
    for b, T in enumerate(lens):
        cs = c.rope[T].double()
        for kv in range(nkv):
            K, V = c.values("K", b, kv), c.values("V", b, kv)
            x = c.y[b].view(-1, hd)[kv * G:(kv + 1) * G].double()
            x0, x1 = x[:, :hd // 2], x[:, hd // 2:]
            q = t.cat([x0 * cs[:, 0] - x1 * cs[:, 1], x1 * cs[:, 0] + x0 * cs[:, 1]], -1)
            want = t.softmax(q @ K.T / math.sqrt(hd), -1) @ V
            rel = (o[b, kv] - want).norm(dim=-1) / want.norm(dim=-1)
            assert (rel <= 2.0 ** -19).all(), (b, T, kv, rel.tolist())


@pytest.mark.parametrize("nkv,G,hd", [(2, 8, 256), (4, 4, 128), (3, 1, 64)])
@pytest.mark.parametrize("ratio", [2.0 ** -10, 2.0 ** -20])
def test_blocks_far_below_others(L, nkv, G, hd, ratio):
    """One block of V large, the others small: a row's weighted scale errs by 2^-22 of itself or 2^-38 of the largest, times
    |code| <= 7.  Weights relative to the largest, 1 / max p in all; 2^-19 covers what the norms above allow a row."""
    c = Cache(L, nkv, G, hd, [5000, 321], 5, powers_of_two)
    t = c.torch
    c.q["Vs"] *= ratio
    c.q["Vs"][..., 0] = 1.0
    c.q["Ks"] *= 0.125
    c.y.normal_(generator=c.g)
    c.y.view(c.B, -1, hd)[:, c.nq + nkv:] *= ratio
    o = c.call()
    for b, T in enumerate(c.lens):
        for kv in range(nkv):
            K, V = c.values("K", b, kv), c.values("V", b, kv)
            q = c.y[b].view(-1, hd)[kv * G:(kv + 1) * G].double()
            p = t.softmax(q @ K.T / math.sqrt(hd), -1)
            tol = 2.0 ** -19 * (p @ V.abs()) + (T + 1) * p.amax(-1, keepdim=True) * 7 * 2.0 ** -38
            err = (o[b, kv] - p @ V).abs()
            assert (err <= tol).all(), (b, kv, float((err / tol).max()))


def test_offsets_past_32_bits(L):
    """Codes of 4.6 GB each: a long last sequence behind short ones, its last heads past 2^32 bytes."""
    lens = [3, 0, 17, 40, 5, 33, 1, 69998]
    c = Cache(L, 64, 1, 256, lens, 6, powers_of_two)
    assert c.q["K"].numel() > 2 ** 32
    c.new_row()
    kept = {n: c.q[n][:, :, -1].clone() for n in ("K", "V")}  # the row behind the longest sequence's last
    o = c.call()
    for b, T in enumerate(lens):
        for kv in range(0, 64, 7):
            want = c.values("V", b, kv).sum(0) / (T + 1)
            err = (o[b, kv] - want).abs()
            assert (err <= 2.0 ** -23 * (1 + 2.0 ** -20) * want.abs()).all(), (b, T, kv)
            codes, _ = quant(c.y[b].view(-1, 256)[64 + kv].cpu().numpy())
            assert (c.q["K"][b, kv, T].cpu().numpy() == pack(codes)).all()
    for n in ("K", "V"):
        assert c.torch.equal(c.q[n][:-1, :, -1], kept[n][:-1])
