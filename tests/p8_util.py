"""A plain form of the paged 8-bit KV cache (the struct hy_kv_p8 of
include/hybrid.h) and of the attention over it, for the tests of its operators.

The cache is compared exactly: its format is a fixed sequence of FP32
operations, and numpy's float32 rounds each of them as the kernels do.

Attention tolerance, per (query head j, output dim d), derived as in
gpu_util.attention_tolerance: with score errors delta_t and relative errors
eps_t of the probabilities, |err| <= sum_t p_t (delta_t + eps_t) |V_t - o| +
rel_sum sum_t p_t |V_t| + 16 u |o|.  Here (u = 2^-24; a tensor-core sum of n
exact products is taken to err by at most 2 gamma(n), truncation included)
  delta_t = 2 gamma(2 hd + 16) scale sum_i |q_i K_ti|    the products of both parts of q with the codes
          + 2^-21 scale sum_i |q_i K_ti|                 q as two fp16 parts (2^-22 each way)
          + 6 u scale sum_i (|a_i| + |b_i|) |K_ti|       RoPE and the score's factors
          + 2^-33 scale max|q| sum_i |K_ti|              fp16 spacing below the head's normalised range
  eps_t   = 2^-20 + 4 u (|s_t| + max |s| + 32)           ex2.approx, its FP32 argument, p as two fp16 parts (2^-21)
  rel_sum = 2 gamma(npos / 8 + 64)                       FP32 sums over a head's positions in 16s, tiles of 16 or more,
            each with its scale, and the joins
and in all npos 2^-37 max |V|: p below fp16's normal range, where its two parts err by half the subnormal spacing, 2^-25, when 1
counts 2^14 (2 2^-25 / 2^14 = 2^-38)."""
import numpy as np

from tests.gpu_util import U32, assert_elementwise, gamma, rope_pair_abs

BLOCK = 16


def to_bf16(x):
    """FP32 rounded to bf16 (half to even), what is not finite then as NaN; the values as FP32."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7fff + ((u >> 16) & 1)) >> 16).astype(np.uint32)
    v = (r << 16).view(np.float32).reshape(x.shape)
    return np.where(np.isfinite(x) & np.isfinite(v), v, np.float32(np.nan)).astype(np.float32)


def bits16(v):
    return (np.ascontiguousarray(v, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def close(x):
    """Codes (int8) and scales of whole blocks x [..., 16, hd] of bf16 values."""
    x = np.asarray(x, dtype=np.float32)
    a = np.abs(x).max((-2, -1))
    bad = np.isnan(a)
    small = ~bad & (a < np.float32(2.0 ** -100))
    safe = np.where(bad | small, np.float32(1), a)
    s = np.where(bad, np.float32(np.nan), np.where(small, np.float32(0), safe / np.float32(127))).astype(np.float32)
    inv = (np.float32(127) / safe).astype(np.float32)
    with np.errstate(invalid="ignore"):
        c = np.rint((x * inv[..., None, None]).astype(np.float32))
        c = np.clip(np.where((bad | small)[..., None, None], 0, c), -127, 127)
    return c.astype(np.int8), s


def rope_np(cap, hd, theta=1e4):
    ang = np.arange(cap)[:, None] * theta ** (-2.0 * np.arange(hd // 2) / hd)
    return np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)


def rotate32(x, cs):
    """RoPE of [..., heads, hd] with cs [..., 1, hd / 2, 2], in the arrays' precision, each operation rounded on its own."""
    h = x.shape[-1] // 2
    c, s = cs[..., 0], cs[..., 1]
    return np.concatenate([x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s], -1)


def attend(yq, cs, K, V, u, t, window, sinks):
    """o and its bound for heads yq [G, hd] (before RoPE) at position t over K, V [n, hd] at positions u."""
    seen = (u <= t) & ((u < sinks) | (u > t - window) if window else True)
    K, V = K[seen], V[seen]
    hd = yq.shape[-1]
    q = rotate32(yq.astype(np.float64), cs.astype(np.float64))
    scale = 1 / np.sqrt(hd)
    s = (q @ K.T) * scale
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    p /= p.sum(-1, keepdims=True)
    o = p @ V
    aK, aq, n = np.abs(K), np.abs(q), len(K)
    delta = (2 * gamma(2 * hd + 16) + 2.0 ** -21) * scale * (aq @ aK.T)
    delta += 6 * U32 * scale * (np.stack([rope_pair_abs(y) for y in yq.astype(np.float64)]) @ aK.T)
    delta += 2.0 ** -33 * scale * aq.max(-1, keepdims=True) * aK.sum(-1)
    w = (delta + 2.0 ** -20 + 4 * U32 * (np.abs(s) + np.abs(top) + 32)) * p
    # sum_t w_t |V_t - o|, in pieces of the positions
    tol = np.zeros_like(o)
    for i in range(0, n, 512):
        tol += np.einsum("gt,gtd->gd", w[:, i:i + 512], np.abs(V[None, i:i + 512] - o[:, None]))
    tol += 2 * gamma(n // 8 + 64) * (p @ np.abs(V)) + 16 * U32 * np.abs(o) + n * 2.0 ** -37 * np.abs(V).max() + 1e-30
    return o, tol


class World:
    """Sequences with random rows, their pages, and the projections of `n` new rows each (decode: one)."""

    def __init__(self, nq, nkv, hd, lens, n=None, page=128, seed=0, window=0, sinks=0, spare=1, pad_y=0, pad_o=0, qmul=1.5,
                 gap_rows=0, far_page=0, kmul=1.0, vmul=1.0):
        import torch
        self.t = torch
        rng = self.rng = np.random.default_rng(seed * 977 + hd + 3 * nq + sum(lens))
        self.nq, self.nkv, self.hd, self.page, self.window, self.sinks = nq, nkv, hd, page, window, sinks
        self.lens, self.n = list(lens), [1] * len(lens) if n is None else list(n)
        B = self.B = len(lens)
        ends = [T + k for T, k in zip(self.lens, self.n)]
        self.max_pages = (max(max(ends), 1) + page - 1) // page + spare
        self.cap = self.max_pages * page
        self.start = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        self.rows = int(self.start[-1]) + gap_rows  # rows of y behind the last sequence's
        self.ldy, self.ldo = (nq + 2 * nkv) * hd + pad_y, nq * hd + pad_o
        self.y = rng.standard_normal((max(self.rows, 1), self.ldy)).astype(np.float32)
        self.y[:, :nq * hd] *= qmul
        self.y[:, nq * hd:(nq + nkv) * hd] *= kmul
        self.y[:, (nq + nkv) * hd:(nq + 2 * nkv) * hd] *= vmul
        self.rope = rope_np(self.cap, hd)
        # the rows so far (as a bf16 cache would hold them), then the new ones
        self.hist = [to_bf16(rng.standard_normal((2, nkv, T, hd)).astype(np.float32) *
                             np.array([kmul, vmul], dtype=np.float32)[:, None, None, None]) for T in self.lens]
        self.table = np.full((B, self.max_pages), -1, dtype=np.int32)
        used = [(b, i) for b in range(B) for i in range(self.max_pages) if self.needs(b, i)]
        self.pool = len(used) + 2 + far_page
        ids = rng.permutation(len(used) + 2)[:len(used)] + far_page
        bad = rng.choice([-1, -7, self.pool, 2 ** 31 - 1], size=self.table.shape)  # entries that no call may follow
        self.table[:] = bad
        for (b, i), p in zip(used, ids):
            self.table[b, i] = p
        self.bpp = page // BLOCK

    def needs(self, b, i):
        """Whether page i of sequence b holds rows that the calls read or close."""
        T, end = self.lens[b], self.lens[b] + self.n[b]
        lo, hi = i * self.page, (i + 1) * self.page
        if lo >= end // BLOCK * BLOCK:
            return False
        if not self.window:
            return True
        return lo < self.sinks or hi > T - self.window + 1 or hi > T // BLOCK * BLOCK

    def fill(self):
        """The device's cache: closed blocks in their pages and open rows in the tails; anything else is noise and NaN."""
        t, nkv, hd, page = self.t, self.nkv, self.hd, self.page
        g = t.Generator(device="cuda")
        g.manual_seed(self.pool * 31 + hd)
        # rows of pages lie apart: page_stride and scale_stride longer than they need be
        self.ps, self.ss = nkv * page * hd + 48, nkv * self.bpp + 3
        self.d = {}
        for k in "KV":
            # (16-byte aligned, at an odd multiple of 16)
            raw = t.randint(-128, 128, (self.pool * self.ps + 16,), generator=g, device="cuda", dtype=t.int8)
            self.d[k] = raw[16:]
            self.d[k + "s"] = t.full((self.pool * self.ss,), float("nan"), device="cuda")
        self.ts = 2 * nkv * BLOCK * hd + 8
        self.d["tail"] = t.full((self.B * self.ts,), float("nan"), dtype=t.bfloat16, device="cuda")
        for b, T in enumerate(self.lens):
            if T < 0:
                continue
            nb = T // BLOCK
            x = self.hist[b][:, :, :nb * BLOCK].reshape(2, nkv, nb, BLOCK, hd)
            c, s = close(x)
            for i in range((nb + self.bpp - 1) // self.bpp):
                p = self.table[b, i]
                if not self.needs(b, i):
                    continue
                lo, hi = i * self.bpp, min(nb, (i + 1) * self.bpp)
                for w, k in enumerate("KV"):
                    pg = self.d[k][int(p) * self.ps:int(p) * self.ps + nkv * page * hd].view(nkv, self.bpp, BLOCK, hd)
                    pg[:, :hi - lo] = t.from_numpy(np.ascontiguousarray(c[w, :, lo:hi])).cuda()
                    sc = self.d[k + "s"][int(p) * self.ss:int(p) * self.ss + nkv * self.bpp].view(nkv, self.bpp)
                    sc[:, :hi - lo] = t.from_numpy(np.ascontiguousarray(s[w, :, lo:hi])).cuda()
            rest = self.hist[b][:, :, nb * BLOCK:]
            tl = self.d["tail"][b * self.ts:b * self.ts + 2 * nkv * BLOCK * hd].view(2, nkv, BLOCK, hd)
            tl[:, :, :T - nb * BLOCK] = t.from_numpy(rest.copy()).cuda().bfloat16()
        f = lambda a: t.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.d |= dict(y=f(self.y), rope=f(self.rope), table=f(self.table), start=f(self.start),
                       len=t.tensor(self.lens, dtype=t.int32, device="cuda"))
        self.o = t.full((max(self.rows, 1), self.ldo), -77.0, device="cuda")
        self.new = t.full((max(self.rows, 1), 2, nkv, hd), -77.0, device="cuda")
        return self

    def kv(self, **over):
        from bandwidth_bound_hybrid_gb300 import capi
        d = self.d
        a = dict(k_codes=d["K"].data_ptr(), v_codes=d["V"].data_ptr(), k_scales=d["Ks"].data_ptr(), v_scales=d["Vs"].data_ptr(),
                 page_stride=self.ps, scale_stride=self.ss, page_tokens=self.page, pool_pages=self.pool, tail=d["tail"].data_ptr(),
                 tail_stride=self.ts * 2, table=d["table"].data_ptr(), max_pages=self.max_pages)
        a.update(over)
        return capi.hy_kv_p8(*a.values())

    # ------------------------------------------------------------ calls
    def _stream(self, stream):
        return self.t.cuda.current_stream().cuda_stream if stream is None else stream

    def append(self, L, stream=None, new=True, **over):
        import ctypes
        d, kv = self.d, self.kv()
        a = dict(y=d["y"].data_ptr(), ldy=self.ldy, n=self.rows, batch=self.B, start=d["start"].data_ptr(), kv=ctypes.byref(kv),
                 nq=self.nq, nkv=self.nkv, hd=self.hd, len=d["len"].data_ptr(), rope=d["rope"].data_ptr(),
                 new=self.new.data_ptr() if new else None, stream=self._stream(stream))
        a.update(over)
        return L.hy_op_kv_append_p8(*a.values())

    def workspace(self, L, prompt=False):
        n = (L.hy_op_attention_p8_prompt_workspace(self.rows, self.B, self.nq, self.nkv, self.hd) if prompt else
             L.hy_op_attention_p8_workspace(self.B, self.nq, self.nkv, self.hd))
        assert n > 0
        # the prompt's needs no zeroing
        return self.t.full((n,), 255 if prompt else 0, dtype=self.t.uint8, device="cuda")

    def decode(self, L, ws, stream=None, new=True, **over):
        import ctypes
        d, kv = self.d, self.kv()
        a = dict(y=d["y"].data_ptr(), ldy=self.ldy, batch=self.B, kv=ctypes.byref(kv), nq=self.nq, nkv=self.nkv, hd=self.hd,
                 window=self.window, sinks=self.sinks, len=d["len"].data_ptr(), rope=d["rope"].data_ptr(), o=self.o.data_ptr(),
                 ldo=self.ldo, new=self.new.data_ptr() if new else None, ws=ws.data_ptr(), stream=self._stream(stream))
        a.update(over)
        return L.hy_op_attention_p8(*a.values())

    def prompt(self, L, ws, stream=None, **over):
        import ctypes
        d, kv = self.d, self.kv()
        a = dict(y=d["y"].data_ptr(), ldy=self.ldy, n=self.rows, batch=self.B, start=d["start"].data_ptr(), kv=ctypes.byref(kv),
                 nq=self.nq, nkv=self.nkv, hd=self.hd, window=self.window, sinks=self.sinks, len=d["len"].data_ptr(),
                 rope=d["rope"].data_ptr(), o=self.o.data_ptr(), ldo=self.ldo, ws=ws.data_ptr(), stream=self._stream(stream))
        a.update(over)
        return L.hy_op_attention_p8_prompt(*a.values())

    # ------------------------------------------------------------ what is expected
    def all_rows(self, b):
        """bf16 rows [2, nkv, T + n, hd] of sequence b after the append."""
        nq, nkv, hd, T, n = self.nq, self.nkv, self.hd, self.lens[b], self.n[b]
        y = self.y[self.start[b]:self.start[b + 1], :(nq + 2 * nkv) * hd].reshape(n, nq + 2 * nkv, hd)
        with np.errstate(invalid="ignore", over="ignore"):
            k = rotate32(y[:, nq:nq + nkv], self.rope[T:T + n][:, None])
        new = to_bf16(np.stack([k, y[:, nq + nkv:]], 0).transpose(0, 2, 1, 3))
        return np.concatenate([self.hist[b], new], 2)

    def held(self, b):
        """Values [2, nkv, T + n, hd] (FP64) as held after the append."""
        x = self.all_rows(b)
        out = x.astype(np.float64)
        nb = x.shape[2] // BLOCK
        if nb:
            c, s = close(x[:, :, :nb * BLOCK].reshape(2, self.nkv, nb, BLOCK, self.hd))
            out[:, :, :nb * BLOCK] = (c.astype(np.float64) * s.astype(np.float64)[..., None, None]).reshape(2, self.nkv, -1, self.hd)
        return out

    def snapshot(self):
        t = self.t
        t.cuda.synchronize()
        return {k: self.d[k].view({t.int8: t.int8, t.float32: t.int32, t.bfloat16: t.int16}[self.d[k].dtype]).clone()
                for k in ("K", "V", "Ks", "Vs", "tail")}

    def check_append(self, before, refused=(), new=True, lost=()):
        """The cache after the append: closed blocks, tails and every other byte as it was; kv_new.  lost: (b, page) not written."""
        t, nkv, hd = self.t, self.nkv, self.hd
        t.cuda.synchronize()
        want = {k: v.clone() for k, v in before.items()}
        nan16 = 0x7fc0
        got_new = self.new.cpu().numpy()
        for b in range(self.B):
            r0, r1 = self.start[b], self.start[b + 1]
            if b in refused:
                if 0 <= r0 <= r1:
                    assert (got_new[r0:r1] == -77).all()
                continue
            T, n = self.lens[b], self.n[b]
            if n == 0:
                continue
            x = self.all_rows(b)
            j0, j1, end = T // BLOCK, (T + n) // BLOCK, T + n
            c, s = close(x[:, :, j0 * BLOCK:j1 * BLOCK].reshape(2, nkv, j1 - j0, BLOCK, hd))
            for j in range(j0, j1):
                p = int(self.table[b, j // self.bpp])
                if (b, j // self.bpp) in lost:
                    continue
                for w, k in enumerate("KV"):
                    pg = want[k][p * self.ps:p * self.ps + nkv * self.page * hd].view(nkv, self.bpp, BLOCK, hd)
                    pg[:, j % self.bpp] = t.from_numpy(c[w, :, j - j0].copy()).cuda()
                    sc = want[k + "s"][p * self.ss:p * self.ss + nkv * self.bpp].view(nkv, self.bpp)
                    sc[:, j % self.bpp] = t.from_numpy(s[w, :, j - j0].copy()).cuda().view(t.int32)
            lo = max(T, j1 * BLOCK)
            tl = want["tail"][b * self.ts:b * self.ts + 2 * nkv * BLOCK * hd].view(2, nkv, BLOCK, hd)
            rows = x[:, :, lo:end]
            rb = np.where(np.isnan(rows), nan16, bits16(rows)).astype(np.uint16)
            tl[:, :, lo - j1 * BLOCK:end - j1 * BLOCK] = t.from_numpy(rb.view(np.int16).copy()).cuda()
            if new:
                h = self.held(b)[:, :, T:].transpose(2, 0, 1, 3)
                with np.errstate(over="ignore"):
                    np.testing.assert_array_equal(got_new[r0:r1], h.astype(np.float32))
        if not new:
            assert (got_new == -77).all()
        else:
            assert (got_new[self.start[self.B]:] == -77).all() or refused
        got = self.snapshot()
        for k in want:
            assert t.equal(got[k], want[k]), (k, (got[k] != want[k]).nonzero()[:4].tolist(), (got[k] != want[k]).sum().item())

    def check_attention(self, refused=(), sample=None):
        """The outputs (and those that stay as they were).  sample: at most so many rows of a sequence, ends and borders first."""
        self.t.cuda.synchronize()
        nq, nkv, hd, G = self.nq, self.nkv, self.hd, self.nq // self.nkv
        got = self.o.cpu().numpy()
        np.testing.assert_array_equal(got[:, nq * hd:], -77.0)
        np.testing.assert_array_equal(got[int(self.start[self.B]):], -77.0) if not refused else None
        for b in range(self.B):
            r0, r1, T = int(self.start[b]), int(self.start[b + 1]), self.lens[b]
            if b in refused:
                assert (got[max(r0, 0):max(r1, 0)] == -77).all()
                continue
            rows = range(r1 - r0)
            if sample and r1 - r0 > sample:
                near = {0, 1, r1 - r0 - 1, (r1 - r0) // 2} | {i for i in rows if (T + i) % 128 in (0, 127)}
                rows = sorted(near | set(self.rng.choice(r1 - r0, sample, replace=False).tolist()))[:4 * sample]
            if not len(rows):
                continue
            held, u = self.held(b), np.arange(T + self.n[b])
            for i in rows:
                t = T + i
                for g in range(nkv):
                    yq = self.y[r0 + i, g * G * hd:(g + 1) * G * hd].reshape(G, hd)
                    o, tol = attend(yq, self.rope[t][None], held[0, g], held[1, g], u, t, self.window, self.sinks)
                    assert_elementwise(got[r0 + i, g * G * hd:(g + 1) * G * hd].reshape(G, hd), o, tol,
                                       f"sequence {b} (T={T}), row {i}, kv head {g}")
