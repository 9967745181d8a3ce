"""The oracle's 4-bit KV cache: worked examples, invariants, agreement with a
numpy form and with the bf16 attention on exact values, and the two-token
closed form of a whole model."""
import dataclasses

import numpy as np

from bandwidth_bound_hybrid_gb300 import accounting as acc
from oracle import oracle as orc
from synth import gen, workloads
from tests import test_oracle_model as tom


def quant_np(x):
    b = np.asarray(x, dtype=np.float32).reshape(-1, 32)
    s = np.minimum(np.abs(b).max(-1) * (np.float32(1) / np.float32(7)), np.float32(65504)).astype(np.float16).astype(np.float32)
    inv = np.where(s > 0, np.float32(1) / np.where(s > 0, s, np.float32(1)), np.float32(0))
    return np.clip(np.rint(b * inv[:, None]), -7, 7).ravel(), s


def test_quant_worked_example():
    x = np.zeros(64)
    x[:4] = [7.0, -3.5, 0.49, 1.5]  # scale 1: codes 7, -4 (half to even), 0, 2 (half to even)
    x[32:35] = [-1.75, 0.125, 0.375]  # scale 0.25: -7, 0 (0.5 to even), 2 (1.5 to even)
    q, s = orc.quant_q4(x)
    assert s.tolist() == [1.0, 0.25]
    assert q[:4].tolist() == [7, -4, 0, 2] and q[32:35].tolist() == [-7, 0, 2] and not q[4:32].any() and not q[35:].any()


def test_quant_against_numpy_and_invariants():
    rng = np.random.default_rng(5)
    for n in (64, 128, 256):
        for mag in (1e-9, 1e-7, 1e-4, 1.0, 30.0, 1e5, 1e7):
            x = (rng.standard_normal(n) * mag).astype(np.float32).astype(np.float64)
            q, s = orc.quant_q4(x)
            qn, sn = quant_np(x)
            np.testing.assert_array_equal(q, qn)
            np.testing.assert_array_equal(s, sn)
            np.testing.assert_array_equal(orc.quant_q4(-x)[0], -q)
            if 1e-3 < mag < 1e5:  # inside fp16's normal scales: within half a step, and the scale's own rounding
                step = np.repeat(s, 32).astype(np.float64)
                assert np.all(np.abs(x - q * step) <= step * (0.5 + 7 * 2.0 ** -11))
                assert np.abs(q).reshape(-1, 32).max(-1).min() == 7


def test_attention_equals_bf16_attention_on_exact_values():
    rng = np.random.default_rng(3)
    nq, nkv, hd, cap, npos = 4, 2, 64, 9, 7
    Kq, Vq = (rng.integers(-7, 8, (nkv, cap, hd)).astype(np.int8) for _ in range(2))
    Ks, Vs = (np.exp2(rng.integers(-4, 3, (nkv, cap, hd // 32))).astype(np.float32) for _ in range(2))
    q = rng.standard_normal((nq, hd))
    Kb, Vb = (gen.f32_to_bf16_bits((c.reshape(nkv, cap, -1, 32) * s[..., None]).astype(np.float32).reshape(nkv, cap, hd))
              for c, s in ((Kq, Ks), (Vq, Vs)))
    np.testing.assert_allclose(orc.attention_q4(q, Kq, Ks, Vq, Vs, npos), orc.attention(q, Kb, Vb, npos), rtol=1e-12, atol=1e-14)


def test_two_token_closed_form(monkeypatch):
    def kv_round(shape, x):
        out = np.empty_like(x)
        for i, r in enumerate(np.atleast_2d(x)):
            q, s = quant_np(r)
            out[i] = q * np.repeat(s, 32).astype(np.float64)
        return out

    monkeypatch.setattr(tom, "_kv_round", kv_round)
    tom._check_closed_form(dataclasses.replace(workloads.TINY, name="tiny-kv4", kv_format=2), ((0, 77), (1023, 1023), (5, 6)))


def test_bytes_of_the_formats():
    assert acc.kv_bytes_per_token(8, 4, 128) == 16384
    assert acc.kv_bytes_per_token(8, 4, 128, kv_format=1) == 8 * 2 * 4 * 132
    assert acc.kv_bytes_per_token(8, 4, 128, kv_format=2) == 8 * 2 * 4 * 72
