"""Argument checks of the 4-bit cache and beam search operators: refused on the
host, before any device call (CPU only)."""
import os
import subprocess
import sys

import pytest

from bandwidth_bound_hybrid_gb300 import capi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 4096  # a 16-byte aligned stand-in address: never read, the calls are refused


@pytest.fixture(scope="module")
def L():
    from bandwidth_bound_hybrid_gb300 import build
    build.build()
    return capi.lib()


def attn(L, **over):
    a = dict(y=A, ldy=(8 + 4) * 64, batch=2, Kq=A, Ks=A, Vq=A, Vs=A, cap=100, nq=8, nkv=2, hd=64, len=A, rope=A, o=A, ldo=8 * 64,
             new=None, ws=A, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return L.hy_op_attention_q4(*a.values())


@pytest.mark.parametrize("over", [dict(y=None), dict(Kq=None), dict(Ks=A + 8), dict(Vq=A + 4), dict(Vs=None), dict(len=None),
                                  dict(rope=None), dict(o=None), dict(ws=None), dict(ws=A + 1), dict(cap=0), dict(cap=-3),
                                  dict(batch=0), dict(batch=9), dict(nq=0), dict(nkv=0), dict(nq=7), dict(ldy=12 * 64 - 1),
                                  dict(ldo=8 * 64 - 1), dict(ldy=-1), dict(y=A + 2), dict(len=A + 1),
                                  dict(rope=A + 4), dict(o=A + 3), dict(new=A + 2)])
def test_attention_q4_bad_arguments(L, over):
    assert attn(L, **over) == capi.HY_ERR_ARG
    assert L.hy_last_error()


@pytest.mark.parametrize("over", [dict(hd=96, ldy=10 ** 6, ldo=10 ** 6), dict(nq=6, ldy=10 ** 6, ldo=10 ** 6),
                                  dict(nq=32, ldy=10 ** 6, ldo=10 ** 6), dict(nq=2048, nkv=2048, ldy=10 ** 6, ldo=10 ** 6),
                                  dict(cap=2 ** 31 - 1, nkv=1024, nq=1024, ldy=10 ** 6, ldo=10 ** 6)])
def test_attention_q4_unsupported_shapes(L, over):
    assert attn(L, **over) == capi.HY_ERR_UNSUPPORTED


def test_attention_q4_workspace_of_bad_shapes(L):
    for shape in ((0, 8, 2, 64), (9, 8, 2, 64), (1, 7, 2, 64), (1, 8, 0, 64), (1, 8, 2, 96), (1, 32, 2, 64), (1, 6, 2, 64)):
        assert L.hy_op_attention_q4_workspace(*shape) == 0


def append(L, **over):
    a = dict(y=A, ldy=12 * 64, n=5, Kq=A, Ks=A, Vq=A, Vs=A, cap=100, nq=8, nkv=2, hd=64, len=A, rope=A, new=None, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return L.hy_op_kv_append_q4(*a.values())


def test_append_q4_refusals(L):
    for over in (dict(y=None), dict(Kq=A + 2), dict(Ks=None), dict(Vq=None), dict(Vs=None), dict(n=-1), dict(cap=0), dict(len=None),
                 dict(rope=None), dict(ldy=12 * 64 - 1), dict(nq=3), dict(y=A + 1), dict(rope=A + 4), dict(new=A + 2), dict(len=A + 2)):
        assert append(L, **over) == capi.HY_ERR_ARG, over
    assert append(L, hd=80, ldy=10 ** 6) == capi.HY_ERR_UNSUPPORTED
    assert append(L, nq=32, ldy=10 ** 6) == capi.HY_ERR_UNSUPPORTED
    assert append(L, n=101) == capi.HY_ERR_CAPACITY
    assert append(L, n=0) == capi.HY_OK
    assert append(L, n=0, y=None) == capi.HY_OK


def select(L, **over):
    a = dict(logits=A, ldl=1000, groups=2, beams=4, vocab=1000, picks=4, score=A, done=None, eos=-1, so=A, po=A, to=A, do=None, ws=A,
             stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return L.hy_op_beam_select(*a.values())


def test_beam_select_refusals(L):
    for over in (dict(logits=None), dict(score=None), dict(so=None), dict(po=None), dict(to=None), dict(ws=None), dict(ws=A + 8),
                 dict(ldl=999), dict(groups=0), dict(beams=0), dict(vocab=0), dict(picks=0), dict(done=A), dict(done=A, eos=1000),
                 dict(beams=1, vocab=3, ldl=3, picks=4), dict(groups=-1), dict(beams=-2), dict(logits=A + 2), dict(score=A + 1),
                 dict(so=A + 2), dict(po=A + 2), dict(to=A + 2), dict(do=A + 2), dict(done=A + 2, eos=1)):
        assert select(L, **over) == capi.HY_ERR_ARG, over
    for over in (dict(beams=17), dict(picks=33), dict(beams=16, vocab=2 ** 28, ldl=2 ** 28), dict(groups=2 ** 30)):
        assert select(L, **over) == capi.HY_ERR_UNSUPPORTED, over
    for shape in ((0, 1, 10), (1, 0, 10), (1, 17, 10), (1, 1, 0)):
        assert L.hy_op_beam_select_workspace(*shape) == 0
    assert L.hy_op_beam_select_workspace(1, 4, 151936) > 0


def reorder(L, **over):
    a = dict(state=A, stride=4096, n_seg=4, pitch=1024, seg=512, groups=2, beams=4, parent=A, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return L.hy_op_beam_reorder(*a.values())


def test_beam_reorder_refusals(L):
    for over in (dict(state=None), dict(state=A + 4), dict(parent=None), dict(stride=4104), dict(pitch=1032), dict(seg=520),
                 dict(seg=-16), dict(groups=0), dict(beams=0), dict(n_seg=0), dict(pitch=496), dict(stride=3568),
                 dict(n_seg=1, stride=496), dict(stride=-4096), dict(pitch=-1024), dict(parent=A + 2)):
        assert reorder(L, **over) == capi.HY_ERR_ARG, over
    for over in (dict(beams=17), dict(groups=65536), dict(n_seg=65536, pitch=512, stride=2 ** 40)):
        assert reorder(L, **over) == capi.HY_ERR_UNSUPPORTED, over


def test_beam_reorder_of_interleaved_states(L):
    """Segment after segment, each of all states: 8 states of 512 bytes need 4096."""
    for over in (dict(stride=512, pitch=4080), dict(stride=496, pitch=4096), dict(stride=528, pitch=4096),
                 dict(stride=512, pitch=2 ** 40, seg=528), dict(stride=2 ** 62, pitch=2 ** 62)):
        assert reorder(L, **over) == capi.HY_ERR_ARG, over


def test_beam_step_refuses_a_state_of_another_size(L):
    from types import SimpleNamespace

    from bandwidth_bound_hybrid_gb300.model import HybridModel
    m = object.__new__(HybridModel)
    m.shape = SimpleNamespace(vocab=1000)
    m.c = m.m = None
    for shape in ((3, 1000), (4, 999)):
        beams = SimpleNamespace(logits=SimpleNamespace(shape=shape))
        with pytest.raises(ValueError, match="beam state"):
            m.beam_step(range(4), beams)


def without_a_gpu(code):
    """Run Python code (with L, the library, and A) in a process that sees no GPU."""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    pre = f"from bandwidth_bound_hybrid_gb300 import capi\nL = capi.lib()\nA = {A}\n"
    return subprocess.run([sys.executable, "-c", pre + code], cwd=ROOT, env=env, capture_output=True, text=True)


@pytest.mark.parametrize("call", [
    "L.hy_op_beam_select(A, 1000, 1, 4, 1000, 4, A, None, -1, A, A, A, None, A, None)",
    "L.hy_op_beam_reorder(A, 64, 1, 64, 64, 1, 4, A, None)",
    "L.hy_op_attention_q4(A, 768, 1, A, A, A, A, 100, 8, 2, 64, A, A, A, 512, None, A, None)",
    "L.hy_op_kv_append_q4(A, 768, 5, A, A, A, A, 100, 8, 2, 64, A, A, None, None)"])
def test_calls_without_a_gpu_return_an_error(L, call):
    """Good arguments on a machine without a usable GPU: an error code and a message, the process lives."""
    r = without_a_gpu(f"print({call}, bool(L.hy_last_error()))")
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
    assert r.stdout.split() == [str(capi.HY_ERR_CUDA), "True"]


def test_attention_q4_workspace_without_a_gpu(L):
    """The partials' size needs the GPU's SM count: 0, not the counters' size alone."""
    r = without_a_gpu("print(L.hy_op_attention_q4_workspace(1, 8, 2, 64))")
    assert r.returncode == 0 and r.stdout.split() == ["0"], (r.stdout, r.stderr[-2000:])
