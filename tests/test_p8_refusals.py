"""Argument checks of the paged 8-bit KV cache's calls: refused on the host, before any device call (CPU only)."""
import ctypes

import pytest

from bandwidth_bound_hybrid_gb300 import capi

A = 4096  # a 16-byte aligned stand-in address: never read, the calls are refused
ARG, UNSUPPORTED = capi.HY_ERR_ARG, capi.HY_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    from bandwidth_bound_hybrid_gb300 import build
    build.build()
    return capi.lib()


def cache(**over):
    a = dict(k_codes=A, v_codes=A, k_scales=A, v_scales=A, page_stride=2 * 128 * 64, scale_stride=2 * 8, page_tokens=128, pool_pages=9,
             tail=A, tail_stride=64 * 2 * 64, table=A, max_pages=5)
    assert set(over) <= set(a)
    a.update(over)
    return capi.hy_kv_p8(*a.values())


def call(L, op, kv=None, null_kv=False, **over):
    kv = kv or cache()
    ref = None if null_kv else ctypes.byref(kv)
    if op == "append":
        a = dict(y=A, ldy=12 * 64, n=5, batch=2, start=A, kv=ref, nq=8, nkv=2, hd=64, len=A, rope=A, new=None, stream=None)
        f = L.hy_op_kv_append_p8
    elif op == "decode":
        a = dict(y=A, ldy=12 * 64, batch=2, kv=ref, nq=8, nkv=2, hd=64, window=0, sinks=0, len=A, rope=A, o=A, ldo=8 * 64, new=None, ws=A,
                 stream=None)
        f = L.hy_op_attention_p8
    else:
        a = dict(y=A, ldy=12 * 64, n=5, batch=2, start=A, kv=ref, nq=8, nkv=2, hd=64, window=0, sinks=0, len=A, rope=A, o=A, ldo=8 * 64,
                 ws=A, stream=None)
        f = L.hy_op_attention_p8_prompt
    assert set(over) <= set(a), over
    a.update(over)
    return f(*a.values())


OPS = ["append", "decode", "prompt"]


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("over", [dict(y=None), dict(y=A + 2), dict(ldy=12 * 64 - 1), dict(ldy=-1), dict(batch=0), dict(batch=-1), dict(nq=0),
                                  dict(nq=7), dict(nkv=0), dict(nkv=-2), dict(hd=0), dict(hd=-64), dict(len=None), dict(len=A + 1), dict(rope=None),
                                  dict(rope=A + 4)])
def test_bad_arguments(L, op, over):
    assert call(L, op, **over) == ARG
    assert L.hy_last_error()


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("over", [dict(k_codes=None), dict(v_codes=A + 8), dict(k_scales=None), dict(v_scales=A + 2), dict(tail=None),
                                  dict(tail=A + 8), dict(table=None), dict(table=A + 2), dict(page_tokens=0), dict(page_tokens=-16),
                                  dict(page_tokens=120), dict(pool_pages=0), dict(pool_pages=-1), dict(max_pages=0), dict(max_pages=-4),
                                  dict(page_stride=2 * 128 * 64 - 16), dict(page_stride=2 * 128 * 64 + 8), dict(page_stride=-16),
                                  dict(scale_stride=15), dict(scale_stride=-1), dict(tail_stride=64 * 2 * 64 - 16),
                                  dict(tail_stride=64 * 2 * 64 + 2), dict(tail_stride=0)])
def test_bad_cache(L, op, over):
    assert call(L, op, cache(**over)) == ARG


@pytest.mark.parametrize("op", OPS)
def test_no_cache(L, op):
    assert call(L, op, null_kv=True) == ARG


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("over", [dict(hd=96), dict(hd=32), dict(nq=6), dict(nq=32), dict(nq=2048, nkv=2048), dict(batch=257)])
def test_unsupported_shapes(L, op, over):
    assert call(L, op, ldy=2 ** 31 - 1, **over) == UNSUPPORTED


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("over", [dict(page_tokens=65552, page_stride=1 << 30, scale_stride=1 << 20),
                                  dict(page_tokens=65536, max_pages=32768, page_stride=1 << 30, scale_stride=1 << 20)])
def test_unsupported_caches(L, op, over):
    assert call(L, op, cache(**over)) == UNSUPPORTED


@pytest.mark.parametrize("op", ["decode", "prompt"])
@pytest.mark.parametrize("over", [dict(o=None), dict(o=A + 2), dict(ldo=8 * 64 - 1), dict(ldo=-5), dict(ws=None), dict(ws=A + 8), dict(window=-1),
                                  dict(sinks=-1)])
def test_bad_attention_arguments(L, op, over):
    assert call(L, op, **over) == ARG


def test_other_pointers(L):
    for op in ("append", "prompt"):
        assert call(L, op, start=None) == ARG
        assert call(L, op, start=A + 1) == ARG
        assert call(L, op, n=-1) == ARG
    for op in ("append", "decode"):
        assert call(L, op, new=A + 1) == ARG
    # lists of tiles and of steps past their counters
    assert call(L, "decode", cache(max_pages=1 << 24), batch=256) == UNSUPPORTED
    assert call(L, "prompt", cache(max_pages=1 << 24), n=1 << 20) == UNSUPPORTED


def test_no_rows_do_nothing(L):
    assert call(L, "append", n=0) == capi.HY_OK
    assert call(L, "append", n=0, y=None) == capi.HY_OK
    assert call(L, "prompt", n=0, y=None, o=None) == capi.HY_OK
    assert call(L, "append", n=0, hd=48) == UNSUPPORTED  # the shape is still checked


def test_workspaces_of_bad_shapes(L):
    for s in ((0, 8, 2, 64), (257, 8, 2, 64), (1, 7, 2, 64), (1, 8, 0, 64), (1, 8, 2, 96), (1, 32, 2, 64), (1, 6, 2, 64)):
        assert L.hy_op_attention_p8_workspace(*s) == 0
        assert L.hy_op_attention_p8_prompt_workspace(10, *s) == 0
    assert L.hy_op_attention_p8_prompt_workspace(-1, 1, 8, 2, 64) == 0
