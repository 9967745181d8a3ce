"""Whole models with the 4-bit KV cache (kv_format 2) against the oracle's, and
sequences copied, reordered and run as beams.

Model gates are those of test_gpu_model (per-layer hidden relative L2 5e-3,
logits 1e-2): the quantised rows are the same on both sides but for the rare
element whose FP32 and FP64 values lie on the two sides of a rounding border."""
import ctypes
import dataclasses

import numpy as np
import pytest

from bandwidth_bound_hybrid_gb300 import capi
from oracle import oracle as orc
from synth import workloads
from tests.gpu_util import rel_l2, to_np

pytestmark = pytest.mark.gpu

KV4_TINY = dataclasses.replace(workloads.TINY, name="tiny-kv4", kv_format=2)
SHAPES = {
    "bf16": workloads.TINY,
    "int8": dataclasses.replace(workloads.TINY, name="tiny-kv8", kv_format=1),
    "4-bit": KV4_TINY,
    "paged": workloads.TINY,
}


@pytest.fixture(scope="module")
def built(gpu):
    from bandwidth_bound_hybrid_gb300 import build
    build.build()
    return True


def _torch():
    import torch
    return torch


def ints(*v):
    return _torch().tensor(list(v), dtype=_torch().int32, device="cuda")


def test_tiny_against_the_oracle(built):
    """128-token prompt (in chunks on the tensor cores), then 16 decode steps."""
    from tests.test_gpu_model import run_parity
    run_parity(KV4_TINY, 128, 16)


def test_tiny_token_by_token(built):
    from tests.test_gpu_model import run_parity
    run_parity(KV4_TINY, 40, 3, prefill_path=False)


@pytest.mark.parametrize("hd,nq,nkv", [(128, 8, 2), (256, 8, 1)])
def test_head_dims_against_the_oracle(built, hd, nq, nkv):
    from tests.test_gpu_model import run_parity
    run_parity(dataclasses.replace(KV4_TINY, name=f"tiny-kv4-{hd}", head_dim=hd, attn_q_heads=nq, attn_kv_heads=nkv), 70, 3)


def test_moe_4bit_weights_against_the_oracle(built):
    """4-bit weights take the batched path for every step and prompt token."""
    from tests.test_gpu_model import run_parity
    shape = dataclasses.replace(KV4_TINY, name="tiny-moe-q4-kv4", ffn=0, n_experts=16, top_k=4, expert_ffn=256, shared_ffn=256,
                                weight_format=1)
    run_parity(shape, 24, 3)


def test_chunked_prefill_equals_token_by_token(built):
    """A prompt over several chunk lengths leaves the cache that single steps leave."""
    torch = _torch()
    from bandwidth_bound_hybrid_gb300.model import HybridModel
    w = workloads.device_weights(KV4_TINY)
    a = HybridModel(KV4_TINY, w, [400])
    b = HybridModel(KV4_TINY, w, [400], flags=capi.HY_FLAG_TOKEN_PREFILL)
    prompt = torch.from_numpy(workloads.prompt_ids(workloads.WORKLOADS["tiny"], n=100)).cuda()
    la, lb = (torch.empty(KV4_TINY.vocab, device="cuda") for _ in range(2))
    for n0, n1 in ((0, 70), (70, 71), (71, 100)):
        a.prefill(0, prompt[n0:n1], la)
        b.prefill(0, prompt[n0:n1], lb)
        assert rel_l2(to_np(la), to_np(lb)) < 1e-2
    ids = ints(0)
    for t in range(3):
        a.decode_step(0, ints(t + 5), ids, la)
        b.decode_step(0, ints(t + 5), ids, lb)
        assert rel_l2(to_np(la), to_np(lb)) < 1e-2
    assert a.check_device() == 0 and b.check_device() == 0


def test_batch_of_ragged_sequences_against_the_oracle(built):
    torch = _torch()
    from bandwidth_bound_hybrid_gb300.model import HybridModel
    lens = [5, 40, 1, 33]
    model = HybridModel(KV4_TINY, workloads.device_weights(KV4_TINY), [64] * 4)
    host = workloads.host_weights(KV4_TINY)
    refs = [orc.Oracle(KV4_TINY, host, 64) for _ in lens]
    rng = np.random.default_rng(0)
    for s, n in enumerate(lens):
        pr = rng.integers(0, KV4_TINY.vocab, n).astype(np.int32)
        model.prefill(s, torch.from_numpy(pr).cuda())
        for t in pr:
            refs[s].forward(int(t), want_hidden=False)
    logits = torch.empty((4, KV4_TINY.vocab), device="cuda")
    ids = torch.empty(4, dtype=torch.int32, device="cuda")
    for _ in range(3):
        toks = rng.integers(0, KV4_TINY.vocab, 4).astype(np.int32)
        model.decode_batch([0, 1, 2, 3], torch.from_numpy(toks).cuda(), ids, logits)
        got = to_np(logits)
        for s in range(4):
            assert rel_l2(got[s], refs[s].forward(int(toks[s]), want_hidden=False)["logits"]) < 1e-2, s
    assert model.check_device() == 0


def test_synthetic_fill_and_long_context(built):
    """The fill's values are quantised by the cache's rule: the oracle from the same rows agrees."""
    torch = _torch()
    from bandwidth_bound_hybrid_gb300.model import HybridModel
    from synth import gen
    shape = dataclasses.replace(KV4_TINY, name="tiny-kv4-attn", n_layers=1, attn_layers=(0,))
    n, cap = 3000, 3010
    model = HybridModel(shape, workloads.device_weights(shape), [cap])
    model.fill_synthetic(0, n, seed=3)
    ref = orc.Oracle(shape, workloads.host_weights(shape), cap)
    hd, nkv = shape.head_dim, shape.attn_kv_heads
    kq, vq = (np.ctypeslib.as_array(ctypes.cast(p, ctypes.POINTER(ctypes.c_int8)), shape=(nkv, cap, hd))
              for p in (ref.cache.k_q, ref.cache.v_q))
    ks, vs = (np.ctypeslib.as_array(ctypes.cast(p, ctypes.POINTER(ctypes.c_float)), shape=(nkv, cap, hd // 32))
              for p in (ref.cache.k_s, ref.cache.v_s))
    for g in range(nkv):
        for w, (q, s) in enumerate(((kq, ks), (vq, vs))):
            vals = gen.fill_values(3 * 1000003 + w * 64 + g, n * hd).reshape(n, hd)
            for r in range(n):
                q[g, r], s[g, r] = orc.quant_q4(vals[r])
    ref.cache.len = n
    logits = torch.empty(shape.vocab, device="cuda")
    ids = ints(0)
    for t in (3, 9):
        model.decode_step(0, ints(t), ids, logits)
        assert rel_l2(to_np(logits), ref.forward(t, want_hidden=False)["logits"]) < 1e-3
    assert model.check_device() == 0


def test_paged_4bit_cache_is_refused(built):
    from bandwidth_bound_hybrid_gb300.model import HybridModel
    with pytest.raises(capi.HybridError) as e:
        HybridModel(KV4_TINY, workloads.device_weights(KV4_TINY), [64], pages=(128, 4))
    assert e.value.code == capi.HY_ERR_UNSUPPORTED


# ------------------------------------------------------------------ copy, reorder, beams
def make(kind, caps):
    from bandwidth_bound_hybrid_gb300.model import HybridModel
    shape = SHAPES[kind]
    pages = (128, 4 * len(caps)) if kind == "paged" else None
    return HybridModel(shape, workloads.device_weights(shape), caps, pages=pages)


def next_logits(model, seqs, token=11):
    torch = _torch()
    lg = torch.empty((len(seqs), model.shape.vocab), device="cuda")
    ids = torch.empty(len(seqs), dtype=torch.int32, device="cuda")
    model.decode_batch(seqs, ints(*[token] * len(seqs)), ids, lg)
    return to_np(lg)


@pytest.mark.parametrize("kind", list(SHAPES))
def test_reorder_moves_whole_states(built, kind):
    """Sequences of different contents (and capacities): after the reordering each continues as its parent would."""
    caps = [300, 290, 310, 280]
    a, b = make(kind, caps), make(kind, caps)
    for m in (a, b):
        for s in range(4):
            m.fill_synthetic(s, 270, seed=10 + s)
    before = next_logits(b, [0, 1, 2, 3])
    for parent in ([1, 0, 3, 2], [2, 2, 2, 2], [0, 0, 1, 3]):
        for s in range(4):
            a.fill_synthetic(s, 270, seed=10 + s)
        a.reorder([0, 1, 2, 3], ints(*parent))
        got = next_logits(a, [0, 1, 2, 3])
        for s in range(4):
            assert rel_l2(got[s], before[parent[s]]) < 1e-4, (parent, s)
            assert rel_l2(got[s], before[(parent[s] + 1) % 4]) > 1e-3
    assert a.check_device() == 0


def test_reorder_and_copy_refusals(built):
    m = make("4-bit", [64, 64, 20])
    m.fill_synthetic(0, 30, seed=1)
    m.fill_synthetic(1, 31, seed=1)
    for call in (lambda: m.reorder([0, 1], ints(0, 0)), lambda: m.reorder([0, 0], ints(0, 0)), lambda: m.reorder([0, 7], ints(0, 0)),
                 lambda: m.reorder([0, 1], ints(0, 0), first=-1), lambda: m.copy(0, 5)):
        with pytest.raises(capi.HybridError) as e:
            call()
        assert e.value.code == capi.HY_ERR_ARG
    with pytest.raises(capi.HybridError) as e:
        m.copy(0, 2)
    assert e.value.code == capi.HY_ERR_CAPACITY and m.seq_len(2) == 0
    m.copy(0, 0)
    m.copy(0, 1)
    assert m.seq_len(1) == 30
    m.reorder([0, 1], ints(5, 0))
    assert m.check_device() == capi.HY_GUARD_BAD_INDEX


@pytest.mark.parametrize("kind", list(SHAPES))
def test_beam_search(built, kind):
    """Four beams for six steps over copies of one prompt; every surviving hypothesis replayed in a sequence of its own has the
    beam's next logits and score."""
    torch = _torch()
    from bandwidth_bound_hybrid_gb300.model import BeamState
    n, P, steps, V = 4, 150, 6, workloads.TINY.vocab
    m = make(kind, [200] * (2 * n))
    prompt = torch.from_numpy(workloads.prompt_ids(workloads.WORKLOADS["tiny"], n=P)).cuda()
    m.prefill(0, prompt[:-1])
    for s in range(1, 2 * n):
        m.copy(0, s)
    last = int(prompt[-1])
    beams = BeamState(n, V, last)
    seqs, hyp = list(range(n)), [[] for _ in range(n)]
    for _ in range(steps):
        m.beam_step(seqs, beams, first=P - 1)
        par, tok = to_np(beams.parent), to_np(beams.tokens)
        hyp = [hyp[par[i]] + [int(tok[i])] for i in range(n)]
    assert len({tuple(h) for h in hyp}) == n
    sc = to_np(beams.scores)
    assert (np.diff(sc) <= 0).all()
    # replay: the same tokens in the other sequences
    lg = torch.empty((n, V), device="cuda")
    ids = torch.empty(n, dtype=torch.int32, device="cuda")
    total = np.zeros(n)
    other = list(range(n, 2 * n))
    for k in range(steps):
        toks = [last] * n if k == 0 else [h[k - 1] for h in hyp]
        m.decode_batch(other, ints(*toks), ids, lg)
        x = to_np(lg).astype(np.float64)
        x -= x.max(-1, keepdims=True)
        total += (x - np.log(np.exp(x).sum(-1, keepdims=True)))[np.arange(n), [h[k] for h in hyp]]
    np.testing.assert_allclose(sc, total, atol=1e-3)
    m.decode_batch(seqs, beams.tokens, ids, lg)
    mine = to_np(lg).copy()
    m.decode_batch(other, beams.tokens, ids, lg)
    theirs = to_np(lg)
    for i in range(n):
        assert rel_l2(mine[i], theirs[i]) < 1e-3
        assert rel_l2(mine[i], theirs[(i + 1) % n]) > 1e-2
    assert m.check_device() == 0


def test_beam_search_with_an_end_token(built):
    """A beam that ends keeps its score while the others go on."""
    torch = _torch()
    from bandwidth_bound_hybrid_gb300.model import BeamState
    m = make("4-bit", [64] * 3)
    m.prefill(0, ints(1, 2, 3))
    for s in (1, 2):
        m.copy(0, s)
    beams = BeamState(3, KV4_TINY.vocab, 4)
    m.beam_step([0, 1, 2], beams, first=3)
    eos = int(beams.tokens[1])
    beams = BeamState(3, KV4_TINY.vocab, 4)
    m2 = make("4-bit", [64] * 3)
    m2.prefill(0, ints(1, 2, 3))
    for s in (1, 2):
        m2.copy(0, s)
    m2.beam_step([0, 1, 2], beams, eos=eos, first=3)
    assert to_np(beams.done).tolist() == [0, 1, 0]
    ended = float(beams.scores[1])
    for _ in range(4):
        m2.beam_step([0, 1, 2], beams, eos=eos, first=3)
        d, sc, tk = to_np(beams.done), to_np(beams.scores), to_np(beams.tokens)
        assert ended in sc[d == 1].tolist() and (tk[d == 1] == eos).all()
    assert torch.isfinite(beams.scores).all()


@pytest.mark.parametrize("kind,hd", [("bf16", 64), ("int8", 64), ("paged", 64), ("4-bit", 64), ("4-bit", 128), ("4-bit", 256)])
def test_reorder_leaves_the_rows_before_first(built, kind, hd):
    """Unlike sequences reordered from a row inside a 16-byte piece of the scales: every row before it stays the sequence's own,
    every later one is the parent's.  In a one-layer model the rows of a position depend on its token alone, so the
    sequence goes on exactly as one does that was prompted with its own tokens up to `first` and its parent's from there."""
    torch = _torch()
    from bandwidth_bound_hybrid_gb300.model import HybridModel
    shape = dataclasses.replace(SHAPES[kind], name=f"{kind}-{hd}", n_layers=1, attn_layers=(0,), head_dim=hd, attn_q_heads=8,
                                attn_kv_heads=2)
    m = HybridModel(shape, workloads.device_weights(shape), [24, 30, 24, 30], pages=(128, 4) if kind == "paged" else None)
    rng = np.random.default_rng(hd)
    for n in (13, 16):
        for first in (0, 1, 2, 3, 5, 7, 8, 11, n - 1, n):
            prompts = rng.integers(0, shape.vocab, (2, n)).astype(np.int32)
            for s in range(4):
                m.reset(s)
            for s in range(2):
                m.prefill(s, torch.from_numpy(prompts[s]).cuda())
                mixed = np.concatenate([prompts[s, :first], prompts[1 - s, first:]])
                m.prefill(2 + s, torch.from_numpy(mixed).cuda())
            m.reorder([0, 1], ints(1, 0), first=first)
            got = next_logits(m, [0, 1, 2, 3])
            np.testing.assert_array_equal(got[:2], got[2:], err_msg=f"{n} rows from {first} on")
    assert m.check_device() == 0


@pytest.mark.parametrize("kind", list(SHAPES))
def test_copy_over_longer_and_shorter_sequences(built, kind):
    """What the destination held before, longer or shorter or nothing, does not show; the source stays as it is."""
    m = make(kind, [300, 310, 290, 300])
    m.fill_synthetic(0, 150, seed=1)
    m.fill_synthetic(1, 280, seed=2)
    m.fill_synthetic(2, 3, seed=3)
    for s in (1, 2, 3):
        m.copy(0, s)
        assert m.seq_len(s) == 150
    got = [next_logits(m, [s])[0] for s in range(4)]
    for s in (1, 2, 3):
        assert rel_l2(got[s], got[0]) < 1e-5
    m.reset(3)
    m.copy(3, 1)  # an empty sequence
    assert m.seq_len(1) == 0 and m.seq_len(0) == 151
    assert rel_l2(next_logits(m, [1])[0], next_logits(m, [3])[0]) < 1e-5
    assert m.check_device() == 0


@pytest.mark.parametrize("kind", list(SHAPES))
def test_one_beam_is_the_greedy_search(built, kind):
    torch = _torch()
    from bandwidth_bound_hybrid_gb300.model import BeamState
    m = make(kind, [100, 100])
    prompt = torch.from_numpy(workloads.prompt_ids(workloads.WORKLOADS["tiny"], n=40)).cuda()
    m.prefill(0, prompt[:-1])
    m.copy(0, 1)
    beams = BeamState(1, m.shape.vocab, int(prompt[-1]))
    tok, ids = prompt[-1:].clone(), ints(0)
    for _ in range(8):
        m.beam_step([0], beams, first=39)
        m.decode_step(1, tok, ids)
        tok.copy_(ids)
        assert beams.tokens.tolist() == ids.tolist() and beams.parent.tolist() == [0]
    assert m.check_device() == 0
