"""HybridModel.beam_step's refusals, over a stand-in for the library (CPU only):
a step that the selection or the reordering would refuse is refused before any
sequence goes on."""
import types

import pytest
import torch

from bandwidth_bound_hybrid_gb300 import capi, model

V = 50


class Library:
    """Records the calls; sequence lengths as given."""

    def __init__(self, lens):
        self.lens, self.calls = lens, []

    def hy_seq_len(self, cache, seq):
        return self.lens[seq]

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return capi.HY_OK
        return call


def step(monkeypatch, n=3, lens=(7, 7, 7, 9), seqs=(0, 1, 2), **kw):
    lib = Library(list(lens))
    monkeypatch.setattr(capi, "lib", lambda: lib)
    m = model.HybridModel.__new__(model.HybridModel)
    m.shape, m.m, m.c = types.SimpleNamespace(vocab=V), 1, 1
    i32 = dict(dtype=torch.int32)
    beams = types.SimpleNamespace(tokens=torch.zeros(n, **i32), scores=torch.zeros(n), done=torch.zeros(n, **i32),
                                  parent=torch.zeros(n, **i32), ids=torch.zeros(n, **i32), logits=torch.zeros(n, V),
                                  workspace=torch.zeros(256))
    try:
        m.beam_step(seqs, beams, stream=types.SimpleNamespace(cuda_stream=0), **kw)
    finally:
        m.m = m.c = None
        step.calls = lib.calls
    return lib.calls


def test_a_good_step_decodes_selects_and_reorders(monkeypatch):
    want = ["hy_decode_step", "hy_op_beam_select", "hy_seq_reorder"]
    for kw in (dict(), dict(eos=-1), dict(eos=0), dict(eos=V - 1, first=7), dict(seqs=range(3))):
        assert step(monkeypatch, **kw) == want


@pytest.mark.parametrize("kw", [dict(eos=V), dict(eos=V + 9), dict(first=-1), dict(lens=(7, 7, 8, 9)), dict(seqs=(0, 1, 3)),
                                dict(n=2), dict(seqs=(0, 1))])
def test_refused_before_any_call(monkeypatch, kw):
    with pytest.raises(ValueError):
        step(monkeypatch, **kw)
    assert step.calls == []


@pytest.mark.parametrize("n", [-1, 0, 9, 16])
def test_beam_state_of_more_beams_than_a_step_takes(n):
    with pytest.raises(ValueError, match="1..8"):
        model.BeamState(n, V, 0)
