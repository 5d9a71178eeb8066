"""What MoETrainLayer keeps between its passes, with the library's calls replaced by recorders: nothing
here needs a GPU."""
import dataclasses

import pytest
import torch

import synth


@pytest.fixture
def layer(monkeypatch):
    """(a layer on the CPU, the names of the calls it made)"""
    import __graft_entry__
    __graft_entry__.build()
    from combine_grouped_gemm_gb300 import train
    calls = []
    for name in ("route", "dispatch", "act_save", "act_load", "combine", "combine_grad",
                 "grouped_mm", "grouped_mm_dx", "grouped_mm_dw", "swiglu_save", "swiglu_grad"):
        monkeypatch.setattr(train, name, lambda *a, _name=name, **k: calls.append(_name))
    cfg = dataclasses.replace(synth.CONFIGS["tiny"], T=8, d_ff_shared=128, R=1)
    z = torch.zeros
    W = dict(w13=z(1), w2=z(1), ws13=z(1), ws2=z(1))

    def make(**kw):
        del calls[:]
        return train.MoETrainLayer(cfg, None, None, W, "cpu", **kw), calls
    make.x = z((cfg.T, cfg.d), dtype=torch.bfloat16)
    return make


def test_one_backward_a_forward(layer):
    """backward writes over what the forward left (the expert rows, the gate/up codes' buffers), so
    a second one, or one before any forward, has nothing to work on."""
    lay, calls = layer()
    with pytest.raises(RuntimeError, match="forward"):
        lay.backward(layer.x)
    assert not calls
    for _ in range(2):
        lay.forward(layer.x)
        lay.forward(layer.x)   # the last one counts
        lay.backward(layer.x)
        done = len(calls)
        with pytest.raises(RuntimeError, match="forward"):
            lay.backward(layer.x, accumulate=True)
        assert len(calls) == done


def test_sums_need_fp32_gradients(layer):
    """Refused before the first call, so that the forward's values are still there."""
    lay, calls = layer(grad_dtype=torch.bfloat16)
    lay.forward(layer.x)
    done = len(calls)
    with pytest.raises(ValueError, match="float32"):
        lay.backward(layer.x, accumulate=True)
    assert len(calls) == done
    lay.backward(layer.x)


def test_gradients_start_at_zero(layer, monkeypatch):
    """So that every micro-batch, the first one too, may be added. (The layer's memory comes filled
    with 7s here, as any bytes may.)"""
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **k).fill_(7))
    lay, _ = layer()
    for n in ("dw13", "dw2", "dws13", "dws2"):
        assert not bool(lay.grads[n].any()), n


def test_rows_of_another_size_are_refused(layer):
    """The router and the combine read and write T rows of d whatever they are given."""
    lay, calls = layer()
    x = layer.x
    for bad in (x[:-1], x[:, :-8], x.float(), None):
        with pytest.raises(ValueError, match="x must be"):
            lay.forward(bad)
        if bad is not None:
            with pytest.raises(ValueError, match="y must be"):
                lay.forward(x, bad)
    assert not calls
