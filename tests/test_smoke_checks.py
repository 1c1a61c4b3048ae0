"""The smoke check fails where an operator's result is not a number or off."""
import math

import pytest
import torch

import __graft_entry__ as entry


@pytest.mark.parametrize("errors", [[math.nan, 0.0], [0.0, math.nan], [torch.tensor([[0.0, math.nan]]), torch.zeros(2, 3)]])
def test_the_worst_error_is_nan_if_one_is(errors):
    assert math.isnan(entry._worst(errors))


def test_the_worst_error():
    assert entry._worst([0.25, torch.tensor([[1.0], [-3.0]]), -1.0]) == 1.0


@pytest.fixture
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from head_attention_forward_02_gb300 import build
    build.build()
    return torch.device("cuda", 0)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["o", "lse", "lse_off", "cache"])
def test_pages(dev, monkeypatch, what):
    from head_attention_forward_02_gb300 import fmha
    entry._smoke_pages(dev)                              # as it is: no error
    attend, write = fmha.page_fwd, fmha.page_write

    def page_fwd(*args, **kw):
        o, lse = attend(*args, **kw)
        if what == "o":
            o[0, 0, 0] = math.nan
        elif what != "cache":
            lse[-1, -1] += math.nan if what == "lse" else 0.1
        return o, lse

    def page_write(k, v, slots, *pool):
        write(k, v, slots, *pool)
        if what == "cache":
            pool[3][slots[:1].long() // 32] = math.nan

    monkeypatch.setattr(fmha, "page_fwd", page_fwd)
    monkeypatch.setattr(fmha, "page_write", page_write)
    with pytest.raises(RuntimeError):
        entry._smoke_pages(dev)


@pytest.mark.gpu
def test_gradients(dev, monkeypatch):
    from head_attention_forward_02_gb300 import fmha
    back = fmha.bwd

    def bwd(*args, **kw):
        dq, dk, dv = back(*args, **kw)
        dk[0, 0, 0, 0] = math.nan
        return dq, dk, dv

    monkeypatch.setattr(fmha, "bwd", bwd)
    with pytest.raises(RuntimeError, match="backward"):
        entry.smoke()
