"""Copies of 4-bit expert weights: copy, deepcopy, pickle and torch.save (no GPU)."""

import copy
import io
import pickle

import pytest
import torch

import sparse_mixture_experts_warp_b200 as M


def _filled(zeros):
    w = M.empty_w4(2, 64, 192, 64, zeros, device="cpu")
    for i, t in enumerate(t for t in (w.codes, w.scales, w.zeros, w.row_scale) if t is not None):
        b = t.view(torch.uint8)
        b.copy_((torch.arange(b.numel()) * (i + 3) % 120).view(b.shape))
    return w


def _saved(w):
    f = io.BytesIO()
    torch.save({"experts": w}, f)
    f.seek(0)
    return torch.load(f, weights_only=False)["experts"]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("again,shared", [
    (copy.copy, True), (copy.deepcopy, False), (_saved, False),
    (lambda w: pickle.loads(pickle.dumps(w)), False)])
def test_copies_of_a_w4(again, shared, zeros):
    """copy, deepcopy, pickle and torch.save give a W4 of the same values whose handle has its own
    tensors' addresses."""
    w = _filled(zeros)
    c = again(w)
    assert isinstance(c, M.W4) and (c.G, c.N, c.K, c.group) == (w.G, w.N, w.K, w.group)
    for name in ("codes", "scales", "zeros", "row_scale"):
        a, b = getattr(w, name), getattr(c, name)
        if a is None:
            assert b is None
            continue
        assert a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert (a.data_ptr() == b.data_ptr()) == shared
        assert getattr(c._ref()._obj, name) == b.data_ptr()
        assert getattr(w._ref()._obj, name) == a.data_ptr()
    with pytest.raises(AttributeError):
        c.codes = w.codes


def test_a_network_that_holds_a_w4_is_copied():
    class Layer(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.up = _filled(False)

    a = Layer()
    b = copy.deepcopy(a)
    assert torch.equal(a.up.codes, b.up.codes) and a.up.codes.data_ptr() != b.up.codes.data_ptr()
