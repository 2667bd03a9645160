"""What copies and pickles of 4-bit weights and of their layers hold, without a GPU."""
import copy
import io
import pickle

import pytest
import torch

sp = pytest.importorskip("unstructured_sparse_linear_gb300")


def elsewhere():
    """A weight whose arrays came back from a file on another device than the one they were on."""
    codes, scales = torch.arange(96, dtype=torch.uint8).view(3, 32), torch.arange(6, dtype=torch.uint8).view(3, 2)
    return sp.Mx4._of(codes, scales, (3, 33), torch.float16, torch.device("cuda", 0))


def saved(W):
    f = io.BytesIO()
    torch.save(W, f)
    f.seek(0)
    return torch.load(f, map_location="cpu", weights_only=False)


@pytest.mark.parametrize("again", [copy.deepcopy, lambda W: pickle.loads(pickle.dumps(W)), saved], ids=["copy", "pickle", "file"])
def test_a_weight_is_where_its_arrays_are(again):
    W = elsewhere()
    V = again(W)
    assert V.device == torch.device("cpu") and V.shape == (3, 33) and V.dtype is torch.float16
    assert torch.equal(V.codes, W.codes) and torch.equal(V.scales, W.scales) and V.codes is not W.codes
    X = torch.zeros(2, 33, dtype=torch.float16)
    for call in (lambda: sp.mx4_linear(X, V), lambda: sp.mx4_linear_grad(X[:, :3], V), lambda: sp.mx4_dequantize(V)):
        with pytest.raises(ValueError, match="W is on cpu"):
            call()


def test_a_layer_pickled_before_it_had_four_bits():
    layer = sp.RosaLinear(torch.randn(6, 8), 2, scale=0.5)
    state = layer.__getstate__()
    state = {k: v for k, v in state.items() if k not in ("dropout", "_quantized")}
    state["_buffers"] = {k: v for k, v in state["_buffers"].items() if k not in ("codes", "scales")}
    old = sp.RosaLinear.__new__(sp.RosaLinear)
    old.__setstate__(state)
    assert old.dropout == 0.0 and old.quantized is None and old.scale == 0.5
    assert torch.equal(old.merged(None), layer.weight) and set(old.state_dict()) == set(layer.state_dict())
    assert set(copy.deepcopy(old)._buffers) == set(layer._buffers)


class Named(sp.Mx4):
    """A weight with an attribute of its own."""


def test_a_kind_of_weight_and_an_older_file():
    W = elsewhere()
    N = Named._of(W.codes, W.scales, W.shape, W.dtype, W.device)
    N.name = "up"
    V = copy.deepcopy(N)
    assert type(V) is Named and V.name == "up" and V.device == torch.device("cpu")
    # (what object's own reduction, which earlier files were written with, restores)
    old = sp.Mx4.__new__(sp.Mx4)
    old.__setstate__((None, dict(_codes=W.codes, _scales=W.scales, _shape=(3, 33), dtype=W.dtype, device=torch.device("cuda", 0))))
    assert old.device == torch.device("cpu") and old.shape == (3, 33)
