"""clip_grads' outputs as autograd sees them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_saved_output_that_was_written_is_noticed(flat, in_place):
    def tensors():
        whole = torch.ones(300, device=DEV)
        return list(whole.split([100, 150, 50])) if flat else [x.clone() for x in whole.split([100, 150, 50])]

    grads = tensors()
    outs = grads if in_place else tensors()
    s = sp.GradSet(grads, out=None if in_place else outs)
    w = torch.ones(150, device=DEV, requires_grad=True)
    loss = (outs[1] * w).sum()  # saves outs[1]
    versions = [g._version for g in grads]
    norm = sp.grad_norm(s)  # writes nothing
    assert [g._version for g in grads] == versions
    assert torch.equal(sp.clip_grads(s, 1.0), norm)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    if not in_place:  # the gradients were only read
        loss = (grads[1] * w).sum()
        sp.clip_grads(s, 1.0)
        loss.backward()
        assert torch.equal(w.grad, grads[1])


def test_inference_tensors_and_empty_sets():
    with torch.inference_mode():
        whole = torch.full((300,), 2.0, device=DEV)
        parts = list(whole.split(100))
    sp.clip_grads(parts, 1.0)
    assert abs(float(torch.linalg.vector_norm(whole)) - 1.0) < 1e-5
    assert float(sp.clip_grads([], 1.0)) == 0.0
