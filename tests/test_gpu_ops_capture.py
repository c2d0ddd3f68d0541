"""Scratch that a captured call keeps: a graph may replay beside later calls."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsq():
    import block_scaled_precision_03_gb300 as b
    b.lib()
    return b


@pytest.mark.parametrize("given", [False, True])
def test_a_captured_clip_has_scratch_of_its_own(bsq, given):
    # the stream that captures is the current one, or is passed while another one is current
    grad, out, norm = torch.full((1000,), 3.0, device="cuda"), torch.empty(1000, device="cuda"), torch.empty(1, device="cuda")
    grads = bsq.GradList([grad], [out])
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(other if given else side):
            stream = side if given else None
            held = grads.workspace(stream)
            again = grads.workspace(stream)
            bsq.clip_grad_norm_into(grads, 1.0, norm, stream=stream)
    later = grads.workspace(side)
    assert len({held.data_ptr(), again.data_ptr(), later.data_ptr()}) == 3
    assert grads.workspace(side).data_ptr() == later.data_ptr()
    graph.replay()
    torch.cuda.synchronize()
    assert abs(float(norm) - 3.0 * 1000 ** 0.5) < 1e-4 and abs(float(out[0]) - 1000 ** -0.5) < 1e-6
