"""What the Python wrappers of the routed-field and distillation calls refuse
(no GPU): everything here is refused before the library is called."""
import pytest
import torch

import volume_rendering_amd as v
from volume_rendering_amd import _binding as B

I32 = torch.int32


def _calls(ws):
    """Each call with a workspace; every other tensor is as it has to be, but on the host."""
    z = torch.zeros
    yield lambda: v.nerf_route_plan(z(4, 2, dtype=I32), 3, z(4, dtype=I32), z(8, dtype=I32), z(4, 2, dtype=I32),
                                    workspace=ws)
    yield lambda: v.nerf_expert_linear_grad(z(8, 5), z(8, 7), z(3, 5, 7), z(4, dtype=I32), z(8, 7), z(3, 5, 7),
                                            workspace=ws)
    yield lambda: v.nerf_distill_topk(z(4, 9), z(4, 2), z(4, 2, dtype=I32), 1.0, z(4), workspace=ws)


@pytest.mark.parametrize("ws,why", [(torch.empty(4096, dtype=torch.uint8), "workspace: not a device tensor"),
                                    (torch.empty((64, 128), dtype=torch.uint8)[:, ::2], "workspace: .*contiguous"),
                                    (torch.empty((64, 64), dtype=torch.uint8).t()[1:], "workspace: .*contiguous")])
def test_workspaces_are_contiguous_device_tensors(ws, why):
    with pytest.raises(v.NerfError, match=why):
        B._ws(ws)
    for call in _calls(ws):
        with pytest.raises(v.NerfError):
            call()


def test_no_workspace_is_a_workspace():
    assert B._ws(None) == (0, 0)


def test_gradient_of_a_layer_needs_x_or_weight():
    z = torch.zeros
    with pytest.raises(v.NerfError, match="x and weight"):
        v.nerf_expert_linear_grad(z(8, 5), None, None, z(4, dtype=I32), z(8, 7))
    # one of them is enough to name the shapes: what is refused next is the host tensor
    with pytest.raises(v.NerfError, match="dz: not a device tensor"):
        v.nerf_expert_linear_grad(z(8, 5), None, z(3, 5, 7), z(4, dtype=I32), z(8, 7))
    with pytest.raises(v.NerfError, match="dz: not a device tensor"):
        v.nerf_expert_linear_grad(z(8, 5), z(8, 7), None, z(4, dtype=I32), None, z(3, 5, 7))
    with pytest.raises(v.NerfError, match="weight: 2 dimensions"):
        v.nerf_expert_linear_grad(z(8, 5), None, z(5, 7), z(4, dtype=I32), z(8, 7))
    with pytest.raises(v.NerfError, match="x: "):
        v.nerf_expert_linear_grad(z(8, 5), z(8, 6), z(3, 5, 7), z(4, dtype=I32), z(8, 7))
