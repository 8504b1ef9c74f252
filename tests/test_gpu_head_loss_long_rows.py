"""The loss over heads whose rows are so long, or so far apart, that pieces of the usual number of rows
would reach 4 GiB. Bounds as in test_gpu_head_loss; the workspace is what the size query asks for."""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from parity import dev
from test_gpu_head_loss import check, make

pytestmark = pytest.mark.gpu


def calls(own, X, t, scale):
    """(loss alone, loss, dX), each call with a workspace of its own query's size."""
    one, both = (torch.empty(qn.head_loss_workspace_bytes(own, X.shape[0], grad=g), dtype=torch.uint8, device=dev())
                 for g in (False, True))
    return (qn.head_loss(own, X, t, workspace=one), *qn.head_loss_grad(own, X, t, scale=scale, workspace=both))


@pytest.mark.parametrize("V,d,head", [(65600, 32768, "bf16"), (33024, 65536, "int8")])
def test_long_rows(V, d, head):
    own, full, X, t, scale = make(V, d, 17, 0.1, head)
    alone, loss, dX = calls(own, X, t, scale)
    check(full, X, t, scale, alone, None)
    check(full, X, t, scale, loss, dX)


@pytest.mark.parametrize("m", [17, 300])
def test_rows_far_apart(m):
    V, d = 66001, 64
    own, full, X, t, scale = make(V, d, m, 0.1)
    wide = torch.empty(V, 40000, dtype=torch.bfloat16, device=dev())
    view = wide[:, 19968:19968 + d]
    view.copy_(own)
    alone, loss, dX = calls(view, X, t, scale)
    check(full, X, t, scale, alone, None)
    check(full, X, t, scale, loss, dX)
