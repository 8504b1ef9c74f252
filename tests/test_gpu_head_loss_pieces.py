"""The loss alone over several pieces of the vocabulary (65536 rows a piece, where the gradient's have
32768), NF4 heads without a second level in several, and rows that grow from piece to piece. Bounds as
in test_gpu_head_loss."""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from parity import dev
from test_gpu_head_loss import check, make

pytestmark = pytest.mark.gpu


# one row past a piece, two and three pieces; tiles of 64 and of 256; all second levels
@pytest.mark.parametrize("V,m,head", [(65537, 17, "bf16"), (65537, 300, "bf16"), (131100, 70, "bf16"), (131100, 300, "bf16"),
                                      (65600, 17, "none"), (65600, 300, "none"), (131136, 130, "fp8"), (65600, 40, "int8")])
def test_loss_alone_over_pieces(V, m, head):
    print("[head loss] alone", V, m, head, flush=True)
    own, full, X, t, scale = make(V, 64, m, 0.2, head)
    # targets on both sides of the pieces' ends
    live = ((t >= 0) & (t < V)).nonzero()[:, 0]
    ends = torch.tensor([0, 32767, 32768, V // 2, 65535, V - 1], device=dev())
    t[live[:6]] = ends[:live.numel()]
    alone = qn.head_loss(own, X, t)
    check(full, X, t, scale, alone, None)
    assert torch.equal(qn.head_loss(own, X, t), alone)


@pytest.mark.parametrize("V,m,head", [(33024, 20, "none"), (65600, 300, "none"), (131136, 70, "none"), (65600, 130, "fp8")])
def test_gradient_of_an_nf4_head_over_pieces(V, m, head):
    print("[head loss] gradient", V, m, head, flush=True)
    own, full, X, t, scale = make(V, 128, m, 0.2, head)
    loss, dX = qn.head_loss_grad(own, X, t, scale=scale)
    check(full, X, t, scale, loss, dX)
    check(full, X, t, scale, qn.head_loss(own, X, t), None)


@pytest.mark.parametrize("m", [60, 270])
def test_later_pieces_far_above_the_earlier_ones(m):
    """Logits that leave float32's range of exponentials in the loss's second piece, and still larger
    ones in its third, which bring the row to a new scale twice."""
    V, d = 131100, 64
    own, full, X, t, scale = make(V, d, m)
    own[70000:70003] = (X[:3].float() * 8).bfloat16()
    own[70010] = (X[50].float() * 4).bfloat16()
    own[V - 2] = (X[50].float() * 16).bfloat16()
    own[V - 1] = (X[1].float() * 24).bfloat16()
    t[:3], t[50] = torch.tensor([5, 65535, 65536], device=dev()), 3
    check(own.double(), X, t, scale, qn.head_loss(own, X, t), None)
    loss, dX = qn.head_loss_grad(own, X, t, scale=scale)
    check(own.double(), X, t, scale, loss, dX)
