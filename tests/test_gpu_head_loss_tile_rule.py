"""The loss on both sides of its choice between tiles of 64 and of 256: up to 64 tokens, and up to 128 where
the small tiles are at most two rounds of the chip (1024) in a piece. Bounds as in test_gpu_head_loss."""
import pytest

import bit_nf4_quantized_05_amd as qn
from test_gpu_head_loss import check, make

pytestmark = pytest.mark.gpu


# a piece of the loss and of the gradient: 1024 and 1026 small tiles, 2048 and over, one row of them
@pytest.mark.parametrize("V,m,head", [(32768, 65, "bf16"), (32769, 65, "bf16"), (65536, 64, "bf16"), (65536, 65, "bf16"),
                                      (65600, 128, "int8"), (32832, 128, "int8"), (16384, 256, "bf16"), (16385, 256, "bf16")])
def test_loss_and_gradient(V, m, head):
    print("[head loss] tile rule", V, m, head, flush=True)
    own, full, X, t, scale = make(V, 128, m, 0.2, head)
    loss, dX = qn.head_loss_grad(own, X, t, scale=scale)
    check(full, X, t, scale, loss, dX)
    check(full, X, t, scale, qn.head_loss(own, X, t), None)
