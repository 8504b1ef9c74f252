"""The gated block's forward on both sides of its choice between tiles of 64 and of 256: small tiles up to
two rounds of the chip (1024) and up to 96 large ones. Bounds as in test_gpu_gated."""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from test_gpu_gated import check_forward, make

pytestmark = pytest.mark.gpu


# 688 small tiles, 1032 and 1376; 1024 and 1088; 96 and 98 large ones
@pytest.mark.parametrize("d_ff,d_in,m", [(11008, 128, 128), (11008, 128, 129), (11008, 128, 256), (2048, 192, 1024),
                                         (2048, 192, 1025), (12288, 64, 70), (12544, 64, 70)])
def test_forward(d_ff, d_in, m):
    print("[gated] tile rule", d_ff, d_in, m, flush=True)
    layer, normal = make(d_ff, d_in, 16, "gelu")
    X = normal(m, d_in).bfloat16()
    H, GU = qn.gated_fwd(layer, X, save=True)
    check_forward(layer, X, H, GU)
    assert torch.equal(qn.gated_fwd(layer, X), H)
