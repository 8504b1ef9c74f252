"""The gated block's forward on batches so long that G and U together would pass 4 GiB: it is taken
where they are not kept. Bounds as in test_gpu_gated."""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from parity import dev
from test_gpu_gated import check_forward, make

pytestmark = pytest.mark.gpu


def test_forward_whose_gate_and_up_would_pass_4_gib():
    f, d, m = 16384, 64, 70001
    layer, normal = make(f, d, 16, "silu")
    X = normal(m, d).bfloat16()
    H = qn.gated_fwd(layer, X)
    rows = torch.tensor([0, 1, 255, 256, 32767, 32768, 65535, 65536, m - 2, m - 1], device=dev())
    check_forward(layer, X[rows], H[rows], None)
    with pytest.raises(qn.QLoRAError, match="4 GiB"):
        qn.gated_fwd(layer, X, save=True)
