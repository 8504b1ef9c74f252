"""The gated block's and the head loss's calls stay inside a workspace of exactly their query's size, and
their results do not depend on what it held: the bytes after it keep their pattern, and a workspace of
ones gives the bits of one of zeros."""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from parity import dev
from test_gpu_gated import make as make_layer
from test_gpu_head_loss import make as make_head

pytestmark = pytest.mark.gpu

GUARD = 1 << 16


def guarded(need, call):
    """call's tensors with a workspace of `need` bytes out of a larger buffer."""
    got = []
    for fill in (0, 0xFF):
        buf = torch.full((need + GUARD,), 0xA5, dtype=torch.uint8, device=dev())
        buf[:need].fill_(fill)
        got.append([t.clone() for t in call(buf[:need])])
        torch.cuda.synchronize()
        assert (buf[need:] == 0xA5).all()
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d_ff,d_in,m,r", [(64, 64, 1, 0), (704, 1088, 1, 16), (192, 4160, 3, 9), (320, 2112, 17, 33), (128, 320, 40, 256),
                                           (704, 1024, 64, 17), (704, 1024, 65, 17), (2112, 512, 300, 64), (6400, 320, 300, 33),
                                           (64, 4160, 1025, 256), (4160, 192, 130, 1), (1024, 64, 4000, 40)])
def test_gated(d_ff, d_in, m, r):
    print("[gated] workspace", d_ff, d_in, m, r, flush=True)
    layer, normal = make_layer(d_ff, d_in, r, "silu")
    X, dH = normal(m, d_in).bfloat16(), normal(m, d_ff).bfloat16()
    _, GU = qn.gated_fwd(layer, X, save=True)
    guarded(qn.gated_fwd_workspace_bytes(d_ff, d_in, m, r), lambda ws: qn.gated_fwd(layer, X, save=True, workspace=ws))
    guarded(qn.gated_bwd_workspace_bytes(d_ff, d_in, m, r), lambda ws: qn.gated_bwd(layer, GU, dH, workspace=ws))


@pytest.mark.parametrize("V,d,m,head,ldw", [(1, 64, 1, "bf16", 0), (1001, 256, 203, "bf16", 0), (1001, 256, 203, "bf16", 300 * 8),
                                            (33000, 128, 65, "bf16", 0), (66001, 64, 300, "bf16", 40000), (66001, 64, 17, "bf16", 70000),
                                            (4160, 320, 300, "int8", 0), (33024, 128, 128, "none", 0), (512, 64, 9001, "bf16", 0)])
def test_head_loss(V, d, m, head, ldw):
    print("[head loss] workspace", V, d, m, head, ldw, flush=True)
    own, _, X, t, scale = make_head(V, d, m, 0.3, head)
    if ldw:
        wide = torch.empty(V, ldw, dtype=torch.bfloat16, device=dev())
        view = wide[:, 8:8 + d]
        view.copy_(own)
        own = view
    guarded(qn.head_loss_workspace_bytes(own, m), lambda ws: [qn.head_loss(own, X, t, workspace=ws)])
    guarded(qn.head_loss_workspace_bytes(own, m, grad=True), lambda ws: qn.head_loss_grad(own, X, t, scale=scale, workspace=ws))
