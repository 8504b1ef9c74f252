"""A device step number below 1: the host number is refused, the device one cannot be, and the
step then changes nothing (the formula would divide by 1 - beta^0 = 0)."""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from parity import dev

pytestmark = pytest.mark.gpu


def _state(bits, p_dtype, seed):
    gen = torch.Generator(device=dev()).manual_seed(seed)
    params = [torch.randn(n, generator=gen, device=dev()).to(p_dtype) for n in (700, 1, 4096)]
    grads = [torch.randn(p.shape, generator=gen, device=dev()) for p in params]
    copies = [p.bfloat16() for p in params] if p_dtype == torch.float32 else None
    return qn.adamw_state(params, grads, copies=copies, bits=bits)


def _tensors(st):
    return st.params + (st.copies or []) + [st.m, st.v] + ([st.m_scale, st.v_scale] if st.bits == 8 else [])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("device_lr", [False, True])
def test_steps_below_1_change_nothing(bits, p_dtype, device_lr):
    print(f"[adamw] device steps below 1, bits={bits}, p={p_dtype}, device rate {device_lr}", flush=True)
    lr = torch.tensor([1e-2], device=dev()) if device_lr else 1e-2
    st, ref = _state(bits, p_dtype, 1), _state(bits, p_dtype, 1)
    for t in (0, -1, -(2 ** 63), 1, 0, 2):
        step = torch.tensor([t], dtype=torch.int64, device=dev())
        qn.adamw_step(st, step, lr)
        if t >= 1:
            qn.adamw_step(ref, step, lr)
        torch.cuda.synchronize()
        for a, b in zip(_tensors(st), _tensors(ref)):
            assert torch.equal(a, b), t


def test_counter_raised_after_the_captured_step():
    """A counter that starts at zero and is raised behind the step: the first replay changes
    nothing, the following ones are steps 1, 2, .."""
    print("[adamw] counter raised after the step", flush=True)
    st, ref = _state(8, torch.float32, 2), _state(8, torch.float32, 2)
    t = torch.zeros(1, dtype=torch.int64, device=dev())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qn.adamw_step(st, t, 1e-2)
        t += 1
    for k in range(4):
        (torch.randn(64, 64, device=dev()) @ torch.randn(64, 64, device=dev())).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        if k >= 1:
            qn.adamw_step(ref, torch.tensor([k], device=dev()), 1e-2)
        for a, b in zip(_tensors(st), _tensors(ref)):
            assert torch.equal(a, b), k
        assert torch.isfinite(st.params[0]).all()
