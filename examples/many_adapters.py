"""Several LoRA adapters trained on one frozen NF4 layer, then served side by side.

    python examples/many_adapters.py

Each user's adapter is fitted to a target of its own on batches that mix the users' tokens
(multi_plan, multi_linear_fwd, multi_linear_bwd, adamw_step with 8-bit moments), and the
trained pool then answers a decode batch of one token per user, captured in a graph.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import bit_nf4_quantized_05_amd as qn  # noqa: E402


def train(d_out=512, d_in=512, users=5, rank=16, tokens=400, steps=60, seed=0, log=print):
    """(layer, pool, first loss, last loss) after `steps` AdamW steps over all users' adapters."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    layer = qn.quantize(rand(d_out, d_in) * 0.02)
    W = qn.double_dequant(layer).float()

    # what each user wants: the frozen layer plus a change of rank 4 of their own
    change = [rand(d_out, 4) @ rand(4, d_in) * 0.01 for _ in range(users)]

    pool = qn.alloc_pool(users, rank, d_out, d_in, dev)
    for u in range(users):
        pool.set(u, rand(rank, d_in) * d_in ** -0.5, torch.zeros(d_out, rank, device=dev), 2.0)
    masters = [pool.A.float(), pool.B.float()]                       # float32 parameters; the pool is their copy
    grads = [torch.empty_like(m) for m in masters]
    opt = qn.adamw_state(masters, grads, copies=[pool.A, pool.B], bits=8)

    # the batch: requests of different lengths, packed; user -1 is a request without an adapter
    bounds = torch.linspace(0, tokens, users + 2).long().tolist()
    ids = torch.full((tokens,), -1, dtype=torch.int32, device=dev)
    for u in range(users):
        ids[bounds[u]:bounds[u + 1]] = u
    plan = qn.multi_plan(ids, users)
    ws = torch.empty(max(qn.multi_linear_fwd_workspace_bytes(d_out, d_in, tokens, pool.r, users),
                         qn.multi_linear_bwd_workspace_bytes(d_out, d_in, tokens, pool.r, users)),
                     dtype=torch.uint8, device=dev)
    clip = torch.empty(1, device=dev)
    first = last = None
    for step in range(1, steps + 1):
        X = rand(tokens, d_in).bfloat16()
        want = X.float() @ W.T
        for u in range(users):
            rows = slice(bounds[u], bounds[u + 1])
            want[rows] += X[rows].float() @ change[u].T
        Y = qn.multi_linear_fwd(layer, pool, plan, X, workspace=ws)
        err = Y.float() - want
        err[bounds[users]:] = 0                                      # nothing to learn without an adapter
        last = err.square().mean().item()
        first = last if first is None else first
        dY = (err * (2.0 / d_out)).bfloat16()
        qn.multi_linear_bwd(layer, pool, plan, X, dY, dA=grads[0], dB=grads[1], workspace=ws)
        norm = torch.stack([g.norm() for g in grads]).norm()
        torch.clamp(10.0 / (norm + 1e-6), max=1.0, out=clip[0])
        qn.adamw_step(opt, step, 5e-3, grad_scale=clip)
        if step == 1 or step % 20 == 0:
            log(f"step {step:3d}  loss {last:.5f}")
    return layer, pool, first, last


def serve(layer, pool, calls=4, log=print):
    """One token per user and call from a captured graph; the largest difference to each
    user's adapter applied alone."""
    dev, users = pool.device, pool.n
    X = torch.zeros(users, layer.d_in, dtype=torch.bfloat16, device=dev)
    ids = torch.zeros(users, dtype=torch.int32, device=dev)
    Y = torch.empty(users, layer.d_out, dtype=torch.bfloat16, device=dev)
    ws = torch.empty(qn.multi_linear_fwd_workspace_bytes(layer.d_out, layer.d_in, users, pool.r, users),
                     dtype=torch.uint8, device=dev)
    plan = qn.multi_plan(ids, users)

    def call():
        qn.multi_plan(ids, users, out=plan)
        qn.multi_linear_fwd(layer, pool, plan, X, out=Y, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    worst = 0.0
    for _ in range(calls):
        who = torch.randperm(users, device=dev).int()
        ids.copy_(who)
        X.copy_(torch.randn(users, layer.d_in, device=dev))
        graph.replay()
        for t, u in enumerate(who.tolist()):
            alone = qn.linear_fwd(layer, pool.A[u], pool.B[u], pool.s[u].item(), X[t:t + 1])
            worst = max(worst, ((Y[t] - alone[0]).float().norm() / alone.float().norm()).item())
    log(f"served {calls} batches of {users} users; largest difference to the adapters alone {worst:.4f}")
    return worst


if __name__ == "__main__":
    layer, pool, first, last = train()
    serve(layer, pool)
