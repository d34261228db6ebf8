"""One linear-attention block, as a model would run it: a training step and a served request.

    x, n   = residual norm of the stream and the previous block's output
    q, k, v, gate, a = slices of one projection of n          (not copied apart)
    decay  = -exp(A_log) softplus(a + dt_bias)                (gate_decay)
    o, h   = linear attention with a decay per head           (chunked; token by token when serving)
    y      = norm of o per head, times silu(gate)             (gated norm)
    x', n' = residual norm of x and y's output projection

Projections are library matrix products; everything between them is this framework's kernels.
``python examples/linear_block.py`` checks that served tokens equal the prefill's and times both.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import delta_rule_linear_gb300 as kda  # noqa: E402

SCALE = 0.5      # residual scale


def make_params(D=512, H=4, m=1, dk=64, dv=64, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    HV = H * m
    # q, k, v, gate, a; a is padded so that a token's row is a multiple of 16 bytes, which views need
    widths = (H * dk, H * dk, HV * dv, HV * dv, -(-HV // 8) * 8)
    rn = lambda *s, std=1.0: std * torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return dict(H=H, HV=HV, dk=dk, dv=dv, widths=widths,
                w_in=1 + 0.1 * rn(D), w_gate=1 + 0.1 * rn(dv), w_out=1 + 0.1 * rn(D),
                A_log=0.1 * rn(HV), dt_bias=-3 + 0.1 * rn(HV),
                W=rn(D, sum(widths), std=D ** -0.5).to(dtype), Wo=rn(HV * dv, D, std=(HV * dv) ** -0.5).to(dtype))


def _project(p, n):
    """q, k, v, gate as strided head views of the projection, and the decay's raw gate in fp32."""
    q, k, v, gate, a = (n @ p["W"]).split(p["widths"], -1)
    return (q.unflatten(-1, (p["H"], -1)), k.unflatten(-1, (p["H"], -1)), v.unflatten(-1, (p["HV"], -1)),
            gate.unflatten(-1, (p["HV"], -1)), a[..., :p["HV"]].float().contiguous())


def forward(p, x, y, state=None):
    """x [B,T,D] fp32 stream, y [B,T,D] the previous block's output.  Returns (x', n', memory, saved)."""
    x1, n1 = kda.residual_norm_fwd(x, y, p["w_in"], scale=SCALE)
    q, k, v, gate, a = _project(p, n1)
    decay = kda.gate_decay(a, p["A_log"], p["dt_bias"])
    o, h = kda.linear_chunk_fwd(q, k, v, decay, state)
    u = kda.gated_norm_fwd(o, gate, p["w_gate"])
    z = u.flatten(-2) @ p["Wo"]
    x2, n2 = kda.residual_norm_fwd(x1, z, p["w_out"], scale=SCALE)
    return x2, n2, h, (x1, n1, q, k, v, gate, a, decay, state, o, u, x2)


def backward(p, saved, dn2, dx2=None, dh=None):
    """Gradients of the parameters and inputs, given those of n' (and of x' and the memory)."""
    x1, n1, q, k, v, gate, a, decay, state, o, u, x2 = saved
    g2 = kda.residual_norm_bwd(dn2, dx2, x2, p["w_out"], scale=SCALE)
    dz = g2["dy"]
    du = (dz @ p["Wo"].T).unflatten(-1, (p["HV"], -1))
    gg = kda.gated_norm_bwd(du, o, gate, p["w_gate"])
    ga = kda.linear_chunk_bwd(q, k, v, decay, state, gg["dx"], dh)
    t = a + p["dt_bias"]
    da = ga["ddecay"] * -p["A_log"].exp() * torch.sigmoid(t)
    dp = torch.cat([ga["dq"].flatten(-2), ga["dk"].flatten(-2), ga["dv"].flatten(-2), gg["dgate"].flatten(-2),
                    torch.nn.functional.pad(da.to(q.dtype), (0, p["widths"][-1] - p["HV"]))], -1)
    g1 = kda.residual_norm_bwd(dp @ p["W"].T, g2["dx"], x1, p["w_in"], scale=SCALE)
    return dict(x=g1["dx"], y=g1["dy"], w_in=g1["dw"], w_gate=gg["dw"], w_out=g2["dw"],
                A_log=(ga["ddecay"] * decay).sum((0, 1)), dt_bias=da.sum((0, 1)),
                W=n1.flatten(0, 1).T @ dp.flatten(0, 1), Wo=u.flatten(2).flatten(0, 1).T @ dz.flatten(0, 1),
                **({"state": ga["dh0"]} if state is not None else {}))


def step(p, x, y, state):
    """One token for every request: x [B,D] fp32, y [B,D]; the memory is updated in place."""
    x1, n1 = kda.residual_norm_fwd(x, y, p["w_in"], scale=SCALE)
    q, k, v, gate, a = _project(p, n1)
    o = kda.linear_decode_step(q, k, v, kda.gate_decay(a, p["A_log"], p["dt_bias"]), state)
    u = kda.gated_norm_fwd(o, gate, p["w_gate"])
    return kda.residual_norm_fwd(x1, u.flatten(-2) @ p["Wo"], p["w_out"], scale=SCALE)


def serve(p, x, y, prompt):
    """Prefills `prompt` tokens and serves the others one at a time; returns all tokens' n' and the memory."""
    _, n, h, _ = forward(p, x[:, :prompt].contiguous(), y[:, :prompt].contiguous())
    out = [n]
    for t in range(prompt, x.shape[1]):
        out.append(step(p, x[:, t].contiguous(), y[:, t].contiguous(), h)[1][:, None])
    return torch.cat(out, 1), h


def main():
    B, T, D, prompt = 4, 1024, 2048, 1000
    p = make_params(D, H=16, dk=128, dv=128)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((B, T, D), generator=g, device="cuda")
    y = torch.randn((B, T, D), generator=g, device="cuda").bfloat16()
    _, n, h, saved = forward(p, x, y)
    got, hs = serve(p, x, y, prompt)
    rel = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())  # noqa: E731
    print(f"served tokens against the prefill's: {rel(got[:, prompt:], n[:, prompt:]):.1e}, memory {rel(hs, h):.1e}")
    dn = torch.randn(n.shape, generator=g, device="cuda").bfloat16()
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    for i in range(4):
        if i == 3:
            ev[0].record()
        _, _, _, saved = forward(p, x, y)
        backward(p, saved, dn)
    ev[1].record()
    xs, ys = x[:, 0].contiguous(), y[:, 0].contiguous()
    for _ in range(100):
        step(p, xs, ys, hs)
    ev[2].record()
    torch.cuda.synchronize()
    print(f"training step {ev[0].elapsed_time(ev[1]):.3f} ms ({B} x {T} tokens); served step "
          f"{ev[1].elapsed_time(ev[2]) / 100:.3f} ms ({B} requests)")


if __name__ == "__main__":
    main()
