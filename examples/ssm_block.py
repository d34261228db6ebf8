"""One state space block, as a model would run it: a training step, and a served request with beam search.

    x, n      = residual norm of the stream and the previous block's output
    u, z      = slices of one projection of n                      (not copied apart)
    c, window = short convolution of u over tokens, silu
    r, B, C   = slices of one projection of c;  dt = r W_dt
    y, h      = state space scan of c with time steps dt, gated by z     (chunked; token by token when serving)
    x', n'    = residual norm of x and y's output projection

Projections are library matrix products; everything between them is this framework's kernels.  When serving, beam_select
takes the best continuations of a request's beams and beam_reorder moves their windows and memories along.
``python examples/ssm_block.py`` checks that served tokens equal the prefill's and times both.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import delta_rule_linear_gb300 as kda  # noqa: E402

K = 4            # taps of the convolution


def make_params(D=512, Di=1024, N=16, rank=32, V=1000, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s, std=1.0: std * torch.randn(s, generator=g, device="cuda")  # noqa: E731
    step = torch.exp(-6.9 + 4.6 * torch.rand(Di, generator=g, device="cuda"))        # 1e-3 to 0.1
    return dict(D=D, Di=Di, N=N, rank=rank,
                w_in=1 + 0.1 * rn(D), w_out=1 + 0.1 * rn(D), conv_w=rn(Di, K, std=K ** -0.5), conv_b=0.1 * rn(Di),
                A_log=torch.log(torch.arange(1, N + 1, device="cuda").float()).expand(Di, N).contiguous() + 0.1 * rn(Di, N),
                skip=1 + 0.1 * rn(Di), dt_bias=step + torch.log(-torch.expm1(-step)),
                W=rn(D, 2 * Di, std=D ** -0.5).to(dtype), Wx=rn(Di, rank + 2 * N, std=Di ** -0.5).to(dtype),
                Wdt=rn(rank, Di, std=0.5 * rank ** -0.5).to(dtype), Wo=rn(Di, D, std=Di ** -0.5).to(dtype),
                embed=rn(V, D, std=2 * D ** -0.5).to(dtype))


def _sizes(p):
    return [p["rank"], p["N"], p["N"]]


def forward(p, x, y, window=None, state=None):
    """x [B,T,D] fp32 stream, y [B,T,D] the previous block's output.  Returns (x', n', window, memory, saved)."""
    x1, n1 = kda.residual_norm_fwd(x, y, p["w_in"])
    u, z = (n1 @ p["W"]).chunk(2, -1)
    c, win = kda.conv_fwd(u, p["conv_w"], p["conv_b"], window)
    r, B, C = (c @ p["Wx"]).split(_sizes(p), -1)
    dt = r @ p["Wdt"]
    v, h = kda.ssm_chunk_fwd(c, dt, -p["A_log"].exp(), B, C, state, skip=p["skip"], gate=z, dt_bias=p["dt_bias"])
    x2, n2 = kda.residual_norm_fwd(x1, v @ p["Wo"], p["w_out"])
    return x2, n2, win, h, (x1, n1, u, z, c, r, B, C, dt, v, window, state, x2)


def backward(p, saved, dn2, dx2=None, dwin=None, dh=None):
    """Gradients of the parameters and inputs, given those of n' (and of x', the window and the memory)."""
    x1, n1, u, z, c, r, B, C, dt, v, window, state, x2 = saved
    flat = lambda t: t.flatten(0, 1)  # noqa: E731
    g2 = kda.residual_norm_bwd(dn2, dx2, x2, p["w_out"])
    dv = g2["dy"] @ p["Wo"].T
    A = -p["A_log"].exp()
    gs = kda.ssm_chunk_bwd(dv, c, dt, A, B, C, state, dh, skip=p["skip"], gate=z, dt_bias=p["dt_bias"])
    dr = gs["ddt"] @ p["Wdt"].T
    dproj = torch.cat([dr, gs["dB"], gs["dC"]], -1)
    gc = kda.conv_bwd(gs["dx"] + dproj @ p["Wx"].T, u, p["conv_w"], p["conv_b"], window, dwin)
    dp = torch.cat([gc["dx"], gs["dgate"]], -1)
    g1 = kda.residual_norm_bwd(dp @ p["W"].T, g2["dx"], x1, p["w_in"])
    return dict(x=g1["dx"], y=g1["dy"], w_in=g1["dw"], w_out=g2["dw"], conv_w=gc["dw"], conv_b=gc["dbias"], A_log=gs["dA"] * A,
                skip=gs["dskip"], dt_bias=gs["ddt_bias"], W=flat(n1).T @ flat(dp), Wx=flat(c).T @ flat(dproj),
                Wdt=flat(r).T @ flat(gs["ddt"]), Wo=flat(v).T @ flat(g2["dy"]),
                **({"window": gc["dstate"]} if window is not None else {}), **({"state": gs["dh0"]} if state is not None else {}))


def step(p, x, y, window, state):
    """One token for every request (or beam): x [B,D] fp32, y [B,D]; window and memory are updated in place."""
    x1, n1 = kda.residual_norm_fwd(x, y, p["w_in"])
    u, z = (n1 @ p["W"]).chunk(2, -1)
    c = kda.conv_decode_step(u, p["conv_w"], window, p["conv_b"])
    r, B, C = (c @ p["Wx"]).split(_sizes(p), -1)
    v = kda.ssm_decode_step(c, r @ p["Wdt"], -p["A_log"].exp(), B, C, state, skip=p["skip"], gate=z, dt_bias=p["dt_bias"])
    return kda.residual_norm_fwd(x1, v @ p["Wo"], p["w_out"])


def serve(p, x, y, prompt):
    """Prefills `prompt` tokens and serves the others one at a time; all tokens' n', the window and the memory."""
    _, n, win, h, _ = forward(p, x[:, :prompt].contiguous(), y[:, :prompt].contiguous())
    out = [n]
    for t in range(prompt, x.shape[1]):
        out.append(step(p, x[:, t].contiguous(), y[:, t].contiguous(), win, h)[1][:, None])
    return torch.cat(out, 1), win, h


def tokens_in(p, tokens):
    """The stream and a first block output (zeros) of tokens [...]."""
    e = p["embed"][tokens]
    return e.float(), torch.zeros_like(e)


def search(p, prompt, W, new, eos):
    """Beam search: prompt [B,T] tokens, W beams, up to `new` tokens.  Returns (tokens [B,W,new], scores [B,W])."""
    B = prompt.shape[0]
    _, n, win, h, _ = forward(p, *tokens_in(p, prompt))
    win, h = win.repeat_interleave(W, 0), h.repeat_interleave(W, 0)      # every beam its own
    logits = (n[:, -1:] @ p["embed"].T).expand(B, W, -1).contiguous()
    scores = torch.full((B, W), -float("inf"), device="cuda")
    scores[:, 0] = 0.0                                                    # the beams are still the same: one counts
    finished = torch.zeros((B, W), dtype=torch.bool, device="cuda")
    seqs = torch.zeros((B, W, new), dtype=torch.int32, device="cuda")
    for t in range(new):
        scores, parents, tokens = kda.beam_select(logits, scores, finished=finished, eos=eos)
        seqs[:, :, t] = tokens if t == 0 else 0
        if t:
            kda.beam_reorder([win, h, seqs, finished], parents)
            seqs[:, :, t] = tokens
        finished |= tokens == eos
        x, y = tokens_in(p, tokens.flatten())
        _, n = step(p, x, y, win, h)
        logits = (n @ p["embed"].T).unflatten(0, (B, W))
    return seqs, scores


def main():
    B, T, D, prompt = 4, 1024, 2048, 1000
    p = make_params(D, Di=2 * D, rank=D // 16, V=32000)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((B, T, D), generator=g, device="cuda")
    y = torch.randn((B, T, D), generator=g, device="cuda").bfloat16()
    _, n, win, h, saved = forward(p, x, y)
    got, ws, hs = serve(p, x, y, prompt)
    rel = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())  # noqa: E731
    print(f"served tokens against the prefill's: {rel(got[:, prompt:], n[:, prompt:]):.1e}, memory {rel(hs, h):.1e}")
    dn = torch.randn(n.shape, generator=g, device="cuda").bfloat16()
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    for i in range(4):
        if i == 3:
            ev[0].record()
        saved = forward(p, x, y)[-1]
        backward(p, saved, dn)
    ev[1].record()
    xs, ys = x[:, 0].contiguous(), y[:, 0].contiguous()
    for _ in range(100):
        step(p, xs, ys, ws, hs)
    ev[2].record()
    tokens = torch.randint(0, 32000, (B, 200), generator=g, device="cuda")
    seqs, scores = search(p, tokens, 4, 20, eos=2)
    ev[3].record()
    torch.cuda.synchronize()
    print(f"training step {ev[0].elapsed_time(ev[1]):.3f} ms ({B} x {T} tokens); served step "
          f"{ev[1].elapsed_time(ev[2]) / 100:.3f} ms ({B} requests); 20 tokens of 4 beams {ev[2].elapsed_time(ev[3]):.1f} ms, "
          f"best score {float(scores[0, 0]):.2f}")


if __name__ == "__main__":
    main()
