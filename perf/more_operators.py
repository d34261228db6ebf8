"""Cases, plain forms and 64-bit references of the short convolution, the state space scan and beam search.

A state space block keeps, beside the linear-attention layers of a model, one small memory per channel:

    short convolution   y_t = act(bias + sum_j w[:, j] x_{t-K+1+j})           (per channel, K taps back in time)
    state space scan    dt_t = softplus(dt_t + dt_bias),
                        h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,   y_t = (C_t . h_t + skip x_t) silu(gate_t)

with h_t a [D, N] memory, A [D, N] a decay per channel and state, B_t and C_t [G, N] shared by the channels of a group:
for prompts (equal lengths or packed), for single tokens, and as gradients.  Beam search over what such layers answer
takes the best of the W beams' continuations and moves the recurrent memories along:

    selection    total[w, v] = score_w + log softmax(logits_w)[v];  the k largest, ties to the lowest w V + v
    reordering   state[b, w] <- state[b, parent[b, w]], in place

`run` computes a case either by elementary torch operations in 32 bits (totals of the selection in 64, since candidates
may lie next to one another), or by the calls of delta_rule_linear_gb300 where `own` is true.
"""
import math
import random

import torch

own = False

# ------------------------------------------------------------------------------------ cases


def listed():
    return [
        # The convolution before a block's scan at the training shape; x is a slice of the block's input projection.
        dict(name="conv_train", op="conv", dtype="bf16", B=2, T=2048, C=4096, K=4, act="silu", bias=True, h0=False, fused=True),
        # Sixteen packed prompts of 256 to 4096 tokens that continue from kept windows.
        dict(name="conv_packed", op="conv_varlen", dtype="bf16", N=16, lo=256, hi=4096, lens=0, C=2048, K=4, act="silu",
             bias=False, h0=True, fused=False),
        # Its gradients at the training shape.
        dict(name="conv_grad", op="conv_bwd", dtype="bf16", B=2, T=2048, C=4096, K=4, act="silu", bias=True, h0=False, fused=True),
        # A short prompt of a small fp32 model: where the call itself is what counts.
        dict(name="ssm_short_fp32", op="ssm", dtype="f32", B=1, T=45, D=250, N=16, G=1, gate=True, h0=False),
        # The training-shape scan: two sequences, 4096 channels of 16 states, gated.
        dict(name="ssm_train", op="ssm", dtype="bf16", B=2, T=2048, D=4096, N=16, G=1, gate=True, h0=False),
        # One long prompt that continues from a carried memory.
        dict(name="ssm_long", op="ssm", dtype="bf16", B=1, T=32768, D=4096, N=16, G=1, gate=True, h0=True),
        # One token for each of 256 requests: bound by the memories.
        dict(name="ssm_step_256", op="ssm_step", dtype="bf16", B=256, D=4096, N=16, G=1, gate=True),
        # Gradients of the scan at the training shape.
        dict(name="ssm_grad", op="ssm_bwd", dtype="bf16", B=2, T=2048, D=4096, N=16, G=1, gate=True, h0=False),
        # One step of 64 requests with 8 beams over a large vocabulary.
        dict(name="select_64x8", op="select", dtype="bf16", B=64, W=8, V=131072, k=8, finished=True, first=False),
        # The same for three requests with 4 beams, an odd vocabulary and fp32 logits; twice the beams are asked for.
        dict(name="select_3x4", op="select", dtype="f32", B=3, W=4, V=50021, k=8, finished=False, first=False),
        # The memories of two linear-attention and two state space layers follow the beams: 32 requests of 4 beams.
        dict(name="reorder_32x4", op="reorder", dtype="bf16", B=32, W=4, layers=2, H=16, dk=128, D=4096, N=16, K=4),
        # The same for two requests of 5 beams and small layers: latency.
        dict(name="reorder_2x5", op="reorder", dtype="bf16", B=2, W=5, layers=4, H=2, dk=64, D=250, N=16, K=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_varlen", "conv_step", "conv_bwd", "ssm", "ssm", "ssm_varlen", "ssm_step", "ssm_bwd",
                     "ssm_bwd", "select", "select", "reorder"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("conv"):
        c = dict(op=op, dtype=dt, C=rng.choice([2048, 4096, _log_int(rng, 16, 8192)]), K=rng.choice([2, 3, 4, 4]),
                 act=rng.choice(["silu", "silu", "none"]), bias=rng.random() < 0.5, h0=rng.random() < 0.5)
        most = (1 << 26) // c["C"]
        if op == "conv_step":
            return dict(c, B=_log_int(rng, 1, 512), fused=rng.random() < 0.5)
        if op == "conv_varlen":
            hi = _log_int(rng, 8, 4096)
            return dict(c, N=max(1, min(_log_int(rng, 1, 64), most // hi)), lo=max(1, hi // 16), hi=hi,
                        lens=rng.randrange(1 << 16), fused=rng.random() < 0.5)
        B = _log_int(rng, 1, 8)
        return dict(c, B=B, T=_log_int(rng, 1, max(2, min(32768, most // B))), fused=rng.random() < 0.5)
    if op.startswith("ssm"):
        N = rng.choice([8, 16, 16, 16, 32, 64])
        D = rng.choice([2048, 4096, _log_int(rng, 16, 4096)])
        G = rng.choice([g for g in (1, 1, 1, 2, 3, 4, 8) if D % g == 0])
        c = dict(op=op, dtype=dt, D=D, N=N, G=G, gate=rng.random() < 0.7, h0=rng.random() < 0.5)
        if op == "ssm_step":
            return dict(c, B=_log_int(rng, 1, min(256, (1 << 24) // (D * N))))
        most = (1 << 28 if op == "ssm_bwd" else 1 << 30) // (D * N)       # tokens
        if op == "ssm_varlen":
            hi = _log_int(rng, 8, min(4096, most))
            return dict(c, N_seq=max(1, min(_log_int(rng, 1, 24), most // hi)), lo=max(1, hi // 16), hi=hi,
                        lens=rng.randrange(1 << 16))
        B = min(_log_int(rng, 1, 8), most)
        return dict(c, B=B, T=_log_int(rng, 1, max(2, min(32768 if op == "ssm" else 4096, most // B))))
    W = _log_int(rng, 1, 16)
    if op == "select":
        V = _log_int(rng, 500, 131072)
        return dict(op=op, dtype=dt, B=max(1, min(_log_int(rng, 1, 64), (1 << 26) // (W * V))), W=W, V=V,
                    k=rng.choice([W, W, min(2 * W, 32)]), finished=rng.random() < 0.5, first=rng.random() < 0.2)
    H, D = _log_int(rng, 1, 16), _log_int(rng, 16, 4096)
    return dict(op=op, dtype=dt, B=max(1, min(_log_int(rng, 1, 64), 256 // W)), W=W, layers=rng.randint(1, 4), H=H,
                dk=rng.choice([32, 64, 128]), D=D, N=rng.choice([8, 16, 32]), K=rng.choice([2, 3, 4]))


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _lens(c, n):
    r = random.Random(c["lens"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(n)]


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    op = c["op"]
    if op.startswith("conv"):
        C, K = c["C"], c["K"]
        w = C * K * 4 + (C * 4 if c["bias"] else 0)
        if op == "conv_step":
            n = c["B"] * C
            return {"bytes": 2 * n * e + 2 * n * (K - 1) * e + w, "flops": (2 * K + 5) * n}
        seqs = c["N"] if op == "conv_varlen" else c["B"]
        n = (sum(_lens(c, seqs)) if op == "conv_varlen" else seqs * c["T"]) * C
        st = seqs * (K - 1) * C * e
        if op == "conv_bwd":        # x, d_y (and both windows' gradients) in; dx, dw out
            return {"bytes": 3 * n * e + 2 * w + (3 if c["h0"] else 1) * st, "flops": (6 * K + 10) * n}
        return {"bytes": 2 * n * e + w + (2 if c["h0"] else 1) * st, "flops": (2 * K + 5) * n}
    if op.startswith("ssm"):
        D, N, G = c["D"], c["N"], c["G"]
        seqs = c["N_seq"] if op == "ssm_varlen" else c["B"]
        rows = sum(_lens(c, seqs)) if op == "ssm_varlen" else seqs * c.get("T", 1)
        x, bc, st, par = rows * D * e, rows * G * N * e, seqs * D * N * 4, D * N * 4 + 2 * D * 4
        cells = rows * D * N
        if op == "ssm_bwd":         # x, dt, (gate,) d_y, B, C, final memory's gradient in; the gradients out
            return {"bytes": (7 if c["gate"] else 5) * x + 4 * bc + (3 if c["h0"] else 1) * st + 2 * par, "flops": 20 * cells}
        if op == "ssm_step":
            return {"bytes": (4 if c["gate"] else 3) * x + 2 * bc + 2 * st + par, "flops": 6 * cells}
        return {"bytes": (4 if c["gate"] else 3) * x + 2 * bc + (2 if c["h0"] else 1) * st + par, "flops": 6 * cells}
    if op == "select":
        n = c["B"] * c["W"] * c["V"]
        return {"bytes": n * e + 4 * c["B"] * c["W"] + 12 * c["B"] * c["k"], "flops": 3 * n}
    W = c["W"]
    row = c["layers"] * (c["H"] * c["dk"] * c["dk"] * 4 + c["D"] * c["N"] * 4 + (c["K"] - 1) * c["D"] * e)
    # beams that take another's memory are written, the different ones they take it from are read (in the mean)
    moved, taken = W - 1, W * (1 - (1 - 1 / W) ** (W - 1)) if W > 1 else 0
    return {"bytes": int(c["B"] * row * (moved + taken)) + 4 * c["B"] * W + 1, "flops": 1}


# ------------------------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32)


def prepare(c, seed):
    g = _gen(seed)
    rn = lambda *s, dt=torch.float32: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    ru = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    dt, op = _dt(c["dtype"]), c["op"]
    s = dict(case=c)
    if op.startswith("conv"):
        C, K = c["C"], c["K"]
        if op == "conv_varlen":
            s["cu_host"] = _cu(_lens(c, c["N"]))
            s["cu"] = s["cu_host"].cuda()
            B, T, n = 1, int(s["cu_host"][-1]), c["N"]
        else:
            B, T, n = c["B"], c.get("T", 1), c["B"]
        pad = 2 * C if c["fused"] else C          # the convolution's input beside the block's gate
        s["x"] = rn(B, T, pad, dt=dt)[..., :C]
        s["w"] = rn(C, K) * K ** -0.5
        s["bias"] = 0.1 * rn(C) if c["bias"] else None
        if op == "conv_step":
            s["state"] = rn(n, K - 1, C, dt=dt)
            s["x"] = s["x"][:, 0]
        else:
            s["h0"] = rn(n, K - 1, C, dt=dt) if c["h0"] else None
        if op == "conv_bwd":
            s["d_y"], s["dhT"] = rn(B, T, C, dt=dt), rn(n, K - 1, C, dt=dt)
        return s
    if op.startswith("ssm"):
        D, N, G = c["D"], c["N"], c["G"]
        if op == "ssm_varlen":
            s["cu_host"] = _cu(_lens(c, c["N_seq"]))
            s["cu"] = s["cu_host"].cuda()
            B, T, n = 1, int(s["cu_host"][-1]), c["N_seq"]
        else:
            B, T, n = c["B"], c.get("T", 1), c["B"]
        # decays -1 .. -N, time steps of 1e-3 to 0.1 around which the input moves them
        s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * (0.1 * rn(D, N)).exp()
        step = torch.exp(math.log(1e-3) + math.log(100.0) * ru(D))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))          # softplus(dt_bias) = step
        s["x"], s["dt"] = rn(B, T, D, dt=dt), (0.5 * rn(B, T, D)).to(dt)
        s["B"], s["C"] = rn(B, T, G, N, dt=dt), rn(B, T, G, N, dt=dt)
        s["skip"] = 1.0 + 0.1 * rn(D)
        s["gate"] = rn(B, T, D, dt=dt) if c["gate"] else None
        if op == "ssm_step":
            for name in ("x", "dt", "B", "C", "gate"):
                s[name] = s[name][:, 0] if s[name] is not None else None
            s["state"] = rn(n, D, N)
        else:
            s["h0"] = 0.1 * rn(n, D, N) if c["h0"] else None
        if op == "ssm_bwd":
            s["d_y"], s["dhT"] = rn(B, T, D, dt=dt), 0.1 * rn(n, D, N)
        return s
    B, W = c["B"], c["W"]
    if op == "select":
        s["logits"] = (3.0 * rn(B, W, c["V"])).to(dt)
        s["scores"] = (-10.0 - 0.7 * rn(B, W).abs().cumsum(1)).contiguous()
        if c["first"]:                  # all beams of a request are still the same: only the first one counts
            s["scores"][:, 1:] = -math.inf
        s["finished"] = (ru(B, W) < 0.2) if c["finished"] else None
        return s
    s["states"] = []
    for _ in range(c["layers"]):
        s["states"] += [rn(B * W, c["H"], c["dk"], c["dk"]), rn(B * W, c["D"], c["N"]), rn(B * W, c["K"] - 1, c["D"], dt=dt)]
    s["parents"] = torch.randint(0, W, (B, W), generator=g, device="cuda", dtype=torch.int32)
    return s


EOS = 2

# ------------------------------------------------------------------------------------ plain forms


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _conv(x, w, bias, h0, act):
    """[B, T, C] in 32 bits with the window h0 [B, K-1, C] before it: (y, all rows with the window)."""
    T, K = x.shape[1], w.shape[1]
    rows = torch.cat([h0 if h0 is not None else x.new_zeros(x.shape[0], K - 1, x.shape[2]), x], 1)
    y = sum(w[:, j] * rows[:, j:j + T] for j in range(K))
    if bias is not None:
        y = y + bias
    return (_silu(y) if act == "silu" else y), rows


def _softplus(x):
    return x.clamp(min=0.0) + torch.log1p(torch.exp(-x.abs()))


def _scan(x, dt, A, Bm, Cm, h0):
    """The recurrence on 32-bit [B, T, D] (dt >= 0 after its softplus; 0 leaves the memory as it is): all chunks walked
    side by side from empty memories, the memories chained over the chunks, then what each chunk had before it."""
    B, T, D = x.shape
    G, N = Bm.shape[2:]
    L = max(1, math.isqrt(T))
    n = -(-T // L)
    pad = n * L - T

    def chunks(t):
        t = torch.cat([t, t.new_zeros(B, pad, *t.shape[2:])], 1) if pad else t
        return t.unflatten(1, (n, L))

    heads = lambda t: t.repeat_interleave(D // G, -2) if G > 1 else t  # noqa: E731
    x, dt, Bm, Cm = chunks(x), chunks(dt), chunks(Bm), chunks(Cm)
    h = x.new_zeros(B, n, D, N)
    y = []
    for j in range(L):
        h = torch.exp(dt[:, :, j, :, None] * A) * h + (dt[:, :, j] * x[:, :, j])[..., None] * heads(Bm[:, :, j])
        y.append((h * heads(Cm[:, :, j])).sum(-1))
    run = dt.cumsum(2)
    all_ = torch.exp(run[:, :, -1, :, None] * A)
    carry = [h0 if h0 is not None else x.new_zeros(B, D, N)]
    for i in range(n):
        carry.append(all_[:, i] * carry[-1] + h[:, i])
    before = torch.stack(carry[:-1], 1)
    y = [y[j] + (before * torch.exp(run[:, :, j, :, None] * A) * heads(Cm[:, :, j])).sum(-1) for j in range(L)]
    return torch.stack(y, 2).flatten(1, 2)[:, :T], carry[-1]


def _ssm(x, dt, A, Bm, Cm, skip, gate, bias, h0, ok=None):
    step = _softplus(dt + bias)
    if ok is not None:
        step = torch.where(ok[..., None], step, 0.0)
    y, h = _scan(x, step, A, Bm, Cm, h0)
    y = y + skip * x
    return (y * _silu(gate) if gate is not None else y), h


def _padded(cu):
    """Rows of packed sequences as [N, most], and which of them are there."""
    cu = cu.to(torch.int64)
    lens = cu[1:] - cu[:-1]
    most = int(lens.max())
    at = cu[:-1, None] + torch.arange(most)
    ok = torch.arange(most) < lens[:, None]
    return torch.where(ok, at, 0).cuda(), ok.cuda(), lens.cuda()


def _plain(s):
    c = s["case"]
    op = c["op"]
    f = lambda t: None if t is None else t.float()  # noqa: E731
    if op in ("conv", "conv_varlen"):
        dt, K = s["x"].dtype, c["K"]
        if op == "conv":
            y, rows = _conv(f(s["x"]), s["w"], s["bias"], f(s["h0"]), c["act"])
            return dict(y=y.to(dt), state=rows[:, rows.shape[1] - (K - 1):].to(dt))
        at, ok, lens = _padded(s["cu_host"])
        y, rows = _conv(f(s["x"])[0][at], s["w"], s["bias"], f(s["h0"]), c["act"])
        last = lens[:, None] + torch.arange(K - 1, device="cuda")
        return dict(y=y[ok][None].to(dt), state=rows.gather(1, last[..., None].expand(-1, -1, c["C"])).to(dt))
    if op == "conv_step":
        y, rows = _conv(f(s["x"])[:, None], s["w"], s["bias"], f(s["state"]), c["act"])
        s["state"].copy_(rows[:, 1:])
        return dict(y=y[:, 0].to(s["x"].dtype), state=s["state"])
    if op == "conv_bwd":
        dt, K = s["x"].dtype, c["K"]
        wrt = dict(dx=f(s["x"]).clone(), dw=s["w"].clone())
        if c["bias"]:
            wrt["dbias"] = s["bias"].clone()
        if c["h0"]:
            wrt["dstate"] = f(s["h0"]).clone()
        for t in wrt.values():
            t.requires_grad_(True)
        y, rows = _conv(wrt["dx"], wrt["dw"], wrt.get("dbias"), wrt.get("dstate"), c["act"])
        got = torch.autograd.grad([y, rows[:, rows.shape[1] - (K - 1):]], list(wrt.values()), [f(s["d_y"]), f(s["dhT"])])
        out = dict(zip(wrt, got))
        return {n: (t.to(dt) if n in ("dx", "dstate") else t) for n, t in out.items()}
    if op == "ssm":
        y, h = _ssm(*(f(s[n]) for n in ("x", "dt", "A", "B", "C", "skip", "gate", "dt_bias", "h0")))
        return dict(y=y.to(s["x"].dtype), h=h)
    if op == "ssm_varlen":
        at, ok, _ = _padded(s["cu_host"])
        tok = [None if s[n] is None else f(s[n])[0][at] for n in ("x", "dt", "B", "C", "gate")]
        y, h = _ssm(tok[0], tok[1], s["A"], tok[2], tok[3], s["skip"], tok[4], s["dt_bias"], s["h0"], ok)
        return dict(y=y[ok][None].to(s["x"].dtype), h=h)
    if op == "ssm_step":
        x, st = f(s["x"]), s["state"]
        step = _softplus(f(s["dt"]) + s["dt_bias"])
        heads = lambda t: f(t).repeat_interleave(c["D"] // c["G"], 1)  # noqa: E731
        st.mul_(torch.exp(step[..., None] * s["A"]))
        st.add_((step * x)[..., None] * heads(s["B"]))
        y = (st * heads(s["C"])).sum(-1) + s["skip"] * x
        if c["gate"]:
            y = y * _silu(f(s["gate"]))
        return dict(y=y.to(s["x"].dtype), state=st)
    if op == "ssm_bwd":
        dt = s["x"].dtype
        names = ["x", "dt", "A", "B", "C", "skip"] + (["gate"] if c["gate"] else []) + ["dt_bias"] + (["h0"] if c["h0"] else [])
        leaf = {n: f(s[n]).clone().requires_grad_(True) for n in names}
        y, h = _ssm(*(leaf.get(n) for n in ("x", "dt", "A", "B", "C", "skip", "gate", "dt_bias", "h0")))
        got = torch.autograd.grad([y, h], list(leaf.values()), [f(s["d_y"]), s["dhT"]])
        return {"d" + n: (t.to(dt) if n in ("x", "dt", "B", "C", "gate") else t) for n, t in zip(leaf, got)}
    if op == "select":
        x = s["logits"].double()
        m = x.amax(-1, keepdim=True)
        total = s["scores"].double()[..., None] + (x - m - torch.exp(x - m).sum(-1, keepdim=True).log())
        if s["finished"] is not None:      # a finished beam goes on as it is, with one candidate
            end = torch.full_like(total, -math.inf)
            end[..., EOS] = s["scores"].double()
            total = torch.where(s["finished"][..., None], end, total)
        best, at = total.flatten(1).sort(dim=1, descending=True, stable=True)
        at = at[:, :c["k"]]
        return dict(scores=best[:, :c["k"]].float(), parents=(at // c["V"]).int(), tokens=(at % c["V"]).int())
    rows = (torch.arange(c["B"], device="cuda")[:, None] * c["W"] + s["parents"]).flatten()
    for t in s["states"]:
        t.copy_(t[rows])
    return list(s["states"])


# ------------------------------------------------------------------------------------ the framework's calls


def run(s):
    if not own:
        return _plain(s)
    import delta_rule_linear_gb300 as kda
    c = s["case"]
    op = c["op"]
    if op.startswith("conv"):
        act = c["act"] if c["act"] != "none" else None
        if op == "conv":
            y, st = kda.conv_fwd(s["x"], s["w"], s["bias"], s["h0"], activation=act)
            return dict(y=y, state=st)
        if op == "conv_varlen":
            y, st = kda.conv_varlen_fwd(s["x"], s["w"], s["cu"], s["bias"], s["h0"], activation=act, cu_seqlens_cpu=s["cu_host"])
            return dict(y=y, state=st)
        if op == "conv_step":
            y = kda.conv_decode_step(s["x"], s["w"], s["state"], s["bias"], activation=act)
            return dict(y=y, state=s["state"])
        return kda.conv_bwd(s["d_y"], s["x"], s["w"], s["bias"], s["h0"], s["dhT"], activation=act)
    if op.startswith("ssm"):
        kw = dict(skip=s["skip"], gate=s["gate"], dt_bias=s["dt_bias"])
        tok = (s["x"], s["dt"], s["A"], s["B"], s["C"])
        if op == "ssm":
            y, h = kda.ssm_chunk_fwd(*tok, s["h0"], **kw)
            return dict(y=y, h=h)
        if op == "ssm_varlen":
            y, h = kda.ssm_varlen_fwd(*tok, s["cu"], s["h0"], cu_seqlens_cpu=s["cu_host"], **kw)
            return dict(y=y, h=h)
        if op == "ssm_step":
            y = kda.ssm_decode_step(*tok, s["state"], **kw)
            return dict(y=y, state=s["state"])
        return kda.ssm_chunk_bwd(s["d_y"], *tok, s["h0"], s["dhT"], **kw)
    if op == "select":
        best, parents, tokens = kda.beam_select(s["logits"], s["scores"], c["k"], finished=s["finished"], eos=EOS)
        return dict(scores=best, parents=parents, tokens=tokens)
    return kda.beam_reorder(s["states"], s["parents"])


# ------------------------------------------------------------------------------------ 64-bit references


def _sequences(c, s, n):
    """(first row, rows) of each sequence in [B * T] rows."""
    if "cu_host" in s:
        cu = s["cu_host"].tolist()
        return list(zip(cu, (b - a for a, b in zip(cu, cu[1:]))))
    T = c.get("T", 1)
    return [(b * T, T) for b in range(n)]


def _conv64(c, s):
    """Tap by tap over rows of one sequence at a time: pre-activations of all rows, and the gradients if d_y is there."""
    K, C = c["K"], c["C"]
    x, w = s["x"].double().reshape(-1, C), s["w"].double()
    n = c["N"] if "cu_host" in s else c["B"]
    h0 = s.get("h0") if s.get("h0") is not None else s.get("state")
    h0 = h0.double() if h0 is not None else x.new_zeros(n, K - 1, C)
    pre, last = torch.empty_like(x), torch.empty(n, K - 1, C, dtype=torch.float64, device="cuda")
    dx, dw, dh = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(h0)
    dpre = None
    silu = c["act"] == "silu"
    dbias = x.new_zeros(C)
    for i, (a, T) in enumerate(_sequences(c, s, n)):
        r = torch.cat([h0[i], x[a:a + T]])
        p = torch.zeros(T, C, dtype=torch.float64, device="cuda")
        for j in range(K):
            p += r[j:j + T] * w[:, j]
        if s["bias"] is not None:
            p += s["bias"].double()
        pre[a:a + T], last[i] = p, r[T:]
        if "d_y" not in s:
            continue
        dpre = s["d_y"].double().reshape(-1, C)[a:a + T]
        if silu:
            sg = torch.sigmoid(p)
            dpre = dpre * sg * (1 + p * (1 - sg))
        dr = torch.zeros_like(r)
        dr[T:] += s["dhT"].double()[i]
        for j in range(K):
            dr[j:j + T] += dpre * w[:, j]
            dw[:, j] += (dpre * r[j:j + T]).sum(0)
        dbias += dpre.sum(0)
        dh[i], dx[a:a + T] = dr[:K - 1], dr[K - 1:]
    y = pre * torch.sigmoid(pre) if silu else pre
    return y, last, dx, dw, dbias, dh


def _ssm64(c, s, n):
    """Token by token; sequences of different lengths go on side by side until each one's end."""
    D, N, G = c["D"], c["N"], c["G"]
    rows = lambda t: t.double().reshape(-1, *t.shape[-1:]) if t.dim() == s["x"].dim() else t.double().reshape(-1, G, N)  # noqa: E731
    x, dt, Bm, Cm = (rows(s[k]) for k in ("x", "dt", "B", "C"))
    gate = rows(s["gate"]) if s["gate"] is not None else None
    A, skip = s["A"].double(), s["skip"].double()
    raw = dt + s["dt_bias"].double()
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    seqs = _sequences(c, s, n)
    first = torch.tensor([a for a, _ in seqs], device="cuda")
    lens = [t for _, t in seqs]
    h = s.get("h0") if s.get("h0") is not None else s.get("state")
    h = h.double().clone() if h is not None else torch.zeros(n, D, N, dtype=torch.float64, device="cuda")
    order = sorted(range(n), key=lambda i: -lens[i])
    at = torch.tensor(order, device="cuda")
    first, h = first[at], h[at]
    most = max(lens)
    live = [sum(1 for l in lens if l > t) for t in range(most)]
    grad = "d_y" in s
    raw_y = torch.empty_like(x)
    spread = lambda t: t[:, :, None].expand(-1, -1, D // G, -1).reshape(-1, D, N)  # noqa: E731
    kept = []
    for t in range(most):
        m = live[t]
        r = first[:m] + t
        a, u = torch.exp(dt[r, :, None] * A), (dt[r] * x[r])[..., None]
        new = a * h[:m] + u * spread(Bm[r])
        if grad:
            kept.append(h[:m].clone())
        h[:m] = new
        raw_y[r] = (new * spread(Cm[r])).sum(-1) + skip * x[r]
    sg = torch.sigmoid(gate) if gate is not None else None
    y = raw_y * gate * sg if gate is not None else raw_y
    back = torch.empty_like(at)
    back[at] = torch.arange(n, device="cuda")
    if not grad:
        return y, h[back], None
    dy = s["d_y"].double().reshape(-1, D)
    out = {}
    if gate is not None:
        out["dgate"] = dy * raw_y * sg * (1 + gate * (1 - sg))
        dy = dy * gate * sg
    out["dx"], out["ddt"] = skip * dy, torch.zeros_like(x)
    out["dskip"] = (dy * x).sum(0)
    out["dA"], out["dB"], out["dC"] = torch.zeros_like(A), torch.zeros_like(Bm), torch.zeros_like(Cm)
    fold = lambda t: t.reshape(-1, G, D // G, N).sum(2)  # noqa: E731
    D_h = s["dhT"].double()[at].clone()
    for t in range(most - 1, -1, -1):
        m = live[t]
        r = first[:m] + t
        a, u = torch.exp(dt[r, :, None] * A), (dt[r] * x[r])[..., None]
        now = a * kept[t] + u * spread(Bm[r])
        g = D_h[:m] + dy[r][..., None] * spread(Cm[r])
        out["dC"][r] = fold(dy[r][..., None] * now)
        out["dB"][r] = fold(u * g)
        gB = (g * spread(Bm[r])).sum(-1)
        ga = g * a
        e = ga * kept[t]
        out["dx"][r] += dt[r] * gB
        out["ddt"][r] = x[r] * gB + (e * A).sum(-1)
        out["dA"] += (e * dt[r][..., None]).sum(0)
        D_h[:m] = ga
    out["ddt"] *= torch.sigmoid(raw)
    out["ddt_bias"] = out["ddt"].sum(0)
    out["dh0"] = D_h[back]
    return y, h[back], out


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op.startswith("conv"):
        y, last, dx, dw, dbias, dh = _conv64(c, s)
        if op != "conv_bwd":
            return dict(y=y.reshape(s["x"].shape), state=last)
        out = dict(dx=dx.reshape(s["x"].shape), dw=dw)
        if c["bias"]:
            out["dbias"] = dbias
        if c["h0"]:
            out["dstate"] = dh
        return out
    if op.startswith("ssm"):
        n = c["N_seq"] if op == "ssm_varlen" else c["B"]
        y, h, grads = _ssm64(c, s, n)
        if op == "ssm_step":
            return dict(y=y.reshape(s["x"].shape), state=h)
        if op != "ssm_bwd":
            return dict(y=y.reshape(s["x"].shape), h=h)
        shape = dict(dx="x", ddt="dt", dA="A", dB="B", dC="C", dskip="skip", dgate="gate", ddt_bias="dt_bias", dh0="h0")
        names = [k for k in shape if (k != "dgate" or c["gate"]) and (k != "dh0" or c["h0"])]
        order = ["dx", "ddt", "dA", "dB", "dC", "dskip", "dgate", "ddt_bias", "dh0"]
        return {k: grads[k].reshape(s[shape[k]].shape) for k in order if k in names}
    if op == "select":
        import numpy as np
        B, W, V, k = c["B"], c["W"], c["V"], c["k"]
        x, sc = s["logits"].double(), s["scores"].double()
        total = (sc - torch.logsumexp(x, -1))[..., None] + x
        out = dict(scores=[], parents=[], tokens=[])
        for b in range(B):
            row = total[b].cpu().numpy()
            if s["finished"] is not None:
                for w in range(W):
                    if bool(s["finished"][b, w]):
                        row[w] = -np.inf
                        row[w, EOS] = float(sc[b, w])
            row = row.reshape(-1)
            least = np.partition(row, row.size - k)[row.size - k]
            cand = np.flatnonzero(row >= least)
            cand = cand[np.lexsort((cand, -row[cand]))][:k]
            out["scores"].append(row[cand])
            out["parents"].append(cand // V)
            out["tokens"].append(cand % V)
        return dict(scores=torch.from_numpy(np.stack(out["scores"])).cuda(),
                    parents=torch.from_numpy(np.stack(out["parents"])).int().cuda(),
                    tokens=torch.from_numpy(np.stack(out["tokens"])).int().cuda())
    W = c["W"]
    out = []
    for t in s["states"]:
        src = t.unflatten(0, (c["B"], W))
        out.append(torch.stack([src[b][s["parents"][b].long()] for b in range(c["B"])]).flatten(0, 1).double())
    return out
