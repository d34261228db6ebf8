"""Cases, plain forms and 64-bit references of the linear-attention operators and block norms.

Linear attention with one log decay per value head and token (a fixed one per head: the same
value at every token), h_t a [dk, dv] memory per head, s the query scale:

    h_t = exp(decay_t) h_{t-1} + k_t v_t^T,      o_t = h_t^T (s q_t)

as chunked prefill (equal-length or packed sequences), as a single-token step that updates the
memory in place, and as the gradients of the prefill; and the norms around such a block:

    gated norm      y = x rsqrt(mean(x^2) + eps) w act(gate)              (per head, after it)
    residual norm   x' = x + c y,   n = x' rsqrt(mean(x'^2) + eps) w      (per token, before the next)

`run` computes a case either by elementary torch operations in 32 bits, or by the calls of
delta_rule_linear_gb300 where `own` is true.
"""
import math
import random

import torch

own = False

CHUNK = 128     # tokens per chunk of the plain form

# ------------------------------------------------------------------------------------ cases


def listed():
    return [
        # A short prompt of a small fp32 model: where the call itself is what counts.
        dict(name="fwd_short_fp32", op="fwd", dtype="f32", B=1, T=45, H=2, m=1, dk=32, dv=32,
             decay="small", h0=False, fused=False),
        # The training-shape prefill: two sequences, q, k and v slices of one projection.
        dict(name="fwd_train", op="fwd", dtype="bf16", B=2, T=2048, H=16, m=1, dk=128, dv=128,
             decay="train", h0=False, fused=True),
        # One long prompt that continues from a carried memory.
        dict(name="fwd_long", op="fwd", dtype="bf16", B=1, T=32768, H=32, m=1, dk=128, dv=128,
             decay="long", h0=True, fused=False),
        # Sixteen packed prompts of 256 to 4096 tokens, memories kept per prompt.
        dict(name="fwd_packed", op="varlen", dtype="bf16", N=16, lo=256, hi=4096, lens=0, H=16, m=1,
             dk=64, dv=64, decay="small", h0=False, fused=False),
        # One token for each of 256 requests: the serving step, bound by the memories.
        dict(name="step_256", op="step", dtype="bf16", B=256, H=32, m=1, dk=128, dv=128, decay="small"),
        # One token for three requests, two value heads to a key head: latency.
        dict(name="step_3_grouped", op="step", dtype="bf16", B=3, H=4, m=2, dk=128, dv=64, decay="small"),
        # Gradients at the training shape.
        dict(name="bwd_train", op="bwd", dtype="bf16", B=2, T=2048, H=16, m=1, dk=128, dv=128,
             decay="train", h0=True, fused=True),
        # Gradients of an odd length in fp32, one key head shared by two value heads.
        dict(name="bwd_odd_fp32", op="bwd", dtype="f32", B=1, T=301, H=2, m=2, dk=64, dv=32,
             decay="small", h0=False, fused=False),
        # The norm and gate behind a long prompt's attention, 32 heads of 128 per token.
        dict(name="gated_norm_long", op="gnorm", dtype="bf16", rows=32768, H=32, d=128, act="silu"),
        # The same at the training shape, backwards.
        dict(name="gated_norm_grad", op="gnorm_bwd", dtype="bf16", rows=4096, H=16, d=128, act="silu"),
        # Residual and norm of one serving step: 256 tokens of width 4096.
        dict(name="residual_norm_step", op="rnorm", dtype="bf16", res="bf16", rows=256, d=4096, vec=False),
        # Residual and norm backwards at the training shape, fp32 residual stream, learned scale.
        dict(name="residual_norm_grad", op="rnorm_bwd", dtype="bf16", res="f32", rows=4096, d=2048, vec=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "varlen", "step", "bwd", "gnorm", "gnorm_bwd", "rnorm", "rnorm_bwd"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    heads = dict(H=_log_int(rng, 1, 32), m=rng.choice([1, 1, 2, 4]), dk=rng.choice([32, 64, 128, 128]))
    heads["dv"] = rng.choice([heads["dk"], heads["dk"], 32, 64, 128])
    decay = rng.choice(["small", "train", "long"])
    if op in ("fwd", "bwd"):
        B = _log_int(rng, 1, 8)
        most = (1 << 20) if op == "fwd" else (1 << 16)      # tokens x value heads
        if dt == "f32":
            most = min(most, 1 << 17)
        if heads["H"] * heads["m"] > 32:
            heads["m"] = 1
        top = max(2, min(32768 if op == "fwd" else 4096, most // (B * heads["H"] * heads["m"])))
        return dict(op=op, dtype=dt, B=B, T=_log_int(rng, 1, top), **heads, decay=decay,
                    h0=rng.random() < 0.5, fused=rng.random() < 0.5)
    if op == "varlen":
        hi = _log_int(rng, 16, 4096)
        if heads["H"] * heads["m"] > 16:
            heads.update(H=16, m=1)
        return dict(op=op, dtype=dt, N=_log_int(rng, 1, 24 if dt == "bf16" else 4), lo=max(1, hi // 16), hi=hi,
                    lens=rng.randrange(1 << 16), **heads, decay=decay, h0=rng.random() < 0.5, fused=False)
    if op == "step":
        return dict(op=op, dtype=dt, B=_log_int(rng, 1, 256), H=min(heads["H"], 32 // heads["m"]), m=heads["m"],
                    dk=heads["dk"], dv=heads["dv"], decay=decay)
    if op in ("gnorm", "gnorm_bwd"):
        return dict(op=op, dtype=dt, rows=_log_int(rng, 1, 32768 if op == "gnorm" else 8192), H=_log_int(rng, 1, 32),
                    d=rng.choice([32, 64, 128, 128, 256, rng.randrange(20, 250)]), act=rng.choice(["silu", "sigmoid"]))
    d = rng.choice([1024, 2048, 4096, 8192, _log_int(rng, 64, 8192)])
    rows = _log_int(rng, 1, 32768 if op == "rnorm" else 8192)
    return dict(op=op, dtype=dt, res=rng.choice([dt, "f32"]), rows=min(rows, (1 << 27) // d), d=d, vec=rng.random() < 0.5)


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _lens(c):
    r = random.Random(c["lens"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["N"])]


def work(c):
    e = 2 if c.get("dtype") == "bf16" else 4
    if c["op"] in ("fwd", "varlen", "bwd", "step"):
        HV = c["H"] * c["m"]
        n = c["B"] if c["op"] != "varlen" else c["N"]
        rows = sum(_lens(c)) if c["op"] == "varlen" else c["B"] * c.get("T", 1)
        st = n * HV * c["dk"] * c["dv"] * 4
        qk, v = rows * c["H"] * c["dk"] * e, rows * HV * c["dv"] * e
        dec = rows * HV * 4
        cells = rows * HV * c["dk"] * c["dv"]
        if c["op"] == "bwd":
            # q, k, v, d_o, decay, dfinal_state (and the initial memory) in; five gradients out
            return {"bytes": 4 * qk + 3 * v + 2 * dec + st + (2 * st if c["h0"] else 0), "flops": 10 * cells}
        if c["op"] == "step":
            return {"bytes": 2 * qk + 2 * v + dec + 2 * st, "flops": 4 * cells}
        return {"bytes": 2 * qk + 2 * v + dec + (2 if c["h0"] else 1) * st, "flops": 4 * cells}
    if c["op"] in ("gnorm", "gnorm_bwd"):
        n = c["rows"] * c["H"] * c["d"]
        return {"bytes": (3 if c["op"] == "gnorm" else 5) * n * e + 4 * c["d"], "flops": (10 if c["op"] == "gnorm" else 25) * n}
    n, r = c["rows"] * c["d"], 4 if c["res"] == "f32" else 2
    if c["op"] == "rnorm":
        return {"bytes": 2 * n * r + 2 * n * e + 4 * c["d"], "flops": 7 * n}
    # d_n, d_x', x' (and y for a learned scale's gradient) in; dx, dy out
    return {"bytes": 3 * n * r + (2 + c["vec"]) * n * e + 12 * c["d"], "flops": 14 * n}


# ------------------------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _decay(g, kind, shape):
    z = torch.randn(shape, generator=g, device="cuda")
    if kind == "small":
        return -0.01 * z.abs()
    if kind == "train":
        return -0.05 * z.abs()
    return -torch.log1p(torch.exp(z - 4.0))        # strongly retentive


def prepare(c, seed):
    g = _gen(seed)
    rn = lambda *s, dt=torch.float32: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    dt = _dt(c["dtype"])
    s = dict(case=c)
    if c["op"] in ("fwd", "varlen", "bwd"):
        H, HV, dk, dv = c["H"], c["H"] * c["m"], c["dk"], c["dv"]
        if c["op"] == "varlen":
            lens = _lens(c)
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
            s["cu_host"] = torch.tensor(cu, dtype=torch.int32)      # a scheduler has the lengths at hand
            B, T, N = 1, cu[-1], c["N"]
        else:
            B, T, N = c["B"], c["T"], c["B"]
        if c["fused"]:     # slices of one projection's output, not copied apart
            z = rn(B, T, 2 * H * dk + HV * dv, dt=dt)
            q, k, v = z[..., :H * dk], z[..., H * dk:2 * H * dk], z[..., 2 * H * dk:]
            s["q"], s["k"], s["v"] = (x.unflatten(-1, (h, -1)) for x, h in ((q, H), (k, H), (v, HV)))
        else:
            s["q"], s["k"], s["v"] = rn(B, T, H, dk, dt=dt), rn(B, T, H, dk, dt=dt), rn(B, T, HV, dv, dt=dt)
        s["decay"] = _decay(g, c["decay"], (B, T, HV))
        s["h0"] = 0.02 * rn(N, HV, dk, dv) if c["h0"] else None
        if c["op"] == "bwd":
            s["d_o"], s["dhT"] = rn(B, T, HV, dv, dt=dt), 0.02 * rn(N, HV, dk, dv)
    elif c["op"] == "step":
        B, H, HV, dk, dv = c["B"], c["H"], c["H"] * c["m"], c["dk"], c["dv"]
        s["q"], s["k"], s["v"] = rn(B, 1, H, dk, dt=dt), rn(B, 1, H, dk, dt=dt), rn(B, 1, HV, dv, dt=dt)
        s["decay"] = _decay(g, c["decay"], (B, 1, HV))
        s["state"] = rn(B, HV, dk, dv)
    elif c["op"] in ("gnorm", "gnorm_bwd"):
        s["x"], s["gate"] = rn(c["rows"], c["H"], c["d"], dt=dt), rn(c["rows"], c["H"], c["d"], dt=dt)
        s["w"] = 1.0 + 0.1 * rn(c["d"])
        if c["op"] == "gnorm_bwd":
            s["d_y"] = rn(c["rows"], c["H"], c["d"], dt=dt)
    else:
        s["x"], s["y"] = rn(c["rows"], c["d"], dt=_dt(c["res"])), rn(c["rows"], c["d"], dt=dt)
        s["w"] = 1.0 + 0.1 * rn(c["d"])
        s["c"] = 0.5 + 0.05 * rn(c["d"]) if c["vec"] else 0.5
        if c["op"] == "rnorm_bwd":
            s["d_n"], s["d_x"] = rn(c["rows"], c["d"], dt=dt), rn(c["rows"], c["d"], dt=_dt(c["res"]))
    return s


EPS = 1e-6

# ------------------------------------------------------------------------------------ plain forms


def _attend(q, k, v, decay, h0, scale):
    """Chunked linear attention on fp32 [B, T, HV, .]: (o, final memory)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    C = min(CHUNK, T)
    n = -(-T // C)
    pad = n * C - T

    def chunks(x):
        x = torch.cat([x, x.new_zeros(B, pad, *x.shape[2:])], 1) if pad else x
        return x.unflatten(1, (n, C)).movedim(3, 1)          # [B, H, n, C, ...]

    q, k, v, g = chunks(q * scale), chunks(k), chunks(v), chunks(decay)
    G = g.cumsum(-1)                                          # [B, H, n, C]
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    D = (G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf).exp()
    o = ((q @ k.transpose(-1, -2)) * D) @ v
    kv = (k * (G[..., -1:] - G).exp()[..., None]).transpose(-1, -2) @ v      # [B, H, n, dk, dv]
    # memory before chunk i: what every chunk j < i left, decayed by the chunks between them
    tot = G[..., -1]                                          # [B, H, n]
    late = torch.ones(n + 1, n, dtype=torch.bool, device=q.device).tril(-1)  # j < i
    between = torch.ones(n, n, dtype=torch.bool, device=q.device).tril(-1)   # chunk l after chunk j
    seg = (tot[..., :, None] * between).cumsum(-2)            # sum of chunks j+1 .. l at [l, j]
    seg = torch.cat([seg.new_zeros(B, H, 1, n), seg], -2).masked_fill(~late, -math.inf).exp()
    S = (seg @ kv.flatten(-2)).unflatten(-1, (dk, dv))        # [B, H, n + 1, dk, dv]
    if h0 is not None:
        run0 = torch.cat([tot.new_zeros(B, H, 1), tot.cumsum(-1)], -1).exp()
        S = S + run0[..., None, None] * h0[:, :, None]
    o = o + G.exp()[..., None] * (q @ S[:, :, :-1])
    return o.movedim(1, 3).flatten(1, 2)[:, :T], S[:, :, -1]


def _spread(x, m):
    """q/k heads to value heads: consecutive value heads share one."""
    return x.repeat_interleave(m, 2) if m > 1 else x


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op in ("fwd", "bwd", "varlen"):
        scale = c["dk"] ** -0.5
        dt = s["q"].dtype
    if op == "fwd":
        q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
        o, hT = _attend(_spread(q, c["m"]), _spread(k, c["m"]), v, s["decay"], s["h0"], scale)
        return dict(o=o.to(dt), h=hT)
    if op == "varlen":
        cu = s["cu_host"].to(torch.int64)
        lens = cu[1:] - cu[:-1]
        most = int(lens.max())
        at = cu[:-1, None] + torch.arange(most)               # [N, most] row of each padded place
        ok = torch.arange(most) < lens[:, None]
        at, ok = torch.where(ok, at, 0).cuda(), ok.cuda()
        take = lambda x: torch.where(ok.view(*ok.shape, *[1] * (x.dim() - 2)), x[0, at].float(), 0.0)  # noqa: E731
        q, k, v, g = (take(x) for x in (s["q"], s["k"], s["v"], s["decay"]))
        o, hT = _attend(_spread(q, c["m"]), _spread(k, c["m"]), v, g, s["h0"], scale)
        return dict(o=o[ok][None].to(dt), h=hT)
    if op == "bwd":
        leaf = [x.float().requires_grad_(True) for x in (s["q"].detach(), s["k"].detach(), s["v"].detach())]
        dec = s["decay"].clone().requires_grad_(True)
        h0 = s["h0"].clone().requires_grad_(True) if s["h0"] is not None else None
        o, hT = _attend(_spread(leaf[0], c["m"]), _spread(leaf[1], c["m"]), leaf[2], dec, h0, scale)
        wrt = leaf + [dec] + ([h0] if h0 is not None else [])
        got = torch.autograd.grad([o, hT], wrt, [s["d_o"].float(), s["dhT"]])
        out = dict(dq=got[0].to(dt), dk=got[1].to(dt), dv=got[2].to(dt), ddecay=got[3])
        if h0 is not None:
            out["dh0"] = got[4]
        return out
    if op == "step":
        q, k = (_spread(x.float(), c["m"])[:, 0] for x in (s["q"], s["k"]))
        st = s["state"]
        st.mul_(s["decay"].exp()[:, 0, :, None, None])
        st.add_(k[..., :, None] * s["v"].float()[:, 0, :, None, :])
        o = (st * (q * c["dk"] ** -0.5)[..., :, None]).sum(-2)
        return dict(o=o[:, None].to(s["v"].dtype), state=st)
    if op in ("gnorm", "gnorm_bwd"):
        x, a, w = s["x"].float(), s["gate"].float(), s["w"]
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        sg = 1.0 / (1.0 + torch.exp(-a))
        act = a * sg if c["act"] == "silu" else sg
        if op == "gnorm":
            return dict(y=(x * r * w * act).to(s["x"].dtype))
        dact = sg * (1.0 + a * (1.0 - sg)) if c["act"] == "silu" else sg * (1.0 - sg)
        dy, xn = s["d_y"].float(), x * r
        t = dy * act * w
        dx = r * (t - xn * (t * xn).mean(-1, keepdim=True))
        return dict(dx=dx.to(s["x"].dtype), dgate=(dy * xn * w * dact).to(s["x"].dtype),
                    dw=(dy * act * xn).sum((0, 1)))
    x, y, w = s["x"].float(), s["y"].float(), s["w"]
    if op == "rnorm":
        z = x + s["c"] * y
        n = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS) * w
        return dict(x=z.to(s["x"].dtype), n=n.to(s["y"].dtype))
    # gradients at x' = s["x"]
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xn, dn = x * r, s["d_n"].float()
    t = dn * w
    dx = s["d_x"].float() + r * (t - xn * (t * xn).mean(-1, keepdim=True))
    out = dict(dx=dx.to(s["x"].dtype), dy=(s["c"] * dx).to(s["y"].dtype), dw=(dn * xn).sum(0))
    if c["vec"]:
        out["dscale"] = (dx * y).sum(0)
    return out


# ------------------------------------------------------------------------------------ the framework's calls


def run(s):
    if not own:
        return _plain(s)
    import delta_rule_linear_gb300 as kda
    c = s["case"]
    op = c["op"]
    if op == "fwd":
        o, h = kda.linear_chunk_fwd(s["q"], s["k"], s["v"], s["decay"], s["h0"])
        return dict(o=o, h=h)
    if op == "varlen":
        o, h = kda.linear_varlen_fwd(s["q"], s["k"], s["v"], s["cu"], s["decay"], s["h0"], cu_seqlens_cpu=s["cu_host"])
        return dict(o=o, h=h)
    if op == "bwd":
        return kda.linear_chunk_bwd(s["q"], s["k"], s["v"], s["decay"], s["h0"], s["d_o"], s["dhT"])
    if op == "step":
        o = kda.linear_decode_step(s["q"], s["k"], s["v"], s["decay"], s["state"])
        return dict(o=o, state=s["state"])
    if op == "gnorm":
        return dict(y=kda.gated_norm_fwd(s["x"], s["gate"], s["w"], eps=EPS, activation=c["act"]))
    if op == "gnorm_bwd":
        return kda.gated_norm_bwd(s["d_y"], s["x"], s["gate"], s["w"], eps=EPS, activation=c["act"])
    if op == "rnorm":
        x, n = kda.residual_norm_fwd(s["x"], s["y"], s["w"], scale=s["c"], eps=EPS)
        return dict(x=x, n=n)
    return kda.residual_norm_bwd(s["d_n"], s["d_x"], s["x"], s["w"], s["y"] if c["vec"] else None, scale=s["c"], eps=EPS)


# ------------------------------------------------------------------------------------ 64-bit references


def _walk(q, k, v, g, h):
    """The recurrence token by token on fp64 [T, P, .] (P = sequence and head pairs), h [P, dk, dv]."""
    o = v.new_empty(v.shape)
    a = g.exp()
    for t in range(q.shape[0]):
        h = torch.baddbmm(h * a[t, :, None, None], k[t, :, :, None], v[t, :, None, :])
        o[t] = torch.bmm(q[t, :, None, :], h)[:, 0]
    return o, h


def _pairs(x, m=1):
    """[B, T, H, ...] to fp64 [T, B * HV, ...]."""
    x = x.double()
    if m > 1:
        x = x[:, :, :, None].expand(-1, -1, -1, m, *[-1] * (x.dim() - 3)).flatten(2, 3)
    return x.movedim(1, 0).flatten(1, 2)


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op in ("fwd", "bwd", "varlen", "step"):
        H, m, dk, dv = c["H"], c["m"], c["dk"], c["dv"]
        HV, scale = H * m, c["dk"] ** -0.5
    if op == "fwd":
        B, T = c["B"], c["T"]
        if B * T * HV * dk * dv > 1 << 35:
            return None                                # half a minute of token steps
        h = s["h0"].double().flatten(0, 1) if s["h0"] is not None else torch.zeros(B * HV, dk, dv, dtype=torch.float64, device="cuda")
        o, h = _walk(_pairs(s["q"], m) * scale, _pairs(s["k"], m), _pairs(s["v"]), _pairs(s["decay"]), h)
        return dict(o=o.unflatten(1, (B, HV)).movedim(0, 1).contiguous(), h=h.unflatten(0, (B, HV)))
    if op == "varlen":
        cu, N = s["cu_host"].tolist(), c["N"]
        most = max(b - a for a, b in zip(cu, cu[1:]))
        put = lambda x: torch.stack([torch.cat([x[0, a:b].double(), torch.zeros(most - (b - a), *x.shape[2:], dtype=torch.float64, device="cuda")])  # noqa: E731
                                     for a, b in zip(cu, cu[1:])])
        h = s["h0"].double().flatten(0, 1) if s["h0"] is not None else torch.zeros(N * HV, dk, dv, dtype=torch.float64, device="cuda")
        o, h = _walk(_pairs(put(s["q"]), m) * scale, _pairs(put(s["k"]), m), _pairs(put(s["v"])), _pairs(put(s["decay"])), h)
        o = o.unflatten(1, (N, HV)).movedim(0, 1)
        return dict(o=torch.cat([o[n, :b - a] for n, (a, b) in enumerate(zip(cu, cu[1:]))])[None], h=h.unflatten(0, (N, HV)))
    if op == "step":
        st = s["state"].double() * s["decay"].double().exp()[:, 0, :, None, None]
        st = st + torch.einsum("bhi,bhj->bhij", _pairs(s["k"], m)[0].unflatten(0, (-1, HV)), s["v"].double()[:, 0])
        o = torch.einsum("bhi,bhij->bhj", _pairs(s["q"], m)[0].unflatten(0, (-1, HV)) * scale, st)
        return dict(o=o[:, None], state=st)
    if op == "bwd":
        # forward: h_t and dq_t = s h_t do_t; backward: the memory's gradient D_t (before its decay),
        # dk_t = D_t v_t, dv_t = D_t^T k_t, ddecay_t = exp(decay_t) <h_{t-1}, D_t>, where D_t collects s q_t do_t
        B, T = c["B"], c["T"]
        q, k, v, g, do = _pairs(s["q"], m) * scale, _pairs(s["k"], m), _pairs(s["v"]), _pairs(s["decay"]), _pairs(s["d_o"])
        a = g.exp()
        P = B * HV
        h = s["h0"].double().flatten(0, 1) if s["h0"] is not None else torch.zeros(P, dk, dv, dtype=torch.float64, device="cuda")
        if T * P * dk * dv * 8 > 40 << 30:
            return None                                # every token's memory is kept below
        kept = torch.empty(T + 1, P, dk, dv, dtype=torch.float64, device="cuda")
        kept[0] = h
        dq, dkk, dvv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        for t in range(T):
            kept[t + 1] = torch.baddbmm(kept[t] * a[t, :, None, None], k[t, :, :, None], v[t, :, None, :])
            dq[t] = torch.bmm(kept[t + 1], do[t, :, :, None])[:, :, 0] * scale
        dd = torch.empty_like(g)
        D = s["dhT"].double().flatten(0, 1)
        for t in range(T - 1, -1, -1):
            D = torch.baddbmm(D, q[t, :, :, None], do[t, :, None, :])
            dkk[t] = torch.bmm(D, v[t, :, :, None])[:, :, 0]
            dvv[t] = torch.bmm(k[t, :, None, :], D)[:, 0]
            D = D * a[t, :, None, None]
            dd[t] = (kept[t] * D).sum((-1, -2))
        back = lambda x: x.unflatten(1, (B, HV)).movedim(0, 1).contiguous()  # noqa: E731
        fold = lambda x: back(x).unflatten(2, (H, m)).sum(3)  # noqa: E731
        out = dict(dq=fold(dq), dk=fold(dkk), dv=back(dvv), ddecay=back(dd))
        if c["h0"]:
            out["dh0"] = D.unflatten(0, (B, HV))
        return out
    s = {n: (x.double() if isinstance(x, torch.Tensor) else x) for n, x in s.items()}
    if op in ("gnorm", "gnorm_bwd"):
        x = s["x"].requires_grad_(True)
        a, w = s["gate"].requires_grad_(True), s["w"].requires_grad_(True)
        y = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w * (torch.sigmoid(a) * (a if c["act"] == "silu" else 1.0))
        if op == "gnorm":
            return dict(y=y.detach())
        dx, da, dw = torch.autograd.grad(y, [x, a, w], s["d_y"])
        return dict(dx=dx, dgate=da, dw=dw)
    if op == "rnorm":
        z = s["x"] + s["c"] * s["y"]
        return dict(x=z, n=z / (z.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * s["w"])
    z, w = s["x"].requires_grad_(True), s["w"].requires_grad_(True)
    n = z / (z.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w
    dz, dw = torch.autograd.grad([n, z * 1.0], [z, w], [s["d_n"], s["d_x"]])
    out = dict(dx=dz, dy=s["c"] * dz, dw=dw)
    if c["vec"]:
        out["dscale"] = (dz * s["y"]).sum(0)
    return out
