"""Measured cases of the operators around a Mamba-2 layer's state space duality (SSD).

A Mamba-2 layer projects its input to rows [z | x B C | dt], passes x B C through
a short causal convolution, runs the SSD over the heads, and normalises the
gated result.  The operators, on packed sequences of different lengths
(cu_seqlens) and on a cache of windows and states addressed by slots:

  conv    ssm_conv1d_fwd / ssm_conv1d_bwd / ssm_conv1d_step
  ssd     ssm_ssd_varlen_fwd (prompts)
  step    ssm_ssd_step (one token per sequence)
  norm    ssm_gated_norm_fwd / ssm_gated_norm_bwd

Layer sizes: "2.7B-like" is 80 heads of 64, one group, state 128, width 5120
(convolution over 5376 channels); "130M-like" is 24 heads of 64, width 1536
(convolution over 1792).
"""
import math

import torch

own = False

P, N, K = 64, 128, 4  # head dimension, state dimension, convolution width


def listed():
    return [
        # prompts of different lengths packed into one pass of a 2.7B-like layer; x B C is
        # read as a slice of the projection's rows; two sequences continue from a window
        dict(name="conv prompts", op="conv", lens="4096,1,2048,517,6000,33,2,3420", pad=0, width=5120, groups=1, bf16=True, sliced=True, initial=True),
        # a short float32 batch with rows behind the last sequence (a captured graph's padding)
        dict(name="conv small f32", op="conv", lens="300,7,1,400,0,64", pad=5, width=1536, groups=1, bf16=False, sliced=False, initial=True),
        # training: the gradients over packed documents, 2.7B-like
        dict(name="conv gradients", op="conv_bwd", lens="8192,511,1025,3000,3656", pad=0, width=5120, groups=1, bf16=True, sliced=True),
        # the same for an odd float32 batch of a 130M-like layer
        dict(name="conv gradients f32", op="conv_bwd", lens="1000,77,1,233", pad=3, width=1536, groups=1, bf16=False, sliced=False),
        # the decode batch of the benchmark: 256 sequences, one token each
        dict(name="conv step", op="conv_step", batch=256, width=5120, groups=1, bf16=True, sliced=True),
        # the benchmark's SSD shape: four prompts of 4096 through a 2.7B-like layer
        dict(name="ssd 4 x 4096", op="ssd", lens="4096,4096,4096,4096", pad=0, heads=80, groups=1, initial=False),
        # a serving batch of a 130M-like layer: many short prompts, some going on from a state
        dict(name="ssd ragged", op="ssd", lens="1,130,7,512,1024,64,255,256,257,900,0,33,2048,128,127,129,600,77,5,383", pad=9, heads=24, groups=1, initial=True),
        # one long prompt alone, 130M-like: few heads, many steps
        dict(name="ssd one long", op="ssd", lens="32768", pad=0, heads=24, groups=1, initial=False),
        # the decode batch of a 2.7B-like layer: bound by the states' bytes
        dict(name="step 256", op="step", batch=256, heads=80, groups=1, bf16=True),
        # one sequence alone: latency
        dict(name="step 1", op="step", batch=1, heads=24, groups=1, bf16=True),
        # after the SSD: the gated norm of 16384 tokens, z a slice of the projection's rows
        dict(name="norm", op="norm", rows=16384, width=5120, groups=1, bf16=True, gate_first=True, sliced=True),
        # its gradients
        dict(name="norm gradients", op="norm_bwd", rows=16384, width=5120, groups=1, bf16=True, gate_first=True, sliced=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, total, most):
    """Up to `most` lengths, from nothing to long, that sum to about `total` at most."""
    got = []
    for _ in range(rng.randint(1, most)):
        left = total - sum(got)
        if left < 1:
            break
        got.append(0 if rng.random() < 0.05 else _spread(rng, 1, left))
    if sum(got) == 0:
        got.append(_spread(rng, 1, total))
    rng.shuffle(got)
    return ",".join(map(str, got))


def draw(rng):
    op = rng.choice(["conv", "conv_bwd", "conv_step", "ssd", "ssd", "step", "norm", "norm_bwd"])
    heads = rng.choice([2, 8, 23, 24, 32, 40, 80])
    groups = rng.choice([g for g in (1, 2, 8) if heads % g == 0])
    bf16 = rng.random() < 0.7
    if op in ("conv", "conv_bwd"):
        c = dict(op=op, lens=_lens(rng, _spread(rng, 50, 16000), 40), pad=rng.choice([0, 0, 1, 17]), width=heads * P, groups=groups, bf16=bf16, sliced=rng.random() < 0.5)
        return dict(c, initial=rng.random() < 0.5) if op == "conv" else c
    if op == "conv_step":
        return dict(op=op, batch=_spread(rng, 1, 256), width=heads * P, groups=groups, bf16=bf16, sliced=rng.random() < 0.5)
    if op == "ssd":
        return dict(op=op, lens=_lens(rng, _spread(rng, 50, 16000), 40), pad=rng.choice([0, 0, 1, 17]), heads=heads, groups=groups, initial=rng.random() < 0.5)
    if op == "step":
        return dict(op=op, batch=_spread(rng, 1, 256), heads=heads, groups=groups, bf16=bf16)
    return dict(op=op, rows=_spread(rng, 1, 16000), width=heads * P, groups=groups, bf16=bf16, gate_first=rng.random() < 0.7, sliced=rng.random() < 0.5)


def _lengths(case):
    return [int(v) for v in case["lens"].split(",")]


def _rows(g, rows, width, after, sliced, dtype):
    """Rows of N(0, 1) values; sliced: a slice of wider rows, as the projection leaves them."""
    wide = torch.randn(rows, width + (after if sliced else 0), generator=g, device="cuda").to(dtype)
    return wide[:, :width]


def _silu_rows(g, rows, width, dtype):
    """Rows as the convolution's activation leaves them."""
    v = torch.randn(rows, width, generator=g, device="cuda")
    return (v * torch.sigmoid(v)).to(dtype)


def _head_parameters(g, heads):
    dt0 = torch.exp(torch.empty(heads, device="cuda").uniform_(math.log(1e-3), math.log(1e-1), generator=g))
    return dict(A=-torch.empty(heads, device="cuda").uniform_(1.0, 16.0, generator=g), dt_bias=torch.log(torch.expm1(dt0)),
                D=torch.ones(heads, device="cuda"))


def _packed(g, case):
    lens = _lengths(case)
    n = len(lens)
    at = [0]
    for v in lens:
        at.append(at[-1] + v)
    s = dict(lens=lens, tokens=at[-1] + case["pad"], cu=torch.tensor(at, dtype=torch.int32, device="cuda"))
    s["slots"] = torch.randperm(n + 2, generator=g, device="cuda")[:n].to(torch.int32)
    s["has_initial"] = torch.rand(n, generator=g, device="cuda") < 0.5 if case.get("initial") else None
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    dtype = torch.bfloat16 if case.get("bf16", True) else torch.float32
    s = dict(op=op)
    if op in ("conv", "conv_bwd", "conv_step"):
        dim = case["width"] + 2 * case["groups"] * N
        s["w"] = torch.randn(dim, K, generator=g, device="cuda") * 0.5
        s["bias"] = torch.randn(dim, generator=g, device="cuda") * 0.2
        if op == "conv_step":
            b = case["batch"]
            s["x"] = _rows(g, b, dim, case["width"] + 64, case["sliced"], dtype)
            s["windows"] = torch.randn(b + 2, K - 1, dim, generator=g, device="cuda").to(dtype)
            s["slots"] = torch.randperm(b + 2, generator=g, device="cuda")[:b].to(torch.int32)
            return s
        s.update(_packed(g, case))
        s["x"] = _rows(g, s["tokens"], dim, case["width"] + 64, case["sliced"], dtype)
        if op == "conv":
            s["windows"] = torch.randn(len(s["lens"]) + 2, K - 1, dim, generator=g, device="cuda").to(dtype)
            s["out"] = torch.zeros(s["tokens"], dim, dtype=dtype, device="cuda")
        else:
            s["dy"] = torch.randn(s["tokens"], dim, generator=g, device="cuda").to(dtype)
            s["dx"] = torch.zeros(s["tokens"], dim, dtype=dtype, device="cuda")
        return s
    if op in ("ssd", "step"):
        h, gr = case["heads"], case["groups"]
        s.update(_head_parameters(g, h))
        if op == "ssd":
            s.update(_packed(g, case))
            rows, slots, dtype = s["tokens"], len(s["lens"]) + 2, torch.bfloat16
            s["out"] = torch.zeros(rows, h, P, dtype=dtype, device="cuda")
        else:
            rows, slots = case["batch"], case["batch"] + 2
            s["slots"] = torch.randperm(slots, generator=g, device="cuda")[:rows].to(torch.int32)
        xbc = _silu_rows(g, rows, h * P + 2 * gr * N, dtype)  # the convolution's rows, read in place
        s["x"] = xbc[:, :h * P].unflatten(1, (h, P))
        s["B"] = xbc[:, h * P:h * P + gr * N].unflatten(1, (gr, N))
        s["C"] = xbc[:, h * P + gr * N:].unflatten(1, (gr, N))
        s["dt"] = (torch.randn(rows, h, generator=g, device="cuda") * 0.1).to(dtype)
        s["states"] = torch.randn(slots, h, P, N, generator=g, device="cuda") * 0.01  # the magnitude that these inputs lead to
        return s
    rows, d = case["rows"], case["width"]
    s.update(groups=case["groups"], gate_first=case["gate_first"], eps=1e-5)
    s["x"] = (torch.randn(rows, d, generator=g, device="cuda") * 2).to(dtype)
    s["z"] = _rows(g, rows, d, d + 320, case["sliced"], dtype)
    s["weight"] = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    if op == "norm_bwd":
        s["dout"] = torch.randn(rows, d, generator=g, device="cuda").to(dtype)
    return s


def run(s):
    if own:
        return _run_own(s)
    return {"conv": _conv, "conv_bwd": _conv_bwd, "conv_step": _conv_step, "ssd": _ssd, "step": _step, "norm": _norm, "norm_bwd": _norm_bwd}[s["op"]](s)


def _run_own(s):
    import selective_state_space_38_b200 as ssm
    op = s["op"]
    if op == "conv":
        y = ssm.ssm_conv1d_fwd(s["x"], s["w"], s["bias"], s["cu"], windows=s["windows"], slots=s["slots"], has_initial=s["has_initial"], out=s["out"])
        return y, s["windows"]
    if op == "conv_bwd":
        return ssm.ssm_conv1d_bwd(s["x"], s["w"], s["bias"], s["cu"], s["dy"], dx=s["dx"])
    if op == "conv_step":
        return ssm.ssm_conv1d_step(s["windows"], s["x"], s["w"], s["bias"], slots=s["slots"]), s["windows"]
    if op == "ssd":
        y = ssm.ssm_ssd_varlen_fwd(s["x"], s["dt"], s["dt_bias"], True, s["A"], s["B"], s["C"], s["D"], s["cu"], states=s["states"], slots=s["slots"],
                                   has_initial=s["has_initial"], out=s["out"])
        return y, s["states"]
    if op == "step":
        return ssm.ssm_ssd_step(s["states"], s["x"], s["dt"], s["dt_bias"], True, s["A"], s["B"], s["C"], s["D"], slots=s["slots"]), s["states"]
    if op == "norm":
        out, rstd = ssm.ssm_gated_norm_fwd(s["x"], s["weight"], s["z"], groups=s["groups"], eps=s["eps"], gate_first=s["gate_first"])
        return out, rstd
    return ssm.ssm_gated_norm_bwd(s["x"], s["weight"], s["z"], s["dout"], groups=s["groups"], eps=s["eps"], gate_first=s["gate_first"])


# ---- plain forms: elementary torch operations in 32 bits ----------------------------

def _silu(v):
    return v * torch.sigmoid(v)


def _token_sequences(s):
    """Of each token: its sequence, its place in it, and whether it is in one."""
    t = torch.arange(s["tokens"], device="cuda")
    cu = s["cu"].long()
    n = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    valid = n < len(s["lens"])
    n = n.clamp(max=len(s["lens"]) - 1)
    return n, t - cu[n], valid


def _taps(s, windows, has_initial):
    """[tokens, K, dim]: the K inputs of each token's convolution, oldest first."""
    n, at, valid = _token_sequences(s)
    back = torch.arange(K - 1, -1, -1, device="cuda")
    t = torch.arange(s["tokens"], device="cuda")
    src = t[:, None] - back
    pos = at[:, None] - back  # before the sequence's start: the window's places K - 1 + pos
    x = s["x"].float()
    taps = torch.where((pos >= 0)[..., None], x[src.clamp(min=0)], 0.0)
    if windows is not None and has_initial is not None:
        early = ((pos < 0) & (has_initial[n] & valid)[:, None]).nonzero()
        rows = s["slots"].long()[n[early[:, 0]]]
        taps[early[:, 0], early[:, 1]] = windows.float()[rows, K - 1 + pos[early[:, 0], early[:, 1]]]
    return taps, n, at, valid


def _conv(s):
    taps, n, at, valid = _taps(s, s["windows"], s["has_initial"])
    u = (taps * s["w"].t()).sum(1) + s["bias"]
    s["out"][valid] = _silu(u)[valid].to(s["out"].dtype)
    last = (valid & (at == s["cu"].diff().long()[n] - 1)).nonzero()[:, 0]
    s["windows"][s["slots"].long()[n[last]]] = taps[last, 1:].to(s["windows"].dtype)
    return s["out"], s["windows"]


def _conv_bwd(s):
    taps, n, at, valid = _taps(s, None, None)
    u = (taps * s["w"].t()).sum(1) + s["bias"]
    sg = torch.sigmoid(u)
    gr = torch.where(valid[:, None], s["dy"].float() * sg * (1 + u * (1 - sg)), 0.0)
    ahead = torch.arange(K - 1, -1, -1, device="cuda")
    t = torch.arange(s["tokens"], device="cuda")[:, None] + ahead  # tap k of token t + K - 1 - k is token t
    inside = valid[:, None] & (at[:, None] + ahead < s["cu"].diff().long()[n][:, None])
    later = torch.where(inside[..., None], gr[t.clamp(max=s["tokens"] - 1)], 0.0)
    s["dx"][valid] = (later * s["w"].t()).sum(1)[valid].to(s["dx"].dtype)
    dw = (gr[:, None].double() * taps).sum(0).t().float()
    return dict(dx=s["dx"], dw=dw, dbias=gr.double().sum(0).float())


def _conv_step(s):
    rows = s["slots"].long()
    taps = torch.cat([s["windows"][rows], s["x"][:, None]], 1)
    y = _silu((taps.float() * s["w"].t()).sum(1) + s["bias"])
    s["windows"][rows] = taps[:, 1:]
    return y.to(s["x"].dtype), s["windows"]


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(v.clamp(max=20))))


def _ssd(s, Q=128):
    """The chunked (semiseparable) form on the sequences padded to one length."""
    lens, cu = s["lens"], s["cu"].long()
    S, nc = len(lens), -(-max(lens) // Q)
    H, G = s["x"].shape[1], s["B"].shape[1]
    per = H // G
    l = torch.arange(nc * Q, device="cuda")
    inside = l < cu.diff()[:, None]
    idx = torch.where(inside, cu[:-1, None] + l, 0)
    shape = (S, nc, Q)
    x = torch.where(inside[..., None, None], s["x"][idx].float(), 0.0).reshape(*shape, H, P)
    Bm = torch.where(inside[..., None, None], s["B"][idx].float(), 0.0).reshape(*shape, G, N)
    Cm = torch.where(inside[..., None, None], s["C"][idx].float(), 0.0).reshape(*shape, G, N)
    dt = torch.where(inside[..., None], _softplus(s["dt"][idx].float() + s["dt_bias"]), 0.0).reshape(*shape, H)
    cs = (dt.double() * s["A"].double()).cumsum(2).permute(0, 1, 3, 2)  # [S, nc, H, Q], in 64 bits: far steps' differences
    dth = dt.permute(0, 1, 3, 2)
    xh = x.permute(0, 1, 3, 2, 4) * dth[..., None]  # [S, nc, H, Q, P]
    Bh, Ch = (v.permute(0, 1, 3, 2, 4).repeat_interleave(per, 2) for v in (Bm, Cm))
    scores = (Cm.permute(0, 1, 3, 2, 4) @ Bm.permute(0, 1, 3, 4, 2)).repeat_interleave(per, 2)
    seen = torch.ones(Q, Q, dtype=torch.bool, device="cuda").tril()
    scores = scores * torch.exp((cs[..., :, None] - cs[..., None, :]).masked_fill(~seen, -math.inf)).float()
    y = scores @ xh
    del scores
    own_states = (xh * torch.exp(cs[..., -1:] - cs).float()[..., None]).transpose(-1, -2) @ Bh  # [S, nc, H, P, N]
    total = cs[..., -1].cumsum(1).permute(0, 2, 1)  # [S, H, nc]
    ends = torch.cat([torch.zeros_like(total[..., :1]), total], -1)  # up to the start of each chunk, and to the end
    reach = torch.ones(nc + 1, nc, dtype=torch.bool, device="cuda").tril(-1)
    decay = torch.exp((ends[..., :, None] - total[..., None, :]).masked_fill(~reach, -math.inf)).float()
    start = s["states"][s["slots"].long()]
    start = torch.where(s["has_initial"][:, None, None, None], start, 0.0) if s["has_initial"] is not None else torch.zeros_like(start)
    at = decay @ own_states.permute(0, 2, 1, 3, 4).reshape(S, H, nc, P * N) + torch.exp(ends).float()[..., None] * start.reshape(S, H, 1, P * N)
    at = at.reshape(S, H, nc + 1, P, N)
    y = y + torch.exp(cs).float()[..., None] * (Ch @ at[:, :, :-1].permute(0, 2, 1, 4, 3))
    y = y.permute(0, 1, 3, 2, 4) + s["D"][:, None] * x
    s["out"][idx[inside]] = y.reshape(S, nc * Q, H, P)[inside].to(s["out"].dtype)
    some = (cu.diff() > 0).nonzero()[:, 0]
    s["states"][s["slots"].long()[some]] = at[some, :, -1]
    return s["out"], s["states"]


def _step(s):
    rows = s["slots"].long()
    per = s["x"].shape[1] // s["B"].shape[1]
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    x = s["x"].float()
    Bh, Ch = (v.float().repeat_interleave(per, 1) for v in (s["B"], s["C"]))
    st = s["states"][rows]
    st = st * torch.exp(dt * s["A"])[..., None, None] + (dt[..., None] * x)[..., None] * Bh[:, :, None]
    y = (st * Ch[:, :, None]).sum(-1) + s["D"][:, None] * x
    s["states"][rows] = st
    return y.to(s["x"].dtype), s["states"]


def _grouped(v, groups):
    return v.float().unflatten(1, (groups, -1))


def _norm(s):
    x, z, w = _grouped(s["x"], s["groups"]), _grouped(s["z"], s["groups"]), s["weight"].reshape(s["groups"], -1)
    v = x * _silu(z) if s["gate_first"] else x
    rstd = torch.rsqrt((v * v).mean(-1) + s["eps"])
    out = v * rstd[..., None] * w
    out = out if s["gate_first"] else out * _silu(z)
    return out.flatten(1).to(s["x"].dtype), rstd


def _norm_bwd(s):
    x, z, dout = (_grouped(s[k], s["groups"]) for k in ("x", "z", "dout"))
    w = s["weight"].reshape(s["groups"], -1)
    sg = torch.sigmoid(z)
    gate, dgate = z * sg, sg * (1 + z * (1 - sg))
    v = x * gate if s["gate_first"] else x
    rstd = torch.rsqrt((v * v).mean(-1, keepdim=True) + s["eps"])
    unit = v * rstd
    up = dout if s["gate_first"] else dout * gate
    dw = (up * unit).double().sum(0).float().flatten()
    dn = up * w
    dv = rstd * (dn - unit * (dn * unit).mean(-1, keepdim=True))
    dx, dz = (dv * gate, dv * x * dgate) if s["gate_first"] else (dv, dout * unit * w * dgate)
    return dict(dx=dx.flatten(1).to(s["x"].dtype), dz=dz.flatten(1).to(s["x"].dtype), dweight=dw)


# ---- what a pass cannot do without -------------------------------------------------

def work(case):
    op = case["op"]
    es = 2 if case.get("bf16", True) else 4
    if op in ("conv", "conv_bwd", "conv_step"):
        dim = case["width"] + 2 * case["groups"] * N
        par = dim * (K + 1) * 4
        if op == "conv_step":
            t = case["batch"]
            return dict(bytes=t * dim * es * (2 + 2 * (K - 1)) + par, flops=t * dim * (2 * K + 5))
        t = sum(_lengths(case))
        if op == "conv":
            return dict(bytes=2 * t * dim * es + par + len(_lengths(case)) * (K - 1) * dim * es, flops=t * dim * (2 * K + 5))
        return dict(bytes=3 * t * dim * es + 2 * par, flops=t * dim * (6 * K + 12))
    if op in ("ssd", "step"):
        h, g = case["heads"], case["groups"]
        per_token = 2 * h * P * es + h * es + 2 * g * N * es
        state = h * P * N * 4
        if op == "step":
            return dict(bytes=case["batch"] * (per_token + 2 * state), flops=case["batch"] * h * P * N * 5)
        lens = _lengths(case)
        t = sum(lens)
        read = 0.5 if case["initial"] else 0.0  # about half of the sequences go on from a state
        # the chunked form: C B^T once per group, then its product with x, C S and the state's update per head
        return dict(bytes=t * per_token + len(lens) * state * (1 + read), flops=t * (2 * 128 * N * g + h * (2 * 128 * P + 4 * P * N)))
    t, d = case["rows"], case["width"]
    if op == "norm":
        return dict(bytes=3 * t * d * es + d * 4 + t * case["groups"] * 4, flops=t * d * 12)
    return dict(bytes=5 * t * d * es + 2 * d * 4, flops=t * d * 30)


# ---- the definitions in 64 bits ------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "conv_bwd": _exact_conv_bwd, "conv_step": _exact_conv_step, "ssd": _exact_ssd, "step": _exact_step, "norm": _exact_norm,
            "norm_bwd": _exact_norm_bwd}[s["op"]](s)


def _one_conv(x, w, bias, before):
    """silu of the convolution of one sequence [len, dim] after `before` [K - 1, dim]."""
    full = torch.cat([before, x])
    u = bias + sum(full[k:k + len(x)] * w[:, k] for k in range(K))
    return torch.nn.functional.silu(u), full[len(x):]


def _exact_conv(s):
    y, win = s["out"].double(), s["windows"].double()
    x, w, b = s["x"].double(), s["w"].double(), s["bias"].double()
    at = 0
    for n, ln in enumerate(s["lens"]):
        slot = int(s["slots"][n])
        if ln:
            start = win[slot].clone() if s["has_initial"] is not None and bool(s["has_initial"][n]) else torch.zeros_like(win[slot])
            y[at:at + ln], win[slot] = _one_conv(x[at:at + ln], w, b, start)
        at += ln
    return y, win


def _exact_conv_bwd(s):
    x, w, b = (s[k].double().requires_grad_() for k in ("x", "w", "bias"))
    at, loss = 0, 0.0
    for ln in s["lens"]:
        if ln:
            y, _ = _one_conv(x[at:at + ln], w, b, torch.zeros(K - 1, x.shape[1], dtype=torch.float64, device="cuda"))
            loss = loss + (y * s["dy"][at:at + ln].double()).sum()
        at += ln
    dx, dw, db = torch.autograd.grad(loss, (x, w, b))
    return dict(dx=dx, dw=dw, dbias=db)


def _exact_conv_step(s):
    win, x = s["windows"].double(), s["x"].double()
    rows = s["slots"].long()
    ys = s["bias"].double() + x * s["w"][:, K - 1].double()
    for k in range(K - 1):
        ys = ys + win[rows, k] * s["w"][:, k].double()
    new = win.clone()
    for k in range(K - 2):
        new[rows, k] = win[rows, k + 1]
    new[rows, K - 2] = x
    return torch.nn.functional.silu(ys), new


def _recur(st, x, dt, A, B, C, D):
    """One token of every sequence by the recurrence: the new state and y."""
    a = torch.exp(dt * A)
    st = a[..., None, None] * st + (dt[..., None] * x)[..., :, None] * B[..., None, :]
    return st, torch.matmul(st, C[..., None])[..., 0] + D[:, None] * x


def _exact_ssd(s):
    lens, H = s["lens"], s["x"].shape[1]
    per = H // s["B"].shape[1]
    if max(lens) * sum(v > 0 for v in lens) * H > 60_000_000:
        return None
    order = sorted((n for n in range(len(lens)) if lens[n]), key=lambda n: -lens[n])
    y, states = s["out"].double(), s["states"].double()
    A, D, bias = s["A"].double(), s["D"].double(), s["dt_bias"].double()
    rows = s["slots"].long()[torch.tensor(order, device="cuda")]
    begin = s["cu"].long()[:-1][torch.tensor(order, device="cuda")]
    st = states[rows]
    if s["has_initial"] is None:
        st = torch.zeros_like(st)
    else:
        st[~s["has_initial"][torch.tensor(order, device="cuda")]] = 0
    x, B, C = s["x"], s["B"], s["C"]
    dt = torch.nn.functional.softplus(s["dt"].double() + bias)
    live = len(order)
    for l in range(lens[order[0]]):
        while lens[order[live - 1]] <= l:
            live -= 1
        t = begin[:live] + l
        st[:live], y[t] = _recur(st[:live], x[t].double(), dt[t], A, B[t].double().repeat_interleave(per, 1), C[t].double().repeat_interleave(per, 1), D)
    states[rows] = st
    return y, states


def _exact_step(s):
    per = s["x"].shape[1] // s["B"].shape[1]
    states, rows = s["states"].double(), s["slots"].long()
    dt = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double())
    states[rows], y = _recur(states[rows], s["x"].double(), dt, s["A"].double(), s["B"].double().repeat_interleave(per, 1),
                             s["C"].double().repeat_interleave(per, 1), s["D"].double())
    return y, states


def _norm_of(s, x, z, w):
    """The gated norm in 64 bits, and the reciprocal root mean square of each group."""
    rows = x.shape[0]
    gate = torch.nn.functional.silu(z)
    v = (x * gate if s["gate_first"] else x).reshape(rows, s["groups"], -1)
    rms = torch.sqrt(v.square().sum(-1) / v.shape[-1] + s["eps"])
    out = (v / rms[..., None]).reshape(rows, -1) * w
    return (out if s["gate_first"] else out * gate), 1 / rms


def _exact_norm(s):
    return _norm_of(s, s["x"].double(), s["z"].double(), s["weight"].double())


def _exact_norm_bwd(s):
    x, z, w = (s[k].double().requires_grad_() for k in ("x", "z", "weight"))
    out, _ = _norm_of(s, x, z, w)
    dx, dz, dw = torch.autograd.grad(out, (x, z, w), s["dout"].double())
    return dict(dx=dx, dz=dz, dweight=dw)
