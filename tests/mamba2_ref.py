"""Plain float64 references of the operators around the Mamba-2 SSD, on the CPU,
from the definitions, with the error bounds that their GPU tests use.

Half a step of rounding is finfo.eps / 2 relative to the value: 2^-8 for bfloat16
(H16), 2^-24 for float32 (H32)."""
from __future__ import annotations

import math

import torch

H16, H32 = 2.0 ** -8, 2.0 ** -24
F64 = torch.float64


def half(dtype):
    return H16 if dtype == torch.bfloat16 else H32


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def offsets(lens):
    at = [0]
    for v in lens:
        at.append(at[-1] + v)
    return at


def silu(v):
    return v * torch.sigmoid(v)


def conv_sequence(x, w, b, before, act=True):
    """One sequence [len, dim] after `before` [K-1, dim]: (y, the window after it, sum of |terms|)."""
    K = w.shape[1]
    full = torch.cat([before, x])
    u, s = b.expand_as(x).clone(), b.abs().expand_as(x).clone()
    for k in range(K):
        u = u + full[k:k + x.shape[0]] * w[:, k]
        s = s + (full[k:k + x.shape[0]] * w[:, k]).abs()
    return (silu(u) if act else u), full[x.shape[0]:], s


def conv(x, w, b, lens, windows=None, slots=None, initial=None, act=True):
    """Packed convolution: (y [tokens, dim] with NaN behind the last sequence, windows after, bound of |terms|)."""
    x, w = x.to(F64), w.to(F64)
    b = torch.zeros(x.shape[1], dtype=F64) if b is None else b.to(F64)
    K = w.shape[1]
    y, s = torch.full_like(x, math.nan), torch.zeros_like(x)
    win = None if windows is None else windows.to(F64).clone()
    at = offsets(lens)
    for i, n in enumerate(lens):
        if n == 0:
            continue
        slot = i if slots is None else int(slots[i])
        ok = win is not None and 0 <= slot < win.shape[0]
        before = win[slot].clone() if ok and initial is not None and bool(initial[i]) else torch.zeros(K - 1, x.shape[1], dtype=F64)
        y[at[i]:at[i + 1]], after, s[at[i]:at[i + 1]] = conv_sequence(x[at[i]:at[i + 1]], w, b, before, act)
        if ok:
            win[slot] = after
    return y, win, s


def conv_tolerance(y, s, K, dtype):
    """K + 1 float32 steps into u (silu' is at most 1.1), silu to 2^-19 relative, one rounding of y."""
    return 1.1 * (K + 1) * H32 * s + (2.0 ** -19 + half(dtype)) * y.abs() + 1e-30


def softplus(v):
    return torch.nn.functional.softplus(v, threshold=60.0)


def ssd_sequence(x, dt, A, B, C, D, state):
    """The recurrence over one sequence in float64: x [L, H, P], dt [L, H] (after softplus), B, C [L, G, N],
    state [H, P, N].  Returns (y, state)."""
    per = x.shape[1] // B.shape[1]
    y = torch.empty_like(x)
    state = state.clone()
    for t in range(x.shape[0]):
        Bt, Ct = B[t].repeat_interleave(per, 0), C[t].repeat_interleave(per, 0)
        state = torch.exp(dt[t] * A)[:, None, None] * state + (dt[t][:, None] * x[t])[:, :, None] * Bt[:, None]
        y[t] = (state * Ct[:, None]).sum(-1) + D[:, None] * x[t]
    return y, state


def ssd(inp, lens, states=None, slots=None, initial=None, absolute=False):
    """Packed SSD: (y with NaN behind the last sequence, states).  absolute: every term by its magnitude, which
    bounds what the roundings of the terms can amount to."""
    f = (lambda v: v.to(F64).abs()) if absolute else (lambda v: v.to(F64))
    x, B, C = f(inp["x"]), f(inp["B"]), f(inp["C"])
    H = x.shape[1]
    A = inp["A"].to(F64)
    D = torch.zeros(H, dtype=F64) if inp.get("D") is None else f(inp["D"])
    v = inp["dt"].to(F64) + (0.0 if inp.get("dt_bias") is None else inp["dt_bias"].to(F64))
    dt = softplus(v) if inp.get("softplus", True) else (v.abs() if absolute else v)
    if absolute and not inp.get("softplus", True):
        raise ValueError("the bound needs steps of one sign")
    y = torch.full(tuple(x.shape), math.nan, dtype=F64)
    st = None if states is None else f(states).clone()
    at = offsets(lens)
    ends = {}
    for i, n in enumerate(lens):
        if n == 0:
            continue
        slot = i if slots is None else int(slots[i])
        ok = st is not None and 0 <= slot < st.shape[0]
        start = torch.zeros(H, x.shape[2], B.shape[2], dtype=F64)
        if ok and initial is not None and bool(initial[i]):
            start = st[slot].clone()
        rows = slice(at[i], at[i + 1])
        y[rows], end = ssd_sequence(x[rows], dt[rows], A, B[rows], C[rows], D, start)
        ends[i] = end
        if ok:
            st[slot] = end
    return y, st


def ssd_y_tolerance(y, y_abs, dtype=torch.bfloat16):
    """The triangle of C B^T is rounded to bf16 once where it meets x, the state once where it meets C: 2^-8 of
    each term; everything else is float32 or finer (2^-14 of the terms covers sums of 128 products in float32,
    384 accumulations, and the exponentials); one rounding of y."""
    return (H16 + 2.0 ** -14) * y_abs + half(dtype) * y.abs() + 1e-30


def ssd_state_tolerance(s_abs, chunks):
    """24 float32 accumulations of 16 products each per chunk, truncated (2^-22 of the terms), twice that for the
    factors and the scaling."""
    return 48 * 2.0 ** -22 * max(chunks, 1) * s_abs + 1e-30


def norm(x, w, z, groups, eps, gate_first):
    """(out, rstd) in float64."""
    rows = x.shape[0]
    s = torch.ones_like(x) if z is None else silu(z)
    v = (x * s if gate_first else x).reshape(rows, groups, -1)
    r = 1 / torch.sqrt(v.square().mean(-1) + eps)
    out = (v * r[..., None]).reshape(rows, -1) * w
    return (out if gate_first else out * s), r


def ssd_inputs(g, tokens, H, G, dtype=torch.bfloat16, dt_range=(1e-3, 1e-1), P=64, N=128):
    dt0 = torch.exp(torch.empty(H).uniform_(math.log(dt_range[0]), math.log(dt_range[1]), generator=g))
    return dict(x=randn(g, tokens, H, P, dtype=dtype), dt=randn(g, tokens, H, dtype=dtype, scale=0.1),
                dt_bias=torch.log(torch.expm1(dt0)), A=-torch.empty(H).uniform_(1.0, 16.0, generator=g),
                B=randn(g, tokens, G, N, dtype=dtype), C=randn(g, tokens, G, N, dtype=dtype), D=randn(g, H))


def close(got, ref, tol, what):
    got = got.detach().cpu().to(F64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: values that are not finite"
    err = (got - ref).abs()
    bad = err > tol
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance; first at {i}: got "
                             f"{float(got[i])!r}, expected {float(ref[i])!r}, off {float(err[i]):.3e}, allowed "
                             f"{float(torch.as_tensor(tol).expand_as(err)[i]):.3e}; worst ratio {float((err / tol).max()):.2f}")
    return float((err / tol).max()) if err.numel() else 0.0
