"""GPU parity of the time-major causal convolution on packed sequences, its
gradients and its single-token step, against float64 definitions."""
import pytest
import torch

import mamba2_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


def _cu(lens):
    return torch.tensor(ref.offsets(lens), dtype=torch.int32, device="cuda")


def _case(seed, lens, dim, K, dtype, pad=0, bias=True):
    g = ref.gen(seed)
    T = sum(lens) + pad
    n = len(lens)
    return dict(x=ref.randn(g, T, dim, dtype=dtype), w=ref.randn(g, dim, K, scale=0.5), b=ref.randn(g, dim, scale=0.2) if bias else None,
                windows=ref.randn(g, n + 2, K - 1, dim, dtype=dtype), slots=torch.randperm(n + 2, generator=g)[:n].to(torch.int32),
                initial=torch.rand(n, generator=g) < 0.5)


def _cuda(v):
    return None if v is None else v.cuda()


def _fwd_check(c, lens, act=True, x=None, what=""):
    import selective_state_space_38_b200 as ssm
    T, (dim, K), dtype = sum(lens), c["w"].shape, c["x"].dtype
    out = torch.full(tuple(c["x"].shape), 7.0, dtype=dtype, device="cuda")
    win = c["windows"].cuda()
    y = ssm.ssm_conv1d_fwd(c["x"].cuda() if x is None else x, c["w"].cuda(), _cuda(c["b"]), _cu(lens), windows=win,
                           slots=c["slots"].cuda(), has_initial=c["initial"].cuda(), silu=act, out=out)
    ry, rwin, s = ref.conv(c["x"], c["w"], c["b"], lens, c["windows"], c["slots"], c["initial"], act)
    assert (y[T:] == 7.0).all(), "rows behind the last sequence"
    ref.close(y[:T], ry[:T], ref.conv_tolerance(ry[:T], s[:T], K, dtype), f"{what} y")
    assert torch.equal(win.cpu().double(), rwin), f"{what} windows"
    return y


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("dim", [1, 24, 1032, 130])
def test_forward(dtype, K, dim):
    lens = [1, 40, 0, 2, 3, 100, 33]
    _fwd_check(_case(K * 1000 + dim, lens, dim, K, dtype, pad=6), lens, what=f"K={K} dim={dim}")


@pytest.mark.parametrize("lens", [[1], [31], [32], [33], [8, 8, 16, 32, 1], [0, 0, 5], [5, 0, 0], [1] * 70])
def test_forward_lengths(lens):
    _fwd_check(_case(len(lens), lens, 64, 4, torch.bfloat16, pad=1), lens, what=str(lens))


def test_forward_without_activation_bias_and_cache():
    import selective_state_space_38_b200 as ssm
    lens = [20, 50]
    c = _case(3, lens, 40, 4, torch.bfloat16, bias=False)
    _fwd_check(c, lens, act=False, what="identity")
    y = ssm.ssm_conv1d_fwd(c["x"].cuda(), c["w"].cuda(), None, _cu(lens))
    ry, _, s = ref.conv(c["x"], c["w"], None, lens)
    ref.close(y, ry, ref.conv_tolerance(ry, s, 4, torch.bfloat16), "no cache")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("start", [0, 8, 3])
def test_forward_slices(dtype, start):
    """A slice of wider rows: aligned to 16 bytes (start 0 and 8), and not."""
    lens = [40, 3, 60]
    c = _case(4, lens, 64, 4, dtype)
    wide = torch.full((sum(lens), 64 + 16), 5.0, dtype=dtype, device="cuda")
    wide[:, start:start + 64] = c["x"].cuda()
    a = _fwd_check(c, lens, x=wide[:, start:start + 64], what=f"slice {start}")
    assert torch.equal(a, _fwd_check(c, lens))


def test_forward_other_sequences_values_do_not_matter():
    import selective_state_space_38_b200 as ssm
    lens = [30, 20, 40]
    c = _case(5, lens, 48, 4, torch.bfloat16, pad=10)
    call = lambda x: ssm.ssm_conv1d_fwd(x.cuda(), c["w"].cuda(), c["b"].cuda(), _cu(lens))  # noqa: E731
    bad = c["x"].clone()
    bad[30:50], bad[90:] = float("nan"), float("inf")
    a, b = call(c["x"]), call(bad)
    assert torch.equal(a[:30], b[:30]) and torch.equal(a[50:90], b[50:90])


def test_tables_out_of_range_stay_in_bounds():
    """Tables that the host cannot see are clamped: wrong rows at most, and the buffers around stay as they were."""
    import selective_state_space_38_b200 as ssm
    c = _case(6, [64], 32, 4, torch.bfloat16)
    for table in ([-5, 30, 1000], [50, 20, 64], [64, 0, 0]):
        room = torch.full((64 + 64, 32), 7.0, dtype=torch.bfloat16, device="cuda")
        win = torch.full((2 + 2, 3, 32), 7.0, dtype=torch.bfloat16, device="cuda")
        ssm.ssm_conv1d_fwd(c["x"].cuda(), c["w"].cuda(), c["b"].cuda(), torch.tensor(table, dtype=torch.int32, device="cuda"),
                           windows=win[1:3], slots=torch.tensor([5, -3], dtype=torch.int32, device="cuda"),
                           has_initial=torch.tensor([True, True], device="cuda"), out=room[32:96])
        torch.cuda.synchronize()
        assert (room[:32] == 7.0).all() and (room[96:] == 7.0).all() and (win == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [1, 2, 4])
@pytest.mark.parametrize("dim", [1, 130, 1032])
def test_step(dtype, K, dim):
    import selective_state_space_38_b200 as ssm
    b = 5
    c = _case(K + dim, [1] * b, dim, K, dtype)
    slots = c["slots"].clone()
    slots[2] = -1  # a padded row
    win = c["windows"].cuda()
    out = torch.full((b, dim), 7.0, dtype=dtype, device="cuda")
    ssm.ssm_conv1d_step(win, c["x"].cuda(), c["w"].cuda(), c["b"].cuda(), slots=slots.cuda(), out=out)
    ry, rwin, s = ref.conv(c["x"], c["w"], c["b"], [1] * b, c["windows"], slots, [True] * b)
    rows = [0, 1, 3, 4]
    assert (out[2] == 7.0).all()
    tol = ref.conv_tolerance(ry, s, K, dtype)
    if K > 1:
        ref.close(out[rows], ry[rows], tol[rows], "step y")
        assert torch.equal(win.cpu().double(), rwin), "step windows"


def test_steps_equal_forward():
    """A prompt, then tokens one at a time, against one longer sequence."""
    import selective_state_space_38_b200 as ssm
    c = _case(9, [20], 72, 4, torch.float32)
    w, b = c["w"].cuda(), c["b"].cuda()
    win = torch.zeros(1, 3, 72, device="cuda")
    x = c["x"].cuda()
    ys = [ssm.ssm_conv1d_fwd(x[:2], w, b, _cu([2]), windows=win)]
    for t in range(2, 20):
        ys.append(ssm.ssm_conv1d_step(win, x[t:t + 1], w, b))
    ry, rwin, s = ref.conv(c["x"], c["w"], c["b"], [20], torch.zeros(1, 3, 72))
    ref.close(torch.cat(ys), ry, ref.conv_tolerance(ry, s, 4, torch.float32), "steps")
    assert torch.equal(win.cpu().double(), rwin)


def _grads(c, dy, lens, act=True):
    """Gradients by autograd of the float64 definition, and the sums of magnitudes that bound their rounding."""
    x, w = c["x"].double().requires_grad_(), c["w"].double().requires_grad_()
    b = (torch.zeros(x.shape[1]) if c["b"] is None else c["b"]).double().requires_grad_()
    K = w.shape[1]
    at, loss = ref.offsets(lens), 0.0
    for i, n in enumerate(lens):
        if n:
            y, _, _ = ref.conv_sequence(x[at[i]:at[i + 1]], w, b, torch.zeros(K - 1, x.shape[1], dtype=torch.float64), act)
            loss = loss + (y * dy[at[i]:at[i + 1]].double()).sum()
    return torch.autograd.grad(loss, (x, w, b))


def _bwd_check(c, lens, act=True, what="", **views):
    import selective_state_space_38_b200 as ssm
    (dim, K), dtype, T = c["w"].shape, c["x"].dtype, sum(lens)
    g = ref.gen(77)
    dy = ref.randn(g, *c["x"].shape, dtype=dtype)
    dx = torch.full(tuple(c["x"].shape), 7.0, dtype=dtype, device="cuda")
    r = ssm.ssm_conv1d_bwd(views.get("x", c["x"].cuda()), c["w"].cuda(), _cuda(c["b"]), _cu(lens), dy.cuda(), silu=act, dx=dx)
    gx, gw, gb = _grads(c, dy, lens, act)
    # g_t = dy silu'(u): |silu'| <= 1.1, |silu''| <= 0.5, u off by (K + 1) 2^-24 of its terms, silu' by 2^-18
    _, _, s = ref.conv(c["x"], c["w"], c["b"], lens)
    ga = 1.1 * dy.double().abs()
    ge = dy.double().abs() * (0.5 * (K + 1) * ref.H32 * s + 2.0 ** -18)
    ax, ex, aw, ew = torch.zeros_like(gx), torch.zeros_like(gx), torch.zeros_like(gw), torch.zeros_like(gw)
    w, x, at = c["w"].double().abs(), c["x"].double().abs(), ref.offsets(lens)
    for i in range(len(lens)):
        for k in range(K):
            d = K - 1 - k
            lo, hi = at[i], at[i + 1] - d
            if hi <= lo:
                continue
            ax[lo:hi] += w[:, k] * ga[lo + d:hi + d]
            ex[lo:hi] += w[:, k] * ge[lo + d:hi + d]
            aw[:, k] += (ga[lo + d:hi + d] * x[lo:hi]).sum(0)
            ew[:, k] += (ge[lo + d:hi + d] * x[lo:hi]).sum(0)
    assert (r["dx"][T:] == 7.0).all(), "rows behind the last sequence"
    ref.close(r["dx"][:T], gx[:T], (ex + K * ref.H32 * ax + ref.half(dtype) * gx.abs() + 1e-30)[:T], f"{what} dx")
    # sums of 128 rows in a row, then of the tiles: 160 steps of 2^-24 of the terms at most here
    ref.close(r["dw"], gw, ew + 160 * ref.H32 * aw + 1e-30, f"{what} dw")
    if c["b"] is not None:
        live = slice(0, T)
        ref.close(r["dbias"], gb, ge[live].sum(0) + 160 * ref.H32 * ga[live].sum(0) + 1e-30, f"{what} dbias")
    return r


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("dim", [1, 520, 130])
def test_gradients(dtype, K, dim):
    lens = [1, 125, 2, 0, 3, 200, 131]
    _bwd_check(_case(K * 10 + dim, lens, dim, K, dtype, pad=5), lens, what=f"K={K} dim={dim}")


@pytest.mark.parametrize("lens", [[1], [127], [128], [129], [126, 2, 2], [0, 3], [1] * 140])
def test_gradient_lengths(lens):
    _bwd_check(_case(8, lens, 64, 4, torch.bfloat16, pad=2), lens, what=str(lens))


def test_gradients_without_activation_and_bias():
    lens = [70, 90]
    _bwd_check(_case(10, lens, 32, 4, torch.float32, bias=False), lens, act=False, what="identity")


def test_gradients_ignore_other_rows_values():
    import selective_state_space_38_b200 as ssm
    lens = [60, 80]
    c = _case(11, lens, 64, 4, torch.bfloat16, pad=30)
    dy = ref.randn(ref.gen(12), 170, 64, dtype=torch.bfloat16)
    bad, bad_dy = c["x"].clone(), dy.clone()
    bad[140:], bad_dy[140:] = float("nan"), float("inf")
    call = lambda x, d: ssm.ssm_conv1d_bwd(x.cuda(), c["w"].cuda(), c["b"].cuda(), _cu(lens), d.cuda())  # noqa: E731
    a, b = call(c["x"], dy), call(bad, bad_dy)
    assert torch.equal(a["dx"][:140], b["dx"][:140]) and torch.equal(a["dw"], b["dw"]) and torch.equal(a["dbias"], b["dbias"])


def test_gradients_against_differences():
    """The gradients along random directions, against central differences of the float64 definition."""
    import selective_state_space_38_b200 as ssm
    lens = [50, 30]
    c = _case(13, lens, 16, 4, torch.float32)
    g = ref.gen(14)
    dy = ref.randn(g, 80, 16)
    r = ssm.ssm_conv1d_bwd(c["x"].cuda(), c["w"].cuda(), c["b"].cuda(), _cu(lens), dy.cuda())

    def loss(x, w, b):
        return float((ref.conv(x, w, b, lens)[0] * dy.double()).sum())
    args = [c["x"].double(), c["w"].double(), c["b"].double()]
    for i, key in enumerate(("dx", "dw", "dbias")):
        v = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + h * v, args[i] - h * v
        want = (loss(*up) - loss(*dn)) / (2 * h)
        got = float((r[key].cpu().double() * v).sum())
        # the difference quotient is good to about 1e-8 of the terms; float32 gradients to 2^-17 of theirs
        scale = float((r[key].cpu().double().abs() * v.abs()).sum())
        assert abs(got - want) <= 2.0 ** -17 * scale, (key, got, want)


def test_equal_calls_give_equal_bits():
    import selective_state_space_38_b200 as ssm
    lens = [700, 300]
    c = _case(15, lens, 264, 4, torch.bfloat16)
    dy = ref.randn(ref.gen(16), 1000, 264, dtype=torch.bfloat16).cuda()
    call = lambda **kw: ssm.ssm_conv1d_bwd(c["x"].cuda(), c["w"].cuda(), c["b"].cuda(), _cu(lens), dy, **kw)  # noqa: E731
    a = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = call(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], b[k]) for k in a)
