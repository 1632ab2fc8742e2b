"""The packed operators where the first sequence does not start at row 0: the rows in
front of it (a mixed batch's single tokens, say) belong to no sequence.  They are left as
they were, whatever they hold, and nothing of them reaches a sequence or a sum."""
import math

import pytest
import torch

import mamba2_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]
LENS = [3, 40, 0, 1, 90]


def _cu(front, lens):
    return torch.tensor([front + v for v in ref.offsets(lens)], dtype=torch.int32, device="cuda")


def _front(t, front, value):
    """t with `front` rows of a value before it, on the GPU."""
    return torch.cat([torch.full((front, *t.shape[1:]), value, dtype=t.dtype), t]).cuda()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K,dim", [(1, 24), (2, 130), (4, 24), (4, 1032)])
@pytest.mark.parametrize("front", [1, 10, 16, 21, 69])
def test_convolution(dtype, K, dim, front):
    import selective_state_space_38_b200 as ssm
    g = ref.gen(front * 100 + K)
    x, w, b = ref.randn(g, sum(LENS), dim, dtype=dtype), ref.randn(g, dim, K, scale=0.5), ref.randn(g, dim, scale=0.2)
    windows = ref.randn(g, len(LENS), K - 1, dim, dtype=dtype)
    initial = torch.tensor([True, False, True, True, False])
    win, out = windows.cuda(), torch.full((front + x.shape[0], dim), 7.0, dtype=dtype, device="cuda")
    ssm.ssm_conv1d_fwd(_front(x, front, math.nan), w.cuda(), b.cuda(), _cu(front, LENS), windows=win, has_initial=initial.cuda(), out=out)
    ry, rwin, s = ref.conv(x, w, b, LENS, windows, None, initial)
    assert (out[:front] == 7.0).all(), "rows in front"
    ref.close(out[front:], ry, ref.conv_tolerance(ry, s, K, dtype), "y")
    assert torch.equal(win.cpu().double(), rwin), "windows"


@pytest.mark.parametrize("front", [69, 5000])
def test_convolution_of_long_tiles(front):
    """Enough rows for the longest tiles, some of them whole in front of the sequence."""
    import selective_state_space_38_b200 as ssm
    g, n, dim = ref.gen(front), 9500, 2048
    x, w = ref.randn(g, n, dim, dtype=torch.bfloat16), ref.randn(g, dim, 4, scale=0.5)
    out = torch.full((front + n, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    ssm.ssm_conv1d_fwd(_front(x, front, math.inf), w.cuda(), None, _cu(front, [n]), out=out)
    ry, _, s = ref.conv(x, w, None, [n])
    assert (out[:front] == 7.0).all()
    ref.close(out[front:], ry, ref.conv_tolerance(ry, s, 4, torch.bfloat16), "y")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K,dim", [(1, 24), (2, 130), (4, 24), (4, 520)])
@pytest.mark.parametrize("front", [1, 10, 16, 21, 69])
def test_convolution_gradients(dtype, K, dim, front):
    import selective_state_space_38_b200 as ssm
    g, T, at = ref.gen(front * 10 + K), sum(LENS), ref.offsets(LENS)
    x, w, b = ref.randn(g, T, dim, dtype=dtype), ref.randn(g, dim, K, scale=0.5), ref.randn(g, dim, scale=0.2)
    dy = ref.randn(g, T, dim, dtype=dtype)
    dx = torch.full((front + T, dim), 7.0, dtype=dtype, device="cuda")
    r = ssm.ssm_conv1d_bwd(_front(x, front, math.nan), w.cuda(), b.cuda(), _cu(front, LENS), _front(dy, front, math.inf), dx=dx)
    x, w, b, dy = (v.double() for v in (x, w, b, dy))
    leaves = [v.clone().requires_grad_() for v in (x, w, b)]
    loss = sum((ref.conv_sequence(leaves[0][i:j], *leaves[1:], torch.zeros(K - 1, dim, dtype=torch.float64))[0] * dy[i:j]).sum()
               for i, j in zip(at, at[1:]))
    gx, gw, gb = torch.autograd.grad(loss, leaves)
    # g_t = dy silu'(u): |silu'| <= 1.1, |silu''| <= 0.5, u off by (K + 1) 2^-24 of its terms, silu' by 2^-18
    _, _, s = ref.conv(x, w, b, LENS)
    ga, ge = 1.1 * dy.abs(), dy.abs() * (0.5 * (K + 1) * ref.H32 * s + 2.0 ** -18)
    ax, ex, aw, ew = (torch.zeros_like(v) for v in (gx, gx, gw, gw))
    for i, j in zip(at, at[1:]):
        for k in range(K):
            d = K - 1 - k
            if j - d <= i:
                continue
            for a, e, sums in ((ga, ax, aw), (ge, ex, ew)):
                e[i:j - d] += w[:, k].abs() * a[i + d:j]
                sums[:, k] += (a[i + d:j] * x[i:j - d].abs()).sum(0)
    assert (r["dx"][:front] == 7.0).all(), "rows in front"
    ref.close(r["dx"][front:], gx, ex + K * ref.H32 * ax + ref.half(dtype) * gx.abs() + 1e-30, "dx")
    # at most all of the rows and as many tiles one after another
    steps = 2 * T
    ref.close(r["dw"], gw, ew + steps * ref.H32 * aw + 1e-30, "dw")
    ref.close(r["dbias"], gb, ge.sum(0) + steps * ref.H32 * ga.sum(0) + 1e-30, "dbias")


def test_everything_in_front():
    """No row is in a sequence: nothing is written but sums of nothing."""
    import selective_state_space_38_b200 as ssm
    x, w, b = torch.full((40, 24), math.nan, device="cuda"), torch.ones(24, 4, device="cuda"), torch.ones(24, device="cuda")
    out, win = torch.full_like(x, 7.0), torch.full((1, 3, 24), 7.0, device="cuda")
    cu = torch.tensor([40, 40], dtype=torch.int32, device="cuda")
    ssm.ssm_conv1d_fwd(x, w, b, cu, windows=win, out=out)
    assert (out == 7.0).all() and (win == 7.0).all()
    r = ssm.ssm_conv1d_bwd(x, w, b, cu, x, dx=out)
    assert (out == 7.0).all() and (r["dw"] == 0).all() and (r["dbias"] == 0).all()


@pytest.mark.parametrize("front", [1, 70, 300])
def test_ssd(front):
    """The same bits as without the rows in front."""
    import selective_state_space_38_b200 as ssm
    H = 4
    inp = ref.ssd_inputs(ref.gen(front), sum(LENS), H, 2)
    states = ref.randn(ref.gen(1), len(LENS), H, 64, 128)
    initial = torch.tensor([True, False, True, True, False], device="cuda")
    p = {k: v.cuda() for k, v in inp.items()}
    res = []
    for f in (0, front):
        d = {k: _front(inp[k], f, math.nan) for k in ("x", "dt", "B", "C")}
        st, out = states.cuda(), torch.full((f + sum(LENS), H, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        ssm.ssm_ssd_varlen_fwd(d["x"], d["dt"], p["dt_bias"], True, p["A"], d["B"], d["C"], p["D"], _cu(f, LENS), states=st,
                               has_initial=initial, out=out, check=True)
        assert (out[:f] == 7.0).all(), "rows in front"
        res.append((out[f:], st))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
