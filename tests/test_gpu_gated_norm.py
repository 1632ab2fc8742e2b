"""GPU parity of the gated RMS norm and its gradients against float64."""
import pytest
import torch

import mamba2_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


def _case(seed, rows, dim, dtype, gate=True, scale=1.0):
    g = ref.gen(seed)
    return dict(x=ref.randn(g, rows, dim, dtype=dtype, scale=2 * scale), z=ref.randn(g, rows, dim, dtype=dtype) if gate else None,
                w=1 + 0.1 * ref.randn(g, dim), d=ref.randn(g, rows, dim, dtype=dtype))


def _cuda(v):
    return None if v is None else v.cuda()


def _f64(v):
    return None if v is None else v.double()


def _check(c, groups=1, eps=1e-5, gate_first=True, what="", **views):
    import selective_state_space_38_b200 as ssm
    dtype = c["x"].dtype
    x, z, w = _f64(c["x"]), _f64(c["z"]), c["w"].double()
    out, rstd = ssm.ssm_gated_norm_fwd(views.get("x", c["x"].cuda()), c["w"].cuda(), views.get("z", _cuda(c["z"])), groups=groups,
                                       eps=eps, gate_first=gate_first)
    ro, rr = ref.norm(x, w, z, groups, eps, gate_first)
    # v: silu's 2^-19; the mean of squares: twice that and a few additions; the rest single float32 steps
    rel = 2.0 ** -17
    ref.close(rstd, rr, rel * rr, f"{what} rstd")
    ref.close(out, ro, (rel + ref.half(dtype)) * ro.abs() + 1e-30, f"{what} out")

    r = ssm.ssm_gated_norm_bwd(views.get("x", c["x"].cuda()), c["w"].cuda(), views.get("z", _cuda(c["z"])), c["d"].cuda(),
                               groups=groups, eps=eps, gate_first=gate_first)
    leaves = [v.clone().requires_grad_() for v in ([x, w] if z is None else [x, w, z])]
    o, _ = ref.norm(leaves[0], leaves[1], leaves[2] if z is not None else None, groups, eps, gate_first)
    grads = torch.autograd.grad(o, leaves, c["d"].double())
    # magnitudes: dv = r (dn - n m(dn n)) with its two parts by their magnitudes
    rows = x.shape[0]
    s = torch.ones_like(x) if z is None else ref.silu(z)
    ds = torch.zeros_like(x) if z is None else (torch.sigmoid(z) * (1 + z * (1 - torch.sigmoid(z))))
    v = x * s if gate_first else x
    up = c["d"].double() if gate_first else c["d"].double() * s
    R = rr.repeat_interleave(x.shape[1] // groups, 1)
    n = v * R
    dn = (up * w).abs()
    m = (dn * n.abs()).reshape(rows, groups, -1).mean(-1).repeat_interleave(x.shape[1] // groups, 1)
    dv = R * (dn + n.abs() * m)
    ax = dv * s.abs() if gate_first else dv
    rel = 2.0 ** -15  # some ten relative errors of 2^-19 each
    ref.close(r["dx"], grads[0], rel * ax + ref.half(dtype) * grads[0].abs() + 1e-30, f"{what} dx")
    # a block adds up its rows one by one: fewer than 64 here, then the blocks' sums
    ref.close(r["dweight"], grads[1], rel * (up * n).abs().sum(0) + 1e-30, f"{what} dweight")
    if z is None:
        assert r["dz"] is None
    else:
        # silu' = sg (1 + z (1 - sg)) cancels near its zero: an absolute 2^-18 (1 + |z|)
        az = (dv * x.abs() if gate_first else (c["d"].double() * n * w).abs()) * (ds.abs() + 2.0 ** -2 * (1 + z.abs()))
        ref.close(r["dz"], grads[2], rel * az + ref.half(dtype) * grads[2].abs() + 1e-30, f"{what} dz")
    return out, r


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gate_first", [True, False])
@pytest.mark.parametrize("rows,dim,groups", [(1, 1, 1), (3, 8, 1), (5, 64, 1), (7, 264, 1), (4, 1536, 1), (6, 5120, 1),
                                             (9, 640, 8), (3, 1000, 5), (2, 77, 7), (5, 333, 1), (2, 4100, 1)])
def test_shapes(dtype, gate_first, rows, dim, groups):
    _check(_case(rows * 100 + dim, rows, dim, dtype), groups, gate_first=gate_first, what=f"{rows}x{dim}/{groups}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [16384, 9001])
def test_wide_rows(dtype, dim):
    _check(_case(dim, 2, dim, dtype), what=f"wide {dim}")


@pytest.mark.parametrize("dtype", DTYPES)
def test_without_gate_and_many_rows(dtype):
    _check(_case(1, 1300, 96, dtype, gate=False), what="no gate")
    _check(_case(2, 1300, 96, dtype), groups=3, what="many rows")


def test_rows_of_zeros_and_large_values():
    c = _case(3, 6, 128, torch.float32)
    c["x"][1] = 0.0
    c["z"][2] = 0.0
    c["z"][3] = -60.0   # silu and its derivative vanish
    c["z"][4] = 60.0
    c["x"][5] *= 1e4
    _check(c, eps=1e-5, what="extremes")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("start", [0, 8, 5])
def test_slices(dtype, start):
    """z as a slice of wider rows, aligned to 16 bytes and not."""
    c = _case(4, 9, 256, dtype)
    wide = torch.full((9, 272), 5.0, dtype=dtype, device="cuda")
    wide[:, start:start + 256] = c["z"].cuda()
    _check(c, z=wide[:, start:start + 256], what=f"slice {start}")


def test_gradients_into_slices_of_one_buffer():
    """dx and dz may be slices of the same wider rows."""
    import selective_state_space_38_b200 as ssm
    c = _case(5, 12, 128, torch.bfloat16)
    wide = torch.full((12, 264), 7.0, dtype=torch.bfloat16, device="cuda")
    args = (c["x"].cuda(), c["w"].cuda(), c["z"].cuda(), c["d"].cuda())
    a = ssm.ssm_gated_norm_bwd(*args)
    b = ssm.ssm_gated_norm_bwd(*args, dx=wide[:, :128], dz=wide[:, 128:256])
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dz"], b["dz"]) and torch.equal(a["dweight"], b["dweight"])
    assert (wide[:, 256:] == 7.0).all()


def test_gradients_against_differences():
    import selective_state_space_38_b200 as ssm
    c = _case(6, 10, 48, torch.float32)
    g = ref.gen(7)
    for gate_first in (True, False):
        r = ssm.ssm_gated_norm_bwd(c["x"].cuda(), c["w"].cuda(), c["z"].cuda(), c["d"].cuda(), groups=2, gate_first=gate_first)
        args = [c["x"].double(), c["z"].double(), c["w"].double()]

        def loss(x, z, w):
            return float((ref.norm(x, w, z, 2, 1e-5, gate_first)[0] * c["d"].double()).sum())
        for i, key in enumerate(("dx", "dz", "dweight")):
            v = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
            h = 1e-5
            up, dn = list(args), list(args)
            up[i], dn[i] = args[i] + h * v, args[i] - h * v
            want = (loss(*up) - loss(*dn)) / (2 * h)
            got = float((r[key].cpu().double() * v).sum())
            scale = float((r[key].cpu().double().abs() * v.abs()).sum())
            assert abs(got - want) <= 2.0 ** -15 * scale, (key, got, want)


def test_equal_calls_give_equal_bits_on_another_stream():
    import selective_state_space_38_b200 as ssm
    c = _case(8, 3000, 640, torch.bfloat16)
    args = [c[k].cuda() for k in ("x", "w", "z", "d")]
    a = ssm.ssm_gated_norm_bwd(*args, groups=5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = ssm.ssm_gated_norm_bwd(*args, groups=5, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], b[k]) for k in a)
