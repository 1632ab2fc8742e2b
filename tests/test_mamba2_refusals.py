"""Refusals of the operators around the Mamba-2 SSD: bad arguments return a code
(from C) or raise (from Python) before anything is launched.  No GPU needed: the
pointers are never used."""
import ctypes

import pytest
import torch

import mamba2_ref as ref


def _p(i):
    return ctypes.c_void_p(0x10000000 + i * 0x1000000)


def _at(i, off):
    return ctypes.c_void_p(0x10000000 + i * 0x1000000 + off)


@pytest.fixture(scope="module")
def m():
    import selective_state_space_38_b200 as m
    m.get_lib()
    return m


def _conv_dims(m, **over):
    d = dict(tokens=64, dim=128, sequences=2, slots=4, x_stride=128, y_stride=128, dy_stride=128, dx_stride=128, width=4,
             silu=1, act_dtype=1)
    d.update(over)
    return ctypes.byref(m.Conv1dDims(**d))


def test_conv1d_fwd(m):
    def call(**o):
        a = dict(x=_p(1), w=_p(2), b=None, cu=_p(3), win=_p(4), slots=_p(5), init=_p(6), y=_p(7), dims=_conv_dims(m))
        a.update(o)
        return m.get_lib().ssm_conv1d_fwd(a["x"], a["w"], a["b"], a["cu"], a["win"], a["slots"], a["init"], a["y"], a["dims"], None)
    for k in ("x", "w", "cu", "y", "dims"):
        assert call(**{k: None}) == 1, k
    for bad in (dict(tokens=0), dict(dim=0), dict(sequences=0), dict(slots=-1), dict(x_stride=127), dict(y_stride=100)):
        assert call(dims=_conv_dims(m, **bad)) == 1, bad
    for bad in (dict(width=0), dict(width=5), dict(act_dtype=2), dict(tokens=1 << 31), dict(sequences=1 << 31)):
        assert call(dims=_conv_dims(m, **bad)) == 2, bad
    assert call(x=_at(1, 1)) == 3 and call(y=_at(7, 1)) == 3 and call(win=_at(4, 1)) == 3
    assert call(w=_at(2, 2)) == 3 and call(cu=_at(3, 2)) == 3 and call(slots=_at(5, 1)) == 3
    assert call(y=_p(1)) == 1                      # y over x
    assert call(y=_p(4)) == 1                      # y over the windows
    assert call(win=_at(1, 64)) == 1               # windows over x
    assert call(y=_at(1, 128), dims=_conv_dims(m, x_stride=192, y_stride=192)) == 1   # rows that meet


def test_conv1d_step(m):
    def call(**o):
        a = dict(win=_p(4), slots=_p(5), x=_p(1), w=_p(2), b=None, y=_p(7), dims=_conv_dims(m, tokens=4))
        a.update(o)
        return m.get_lib().ssm_conv1d_step(a["win"], a["slots"], a["x"], a["w"], a["b"], a["y"], a["dims"], None)
    for k in ("win", "x", "w", "y", "dims"):
        assert call(**{k: None}) == 1, k
    assert call(slots=None, dims=_conv_dims(m, tokens=5)) == 1   # more rows than the cache has
    assert call(win=_p(1)) == 1 and call(y=_p(4)) == 1
    assert call(dims=_conv_dims(m, tokens=4, act_dtype=5)) == 2
    assert call(x=_at(1, 1)) == 3


def test_conv1d_bwd(m):
    lib = m.get_lib()
    n = ctypes.c_size_t(0)
    assert lib.ssm_conv1d_bwd_workspace_size(_conv_dims(m), ctypes.byref(n)) == 0 and n.value == 4 * 5 * 128 * 4  # four tiles of 16 rows
    assert lib.ssm_conv1d_bwd_workspace_size(None, ctypes.byref(n)) == 1
    assert lib.ssm_conv1d_bwd_workspace_size(_conv_dims(m, width=9), ctypes.byref(n)) == 2

    def call(**o):
        a = dict(x=_p(1), w=_p(2), b=_p(3), cu=_p(4), dy=_p(5), dx=_p(6), dw=_p(7), db=_p(8), ws=_p(9), wsb=n.value, dims=_conv_dims(m))
        a.update(o)
        return lib.ssm_conv1d_bwd(a["x"], a["w"], a["b"], a["cu"], a["dy"], a["dx"], a["dw"], a["db"], a["ws"], a["wsb"], a["dims"], None)
    for k in ("x", "w", "cu", "dy", "dx", "dw", "ws", "dims"):
        assert call(**{k: None}) == 1, k
    assert call(wsb=n.value - 1) == 1
    assert call(ws=_at(9, 8)) == 3 and call(dy=_at(5, 1)) == 3
    assert call(dx=_p(1)) == 1 and call(dw=_p(6)) == 1 and call(ws=_p(5)) == 1
    assert call(dims=_conv_dims(m, dy_stride=1)) == 1


def _ssd_dims(m, **over):
    d = dict(tokens=64, sequences=2, slots=4, heads=8, headdim=64, groups=2, dstate=128, x_stride=512, dt_stride=8, b_stride=256,
             c_stride=256, y_stride=512, act_dtype=1)
    d.update(over)
    return ctypes.byref(m.SsdPackedDims(**d))


BAD_SSD = [(dict(tokens=0), 1), (dict(heads=0), 1), (dict(groups=3), 1), (dict(slots=-1), 1), (dict(x_stride=511), 1),
           (dict(dt_stride=7), 1), (dict(b_stride=255), 1), (dict(c_stride=0), 1), (dict(y_stride=8), 1), (dict(headdim=32), 2),
           (dict(dstate=64), 2), (dict(act_dtype=3), 2), (dict(tokens=1 << 31), 2)]


def test_ssd_varlen(m):
    lib = m.get_lib()
    n = ctypes.c_size_t(0)
    assert lib.ssm_ssd_varlen_fwd_workspace_size(_ssd_dims(m), ctypes.byref(n)) == 0
    small = n.value
    assert lib.ssm_ssd_varlen_fwd_workspace_size(_ssd_dims(m, tokens=5000), ctypes.byref(n)) == 0
    assert n.value > 5 * 8 * 64 * 128 * 4          # one carried state per window of 1024 tokens and head
    assert lib.ssm_ssd_varlen_fwd_workspace_size(_ssd_dims(m, groups=3), ctypes.byref(n)) == 1

    def call(fn="ssm_ssd_varlen_fwd", **o):
        a = dict(x=_p(1), dt=_p(2), bias=None, sp=1, A=_p(3), B=_p(4), C=_p(5), D=None, cu=_p(6), st=None, slots=None, init=None,
                 y=_p(8), ws=_p(9), wsb=1 << 20, dims=_ssd_dims(m))
        a.update(o)
        args = [a[k] for k in ("x", "dt", "bias", "sp", "A", "B", "C", "D", "cu", "st", "slots", "init", "y", "ws", "wsb")]
        return lib.ssm_ssd_varlen_fwd(*args, a["dims"], None) if fn == "ssm_ssd_varlen_fwd" else lib.ssm_debug_ssd_varlen_flag_timeout(*args, 0, a["dims"], None)
    for fn in ("ssm_ssd_varlen_fwd", "ssm_debug_ssd_varlen_flag_timeout"):
        for k in ("x", "dt", "A", "B", "C", "cu", "y", "ws", "dims"):
            assert call(fn, **{k: None}) == 1, k
        for bad, code in BAD_SSD + [(dict(sequences=0), 1), (dict(act_dtype=0), 2), (dict(x_stride=516), 3), (dict(b_stride=260), 3),
                                    (dict(y_stride=513), 3)]:
            assert call(fn, dims=_ssd_dims(m, **bad)) == code, bad
        assert call(fn, wsb=small - 1) == 1
        for k, i in (("x", 1), ("B", 4), ("C", 5), ("y", 8), ("ws", 9)):
            assert call(fn, **{k: _at(i, 8)}) == 3, k
        assert call(fn, dt=_at(2, 1)) == 3 and call(fn, A=_at(3, 2)) == 3 and call(fn, cu=_at(6, 1)) == 3
        assert call(fn, y=_p(1)) == 1 and call(fn, st=_p(8)) == 1 and call(fn, ws=_p(4)) == 1


def test_ssd_step(m):
    def call(**o):
        a = dict(st=_p(10), slots=None, x=_p(1), dt=_p(2), bias=None, sp=1, A=_p(3), B=_p(4), C=_p(5), D=None, out=_p(8),
                 dims=_ssd_dims(m, tokens=4))
        a.update(o)
        return m.get_lib().ssm_ssd_step(a["st"], a["slots"], a["x"], a["dt"], a["bias"], a["sp"], a["A"], a["B"], a["C"], a["D"],
                                        a["out"], a["dims"], None)
    for k in ("st", "x", "dt", "A", "B", "C", "out", "dims"):
        assert call(**{k: None}) == 1, k
    for bad, code in BAD_SSD:
        assert call(dims=_ssd_dims(m, **dict(dict(tokens=4), **bad))) == code, bad
    assert call(dims=_ssd_dims(m, tokens=5)) == 1     # more rows than the cache has
    assert call(st=_at(10, 8)) == 3 and call(B=_at(4, 2)) == 3
    assert call(dims=_ssd_dims(m, tokens=4, c_stride=258)) == 3
    assert call(out=_p(10)) == 1 and call(out=_p(1)) == 1


def _norm_dims(m, **over):
    d = dict(rows=16, dim=256, groups=2, x_stride=256, z_stride=256, dout_stride=256, out_stride=256, dx_stride=256, dz_stride=256,
             eps=1e-5, gate_first=1, act_dtype=1)
    d.update(over)
    return ctypes.byref(m.NormDims(**d))


BAD_NORM = [(dict(rows=0), 1), (dict(dim=0), 1), (dict(groups=3), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(x_stride=255), 1),
            (dict(z_stride=1), 1), (dict(act_dtype=2), 2), (dict(dim=1 << 15, groups=1, x_stride=1 << 15, z_stride=1 << 15, out_stride=1 << 15), 2)]


def test_gated_norm(m):
    lib = m.get_lib()

    def fwd(**o):
        a = dict(x=_p(1), z=_p(2), w=_p(3), out=_p(4), r=_p(5), dims=_norm_dims(m))
        a.update(o)
        return lib.ssm_gated_norm_fwd(a["x"], a["z"], a["w"], a["out"], a["r"], a["dims"], None)
    for k in ("x", "w", "out", "dims"):
        assert fwd(**{k: None}) == 1, k
    for bad, code in BAD_NORM + [(dict(out_stride=1), 1)]:
        assert fwd(dims=_norm_dims(m, **bad)) == code, bad
    assert fwd(x=_at(1, 1)) == 3 and fwd(w=_at(3, 2)) == 3 and fwd(r=_at(5, 2)) == 3
    assert fwd(out=_p(1)) == 1 and fwd(out=_p(2)) == 1 and fwd(r=_p(4)) == 1

    n = ctypes.c_size_t(0)
    assert lib.ssm_gated_norm_bwd_workspace_size(_norm_dims(m), ctypes.byref(n)) == 0
    assert lib.ssm_gated_norm_bwd_workspace_size(_norm_dims(m, groups=3), ctypes.byref(ctypes.c_size_t(0))) == 1

    def bwd(**o):
        a = dict(x=_p(1), z=_p(2), w=_p(3), d=_p(4), dx=_p(5), dz=_p(6), dw=_p(7), ws=_p(8), wsb=n.value, dims=_norm_dims(m))
        a.update(o)
        return lib.ssm_gated_norm_bwd(a["x"], a["z"], a["w"], a["d"], a["dx"], a["dz"], a["dw"], a["ws"], a["wsb"], a["dims"], None)
    for k in ("x", "w", "d", "dx", "dz", "dw", "ws", "dims"):
        assert bwd(**{k: None}) == 1, k
    for bad, code in BAD_NORM[:-1] + [(dict(dout_stride=1), 1), (dict(dx_stride=1), 1), (dict(dz_stride=1), 1)]:
        assert bwd(dims=_norm_dims(m, **bad)) == code, bad
    assert bwd(wsb=n.value - 1) == 1
    assert bwd(dx=_p(1)) == 1 and bwd(dz=_p(5)) == 1 and bwd(ws=_p(4)) == 1
    assert bwd(d=_at(4, 1)) == 3 and bwd(ws=_at(8, 8)) == 3


def test_python_refuses_cpu_tensors_and_wrong_ranks(m):
    x = torch.zeros(4, 8)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        m.ssm_conv1d_fwd(x, torch.zeros(8, 4), None, cu)
    with pytest.raises(ValueError):
        m.ssm_conv1d_bwd(x, torch.zeros(8, 4), None, cu, x)
    with pytest.raises(ValueError):
        m.ssm_conv1d_step(torch.zeros(4, 3, 8), x, torch.zeros(8, 4), None)
    with pytest.raises(ValueError):
        m.ssm_gated_norm_fwd(x, torch.zeros(8))
    with pytest.raises(ValueError):
        m.ssm_gated_norm_bwd(x, torch.zeros(8), None, x)
    x3 = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        m.ssm_ssd_step(torch.zeros(4, 2, 64, 128), x3, torch.zeros(4, 2), None, True, torch.zeros(2), torch.zeros(4, 1, 128), torch.zeros(4, 1, 128))
    with pytest.raises(ValueError):
        m.ssm_ssd_varlen_fwd(x3, torch.zeros(4, 2), None, True, torch.zeros(2), torch.zeros(4, 1, 128), torch.zeros(4, 1, 128), None, cu)


def test_python_refuses_a_stream_of_another_device():
    from selective_state_space_38_b200.mamba2 import _on

    class Stream:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError):
        _on(torch.device("cuda", 0), Stream())


def test_workspace_sizes_of_more_than_the_operators_take(m):
    """Sizes whose products would leave 64 bits are refused before they are formed."""
    lib, n = m.get_lib(), ctypes.c_size_t(0)
    big = 1 << 62
    for query, make, fields in ((lib.ssm_conv1d_bwd_workspace_size, _conv_dims, ("tokens", "dim")),
                                (lib.ssm_ssd_varlen_fwd_workspace_size, _ssd_dims, ("tokens", "sequences", "heads")),
                                (lib.ssm_gated_norm_bwd_workspace_size, _norm_dims, ("rows", "dim"))):
        for k in fields:
            assert query(make(m, **{k: big}), ctypes.byref(n)) == 2, k


def test_row_strides(m):
    from selective_state_space_38_b200.mamba2 import _rows
    t = torch.zeros(6, 40)
    assert _rows(t, name="t")[1] == 40
    assert _rows(t[:, 8:24], name="t") == (t.data_ptr() + 32, 40)
    assert _rows(t[:, 8:24].unflatten(1, (2, 8)), name="t")[1] == 40
    assert _rows(t[:1].expand(1, 40), name="t")[1] == 40
    for bad in (t.t(), t[:, ::2], t[:1].expand(6, 40), torch.zeros(6, 2, 8).transpose(1, 2)):
        with pytest.raises(ValueError):
            _rows(bad, name="t")


def test_reference_convolution_and_ssd_agree_with_library_forms():
    """The float64 references themselves: the convolution against torch's, the SSD against its quadratic form."""
    g = ref.gen(0)
    x, w, b = ref.randn(g, 12, 5).double(), ref.randn(g, 5, 4).double(), ref.randn(g, 5).double()
    y, _, _ = ref.conv(x, w, b, [12], act=False)
    want = torch.nn.functional.conv1d(torch.nn.functional.pad(x.t()[None], (3, 0)), w[:, None], b, groups=5)[0].t()
    assert torch.allclose(y, want, atol=1e-12)
    inp = ref.ssd_inputs(g, 20, 2, 1, dtype=torch.float32)
    y, _ = ref.ssd(inp, [20])
    dt = ref.softplus(inp["dt"].double() + inp["dt_bias"].double())
    cs = (dt * inp["A"].double()).cumsum(0)
    L = torch.stack(
        [torch.exp(cs[:, None, h] - cs[None, :, h]).tril() for h in range(2)])
    G = inp["C"][:, 0].double() @ inp["B"][:, 0].double().t()
    q = torch.einsum("hij,ij,jh,jhp->ihp", L, G, dt, inp["x"].double()) + inp["D"].double()[:, None] * inp["x"].double()
    assert torch.allclose(y, q, atol=1e-9)
