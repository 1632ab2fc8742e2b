"""Binding of the operators around the Mamba-2 SSD on packed sequences: the
time-major causal convolution (forward, gradients, one token), the packed SSD and
its decode step, and the gated norm with its gradients.

Tensors are rows of tokens: the columns of a row lie together, the rows may be
any stride apart, so a slice of a wider projection's rows needs no copy.  Results
and workspaces that a call allocates belong to the stream the call runs on.
"""
from __future__ import annotations

import ctypes

import torch

from . import SSM_BF16, SSM_F32, _act_code, _check, _ptr, get_lib

HEADDIM, DSTATE_SSD = 64, 128
_I64, _I32, _P, _S = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t


class Conv1dDims(ctypes.Structure):
    _fields_ = [("tokens", _I64), ("dim", _I64), ("sequences", _I64), ("slots", _I64), ("x_stride", _I64),
                ("y_stride", _I64), ("dy_stride", _I64), ("dx_stride", _I64), ("width", _I32), ("silu", _I32),
                ("act_dtype", _I32)]


class SsdPackedDims(ctypes.Structure):
    _fields_ = [("tokens", _I64), ("sequences", _I64), ("slots", _I64), ("heads", _I64), ("headdim", _I64),
                ("groups", _I64), ("dstate", _I64), ("x_stride", _I64), ("dt_stride", _I64), ("b_stride", _I64),
                ("c_stride", _I64), ("y_stride", _I64), ("act_dtype", _I32)]


class NormDims(ctypes.Structure):
    _fields_ = [("rows", _I64), ("dim", _I64), ("groups", _I64), ("x_stride", _I64), ("z_stride", _I64),
                ("dout_stride", _I64), ("out_stride", _I64), ("dx_stride", _I64), ("dz_stride", _I64),
                ("eps", ctypes.c_float), ("gate_first", _I32), ("act_dtype", _I32)]


def bind(lib):
    """Argument types of this module's entry points on the loaded library."""
    C, S, N = (ctypes.POINTER(t) for t in (Conv1dDims, SsdPackedDims, NormDims))
    size = ctypes.POINTER(_S)
    I = ctypes.c_int
    lib.ssm_conv1d_fwd.argtypes = [_P] * 8 + [C, _P]
    lib.ssm_conv1d_step.argtypes = [_P] * 6 + [C, _P]
    lib.ssm_conv1d_bwd_workspace_size.argtypes = [C, size]
    lib.ssm_conv1d_bwd.argtypes = [_P] * 9 + [_S, C, _P]
    lib.ssm_ssd_varlen_fwd_workspace_size.argtypes = [S, size]
    lib.ssm_ssd_varlen_fwd.argtypes = [_P, _P, _P, I] + [_P] * 10 + [_S, S, _P]
    lib.ssm_debug_ssd_varlen_flag_timeout.argtypes = [_P, _P, _P, I] + [_P] * 10 + [_S, ctypes.c_uint32, S, _P]
    lib.ssm_ssd_step.argtypes = [_P] * 5 + [I] + [_P] * 5 + [S, _P]
    lib.ssm_gated_norm_fwd.argtypes = [_P] * 5 + [N, _P]
    lib.ssm_gated_norm_bwd_workspace_size.argtypes = [N, size]
    lib.ssm_gated_norm_bwd.argtypes = [_P] * 8 + [_S, N, _P]
    for name in EXPORTS:
        getattr(lib, name).restype = I


EXPORTS = ("ssm_conv1d_fwd", "ssm_conv1d_step", "ssm_conv1d_bwd_workspace_size", "ssm_conv1d_bwd",
           "ssm_ssd_varlen_fwd_workspace_size", "ssm_ssd_varlen_fwd", "ssm_debug_ssd_varlen_flag_timeout",
           "ssm_ssd_step", "ssm_gated_norm_fwd", "ssm_gated_norm_bwd_workspace_size", "ssm_gated_norm_bwd")


def _rows(t, device=None, name="", dtype=None, shape=None):
    """(pointer, row stride) of a tensor whose rows' elements lie together."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    size, strides = t.shape, t.stride()
    if device is not None and t.get_device() != device.index:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and size != shape:
        raise ValueError(f"{name} has shape {tuple(size)}, expected {tuple(shape)}")
    if len(size) == 2:
        width = size[1]
        together = strides[1] == 1 or width == 1
    elif len(size) == 3:
        heads, each = size[1], size[2]
        width = heads * each
        together = (strides[2] == 1 or each == 1) and (strides[1] == each or heads == 1)
    else:
        raise ValueError(f"{name} must have two or three dimensions, got shape {tuple(size)}")
    if not together:
        raise ValueError(f"{name}: the elements of a row must lie together (strides {strides})")
    if size[0] <= 1:
        return t.data_ptr(), width
    if strides[0] < width:
        raise ValueError(f"{name}: rows overlap (strides {strides})")
    return t.data_ptr(), strides[0]


def _flat(t, dtype, device, shape, name):
    """Pointer of a contiguous tensor (None: no tensor); _ptr says what is wrong with others."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device.index and t.is_contiguous():
        return t.data_ptr()
    return _ptr(t, dtype=dtype, device=device, shape=shape, name=name)


def _like(t):
    """A new contiguous tensor of t's shape, type and device."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _cuda(x, rank, name):
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError("this operator needs CUDA tensors")
    if x.dim() != rank:
        raise ValueError(f"{name} must have {rank} dimensions, got shape {tuple(x.shape)}")
    if x.shape[0] < 1:
        raise ValueError(f"{name} has no rows")
    return x.device


def _size(t, i, rank, name):
    """t.shape[i] of a tensor that must have `rank` dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != rank:
        raise ValueError(f"{name} must have {rank} dimensions, got shape {tuple(t.shape)}")
    return t.shape[i]


class _on:
    """The device and the stream of a call; what is allocated meanwhile belongs to that stream."""
    __slots__ = ("device", "stream", "inside")

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        self.device, self.stream, self.inside = device, stream, ()

    def __enter__(self):
        index = self.device.index
        if index != torch._C._cuda_getDevice():
            self.inside += (torch.cuda.device(self.device),)
        if self.stream is not None:
            self.inside += (torch.cuda.stream(self.stream),)
        for c in self.inside:
            c.__enter__()
        return torch._C._cuda_getCurrentRawStream(index) if self.stream is None else self.stream.cuda_stream

    def __exit__(self, *error):
        for c in reversed(self.inside):
            c.__exit__(*error)


def _tables(cu_seqlens, slots, has_initial, device):
    """Pointers of the packed sequences' tables, and the number of sequences."""
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must be [sequences + 1]")
    n = cu_seqlens.shape[0] - 1
    pc = _flat(cu_seqlens, torch.int32, device, (n + 1,), "cu_seqlens")
    ps = _flat(slots, torch.int32, device, (n,), "slots")
    ph = _flat(has_initial, torch.uint8 if getattr(has_initial, "dtype", None) is torch.uint8 else torch.bool, device, (n,),
               "has_initial")
    return pc, ps, ph, n


def _workspace(query, dims, workspace, device):
    """(pointer, bytes, tensor) of the caller's workspace, or of one from torch's caching allocator."""
    if workspace is None:
        n = _S(0)
        _check(query(ctypes.byref(dims), ctypes.byref(n)))
        workspace = torch.empty(int(n.value), dtype=torch.uint8, device=device)
    return _ptr(workspace, dtype=torch.uint8, device=device, name="workspace"), workspace.numel(), workspace


def ssm_conv1d_fwd(x, conv_w, conv_bias, cu_seqlens, windows=None, slots=None, has_initial=None, silu=True,
                   out=None, stream=None):
    """Causal depthwise convolution (width conv_w.shape[1] <= 4) and silu over
    packed sequences.  x [tokens, dim] bfloat16 or float32; conv_w [dim, K] and
    conv_bias [dim] (or None) float32; cu_seqlens [n + 1] int32.  ``windows``
    [slots, K-1, dim] (x's dtype) holds inputs before a sequence, oldest first:
    read for the sequences that ``has_initial`` [n] (bool) marks, and left holding
    every sequence's last K-1 inputs; ``slots`` [n] int32 names the rows.  Returns
    out [tokens, dim]; rows outside the sequences are not written."""
    dev = _cuda(x, 2, "x")
    T, dim = x.shape
    act, f32 = x.dtype, torch.float32
    code = _act_code(x)
    K = _size(conv_w, 1, 2, "conv_w")
    px, xs = _rows(x, dev, "x")
    pw = _flat(conv_w, f32, dev, (dim, K), "conv_w")
    pb = _flat(conv_bias, f32, dev, (dim,), "conv_bias")
    pc, ps, ph, n = _tables(cu_seqlens, slots, has_initial, dev)
    nslots = 0
    if windows is not None:
        nslots = _size(windows, 0, 3, "windows")
    pwin = _flat(windows, act, dev, (nslots, K - 1, dim), "windows")
    with _on(dev, stream) as sp:
        if out is None:
            out = _like(x)
        po, os_ = _rows(out, dev, "out", act, (T, dim))
        dims = Conv1dDims(T, dim, n, nslots, xs, os_, 0, 0, K, int(bool(silu)), code)
        _check(get_lib().ssm_conv1d_fwd(px, pw, pb, pc, pwin if K > 1 else None, ps, ph, po, ctypes.byref(dims), sp))
    return out


def ssm_conv1d_step(windows, x, conv_w, conv_bias, slots=None, silu=True, out=None, stream=None):
    """One token per sequence through the convolution: x [batch, dim]; ``windows``
    [slots, K-1, dim] is read and moved on by one input in place; ``slots`` [batch]
    int32 (None: row b's is b).  Returns out [batch, dim]; a row whose slot is
    outside the cache is padding and is not written."""
    dev = _cuda(x, 2, "x")
    b, dim = x.shape
    act, f32 = x.dtype, torch.float32
    code = _act_code(x)
    K = _size(conv_w, 1, 2, "conv_w")
    px, xs = _rows(x, dev, "x")
    pw = _flat(conv_w, f32, dev, (dim, K), "conv_w")
    pb = _flat(conv_bias, f32, dev, (dim,), "conv_bias")
    ps = _flat(slots, torch.int32, dev, (b,), "slots")
    nslots = _size(windows, 0, 3, "windows") if windows is not None else b
    pwin = _flat(windows, act, dev, (nslots, K - 1, dim), "windows")
    with _on(dev, stream) as sp:
        if out is None:
            out = _like(x)
        po, os_ = _rows(out, dev, "out", act, (b, dim))
        dims = Conv1dDims(b, dim, 0, nslots, xs, os_, 0, 0, K, int(bool(silu)), code)
        _check(get_lib().ssm_conv1d_step(pwin if K > 1 else None, ps, px, pw, pb, po, ctypes.byref(dims), sp))
    return out


def ssm_conv1d_bwd(x, conv_w, conv_bias, cu_seqlens, dy, silu=True, dx=None, stream=None, workspace=None):
    """Gradients of ssm_conv1d_fwd on sequences that start from zeros.  Returns a
    dict: dx [tokens, dim] in x's dtype (rows outside the sequences are not
    written), dw [dim, K] and dbias [dim] (None without conv_bias) float32."""
    dev = _cuda(x, 2, "x")
    T, dim = x.shape
    act, f32 = x.dtype, torch.float32
    code = _act_code(x)
    K = _size(conv_w, 1, 2, "conv_w")
    px, xs = _rows(x, dev, "x")
    pw = _flat(conv_w, f32, dev, (dim, K), "conv_w")
    pb = _flat(conv_bias, f32, dev, (dim,), "conv_bias")
    pc, _, _, n = _tables(cu_seqlens, None, None, dev)
    pdy, dys = _rows(dy, dev, "dy", act, (T, dim))
    with _on(dev, stream) as sp:
        if dx is None:
            dx = _like(x)
        pdx, dxs = _rows(dx, dev, "dx", act, (T, dim))
        dw = _like(conv_w)
        dbias = _like(conv_bias) if conv_bias is not None else None
        dims = Conv1dDims(T, dim, n, 0, xs, 0, dys, dxs, K, int(bool(silu)), code)
        lib = get_lib()
        pws, nws, _keep = _workspace(lib.ssm_conv1d_bwd_workspace_size, dims, workspace, dev)
        _check(lib.ssm_conv1d_bwd(px, pw, pb, pc, pdy, pdx, dw.data_ptr(), None if dbias is None else dbias.data_ptr(),
                                  pws, nws, ctypes.byref(dims), sp))
    return dict(dx=dx, dw=dw, dbias=dbias)


def _ssd_args(x, dt, dt_bias, A, B, C, D, dev):
    """Pointers of the SSD's inputs and its sizes (slots, sequences and out's stride still open)."""
    T, H, P = x.shape
    act, f32 = x.dtype, torch.float32
    for t, name in ((B, "B"), (C, "C")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must be [rows, groups, {DSTATE_SSD}]")
    G, N = B.shape[1], B.shape[2]
    px, xs = _rows(x, dev, "x")
    pdt, dts = _rows(dt, dev, "dt", act, (T, H))
    pB, bs = _rows(B, dev, "B", act, (T, G, N))
    pC, cs = _rows(C, dev, "C", act, (T, G, N))
    pbias = _flat(dt_bias, f32, dev, (H,), "dt_bias")
    pA = _flat(A, f32, dev, (H,), "A")
    pD = _flat(D, f32, dev, (H,), "D")
    dims = SsdPackedDims(T, 0, 0, H, P, G, N, xs, dts, bs, cs, 0, _act_code(x))
    return px, pdt, pbias, pA, pB, pC, pD, dims


def ssm_ssd_varlen_fwd(x, dt, dt_bias, softplus, A, B, C, D, cu_seqlens, states=None, slots=None, has_initial=None,
                       out=None, stream=None, workspace=None, check=False):
    """Mamba-2 SSD over packed sequences on the tensor cores.  x [tokens, heads,
    64], dt [tokens, heads], B, C [tokens, groups, 128] bfloat16; A, dt_bias, D
    [heads] float32 (dt_bias and D may be None); cu_seqlens [n + 1] int32.
    ``states`` [slots, heads, 64, 128] float32 is read for the sequences that
    ``has_initial`` [n] (bool) marks and left holding every sequence's state;
    ``slots`` [n] int32 names the rows.  Returns out [tokens, heads, 64]; rows
    outside the sequences are not written.  ``check=True`` waits for the call
    and raises SSMError when cu_seqlens did not ascend within the tokens or a
    bounded device wait gave up."""
    dev = _cuda(x, 3, "x")
    px, pdt, pbias, pA, pB, pC, pD, dims = _ssd_args(x, dt, dt_bias, A, B, C, D, dev)
    pc, ps, ph, n = _tables(cu_seqlens, slots, has_initial, dev)
    dims.sequences = n
    dims.slots = _size(states, 0, 4, "states") if states is not None else 0
    pst = _flat(states, torch.float32, dev, (dims.slots, dims.heads, dims.headdim, dims.dstate), "states")
    lib = get_lib()
    with _on(dev, stream) as sp:
        if out is None:
            out = _like(x)
        po, dims.y_stride = _rows(out, dev, "out", x.dtype, x.shape)
        pws, nws, _keep = _workspace(lib.ssm_ssd_varlen_fwd_workspace_size, dims, workspace, dev)
        _check(lib.ssm_ssd_varlen_fwd(px, pdt, pbias, int(bool(softplus)), pA, pB, pC, pD, pc, pst, ps, ph, po, pws, nws,
                                      ctypes.byref(dims), sp))
        if check:
            _check(lib.ssm_scan_fwd_status(pws, sp))
    return out


def ssm_ssd_step(states, x, dt, dt_bias, softplus, A, B, C, D=None, slots=None, out=None, stream=None):
    """One decode step of the SSD: x [batch, heads, 64], dt [batch, heads], B, C
    [batch, groups, 128] (all bfloat16 or all float32); ``states`` [slots, heads,
    64, 128] float32 is updated in place; ``slots`` [batch] int32 (None: row b's is
    b).  Returns out [batch, heads, 64]; a row whose slot is outside the cache is
    padding and is not written."""
    dev = _cuda(x, 3, "x")
    px, pdt, pbias, pA, pB, pC, pD, dims = _ssd_args(x, dt, dt_bias, A, B, C, D, dev)
    dims.slots = _size(states, 0, 4, "states")
    pst = _flat(states, torch.float32, dev, (dims.slots, dims.heads, dims.headdim, dims.dstate), "states")
    ps = _flat(slots, torch.int32, dev, (x.shape[0],), "slots")
    with _on(dev, stream) as sp:
        if out is None:
            out = _like(x)
        po, dims.y_stride = _rows(out, dev, "out", x.dtype, x.shape)
        _check(get_lib().ssm_ssd_step(pst, ps, px, pdt, pbias, int(bool(softplus)), pA, pB, pC, pD, po,
                                      ctypes.byref(dims), sp))
    return out


def _norm_args(x, weight, z, groups, eps, gate_first):
    dev = _cuda(x, 2, "x")
    rows, dim = x.shape
    px, xs = _rows(x, dev, "x")
    pz, zs = _rows(z, dev, "z", x.dtype, x.shape)
    pw = _flat(weight, torch.float32, dev, (dim,), "weight")
    dims = NormDims(rows, dim, int(groups), xs, zs, 0, 0, 0, 0, float(eps), int(bool(gate_first)), _act_code(x))
    return dev, px, pz, pw, dims


def ssm_gated_norm_fwd(x, weight, z=None, groups=1, eps=1e-5, gate_first=True, out=None, stream=None):
    """RMS norm over each of ``groups`` equal parts of the rows of x [rows, dim]
    (bfloat16 or float32), fused with the gate silu(z): norm(x silu(z)) weight, or
    with ``gate_first=False`` norm(x) weight silu(z); no gate without z.  weight
    [dim] float32.  Returns (out [rows, dim], rstd [rows, groups] float32)."""
    dev, px, pz, pw, dims = _norm_args(x, weight, z, groups, eps, gate_first)
    with _on(dev, stream) as sp:
        if out is None:
            out = _like(x)
        po, dims.out_stride = _rows(out, dev, "out", x.dtype, x.shape)
        rstd = torch.empty((x.shape[0], max(int(groups), 1)), dtype=torch.float32, device=dev)
        _check(get_lib().ssm_gated_norm_fwd(px, pz, pw, po, rstd.data_ptr(), ctypes.byref(dims), sp))
    return out, rstd


def ssm_gated_norm_bwd(x, weight, z, dout, groups=1, eps=1e-5, gate_first=True, dx=None, dz=None, stream=None,
                       workspace=None):
    """Gradients of ssm_gated_norm_fwd given dout.  Returns a dict: dx and dz (None
    without z) in x's dtype, dweight [dim] float32."""
    dev, px, pz, pw, dims = _norm_args(x, weight, z, groups, eps, gate_first)
    pd, dims.dout_stride = _rows(dout, dev, "dout", x.dtype, x.shape)
    lib = get_lib()
    with _on(dev, stream) as sp:
        if dx is None:
            dx = _like(x)
        if z is None:
            dz = None
        elif dz is None:
            dz = _like(x)
        pdx, dims.dx_stride = _rows(dx, dev, "dx", x.dtype, x.shape)
        pdz, dims.dz_stride = _rows(dz, dev, "dz", x.dtype, x.shape)
        dweight = _like(weight)
        pws, nws, _keep = _workspace(lib.ssm_gated_norm_bwd_workspace_size, dims, workspace, dev)
        _check(lib.ssm_gated_norm_bwd(px, pz, pw, pd, pdx, pdz, dweight.data_ptr(), pws, nws, ctypes.byref(dims), sp))
    return dict(dx=dx, dz=dz, dweight=dweight)
