// mamba2.cu -- C ABI entry points of the operators around the Mamba-2 SSD on
// packed sequences: the time-major causal convolution, the packed SSD, its
// decode step and the gated norm.  Host-side validation and kernel launch, by
// the rules of ssm_scan.cu: every check before anything is enqueued.

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <type_traits>

#include "ssm_scan.h"
#include "host.h"
#include "conv1d.cuh"
#include "gated_norm.cuh"
#include "ssd_step.cuh"
#include "ssd_varlen.cuh"

namespace {

using namespace ssm;
using namespace ssm_host;

// `rows` rows of `width` bytes, `stride` bytes apart (an ordinary buffer is one row)
struct Rows {
    const void *p;
    int64_t rows, width, stride;
};

Rows flat(const void *p, int64_t bytes) { return Rows{p, 1, bytes, bytes}; }

// Whether two sets of rows share a byte.  Rows of the same stride may lie next to
// each other in one wider buffer (slices of a projection's rows).
bool overlap(const Rows &a, const Rows &b) {
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return false;
    const Span sa{a.p, static_cast<size_t>((a.rows - 1) * a.stride + a.width)};
    const Span sb{b.p, static_cast<size_t>((b.rows - 1) * b.stride + b.width)};
    if (!ssm_host::overlap(sa, sb)) return false;
    if (a.rows == 1 || b.rows == 1 || a.stride != b.stride) return true;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const int64_t s = a.stride;
    const int64_t off = pb >= pa ? static_cast<int64_t>((pb - pa) % s) : (s - static_cast<int64_t>((pa - pb) % s)) % s;
    return off < a.width || off + b.width > s;
}

template <size_t NI, size_t NO>
bool outputs_clash(const Rows (&ins)[NI], const Rows (&outs)[NO]) {
    for (size_t o = 0; o < NO; ++o) {
        for (const Rows &in : ins)
            if (overlap(outs[o], in)) return true;
        for (size_t q = o + 1; q < NO; ++q)
            if (overlap(outs[o], outs[q])) return true;
    }
    return false;
}

bool dtype_ok(int32_t t) { return t == SSM_F32 || t == SSM_BF16; }
bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// sizes whose byte offsets stay well inside int64
bool rows_ok(int64_t rows, int64_t stride) {
    return rows >= 0 && stride >= 0 && static_cast<double>(rows) * static_cast<double>(stride) < 4.0e18 / 16.0;
}

// ---- convolution ---------------------------------------------------------------------

// The checks that the three convolution entries share; on success fills `p`.
// vec: every row of every buffer allows 16-byte accesses.
int conv_setup(const void *x, const float *w, const float *bias, const ssm_conv1d_dims_t *d, Conv1dParams *p) {
    if (!d || !x || !w) return SSM_ERR_INVALID_ARG;
    if (d->tokens < 1 || d->dim < 1 || d->slots < 0) return SSM_ERR_INVALID_ARG;
    if (d->width < 1 || d->width > 4 || !dtype_ok(d->act_dtype)) return SSM_ERR_UNSUPPORTED;
    if (d->tokens > INT32_MAX || d->slots > INT32_MAX || d->dim > INT32_MAX) return SSM_ERR_UNSUPPORTED;
    if (d->x_stride < d->dim || !rows_ok(d->tokens, d->x_stride)) return SSM_ERR_INVALID_ARG;
    const size_t es = d->act_dtype == SSM_F32 ? 4 : 2;
    if (!aligned_to(x, es) || !aligned4(w) || !aligned4(bias)) return SSM_ERR_MISALIGNED;
    memset(p, 0, sizeof *p);
    p->x = x, p->w = w, p->bias = bias;
    p->dim = d->dim, p->x_stride = d->x_stride, p->silu = d->silu ? 1 : 0;
    p->seq.tokens = d->tokens, p->seq.nslots = static_cast<int32_t>(d->slots);
    return SSM_OK;
}

// The packed sequences of the forward pass and of the gradients (the step has none).
int conv_sequences(const int32_t *cu_seqlens, const ssm_conv1d_dims_t *d, Conv1dParams *p) {
    if (!cu_seqlens || d->sequences < 1) return SSM_ERR_INVALID_ARG;
    if (d->sequences > INT32_MAX) return SSM_ERR_UNSUPPORTED;
    if (!aligned4(cu_seqlens)) return SSM_ERR_MISALIGNED;
    p->seq.cu = cu_seqlens, p->seq.sequences = static_cast<int32_t>(d->sequences);
    return SSM_OK;
}

bool vector_rows(std::initializer_list<const void *> ptrs, std::initializer_list<int64_t> strides, int64_t dim,
                 int32_t act_dtype) {
    const int64_t v = act_dtype == SSM_F32 ? 4 : 8;
    bool ok = dim % v == 0;
    for (const void *q : ptrs) ok = ok && aligned16(q);
    for (int64_t s : strides) ok = ok && s % v == 0;
    return ok;
}

uint32_t conv_cblocks(int64_t dim, int v) {
    return static_cast<uint32_t>((dim + static_cast<int64_t>(kConvThreads) * v - 1) / (static_cast<int64_t>(kConvThreads) * v));
}

// f(type, vector length, width) with the three as compile-time constants
template <typename F>
int conv_dispatch(int32_t act_dtype, bool vec, int k, F f) {
    auto by_width = [&](auto t, auto v) {
        switch (k) {
            case 1: return f(t, v, std::integral_constant<int, 1>());
            case 2: return f(t, v, std::integral_constant<int, 2>());
            case 3: return f(t, v, std::integral_constant<int, 3>());
            default: return f(t, v, std::integral_constant<int, 4>());
        }
    };
    if (act_dtype == SSM_BF16)
        return vec ? by_width(bf16raw(), std::integral_constant<int, 8>()) : by_width(bf16raw(), std::integral_constant<int, 1>());
    return vec ? by_width(float(), std::integral_constant<int, 4>()) : by_width(float(), std::integral_constant<int, 1>());
}

int launched() { return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA; }

// A kernel whose blocks may come while the one before it on the stream still runs; it waits for
// that one's end itself (wait_previous).
template <typename... P, typename... A>
bool launch_after(void (*kernel)(P...), dim3 grid, dim3 block, int smem, cudaStream_t stream, const A &...args) {
    cudaLaunchAttribute after;
    after.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    after.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid, cfg.blockDim = block, cfg.dynamicSmemBytes = static_cast<size_t>(smem), cfg.stream = stream;
    cfg.attrs = &after, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

constexpr int64_t kConvBlocks = 1184;

// Rows of a tile.  A tile reads K - 1 rows before its own (and, for the gradients,
// after them) and its taps again, so tiles are long; but few rows are cut shorter,
// down to 16, until some eight blocks of 64 threads stand for each SM.
int64_t conv_tile(int64_t tokens, int64_t dim, int64_t longest) {
    const int64_t cblocks = (dim + 4 * kConvThreads - 1) / (4 * kConvThreads);
    int64_t tile = longest;
    while (tile > 16 && (tokens + tile - 1) / tile * cblocks < kConvBlocks) tile /= 2;
    return tile;
}
// For the gradients at most 256 tiles: their partial sums stay small beside the rows.
int64_t conv_bwd_tile(int64_t tokens, int64_t dim) {
    return std::max<int64_t>(conv_tile(tokens, dim, 128), ((tokens + 255) / 256 + 3) / 4 * 4);
}
int64_t conv_bwd_tiles(int64_t tokens, int64_t dim) { return (tokens + conv_bwd_tile(tokens, dim) - 1) / conv_bwd_tile(tokens, dim); }
size_t conv_bwd_bytes(const ssm_conv1d_dims_t *d) {
    return static_cast<size_t>(conv_bwd_tiles(d->tokens, d->dim)) * (d->width + 1) * d->dim * 4;
}

}  // namespace

extern "C" {

int ssm_conv1d_fwd(const void *x, const float *w, const float *bias, const int32_t *cu_seqlens, void *windows,
                   const int32_t *slots, const uint8_t *has_initial, void *y, const ssm_conv1d_dims_t *dims,
                   ssm_stream_t stream) {
    Conv1dParams p;
    int rc = conv_setup(x, w, bias, dims, &p);
    if (rc == SSM_OK) rc = conv_sequences(cu_seqlens, dims, &p);
    if (rc != SSM_OK) return rc;
    if (!y) return SSM_ERR_INVALID_ARG;
    if (dims->y_stride < dims->dim || !rows_ok(dims->tokens, dims->y_stride)) return SSM_ERR_INVALID_ARG;
    const int64_t es = dims->act_dtype == SSM_F32 ? 4 : 2, K = dims->width;
    if (!aligned_to(y, es) || !aligned_to(windows, es) || !aligned4(slots)) return SSM_ERR_MISALIGNED;
    if (!rows_ok(dims->slots, (K - 1) * dims->dim)) return SSM_ERR_INVALID_ARG;
    const int64_t cache = windows ? dims->slots * (K - 1) * dims->dim * es : 0;
    const Rows ins[] = {{x, dims->tokens, dims->dim * es, dims->x_stride * es}, flat(w, dims->dim * K * 4),
                        flat(bias, dims->dim * 4), flat(cu_seqlens, (dims->sequences + 1) * 4),
                        flat(slots, dims->sequences * 4), flat(has_initial, dims->sequences)};
    const Rows outs[] = {{y, dims->tokens, dims->dim * es, dims->y_stride * es}, flat(windows, cache)};
    if (outputs_clash(ins, outs)) return SSM_ERR_INVALID_ARG;
    p.windows = windows, p.y = y, p.y_stride = dims->y_stride;
    p.seq.slots = slots, p.seq.has_initial = has_initial;
    const bool vec = vector_rows({x, y, windows, w, bias}, {dims->x_stride, dims->y_stride}, dims->dim, dims->act_dtype);
    p.tile = conv_tile(dims->tokens, dims->dim, 64);
    const int64_t tiles = (dims->tokens + p.tile - 1) / p.tile;
    if ((std::max<int64_t>(tiles, dims->sequences)) * conv_cblocks(dims->dim, 1) > INT32_MAX) return SSM_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return conv_dispatch(dims->act_dtype, vec, dims->width, [&](auto t, auto v, auto k) {
        using T = decltype(t);
        // four channels a thread (8 bytes of bf16): with eight, 144 registers leave 14 warps an SM (117 us
        // against 81 for 16384 x 5376)
        constexpr int V = v > 4 ? 4 : v;
        p.cblocks = conv_cblocks(p.dim, V);
        conv1d_fwd_kernel<T, V, k><<<static_cast<unsigned>(tiles * p.cblocks), kConvThreads, 0, s>>>(p);
        p.cblocks = conv_cblocks(p.dim, v);
        if (windows && k > 1 &&
            !launch_after(conv1d_window_kernel<T, v, k>, dim3(static_cast<unsigned>(p.seq.sequences * static_cast<int64_t>(p.cblocks))),
                          dim3(kConvThreads), 0, s, p))
            return static_cast<int>(SSM_ERR_CUDA);
        return launched();
    });
}

int ssm_conv1d_step(void *windows, const int32_t *slots, const void *x, const float *w, const float *bias, void *y,
                    const ssm_conv1d_dims_t *dims, ssm_stream_t stream) {
    Conv1dParams p;
    const int rc = conv_setup(x, w, bias, dims, &p);
    if (rc != SSM_OK) return rc;
    const int64_t es = dims->act_dtype == SSM_F32 ? 4 : 2, K = dims->width;
    if (!y || (K > 1 && !windows)) return SSM_ERR_INVALID_ARG;
    if (!slots && dims->tokens > dims->slots) return SSM_ERR_INVALID_ARG;
    if (dims->y_stride < dims->dim || !rows_ok(dims->tokens, dims->y_stride)) return SSM_ERR_INVALID_ARG;
    if (!aligned_to(y, es) || !aligned_to(windows, es) || !aligned4(slots)) return SSM_ERR_MISALIGNED;
    if (!rows_ok(dims->slots, (K - 1) * dims->dim)) return SSM_ERR_INVALID_ARG;
    const Rows ins[] = {{x, dims->tokens, dims->dim * es, dims->x_stride * es}, flat(w, dims->dim * K * 4),
                        flat(bias, dims->dim * 4), flat(slots, dims->tokens * 4)};
    const Rows outs[] = {{y, dims->tokens, dims->dim * es, dims->y_stride * es},
                         flat(windows, windows ? dims->slots * (K - 1) * dims->dim * es : 0)};
    if (outputs_clash(ins, outs)) return SSM_ERR_INVALID_ARG;
    p.windows = windows, p.y = y, p.y_stride = dims->y_stride;
    p.seq.slots = slots, p.seq.sequences = static_cast<int32_t>(dims->tokens);
    const bool vec = vector_rows({x, y, windows, w, bias}, {dims->x_stride, dims->y_stride}, dims->dim, dims->act_dtype);
    if (dims->tokens * conv_cblocks(dims->dim, 1) > INT32_MAX) return SSM_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return conv_dispatch(dims->act_dtype, vec, dims->width, [&](auto t, auto v, auto k) {
        p.cblocks = conv_cblocks(p.dim, v);
        conv1d_step_kernel<decltype(t), v, k><<<static_cast<unsigned>(dims->tokens * p.cblocks), kConvThreads, 0, s>>>(p);
        return launched();
    });
}

int ssm_conv1d_bwd_workspace_size(const ssm_conv1d_dims_t *dims, size_t *bytes) {
    if (!dims || !bytes || dims->tokens < 1 || dims->dim < 1) return SSM_ERR_INVALID_ARG;
    if (dims->width < 1 || dims->width > 4 || dims->tokens > INT32_MAX || dims->dim > INT32_MAX) return SSM_ERR_UNSUPPORTED;
    *bytes = conv_bwd_bytes(dims);
    return SSM_OK;
}

int ssm_conv1d_bwd(const void *x, const float *w, const float *bias, const int32_t *cu_seqlens, const void *dy, void *dx,
                   float *dw, float *dbias, void *workspace, size_t workspace_bytes, const ssm_conv1d_dims_t *dims,
                   ssm_stream_t stream) {
    Conv1dParams p;
    int rc = conv_setup(x, w, bias, dims, &p);
    if (rc == SSM_OK) rc = conv_sequences(cu_seqlens, dims, &p);
    if (rc != SSM_OK) return rc;
    if (!dy || !dx || !dw || !workspace) return SSM_ERR_INVALID_ARG;
    if (dims->dy_stride < dims->dim || dims->dx_stride < dims->dim || !rows_ok(dims->tokens, dims->dy_stride) ||
        !rows_ok(dims->tokens, dims->dx_stride))
        return SSM_ERR_INVALID_ARG;
    if (workspace_bytes < conv_bwd_bytes(dims)) return SSM_ERR_INVALID_ARG;
    const int64_t es = dims->act_dtype == SSM_F32 ? 4 : 2, K = dims->width;
    if (!aligned_to(dy, es) || !aligned_to(dx, es) || !aligned4(dw) || !aligned4(dbias) || !aligned16(workspace))
        return SSM_ERR_MISALIGNED;
    const Rows ins[] = {{x, dims->tokens, dims->dim * es, dims->x_stride * es}, flat(w, dims->dim * K * 4),
                        flat(bias, dims->dim * 4), flat(cu_seqlens, (dims->sequences + 1) * 4),
                        {dy, dims->tokens, dims->dim * es, dims->dy_stride * es}};
    const Rows outs[] = {{dx, dims->tokens, dims->dim * es, dims->dx_stride * es}, flat(dw, dims->dim * K * 4),
                         flat(dbias, dims->dim * 4), flat(workspace, static_cast<int64_t>(workspace_bytes))};
    if (outputs_clash(ins, outs)) return SSM_ERR_INVALID_ARG;
    p.dy = dy, p.dx = dx, p.dy_stride = dims->dy_stride, p.dx_stride = dims->dx_stride;
    p.partial = static_cast<float *>(workspace), p.dw = dw, p.dbias = dbias;
    p.tile = conv_bwd_tile(dims->tokens, dims->dim);
    const int64_t tiles = conv_bwd_tiles(dims->tokens, dims->dim);
    const bool vec = vector_rows({x, dy, dx, w, bias}, {dims->x_stride, dims->dy_stride, dims->dx_stride}, dims->dim, dims->act_dtype);
    if (tiles * conv_cblocks(dims->dim, 1) > INT32_MAX) return SSM_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return conv_dispatch(dims->act_dtype, vec, dims->width, [&](auto t, auto v, auto k) {
        // four channels a thread, two where that would leave SMs without blocks (16384 x 5376 bf16:
        // 139 us with four, 148 with two; 1314 x 1792 float32: 30 and 19; both with blocks of 128)
        constexpr int V4 = v > 4 ? 4 : v, V2 = v > 2 ? 2 : v;
        p.cblocks = conv_cblocks(p.dim, V4);
        if (tiles * p.cblocks >= kConvBlocks) {
            conv1d_bwd_kernel<decltype(t), V4, k><<<static_cast<unsigned>(tiles * p.cblocks), kConvThreads, 0, s>>>(p);
        } else {
            p.cblocks = conv_cblocks(p.dim, V2);
            conv1d_bwd_kernel<decltype(t), V2, k><<<static_cast<unsigned>(tiles * p.cblocks), kConvThreads, 0, s>>>(p);
        }
        const float *partial = p.partial;
        const int width = k;
        if (!launch_after(conv1d_reduce_kernel, dim3(static_cast<unsigned>((p.dim + 31) / 32), k + 1), dim3(32, 8), 0, s, partial, p.dw,
                          p.dbias, p.dim, tiles, width))
            return static_cast<int>(SSM_ERR_CUDA);
        return launched();
    });
}

}  // extern "C"

// ---- gated norm ------------------------------------------------------------------------

namespace {

constexpr int kNormThreads = 512;      // threads that share a row's group at most
constexpr int kNormSmallBlock = 128;   // threads of a block whose rows need one warp or less
// blocks of the gradient kernel in all: two for each of 148 SMs (592: 186 us against 181 for 16384 rows of 5120)
constexpr int kNormBwdBlocks = 296;

// How the threads share a row's group of `gdim` columns: vectors of V elements,
// NV to a thread, `tpr` threads.
struct NormShape {
    int v, nv, tpr, rpb;  // rpb: rows to a block
};

// A thread takes one vector where a warp covers the group, else `want` elements
// (32 at most, more only where 512 threads would not reach).
bool norm_shape(int64_t gdim, int v, int want, NormShape *s) {
    const int64_t nvec = (gdim + v - 1) / v;
    s->v = v;
    if (nvec <= 32) {
        s->nv = 1;
        for (s->tpr = 1; s->tpr < nvec; s->tpr *= 2) {}
        s->rpb = kNormSmallBlock / s->tpr;
        return true;
    }
    for (int ept : {want, 32}) {
        s->nv = ept / v;
        const int64_t t = (nvec + 32 * s->nv - 1) / (32 * s->nv) * 32;
        s->tpr = static_cast<int>(std::min<int64_t>(t, INT32_MAX));
        s->rpb = t == 32 ? kNormSmallBlock / 32 : 1;
        if (t <= kNormThreads) return true;
    }
    return false;
}

int norm_setup(const void *x, const void *z, const float *weight, const ssm_norm_dims_t *d, NormParams *p) {
    if (!d || !x || !weight) return SSM_ERR_INVALID_ARG;
    if (d->rows < 1 || d->dim < 1 || d->groups < 1 || d->dim % d->groups != 0) return SSM_ERR_INVALID_ARG;
    if (!(d->eps >= 0.0f)) return SSM_ERR_INVALID_ARG;
    if (!dtype_ok(d->act_dtype)) return SSM_ERR_UNSUPPORTED;
    if (d->dim / d->groups > 16384 || d->dim > INT32_MAX || d->groups > 65535 || d->rows > INT32_MAX) return SSM_ERR_UNSUPPORTED;
    if (d->x_stride < d->dim || (z && d->z_stride < d->dim) || !rows_ok(d->rows, d->x_stride) || !rows_ok(d->rows, z ? d->z_stride : 0))
        return SSM_ERR_INVALID_ARG;
    const size_t es = d->act_dtype == SSM_F32 ? 4 : 2;
    if (!aligned_to(x, es) || !aligned_to(z, es) || !aligned4(weight)) return SSM_ERR_MISALIGNED;
    memset(p, 0, sizeof *p);
    p->x = x, p->z = z, p->weight = weight;
    p->rows = d->rows, p->dim = d->dim, p->gdim = d->dim / d->groups, p->groups = static_cast<int32_t>(d->groups);
    p->x_stride = d->x_stride, p->z_stride = d->z_stride, p->eps = d->eps;
    return SSM_OK;
}

// f(type, vector length, vectors a thread, gate, gate first) as compile-time constants
template <typename F>
int norm_dispatch(int32_t act_dtype, const NormShape &s, bool gate, bool gate_first, F f) {
    auto by_gate = [&](auto t, auto v, auto nv) {
        if (!gate) return f(t, v, nv, std::false_type(), std::false_type());
        return gate_first ? f(t, v, nv, std::true_type(), std::true_type()) : f(t, v, nv, std::true_type(), std::false_type());
    };
    auto by_nv = [&](auto t, auto v) {
        if (s.nv == 1) return by_gate(t, v, std::integral_constant<int, 1>());
        if (s.nv * s.v == 16) return by_gate(t, v, std::integral_constant<int, 16 / v>());
        return by_gate(t, v, std::integral_constant<int, 32 / v>());
    };
    if (act_dtype == SSM_BF16)
        return s.v == 8 ? by_nv(bf16raw(), std::integral_constant<int, 8>()) : by_nv(bf16raw(), std::integral_constant<int, 1>());
    return s.v == 4 ? by_nv(float(), std::integral_constant<int, 4>()) : by_nv(float(), std::integral_constant<int, 1>());
}

// blocks of the gradient kernel for each group, with `rpb` rows to a block
int64_t norm_bwd_blocks(int64_t rows, int64_t groups, int rpb) {
    return std::max<int64_t>(1, std::min<int64_t>((rows + rpb - 1) / rpb, kNormBwdBlocks / groups));
}

// Slots of partial sums at most, whatever the alignment of the rows turns out to be.
size_t norm_bwd_bytes(const ssm_norm_dims_t *d) {
    int64_t slots = 1;
    for (int v : {d->act_dtype == SSM_F32 ? 4 : 8, 1}) {
        NormShape s;
        if (norm_shape(d->dim / d->groups, v, 16, &s))
            slots = std::max<int64_t>(slots, norm_bwd_blocks(d->rows, d->groups, s.rpb) * s.rpb);
    }
    return static_cast<size_t>(slots) * d->dim * 4;
}

}  // namespace

extern "C" {

int ssm_gated_norm_fwd(const void *x, const void *z, const float *weight, void *out, float *rstd,
                       const ssm_norm_dims_t *dims, ssm_stream_t stream) {
    NormParams p;
    const int rc = norm_setup(x, z, weight, dims, &p);
    if (rc != SSM_OK) return rc;
    if (!out || dims->out_stride < dims->dim || !rows_ok(dims->rows, dims->out_stride)) return SSM_ERR_INVALID_ARG;
    const int64_t es = dims->act_dtype == SSM_F32 ? 4 : 2;
    if (!aligned_to(out, es) || !aligned4(rstd)) return SSM_ERR_MISALIGNED;
    const int64_t wb = dims->dim * es;
    const Rows ins[] = {{x, dims->rows, wb, dims->x_stride * es}, {z, z ? dims->rows : 0, wb, dims->z_stride * es}, flat(weight, dims->dim * 4)};
    const Rows outs[] = {{out, dims->rows, wb, dims->out_stride * es}, flat(rstd, rstd ? dims->rows * dims->groups * 4 : 0)};
    if (outputs_clash(ins, outs)) return SSM_ERR_INVALID_ARG;
    p.out = out, p.rstd = rstd, p.out_stride = dims->out_stride;
    const bool vec = vector_rows({x, z, out, weight}, {dims->x_stride, z ? dims->z_stride : 0, dims->out_stride}, p.gdim, dims->act_dtype);
    NormShape s;
    if (!norm_shape(p.gdim, vec ? (es == 4 ? 4 : 8) : 1, 32, &s)) return SSM_ERR_UNSUPPORTED;
    const int64_t blocks = (p.rows * p.groups + s.rpb - 1) / s.rpb;
    if (blocks > INT32_MAX) return SSM_ERR_UNSUPPORTED;
    return norm_dispatch(dims->act_dtype, s, z != nullptr, dims->gate_first != 0, [&](auto t, auto v, auto nv, auto gate, auto first) {
        gated_norm_fwd_kernel<decltype(t), v, nv, gate, first>
            <<<static_cast<unsigned>(blocks), s.tpr * s.rpb, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p, s.tpr);
        return launched();
    });
}

int ssm_gated_norm_bwd_workspace_size(const ssm_norm_dims_t *dims, size_t *bytes) {
    if (!dims || !bytes || dims->rows < 1 || dims->dim < 1 || dims->groups < 1 || dims->dim % dims->groups != 0)
        return SSM_ERR_INVALID_ARG;
    if (dims->rows > INT32_MAX || dims->dim > INT32_MAX) return SSM_ERR_UNSUPPORTED;
    *bytes = norm_bwd_bytes(dims);
    return SSM_OK;
}

int ssm_gated_norm_bwd(const void *x, const void *z, const float *weight, const void *dout, void *dx, void *dz,
                       float *dweight, void *workspace, size_t workspace_bytes, const ssm_norm_dims_t *dims,
                       ssm_stream_t stream) {
    NormParams p;
    const int rc = norm_setup(x, z, weight, dims, &p);
    if (rc != SSM_OK) return rc;
    if (!dout || !dx || !dweight || !workspace || (z && !dz)) return SSM_ERR_INVALID_ARG;
    if (!z) dz = nullptr;
    if (dims->dout_stride < dims->dim || dims->dx_stride < dims->dim || (dz && dims->dz_stride < dims->dim) ||
        !rows_ok(dims->rows, dims->dout_stride) || !rows_ok(dims->rows, dims->dx_stride) || !rows_ok(dims->rows, dz ? dims->dz_stride : 0))
        return SSM_ERR_INVALID_ARG;
    if (workspace_bytes < norm_bwd_bytes(dims)) return SSM_ERR_INVALID_ARG;
    const int64_t es = dims->act_dtype == SSM_F32 ? 4 : 2, wb = dims->dim * es;
    if (!aligned_to(dout, es) || !aligned_to(dx, es) || !aligned_to(dz, es) || !aligned4(dweight) || !aligned16(workspace))
        return SSM_ERR_MISALIGNED;
    const Rows ins[] = {{x, dims->rows, wb, dims->x_stride * es}, {z, z ? dims->rows : 0, wb, dims->z_stride * es},
                        flat(weight, dims->dim * 4), {dout, dims->rows, wb, dims->dout_stride * es}};
    const Rows outs[] = {{dx, dims->rows, wb, dims->dx_stride * es}, {dz, dz ? dims->rows : 0, wb, dims->dz_stride * es},
                         flat(dweight, dims->dim * 4), flat(workspace, static_cast<int64_t>(workspace_bytes))};
    if (outputs_clash(ins, outs)) return SSM_ERR_INVALID_ARG;
    p.dout = dout, p.dx = dx, p.dz = dz, p.partial = static_cast<float *>(workspace);
    p.dout_stride = dims->dout_stride, p.dx_stride = dims->dx_stride, p.dz_stride = dims->dz_stride;
    const bool vec = vector_rows({x, z, dout, dx, dz, weight},
                                 {dims->x_stride, z ? dims->z_stride : 0, dims->dout_stride, dims->dx_stride, dz ? dims->dz_stride : 0},
                                 p.gdim, dims->act_dtype);
    NormShape s;
    if (!norm_shape(p.gdim, vec ? (es == 4 ? 4 : 8) : 1, 16, &s)) return SSM_ERR_UNSUPPORTED;
    const int64_t blocks = norm_bwd_blocks(p.rows, p.groups, s.rpb);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return norm_dispatch(dims->act_dtype, s, z != nullptr, dims->gate_first != 0, [&](auto t, auto v, auto nv, auto gate, auto first) {
        // 16 elements a thread fit the 96 registers with which two blocks of 320 threads share an SM
        // (three at 64 registers spilled: 196 us against 181 for 16384 rows of 5120, before the weights
        // stayed in registers)
        const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(p.groups));
        const int threads = s.tpr * s.rpb, smem = norm_bwd_smem(threads, nv, v * static_cast<int>(es), gate);
        auto launch = [&](auto kernel) {
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return SSM_ERR_CUDA;
            kernel<<<grid, threads, smem, st>>>(p, s.tpr);
            return SSM_OK;
        };
        int rc2 = -1;
        if constexpr (nv * v <= 16) {
            if (threads <= 320) rc2 = launch(gated_norm_bwd_kernel<decltype(t), v, nv, gate, first, 320, 2>);
        }
        if (rc2 < 0) rc2 = launch(gated_norm_bwd_kernel<decltype(t), v, nv, gate, first, kNormThreads, 1>);
        if (rc2 != SSM_OK) return rc2;
        const float *partial = p.partial;
        const int64_t slots = blocks * s.rpb;
        if (!launch_after(norm_reduce_kernel, dim3(static_cast<unsigned>((p.dim + 31) / 32)), dim3(32, 32), 0, st, partial, dweight, p.dim, slots))
            return static_cast<int>(SSM_ERR_CUDA);
        return launched();
    });
}

}  // extern "C"

// ---- SSD on packed sequences and on single tokens -----------------------------------------

namespace {

// The checks that the packed forward and the step share.
int ssd_setup(const void *x, const void *dt, const float *dt_bias, const float *A, const void *B, const void *C,
              const float *D, const int32_t *slots, const void *out, const ssm_ssd_packed_dims_t *d) {
    if (!d || !x || !dt || !A || !B || !C || !out) return SSM_ERR_INVALID_ARG;
    if (d->tokens < 1 || d->heads < 1 || d->groups < 1 || d->headdim < 1 || d->dstate < 1 || d->slots < 0 || d->heads % d->groups != 0)
        return SSM_ERR_INVALID_ARG;
    if (d->headdim != kSsdP || d->dstate != kSsdN || !dtype_ok(d->act_dtype)) return SSM_ERR_UNSUPPORTED;
    if (d->tokens > INT32_MAX - kVarQ || d->slots > INT32_MAX || d->heads > 65535) return SSM_ERR_UNSUPPORTED;
    const int64_t inner = d->heads * kSsdP, bc = d->groups * kSsdN;
    if (d->x_stride < inner || d->y_stride < inner || d->dt_stride < d->heads || d->b_stride < bc || d->c_stride < bc)
        return SSM_ERR_INVALID_ARG;
    for (int64_t s : {d->x_stride, d->y_stride, d->dt_stride, d->b_stride, d->c_stride})
        if (!rows_ok(d->tokens, s)) return SSM_ERR_INVALID_ARG;
    if (!rows_ok(d->slots, d->heads * kSsdP * kSsdN)) return SSM_ERR_INVALID_ARG;
    for (const void *q : {static_cast<const void *>(A), static_cast<const void *>(dt_bias), static_cast<const void *>(D),
                          static_cast<const void *>(slots)})
        if (!aligned4(q)) return SSM_ERR_MISALIGNED;
    return SSM_OK;
}

// [tokens][n][64 or 128] bf16 rows of a stride of their own, boxes of 64 x 1 x 128 rows
bool var_map(CUtensorMap *m, const void *base, uint64_t inner, uint64_t n, uint64_t tokens, int64_t stride) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t dims[3] = {inner, n, tokens};
    const cuuint64_t strides[2] = {inner * 2, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[3] = {64, 1, kVarQ}, estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t var_pairs(const ssm_ssd_packed_dims_t *d) {
    return d->groups * ((d->heads / d->groups + kVarHeads - 1) / kVarHeads);
}

// Tokens of a segment of the two passes: two to seven chunks, about three segments to each of 148
// SMs (a segment costs about half a chunk more for its state, and the last ones should even out;
// one sequence of 32768 with 24 heads: 193 us with seven chunks, 229 with five; 20 ragged ones: 82
// with two, 88 with three); longer where a thousand segments or sixteen to each SM would not do,
// which bounds the states in the workspace.
int64_t var_segment(const ssm_ssd_packed_dims_t *d) {
    const int64_t chunks = (d->tokens + kVarQ - 1) / kVarQ;
    const double work = static_cast<double>(chunks) * static_cast<double>(var_pairs(d)) / 148.0;
    int64_t c = static_cast<int64_t>(std::min(std::max(std::ceil(work / 3.0), 2.0), 7.0));
    c = std::max<int64_t>(c, static_cast<int64_t>(std::min(work / 16.0, static_cast<double>(chunks))));
    c = std::max<int64_t>(c, (chunks + kVarMaxWindows - 1) / kVarMaxWindows);
    return c * kVarQ;
}

// Workspace: [0, 256) header, the units, the later segments, the flags, the decays, then (256-byte
// aligned) the states that pass between segments or CTAs, and the starting states of the sequences
// of several segments (each has a window in which its second one starts, so they are no more than those).
size_t var_layout(const ssm_ssd_packed_dims_t *d, uint8_t *base, VarWork *w) {
    const int64_t windows = (d->tokens + var_segment(d) - 1) / var_segment(d);
    size_t at = 256;
    const size_t list = at;
    at += static_cast<size_t>(windows) * sizeof(int2);
    const size_t units = at;
    at += static_cast<size_t>(d->sequences + 1) * 4;
    const size_t flags = at;
    at += kVarMaxCtas * 4;
    const size_t decay = at;
    at += static_cast<size_t>(windows) * d->heads * 4;
    const size_t carry = at = (at + 255) / 256 * 256;
    at += std::max<size_t>(static_cast<size_t>(windows > 1 ? windows : 0) * d->heads, kVarMaxCtas * kVarHeads) * kSsdP * kSsdN * 4;
    const size_t start = at;
    at += static_cast<size_t>(windows > 1 ? std::min(d->sequences, windows) : 0) * d->heads * kSsdP * kSsdN * 4;
    if (w) {
        w->queue = reinterpret_cast<uint32_t *>(base);
        w->error = reinterpret_cast<uint32_t *>(base + 16);
        w->extras = reinterpret_cast<uint32_t *>(base + 20);
        w->several = reinterpret_cast<uint32_t *>(base + 24);
        w->mode = reinterpret_cast<uint32_t *>(base + 28);
        w->range = reinterpret_cast<uint32_t *>(base + 32);
        w->units = reinterpret_cast<uint32_t *>(base + units);
        w->list = reinterpret_cast<int2 *>(base + list);
        w->flags = reinterpret_cast<uint32_t *>(base + flags);
        w->decay = reinterpret_cast<float *>(base + decay);
        w->carry = reinterpret_cast<float *>(base + carry);
        w->start = reinterpret_cast<float *>(base + start);
    }
    return at;
}

int ssd_varlen_impl(const void *x, const void *dt, const float *dt_bias, int softplus, const float *A, const void *B,
                    const void *C, const float *D, const int32_t *cu_seqlens, float *states, const int32_t *slots,
                    const uint8_t *has_initial, void *y, void *workspace, size_t workspace_bytes,
                    const ssm_ssd_packed_dims_t *dims, ssm_stream_t stream, uint32_t flag_want, uint32_t spin_limit) {
    const int rc = ssd_setup(x, dt, dt_bias, A, B, C, D, slots, y, dims);
    if (rc != SSM_OK) return rc;
    if (dims->act_dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
    if (!cu_seqlens || !workspace || dims->sequences < 1) return SSM_ERR_INVALID_ARG;
    if (dims->sequences > INT32_MAX / 4) return SSM_ERR_UNSUPPORTED;
    // TMA rows and 16-byte stores
    for (const void *q : {x, B, C, static_cast<const void *>(y), static_cast<const void *>(states), static_cast<const void *>(workspace)})
        if (!aligned16(q)) return SSM_ERR_MISALIGNED;
    for (int64_t s : {dims->x_stride, dims->b_stride, dims->c_stride, dims->y_stride})
        if (s % 8 != 0) return SSM_ERR_MISALIGNED;
    for (int64_t s : {dims->x_stride, dims->b_stride, dims->c_stride})
        if (s * 2 >= (int64_t(1) << 40)) return SSM_ERR_UNSUPPORTED;
    if (!aligned_to(dt, 2) || !aligned4(cu_seqlens)) return SSM_ERR_MISALIGNED;
    if (workspace_bytes < var_layout(dims, nullptr, nullptr)) return SSM_ERR_INVALID_ARG;
    const int64_t T = dims->tokens, H = dims->heads, G = dims->groups;
    const Rows ins[] = {{x, T, H * kSsdP * 2, dims->x_stride * 2}, {dt, T, H * 2, dims->dt_stride * 2},
                        {B, T, G * kSsdN * 2, dims->b_stride * 2}, {C, T, G * kSsdN * 2, dims->c_stride * 2},
                        flat(A, H * 4), flat(dt_bias, H * 4), flat(D, H * 4), flat(cu_seqlens, (dims->sequences + 1) * 4),
                        flat(slots, dims->sequences * 4), flat(has_initial, dims->sequences)};
    const Rows outs[] = {{y, T, H * kSsdP * 2, dims->y_stride * 2},
                         flat(states, states ? dims->slots * H * kSsdP * kSsdN * 4 : 0),
                         flat(workspace, static_cast<int64_t>(workspace_bytes))};
    if (outputs_clash(ins, outs)) return SSM_ERR_INVALID_ARG;
    VarParams p;
    memset(&p, 0, sizeof p);
    p.dt = dt, p.dt_bias = dt_bias, p.A = A, p.D = D, p.states = states, p.y = y;
    p.seq.cu = cu_seqlens, p.seq.slots = slots, p.seq.has_initial = has_initial;
    p.seq.tokens = T, p.seq.sequences = static_cast<int32_t>(dims->sequences), p.seq.nslots = static_cast<int32_t>(dims->slots);
    p.dt_stride = dims->dt_stride, p.y_stride = dims->y_stride;
    p.heads = static_cast<int32_t>(H), p.groups = static_cast<int32_t>(G), p.pairs = static_cast<int32_t>(var_pairs(dims));
    p.segment = static_cast<int32_t>(var_segment(dims));
    p.windows = static_cast<int32_t>((T + p.segment - 1) / p.segment);
    p.flag_want = flag_want, p.spin_limit = spin_limit, p.softplus = softplus ? 1 : 0;
    var_layout(dims, static_cast<uint8_t *>(workspace), &p.work);
    const int64_t units = (T / kVarQ + dims->sequences) * p.pairs;  // chunks of all pairs, at most
    if (units > INT32_MAX / 16) return SSM_ERR_UNSUPPORTED;
    VarMaps tm;
    memset(&tm, 0, sizeof tm);
    if (!var_map(&tm.x, x, kSsdP, H, T, dims->x_stride) || !var_map(&tm.B, B, kSsdN, G, T, dims->b_stride) ||
        !var_map(&tm.C, C, kSsdN, G, T, dims->c_stride))
        return SSM_ERR_CUDA;
    int sms = 0;
    if (current_sms(&sms) != SSM_OK) return SSM_ERR_CUDA;
    p.ctas = static_cast<int32_t>(std::min<int64_t>({units, sms, kVarMaxCtas}));
    if (cudaFuncSetAttribute(ssd_varlen_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, VarSmem::kTotal) != cudaSuccess ||
        cudaFuncSetAttribute(ssd_varlen_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, VarSmem::kTotal) != cudaSuccess)
        return SSM_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const unsigned ctas = static_cast<unsigned>(p.ctas);
    ssd_varlen_setup_kernel<<<1, 1024, 0, s>>>(p);
    if (p.windows > 1) {  // some sequence may have more than one segment
        // about eight blocks to an SM at most: where there is nothing to join they cost what they are launched for
        const unsigned several = static_cast<unsigned>(
            std::min<int64_t>({dims->sequences, p.windows, std::max<int64_t>(1, 1184 / (H * 8))}));
        if (!launch_after(ssd_varlen_kernel<true>, dim3(ctas), dim3(kVarSummaryThreads), VarSmem::kTotal, s, p, tm) ||
            !launch_after(ssd_varlen_combine_kernel, dim3(static_cast<unsigned>(H) * 8, several), dim3(256), 0, s, p))
            return SSM_ERR_CUDA;
    }
    if (!launch_after(ssd_varlen_kernel<false>, dim3(ctas), dim3(kVarThreads), VarSmem::kTotal, s, p, tm)) return SSM_ERR_CUDA;
    return launched();
}

}  // namespace

extern "C" {

int ssm_ssd_varlen_fwd_workspace_size(const ssm_ssd_packed_dims_t *dims, size_t *bytes) {
    if (!dims || !bytes || dims->tokens < 1 || dims->sequences < 1 || dims->heads < 1 || dims->groups < 1 ||
        dims->heads % dims->groups != 0)
        return SSM_ERR_INVALID_ARG;
    if (dims->tokens > INT32_MAX - kVarQ || dims->sequences > INT32_MAX / 4 || dims->heads > 65535) return SSM_ERR_UNSUPPORTED;
    *bytes = var_layout(dims, nullptr, nullptr);
    return SSM_OK;
}

int ssm_ssd_varlen_fwd(const void *x, const void *dt, const float *dt_bias, int softplus, const float *A, const void *B,
                       const void *C, const float *D, const int32_t *cu_seqlens, float *states, const int32_t *slots,
                       const uint8_t *has_initial, void *y, void *workspace, size_t workspace_bytes,
                       const ssm_ssd_packed_dims_t *dims, ssm_stream_t stream) {
    return ssd_varlen_impl(x, dt, dt_bias, softplus, A, B, C, D, cu_seqlens, states, slots, has_initial, y, workspace,
                           workspace_bytes, dims, stream, 1u, kSsdFlagLimit);
}

int ssm_debug_ssd_varlen_flag_timeout(const void *x, const void *dt, const float *dt_bias, int softplus, const float *A,
                                      const void *B, const void *C, const float *D, const int32_t *cu_seqlens,
                                      float *states, const int32_t *slots, const uint8_t *has_initial, void *y,
                                      void *workspace, size_t workspace_bytes, uint32_t spin_limit,
                                      const ssm_ssd_packed_dims_t *dims, ssm_stream_t stream) {
    return ssd_varlen_impl(x, dt, dt_bias, softplus, A, B, C, D, cu_seqlens, states, slots, has_initial, y, workspace,
                           workspace_bytes, dims, stream, 1u << 30, spin_limit);  // no flag ever reaches this
}

int ssm_ssd_step(float *states, const int32_t *slots, const void *x, const void *dt, const float *dt_bias, int softplus,
                 const float *A, const void *B, const void *C, const float *D, void *out,
                 const ssm_ssd_packed_dims_t *dims, ssm_stream_t stream) {
    const int rc = ssd_setup(x, dt, dt_bias, A, B, C, D, slots, out, dims);
    if (rc != SSM_OK) return rc;
    if (!states || (!slots && dims->tokens > dims->slots)) return SSM_ERR_INVALID_ARG;
    const int64_t es = dims->act_dtype == SSM_F32 ? 4 : 2;
    // B and C are read four elements at a time, the states as 16-byte vectors
    if (!aligned16(states) || !aligned_to(B, 4 * es) || !aligned_to(C, 4 * es) || dims->b_stride % 4 != 0 || dims->c_stride % 4 != 0)
        return SSM_ERR_MISALIGNED;
    if (!aligned_to(x, es) || !aligned_to(dt, es) || !aligned_to(out, es)) return SSM_ERR_MISALIGNED;
    const int64_t b = dims->tokens, H = dims->heads, G = dims->groups;
    const Rows ins[] = {{x, b, H * kSsdP * es, dims->x_stride * es}, {dt, b, H * es, dims->dt_stride * es},
                        {B, b, G * kSsdN * es, dims->b_stride * es}, {C, b, G * kSsdN * es, dims->c_stride * es},
                        flat(A, H * 4), flat(dt_bias, H * 4), flat(D, H * 4), flat(slots, b * 4)};
    const Rows outs[] = {{out, b, H * kSsdP * es, dims->y_stride * es}, flat(states, dims->slots * H * kSsdP * kSsdN * 4)};
    if (outputs_clash(ins, outs)) return SSM_ERR_INVALID_ARG;
    const int64_t blocks = b * H * (kSsdStepP / kSsdStepTile);
    if (blocks > INT32_MAX) return SSM_ERR_UNSUPPORTED;
    SsdStepParams p;
    memset(&p, 0, sizeof p);
    p.states = states, p.slots = slots, p.x = x, p.dt = dt, p.B = B, p.C = C;
    p.dt_bias = dt_bias, p.A = A, p.D = D, p.out = out;
    p.x_stride = dims->x_stride, p.dt_stride = dims->dt_stride, p.b_stride = dims->b_stride, p.c_stride = dims->c_stride;
    p.out_stride = dims->y_stride;
    p.nslots = static_cast<int32_t>(dims->slots), p.heads = static_cast<int32_t>(H), p.groups = static_cast<int32_t>(G);
    p.softplus = softplus ? 1 : 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dims->act_dtype == SSM_BF16) ssd_step_kernel<bf16raw><<<static_cast<unsigned>(blocks), kSsdStepThreads, 0, s>>>(p);
    else ssd_step_kernel<float><<<static_cast<unsigned>(blocks), kSsdStepThreads, 0, s>>>(p);
    return launched();
}

}  // extern "C"
