// gated_norm.cuh -- the RMS norm of a Mamba-2 block fused with its gate, and its
// gradients.  The columns fall into `groups` equal parts, each normalised alone.
// With s = silu(z) (1 without z), r = 1 / sqrt(mean(v^2) + eps) over a group:
//
//   gate first:  v = x s,  out = v r w          norm first:  v = x,  out = v r w s
//
// Gradients, with n = v r and m(.) the mean over the group:
//   up = dout (gate first) or dout s,  dw = sum over rows of up n,
//   dn = up w,  dv = r (dn - n m(dn n)),
//   gate first: dx = dv s, dz = dv x s'     norm first: dx = dv, dz = dout n w s'
//
// Some 15 (forward) to 30 (gradients) operations per element: bound by HBM (3
// and 5 passes over the rows).  A row's group is held in the registers of the
// threads that share it, so each input is read once; the statistics are sums
// of float32 over lanes, then over warps in a fixed order.
#pragma once

#include "packed.cuh"

namespace ssm {

struct NormParams {
    const void *x, *z, *dout;  // [rows][dim], rows x_stride, z_stride, dout_stride apart; z may be NULL
    const float *weight;       // [dim]
    void *out;                 // [rows][dim], rows out_stride apart
    float *rstd;               // [rows][groups] or NULL
    void *dx, *dz;             // [rows][dim], rows dx_stride, dz_stride apart; dz NULL without z
    float *partial;            // [blocks per group][dim]
    int64_t rows, dim, gdim;   // gdim = dim / groups
    int64_t x_stride, z_stride, dout_stride, out_stride, dx_stride, dz_stride;
    int32_t groups;
    float eps;
};

// The sum over the threads that share a row: `threads` of them (a power of two
// up to 32, or whole warps).  slots: one float per warp of the block.  With more
// than one warp to a row the block holds that one row, and every thread gets the
// warps' sums added in the same order.
__device__ __forceinline__ float norm_row_sum(float v, int threads, float *slots) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < threads) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (threads <= 32) return v;
    const int warps = threads >> 5;
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = slots[0];
    for (int i = 1; i < warps; ++i) s += slots[i];
    return s;
}

// TPR threads share a row's group: thread j takes vectors j, j + TPR, ... (NV of
// them at most, V elements each).  grid.x: the (row, group) pairs, blockDim.x /
// TPR to a block.
template <typename T, int V, int NV, bool GATE, bool GATE_FIRST>
__global__ void __launch_bounds__(512) gated_norm_fwd_kernel(const NormParams p, int tpr) {
    using R = Row<T, V>;
    constexpr bool kAccurate = Act<T>::kBytes == 4;
    __shared__ float slots[32];
    const int j = threadIdx.x % tpr;
    const int64_t pairs = p.rows * p.groups;
    const int64_t pair = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool live = pair < pairs;  // others still join the sums
    const int64_t row = (live ? pair : pairs - 1) / p.groups, col0 = ((live ? pair : pairs - 1) % p.groups) * p.gdim;
    typename R::Raw rx[NV], rz[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = (static_cast<int64_t>(i) * tpr + j) * V;
        rx[i] = c < p.gdim ? R::load_raw(p.x, row * p.x_stride + col0 + c) : R::zero_raw();
        if constexpr (GATE) rz[i] = c < p.gdim ? R::load_raw(p.z, row * p.z_stride + col0 + c) : R::zero_raw();
    }
    float v[NV][V], ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            v[i][e] = R::get(rx[i], e);
            if constexpr (GATE && GATE_FIRST) {
                const float z = R::get(rz[i], e);
                v[i][e] *= z * sigmoid_of<kAccurate>(z);
            }
            ss = fmaf(v[i][e], v[i][e], ss);
        }
    ss = norm_row_sum(ss, tpr, slots);
    const float r = 1.0f / sqrtf(ss / static_cast<float>(p.gdim) + p.eps);
    if (!live) return;
    if (p.rstd && j == 0) p.rstd[pair] = r;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = (static_cast<int64_t>(i) * tpr + j) * V;
        if (c >= p.gdim) continue;
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            o[e] = v[i][e] * r * __ldg(p.weight + col0 + c + e);
            if constexpr (GATE && !GATE_FIRST) {
                const float z = R::get(rz[i], e);
                o[e] *= z * sigmoid_of<kAccurate>(z);
            }
        }
        R::store(p.out, row * p.out_stride + col0 + c, o);
    }
}

// Gradients.  Block (b, g) takes rows b R, b R + 1, ... of group g (R rows share
// the block when a row needs one warp or less) at a stride of the grid, and keeps
// the sums of dw over its rows in registers; they go to `partial`, one row of it
// per block and row slot, added in a fixed order by norm_reduce_kernel.
template <typename T, int V, int NV, bool GATE, bool GATE_FIRST>
__global__ void __launch_bounds__(512) gated_norm_bwd_kernel(const NormParams p, int tpr) {
    using R = Row<T, V>;
    constexpr bool kAccurate = Act<T>::kBytes == 4;
    __shared__ float slots[2][2][32];
    const int j = threadIdx.x % tpr, rpb = blockDim.x / tpr;
    const int64_t col0 = static_cast<int64_t>(blockIdx.y) * p.gdim;
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * rpb + threadIdx.x / tpr;
    const int64_t step = static_cast<int64_t>(gridDim.x) * rpb;
    float dw[NV][V] = {};
    int flip = 0;  // the sums' shared slots alternate: one barrier per sum is enough
    const int64_t trips = (p.rows + step - 1) / step;
    for (int64_t k = 0; k < trips; ++k, flip ^= 1) {
        const bool live = slot + k * step < p.rows;
        const int64_t row = live ? slot + k * step : p.rows - 1;
        typename R::Raw rx[NV], rz[NV], rd[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (static_cast<int64_t>(i) * tpr + j) * V;
            const bool in = c < p.gdim;
            rx[i] = in ? R::load_raw(p.x, row * p.x_stride + col0 + c) : R::zero_raw();
            if constexpr (GATE) rz[i] = in ? R::load_raw(p.z, row * p.z_stride + col0 + c) : R::zero_raw();
            rd[i] = in ? R::load_raw(p.dout, row * p.dout_stride + col0 + c) : R::zero_raw();
        }
        float ss = 0.0f, dot = 0.0f;  // sum of v^2, and of (up w) v
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (static_cast<int64_t>(i) * tpr + j) * V;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float v = R::get(rx[i], e), up = R::get(rd[i], e);
                if constexpr (GATE) {
                    const float z = R::get(rz[i], e), s = z * sigmoid_of<kAccurate>(z);
                    if constexpr (GATE_FIRST) v *= s;
                    else up *= s;
                }
                ss = fmaf(v, v, ss);
                dot = fmaf(up * (c < p.gdim ? __ldg(p.weight + col0 + c + e) : 0.0f), v, dot);
            }
        }
        ss = norm_row_sum(ss, tpr, slots[flip][0]);
        dot = norm_row_sum(dot, tpr, slots[flip][1]);
        const float r = 1.0f / sqrtf(ss / static_cast<float>(p.gdim) + p.eps);
        const float mean = dot * r / static_cast<float>(p.gdim);  // m(dn n)
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (static_cast<int64_t>(i) * tpr + j) * V;
            if (c >= p.gdim) continue;
            float dx[V], dz[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float x = R::get(rx[i], e), d = R::get(rd[i], e), w = __ldg(p.weight + col0 + c + e);
                if constexpr (GATE) {
                    const float z = R::get(rz[i], e), sg = sigmoid_of<kAccurate>(z), s = z * sg;
                    const float ds = sg * fmaf(z, 1.0f - sg, 1.0f);
                    if constexpr (GATE_FIRST) {
                        const float n = x * s * r;
                        const float dv = r * fmaf(-n, mean, d * w);
                        dw[i][e] = fmaf(d, n, dw[i][e]);
                        dx[e] = dv * s;
                        dz[e] = dv * x * ds;
                    } else {
                        const float n = x * r, up = d * s;
                        dw[i][e] = fmaf(up, n, dw[i][e]);
                        dx[e] = r * fmaf(-n, mean, up * w);
                        dz[e] = d * n * w * ds;
                    }
                } else {
                    const float n = x * r;
                    dw[i][e] = fmaf(d, n, dw[i][e]);
                    dx[e] = r * fmaf(-n, mean, d * w);
                }
            }
            R::store(p.dx, row * p.dx_stride + col0 + c, dx);
            if constexpr (GATE) R::store(p.dz, row * p.dz_stride + col0 + c, dz);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = (static_cast<int64_t>(i) * tpr + j) * V;
        if (c >= p.gdim) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) p.partial[slot * p.dim + col0 + c + e] = dw[i][e];
    }
}

// dweight[c] = sum over the slots of partial[slot][c], in a fixed order.  grid: dim / 32
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float *partial, float *dweight, int64_t dim, int64_t slots) {
    __shared__ float part[32][33];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float s = 0.0f;
    if (c < dim) {
#pragma unroll 4
        for (int64_t t = threadIdx.y; t < slots; t += 32) s += __ldg(partial + t * dim + c);
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < dim) {
        for (int r = 1; r < 32; ++r) s += part[r][threadIdx.x];
        dweight[c] = s;
    }
}

}  // namespace ssm
