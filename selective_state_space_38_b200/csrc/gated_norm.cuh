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
// of float32 over lanes, then over warps in a fixed order.  Measured, 16384 rows of
// 5120 bf16 columns with the gate first, queued back to back: forward 86 us, 5.8 TB/s,
// 89 % of the copy rate; gradients 157 us, 5.3 TB/s, 81 %; called one by one 94 and
// 172 us, 81 and 74 %.
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
        float o[V], w[V];
        load_params<V, (V > 1)>(p.weight + col0 + c, w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            o[e] = v[i][e] * r * w[e];
            if constexpr (GATE && !GATE_FIRST) {
                const float z = R::get(rz[i], e);
                o[e] *= z * sigmoid_of<kAccurate>(z);
            }
        }
        R::store(p.out, row * p.out_stride + col0 + c, o);
    }
}

// Gradients.  Block (b, g) takes rows b R, b R + 1, ... of group g (R rows share
// the block when a row needs one warp or less) at a stride of the grid.  Whole
// 16-byte vectors come through shared memory, each thread's own by cp.async, so
// that the next rows are on their way without holding registers; both sums cross
// the block at once; the weights stay in registers where they fit (16 elements a thread:
// 156 us for 16384 x 5120 bf16, against 180 with the weights loaded for each row; 8 a
// thread, with twice the warps, spill and cross more warps per row: 241).  dw over the block's rows stays in registers and goes to
// `partial`, one row of it per block and row slot, added in a fixed order by
// norm_reduce_kernel.  THREADS, BLOCKS: the block's threads at most and the blocks
// that share an SM, which bound the registers.
// Rows in shared memory: this one and the next; only this one where a thread has
// eight vectors (float32 rows beyond 8192 columns), which would not fit twice.
__host__ __device__ constexpr int norm_stages(int nv) { return nv < 8 ? 2 : 1; }
// shared memory of a block: x, dout and z vectors of its threads, a stage after another
__host__ __device__ constexpr int norm_bwd_smem(int threads, int nv, int bytes, bool gate) {
    return bytes == 16 ? norm_stages(nv) * (gate ? 3 : 2) * nv * threads * 16 : 0;
}

template <typename T, int V, int NV, bool GATE, bool GATE_FIRST, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) gated_norm_bwd_kernel(const NormParams p, int tpr) {
    release_next();
    using R = Row<T, V>;
    constexpr bool kAccurate = Act<T>::kBytes == 4, kAsync = V * Act<T>::kBytes == 16;
    constexpr int kArrays = GATE ? 3 : 2, kStages = norm_stages(NV);
    extern __shared__ __align__(16) uint4 rows_smem[];
    __shared__ float2 slots[2][32];
    const int j = threadIdx.x % tpr, rpb = blockDim.x / tpr;
    const int64_t col0 = static_cast<int64_t>(blockIdx.y) * p.gdim;
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * rpb + threadIdx.x / tpr;
    const int64_t step = static_cast<int64_t>(gridDim.x) * rpb;
    const float inv = 1.0f / static_cast<float>(p.gdim);
    using Ln = Lanes<R::kL>;
    constexpr int kL = R::kL, kN = R::kN;
    Ln dw[NV][kN];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < kN; ++e) dw[i][e] = lanes<kL>(0.0f);
    typename R::Raw reg[kAsync ? 1 : kArrays][kAsync ? 1 : NV];
    constexpr int kE = Act<T>::kBytes;
    // the row's first vector of this thread, in each array; vector i is `apart` bytes times i on
    const int64_t first = col0 + static_cast<int64_t>(j) * V;
    const char *px = static_cast<const char *>(p.x) + (slot * p.x_stride + first) * kE;
    const char *pd = static_cast<const char *>(p.dout) + (slot * p.dout_stride + first) * kE;
    const char *pz = static_cast<const char *>(p.z) + (GATE ? (slot * p.z_stride + first) * kE : 0);
    char *pdx = static_cast<char *>(p.dx) + (slot * p.dx_stride + first) * kE;
    char *pdz = static_cast<char *>(p.dz) + (GATE ? (slot * p.dz_stride + first) * kE : 0);
    const int64_t sx = step * p.x_stride * kE, sd = step * p.dout_stride * kE, sz = step * p.z_stride * kE,
                  sdx = step * p.dx_stride * kE, sdz = step * p.dz_stride * kE;
    const int apart = tpr * V * kE;
    bool has[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) has[i] = (static_cast<int64_t>(i) * tpr + j) * V < p.gdim;
    // the weights stay in registers where they fit
    constexpr bool kKeep = NV * V <= 16;
    float keep[kKeep ? NV : 1][V] = {};
    if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (has[i]) load_params<V, (V > 1)>(p.weight + first + static_cast<int64_t>(i) * tpr * V, keep[i]);
    }
    auto weight = [&](int i, float (&w)[V]) {
        if constexpr (kKeep) {
#pragma unroll
            for (int e = 0; e < V; ++e) w[e] = keep[i][e];
        } else {
            if (has[i]) load_params<V, (V > 1)>(p.weight + first + static_cast<int64_t>(i) * tpr * V, w);
        }
    };
    // this thread's vector i of array a (x, dout, z) of a stage
    auto at = [&](int stage, int a, int i) -> uint4 & { return rows_smem[((stage * kArrays + a) * NV + i) * blockDim.x + threadIdx.x]; };
    auto load = [&](int stage, int64_t row) {  // the row that px, pd and pz are on; they move on
        const bool in = row < p.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool some = in && has[i];
            if constexpr (kAsync) {
                if (some) {
                    copy16_async(&at(stage, 0, i), px + i * apart);
                    copy16_async(&at(stage, 1, i), pd + i * apart);
                    if constexpr (GATE) copy16_async(&at(stage, 2, i), pz + i * apart);
                } else {
                    at(stage, 0, i) = at(stage, 1, i) = make_uint4(0, 0, 0, 0);
                    if constexpr (GATE) at(stage, 2, i) = make_uint4(0, 0, 0, 0);
                }
            } else {
                reg[0][i] = some ? R::load_raw(px + i * apart, 0) : R::zero_raw();
                reg[1][i] = some ? R::load_raw(pd + i * apart, 0) : R::zero_raw();
                if constexpr (GATE) reg[2][i] = some ? R::load_raw(pz + i * apart, 0) : R::zero_raw();
            }
        }
        if constexpr (kAsync) copy_async_commit();
        px += sx, pd += sd, pz += sz;
    };
    auto get = [&](int stage, int a, int i) -> typename R::Raw {
        if constexpr (kAsync) {
            const uint4 v = at(stage, a, i);
            typename R::Raw r;
            r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
            return r;
        } else {
            return reg[a][i];
        }
    };
    const int trips = static_cast<int>((p.rows + step - 1) / step);  // the same for every thread: all join the sums
    constexpr int kAhead = kAsync ? kStages - 1 : 0;
    if constexpr (kAhead > 0) load(0, slot);
    int64_t row = slot;
    int st = 0;
    for (int k = 0; k < trips; ++k, row += step, st = kStages - 1 - st, pdx += sdx, pdz += sdz) {
        load(kAhead > 0 ? 1 - st : 0, row + kAhead * step);  // (past the last row: zeros, so that the count of groups stays)
        if constexpr (kAsync) copy_async_wait<kAhead>();
        Ln sg[GATE ? NV : 1][kN];     // sigmoid(z)
        Ln ss2 = lanes<kL>(0.0f), dot2 = lanes<kL>(0.0f);  // sums of v^2, and of (up w) v
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float w[V] = {};
            weight(i, w);
            const typename R::Raw cx = get(st, 0, i), cd = get(st, 1, i), cz = get(st, GATE ? 2 : 0, i);
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                Ln v = R::pair(cx, e), up = R::pair(cd, e);
                if constexpr (GATE) {
                    const Ln z = R::pair(cz, e);
                    sg[i][e] = sigmoid_lanes<kAccurate, kL>(z);
                    if constexpr (GATE_FIRST) v = v * (z * sg[i][e]);
                    else up = up * (z * sg[i][e]);
                }
                ss2 = Ln::fma(v, v, ss2);
                dot2 = Ln::fma(up * Ln::of(w[e * kL], w[e * kL + kL - 1]), v, dot2);
            }
        }
        float ss = ss2.get(0), dot = dot2.get(0);
        if constexpr (kL > 1) ss += ss2.get(1), dot += dot2.get(1);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o < tpr) {
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
                dot += __shfl_xor_sync(0xffffffffu, dot, o);
            }
        if (tpr > 32) {  // one row to the block; the slots alternate, so one barrier per row is enough
            float2 *sl = slots[k & 1];
            if ((threadIdx.x & 31) == 0) sl[threadIdx.x >> 5] = make_float2(ss, dot);
            __syncthreads();
            ss = dot = 0.0f;
            for (int i = 0; i < tpr >> 5; ++i) ss += sl[i].x, dot += sl[i].y;
        }
        const float r = 1.0f / sqrtf(ss * inv + p.eps);
        const float mean = dot * r * inv;  // m(dn n)
        if (row >= p.rows) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!has[i]) continue;
            float w[V];
            Ln dx[kN], dz[kN];
            weight(i, w);
            const typename R::Raw cx = get(st, 0, i), cd = get(st, 1, i), cz = get(st, GATE ? 2 : 0, i);
            const Ln r2 = lanes<kL>(r), m2 = lanes<kL>(-mean), one = lanes<kL>(1.0f);
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                const Ln x = R::pair(cx, e), d = R::pair(cd, e), we = Ln::of(w[e * kL], w[e * kL + kL - 1]);
                if constexpr (GATE) {
                    const Ln z = R::pair(cz, e), g = sg[i][e], s = z * g;
                    const Ln ds = g * Ln::fma(z, Ln::fma(g, lanes<kL>(-1.0f), one), one);
                    if constexpr (GATE_FIRST) {
                        const Ln n = x * s * r2;
                        const Ln dv = r2 * Ln::fma(n, m2, d * we);
                        dw[i][e] = Ln::fma(d, n, dw[i][e]);
                        dx[e] = dv * s;
                        dz[e] = dv * x * ds;
                    } else {
                        const Ln n = x * r2, up = d * s;
                        dw[i][e] = Ln::fma(up, n, dw[i][e]);
                        dx[e] = r2 * Ln::fma(n, m2, up * we);
                        dz[e] = d * n * we * ds;
                    }
                } else {
                    const Ln n = x * r2;
                    dw[i][e] = Ln::fma(d, n, dw[i][e]);
                    dx[e] = r2 * Ln::fma(n, m2, d * we);
                }
            }
            R::store(pdx + i * apart, 0, dx);
            if constexpr (GATE) R::store(pdz + i * apart, 0, dz);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!has[i]) continue;
        const int64_t c = first + static_cast<int64_t>(i) * tpr * V;
#pragma unroll
        for (int e = 0; e < V; ++e) p.partial[slot * p.dim + c + e] = dw[i][e / kL].get(e % kL);
    }
}

// dweight[c] = sum over the slots of partial[slot][c], in a fixed order.  grid: dim / 32
// (`partial` is loaded from L2: its blocks come while the kernel before still writes it,
// so the read-only path, which may keep what it held before the wait, is not for it)
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float *partial, float *dweight, int64_t dim, int64_t slots) {
    __shared__ float part[32][33];
    wait_previous();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float s = 0.0f;
    if (c < dim) {
#pragma unroll 4
        for (int64_t t = threadIdx.y; t < slots; t += 32) s += __ldcg(partial + t * dim + c);
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < dim) {
        for (int r = 1; r < 32; ++r) s += part[r][threadIdx.x];
        dweight[c] = s;
    }
}

}  // namespace ssm
