// conv1d.cuh -- the short causal depthwise convolution of a Mamba-2 block on
// time-major rows x[t][c] of packed sequences, its gradients, and one token.
//
//   u_t[c] = bias[c] + sum_{k < K} w[c][k] x_{t-K+1+k}[c],   y = silu(u)  (or u)
//
// where rows before the sequence's first are the K - 1 stored inputs of its
// window (oldest first), or zeros.  Gradients, with g_t = dy_t silu'(u_t):
//   dx_s = sum_k w[k] g_{s+K-1-k} (rows of the same sequence),
//   dw[k] = sum_t g_t x_{t-K+1+k},   dbias = sum_t g_t.
//
// A few operations per element: bound by HBM (forward 2, gradients 3 passes
// over the rows).  A thread owns V neighbouring channels and walks down a tile
// of rows with the last K - 1 inputs in registers, so each row is read once but
// for the K - 1 rows before a tile; the rows of a batch are loaded ahead of
// their use to keep enough bytes in flight.
#pragma once

#include "packed.cuh"

namespace ssm {

struct Conv1dParams {
    const void *x;        // [tokens][dim], rows x_stride elements apart
    const float *w;       // [dim][K]
    const float *bias;    // [dim] or NULL
    void *windows;        // [slots][K - 1][dim] or NULL
    void *y;              // [tokens][dim], rows y_stride apart
    // gradients
    const void *dy;       // rows dy_stride apart
    void *dx;             // rows dx_stride apart
    float *partial;       // [tiles][K + 1][dim]
    float *dw, *dbias;    // [dim][K], [dim] (dbias may be NULL)
    Packed seq;
    int64_t dim, x_stride, y_stride, dy_stride, dx_stride;
    int64_t tile;         // rows of a tile of the gradient kernel
    uint32_t cblocks;     // channel blocks: block i takes channel block i % cblocks of tile (or row) i / cblocks
    int silu;
};

constexpr int kConvThreads = 128;
constexpr int kConvTile = 32;   // rows of a tile of the forward kernel
constexpr int kConvBatch = 8;   // rows loaded ahead

// The K - 1 inputs before row t of sequence n (which starts at `start`): h[d]
// is the row d + 1 back.  Rows before the start come from the window when the
// sequence goes on from one.
template <typename T, int V, int K>
__device__ __forceinline__ void conv_history(const Conv1dParams &p, int n, int64_t start, int64_t t, int64_t c,
                                             float (&h)[K > 1 ? K - 1 : 1][V]) {
    if constexpr (K > 1) {
        using R = Row<T, V>;
        const int64_t pos = t > start ? t - start : 0;
        int slot = -1;
        if (pos < K - 1 && p.windows && p.seq.has_initial && p.seq.has_initial[n]) slot = packed_slot(p.seq, n);
#pragma unroll
        for (int d = 0; d < K - 1; ++d) {
            typename R::Raw r = R::zero_raw();
            if (pos - d - 1 >= 0) r = R::load_raw(p.x, (t - d - 1) * p.x_stride + c);
            else if (slot >= 0) r = R::load_raw(p.windows, (static_cast<int64_t>(slot) * (K - 1) + (K - 1 + pos - d - 1)) * p.dim + c);
#pragma unroll
            for (int e = 0; e < V; ++e) h[d][e] = R::get(r, e);
        }
    }
}

template <typename T, int V, int K>
__device__ __forceinline__ void conv_taps(const Conv1dParams &p, int64_t c, float (&w)[K][V], float (&b)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int k = 0; k < K; ++k) w[k][e] = __ldg(p.w + (c + e) * K + k);
        b[e] = p.bias ? __ldg(p.bias + c + e) : 0.0f;
    }
}

// grid: row tiles x channel blocks, the channel blocks of a tile next to each other
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads) conv1d_fwd_kernel(const Conv1dParams p) {
    using R = Row<T, V>;
    constexpr bool kAccurate = Act<T>::kBytes == 4;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / p.cblocks) * kConvTile;
    const int64_t t1 = min(t0 + kConvTile, p.seq.tokens);
    int n = packed_find(p.seq, t0);  // the whole block walks the same rows: n and its bounds are uniform
    if (n >= p.seq.sequences) return;
    const int64_t c = (static_cast<int64_t>(blockIdx.x % p.cblocks) * kConvThreads + threadIdx.x) * V;
    if (c >= p.dim) return;
    float w[K][V], b[V], h[K > 1 ? K - 1 : 1][V];
    conv_taps<T, V, K>(p, c, w, b);
    int64_t start = packed_at(p.seq, n), end = packed_at(p.seq, n + 1);
    conv_history<T, V, K>(p, n, start, t0, c, h);
    for (int64_t t = t0; t < t1; t += kConvBatch) {
        typename R::Raw raw[kConvBatch];
#pragma unroll
        for (int i = 0; i < kConvBatch; ++i)
            raw[i] = t + i < t1 ? R::load_raw(p.x, (t + i) * p.x_stride + c) : R::zero_raw();
#pragma unroll
        for (int i = 0; i < kConvBatch; ++i) {
            if (t + i >= t1) break;
            if (t + i >= end) {
                do {
                    if (++n >= p.seq.sequences) return;  // rows behind the last sequence stay as they were
                    start = packed_at(p.seq, n);
                    end = packed_at(p.seq, n + 1);
                } while (t + i >= end);
                conv_history<T, V, K>(p, n, start, t + i, c, h);
            }
            float y[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float x = R::get(raw[i], e);
                float u = fmaf(w[K - 1][e], x, b[e]);
#pragma unroll
                for (int d = 0; d < K - 1; ++d) u = fmaf(w[K - 2 - d][e], h[d][e], u);
#pragma unroll
                for (int d = K - 2; d > 0; --d) h[d][e] = h[d - 1][e];
                if constexpr (K > 1) h[0][e] = x;
                y[e] = p.silu ? u * sigmoid_of<kAccurate>(u) : u;
            }
            R::store(p.y, (t + i) * p.y_stride + c, y);
        }
    }
}

// The window after each sequence: its last K - 1 inputs (of the old window when
// the sequence is shorter).  A kernel of its own, after the convolution: the
// first rows' tile reads the old window and the last rows' tile would write it.
// grid: sequences x channel blocks
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads) conv1d_window_kernel(const Conv1dParams p) {
    using R = Row<T, V>;
    const int64_t c = (static_cast<int64_t>(blockIdx.x % p.cblocks) * kConvThreads + threadIdx.x) * V;
    if (c >= p.dim) return;
    {
        const int n = static_cast<int>(blockIdx.x / p.cblocks);
        const int slot = packed_slot(p.seq, n);
        const int64_t start = packed_at(p.seq, n), len = packed_at(p.seq, n + 1) - start;
        if (slot < 0 || len <= 0) return;
        const bool init = p.seq.has_initial && p.seq.has_initial[n];
        const int64_t win = static_cast<int64_t>(slot) * (K - 1);
        typename R::Raw v[K > 1 ? K - 1 : 1];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int64_t pos = len - (K - 1) + j;
            v[j] = R::zero_raw();
            if (pos >= 0) v[j] = R::load_raw(p.x, (start + pos) * p.x_stride + c);
            else if (init) v[j] = R::load_raw_rw(p.windows, (win + K - 1 + pos) * p.dim + c);
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) R::store_raw(p.windows, (win + j) * p.dim + c, v[j]);
    }
}

// One token per sequence: row b of x through the window of its slot, which moves
// on by one input.  A row whose slot is outside the cache is padding: its row of
// y stays as it was.  grid: rows x channel blocks
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads) conv1d_step_kernel(const Conv1dParams p) {
    using R = Row<T, V>;
    constexpr bool kAccurate = Act<T>::kBytes == 4;
    const int64_t c = (static_cast<int64_t>(blockIdx.x % p.cblocks) * kConvThreads + threadIdx.x) * V;
    if (c >= p.dim) return;
    const int64_t b = blockIdx.x / p.cblocks;
    const typename R::Raw x = R::load_raw(p.x, b * p.x_stride + c);
    float w[K][V], u[V];
    conv_taps<T, V, K>(p, c, w, u);
    const int slot = packed_slot(p.seq, static_cast<int>(b));
    if (slot < 0) return;
    const int64_t win = static_cast<int64_t>(slot) * (K - 1);
    typename R::Raw old[K > 1 ? K - 1 : 1];
    if constexpr (K > 1) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) old[j] = R::load_raw_rw(p.windows, (win + j) * p.dim + c);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) u[e] = fmaf(w[j][e], R::get(old[j], e), u[e]);
        u[e] = fmaf(w[K - 1][e], R::get(x, e), u[e]);
        if (p.silu) u[e] *= sigmoid_of<kAccurate>(u[e]);
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j) R::store_raw(p.windows, (win + j) * p.dim + c, j + 1 < K - 1 ? old[j + 1] : x);
    R::store(p.y, b * p.y_stride + c, u);
}

// Gradients.  A thread walks its tile's rows and K - 1 rows on: g_t is formed
// from the recomputed u_t, dx_{t-K+1} is complete at row t.  eh[d] is the end of
// row t - d's sequence (-1: none), so that no gradient crosses into another
// sequence's rows.  The sums over the tile's rows stay in registers and go to
// `partial`, which conv1d_reduce_kernel adds in a fixed order: the result does
// not depend on the order in which blocks run.
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads) conv1d_bwd_kernel(const Conv1dParams p) {
    using R = Row<T, V>;
    constexpr bool kAccurate = Act<T>::kBytes == 4;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / p.cblocks) * p.tile;
    const int64_t t1 = min(t0 + p.tile, p.seq.tokens);
    int n = packed_find(p.seq, t0);
    const int64_t c = (static_cast<int64_t>(blockIdx.x % p.cblocks) * kConvThreads + threadIdx.x) * V;
    if (c >= p.dim) return;
    float w[K][V], b[V], h[K > 1 ? K - 1 : 1][V], g[K][V] = {}, dw[K][V] = {}, db[V] = {};
    conv_taps<T, V, K>(p, c, w, b);
    int64_t start = 0, end = -1, eh[K];
#pragma unroll
    for (int d = 0; d < K; ++d) eh[d] = -1;
    if (n < p.seq.sequences) {
        start = packed_at(p.seq, n);
        end = packed_at(p.seq, n + 1);
        conv_history<T, V, K>(p, n, start, t0, c, h);
    }
    const int64_t last = t1 + K - 1;  // the rows after the tile complete its last gradients
    for (int64_t t = t0; t < last; t += 4) {
        typename R::Raw rx[4], rd[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = t + i < last && t + i < p.seq.tokens;
            rx[i] = in ? R::load_raw(p.x, (t + i) * p.x_stride + c) : R::zero_raw();
            rd[i] = in ? R::load_raw(p.dy, (t + i) * p.dy_stride + c) : R::zero_raw();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t s = t + i;
            if (s >= last) break;
            if (n < p.seq.sequences && s >= end) {
                do {
                    if (++n >= p.seq.sequences) break;
                    start = packed_at(p.seq, n);
                    end = packed_at(p.seq, n + 1);
                } while (s >= end);
                if (n < p.seq.sequences) conv_history<T, V, K>(p, n, start, s, c, h);
            }
            const bool live = n < p.seq.sequences && s < p.seq.tokens;
#pragma unroll
            for (int d = K - 1; d > 0; --d) {
                eh[d] = eh[d - 1];
#pragma unroll
                for (int e = 0; e < V; ++e) g[d][e] = g[d - 1][e];
            }
            eh[0] = live ? end : -1;
            if (live) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float x = R::get(rx[i], e), dy = R::get(rd[i], e);
                    float u = fmaf(w[K - 1][e], x, b[e]);
#pragma unroll
                    for (int d = 0; d < K - 1; ++d) u = fmaf(w[K - 2 - d][e], h[d][e], u);
                    float gv = dy;
                    if (p.silu) {
                        const float sg = sigmoid_of<kAccurate>(u);
                        gv = dy * (sg * fmaf(u, 1.0f - sg, 1.0f));
                    }
                    g[0][e] = gv;
                    if (s < t1) {
                        db[e] += gv;
                        dw[K - 1][e] = fmaf(gv, x, dw[K - 1][e]);
#pragma unroll
                        for (int d = 0; d < K - 1; ++d) dw[K - 2 - d][e] = fmaf(gv, h[d][e], dw[K - 2 - d][e]);
                    }
#pragma unroll
                    for (int d = K - 2; d > 0; --d) h[d][e] = h[d - 1][e];
                    if constexpr (K > 1) h[0][e] = x;
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) g[0][e] = 0.0f;
            }
            const int64_t r = s - (K - 1);  // the row whose gradient is complete
            if (r >= t0 && eh[K - 1] >= 0) {
                float dx[V] = {};
#pragma unroll
                for (int d = 0; d < K; ++d)  // g[d] is row s - d; its tap on row r is K - 1 - (K - 1 - d) = d
                    if (s - d < eh[K - 1]) {
#pragma unroll
                        for (int e = 0; e < V; ++e) dx[e] = fmaf(w[d][e], g[d][e], dx[e]);
                    }
                R::store(p.dx, r * p.dx_stride + c, dx);
            }
        }
    }
    float *q = p.partial + static_cast<int64_t>(blockIdx.x / p.cblocks) * (K + 1) * p.dim + c;
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) q[k * p.dim + e] = k < K ? dw[k][e] : db[e];
}

// dst[c * stride_c + k] = sum over tiles of partial[tile][k][c], tiles in order
// within each of the 8 rows of a block and the rows in order.  grid: (dim / 32, K + 1)
__global__ void __launch_bounds__(256) conv1d_reduce_kernel(const float *partial, float *dw, float *dbias, int64_t dim,
                                                            int64_t tiles, int K) {
    __shared__ float part[8][32];
    const int k = blockIdx.y;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float s = 0.0f;
    if (c < dim) {
#pragma unroll 8
        for (int64_t t = threadIdx.y; t < tiles; t += 8) s += __ldg(partial + (t * (K + 1) + k) * dim + c);
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < dim) {
        for (int r = 1; r < 8; ++r) s += part[r][threadIdx.x];
        if (k < K) dw[c * K + k] = s;
        else if (dbias) dbias[c] = s;
    }
}

}  // namespace ssm
