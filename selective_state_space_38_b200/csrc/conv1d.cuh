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
// their use to keep enough bytes in flight.  Measured, 5376 bf16 channels as slices
// of wider rows, K = 4, silu: forward of 16117 rows 70 us, 5.0 TB/s, 75 % of the
// copy rate, some 5 us of it the windows' kernel (the same walk that only copies takes
// 60 us; the rest is the latency of the 51 instructions a row and thread at 24 warps
// an SM: more warps with fewer rows ahead were slower, 77); gradients of 16384 rows 135 us, 3.9 TB/s, 60 % (some 100
// instructions a row and thread, whose 128 registers leave 16 warps an SM; issue slots
// and FMA pipe at half of their rates); one token for 256 rows 10 us, launch included.
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
    int64_t tile;         // rows of a tile
    uint32_t cblocks;     // channel blocks: block i takes channel block i % cblocks of tile (or row) i / cblocks
    int silu;
};

constexpr int kConvThreads = 64;  // (of 5376 bf16 channels forward and gradients 70 and 135 us; with 128 threads 74 and 137)
constexpr int kConvBatch = 8;   // rows loaded ahead
constexpr int kConvBwdBatch = 4;

// The sequences of a block's tile, rows counted from the tile's first (32 bits).  All
// rows are walked by every thread of the block in step, so the current sequence is
// the block's; the first 32 from the tile's start wait in shared memory, since each
// would cost dependent loads.  Rows before the first sequence's start are in none; behind
// it a sequence starts where the one before ends.
struct ConvWalk {
    int n;           // the current sequence (`sequences`: none any more)
    int start, end;  // its rows
    int slot;        // the window it goes on from, or -1
    const int *ends, *slots;
    int base;
    int64_t t0;

    __device__ __forceinline__ int rel(int64_t t) const {
        const int64_t d = t - t0;
        return static_cast<int>(d < -(1 << 30) ? -(1 << 30) : d > (1 << 30) ? (1 << 30) : d);
    }
    __device__ __forceinline__ void stage(const Conv1dParams &p, int64_t first, int *e, int *s) {
        t0 = first, ends = e, slots = s;
        n = base = packed_find(p.seq, t0);
        start = 0, end = -1, slot = -1;
        if (threadIdx.x < 32) {
            const int i = threadIdx.x, m = base + i;
            const bool in = m < p.seq.sequences;
            e[i] = in ? rel(packed_at(p.seq, m + 1)) : 0;
            s[i] = in && p.windows && p.seq.has_initial && p.seq.has_initial[m] ? packed_slot(p.seq, m) : -1;
        }
        __syncthreads();
    }
    __device__ __forceinline__ void enter(const Conv1dParams &p) {  // sequence n
        const int i = n - base;
        if (i < 32) {
            start = i > 0 ? ends[i - 1] : rel(packed_at(p.seq, n));
            end = ends[i];
            slot = slots[i];
        } else {
            start = rel(packed_at(p.seq, n));
            end = rel(packed_at(p.seq, n + 1));
            slot = p.windows && p.seq.has_initial && p.seq.has_initial[n] ? packed_slot(p.seq, n) : -1;
        }
    }
    // on to the sequence that row r is in; false: behind the last one
    __device__ __forceinline__ bool to(const Conv1dParams &p, int r) {
        do {
            if (n + 1 >= p.seq.sequences) {
                n = p.seq.sequences;
                return false;
            }
            ++n;
            enter(p);
        } while (r >= end);
        return true;
    }
};

// A thread's V channels: taps, bias and the last K - 1 inputs (h[d]: d + 1 rows back).
template <typename T, int V, int K>
struct ConvChannels {
    using R = Row<T, V>;
    static constexpr int kL = R::kL, kN = R::kN, kH = K > 1 ? K - 1 : 1;
    Lanes<kL> w[K][kN], b[kN], h[kH][kN];

    __device__ __forceinline__ void taps(const Conv1dParams &p, int64_t c) {
        float f[K * V], g[V];
        load_params<K * V, (V > 1)>(p.w + c * K, f);
        if (p.bias) {
            load_params<V, (V > 1)>(p.bias + c, g);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) g[e] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
#pragma unroll
            for (int k = 0; k < K; ++k) w[k][i] = Lanes<kL>::of(f[i * kL * K + k], f[(i * kL + kL - 1) * K + k]);
            b[i] = Lanes<kL>::of(g[i * kL], g[i * kL + kL - 1]);
        }
    }
    // The inputs before row `at` of the current sequence: its rows, before its first the
    // window it goes on from, else zeros.
    __device__ __forceinline__ void history(const Conv1dParams &p, const ConvWalk &q, int at, int64_t c) {
        const int pos = max(at - q.start, 0);
#pragma unroll
        for (int d = 0; d < K - 1; ++d) {
            typename R::Raw r = R::zero_raw();
            if (pos - d - 1 >= 0) r = R::load_raw(p.x, (q.t0 + at - d - 1) * p.x_stride + c);
            else if (q.slot >= 0) r = R::load_raw(p.windows, (static_cast<int64_t>(q.slot) * (K - 1) + (K - 1 + pos - d - 1)) * p.dim + c);
#pragma unroll
            for (int i = 0; i < kN; ++i) h[d][i] = R::pair(r, i);
        }
    }
    // u of one row; the history moves on
    __device__ __forceinline__ void row(const Lanes<kL> (&x)[kN], Lanes<kL> (&u)[kN]) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            u[i] = Lanes<kL>::fma(w[K - 1][i], x[i], b[i]);
#pragma unroll
            for (int d = 0; d < K - 1; ++d) u[i] = Lanes<kL>::fma(w[K - 2 - d][i], h[d][i], u[i]);
#pragma unroll
            for (int d = K - 2; d > 0; --d) h[d][i] = h[d - 1][i];
            if constexpr (K > 1) h[0][i] = x[i];
        }
    }
};

// grid: row tiles x channel blocks, the channel blocks of a tile next to each other
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads, 12) conv1d_fwd_kernel(const Conv1dParams p) {
    release_next();
    using R = Row<T, V>;
    constexpr bool kAccurate = Act<T>::kBytes == 4;
    constexpr int kL = R::kL, kN = R::kN;
    __shared__ int ends[32], slots[32];
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / p.cblocks) * p.tile;
    const int rows = static_cast<int>(min(p.tile, p.seq.tokens - t0));
    ConvWalk q;
    q.stage(p, t0, ends, slots);
    const int64_t c = (static_cast<int64_t>(blockIdx.x % p.cblocks) * kConvThreads + threadIdx.x) * V;
    if (q.n >= p.seq.sequences || c >= p.dim) return;
    // the rows' bytes from the tile's first
    const char *x = static_cast<const char *>(p.x) + (t0 * p.x_stride + c) * Act<T>::kBytes;
    char *y = static_cast<char *>(p.y) + (t0 * p.y_stride + c) * Act<T>::kBytes;
    const int64_t xs = p.x_stride * Act<T>::kBytes, ys = p.y_stride * Act<T>::kBytes;
    ConvChannels<T, V, K> ch;
    typename R::Raw raw[kConvBatch];
    auto load = [&](int r) {  // rows r, r + 1, ...: `x` is row r's
        if (r + kConvBatch <= rows) {
#pragma unroll
            for (int i = 0; i < kConvBatch; ++i) raw[i] = R::load_raw(x + i * xs, 0);
        } else {
#pragma unroll
            for (int i = 0; i < kConvBatch; ++i)
                if (r + i < rows) raw[i] = R::load_raw(x + i * xs, 0);
        }
        x += kConvBatch * xs;
    };
    load(0);
    q.enter(p);
    int first = 0;
    if (q.start > 0) {  // rows before the first sequence stay as they were
        first = min(q.start, rows);
        x += (first - kConvBatch) * xs, y += first * ys;
        load(first);
    }
    ch.taps(p, c);
    ch.history(p, q, first, c);
    auto row = [&](const typename R::Raw &r) {  // `y` is its row
        Lanes<kL> v[kN], u[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = R::pair(r, i);
        ch.row(v, u);
        if (p.silu) {
#pragma unroll
            for (int i = 0; i < kN; ++i) u[i] = u[i] * sigmoid_lanes<kAccurate, kL>(u[i]);
        }
        R::store(y, 0, u);
        y += ys;
    };
    for (int r = first; r < rows; r += kConvBatch) {
        typename R::Raw now[kConvBatch];
#pragma unroll
        for (int i = 0; i < kConvBatch; ++i) now[i] = raw[i];
        load(r + kConvBatch);
        if (r + kConvBatch <= min(rows, q.end)) {  // rows of one sequence: the history's moves are renamings
#pragma unroll
            for (int i = 0; i < kConvBatch; ++i) row(now[i]);
            continue;
        }
#pragma unroll
        for (int i = 0; i < kConvBatch; ++i) {
            if (r + i >= rows) break;
            if (r + i >= q.end) {
                if (!q.to(p, r + i)) return;  // rows behind the last sequence stay as they were
                ch.history(p, q, r + i, c);
            }
            row(now[i]);
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
    wait_previous();
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
    ConvChannels<T, V, K> ch;
    ch.taps(p, c);
    const int slot = packed_slot(p.seq, static_cast<int>(b));
    if (slot < 0) return;
    const int64_t win = static_cast<int64_t>(slot) * (K - 1);
    typename R::Raw old[K > 1 ? K - 1 : 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) old[j] = R::load_raw_rw(p.windows, (win + j) * p.dim + c);
    Lanes<R::kL> v[R::kN], u[R::kN];
#pragma unroll
    for (int i = 0; i < R::kN; ++i) {
        v[i] = R::pair(x, i);
#pragma unroll
        for (int d = 0; d < K - 1; ++d) ch.h[d][i] = R::pair(old[K - 2 - d], i);
    }
    ch.row(v, u);
    if (p.silu) {
#pragma unroll
        for (int i = 0; i < R::kN; ++i) u[i] = u[i] * sigmoid_lanes<kAccurate, R::kL>(u[i]);
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
__global__ void __launch_bounds__(kConvThreads, 8) conv1d_bwd_kernel(const Conv1dParams p) {
    release_next();
    using R = Row<T, V>;
    constexpr bool kAccurate = Act<T>::kBytes == 4;
    constexpr int kL = R::kL, kN = R::kN, kB = kConvBwdBatch;
    using Ln = Lanes<kL>;
    __shared__ int ends[32], slots[32];
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / p.cblocks) * p.tile;
    const int rows = static_cast<int>(min(p.tile, p.seq.tokens - t0));
    ConvWalk q;
    q.stage(p, t0, ends, slots);
    const int64_t c = (static_cast<int64_t>(blockIdx.x % p.cblocks) * kConvThreads + threadIdx.x) * V;
    if (c >= p.dim) return;
    ConvChannels<T, V, K> ch;
    Ln g[K][kN], dw[K][kN], db[kN];
    int eh[K];
#pragma unroll
    for (int d = 0; d < K; ++d) {
        eh[d] = -1;
#pragma unroll
        for (int i = 0; i < kN; ++i) g[d][i] = dw[d][i] = lanes<kL>(0.0f);
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) db[i] = lanes<kL>(0.0f);
    // the rows after the tile complete its last gradients; there may be fewer of them
    const int last = rows + K - 1, have = static_cast<int>(min(static_cast<int64_t>(last), p.seq.tokens - t0));
    const char *x = static_cast<const char *>(p.x) + (t0 * p.x_stride + c) * Act<T>::kBytes;
    const char *dy = static_cast<const char *>(p.dy) + (t0 * p.dy_stride + c) * Act<T>::kBytes;
    char *dx = static_cast<char *>(p.dx) + ((t0 - (K - 1)) * p.dx_stride + c) * Act<T>::kBytes;  // of the row whose gradient is complete
    const int64_t xs = p.x_stride * Act<T>::kBytes, dys = p.dy_stride * Act<T>::kBytes, dxs = p.dx_stride * Act<T>::kBytes;
    typename R::Raw rx[kB], rd[kB];
    auto load = [&](int r) {  // rows r, r + 1, ...: `x` and `dy` are row r's
        if (r + kB <= have) {
#pragma unroll
            for (int i = 0; i < kB; ++i) rx[i] = R::load_raw(x + i * xs, 0), rd[i] = R::load_raw(dy + i * dys, 0);
        } else {
#pragma unroll
            for (int i = 0; i < kB; ++i)
                if (r + i < have) rx[i] = R::load_raw(x + i * xs, 0), rd[i] = R::load_raw(dy + i * dys, 0);
        }
        x += kB * xs, dy += kB * dys;
    };
    load(0);
    ch.taps(p, c);
    if (q.n < p.seq.sequences) {
        q.enter(p);
        ch.history(p, q, 0, c);
    }
    // g of a row that is in a sequence, and its part of the sums
    auto row = [&](const typename R::Raw &rxi, const typename R::Raw &rdi, bool count) {
        Ln x[kN], u[kN], hx[ConvChannels<T, V, K>::kH][kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            x[i] = R::pair(rxi, i);
#pragma unroll
            for (int d = 0; d < K - 1; ++d) hx[d][i] = ch.h[d][i];
        }
        ch.row(x, u);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            Ln gv = R::pair(rdi, i);
            if (p.silu) {
                const Ln sg = sigmoid_lanes<kAccurate, kL>(u[i]);
                const Ln one = lanes<kL>(1.0f);
                gv = gv * (sg * Ln::fma(u[i], Ln::fma(sg, lanes<kL>(-1.0f), one), one));
            }
#pragma unroll
            for (int d = K - 1; d > 0; --d) g[d][i] = g[d - 1][i];
            g[0][i] = gv;
            if (count) {
                db[i] = db[i] + gv;
                dw[K - 1][i] = Ln::fma(gv, x[i], dw[K - 1][i]);
#pragma unroll
                for (int d = 0; d < K - 1; ++d) dw[K - 2 - d][i] = Ln::fma(gv, hx[d][i], dw[K - 2 - d][i]);
            }
        }
    };
    for (int r = 0; r < last; r += kB) {
        typename R::Raw nx[kB], nd[kB];
#pragma unroll
        for (int i = 0; i < kB; ++i) nx[i] = rx[i], nd[i] = rd[i];
        load(r + kB);
        // rows of one sequence whose K - 1 rows before are the same sequence's and the tile's
        if (r - (K - 1) >= max(0, q.start) && r + kB <= min(rows, q.end)) {
#pragma unroll
            for (int e = 0; e < kB; ++e) {
                row(nx[e], nd[e], true);
                Ln v[kN];
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    v[i] = ch.w[0][i] * g[0][i];
#pragma unroll
                    for (int d = 1; d < K; ++d) v[i] = Ln::fma(ch.w[d][i], g[d][i], v[i]);
                }
                R::store(dx, 0, v);
                dx += dxs;
            }
#pragma unroll
            for (int d = 0; d < K; ++d) eh[d] = q.end;
            continue;
        }
#pragma unroll
        for (int e = 0; e < kB; ++e) {
            const int s = r + e;
            if (s >= last) break;
            if (q.n < p.seq.sequences && s >= q.end && q.to(p, s)) ch.history(p, q, s, c);
            const bool live = q.n < p.seq.sequences && s >= q.start && s < have;
#pragma unroll
            for (int d = K - 1; d > 0; --d) eh[d] = eh[d - 1];
            eh[0] = live ? q.end : -1;
            if (live) {
                row(nx[e], nd[e], s < rows);
            } else {
#pragma unroll
                for (int i = 0; i < kN; ++i) {
#pragma unroll
                    for (int d = K - 1; d > 0; --d) g[d][i] = g[d - 1][i];
                    g[0][i] = lanes<kL>(0.0f);
                }
            }
            if (s >= K - 1 && eh[K - 1] >= 0) {  // the row s - (K - 1), when it is in a sequence
                Ln v[kN];
#pragma unroll
                for (int i = 0; i < kN; ++i) v[i] = lanes<kL>(0.0f);
#pragma unroll
                for (int d = 0; d < K; ++d)  // g[d] is row s - d: its tap on row s - (K - 1) is d
                    if (s - d < eh[K - 1]) {
#pragma unroll
                        for (int i = 0; i < kN; ++i) v[i] = Ln::fma(ch.w[d][i], g[d][i], v[i]);
                    }
                R::store(dx, 0, v);
            }
            dx += dxs;
        }
    }
    float *o = p.partial + static_cast<int64_t>(blockIdx.x / p.cblocks) * (K + 1) * p.dim + c;
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) o[k * p.dim + e] = (k < K ? dw[k][e / kL] : db[e / kL]).get(e % kL);
}

// dst[c * stride_c + k] = sum over tiles of partial[tile][k][c], tiles in order
// within each of the 8 rows of a block and the rows in order.  grid: (dim / 32, K + 1)
// (`partial` is loaded from L2: its blocks come while the kernel before still writes it,
// so the read-only path, which may keep what it held before the wait, is not for it)
__global__ void __launch_bounds__(256) conv1d_reduce_kernel(const float *partial, float *dw, float *dbias, int64_t dim,
                                                            int64_t tiles, int K) {
    __shared__ float part[8][32];
    wait_previous();
    const int k = blockIdx.y;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float s = 0.0f;
    if (c < dim) {
#pragma unroll 8
        for (int64_t t = threadIdx.y; t < tiles; t += 8) s += __ldcg(partial + (t * (K + 1) + k) * dim + c);
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
