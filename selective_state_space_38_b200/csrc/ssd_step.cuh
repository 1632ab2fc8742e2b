// ssd_step.cuh -- one token of the Mamba-2 SSD for every row of a decode batch,
// against float32 states in cache slots.  Per row b and head h, with
// dt = softplus(dt_raw + dt_bias[h]):
//
//   H[p][n] <- exp(dt A[h]) H[p][n] + dt x[p] B[n],   y[p] = sum_n H[p][n] C[n] + D[h] x[p]
//
// Three float32 operations for the 8 bytes that each state element moves: bound
// by HBM (two passes over the states).  Eight lanes share a row p of the state,
// each with 16 of its 128 elements as four 16-byte vectors at a stride of 128
// bytes, so a warp's load covers four whole 128-byte lines, B and C stay in
// registers for all of a thread's rows, and three shuffles finish a readout.
// Measured, 256 rows of 80 heads (1348 MB): 207 us, 6.5 TB/s, 99 % of the copy
// rate; one row of 24 heads: 7 us, launch included.
#pragma once

#include "packed.cuh"

namespace ssm {

constexpr int kSsdStepP = 64, kSsdStepN = 128;  // head and state dimensions
constexpr int kSsdStepThreads = 128;
constexpr int kSsdStepRows = 2;                                  // rows p per thread
constexpr int kSsdStepTile = kSsdStepThreads / 8 * kSsdStepRows; // rows p per block

struct SsdStepParams {
    float *states;           // [slots][H][P][N]
    const int32_t *slots;    // [batch] or NULL (row b's is b)
    const void *x, *dt, *B, *C;  // rows x_stride, dt_stride, b_stride, c_stride apart
    const float *dt_bias, *A, *D;
    void *out;               // [batch][H][P], rows out_stride apart
    int64_t x_stride, dt_stride, b_stride, c_stride, out_stride;
    int32_t nslots, heads, groups;
    int softplus;
};

// grid: batch x heads x (P / kSsdStepTile)
template <typename T>
__global__ void __launch_bounds__(kSsdStepThreads) ssd_step_kernel(const SsdStepParams p) {
    using AT = Act<T>;
    using R = Row<T, 4>;
    constexpr int kParts = kSsdStepP / kSsdStepTile;
    const uint32_t part = blockIdx.x % kParts, bh = blockIdx.x / kParts;
    const int64_t b = bh / static_cast<uint32_t>(p.heads);
    const int h = static_cast<int>(bh % static_cast<uint32_t>(p.heads));
    const int q = threadIdx.x & 7, r0 = part * kSsdStepTile + (threadIdx.x >> 3);
    const int slot = p.slots ? __ldg(p.slots + b) : static_cast<int>(b);
    if (slot < 0 || slot >= p.nslots) return;  // padding: nothing is read or written
    float *st = p.states + ((static_cast<int64_t>(slot) * p.heads + h) * kSsdStepP + r0) * kSsdStepN + 4 * q;
    // every load of the block's state is issued before its first use
    float4 s[kSsdStepRows][4];
#pragma unroll
    for (int k = 0; k < kSsdStepRows; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s[k][i] = *reinterpret_cast<const float4 *>(st + k * (kSsdStepThreads / 8) * kSsdStepN + 32 * i);
    const int g = h / (p.heads / p.groups);
    float B[4][4], C[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const typename R::Raw rb = R::load_raw(p.B, b * p.b_stride + g * kSsdStepN + 32 * i + 4 * q);
        const typename R::Raw rc = R::load_raw(p.C, b * p.c_stride + g * kSsdStepN + 32 * i + 4 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e) B[i][e] = R::get(rb, e), C[i][e] = R::get(rc, e);
    }
    float dt = AT::load(p.dt, b * p.dt_stride + h);
    if (p.dt_bias) dt += __ldg(p.dt_bias + h);
    if (p.softplus) dt = softplus_accurate(dt);  // one per thread: the states keep float32's precision
    const float a = expf(dt * __ldg(p.A + h));
    const float Dh = p.D ? __ldg(p.D + h) : 0.0f;
#pragma unroll
    for (int k = 0; k < kSsdStepRows; ++k) {
        const int row = r0 + k * (kSsdStepThreads / 8);
        const float x = AT::load(p.x, b * p.x_stride + h * kSsdStepP + row);
        const float u = dt * x;
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float4 v = s[k][i];
            v.x = fmaf(a, v.x, u * B[i][0]);
            v.y = fmaf(a, v.y, u * B[i][1]);
            v.z = fmaf(a, v.z, u * B[i][2]);
            v.w = fmaf(a, v.w, u * B[i][3]);
            *reinterpret_cast<float4 *>(st + k * (kSsdStepThreads / 8) * kSsdStepN + 32 * i) = v;
            y = fmaf(v.x, C[i][0], fmaf(v.y, C[i][1], fmaf(v.z, C[i][2], fmaf(v.w, C[i][3], y))));
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (q == 0) AT::store(p.out, b * p.out_stride + h * kSsdStepP + row, fmaf(Dh, x, y));
    }
}

}  // namespace ssm
