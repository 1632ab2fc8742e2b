// packed.cuh -- helpers of the time-major operators around the SSD: rows of
// activations read V elements at a time, and packed sequences (cu_seqlens).
#pragma once

#include "common.cuh"

namespace ssm {

// V consecutive elements at p (aligned to V elements; V = 1, 4 or, for bf16, 8)
// as floats, and back.
template <typename T, int V>
struct Row {
    // V elements as they are in memory
    struct Raw {
        uint32_t w[V * Act<T>::kBytes >= 4 ? V * Act<T>::kBytes / 4 : 1];
    };
    // CONST: the kernel does not write these bytes (the read-only path); else a plain load
    template <bool CONST = true>
    __device__ __forceinline__ static Raw load_raw(const void *base, int64_t i) {
        Raw r;
        const char *p = static_cast<const char *>(base) + i * Act<T>::kBytes;
        if constexpr (V * Act<T>::kBytes == 16) {
            const uint4 *q = reinterpret_cast<const uint4 *>(p);
            const uint4 v = CONST ? __ldg(q) : *q;
            r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
        } else if constexpr (V * Act<T>::kBytes == 8) {
            const uint2 *q = reinterpret_cast<const uint2 *>(p);
            const uint2 v = CONST ? __ldg(q) : *q;
            r.w[0] = v.x, r.w[1] = v.y;
        } else if constexpr (Act<T>::kBytes == 4) {
            const uint32_t *q = reinterpret_cast<const uint32_t *>(p);
            r.w[0] = CONST ? __ldg(q) : *q;
        } else {
            const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
            r.w[0] = CONST ? __ldg(q) : *q;
        }
        return r;
    }
    __device__ __forceinline__ static Raw load_raw_rw(const void *base, int64_t i) { return load_raw<false>(base, i); }
    __device__ __forceinline__ static Raw zero_raw() {
        Raw r;
#pragma unroll
        for (uint32_t &w : r.w) w = 0;
        return r;
    }
    __device__ __forceinline__ static float get(const Raw &r, int e) {
        if constexpr (Act<T>::kBytes == 4) return __uint_as_float(r.w[e]);
        else if constexpr (V == 1) return __uint_as_float(r.w[0] << 16);
        else return (e & 1) ? __uint_as_float(r.w[e / 2] & 0xffff0000u) : __uint_as_float(r.w[e / 2] << 16);
    }
    // one rounding (to nearest even) when T is bf16
    __device__ __forceinline__ static void store(void *base, int64_t i, const float (&v)[V]) {
        char *p = static_cast<char *>(base) + i * Act<T>::kBytes;
        if constexpr (Act<T>::kBytes == 4 && V == 4) {
            *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        } else if constexpr (Act<T>::kBytes == 2 && V == 8) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                       pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        } else if constexpr (Act<T>::kBytes == 2 && V == 4) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) Act<T>::store(base, i + e, v[e]);
        }
    }
    __device__ __forceinline__ static void store_raw(void *base, int64_t i, const Raw &r) {
        char *p = static_cast<char *>(base) + i * Act<T>::kBytes;
        if constexpr (V * Act<T>::kBytes == 16) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        } else if constexpr (V * Act<T>::kBytes == 8) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(r.w[0], r.w[1]);
        } else if constexpr (Act<T>::kBytes == 4) {
            *reinterpret_cast<uint32_t *>(p) = r.w[0];
        } else {
            *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(r.w[0]);
        }
    }
};

// silu(v) and its derivative sg (1 + v (1 - sg)), sg = 1 / (1 + e^-v).  For
// float32 activations with expf and a true division; for bf16 with the MUFU
// forms, whose 2^-21 or so is far below the output's half step of 2^-8.
template <bool ACCURATE>
__device__ __forceinline__ float sigmoid_of(float v) {
    if constexpr (ACCURATE) return 1.0f / (1.0f + expf(-v));
    else return rcp_approx(1.0f + ex2_approx(-v * kLog2e));
}

// Packed sequences: cu[0..n], where sequence i is rows [cu[i], cu[i + 1]).  The
// values are device data that the host cannot check, so every one is clamped to
// [0, tokens] here: a bad table gives wrong rows, never an access out of range.
struct Packed {
    const int32_t *cu;          // [sequences + 1]
    const int32_t *slots;       // [sequences] rows of the cache, or NULL (slot i = sequence i)
    const uint8_t *has_initial; // [sequences] or NULL (none)
    int64_t tokens;
    int32_t sequences, nslots;
};

__device__ __forceinline__ int64_t packed_at(const Packed &p, int i) {
    const int64_t v = __ldg(p.cu + i);
    return v < 0 ? 0 : v > p.tokens ? p.tokens : v;
}

// The cache row of sequence i, or -1 when it has none (a slot outside the cache
// stands for padding: nothing is read or written there).
__device__ __forceinline__ int packed_slot(const Packed &p, int i) {
    const int s = p.slots ? __ldg(p.slots + i) : i;
    return s >= 0 && s < p.nslots ? s : -1;
}

// The first sequence that ends after row t (`sequences` when none does): the
// count of those that end at or before it, one warp together.
__device__ __forceinline__ int packed_find(const Packed &p, int64_t t) {
    int c = 0;
    for (int i = threadIdx.x & 31; i < p.sequences; i += 32) c += packed_at(p, i + 1) <= t;
    return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(c)));
}

}  // namespace ssm
