// packed.cuh -- helpers of the time-major operators around the SSD: rows of
// activations read V elements at a time, and packed sequences (cu_seqlens).
#pragma once

#include "common.cuh"

namespace ssm {

// One or two float32 values that go through an operation together (two: the f32x2
// instructions, one issue slot for both, each rounded as by itself).
template <int L>
struct Lanes;
template <>
struct Lanes<1> {
    float v;
    __device__ __forceinline__ static Lanes of(float a, float) { return {a}; }
    __device__ __forceinline__ float get(int) const { return v; }
    __device__ __forceinline__ friend Lanes operator*(Lanes a, Lanes b) { return {a.v * b.v}; }
    __device__ __forceinline__ friend Lanes operator+(Lanes a, Lanes b) { return {a.v + b.v}; }
    __device__ __forceinline__ static Lanes fma(Lanes a, Lanes b, Lanes c) { return {fmaf(a.v, b.v, c.v)}; }
};
template <>
struct Lanes<2> {
    uint64_t v;
    __device__ __forceinline__ static Lanes of(float a, float b) {
        Lanes r;
        asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
        return r;
    }
    __device__ __forceinline__ float get(int i) const {
        float a, b;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
        return i ? b : a;
    }
    __device__ __forceinline__ friend Lanes operator*(Lanes a, Lanes b) {
        Lanes r;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
        return r;
    }
    __device__ __forceinline__ friend Lanes operator+(Lanes a, Lanes b) {
        Lanes r;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
        return r;
    }
    __device__ __forceinline__ static Lanes fma(Lanes a, Lanes b, Lanes c) {
        Lanes r;
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
        return r;
    }
};
template <int L>
__device__ __forceinline__ Lanes<L> lanes(float a) { return Lanes<L>::of(a, a); }

// V consecutive elements at p (aligned to V elements; V = 1, 2, 4 or, for bf16, 8)
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
        } else if constexpr (V * Act<T>::kBytes == 4) {
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
    static constexpr int kL = V % 2 == 0 ? 2 : 1, kN = V / kL;  // values that go together, and how many such
    __device__ __forceinline__ static Lanes<kL> pair(const Raw &r, int i) {
        return Lanes<kL>::of(get(r, i * kL), kL > 1 ? get(r, i * kL + kL - 1) : 0.0f);
    }
    __device__ __forceinline__ static void store(void *base, int64_t i, const Lanes<kL> (&v)[kN]) {
        float f[V];
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = v[e / kL].get(e % kL);
        store(base, i, f);
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
        } else if constexpr (Act<T>::kBytes == 4 && V == 2) {
            *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
        } else if constexpr (Act<T>::kBytes == 2 && V == 2) {
            *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(v[0], v[1]);
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
        } else if constexpr (V * Act<T>::kBytes == 4) {
            *reinterpret_cast<uint32_t *>(p) = r.w[0];
        } else {
            *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(r.w[0]);
        }
    }
};

// 16 bytes global -> shared without a register round trip.
__device__ __forceinline__ void copy16_async(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() {  // until at most N groups are pending
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The kernels of a call may follow each other by programmatic dependent launch: each lets
// the next one's blocks come while it runs, and waits for the one before to be over (its
// writes seen) before it reads anything of its.  Every block waits, also one with nothing
// to do: the kernel after takes this one's end for the end of both.
__device__ __forceinline__ void release_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// N consecutive float32 parameters: as 16-byte vectors when VEC (the host checks their
// alignment with the rows'), else one by one.
template <int N, bool VEC>
__device__ __forceinline__ void load_params(const float *p, float (&v)[N]) {
    if constexpr (VEC && N % 4 == 0) {  // (N / 4 vectors lie together, so N floats' alignment is 16 bytes)
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(p) + i);
            v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __ldg(p + i);
    }
}

// silu(v) and its derivative sg (1 + v (1 - sg)), sg = 1 / (1 + e^-v).  For
// float32 activations with expf and a true division; for bf16 with the MUFU
// forms, whose 2^-21 or so is far below the output's half step of 2^-8.
template <bool ACCURATE>
__device__ __forceinline__ float sigmoid_of(float v) {
    if constexpr (ACCURATE) return 1.0f / (1.0f + expf(-v));
    else return rcp_approx(1.0f + ex2_approx(-v * kLog2e));
}

// sigmoid of one or two values: the multiplications and the sum together.
template <bool ACCURATE, int L>
__device__ __forceinline__ Lanes<L> sigmoid_lanes(Lanes<L> v) {
    if constexpr (ACCURATE) {
        return Lanes<L>::of(sigmoid_of<true>(v.get(0)), L > 1 ? sigmoid_of<true>(v.get(L - 1)) : 0.0f);
    } else {
        const Lanes<L> t = v * lanes<L>(-kLog2e);
        const Lanes<L> e = lanes<L>(1.0f) + Lanes<L>::of(ex2_approx(t.get(0)), L > 1 ? ex2_approx(t.get(L - 1)) : 0.0f);
        return Lanes<L>::of(rcp_approx(e.get(0)), L > 1 ? rcp_approx(e.get(L - 1)) : 0.0f);
    }
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
