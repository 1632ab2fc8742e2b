// ssd_varlen.cuh -- the Mamba-2 SSD over packed sequences of different lengths,
// with float32 states in cache slots, on the 5th-generation tensor cores.
//
//   H_t = exp(dt_t A) H_{t-1} + dt_t x_t B_t^T,   y_t = H_t C_t + D x_t   per head
//
// over chunks of Q = 128 steps.  With d_i = cs_i - cs_last (cs the running sum of
// dt A in the chunk, T its last value) and S the state before the chunk:
//
//   Yd_i  = sum_{j <= i} (C_i . B_j) exp(d_i - d_j) dt_j x_j,   Yo_i = C_i S
//   y_i   = Yd_i + exp(d_i + T) Yo_i + D x_i
//   S_new = exp(T) S + sum_j exp(-d_j) dt_j x_j B_j^T
//
// C B^T is the same for every head of a group: it is formed once for the two heads
// that a CTA walks together.  Where |d| stays below kVarRange = 80 the decays
// factor, exp(d_i - d_j) dt_j = exp(d_i) w_j with w_j = exp(-d_j) dt_j, the same
// w_j that scales x for the state; else they are taken element by element.  (With
// softplus d runs one way, so the factors' product stays below e^80 even where the
// mask drops it; without it the limit is half of that.  The
// row factor is not left to the end, though that would save the per-head matrix:
// the tensor core aligns a sum's products to the largest, and counts a masked zero
// as 2^-126 times its x; with x scaled over e^110 the first rows of a chunk came
// out wrong by their whole value, and shorter chunks made heads of strong decay
// the longest chain.)  The state accumulates in tensor memory on exp(T) S itself.
//
// Roundings to bf16 are those of the tensor core's operands: C B^T with its decays
// once, S once where it meets C (each at most the half step that y's own rounding
// is), and exp(-d) dt x as a sum of three bf16 parts, 24 bits, where it meets B.
// The state itself stays float32.  d is summed from the chunk's end, so the steps
// that count most for the state have the smallest rounding.
//
// Per pair of heads and chunk: 96 KB loaded through TMA and six products of
// 128 x 128 x 128, 3072 cycles of the tensor pipe at 8192 bf16 flops a cycle;
// shared memory carries about 670 KB for them and their operands, 5200 cycles at
// 128 bytes a cycle, which bounds the chunk.  One CTA per SM: one warp issues the
// TMA loads and one the MMAs, a table warp walks the work list a chunk ahead
// (running sums and factors), and sixteen epilogue warps work in two halves: eight
// on the state (S and its operand, the parts of x), eight on the output (C B^T with
// its decays, y), so that a chunk's y is written while the next one's state and
// operands are formed.  Every wait is bounded.
//
// Long sequences are cut into segments.  Chained, a segment waits for the state of
// the one before; where that would leave SMs idle (few heads, long sequences) the
// setup kernel chooses the two-pass schedule instead: the segments' own states
// first, from zeros and without outputs, all at once, then the states at their
// starts (ssd_varlen_combine_kernel), then every segment by itself.
#pragma once

#include <cuda.h>

#include "packed.cuh"
#include "tcgen05.cuh"

namespace ssm {

constexpr int kVarQ = 128;          // steps of a chunk at most
constexpr int kVarSegment = 1024;   // tokens of a work item at least (all but a sequence's last)
constexpr int kVarMaxWindows = 1024;
constexpr float kVarRange = 80.0f;
constexpr int kVarHalf = 256;       // epilogue threads on the state, and on the output
constexpr int kVarThreads = 2 * kVarHalf + 96;  // + a warp for the MMAs, the loads and the tables each
constexpr int kVarHeads = 2;        // heads walked together
constexpr int kVarParts = 3;        // bf16 parts of exp(-d) dt x

// Workspace: header (error word at 16, where ssm_scan_fwd_status reads it), the
// work list's later segments, and for each of them (by the window of `segment`
// tokens it starts in) a flag per pair, a decay and a state per head.
struct VarWork {
    uint32_t *queue, *error, *extras;  // item counters of the passes (2); error word; later segments
    uint32_t *several, *parallel;      // sequences of more than one segment; the two-pass schedule
    int2 *list;                        // [windows] (sequence, segment) of the later segments
    uint32_t *flags;                   // [windows][pairs] the state at the segment's start is written
    float *decay;                      // [windows][heads] of the segment before it
    float *carry;                      // [windows][heads][P][N] the state at its start
};

struct VarMaps {
    CUtensorMap x, B, C;  // [tokens][heads or groups][64 or 128], boxes of 64 x 1 x 128 rows
};

struct VarParams {
    const void *dt;
    const float *dt_bias, *A, *D;
    float *states;          // [slots][H][P][N] or NULL
    void *y;                // [tokens][H][P], rows y_stride apart
    Packed seq;
    VarWork work;
    int64_t dt_stride, y_stride;
    int32_t heads, groups, pairs;  // pairs: of all groups
    int32_t segment, windows, sms;
    uint32_t flag_want, spin_limit;
    int softplus;
};

// What the table warp hands on with each chunk.
struct VarChunk {
    int32_t t0, rows;        // first token, steps
    int32_t h0, nh, g;       // first head, heads (1 or 2), group
    int32_t first, last;     // of the item
    int32_t stop;
    const float *src;        // the state before the item, or NULL (zeros)
    float *dst;              // where its state goes, or NULL
    uint32_t *flag;          // hand-off: set once dst is written, or NULL
    float decay[2], total[2], D[2];  // exp(T), T
    int32_t factored[2];
};

// A segment of a sequence for a pair of heads, as the table warp sees it (A, bias
// and D: of the lane's head).
struct VarItem {
    bool valid, more;        // more: the sequence goes on behind it
    int32_t h0, nh, g, seg;
    int64_t first, stop, window;  // window: of the segment's start
    float *state;
    const float *src;
    float A, bias, D;
};

struct VarSmem {
    static constexpr int kTile = 128 * 128;           // [128 rows][64] bf16, 128-byte swizzle
    static constexpr int kC = 0, kB = 2 * kTile;      // [t][n]: n < 64, n >= 64
    static constexpr int kX = 4 * kTile;              // [t][p] of each head
    static constexpr int kXp = 6 * kTile;             // exp(-d) dt x: parts x heads tiles
    static constexpr int kS = kXp + kVarParts * kVarHeads * kTile;  // S [n][p] of each head
    static constexpr int kTabD = kS + kVarHeads * kTile;            // d [head][128]
    static constexpr int kTabW = kTabD + kVarHeads * 512;           // w where the decays factor, else dt
    static constexpr int kInfo = kTabW + kVarHeads * 512;
    static constexpr int kBar = kInfo + 256;                        // of even and of odd chunks
    static constexpr int kTotal = kBar + 128;
};
static_assert(sizeof(VarChunk) <= 128, "");
static_assert(VarSmem::kTotal <= 227 * 1024, "shared memory of the packed SSD kernel");

// The work list: one segment per sequence first, then the later segments of the
// longer ones by their number, so that a segment's predecessor always stands
// before it.  Two later segments never start in the same window of `segment`
// tokens (those of one sequence are `segment` apart, those of the next sequence
// start more than that behind its start), so a window's index names one.  One block.
__global__ void __launch_bounds__(1024) ssd_varlen_setup_kernel(const VarParams p) {
    __shared__ int2 at[kVarMaxWindows];
    __shared__ uint32_t later, several, filled, bad;
    __shared__ int longest;
    if (threadIdx.x == 0) later = 0, several = 0, filled = 0, bad = 0, longest = 1;
    for (int k = threadIdx.x; k < p.windows; k += blockDim.x) at[k] = make_int2(-1, 0);
    for (int k = threadIdx.x; k < p.windows * p.pairs; k += blockDim.x) p.work.flags[k] = 0;
    __syncthreads();
    for (int n = threadIdx.x; n < p.seq.sequences; n += blockDim.x) {
        const int32_t a = p.seq.cu[n], b = p.seq.cu[n + 1];
        if (a < 0 || b < a || b > p.seq.tokens) {
            bad = 1;
            continue;
        }
        const int segs = (b - a + p.segment - 1) / p.segment;
        for (int s = 1; s < segs; ++s) at[a / p.segment + s] = make_int2(n, s);  // the window of a + s segment
        if (segs > 0) atomicAdd(&filled, 1u);
        if (segs > 1) {
            atomicAdd(&several, 1u);
            atomicMax(&longest, segs);
        }
    }
    __syncthreads();
    for (int k = threadIdx.x; k < p.windows; k += blockDim.x) {
        const int2 v = at[k];
        if (v.x < 0) continue;
        int rank = 0;
        for (int o = 0; o < p.windows; ++o)
            rank += at[o].x >= 0 && (at[o].y < v.y || (at[o].y == v.y && o < k));
        p.work.list[rank] = v;
        atomicAdd(&later, 1u);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        p.work.queue[0] = p.work.queue[1] = 0;
        *p.work.extras = later;
        *p.work.several = several;
        // the chain of the longest sequence against the segments that each SM takes, with
        // half as much again for the first pass and two segments for its launches
        const int64_t items = static_cast<int64_t>(filled + later) * p.pairs;
        *p.work.parallel = p.flag_want == 1u && 2ll * longest * p.sms > 3ll * items + 4ll * p.sms;
        *p.work.error = bad ? 4u : 0u;  // a table that does not ascend within the tokens: nothing is run
    }
}

// The states at the segments' starts from the segments' own: S_{s+1} = exp(T_s) S_s
// + E_s, in place.  grid: (heads x 8, sequences of more than one segment at most)
__global__ void __launch_bounds__(256) ssd_varlen_combine_kernel(const VarParams p) {
    if ((*p.work.error & 4u) || !*p.work.parallel) return;
    const int h = blockIdx.x / 8;
    const int64_t e = (blockIdx.x % 8) * 256 + threadIdx.x;  // a 16-byte vector of the state
    for (uint32_t i = blockIdx.y; i < *p.work.several; i += gridDim.y) {
        const int n = p.work.list[i].x;  // the second segments come first in the list
        const int64_t begin = p.seq.cu[n], end = p.seq.cu[n + 1];
        const int segs = static_cast<int>((end - begin + p.segment - 1) / p.segment);
        const int slot = p.states ? packed_slot(p.seq, n) : -1;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (slot >= 0 && p.seq.has_initial && p.seq.has_initial[n])
            s = reinterpret_cast<const float4 *>(p.states + (static_cast<int64_t>(slot) * p.heads + h) * (kSsdP * kSsdN))[e];
#pragma unroll 4
        for (int k = 1; k < segs; ++k) {
            const int64_t at = (begin / p.segment + k) * p.heads + h;
            float4 *c = reinterpret_cast<float4 *>(p.work.carry + at * (kSsdP * kSsdN)) + e;
            const float a = p.work.decay[at];
            const float4 v = *c;
            s.x = fmaf(a, s.x, v.x), s.y = fmaf(a, s.y, v.y), s.z = fmaf(a, s.z, v.z), s.w = fmaf(a, s.w, v.w);
            *c = s;
        }
    }
}

// SUMMARY: the first pass of the two-pass schedule, which forms the segments' own
// states only; nothing to do when the setup kernel chose the chained schedule.
template <bool SUMMARY>
__global__ void __launch_bounds__(kVarThreads, 1)
    ssd_varlen_kernel(const VarParams p, const __grid_constant__ VarMaps tm) {
    extern __shared__ __align__(1024) uint8_t var_smem[];
    using S = VarSmem;
    uint8_t *sm = var_smem;
    float *tabD = reinterpret_cast<float *>(sm + S::kTabD), *tabW = reinterpret_cast<float *>(sm + S::kTabW);
    VarChunk *info = reinterpret_cast<VarChunk *>(sm + S::kInfo);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + S::kBar);
    uint64_t *bFull = bar, *bX = bar + 1;                          // tables and info written; X landed
    uint64_t *mG = bar + 2, *mC = bar + 3, *mS = bar + 4, *mY = bar + 5;  // C B^T; C S; the state; Yd done
    uint64_t *bCB = bar + 6;                                       // C and B landed
    uint64_t *bEmpty = bar + 7;                                    // info read by everyone, tables done with
    uint64_t *bS = bar + 8, *bE1 = bar + 9, *bOut = bar + 10;      // S; the parts of x; a handed-on state written
    uint64_t *bE2 = bar + 11, *bYf = bar + 12;                     // C B^T with its decays written; y out of the S tile
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + 13);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t *error = p.work.error;

    // the swizzled tiles need 1024-byte alignment; a work list that was refused has no items
    if ((smem_u32(sm) & 1023u) != 0) {
        if (tid == 0) atomicOr(error, 2u);
        return;
    }
    if (*reinterpret_cast<volatile uint32_t *>(error) & 4u) return;
    const bool parallel = *reinterpret_cast<volatile uint32_t *>(p.work.parallel) != 0;
    if (SUMMARY && !parallel) return;
    if (tid == 0) {
        for (int i = 0; i < 13; ++i) {
            const uint32_t n = i == 7 ? (SUMMARY ? 1 : 2) * kVarHalf + 2 : i > 7 ? kVarHalf : i == 6 && !SUMMARY ? 2 : 1;
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar + i)), "r"(n));
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tslot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tbase = *reinterpret_cast<volatile uint32_t *>(tslot);
    // TMEM columns: C B^T (128; its two heads' matrices replace it, as bf16 pairs: of
    // every 16 columns the first 8 for head 0, the others for head 1), Yd, Yo and S (128
    // each: head h's column p in 64 h + p; lane n holds S[p][n])
    const uint32_t tG = tbase, tYd = tbase + 128, tYo = tbase + 256, tS = tbase + 384;
    constexpr int kN = 64 * kVarHeads;

    // The waits of the two issuing warps, which stay converged: a bounded one, and a test.
    auto wait = [&](uint64_t *b, uint32_t ph) -> bool { return __all_sync(0xffffffffu, ssd_wait(b, ph, error)); };
    auto test = [&](uint64_t *b, uint32_t ph) -> bool { return __any_sync(0xffffffffu, ssd_try(smem_u32(b), ph)); };
    auto give_up = [&](uint32_t n) -> bool {  // after n tests in vain
        if (n >= kSsdWaitLimit && lane == 0) atomicOr(error, 2u);
        return n >= kSsdWaitLimit || ((n & 1023u) == 1023u && __any_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(error) != 0));
    };
    if (warp == 2 * kVarHalf / 32) {
        // ---- the products, issued by one elected lane -----------------------------------
        const uint32_t aC = smem_u32(sm + S::kC), aB = smem_u32(sm + S::kB), aX = smem_u32(sm + S::kX),
                       aXp = smem_u32(sm + S::kXp), aS = smem_u32(sm + S::kS);
        uint32_t nG = 0, nC = 0, nS = 0, nY = 0;  // issued
        for (uint32_t u = 0;; ++u) {
            const uint32_t ph = u & 1u;
            if (!wait(bFull, ph)) break;
            const int heads = info[ph].nh;
            const bool stop = info[ph].stop;
            __syncwarp();
            if (lane == 0) ssd_arrive(bEmpty);
            // (Yd before has read what C B^T replaces: mY)
            if (stop || !wait(bCB, ph) || (!SUMMARY && u > 0 && !wait(mY, ph ^ 1u))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if constexpr (!SUMMARY) {
                if (ssd_elect()) {  // C B^T
                    constexpr uint32_t id = ssd_idesc(128, 128, 0, 0);
                    const uint64_t dC = ssd_desc(aC, 16, 1024), dB = ssd_desc(aB, 16, 1024);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t o = ((k / 4) * S::kTile + (k % 4) * 32) >> 4;
                        ssd_mma(tG, dC + o, dB + o, id, k > 0);
                    }
                    ssd_commit(mG);
                }
                __syncwarp();
                nG = u + 1;
                if (!wait(bS, ph)) break;  // (S is written after the y before was read)
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                if (ssd_elect()) {  // Yo = C S
                    constexpr uint32_t id = ssd_idesc(128, kN, 0, 1);
                    const uint64_t dC = ssd_desc(aC, 16, 1024), dS = ssd_desc(aS, S::kTile, 1024);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        ssd_mma(tYo, dC + (((k / 4) * S::kTile + (k % 4) * 32) >> 4), dS + ((2048 * k) >> 4), id, k > 0);
                    ssd_commit(mC);
                }
                __syncwarp();
                nC = u + 1;
            }
            // the state's products and Yd, whichever has its operands first
            bool state = false, yd = SUMMARY;
            for (uint32_t n = 0; !(state && yd) && !give_up(n); ++n) {
                if (!state && test(bE1, ph)) {
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    if (ssd_elect()) {  // S += B^T (exp(-d) dt x), the smallest part first
                        constexpr uint32_t id = ssd_idesc(128, kN, 1, 1);
                        const uint64_t dB = ssd_desc(aB, S::kTile, 1024), dX = ssd_desc(aXp, S::kTile, 1024);
#pragma unroll
                        for (int part = kVarParts - 1; part >= 0; --part)
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                ssd_mma(tS, dB + ((2048 * k) >> 4), dX + ((part * kVarHeads * S::kTile + 2048 * k) >> 4), id, 1);
                        ssd_commit(mS);
                    }
                    __syncwarp();
                    state = true;
                    nS = u + 1;
                }
                if (!SUMMARY && !yd && test(bE2, ph)) {
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    if (ssd_elect()) {  // Yd = (C B^T with its decays) x, per head
                        constexpr uint32_t id = ssd_idesc(128, 64, 0, 1);
                        const uint64_t dX = ssd_desc(aX, S::kTile, 1024);
#pragma unroll
                        for (int i = 0; i < kVarHeads; ++i)
                            if (i < heads) {
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    ssd_mma_ts(tYd + 64 * i, tG + 16 * k + 8 * i, dX + ((i * S::kTile + 2048 * k) >> 4), id, k > 0);
                            }
                        ssd_commit(mY);
                    }
                    __syncwarp();
                    yd = true;
                    nY = u + 1;
                }
            }
            if (!(state && yd)) break;
        }
        // nothing in flight when the CTA ends (a phase that was waited for before is over: the
        // test of its parity says so at once)
        if (nG > 0) ssd_drain(mG, (nG - 1) & 1u, error);
        if (nC > 0) ssd_drain(mC, (nC - 1) & 1u, error);
        if (nS > 0) ssd_drain(mS, (nS - 1) & 1u, error);
        if (nY > 0) ssd_drain(mY, (nY - 1) & 1u, error);
        __syncwarp();
    } else if (warp == 2 * kVarHalf / 32 + 2) {
        // ---- the loads: C once C S has read the chunk's before, B once its state's products
        // have, X once its Yd and the epilogue have ---------------------------------------
        uint32_t nX = 0, nCB = 0;  // issued in full
        bool half = false;         // C is on its way without B
        for (uint32_t u = 0;; ++u) {
            const uint32_t ph = u & 1u, pv = ph ^ 1u;
            if (!wait(bFull, ph)) break;
            const int t0 = info[ph].t0, h0 = info[ph].h0, nh = info[ph].nh, g = info[ph].g;
            const bool stop = info[ph].stop;
            __syncwarp();
            if (lane == 0) ssd_arrive(bEmpty);
            if (stop) break;
            bool c = SUMMARY, b = false, x = false;
            for (uint32_t n = 0; !(c && b && x) && !give_up(n); ++n) {
                if (!SUMMARY && !c && (u == 0 || test(mC, pv))) {
                    if (ssd_elect()) {
                        mbar_arrive_expect_tx(bCB, 2 * S::kTile);
                        tma_load_3d(sm + S::kC, &tm.C, 0, g, t0, bCB);
                        tma_load_3d(sm + S::kC + S::kTile, &tm.C, 64, g, t0, bCB);
                    }
                    __syncwarp();
                    c = half = true;
                }
                if (!b && c && (u == 0 || test(mS, pv))) {
                    if (ssd_elect()) {
                        mbar_arrive_expect_tx(bCB, 2 * S::kTile);
                        tma_load_3d(sm + S::kB, &tm.B, 0, g, t0, bCB);
                        tma_load_3d(sm + S::kB + S::kTile, &tm.B, 64, g, t0, bCB);
                    }
                    __syncwarp();
                    b = true;
                    half = false;
                    ++nCB;
                }
                if (!x && (u == 0 || (test(bE1, pv) && (SUMMARY || test(mY, pv))))) {
                    if (ssd_elect()) {
                        mbar_arrive_expect_tx(bX, nh * S::kTile);
                        for (int i = 0; i < nh; ++i) tma_load_3d(sm + S::kX + i * S::kTile, &tm.x, 0, h0 + i, t0, bX);
                    }
                    __syncwarp();
                    x = true;
                    ++nX;
                }
            }
            if (!(c && b && x)) break;
        }
        // nothing in flight when the CTA ends: a C without its B is let land by completing
        // the barrier's arrivals
        if (half) {
            if (lane == 0) ssd_arrive(bCB);
            ++nCB;
        }
        if (nX > 0) ssd_drain(bX, (nX - 1) & 1u, error);
        if (nCB > 0) ssd_drain(bCB, (nCB - 1) & 1u, error);
        __syncwarp();
    } else if (warp == 2 * kVarHalf / 32 + 1) {
        // ---- table warp: items, running sums and factors.  Half a warp per head, eight
        // rows per lane; the next chunk's dt is on its way while this one's are formed. ----
        const uint32_t sequences = SUMMARY ? 0u : static_cast<uint32_t>(p.seq.sequences);
        const uint32_t total = (sequences + *reinterpret_cast<volatile uint32_t *>(p.work.extras)) * static_cast<uint32_t>(p.pairs);
        const int HG = p.heads / p.groups, pairs_per_group = p.pairs / p.groups;
        const int hh = lane >> 4, sub = lane & 15;
        uint32_t u = 0;
        auto fetch = [&]() -> VarItem {  // the next item of the list that has tokens
            VarItem it;
            it.valid = false;
            for (;;) {
                uint32_t q = 0;
                if (lane == 0) q = atomicAdd(p.work.queue + (SUMMARY ? 1 : 0), 1u);
                q = __shfl_sync(0xffffffffu, q, 0);
                if (q >= total) return it;
                const uint32_t e = q / static_cast<uint32_t>(p.pairs);
                const int pair = static_cast<int>(q % static_cast<uint32_t>(p.pairs));
                int n = static_cast<int>(e);
                it.seg = 0;
                if (e >= sequences) {
                    const int2 v = p.work.list[e - sequences];
                    n = v.x, it.seg = SUMMARY ? v.y - 1 : v.y;  // (a later segment's start needs the one before)
                }
                const int64_t begin = packed_at(p.seq, n), end = packed_at(p.seq, n + 1);
                it.first = begin + static_cast<int64_t>(it.seg) * p.segment;
                it.stop = min(it.first + p.segment, end);
                if (it.first >= it.stop) continue;
                it.valid = true;
                it.more = it.stop < end;
                it.g = pair / pairs_per_group;
                it.h0 = it.g * HG + (pair % pairs_per_group) * kVarHeads;
                it.nh = min(kVarHeads, (it.g + 1) * HG - it.h0);
                it.window = begin / p.segment + it.seg;
                const int slot = p.states ? packed_slot(p.seq, n) : -1;
                it.state = slot >= 0 ? p.states + (static_cast<int64_t>(slot) * p.heads + it.h0) * (kSsdP * kSsdN) : nullptr;
                it.src = it.state && p.seq.has_initial && p.seq.has_initial[n] ? it.state : nullptr;
                if (it.seg > 0) it.src = p.work.carry + (it.window * p.heads + it.h0) * (kSsdP * kSsdN);
                if (SUMMARY) it.src = nullptr;
                const int h = it.h0 + (hh < it.nh ? hh : 0);
                it.A = p.A[h];
                it.bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
                it.D = p.D ? p.D[h] : 0.0f;
                return it;
            }
        };
        uint16_t raw[8];
        auto load_dt = [&](const VarItem &it, int64_t t) {
            const uint16_t *src = static_cast<const uint16_t *>(p.dt) + it.h0 + hh;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int64_t r = t + 8 * sub + k;
                raw[k] = r < it.stop && hh < it.nh ? __ldg(src + r * p.dt_stride) : static_cast<uint16_t>(0);
            }
        };
        auto ready = [&]() -> bool {  // everyone has read the chunk before
            const bool ok = u == 0 || ssd_wait(bEmpty, (u - 1) & 1u, error);
            return __all_sync(0xffffffffu, ok);
        };
        bool ok = true;
        VarItem it = fetch();
        if (it.valid) load_dt(it, it.first);
        while (ok && it.valid) {
            VarItem nxt;
            nxt.valid = false;
            float item_total = 0.0f;
            for (int64_t t = it.first; t < it.stop; t += kVarQ) {
                const int rows = static_cast<int>(min(static_cast<int64_t>(kVarQ), it.stop - t));
                const bool last_chunk = t + rows >= it.stop;
                float dt[8], d[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    dt[k] = __uint_as_float(static_cast<uint32_t>(raw[k]) << 16) + it.bias;
                    if (p.softplus) dt[k] = softplus_accurate(dt[k]);
                    if (8 * sub + k >= rows || hh >= it.nh) dt[k] = 0.0f;
                }
                if (!last_chunk) load_dt(it, t + rows);
                // d_j = minus the sum of the later rows' dt A
                float after = 0.0f;
#pragma unroll
                for (int k = 7; k >= 0; --k) {
                    d[k] = after;
                    after -= dt[k] * it.A;
                }
                float sum = after;
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) {
                    const float v = __shfl_down_sync(0xffffffffu, sum, o, 16);
                    if (sub + o < 16) sum += v;
                }
                const float T = -__shfl_sync(0xffffffffu, sum, 0, 16);
                float later = __shfl_down_sync(0xffffffffu, sum, 1, 16);
                if (sub == 15) later = 0.0f;
                float most = 0.0f, w[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    d[k] += later;
                    most = fmaxf(most, fabsf(d[k]));
                    w[k] = expf(-d[k]) * dt[k];
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                const bool factored = most <= (p.softplus ? kVarRange : 0.5f * kVarRange);
                item_total += T;
                if (!SUMMARY && !parallel && t == it.first && it.seg > 0) {  // the segment before, taken earlier by some CTA
                    bool got = false;
                    if (lane == 0) {
                        const uint32_t *flag = p.work.flags + it.window * p.pairs + it.g * pairs_per_group +
                                               (it.h0 - it.g * HG) / kVarHeads;
                        for (uint32_t i = 0; i < p.spin_limit; ++i) {
                            if (ld_acquire(flag) >= p.flag_want) {
                                got = true;
                                break;
                            }
                            if ((i & 255u) == 255u && *reinterpret_cast<volatile uint32_t *>(error) != 0) break;
                            __nanosleep(64);
                        }
                        if (!got) atomicOr(error, 2u);
                    }
                    ok = __shfl_sync(0xffffffffu, static_cast<int>(got), 0) != 0;
                }
                if (!ok || !ready()) {
                    ok = false;
                    break;
                }
                float4 *pd = reinterpret_cast<float4 *>(tabD + hh * kVarQ + 8 * sub), *pw = reinterpret_cast<float4 *>(tabW + hh * kVarQ + 8 * sub);
                pd[0] = make_float4(d[0], d[1], d[2], d[3]), pd[1] = make_float4(d[4], d[5], d[6], d[7]);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (!factored) w[k] = dt[k];
                pw[0] = make_float4(w[0], w[1], w[2], w[3]), pw[1] = make_float4(w[4], w[5], w[6], w[7]);
                VarChunk *out = info + (u & 1u);
                if (sub == 0) {
                    out->decay[hh] = expf(T), out->total[hh] = T, out->D[hh] = it.D;
                    out->factored[hh] = factored;
                    if (SUMMARY && last_chunk && hh < it.nh) p.work.decay[(it.window + 1) * p.heads + it.h0 + hh] = expf(item_total);
                }
                if (lane == 0) {
                    out->t0 = static_cast<int>(t), out->rows = rows;
                    out->h0 = it.h0, out->nh = it.nh, out->g = it.g;
                    out->first = t == it.first, out->last = last_chunk;
                    out->stop = 0;
                    out->src = it.src;
                    const bool hand = SUMMARY || (it.more && !parallel);
                    out->dst = hand ? p.work.carry + ((it.window + 1) * p.heads + it.h0) * (kSsdP * kSsdN)
                                     : it.more ? nullptr : it.state;
                    out->flag = hand && !SUMMARY ? p.work.flags + (it.window + 1) * p.pairs + it.g * pairs_per_group +
                                                        (it.h0 - it.g * HG) / kVarHeads
                                                  : nullptr;
                }
                __syncwarp();
                if (lane == 0) ssd_arrive(bFull);
                ++u;
                // the next item, and its first dt, while this chunk is worked on
                if (t == it.first) nxt = fetch();
                if (last_chunk && nxt.valid) load_dt(nxt, nxt.first);
            }
            it = nxt;
        }
        if (ready() && lane == 0) {
            info[u & 1u].stop = 1;
            ssd_arrive(bFull);
        }
        __syncwarp();
    } else if (tid < kVarHalf) {
        // ---- the state's warps: a thread has row 32 quad + lane of every [128][..] tile (its
        // TMEM lane) and the 64 columns of head `head` --------------------------------------
        using L2 = Lanes<2>;
        const int quad = warp & 3, head = warp >> 2, row = quad * 32 + lane;
        const uint32_t tSh = tS + (static_cast<uint32_t>(quad * 32) << 16) + 64 * head;
        const uint8_t *xraw = sm + S::kX + head * S::kTile;
        uint8_t *stile = sm + S::kS + head * S::kTile;
        uint32_t handed = 0;  // states handed on by this CTA so far
        for (uint32_t u = 0;; ++u) {
            const uint32_t ph = u & 1u;
            if (u > 0) {
                if (!__all_sync(0xffffffffu, ssd_wait(mS, ph ^ 1u, error))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                // the state after an item leaves before anything waits for the next chunk, which
                // may need it; handed on once every thread's part is written
                const VarChunk &c = info[ph ^ 1u];
                if (float *dst = c.dst; c.last && dst) {
                    if (head < c.nh) {
#pragma unroll
                        for (int q0 = 0; q0 < 64; q0 += 16) {
                            float v[16];
                            ssd_ld16(tSh + q0, v);
#pragma unroll
                            for (int e = 0; e < 16; ++e) dst[(head * kSsdP + q0 + e) * kSsdN + row] = v[e];
                        }
                    }
                    if (c.flag) {
                        ssd_arrive(bOut);
                        if (tid == 0 && ssd_wait(bOut, handed & 1u, error)) {
                            __threadfence();  // everyone's part, seen through the barrier, before the flag
                            st_release(c.flag, 1u);
                        }
                        ++handed;
                        __syncwarp();
                    }
                }
            }
            if (!__all_sync(0xffffffffu, ssd_wait(bFull, ph, error))) break;
            const VarChunk &c = info[ph];
            if (c.stop) break;
            const int rows = c.rows;
            const bool first = c.first, live = head < c.nh;
            const float *src = c.src;
            const L2 decay = lanes<2>(c.decay[head]);
            float w = tabW[head * kVarQ + row];
            if (!c.factored[head]) w *= expf(-tabD[head * kVarQ + row]);
            ssd_arrive(bEmpty);

            // S as bf16 to its operand tile [n][p] (the y before passed through it); exp(T) S,
            // float32, to tensor memory
            if (!SUMMARY && u > 0 && !__all_sync(0xffffffffu, ssd_wait(bYf, ph ^ 1u, error))) break;
            auto put = [&](int q0, const float (&v)[16]) {
                uint32_t r[16];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const L2 d = decay * L2::of(v[e], v[e + 1]);
                    r[e] = __float_as_uint(d.get(0)), r[e + 1] = __float_as_uint(d.get(1));
                }
                ssd_st16(tSh + q0, r);
                if constexpr (!SUMMARY) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        *reinterpret_cast<uint4 *>(stile + ssd_sw128(row, q0 + 8 * k)) =
                            make_uint4(pack_bf16x2(v[8 * k], v[8 * k + 1]), pack_bf16x2(v[8 * k + 2], v[8 * k + 3]),
                                       pack_bf16x2(v[8 * k + 4], v[8 * k + 5]), pack_bf16x2(v[8 * k + 6], v[8 * k + 7]));
                }
            };
#pragma unroll
            for (int q0 = 0; q0 < 64; q0 += 32) {
                float v[16], v2[16];
                if (!first) {
                    ssd_ld16x2(tSh + q0, v, tSh + q0 + 16, v2);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float *at = src + (head * kSsdP + q0 + e) * kSsdN + row;
                        v[e] = src && live ? __ldcg(at) : 0.0f;
                        v2[e] = src && live ? __ldcg(at + 16 * kSsdN) : 0.0f;
                    }
                }
                put(q0, v);
                put(q0 + 16, v2);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            if constexpr (!SUMMARY) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                ssd_arrive(bS);
            }

            // exp(-d) dt x as three bf16 parts; rows past the chunk's end are zeros whatever
            // they hold (another sequence's values, or none)
            if (!__all_sync(0xffffffffu, ssd_wait(bX, ph, error))) break;
            const bool in = row < rows && live;
            const L2 w2 = lanes<2>(w), minus = lanes<2>(-1.0f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t o = ssd_sw128(row, 8 * k);
                uint4 xv = *reinterpret_cast<const uint4 *>(xraw + o);
                if (!in) xv = make_uint4(0, 0, 0, 0);
                const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
                uint32_t part[kVarParts][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    L2 v = w2 * L2::of(__uint_as_float(xw[e] << 16), __uint_as_float(xw[e] & 0xffff0000u));
#pragma unroll
                    for (int i = 0; i < kVarParts; ++i) {
                        part[i][e] = pack_bf16x2(v.get(0), v.get(1));
                        if (i + 1 < kVarParts)
                            v = L2::fma(minus, L2::of(__uint_as_float(part[i][e] << 16), __uint_as_float(part[i][e] & 0xffff0000u)), v);
                    }
                }
#pragma unroll
                for (int i = 0; i < kVarParts; ++i)
                    *reinterpret_cast<uint4 *>(sm + S::kXp + (i * kVarHeads + head) * S::kTile + o) =
                        make_uint4(part[i][0], part[i][1], part[i][2], part[i][3]);
            }
            // B's rows past the end meet zeros, but a NaN there would not vanish
            if (rows < kVarQ) {
                if (!__all_sync(0xffffffffu, ssd_wait(bCB, ph, error))) break;
                if (row >= rows) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint4 *>(sm + S::kB + head * S::kTile + ssd_sw128(row, 8 * k)) = make_uint4(0, 0, 0, 0);
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            ssd_arrive(bE1);
        }
    } else if constexpr (!SUMMARY) {
        // ---- the output's warps: a thread has row 32 quad + lane and, of C B^T, 64 columns
        // j, of y, the 64 columns of head `half` ----------------------------------------------
        using L2 = Lanes<2>;
        const int quad = warp & 3, half = (warp >> 2) & 1, row = quad * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
        uint8_t *xraw = sm + S::kX + half * S::kTile;
        for (uint32_t u = 0;; ++u) {
            const uint32_t ph = u & 1u;
            if (!__all_sync(0xffffffffu, ssd_wait(bFull, ph, error))) break;
            // read again where it is needed: this chunk's is overwritten only after everyone
            // has come to the next chunk's C B^T
            const VarChunk &c = info[ph];
            if (c.stop) break;
            const int rows = c.rows;
            const bool live = half < c.nh;
            const int fac0 = c.factored[0], fac1 = c.factored[1];
            const float di0 = tabD[row], di1 = tabD[kVarQ + row];
            // the raw row, for D x; rows past the end as zeros, also in Yd's operand
            if (!__all_sync(0xffffffffu, ssd_wait(bX, ph, error))) break;
            uint32_t xr[32];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t o = ssd_sw128(row, 8 * k);
                if (live && row >= rows) *reinterpret_cast<uint4 *>(xraw + o) = make_uint4(0, 0, 0, 0);
                const uint4 xv = *reinterpret_cast<const uint4 *>(xraw + o);
                xr[4 * k] = xv.x, xr[4 * k + 1] = xv.y, xr[4 * k + 2] = xv.z, xr[4 * k + 3] = xv.w;
            }
            if (rows < kVarQ) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");

            // C B^T with the decays of both heads, as bf16, over its own columns: this thread's
            // 64 columns j of its row i, 16 at a time
            if (!__all_sync(0xffffffffu, ssd_wait(mG, ph, error))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
            for (int q0 = 0; q0 < 64; q0 += 16) {
                const int j0 = 64 * half + q0;
                uint32_t r[16];
                if (j0 > quad * 32 + 31) {  // above the diagonal for every row of the warp
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[e] = 0;
                } else {
                    float v[16];
                    ssd_ld16(tG + lane_off + j0, v);
#pragma unroll
                    for (int e = 0; e < 16; ++e)  // the causal mask, by selection: a zero whatever the later rows hold
                        if (j0 + e > row) v[e] = 0.0f;
#pragma unroll
                    for (int i = 0; i < kVarHeads; ++i) {
                        const float4 *wj = reinterpret_cast<const float4 *>(tabW + i * kVarQ + j0);
                        const float dr = i ? di1 : di0;
                        if (i ? fac1 : fac0) {
                            const L2 e = lanes<2>(expf(dr));
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float4 f = wj[k];
                                const L2 a = L2::of(v[4 * k], v[4 * k + 1]) * (e * L2::of(f.x, f.y));
                                const L2 b = L2::of(v[4 * k + 2], v[4 * k + 3]) * (e * L2::of(f.z, f.w));
                                r[8 * i + 2 * k] = pack_bf16x2(a.get(0), a.get(1));
                                r[8 * i + 2 * k + 1] = pack_bf16x2(b.get(0), b.get(1));
                            }
                        } else {
                            // (the mask's columns may have factors up to infinity: left out too)
                            const float4 *dj = reinterpret_cast<const float4 *>(tabD + i * kVarQ + j0);
                            auto factor = [&](float dc, float dtc, int j) {
                                return j <= row ? ex2_approx((dr - dc) * kLog2e) * dtc : 0.0f;
                            };
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float4 f = wj[k], dd = dj[k];
                                const int j = j0 + 4 * k;
                                r[8 * i + 2 * k] = pack_bf16x2(v[4 * k] * factor(dd.x, f.x, j), v[4 * k + 1] * factor(dd.y, f.y, j + 1));
                                r[8 * i + 2 * k + 1] = pack_bf16x2(v[4 * k + 2] * factor(dd.z, f.z, j + 2), v[4 * k + 3] * factor(dd.w, f.w, j + 3));
                            }
                        }
                    }
                }
                ssd_st16(tG + lane_off + j0, r);
            }
            ssd_arrive(bEmpty);
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            ssd_arrive(bE2);

            if (!__all_sync(0xffffffffu, ssd_wait(mY, ph, error))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            // y = Yd + exp(d + T) Yo + D x
            const uint32_t col = lane_off + 64 * half;
            const L2 eo = lanes<2>(expf((half ? di1 : di0) + c.total[half])), D = lanes<2>(c.D[half]);
#pragma unroll
            for (int q0 = 0; q0 < 64; q0 += 16) {
                float yd[16], yo[16];
                ssd_ld16x2(tYo + col + q0, yo, tYd + col + q0, yd);
#pragma unroll
                for (int e = 0; e < 8; ++e) {  // y takes x's place
                    const uint32_t x = xr[q0 / 2 + e];
                    const L2 v = L2::fma(eo, L2::of(yo[2 * e], yo[2 * e + 1]),
                                         L2::fma(D, L2::of(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)),
                                                 L2::of(yd[2 * e], yd[2 * e + 1])));
                    xr[q0 / 2 + e] = pack_bf16x2(v.get(0), v.get(1));
                }
            }
            // through this warp's rows of the S tile (its product with C is done, and the next
            // S is written after bYf), so that each store writes whole 128-byte lines
            uint8_t *stage = sm + S::kS + half * S::kTile;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                *reinterpret_cast<uint4 *>(stage + ssd_sw128(row, 8 * k)) = make_uint4(xr[4 * k], xr[4 * k + 1], xr[4 * k + 2], xr[4 * k + 3]);
            __syncwarp();
            uint4 line[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                line[k] = *reinterpret_cast<const uint4 *>(stage + ssd_sw128(quad * 32 + 4 * k + (lane >> 3), 8 * (lane & 7)));
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            ssd_arrive(bYf);
            if (live) {
                const int r0 = quad * 32 + (lane >> 3);
                uint16_t *yg = static_cast<uint16_t *>(p.y) + static_cast<int64_t>(c.t0 + r0) * p.y_stride + (c.h0 + half) * kSsdP + 8 * (lane & 7);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (r0 + 4 * k < rows) *reinterpret_cast<uint4 *>(yg) = line[k];
                    yg += 4 * p.y_stride;
                }
            }
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tbase));
}

}  // namespace ssm
