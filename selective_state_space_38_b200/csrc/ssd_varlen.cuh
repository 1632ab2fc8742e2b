// ssd_varlen.cuh -- the Mamba-2 SSD over packed sequences of different lengths,
// with float32 states in cache slots, on the 5th-generation tensor cores.
//
//   H_t = exp(dt_t A) H_{t-1} + dt_t x_t B_t^T,   y_t = H_t C_t + D x_t   per head
//
// over chunks of Q = 128 steps.  With d_i = cs_i - cs_last (cs the running sum of
// dt A in the chunk, T its last value), w_j = exp(-d_j) dt_j and S the state before
// the chunk:
//
//   Y_i   = sum_{j <= i} (C_i . B_j) w_j x_j + C_i (exp(T) S),   y_i = exp(d_i) Y_i + D x_i
//   S_new = exp(T) S + sum_j w_j x_j B_j^T
//
// C B^T is the same for every head of a group: it is formed once for the two heads
// that a CTA walks together; with its columns scaled by w and the later ones masked
// it meets x itself, and the row factor exp(d_i) waits for the end.  (Scaling x by w
// instead would save the per-head matrix, but the tensor core aligns a sum's products
// to the largest and counts a masked zero as 2^-126 times its x: with x scaled over
// e^110 the first rows of a chunk came out wrong by their whole value.)  Where the
// decays span more than e^kVarRange the factors would leave bfloat16's range: there the
// matrix takes its decays against a row factor exp(cs_i), held to e^-70 at least, and S comes
// unscaled.  Its decays are then, for a block of 16 columns from j0 on, one factor of
// the row, exp(c_i - d_j0), times w_j = exp(d_j0 - d_j) dt_j, or, where d moves by more
// than kVarSpan within 16 steps, formed one by one.  (One by one throughout, the heads
// of such decays took 1.25 times the others' time, and at 4 x 4096 their CTAs 220 us
// where the median took 180.)  The state accumulates in tensor memory on exp(T) S.
// The matrix and S also take a power of two, 2^k, and the row's factor 2^-k, with k
// from the middle of the decays' exponents: the factors then span e^-35 to e^35 instead
// of e^-70 to 1 or 1 to e^70, so that neither small operands fall below bfloat16's
// normal values (without it a state of 1e-11 vanished at T = -69) nor large ones pass
// float32's (C B^T dt x of 1e8 at T = -71).
//
// Roundings to bf16 are those of the tensor core's operands: C B^T with its factors
// once, S once where it meets C (each at most the half step that y's own rounding
// is), and w x as a sum of three bf16 parts, 24 bits, where it meets B.  The state
// itself stays float32.  d is summed from the chunk's end, so the steps that count
// most for the state have the smallest rounding.
//
// Per pair of heads and chunk: 96 KB loaded through TMA and six products of
// 128 x 128 x 128, 512 cycles of the tensor pipe each at 8192 bf16 flops a cycle;
// shared memory carries about 640 KB for them and their operands, 5000 cycles at
// 128 bytes a cycle, and bounds it together with the chain from a chunk's state to the
// next one's (about 8600 cycles are measured).  Replayed in a graph, 4 x 4096 tokens of
// 80 heads in one group take 191 us: 340 TFLOP/s, 20 % of the dense rate, 1.9 TB/s; 20
// ragged prompts of 24 heads 81 us; one of 32768 tokens and 24 heads 190 us (called one
// by one 203, 81 and 196).  One CTA per SM.  One warp issues the TMA loads and one the
// MMAs, one walks the work list, one forms the chunks' running sums and factors, and
// sixteen epilogue warps work in two halves: eight on the state (S and its operand,
// the parts of w x), eight on the output (y), so that a chunk's y is written while the
// next one's state and operands are formed; C B^T takes its factors from all sixteen
// (only the warps of the last rows have whole rows of it to do): the output's warps
// have the time for three quarters of them.  Every wait is bounded.
//
// The work is chains of chunks, one for each sequence and pair of heads.  The setup
// kernel chooses between three schedules.  Ranges, when no chain is longer than a
// CTA's share: the chains form one list, cut into equal ranges, one for each CTA.  A
// range is then the end of one chain (its tail), whole chains, and the start of
// another (its head): the CTA walks the head first and hands its state on, the tail
// last, from the state that the CTA before handed on after its own head, so that the
// wait normally finds it there.  Whole chains, from a queue, when some are longer than
// that: those of sequences of more than one segment first, in packed order.  And two passes over segments of the
// sequences when the longest chain would leave the other SMs idle: the segments' own
// states first, from zeros and without outputs, all at once, then the states at their
// starts (ssd_varlen_combine_kernel), then every segment by itself.  In that last pass
// the segments of a sequence run in any order on any CTAs, and the one that ends it
// writes its cache row: so none of them reads that row.  The first one starts from a
// copy that the joining kernel, which reads the row anyhow, leaves in the workspace.
#pragma once

#include <cuda.h>

#include "packed.cuh"
#include "tcgen05.cuh"

namespace ssm {

constexpr int kVarQ = 128;          // steps of a chunk at most
constexpr int kVarMaxWindows = 1024;
constexpr int kVarMaxCtas = 160;
constexpr float kVarRange = 70.0f;   // of the exponents of the factors by columns, and of the rows' on the side of decay
constexpr float kVarGrowth = 85.0f;  // rows' exponents on the side of growth
constexpr float kVarSpan = 40.0f;  // e^40 and e^-87 keep the products of a block's factors well inside float32
constexpr int kVarHalf = 256;       // epilogue threads on the state, and on the output
// + a warp for the MMAs, the tables, the loads and the work list each; the first of the two passes has
// two for the tables, which bound it (in the other a 21st warp leaves 80 registers a thread: 210 us
// against 190 for 4 x 4096)
constexpr int kVarThreads = 2 * kVarHalf + 128, kVarSummaryThreads = kVarThreads + 32;
constexpr int kVarHeads = 2;        // heads walked together
constexpr int kVarParts = 3;        // bf16 parts of w x

// Workspace: header (error word at 16, where ssm_scan_fwd_status reads it); the units
// (chunks x pairs) before each sequence; for the two passes the later segments of the
// sequences and, by the window of `segment` tokens each starts in, a decay and a state
// per head, and the starting states of the sequences of several segments, by their
// number among those; for the ranges a flag and a pair of states per CTA (the carried
// states of both share one place).
struct VarWork {
    uint32_t *queue;                   // item counters of the two passes; order of the CTAs' start
    uint32_t *error, *extras;          // error word; later segments
    uint32_t *several, *mode;          // sequences of more than one segment; the schedule
    uint32_t *range;                   // units of a CTA's range
    uint32_t *units;                   // [sequences + 1]
    int2 *list;                        // [windows] (sequence, segment) of the later segments
    uint32_t *flags;                   // [kVarMaxCtas] a range's head is handed on
    float *decay;                      // [windows][heads] of the segment before the window's
    float *carry;                      // [windows][heads][P][N], or [kVarMaxCtas][2][P][N]
    float *start;                      // [sequences of several segments][heads][P][N]
};

enum VarMode : uint32_t { kVarRanges = 0, kVarTwoPasses = 1, kVarChains = 2 };

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
    int32_t segment, windows, ctas;
    uint32_t flag_want, spin_limit;
    int softplus;
};

// A stretch of a sequence's tokens for a pair of heads, as the work list's warp hands
// it on: where its state comes from and goes.
struct VarItem {
    int32_t first, stop;     // tokens
    int32_t h0, nh, g;       // first head, heads (1 or 2), group
    int32_t valid;
    const float *src;        // the state before it, or NULL (zeros)
    float *dst;              // where its state goes, or NULL
    uint32_t *flag;          // hand-off: set once dst is written, or NULL
    float *decay;            // the two passes' first: receives exp of its sum of dt A, per head
    float A[2], bias[2], D[2];
};

// How C B^T takes a head's decays: by columns, by rows and columns of 16-column blocks, one by one.
enum VarDecays : int32_t { kVarByColumn = 0, kVarByBlock = 1, kVarOneByOne = 2 };

// What the table warp hands on with each chunk.
struct VarChunk {
    int32_t t0, rows;        // first token, steps
    int32_t h0, nh, g;
    int32_t first, last;     // of the item
    int32_t stop;
    const float *src;
    float *dst;
    uint32_t *flag;
    float decay[2], scale[2], D[2];  // exp(T); of S where it meets C
    float ref[2];            // T: cs = d + T, the row factor's exponent where the decays are not by columns
    float down[2], shift[2]; // 2^-k and its exponent k ln 2, where C B^T with its factors and S take 2^k
    int32_t decays[2];       // VarDecays
};

struct VarSmem {
    static constexpr int kTile = 128 * 128;           // [128 rows][64] bf16, 128-byte swizzle
    static constexpr int kC = 0;                      // [t][n]: n < 64, n >= 64
    static constexpr int kB = 2 * kTile, kBufB = 2 * kTile;  // the same, of even and of odd chunks
    static constexpr int kX = kB + 2 * kBufB;         // [t][p] of each head; y passes through it
    static constexpr int kXp = kX + kVarHeads * kTile;  // w x: parts x heads tiles
    // S [n][p] of each head, in the last part's place: C S has read it before the parts are formed
    static constexpr int kS = kXp + (kVarParts - 1) * kVarHeads * kTile;
    static constexpr int kTabD = kXp + kVarParts * kVarHeads * kTile;  // d [head][128]
    static constexpr int kTabW = kTabD + kVarHeads * 512;           // the columns' factors (with decays one by one: dt)
    static constexpr int kInfo = kTabW + kVarHeads * 512;           // of even and of odd chunks
    static constexpr int kItem = kInfo + 256;
    static constexpr int kBar = kItem + 128;
    static constexpr int kTotal = kBar + 192;
};
static_assert(sizeof(VarChunk) <= 128 && sizeof(VarItem) <= 128, "");
static_assert(VarSmem::kTotal <= 227 * 1024, "shared memory of the packed SSD kernel");

// The units before each sequence, the later segments ordered by their number (so that
// the second segments come first), and the choice of the schedule.  Two later segments
// never start in the same window of `segment` tokens (those of one sequence are
// `segment` apart, those of the next sequence start more than that behind its start),
// so a window's index names one.  One block of 1024 threads.
__global__ void __launch_bounds__(1024) ssd_varlen_setup_kernel(const VarParams p) {
    release_next();
    __shared__ int2 at[kVarMaxWindows];
    __shared__ uint32_t sums[32];
    __shared__ uint32_t later, several, filled, bad;
    __shared__ int longest;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) later = 0, several = 0, filled = 0, bad = 0, longest = 0;
    for (int k = tid; k < p.windows; k += 1024) at[k] = make_int2(-1, 0);
    for (int k = tid; k < kVarMaxCtas; k += 1024) p.work.flags[k] = 0;
    __syncthreads();
    uint32_t before = 0;  // units of the sequences of earlier turns
    for (int n0 = 0; n0 < p.seq.sequences; n0 += 1024) {
        const int n = n0 + tid;
        uint32_t units = 0;
        if (n < p.seq.sequences) {
            const int32_t a = p.seq.cu[n], b = p.seq.cu[n + 1];
            if (a < 0 || b < a || b > p.seq.tokens) {
                bad = 1;
            } else {
                const int segs = (b - a + p.segment - 1) / p.segment, chunks = (b - a + kVarQ - 1) / kVarQ;
                units = static_cast<uint32_t>(chunks) * p.pairs;
                if (segs > 1) {
                    for (int s = 1; s < segs; ++s) at[a / p.segment + s] = make_int2(n, s);  // the window of a + s segment
                    atomicAdd(&several, 1u);
                }
                if (chunks > 0) atomicAdd(&filled, 1u);
                atomicMax(&longest, chunks);
            }
        }
        uint32_t run = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += v;
        }
        if (lane == 31) sums[warp] = run;
        __syncthreads();
        uint32_t base = before, all = 0;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) base += sums[w];
            all += sums[w];
        }
        if (n < p.seq.sequences) p.work.units[n + 1] = base + run;
        before += all;
        __syncthreads();
    }
    for (int k = tid; k < p.windows; k += 1024) {
        const int2 v = at[k];
        if (v.x < 0) continue;
        int rank = 0;
        for (int o = 0; o < p.windows; ++o)
            rank += at[o].x >= 0 && (at[o].y < v.y || (at[o].y == v.y && o < k));
        p.work.list[rank] = v;
        atomicAdd(&later, 1u);
    }
    __syncthreads();
    if (tid == 0) {
        p.work.queue[0] = p.work.queue[1] = p.work.queue[2] = 0;
        p.work.units[0] = 0;
        *p.work.extras = later;
        *p.work.several = several;
        // In tenths of a chunk's time: a CTA's share, with six for the start and the end of each
        // chain; the two passes cost 1.4 times that, an uneven last segment, and their launches
        // (four chunks' time).  Measured on 24 heads: one sequence of 32768 tokens 193 us in two
        // passes against some 1300 as chains; 20 sequences, the longest of 2048, 82 against 134.
        const uint32_t share = (before + p.ctas - 1) / p.ctas;
        const int64_t each = (10ll * before + 6ll * filled * p.pairs) / p.ctas;
        const int64_t two = each * 14 / 10 + 10 * (p.segment / kVarQ + 4);
        *p.work.range = max(share, 1u);
        *p.work.mode = share >= static_cast<uint32_t>(longest) || p.flag_want != 1u ? kVarRanges
                       : later > 0 && 10ll * longest > two                          ? kVarTwoPasses
                                                                                    : kVarChains;
        *p.work.error = bad ? 4u : 0u;  // a table that does not ascend within the tokens: nothing is run
    }
}

// The states at the segments' starts from the segments' own: S_{s+1} = exp(T_s) S_s
// + E_s, in place, and a copy of S_0 from the cache where a sequence goes on.  grid: (heads x 8, sequences of more than one segment at most)
__global__ void __launch_bounds__(256) ssd_varlen_combine_kernel(const VarParams p) {
    release_next();
    wait_previous();
    if ((*p.work.error & 4u) || *p.work.mode != kVarTwoPasses) return;
    const int h = blockIdx.x / 8;
    const int64_t e = (blockIdx.x % 8) * 256 + threadIdx.x;  // a 16-byte vector of the state
    for (uint32_t i = blockIdx.y; i < *p.work.several; i += gridDim.y) {
        const int n = p.work.list[i].x;
        const int64_t begin = p.seq.cu[n], end = p.seq.cu[n + 1];
        const int segs = static_cast<int>((end - begin + p.segment - 1) / p.segment);
        const int slot = p.states ? packed_slot(p.seq, n) : -1;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (slot >= 0 && p.seq.has_initial && p.seq.has_initial[n]) {
            s = reinterpret_cast<const float4 *>(p.states + (static_cast<int64_t>(slot) * p.heads + h) * (kSsdP * kSsdN))[e];
            reinterpret_cast<float4 *>(p.work.start + (static_cast<int64_t>(i) * p.heads + h) * (kSsdP * kSsdN))[e] = s;
        }
        for (int k0 = 1; k0 < segs; k0 += 8) {  // eight segments' loads at a time
            float4 v[8];
            float a[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t w = (begin / p.segment + min(k0 + j, segs - 1)) * p.heads + h;
                v[j] = reinterpret_cast<const float4 *>(p.work.carry + w * (kSsdP * kSsdN))[e];
                a[j] = p.work.decay[w];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (k0 + j >= segs) break;
                s.x = fmaf(a[j], s.x, v[j].x), s.y = fmaf(a[j], s.y, v[j].y), s.z = fmaf(a[j], s.z, v[j].z), s.w = fmaf(a[j], s.w, v[j].w);
                reinterpret_cast<float4 *>(p.work.carry + ((begin / p.segment + k0 + j) * p.heads + h) * (kSsdP * kSsdN))[e] = s;
            }
        }
    }
}

// The chunks of a CTA's range, one item after another (one warp together).
struct VarRange {
    // a chain and a place in it
    struct At {
        int n, pair, chunk, chunks;
    };
    const VarParams &p;
    __device__ explicit VarRange(const VarParams &q) : p(q) {}
    __device__ At find(uint32_t unit) const {  // unit < units[sequences]
        int c = 0;
        for (int i = threadIdx.x & 31; i < p.seq.sequences; i += 32) c += p.work.units[i + 1] <= unit;
        At a;
        a.n = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(c)));
        const uint32_t from = p.work.units[a.n];
        a.chunks = static_cast<int>((p.work.units[a.n + 1] - from) / p.pairs);
        a.pair = static_cast<int>((unit - from) / a.chunks);
        a.chunk = static_cast<int>((unit - from) % a.chunks);
        return a;
    }
    __device__ void next_chain(At &a) const {
        a.chunk = 0;
        if (++a.pair < p.pairs) return;
        a.pair = 0;
        do ++a.n;
        while (a.n < p.seq.sequences && p.work.units[a.n + 1] == p.work.units[a.n]);
        if (a.n < p.seq.sequences) a.chunks = static_cast<int>((p.work.units[a.n + 1] - p.work.units[a.n]) / p.pairs);
    }
};

// The exponent of a row's factor.  Where the decays are not taken by columns it is cs_i,
// held to [-70, 85] (beyond, only the state before the chunk would feel it, by e^-70
// of itself; growth by e^85 overflows), and the rest is left to the matrix.  2^k comes
// off here (its rounded exponent changes y by 2^-18 of itself at most).
__device__ __forceinline__ float var_row_exponent(const VarChunk &c, int i, float di) {
    return (c.decays[i] == kVarByColumn ? di : fminf(fmaxf(di + c.ref[i], -kVarRange), kVarGrowth)) - c.shift[i];
}

// C B^T with the factors of both heads, as bf16, over its own columns: of this warp's
// 32 rows the blocks of 16 columns j0, j0 + 32, ... below j1.  One copy of it,
// called: the warps' loops are straight code of thousands of instructions, and the
// instruction cache is what they would wait for.
__device__ __noinline__ void var_factors(const VarChunk &c, const float *tabD, const float *tabW, uint32_t at, int row, int j0,
                                         int j1) {
    using L2 = Lanes<2>;
    const int top = row & ~31;
#pragma unroll 1
    for (; j0 < j1; j0 += 32) {
        const bool some = j0 <= top + 31;  // else above the diagonal for every row of the warp
        float v[16];
        if (some) {
            ssd_ld16(at + j0, v);
            if (j0 + 15 > top) {  // the causal mask, by selection: a zero whatever the later rows hold
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (j0 + e > row) v[e] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < kVarHeads; ++i) {
            uint32_t r[8] = {};
            const float4 *wj = reinterpret_cast<const float4 *>(tabW + i * kVarQ + j0);
            if (some && c.decays[i] != kVarOneByOne) {
                float rf = 1.0f;  // the row's factor of the block; none above the diagonal, where it may overflow
                if (c.decays[i] == kVarByBlock) {
                    const float di = tabD[i * kVarQ + row];
                    rf = j0 <= row ? ex2_approx((di - var_row_exponent(c, i, di) - tabD[i * kVarQ + j0]) * kLog2e) : 0.0f;
                }
                const L2 rf2 = lanes<2>(rf);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 f = wj[k];
                    const L2 lo = L2::of(v[4 * k], v[4 * k + 1]) * rf2 * L2::of(f.x, f.y);
                    const L2 hi = L2::of(v[4 * k + 2], v[4 * k + 3]) * rf2 * L2::of(f.z, f.w);
                    r[2 * k] = pack_bf16x2(lo.get(0), lo.get(1));
                    r[2 * k + 1] = pack_bf16x2(hi.get(0), hi.get(1));
                }
            } else if (some) {
                // (the mask's columns may have factors up to infinity: left out too)
                const float4 *dj = reinterpret_cast<const float4 *>(tabD + i * kVarQ + j0);
                const float di = tabD[i * kVarQ + row], ci = di - var_row_exponent(c, i, di);
                auto factor = [&](float dc, float dtc, int j) {
                    return j <= row ? ex2_approx((ci - dc) * kLog2e) * dtc : 0.0f;
                };
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 f = wj[k], dd = dj[k];
                    const int j = j0 + 4 * k;
                    r[2 * k] = pack_bf16x2(v[4 * k] * factor(dd.x, f.x, j), v[4 * k + 1] * factor(dd.y, f.y, j + 1));
                    r[2 * k + 1] = pack_bf16x2(v[4 * k + 2] * factor(dd.z, f.z, j + 2), v[4 * k + 3] * factor(dd.w, f.w, j + 3));
                }
            }
            ssd_st8(at + j0 + 8 * i, r);
        }
    }
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

// One copy of the wait, too.
__device__ __noinline__ bool var_wait(uint64_t *bar, uint32_t parity, uint32_t *error) {
    return __all_sync(0xffffffffu, ssd_wait(bar, parity, error));
}

// SUMMARY: the first of the two passes, which forms the segments' own states only;
// nothing to do when the setup kernel chose the ranges.
template <bool SUMMARY>
__global__ void __launch_bounds__(SUMMARY ? kVarSummaryThreads : kVarThreads, 1)
    ssd_varlen_kernel(const VarParams p, const __grid_constant__ VarMaps tm) {
    extern __shared__ __align__(1024) uint8_t var_smem[];
    using S = VarSmem;
    // without outputs all sixteen epilogue warps work on the state, half the columns each
    constexpr int kTables = SUMMARY ? 2 : 1;  // warps on the tables
    constexpr int kStateThreads = SUMMARY ? 2 * kVarHalf : kVarHalf, kCols = SUMMARY ? 32 : 64;
    uint8_t *sm = var_smem;
    float *tabD = reinterpret_cast<float *>(sm + S::kTabD), *tabW = reinterpret_cast<float *>(sm + S::kTabW);
    VarChunk *info = reinterpret_cast<VarChunk *>(sm + S::kInfo);
    VarItem *item = reinterpret_cast<VarItem *>(sm + S::kItem);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + S::kBar);
    uint64_t *bFull = bar, *bX = bar + 1;                          // tables and info written; X landed
    uint64_t *mG = bar + 2, *mC = bar + 3, *mS = bar + 4, *mY = bar + 5;  // C B^T; C S; the state; Y done
    uint64_t *bItem = bar + 6, *bTaken = bar + 7;                  // an item written; read
    uint64_t *bCB = bar + 8;                                       // C and B landed
    uint64_t *bEmpty = bar + 9;                                    // info read by everyone, tables done with
    uint64_t *bS = bar + 10, *bE1 = bar + 11, *bOut = bar + 12;    // S; the parts of w x; a handed-on state written
    uint64_t *bE2 = bar + 13, *bYf = bar + 14;                     // C B^T with its factors written; y out of the X tile
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + 15);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t *error = p.work.error;

    // (the first pass does not let the next kernels' blocks come while it has work to do:
    // beside it they cost it 7 %)
    wait_previous();
    // the swizzled tiles need 1024-byte alignment; a work list that was refused has no items
    if ((smem_u32(sm) & 1023u) != 0) {
        if (tid == 0) atomicOr(error, 2u);
        return;
    }
    if (*reinterpret_cast<volatile uint32_t *>(error) & 4u) return;
    const uint32_t mode = *reinterpret_cast<volatile uint32_t *>(p.work.mode);
    if (SUMMARY && mode != kVarTwoPasses) return;
    if (tid == 0) {
        for (int i = 0; i < 15; ++i) {
            const uint32_t n = i == 0 || i == 7 ? kTables : i < 9 ? 1 : i == 9 ? 2 * kVarHalf + 2 : i == 13 ? 2 * kVarHalf : i < 13 ? kStateThreads : kVarHalf;
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
    // every 16 columns the first 8 for head 0, the others for head 1), Y of even and of odd
    // chunks and S (128 each: head h's column p in 64 h + p; lane n holds S[p][n])
    const uint32_t tG = tbase, tY = tbase + 128, tS = tbase + 384;
    constexpr int kN = 64 * kVarHeads;

    // The waits of the warps that stay converged: a bounded one, and a test.
    auto wait = [&](uint64_t *b, uint32_t ph) -> bool { return var_wait(b, ph, error); };
    auto test = [&](uint64_t *b, uint32_t ph) -> bool { return __any_sync(0xffffffffu, ssd_try(smem_u32(b), ph)); };
    auto give_up = [&](uint32_t n) -> bool {  // after n tests in vain
        if (n >= kSsdWaitLimit && lane == 0) atomicOr(error, 2u);
        return n >= kSsdWaitLimit || ((n & 1023u) == 1023u && __any_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(error) != 0));
    };
    constexpr int kMmaWarp = 2 * kVarHalf / 32, kTableWarp = kMmaWarp + 1,
                  kLoadWarp = kTableWarp + kTables, kListWarp = kLoadWarp + 1;
    if (warp == kMmaWarp) {
        // ---- the products, issued by one elected lane -----------------------------------
        const uint32_t aC = smem_u32(sm + S::kC), aB = smem_u32(sm + S::kB), aX = smem_u32(sm + S::kX),
                       aXp = smem_u32(sm + S::kXp), aS = smem_u32(sm + S::kS);
        uint32_t nG = 0, nC = 0, nS = 0, nY = 0;  // issued
        for (uint32_t u = 0;; ++u) {
            const uint32_t ph = u & 1u, tYu = tY + 128 * ph, aBu = aB + S::kBufB * ph;
            if (!wait(bFull, ph)) break;
            const int heads = info[ph].nh;
            const bool stop = info[ph].stop;
            __syncwarp();
            if (!SUMMARY && lane == 0) ssd_arrive(bEmpty);
            // (the products before have read what C B^T replaces: mY)
            if (stop || !wait(bCB, ph) || (!SUMMARY && u > 0 && !wait(mY, ph ^ 1u))) break;
            // (in the first pass the next chunk's B may come from here on, which a later wait for this
            // one's could not tell apart)
            if (SUMMARY && lane == 0) ssd_arrive(bEmpty);
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if constexpr (!SUMMARY) {
                if (ssd_elect()) {  // C B^T
                    constexpr uint32_t id = ssd_idesc(128, 128, 0, 0);
                    const uint64_t dC = ssd_desc(aC, 16, 1024), dB = ssd_desc(aBu, 16, 1024);
#pragma unroll 2
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t o = ((k / 4) * S::kTile + (k % 4) * 32) >> 4;
                        ssd_mma(tG, dC + o, dB + o, id, k > 0);
                    }
                    ssd_commit(mG);
                }
                __syncwarp();
                nG = u + 1;
                if (!wait(bS, ph)) break;  // (and this Y, of two chunks before, was read before that chunk's bYf)
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                if (ssd_elect()) {  // Y = C S
                    constexpr uint32_t id = ssd_idesc(128, kN, 0, 1);
                    const uint64_t dC = ssd_desc(aC, 16, 1024), dS = ssd_desc(aS, S::kTile, 1024);
#pragma unroll 2
                    for (int k = 0; k < 8; ++k)
                        ssd_mma(tYu, dC + (((k / 4) * S::kTile + (k % 4) * 32) >> 4), dS + ((2048 * k) >> 4), id, k > 0);
                    ssd_commit(mC);
                }
                __syncwarp();
                nC = u + 1;
            }
            // the state's products and the rest of Y, whichever has its operands first
            bool state = false, yd = SUMMARY;
            for (uint32_t n = 0; !(state && yd) && !give_up(n); ++n) {
                if (!SUMMARY && !yd && test(bE2, ph) && test(bX, ph)) {  // (bE2 alone does not say that X has landed)
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    if (ssd_elect()) {  // Y += (C B^T with its factors) x, per head
                        constexpr uint32_t id = ssd_idesc(128, 64, 0, 1);
                        const uint64_t dX = ssd_desc(aX, S::kTile, 1024);
#pragma unroll 1
                        for (int i = 0; i < kVarHeads; ++i)
                            if (i < heads) {
#pragma unroll 2
                                for (int k = 0; k < 8; ++k)
                                    ssd_mma_ts(tYu + 64 * i, tG + 16 * k + 8 * i, dX + ((i * S::kTile + 2048 * k) >> 4), id, 1);
                            }
                        ssd_commit(mY);
                    }
                    __syncwarp();
                    yd = true;
                    nY = u + 1;
                }
                if (!state && test(bE1, ph)) {
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    if (ssd_elect()) {  // S += B^T (w x), the smallest part first
                        constexpr uint32_t id = ssd_idesc(128, kN, 1, 1);
                        const uint64_t dB = ssd_desc(aBu, S::kTile, 1024), dX = ssd_desc(aXp, S::kTile, 1024);
#pragma unroll 1
                        for (int part = kVarParts - 1; part >= 0; --part)
#pragma unroll 2
                            for (int k = 0; k < 8; ++k)
                                ssd_mma(tS, dB + ((2048 * k) >> 4), dX + ((part * kVarHeads * S::kTile + 2048 * k) >> 4), id, 1);
                        ssd_commit(mS);
                    }
                    __syncwarp();
                    state = true;
                    nS = u + 1;
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
    } else if (warp == kLoadWarp) {
        // ---- the loads: C once C S has read the chunk's before, and B with it (its buffer is
        // free: that C S had the state after the products that read it); X once the state's
        // warps have read the one before and y, which passes through it, is out of it.  In the
        // first pass B comes with X: the state's warps had waited for the products two chunks
        // before, and the MMA warp has seen the B before land (bEmpty, then bFull) -------------
        uint32_t nX = 0, nCB = 0;  // issued
        for (uint32_t u = 0;; ++u) {
            const uint32_t ph = u & 1u, pv = ph ^ 1u;
            if (!wait(bFull, ph)) break;
            const int t0 = info[ph].t0, h0 = info[ph].h0, nh = info[ph].nh, g = info[ph].g;
            const bool stop = info[ph].stop;
            __syncwarp();
            if (lane == 0) ssd_arrive(bEmpty);
            if (stop) break;
            bool cb = false, x = false;
            for (uint32_t n = 0; !(cb && x) && !give_up(n); ++n) {
                if (!cb && (u == 0 || test(SUMMARY ? bE1 : mC, pv))) {
                    if (ssd_elect()) {
                        uint8_t *b = sm + S::kB + S::kBufB * ph;
                        mbar_arrive_expect_tx(bCB, (SUMMARY ? 2 : 4) * S::kTile);
                        if constexpr (!SUMMARY) {
                            tma_load_3d(sm + S::kC, &tm.C, 0, g, t0, bCB);
                            tma_load_3d(sm + S::kC + S::kTile, &tm.C, 64, g, t0, bCB);
                        }
                        tma_load_3d(b, &tm.B, 0, g, t0, bCB);
                        tma_load_3d(b + S::kTile, &tm.B, 64, g, t0, bCB);
                    }
                    __syncwarp();
                    cb = true;
                    ++nCB;
                }
                if (!x && (u == 0 || (SUMMARY ? cb : test(bE1, pv) && test(bYf, pv)))) {
                    if (ssd_elect()) {
                        mbar_arrive_expect_tx(bX, nh * S::kTile);
                        for (int i = 0; i < nh; ++i) tma_load_3d(sm + S::kX + i * S::kTile, &tm.x, 0, h0 + i, t0, bX);
                    }
                    __syncwarp();
                    x = true;
                    ++nX;
                }
            }
            if (!(cb && x)) break;
        }
        // nothing in flight when the CTA ends
        if (nX > 0) ssd_drain(bX, (nX - 1) & 1u, error);
        if (nCB > 0) ssd_drain(bCB, (nCB - 1) & 1u, error);
        __syncwarp();
    } else if (warp == kListWarp) {
        // ---- the work list: one item ahead of the table warp ------------------------------
        const int HG = p.heads / p.groups, pairs_per_group = p.pairs / p.groups;
        uint32_t k = 0;  // items handed on
        auto hand_on = [&](bool valid, int pair, int64_t first, int64_t stop, const float *src, float *dst, uint32_t *flag,
                           float *decay) -> bool {
            if (k > 0 && !wait(bTaken, (k - 1) & 1u)) return false;
            if (lane == 0) {
                item->valid = valid;
                if (valid) {
                    const int g = pair / pairs_per_group, h0 = g * HG + (pair % pairs_per_group) * kVarHeads;
                    const int nh = min(kVarHeads, (g + 1) * HG - h0);
                    item->first = static_cast<int>(first), item->stop = static_cast<int>(stop);
                    item->h0 = h0, item->nh = nh, item->g = g;
                    item->src = src, item->dst = dst, item->flag = flag, item->decay = decay;
#pragma unroll
                    for (int i = 0; i < kVarHeads; ++i) {
                        const int h = h0 + (i < nh ? i : 0);
                        item->A[i] = p.A[h];
                        item->bias[i] = p.dt_bias ? p.dt_bias[h] : 0.0f;
                        item->D[i] = p.D ? p.D[h] : 0.0f;
                    }
                }
                ssd_arrive(bItem);
            }
            __syncwarp();
            ++k;
            return true;
        };
        auto head_of = [&](int pair) { return (pair / pairs_per_group) * HG + (pair % pairs_per_group) * kVarHeads; };
        // a sequence's place in the cache for a pair of heads, and whether it goes on from it
        auto cache = [&](int n, int pair, const float **initial) -> float * {
            const int slot = p.states ? packed_slot(p.seq, n) : -1;
            float *s = slot >= 0 ? p.states + (static_cast<int64_t>(slot) * p.heads + head_of(pair)) * (kSsdP * kSsdN) : nullptr;
            *initial = s && p.seq.has_initial && p.seq.has_initial[n] ? s : nullptr;
            return s;
        };
        // the sequences of several segments before n (their second segments lead the list, in packed order)
        auto several_before = [&](int n) -> int {
            const int several = static_cast<int>(*reinterpret_cast<volatile uint32_t *>(p.work.several));
            int c = 0;
            for (int i = lane; i < several; i += 32) c += p.work.list[i].x < n;
            return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(c)));
        };
        bool ok = true;
        if (mode != kVarRanges) {
            // segments: every sequence's first, then the later ones of the list; chains: the
            // sequences of several segments (whose second ones lead the list), then the others
            const bool chains = mode == kVarChains;
            const uint32_t lead = chains ? *reinterpret_cast<volatile uint32_t *>(p.work.several) : SUMMARY ? 0u : static_cast<uint32_t>(p.seq.sequences);
            const uint32_t rest = chains ? static_cast<uint32_t>(p.seq.sequences) : *reinterpret_cast<volatile uint32_t *>(p.work.extras);
            const uint32_t total = (lead + rest) * static_cast<uint32_t>(p.pairs);
            while (ok) {
                uint32_t q = 0;
                if (lane == 0) q = atomicAdd(p.work.queue + (SUMMARY ? 1 : 0), 1u);
                q = __shfl_sync(0xffffffffu, q, 0);
                if (q >= total) break;
                const uint32_t e = q / static_cast<uint32_t>(p.pairs);
                const int pair = static_cast<int>(q % static_cast<uint32_t>(p.pairs));
                int n = static_cast<int>(e), seg = 0;
                if (chains) {
                    n = e < lead ? p.work.list[e].x : static_cast<int>(e - lead);
                } else if (SUMMARY || e >= lead) {
                    const int2 v = p.work.list[e - lead];
                    n = v.x, seg = SUMMARY ? v.y - 1 : v.y;  // (a later segment's start needs the one before)
                }
                const int64_t begin = packed_at(p.seq, n), end = packed_at(p.seq, n + 1);
                const int64_t first = begin + static_cast<int64_t>(seg) * p.segment, stop = chains ? end : min(first + p.segment, end);
                if (first >= stop || (chains && e >= lead && end - begin > p.segment)) continue;
                const int64_t window = begin / p.segment + seg;  // of its start; the next one's is the segment behind it
                const int h0 = head_of(pair);
                if constexpr (SUMMARY) {
                    const int64_t w = (window + 1) * p.heads + h0;
                    ok = hand_on(true, pair, first, stop, nullptr, p.work.carry + w * (kSsdP * kSsdN), nullptr, p.work.decay + w);
                } else {
                    const float *src;
                    float *state = cache(n, pair, &src);
                    if (seg > 0) src = p.work.carry + (window * p.heads + h0) * (kSsdP * kSsdN);
                    else if (src && stop < end) src = p.work.start + (static_cast<int64_t>(several_before(n)) * p.heads + h0) * (kSsdP * kSsdN);
                    ok = hand_on(true, pair, first, stop, src, stop < end ? nullptr : state, nullptr, nullptr);
                }
            }
        } else {
            uint32_t order = 0;  // with hand-offs a CTA's range is its place in the order of start
            if (lane == 0) order = atomicAdd(p.work.queue + 2, 1u);
            order = __shfl_sync(0xffffffffu, order, 0);
            const uint32_t W = *reinterpret_cast<volatile uint32_t *>(p.work.range), all = p.work.units[p.seq.sequences];
            const uint64_t s0 = static_cast<uint64_t>(order) * W;
            if (s0 < all) {
                const uint32_t e0 = static_cast<uint32_t>(min(s0 + W, static_cast<uint64_t>(all)));
                const VarRange range(p);
                const VarRange::At from = range.find(static_cast<uint32_t>(s0)), to = range.find(e0 - 1);
                // chunks [c0, c1) of a chain: its state from the cache or the CTA before, to the
                // cache or the next CTA
                auto part = [&](const VarRange::At &a, int c0, int c1) -> bool {
                    const int64_t begin = packed_at(p.seq, a.n), end = packed_at(p.seq, a.n + 1);
                    const float *src;
                    float *dst = cache(a.n, a.pair, &src);
                    uint32_t *flag = nullptr;
                    if (c0 > 0) {  // (order > 0: the first range starts with a chain)
                        bool got = false;
                        if (lane == 0) {
                            for (uint32_t i = 0; i < p.spin_limit; ++i) {
                                if (ld_acquire(p.work.flags + order - 1) >= p.flag_want) {
                                    got = true;
                                    break;
                                }
                                if ((i & 255u) == 255u && *reinterpret_cast<volatile uint32_t *>(error) != 0) break;
                                __nanosleep(64);
                            }
                            if (!got) atomicOr(error, 2u);
                        }
                        if (!__shfl_sync(0xffffffffu, static_cast<int>(got), 0)) return false;
                        src = p.work.carry + static_cast<int64_t>(order - 1) * kVarHeads * (kSsdP * kSsdN);
                    }
                    if (c1 < a.chunks) {
                        dst = p.work.carry + static_cast<int64_t>(order) * kVarHeads * (kSsdP * kSsdN);
                        flag = p.work.flags + order;
                    }
                    return hand_on(true, a.pair, begin + static_cast<int64_t>(c0) * kVarQ,
                                   min(begin + static_cast<int64_t>(c1) * kVarQ, end), src, dst, flag, nullptr);
                };
                if (from.n == to.n && from.pair == to.pair) {
                    ok = part(from, from.chunk, to.chunk + 1);
                } else {
                    const bool head = to.chunk + 1 < to.chunks;  // a chain that the next CTA ends
                    if (head) ok = part(to, 0, to.chunk + 1);
                    VarRange::At a = from;
                    if (a.chunk > 0) range.next_chain(a);
                    for (; ok; range.next_chain(a)) {
                        const bool at_end = a.n == to.n && a.pair == to.pair;
                        if (at_end && head) break;
                        ok = part(a, 0, a.chunks);
                        if (at_end) break;
                    }
                    if (ok && from.chunk > 0) ok = part(from, from.chunk, from.chunks);
                }
            }
        }
        hand_on(false, 0, 0, 0, nullptr, nullptr, nullptr, nullptr);  // (after a failure too, for those who can still hear it)
        __syncwarp();
    } else if (warp >= kTableWarp && warp < kTableWarp + kTables) {
        // ---- the tables: running sums and factors.  Half a warp per head, eight rows per lane
        // (a warp and four where there are two); the next chunk's dt is on its way while this
        // one's are formed. ----------------------------------------------------------------
        constexpr int kLanes = 16 * kTables, kRows = kVarQ / kLanes;
        const int hh = SUMMARY ? warp - kTableWarp : lane >> 4, sub = lane & (kLanes - 1);
        uint32_t u = 0, k = 0;  // chunks handed on, items taken
        // the item at hand, with this head's A, bias and D
        int first_t = 0, stop_t = 0, h0 = 0, nh = 0, g = 0;
        const float *src = nullptr;
        float *dst = nullptr, *decay = nullptr;
        uint32_t *flag = nullptr;
        float A = 0.0f, bias = 0.0f, D = 0.0f;
        auto take = [&]() -> bool {  // the next item; false: none
            const bool got = wait(bItem, k & 1u);
            if (!got) return false;
            const bool valid = item->valid;
            first_t = item->first, stop_t = item->stop, h0 = item->h0, nh = item->nh, g = item->g;
            src = item->src, dst = item->dst, flag = item->flag, decay = item->decay;
            A = item->A[hh], bias = item->bias[hh], D = item->D[hh];
            __syncwarp();
            if (lane == 0) ssd_arrive(bTaken);
            ++k;
            return valid;
        };
        uint16_t raw[kRows];
        auto load_dt = [&](int64_t t) {
            const uint16_t *from = static_cast<const uint16_t *>(p.dt) + h0 + hh;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int64_t r = t + kRows * sub + i;
                raw[i] = r < stop_t && hh < nh ? __ldg(from + r * p.dt_stride) : static_cast<uint16_t>(0);
            }
        };
        auto ready = [&]() -> bool { return u == 0 || wait(bEmpty, (u - 1) & 1u); };  // everyone has read the chunk before
        // The first of the two passes walks an item from its last chunk to its first, the sum of
        // the later chunks' dt A in the columns' factors: its state only collects products.
        auto begin = [&]() -> int { return SUMMARY ? first_t + (stop_t - first_t - 1) / kVarQ * kVarQ : first_t; };
        bool ok = true, more = take();
        int t = begin();
        if (more) load_dt(t);
        float item_total = 0.0f;  // of the item's chunks so far
        while (more) {
            const int rows = min(kVarQ, stop_t - t), next = SUMMARY ? t - kVarQ : t + kVarQ;
            const bool low = t == first_t, high = t + rows >= stop_t, mine = hh < nh;
            const bool first = SUMMARY ? high : low, last = SUMMARY ? low : high;
            float dt[kRows], d[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                dt[i] = __uint_as_float(static_cast<uint32_t>(raw[i]) << 16) + bias;
                if (p.softplus) dt[i] = softplus_accurate(dt[i]);
                if (kRows * sub + i >= rows || !mine) dt[i] = 0.0f;
            }
            if (!last) load_dt(next);
            // d_j = minus the sum of the later rows' dt A
            float after = 0.0f;
#pragma unroll
            for (int i = kRows - 1; i >= 0; --i) {
                d[i] = after;
                after -= dt[i] * A;
            }
            float sum = after;
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) {
                const float v = __shfl_down_sync(0xffffffffu, sum, o, kLanes);
                if (sub + o < kLanes) sum += v;
            }
            const float T = -__shfl_sync(0xffffffffu, sum, 0, kLanes);
            float later = __shfl_down_sync(0xffffffffu, sum, 1, kLanes);
            if (sub == kLanes - 1) later = 0.0f;
            const float half = 0.5f * T;  // d lies between 0 and -T where dt has one sign
            float most = fabsf(half), w[kRows], span = 0.0f;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                d[i] += later;
                most = fmaxf(most, fabsf(d[i] + half));
            }
            const float block = __shfl_sync(0xffffffffu, d[0], lane & ~(16 / kRows - 1));  // d of the first of these 16 rows
#pragma unroll
            for (int i = 0; i < kRows; ++i) span = fmaxf(span, fabsf(block - d[i]));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) {
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                span = fmaxf(span, __shfl_xor_sync(0xffffffffu, span, o));
            }
            if (first) item_total = 0.0f;
            const bool wide = !SUMMARY && most > 0.5f * kVarRange;
            const VarDecays decays = !wide ? kVarByColumn : span <= kVarSpan ? kVarByBlock : kVarOneByOne;
            // the middle of the exponents of the columns' factors, or of the rows', which are those of cs; these
            // go from 0 to T, or where dt changes its sign somewhere on both sides
            const float centre = SUMMARY ? 0.0f : !wide ? -half : most > fabsf(half) + 1.0f ? 0.0f : 0.5f * fminf(fmaxf(T, -kVarRange), kVarGrowth);
            const int k2 = __float2int_rn(centre * kLog2e);  // |k2| < 127
            const float up = __int_as_float((127 + k2) << 23);
            const float from = SUMMARY ? item_total : decays == kVarByColumn ? 0.0f : block, by = decays == kVarByColumn ? up : 1.0f;
#pragma unroll
            for (int i = 0; i < kRows; ++i) w[i] = decays == kVarOneByOne ? dt[i] : expf(from - d[i]) * by * dt[i];
            item_total += T;
            if (!ready()) {
                ok = false;
                break;
            }
#pragma unroll
            for (int i = 0; i < kRows; i += 4) {
                *reinterpret_cast<float4 *>(tabD + hh * kVarQ + kRows * sub + i) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
                *reinterpret_cast<float4 *>(tabW + hh * kVarQ + kRows * sub + i) = make_float4(w[i], w[i + 1], w[i + 2], w[i + 3]);
            }
            VarChunk *out = info + (u & 1u);
            if (sub == 0) {
                out->decay[hh] = expf(T), out->scale[hh] = decays == kVarByColumn ? expf(T) * up : up, out->D[hh] = D;
                out->ref[hh] = T, out->decays[hh] = decays;
                out->down[hh] = __int_as_float((127 - k2) << 23), out->shift[hh] = static_cast<float>(k2) * kLn2;
                if (SUMMARY && last && mine) decay[hh] = expf(item_total);
            }
            if (lane == 0 && (!SUMMARY || hh == 0)) {
                out->t0 = t, out->rows = rows;
                out->h0 = h0, out->nh = nh, out->g = g;
                out->first = first, out->last = last, out->stop = 0;
                out->src = src, out->dst = dst, out->flag = flag;
            }
            __syncwarp();
            if (lane == 0) ssd_arrive(bFull);
            ++u;
            t = next;
            if (last) {
                more = take();
                t = begin();
                if (more) load_dt(t);
            }
        }
        if (ok && ready() && lane == 0) {
            if (!SUMMARY || hh == 0) info[u & 1u].stop = 1;
            ssd_arrive(bFull);
        }
        __syncwarp();
    } else if (tid < kStateThreads) {
        // ---- the state's warps: a thread has row 32 quad + lane of every [128][..] tile (its
        // TMEM lane) and of head `head`'s columns the kCols from c0 --------------------------
        using L2 = Lanes<2>;
        const int quad = warp & 3, head = (warp >> 2) & 1, row = quad * 32 + lane, c0 = SUMMARY ? 32 * (warp >> 3) : 0;
        const uint32_t tSh = tS + (static_cast<uint32_t>(quad * 32) << 16) + 64 * head;
        const uint8_t *xraw = sm + S::kX + head * S::kTile;
        uint8_t *stile = sm + S::kS + head * S::kTile;
        uint32_t handed = 0;  // states handed on by this CTA so far
        for (uint32_t u = 0;; ++u) {
            const uint32_t ph = u & 1u;
            if (u > 0) {
                if (!wait(mS, ph ^ 1u)) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                // the state after an item leaves before anything waits for the next chunk;
                // handed on once every thread's part is written
                const VarChunk &c = info[ph ^ 1u];
                if (float *dst = c.dst; c.last && dst) {
                    if (head < c.nh) {
#pragma unroll 1
                        for (int q0 = c0; q0 < c0 + kCols; q0 += 16) {
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
            if (!wait(bFull, ph)) break;
            const VarChunk &c = info[ph];
            if (c.stop) break;
            const int rows = c.rows;
            const bool first = c.first, live = head < c.nh;
            const float *src = c.src;
            const L2 decay = lanes<2>(c.decay[head]);
            const float scale = c.scale[head];
            float w = tabW[head * kVarQ + row];
            if constexpr (!SUMMARY) {
                if (c.decays[head] == kVarByColumn) w *= c.down[head];
            }
            if (c.decays[head] != kVarByColumn)  // what is missing of exp(-d) dt
                w *= expf(-tabD[head * kVarQ + (c.decays[head] == kVarByBlock ? row & ~15 : row)]);
            if constexpr (SUMMARY) ssd_arrive(bEmpty);

            // exp(T) S, float32, to tensor memory; S, scaled as it meets C, as bf16 to its
            // operand tile [n][p]
            auto put = [&](int q0, const float (&v)[16]) {
                uint32_t r[16];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const L2 dv = decay * L2::of(v[e], v[e + 1]);
                    r[e] = __float_as_uint(dv.get(0)), r[e + 1] = __float_as_uint(dv.get(1));
                }
                ssd_st16(tSh + q0, r);
                if constexpr (!SUMMARY) {
                    uint32_t b[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) b[e] = pack_bf16x2(scale * v[2 * e], scale * v[2 * e + 1]);
                    *reinterpret_cast<uint4 *>(stile + ssd_sw128(row, q0)) = make_uint4(b[0], b[1], b[2], b[3]);
                    *reinterpret_cast<uint4 *>(stile + ssd_sw128(row, q0 + 8)) = make_uint4(b[4], b[5], b[6], b[7]);
                }
            };
#pragma unroll 1
            for (int q0 = c0; q0 < c0 + kCols; q0 += 32) {
                if (SUMMARY && !first) break;  // no decay between its chunks
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
                if (!wait(mG, ph)) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                var_factors(c, tabD, tabW, tG + (static_cast<uint32_t>(quad * 32) << 16), row, 96 + 16 * head, 128);
                ssd_arrive(bEmpty);  // the tables' last readers
                ssd_arrive(bE2);
            }

            // w x as three bf16 parts; rows past the chunk's end are zeros whatever they hold
            // (another sequence's values, or none)
            if (!wait(bX, ph)) break;
            if (!SUMMARY && !wait(mC, ph)) break;  // S read: the last part takes its place
            const bool in = row < rows && live;
            const L2 w2 = lanes<2>(w), minus = lanes<2>(-1.0f);
#pragma unroll 1
            for (int k = c0 / 8; k < (c0 + kCols) / 8; ++k) {
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
                // (with outputs C B^T was waited for, and the next chunk's B may have landed: a wait
                // for this one's could not tell them apart)
                if (SUMMARY && !wait(bCB, ph)) break;
                if (row >= rows) {
#pragma unroll
                    for (int k = c0 / 8; k < (c0 + kCols) / 8; ++k)
                        *reinterpret_cast<uint4 *>(sm + S::kB + S::kBufB * ph + head * S::kTile + ssd_sw128(row, 8 * k)) = make_uint4(0, 0, 0, 0);
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            ssd_arrive(bE1);
        }
    } else if constexpr (!SUMMARY) {
        // ---- the output's warps: a thread has row 32 quad + lane and, of y, the 64 columns of
        // head `half` ---------------------------------------------------------------------------
        using L2 = Lanes<2>;
        const int quad = warp & 3, half = (warp >> 2) & 1, row = quad * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
        uint8_t *xraw = sm + S::kX + half * S::kTile;
        for (uint32_t u = 0;; ++u) {
            const uint32_t ph = u & 1u;
            if (!wait(bFull, ph)) break;
            // read again where it is needed: this chunk's is overwritten only after everyone
            // has come to the next chunk's C B^T
            const VarChunk &c = info[ph];
            if (c.stop) break;
            const int rows = c.rows;
            const bool live = half < c.nh;
            const float e_row = expf(var_row_exponent(c, half, tabD[half * kVarQ + row]));
            // rows past the end as zeros: they are the products' operand
            if (rows < kVarQ) {
                if (!wait(bX, ph)) break;
                if (live && row >= rows) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4 *>(xraw + ssd_sw128(row, 8 * k)) = make_uint4(0, 0, 0, 0);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            if (!wait(mG, ph)) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            var_factors(c, tabD, tabW, tG + lane_off, row, 16 * half, 96);
            ssd_arrive(bEmpty);  // the tables' last readers
            ssd_arrive(bE2);

            // y = exp(.) Y + D x, in x's place in its tile (the products have read it, and the
            // state's warps had before bE1)
            if (!wait(mY, ph) || !wait(bE1, ph)) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t col = tY + 128 * ph + lane_off + 64 * half;
            const L2 eo = lanes<2>(e_row), D = lanes<2>(c.D[half]);
#pragma unroll 1
            for (int q0 = 0; q0 < 64; q0 += 16) {
                float y[16];
                ssd_ld16(col + q0, y);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint4 *at = reinterpret_cast<uint4 *>(xraw + ssd_sw128(row, q0 + 8 * k));
                    const uint4 xv = *at;
                    const uint32_t x[4] = {xv.x, xv.y, xv.z, xv.w};
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const L2 v = L2::fma(eo, L2::of(y[8 * k + 2 * e], y[8 * k + 2 * e + 1]),
                                             D * L2::of(__uint_as_float(x[e] << 16), __uint_as_float(x[e] & 0xffff0000u)));
                        o[e] = pack_bf16x2(v.get(0), v.get(1));
                    }
                    *at = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            // out of it by whole 128-byte lines, this warp's rows
            __syncwarp();
            uint4 line[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                line[k] = *reinterpret_cast<const uint4 *>(xraw + ssd_sw128(quad * 32 + 4 * k + (lane >> 3), 8 * (lane & 7)));
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next load into it
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
