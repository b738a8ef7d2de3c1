// tq_prefill_weights.cu -- chunked-prefill attention that also accumulates the attention
// weights of the chunk's last tokens, on the tcgen05 tensor cores.
//
// Attention.  One CTA takes two tiles of 128 query rows ((chunk token, query head) pairs of
// one kv head) and walks the sequence in steps of 64 tokens, its warps apart by role:
//   warps 0-7       first rotate the queries, while the others bring the first step
//   warps 0-3, 4-7  the rows of tile 0 and of tile 1, one row per thread: scores from
//                   tensor memory, key norms, causal limit, online softmax, the weights as
//                   two fp16 parts back into the same tensor-memory columns; the outputs
//                   accumulate in the threads' registers
//   warps 8-11      dequantise the step's values: fp16 high and low parts, K-major along the
//                   tokens
//   warps 13-15     the keys, as fp16 centroids (exact)
//   warp 12         issues the MMAs: S = q~ C^T with the query's two fp16 parts along K,
//                   O = [p_lo | p_hi | p_hi] [v_hi ; v_lo ; v_hi] with p from tensor memory
// The scores of step s + 1 are formed while step s is in its softmax, and the product of
// step s while step s + 1 is: two score buffers per tile, two stages of operands.
//
// Exactness.  The tensor cores cut an accumulator towards zero at every MMA; left in tensor
// memory over 32768 tokens the output loses 1e-4 of itself.  So each step's product is
// summed from zero and added to the row's fp32 registers, and the weights reach 2^15, where
// their two fp16 parts keep 22 bits down to 2^-18 of the largest.  A record with values past
// fp16 (n s + z reaches 16 times the largest of its fields) holds them at a sixteenth, and its
// products are added sixteen times.
//
// Few rows have few CTAs: their contexts are cut into parts, which leave their sums to the
// CTAs of the second kernel.
//
// Measured (2048 tokens at context 32768, 32 query / 8 kv heads, d 128): 2.6-2.7 ms, of which
// 35 us are the votes (3.8 ms where all 2048 tokens vote); the tensor pipe is active 60 % of the
// cycles of a resident CTA.  A step takes its row warps about 4000 clocks (maximum 700, weights
// 1300, product 700, barriers), against 2560 of MMA arithmetic (2.5 times that of a product of
// single fp16 parts; near 3070 if the scores' operands, 6 KB of shared memory a K step, are
// read at 128 bytes a clock), and a CTA by itself about 10 us; 256 CTAs on 148 SMs leave a
// seventh of the second wave empty.  With one thread issuing under a branch the MMAs were the
// bound (5.1 ms), with keys and values in the same warps those were (3.0 ms).  At d 128 the
// compiler spills 200-360 bytes a thread, at d 64 16-110.
//
// Votes.  token_weights[b][kv][t] += sum over the voting rows r of 2^(s_r,t - lse_r).  The
// attention leaves each voting tile's rotated queries and row statistics in the workspace;
// a second kernel forms the scores again, transposed: S^T = C q~^T with the tokens along M,
// so that a thread owns one token (one tensor-memory lane) and sums its rows' weights in
// registers, in one order.  A row whose scores are not numbers has no vote.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "tq_mma.cuh"

namespace tq {
namespace {

using WArgs = PrefillWeightsArgs;

constexpr int kRows = 128;   // query rows per tile (the M of every MMA)
constexpr int kStep = 64;    // cached tokens per step
constexpr int kVWarps = 4, kKWarps = 3;  // dequantising warps
constexpr int kThreads = 512;
constexpr float kHead = 15.f;  // weights reach 2^kHead
constexpr int kPartSteps = 8;  // a part of a context has at least these steps
constexpr int kMaxParts = 32;
constexpr long long kSMs = 148;
// Registers.  512 threads start with 128 each, the whole file; the row warps take what the
// others give.  A split above what the block was launched with would wait for ever, so the
// launcher refuses a kernel that was compiled to less.
constexpr int kRowRegs = 184, kDqRegs = 88, kIssueRegs = 56;
constexpr int kLaunchRegs = 128;
static_assert(256 * kRowRegs + 128 * kDqRegs + 128 * kIssueRegs <= kThreads * kLaunchRegs, "register split");

// ------------------------------------------------------------------ more PTX helpers
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Whether a thread of two warps says so; a barrier of theirs (id)
__device__ __forceinline__ bool pair_any(uint32_t id, bool yes) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred.aligned q, %2, 64, p;\n"
        " selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)yes), "r"(id)
        : "memory");
    return r != 0;
}
// one arrival per warp, after every lane's work
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
    __syncwarp();
    if (lane == 0) bar_arrive(bar);
}
// Global loads that stay where they are written, ahead of their use by a step.
__device__ __forceinline__ uint32_t ldg_u32(const void* p) {
    uint32_t v;
    asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint16_t ldg_u16(const void* p) {
    uint16_t v;
    asm volatile("ld.global.nc.b16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 ldg_u128(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// The issuing warp runs its loops whole and one elected lane issues, by predicate: the
// descriptors stay in uniform registers.  (Under a branch of one lane every operand is moved
// there anew, 180 clocks an MMA.)
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
    return e;
}
// D (tensor memory) (+)= A (shared memory) B (shared memory)
__device__ __forceinline__ void mma_ss(uint32_t el, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
        : "memory");
}
// D (tensor memory) (+)= A (tensor memory, fp16 pairs) B (shared memory)
__device__ __forceinline__ void mma_ts(uint32_t el, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(el)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t el, uint32_t bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
        "r"(el)
        : "memory");
}
// 16 consecutive 32-bit columns of this thread's lane: the load in flight, and its end (which
// ties the registers, so that no use moves ahead of it)
__device__ __forceinline__ void tmem_ld16_start(uint32_t taddr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :
                 : "memory");
}
// the same registers after a wait that covered their load too
__device__ __forceinline__ void tie(float (&v)[16]) {
    asm volatile(""
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// NaN if one of them is
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// x - h, the part of x that its fp16 rounding h leaves (one mixed-precision fma)
__device__ __forceinline__ float rest_of(float x, __half h) {
    float d;
    asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(d) : "h"(__half_as_ushort(h)), "h"((uint16_t)0xBC00), "f"(x));
    return d;
}

// log2 of a row's sum of 2^score from its maximum and the sum of 2^(score - maximum + kHead);
// NaN where scores that are not numbers leave no sum
__device__ __forceinline__ float row_lse(float m, float l) {
    return l > 0.f ? m - kHead + log2f(l) : __int_as_float(0x7fffffff);
}

// The row tiles of a chunk of qlen tokens that hold the rows of its last `window` tokens.
struct VoteTiles {
    int row0, rows, first, end;  // voting rows [row0, rows); tiles [first, end)
    __device__ __forceinline__ VoteTiles(int qlen, int window, int G) {
        row0 = (window > 0 && window < qlen ? qlen - window : 0) * G;
        rows = qlen * G;
        first = row0 / kRows;
        end = (rows + kRows - 1) / kRows;
    }
    // a tile's voting rows [lo, hi), and the run of its image that holds them in whole core matrices
    __device__ __forceinline__ int lo(int tile) const { return max(row0 - tile * kRows, 0); }
    __device__ __forceinline__ int hi(int tile) const { return min(rows - tile * kRows, kRows); }
    template <int D>
    __device__ __forceinline__ uint32_t from(int tile) const { return (uint32_t)(lo(tile) / 8) * (32u * D); }
    template <int D>
    __device__ __forceinline__ uint32_t bytes(int tile) const {
        return (uint32_t)((hi(tile) + 7) / 8) * (32u * D) - from<D>(tile);
    }
};

// The steps that two row tiles (from row0 on) of a chunk walk over a valid context of L tokens,
// and their cut into parts of at least kPartSteps.
struct Walk {
    int tokens, steps, parts;  // what the widest row sees
    __device__ __forceinline__ Walk(const WArgs& a, int L, int qfull, int rows_b, int G, int row0) {
        const int last_row = min(row0 + 2 * kRows, rows_b) - 1;
        tokens = L >= 0 ? L - qfull + last_row / G + 1 : 0;
        steps = (tokens + kStep - 1) / kStep;
        parts = max(1, min(a.parts, steps / kPartSteps));
    }
    // parts <= 32 and steps < 2^25
    __device__ __forceinline__ int first(int part) const { return steps * part / parts; }
};

// Eight rows of a tile into shared memory as the MMA's A operand: the rotated queries
// q~ = H q * scale log2(e) / sqrt(D), fp16 high parts at K 0 .. D-1, low parts behind.
// K-major, no swizzle: (r/8) 32 D + (k/8) 128 + (r%8) 16 + (k%8) 2.  A warp takes the eight
// rows of a core matrix, lane r + 8 q the chunks 4 j + q (8 dims each) of row r: its stores
// fill whole core matrices (a row per warp met in one bank, 17 000 clocks for 256 rows).
// src: this lane's row, null for a row of zeros; dst: the rows' place.
template <int D>
struct QRows {
    static constexpr int NJ = D / 32;
    uint4 raw[NJ];
    __device__ __forceinline__ void load(const uint16_t* src, int lane) {
#pragma unroll
        for (int j = 0; j < NJ; j++)
            raw[j] = src ? ldg_u128(src + 8 * (4 * j + (lane >> 3))) : make_uint4(0, 0, 0, 0);
    }
    // false: an element is beyond fp16 or not a number, and so will be the row's scores
    __device__ __forceinline__ bool rotate(const WArgs& a, uint32_t dst, int lane) const {
        float2 x[4 * NJ];
#pragma unroll
        for (int j = 0; j < NJ; j++) {
            const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
            for (int e = 0; e < 4; e++)
                x[4 * j + e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
        }
        if (a.rotate) {
            const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll
            for (int e = 0; e < 4 * NJ; e++) x[e] = make_float2(x[e].x + x[e].y, x[e].x - x[e].y);
#pragma unroll
            for (int m = 1; m < 4 * NJ; m <<= 1)
#pragma unroll
                for (int e = 0; e < 4 * NJ; e++)
                    if (!(e & m)) {
                        const float2 p = x[e], q = x[e | m];
                        x[e] = __fadd2_rn(p, q);
                        x[e | m] = __ffma2_rn(q, minus, p);
                    }
#pragma unroll
            for (int m = 8; m < 32; m <<= 1) {
                const float s = lane & m ? -1.f : 1.f;
                const float2 sign = make_float2(s, s);
#pragma unroll
                for (int e = 0; e < 4 * NJ; e++)
                    x[e] = __ffma2_rn(sign, x[e], make_float2(__shfl_xor_sync(kFull, x[e].x, m),
                                                              __shfl_xor_sync(kFull, x[e].y, m)));
            }
        }
        // the +-1 butterfly leaves a factor sqrt(D) that the scale takes out
        const float sc = a.rotate ? a.scale_log2 * rsqrtf((float)D) : a.scale_log2;
        const float2 sc2 = make_float2(sc, sc);
        uint32_t top = 0;  // the largest element, bits of |.|
#pragma unroll
        for (int j = 0; j < NJ; j++) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float2 v = __fmul2_rn(x[4 * j + e], sc2);
                const __half2 h = __floats2half2_rn(v.x, v.y);
                hi[e] = h2u(h);
                lo[e] = pack_h2(rest_of(v.x, __low2half(h)), rest_of(v.y, __high2half(h)));
            }
            top = __vimax3_u16x2(top, hi[0] & 0x7fff7fffu, hi[1] & 0x7fff7fffu);
            top = __vimax3_u16x2(top, hi[2] & 0x7fff7fffu, hi[3] & 0x7fff7fffu);
            store(dst, j, lane, make_uint4(hi[0], hi[1], hi[2], hi[3]), make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
        return ((top + 0x04000400u) & 0x80008000u) == 0;  // 0x7c00: infinite
    }
    __device__ __forceinline__ void zero(uint32_t dst, int lane) const {
#pragma unroll
        for (int j = 0; j < NJ; j++) store(dst, j, lane, make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0));
    }
    static __device__ __forceinline__ void store(uint32_t dst, int j, int lane, uint4 hi, uint4 lo) {
        const uint32_t at = dst + 128u * (4 * j + (lane >> 3)) + 16u * (lane & 7);
        st_s128(at, hi);
        st_s128(at + 16u * D, lo);
    }
};

// ------------------------------------------------------------------ attention
// Shared memory.  K [64 tokens][D] K-major: (t/8) 16 D + (k/8) 128 + (t%8) 16 + (k%8) 2.
// V^T hi, lo [D columns][64 tokens] K-major: (n/8) 1024 + (t/8) 128 + (n%8) 16 + (t%8) 2,
// column n = 8 (2 m + e) + r holding dim 16 m + 2 r + e, so that a warp's stores of one
// (m, e) fill the core matrices they touch.
template <int D>
struct APlan {
    static constexpr uint32_t kQ = 0;                    // two tiles of 512 D
    static constexpr uint32_t kK = kQ + 1024u * D;       // two stages
    static constexpr uint32_t kKStage = 128u * D;
    static constexpr uint32_t kV = kK + 2 * kKStage;     // two stages of hi, lo
    static constexpr uint32_t kVPart = 128u * D, kVStage = 2 * kVPart;
    static constexpr uint32_t kLut = kV + 2 * kVStage;
    static constexpr uint32_t kNorm = kLut + 1024u;      // four steps of 64 floats
    static constexpr uint32_t kBars = kNorm + 4u * 4u * kStep;
    static constexpr uint32_t kMisc = kBars + 32u * 8u;  // tensor-memory base, abort flag, part, parts
    static constexpr uint32_t kSmall = kMisc + 16u;      // two stages: a byte per record, its values at a sixteenth
    static constexpr uint32_t kEnd = kSmall + 16u;
    static_assert(kEnd <= 232448u, "227 KB per CTA");
};
// Barriers.  Step s is phase s / 2 of the ones kept per stage, s / 4 of NORM, s of the rest.
// A warp may be a step ahead of another of its role until it waits for what both feed, so
// what it arrives on before that wait is kept per stage.
enum : uint32_t {
    B_KFULL = 0,   // [stage] keys of the step in place (one arrival per warp that dequantises them)
    B_VFULL = 2,   // [stage] values
    B_KFREE = 4,   // [stage] the scores that read them are done
    B_VFREE = 6,   // [stage] the products are
    B_NORM = 8,    // [step % 4] key norms in place
    B_SFULL = 12,  // [tile][stage] scores done
    B_PFULL = 16,  // [tile][stage] weights written (one arrival per row warp)
    B_OFREE = 20,  // [tile] product taken into the registers (the same)
    B_OFULL = 22,  // [tile] product done
    B_QFULL = 24,  // the queries in place (one arrival per row warp)
    B_COUNT = 25
};
constexpr uint32_t kAbsent = 0x7fc00001u;  // the norm of a token that is not there (a NaN that no fp16 gives)
constexpr int kAgain = 16;  // products of a record whose values are held at a sixteenth
constexpr uint32_t kTileCols = 256, kOCol = 128;  // tensor memory: two score buffers of 64, product

// CUT: the contexts are cut into parts (what a part leaves behind takes registers that whole
// contexts do without: 3 % of a long prompt).
template <int D, bool CUT>
__global__ void __launch_bounds__(kThreads, 1) prefill_rows_kernel(WArgs a) {
    using R = Rec<D>;
    using PL = APlan<D>;
    constexpr uint32_t REC = R::kBytes;
    extern __shared__ __align__(1024) unsigned char psm[];
    const uint32_t base = saddr(psm);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);
    const int b = blockIdx.z, kv = blockIdx.y;
    const int pair = CUT ? blockIdx.x % a.pairs : blockIdx.x, part0 = CUT ? blockIdx.x / a.pairs : 0;
    const int G = a.Hq / a.Hkv;

    const int q0 = a.q_start[b], q1 = a.q_start[b + 1];
    const bool reporter = tid == 0 && kv == 0 && blockIdx.x == 0;
    if (q0 < 0 || q1 < q0 || q1 > a.T) {  // rows outside q / out: nothing is touched
        if (reporter) flag_status(a.status, TQ_STATUS_BAD_LEN);
        return;
    }
    const int qfull = q1 - q0;
    if (qfull > a.max_q_len && reporter) flag_status(a.status, TQ_STATUS_BAD_LEN);
    const int qlen = min(qfull, a.max_q_len);  // a longer chunk is cut: its last rows are not written
    const int rows_b = qlen * G;
    const int row0 = pair * 2 * kRows;
    if (qlen <= 0 || row0 >= rows_b) return;  // the whole CTA leaves together
    int L = a.seq_lens[b];
    if (L < qfull || L > a.max_blocks * kBlock) {  // no valid context: rows get 0
        if (reporter) flag_status(a.status, TQ_STATUS_BAD_LEN);
        L = -1;
    }
    const bool two = row0 + kRows < rows_b;  // the second tile has rows
    const Walk walk(a, L, qfull, rows_b, G, row0);
    if (CUT && part0 >= walk.parts) return;
    // this CTA's steps; tokens are counted from its first one
    const int step0 = CUT ? walk.first(part0) : 0, nsteps = CUT ? walk.first(part0 + 1) - step0 : walk.steps;
    const int maxlim = walk.tokens - kStep * step0;  // tokens the widest row sees

    const uint32_t sQ = base + PL::kQ, sK = base + PL::kK, sV = base + PL::kV;
    const uint32_t sLut = base + PL::kLut, sNorm = base + PL::kNorm, bars = base + PL::kBars;
    const uint32_t sSmall = base + PL::kSmall;
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(psm + PL::kMisc);
    auto bar = [&](uint32_t id) { return bars + 8 * id; };

    // ---- set-up: barriers, tensor memory, the centroid-pair table
    if (tid == 0) {
        for (uint32_t i = 0; i < B_COUNT; i++) {
            const bool keys = i < B_VFULL || (i >= B_NORM && i < B_SFULL);
            const bool rows = i >= B_PFULL && i < B_OFULL;
            bar_init(bar(i), keys ? kKWarps : i < B_KFREE ? kVWarps : rows ? 4 : i == B_QFULL ? 8 : 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        misc[1] = 0;
        misc[2] = (uint32_t)part0;  // for the end: no registers in between
        misc[3] = (uint32_t)walk.parts;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + PL::kMisc),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid < 256) {
        const uint16_t* tab = a.k_tables ? a.k_tables + kv * 16 : nullptr;
        const uint32_t lo = tab ? tab[tid & 15] : a.default_table[tid & 15];
        const uint32_t hi = tab ? tab[tid >> 4] : a.default_table[tid >> 4];
        st_s32(sLut + 4 * tid, lo | (hi << 16));
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = misc[0];
    bool ok = true;  // every wait of this thread's role ended
    // the dequantising roles' records: blocks behind the last one are read as the last one,
    // every field of them masked by the token's position
    const int32_t* bt = a.block_tables + (size_t)b * a.max_blocks + step0 * (kStep / kBlock);
    const int last_blk = (maxlim + kBlock - 1) / kBlock - 1;
    const unsigned char* kvbase = a.cache + (size_t)kv * REC;
    const long long blk_stride = (long long)a.Hkv * REC;
    auto block_id = [&](int s, int j) { return (int)ldg_u32(bt + min(4 * s + j, last_blk)); };
    auto record = [&](int id, bool& there) {
        there = (uint32_t)id < (uint32_t)a.num_blocks;
        if (!there) flag_status(a.status, TQ_STATUS_BAD_BLOCK);
        return kvbase + (there ? id : 0) * blk_stride;
    };

    if (warp < 8) {
        // ================================================================ rows
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
        // ---- the rotated queries of both tiles, while the other warps bring the first step
        {
            const int n8 = (two ? 2 : 1) * kRows / 64;  // eight warps take 64 rows at a time
            QRows<D> cur, next;
            auto load = [&](QRows<D>& to, int i) {
                const int Rr = row0 + 64 * i + 8 * warp + (lane & 7);
                const bool there = i < n8 && Rr < rows_b && L >= 0;
                to.load(there ? a.q + ((size_t)(q0 + Rr / G) * a.Hq + kv * G + Rr % G) * D : nullptr, lane);
            };
            load(cur, 0);
            for (int i = 0; i < n8; i++) {
                load(next, i + 1);
                const uint32_t dst = sQ + (uint32_t)(8 * i + warp) * (32u * D);
                if (row0 + 64 * i + 8 * warp >= rows_b)
                    cur.zero(dst, lane);
                else if (!cur.rotate(a, dst, lane))
                    flag_status(a.status, TQ_STATUS_RANGE);
                cur = next;
            }
            async_proxy_fence();
            warp_arrive(bar(B_QFULL), lane);
        }
        const int tile = warp >> 2;
        const int R_ = row0 + tile * kRows + (tid & 127);  // this thread's row
        const bool row_ok = R_ < rows_b;
        const int ri = R_ / G, rh = R_ % G;
        // it sees positions < lim; a row that is not there sees all, so that its warp takes no masks
        // for it (what it gives is not used)
        const int lim = row_ok ? L - qfull + ri + 1 - kStep * step0 : 0x7fffffff;
        const uint32_t tT = tmem + (uint32_t)tile * kTileCols + ((uint32_t)(32 * (warp & 3)) << 16);
        float o[D];
#pragma unroll
        for (int j = 0; j < D; j++) o[j] = 0.f;
        float m_run = -INFINITY, l_run = 0.f, corr_prev = 1.f;
        // o = o * corr + the product in tensor memory
        auto take = [&](float corr) {
            const float2 c2 = make_float2(corr, corr);
            float t[2][16];
            tmem_ld16_start(tT + kOCol, t[0]);
#pragma unroll
            for (int c = 0; c < D / 16; c++) {
                tmem_ld_wait(t[c & 1]);
                if (c + 1 < D / 16) tmem_ld16_start(tT + kOCol + 16u * (c + 1), t[(c + 1) & 1]);
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    float* oj = o + 16 * c + j;
                    const float2 r =
                        __ffma2_rn(make_float2(oj[0], oj[1]), c2, make_float2(t[c & 1][j], t[c & 1][j + 1]));
                    oj[0] = r.x;
                    oj[1] = r.y;
                }
            }
        };
        const int n = tile == 0 || two ? nsteps : 0;
#pragma unroll 1
        for (int s = 0; s < n && ok; s++) {
            const bool r0 = bar_try(bar(B_NORM + (s & 3)), (uint32_t)(s >> 2) & 1u);
            const bool r1 = bar_try(bar(B_SFULL + 2 * tile + (s & 1)), (uint32_t)(s >> 1) & 1u);
            ok = (r0 || bar_wait(bar(B_NORM + (s & 3)), (uint32_t)(s >> 2) & 1u)) &&
                 (r1 || bar_wait(bar(B_SFULL + 2 * tile + (s & 1)), (uint32_t)(s >> 1) & 1u));
            ok = __all_sync(kFull, ok);
            if (!ok) break;
            tc_after_sync();
            const uint32_t tS = tT + (uint32_t)(s & 1) * kStep;
            const uint32_t nrm = sNorm + (uint32_t)(s & 3) * (4u * kStep);
            // the row's maximum, then the weights; MASK: some row does not see the whole step, or a
            // token is not there.  Its norm makes the maximum NaN, with which the other variant
            // ends, before it has written anything.
            float corr = 1.f;
            float2 l2 = make_float2(0.f, 0.f);
            auto softmax = [&](auto mask) -> bool {
                constexpr bool MASK = decltype(mask)::value;
                // 16 tokens in flight at a time; at D = 64 there are registers for all 64,
                // which then are read and scaled once
                constexpr bool KEEP = D == 64;
                // scores 16 c + j .. + 3 times their norms, plus add
                auto four = [&](const float* xc, int c, int j, float2 add, float2& y, float2& z) {
                    const uint4 nw = ld_s128(nrm + 64u * c + 4u * j);
                    y = __ffma2_rn(make_float2(xc[0], xc[1]),
                                   make_float2(__uint_as_float(nw.x), __uint_as_float(nw.y)), add);
                    z = __ffma2_rn(make_float2(xc[2], xc[3]),
                                   make_float2(__uint_as_float(nw.z), __uint_as_float(nw.w)), add);
                    if constexpr (MASK) {
                        const int t = kStep * s + 16 * c + j;
                        y.x = t < lim && nw.x != kAbsent ? y.x : -INFINITY;
                        y.y = t + 1 < lim && nw.y != kAbsent ? y.y : -INFINITY;
                        z.x = t + 2 < lim && nw.z != kAbsent ? z.x : -INFINITY;
                        z.y = t + 3 < lim && nw.w != kAbsent ? z.y : -INFINITY;
                    }
                };
                constexpr int NX = KEEP ? 4 : 2;
                float x[NX][16];
                float m2[2] = {-INFINITY, -INFINITY};
                const float2 zero = make_float2(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < NX - 1; c++) tmem_ld16_start(tS + 16u * c, x[c]);
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    float(&xc)[16] = x[c % NX];
                    if (KEEP && c == 0) tmem_ld16_start(tS + 48u, x[NX - 1]);
                    if (!KEEP || c == 0) tmem_ld_wait(xc);
                    if (KEEP && c > 0) tie(xc);
                    if (!KEEP && c < 3) tmem_ld16_start(tS + 16u * (c + 1), x[(c + 1) % NX]);
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        float2 y, z;
                        four(xc + j, c, j, zero, y, z);
                        if (KEEP) xc[j] = y.x, xc[j + 1] = y.y, xc[j + 2] = z.x, xc[j + 3] = z.y;
                        m2[0] = MASK ? max3(m2[0], y.x, y.y) : max3_nan(m2[0], y.x, y.y);
                        m2[1] = MASK ? max3(m2[1], z.x, z.y) : max3_nan(m2[1], z.x, z.y);
                    }
                }
                const float mn = MASK ? max3(m_run, m2[0], m2[1]) : max3_nan(m_run, m2[0], m2[1]);
                if (!MASK && __any_sync(kFull, isnan(mn))) return false;
                corr = m_run == -INFINITY ? 1.f : exp2a(m_run - mn);
                m_run = mn;
                // a row that has seen no token yet takes 0 as its reference: 2^-inf = 0
                const float ref = mn == -INFINITY ? 0.f : mn - kHead;
                const float2 nref = make_float2(-ref, -ref);
                if (!KEEP) tmem_ld16_start(tS, x[0]);
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    float(&xc)[16] = x[c % NX];
                    if (!KEEP) {
                        tmem_ld_wait(xc);
                        if (c < 3) tmem_ld16_start(tS + 16u * (c + 1), x[(c + 1) % NX]);
                    }
                    uint32_t w[16];  // high parts of tokens 2j, 2j + 1 in w[j], low parts in w[8 + j]
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        float2 y, z;
                        if (KEEP) {
                            y = __fadd2_rn(make_float2(xc[j], xc[j + 1]), nref);
                            z = __fadd2_rn(make_float2(xc[j + 2], xc[j + 3]), nref);
                        } else {
                            four(xc + j, c, j, nref, y, z);
                        }
                        const float2 p0 = make_float2(exp2a(y.x), exp2a(y.y)), p1 = make_float2(exp2a(z.x), exp2a(z.y));
                        l2 = __fadd2_rn(l2, __fadd2_rn(p0, p1));
                        const __half2 h0 = __floats2half2_rn(p0.x, p0.y), h1 = __floats2half2_rn(p1.x, p1.y);
                        w[j / 2] = h2u(h0);
                        w[j / 2 + 1] = h2u(h1);
                        w[8 + j / 2] = pack_h2(rest_of(p0.x, __low2half(h0)), rest_of(p0.y, __high2half(h0)));
                        w[8 + j / 2 + 1] = pack_h2(rest_of(p1.x, __low2half(h1)), rest_of(p1.y, __high2half(h1)));
                    }
                    tmem_st16u(tS + 16u * c, w);
                }
                return true;
            };
            if (!__all_sync(kFull, kStep * (s + 1) <= lim) || !softmax(std::false_type{})) softmax(std::true_type{});
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_before_sync();
            warp_arrive(bar(B_PFULL + 2 * tile + (s & 1)), lane);
            l_run = fmaf(l_run, corr, l2.x + l2.y);
            if (s > 0) {  // the product of the step before
                ok = __all_sync(kFull, bar_wait(bar(B_OFULL + tile), (uint32_t)(s - 1) & 1u));
                if (!ok) break;
                tc_after_sync();
                take(corr_prev);
                tc_before_sync();
                warp_arrive(bar(B_OFREE + tile), lane);
            }
            corr_prev = corr;
        }
        if (n > 0 && ok) {
            ok = __all_sync(kFull, bar_wait(bar(B_OFULL + tile), (uint32_t)(n - 1) & 1u));
            tc_after_sync();
            if (ok) take(corr_prev);
        }
        tc_before_sync();
        if (!ok) misc[1] = 1;
        // ---- the row's statistics, if it votes
        const VoteTiles vt(qlen, a.window, G);
        const int vtile = 2 * pair + tile - vt.first;
        const int part = CUT ? (int)misc[2] : 0, parts = CUT ? (int)misc[3] : 1;
        if (parts == 1 && vtile >= 0 && 2 * pair + tile < vt.end) {
            const size_t at = ((size_t)b * a.Hkv + kv) * a.wtiles + vtile;
            a.lse[at * kRows + (tid & 127)] = ok && row_ok && R_ >= vt.row0 ? row_lse(m_run, l_run) : INFINITY;
        }
        // ---- the row's output in dim order, or a part's sums, rows side by side, and what they
        // refer to
        const size_t at = (((size_t)b * a.Hkv + kv) * a.pairs + pair) * a.parts + part;
        if (parts > 1)  // (a part that gave up leaves its rows without a vote: their sums are not numbers)
            a.part_stat[at * (2 * kRows) + tid] = make_float2(m_run, ok ? l_run : NAN);
        if (row_ok) {
            const float f = parts > 1 ? 1.f : ok && l_run > 0.f ? 1.f / l_run : 0.f;
            float4* dst = parts > 1 ? a.part_o + at * (2 * kRows * D / 4) + tid
                                    : reinterpret_cast<float4*>(a.out) +
                                          ((size_t)(q0 + ri) * a.Hq + kv * G + rh) * (D / 4);
            const int step = parts > 1 ? 2 * kRows : 1;
#pragma unroll
            for (int m = 0; m < D / 16; m++)
#pragma unroll
                for (int r = 0; r < 8; r += 2, dst += step)  // dims 16 m + 2 r ..: columns of e = 0 and e = 1
                    *dst = make_float4(o[16 * m + r] * f, o[16 * m + 8 + r] * f, o[16 * m + r + 1] * f,
                                       o[16 * m + 8 + r + 1] * f);
        }
    } else if (warp < 12) {
        // ================================================================ values
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDqRegs));
        // tokens 8 vg .. 8 vg + 7 of the step (half vh of record vg / 2, vg = vg0 + 4 n), byte
        // row vr, word vq of its chunks: dims 16 (2 vq + mm) + 2 vr + e of group vq
        constexpr int NI = D / 64;
        const int vr = lane & 7, vq = D == 128 ? lane >> 3 : (lane >> 3) & 1;
        const int vg0 = D == 128 ? warp - 8 : warp - 8 + 4 * (lane >> 4);
        const int vh = vg0 & 1;
        // what a load brings is first touched where it is used, a step later
        uint32_t vw[NI][4], vs[NI][4], vz[NI][4];  // per token pair: codes, scales, zero points
        bool there[NI];
        int id[NI];
        auto ids = [&](int s) {
#pragma unroll
            for (int n = 0; n < NI; n++) id[n] = block_id(s, (vg0 + 4 * n) >> 1);
        };
        auto load = [&]() {
#pragma unroll
            for (int n = 0; n < NI; n++) {
                const unsigned char* rec = record(id[n], there[n]);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int p = 4 * vh + i;
                    vw[n][i] = ldg_u32(rec + R::kVCodes + (8 * p + ((vr + 2 * p) & 7)) * R::kPairChunk + 4 * vq);
                    const int u = (i * R::kGroups + vq) * 8 + 4 * vh;
                    vs[n][i] = ldg_u32(rec + R::kVScale + u);
                    vz[n][i] = ldg_u32(rec + R::kVZero + u);
                }
            }
        };
        // Scale and zero point of the tokens of pair i that are there, else 0 (the fields of others
        // may hold anything)
        auto fields = [&](int s, int n, int i, float2& sf, float2& zf) {
            const int t = kStep * s + 8 * (vg0 + 4 * n) + 2 * i;
            const uint32_t m = there[n] ? (t < maxlim ? 0xffffu : 0u) | (t + 1 < maxlim ? 0xffff0000u : 0u) : 0u;
            sf = __half22float2(u2h(vs[n][i] & m));
            zf = __half22float2(u2h(vz[n][i] & m));
        };
        // Which of the warp's two records, as bits, hold values past fp16; with the other warp of
        // those records (even and odd halves)
        const uint32_t pair_bar = 1 + ((warp - 8) >> 1);
        auto record_of = [&](int n) { return D == 128 ? n : lane >> 4; };
        auto past_fp16 = [&](int s) {
            bool past[2] = {false, false};
#pragma unroll
            for (int n = 0; n < NI; n++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    float2 sf, zf;
                    fields(s, n, i, sf, zf);
                    const float most = fmaxf(fmaxf(fabsf(zf.x), fabsf(fmaf(15.f, sf.x, zf.x))),
                                             fmaxf(fabsf(zf.y), fabsf(fmaf(15.f, sf.y, zf.y))));
                    past[0] |= record_of(n) == 0 && most > 65504.f;
                    past[1] |= record_of(n) == 1 && most > 65504.f;
                }
            const uint32_t first = pair_any(pair_bar, past[0]);
            return first | (uint32_t)pair_any(pair_bar, past[1]) << 1;
        };
        if (nsteps > 0) {
            ids(0);
            load();
            ids(1);
        }
#pragma unroll 1
        for (int s = 0; s < nsteps; s++) {
            const uint32_t st = (uint32_t)s & 1u;
            // does a value pass fp16?  Not while every field is below 2^11 (0x6800): 15 s + |z| < 2^15
            uint32_t top = 0;  // the largest fields, as bits of |.|
#pragma unroll
            for (int n = 0; n < NI; n++)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    top = __vimax3_u16x2(top, vs[n][i] & 0x7fff7fffu, vz[n][i] & 0x7fff7fffu);
            // the two warps of a record agree; one that gave up says so, and they leave together
            uint32_t small = 0;
            if (pair_any(pair_bar, ((top + 0x18001800u) & 0x80008000u) != 0 || !ok)) {
                if (pair_any(pair_bar, !ok)) {
                    ok = false;
                    break;
                }
                small = past_fp16(s);
            }
            if (s >= 2) ok = __all_sync(kFull, bar_wait(bar(B_VFREE + st), ((uint32_t)(s >> 1) + 1u) & 1u));
            if (!ok) continue;  // to the next agreement
            if (vh == 0 && lane < 2) st_s8(sSmall + 4 * st + (uint32_t)((warp - 8) >> 1) + 2u * lane, small >> lane);
#pragma unroll
            for (int n = 0; n < NI; n++) {
                const uint32_t dst = sV + st * PL::kVStage + (uint32_t)(vq * 4096 + (vg0 + 4 * n) * 128 + vr * 16);
                float2 sf[4], zf[4];
#pragma unroll
                for (int i = 0; i < 4; i++) fields(s, n, i, sf[i], zf[i]);
                if (small) {
                    const float f = (small >> record_of(n)) & 1u ? 1.f / kAgain : 1.f;
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        sf[i] = __fmul2_rn(sf[i], make_float2(f, f));
                        zf[i] = __fmul2_rn(zf[i], make_float2(f, f));
                    }
                }
#pragma unroll
                for (int me = 0; me < 4; me++) {  // (mm, e): byte mm of the token's two, nibble e
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const uint32_t w = me >= 2 ? vw[n][i] >> 8 : vw[n][i];
                        // the codes n of the pair as fp16: in the low bits of 1024's mantissa
                        const __half2 nn =
                            me & 1 ? __hfma2(u2h((w & 0x00F000F0u) | 0x64006400u), __floats2half2_rn(0.0625f, 0.0625f),
                                             __floats2half2_rn(-64.f, -64.f))
                                   : __hsub2(u2h((w & 0x000F000Fu) | 0x64006400u), __floats2half2_rn(1024.f, 1024.f));
                        // v = n s + z in fp32, as its fp16 rounding and the rest
                        const float2 v = __ffma2_rn(__half22float2(nn), sf[i], zf[i]);
                        const __half2 h = __floats2half2_rn(v.x, v.y);
                        hi[i] = h2u(h);
                        lo[i] = pack_h2(rest_of(v.x, __low2half(h)), rest_of(v.y, __high2half(h)));
                    }
                    st_s128(dst + 1024u * me, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                    st_s128(dst + PL::kVPart + 1024u * me, make_uint4(lo[0], lo[1], lo[2], lo[3]));
                }
            }
            async_proxy_fence();
            warp_arrive(bar(B_VFULL + st), lane);
            if (s + 1 < nsteps) load();
            ids(s + 2);
        }
        if (!ok) misc[1] = 1;
    } else {
        // one instruction for the whole warpgroup
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp > 12) {
            // ================================================================ keys
            // 16 code bytes (32 dims, part kq) of token kt: D / 32 parts of 64 tokens over 96 threads
            constexpr int kJobs = 64 * (D / 32), NJ = (kJobs + 32 * kKWarps - 1) / (32 * kKWarps);
            const int job0 = tid - 32 * 13;
            uint4 kw[NJ];
            uint16_t kn = 0;
            bool there0 = false;  // of the first job's token, whose norm this thread brings
            int id[NJ];
            auto ids = [&](int s) {
#pragma unroll
                for (int i = 0; i < NJ; i++) id[i] = block_id(s, ((job0 + 32 * kKWarps * i) & 63) >> 4);
            };
            auto load = [&]() {
#pragma unroll
                for (int i = 0; i < NJ; i++) {
                    const int job = job0 + 32 * kKWarps * i, kt = job & 63, kq = job >> 6;
                    bool there;
                    const unsigned char* rec = record(id[i], there);
                    if (job < kJobs) kw[i] = ldg_u128(rec + (kt & 15) * R::kCodeRow + 16 * kq);
                    if (i == 0) {
                        kn = ldg_u16(rec + R::kKNorm + 2 * (kt & 15));
                        there0 = there;
                    }
                }
            };
            if (nsteps > 0) {
                ids(0);
                load();
                ids(1);
            }
#pragma unroll 1
            for (int s = 0; s < nsteps; s++) {
                const uint32_t st = (uint32_t)s & 1u;
                if (s >= 2) ok = __all_sync(kFull, bar_wait(bar(B_KFREE + st), ((uint32_t)(s >> 1) + 1u) & 1u));
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < NJ; i++) {
                    const int job = job0 + 32 * kKWarps * i, kt = job & 63, kq = job >> 6;
                    if (job >= kJobs) continue;
                    const uint32_t row =
                        sK + st * PL::kKStage + (uint32_t)((kt / 8) * (16 * D) + (kt % 8) * 16 + kq * 512);
                    const uint32_t ws[4] = {kw[i].x, kw[i].y, kw[i].z, kw[i].w};
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        const uint32_t w = ws[c];
                        st_s128(row + 128u * c,
                                make_uint4(ld_s32(sLut + 4 * (w & 0xFFu)), ld_s32(sLut + 4 * ((w >> 8) & 0xFFu)),
                                           ld_s32(sLut + 4 * ((w >> 16) & 0xFFu)), ld_s32(sLut + 4 * (w >> 24))));
                    }
                }
                if (job0 < 64) {  // (behind the last token the field may hold anything)
                    const float norm = kStep * s + job0 < maxlim ? half_bits_to_float(kn) : 0.f;
                    st_s32(sNorm + (uint32_t)(s & 3) * (4u * kStep) + 4u * job0,
                           there0 ? __float_as_uint(norm) : kAbsent);
                }
                async_proxy_fence();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(bar(B_KFULL + st));
                    bar_arrive(bar(B_NORM + (s & 3)));
                }
                if (s + 1 < nsteps) load();
                ids(s + 2);
            }
            if (!ok) misc[1] = 1;
        } else {
            // ============================================================ MMA issue
            constexpr uint32_t idS = idesc_f16(kRows, kStep, 0), idO = idesc_f16(kRows, D, 0);
            const uint32_t el = elect_one();
            // what the loops and operands depend on, from lane 0: known to be uniform
            const int tiles = __shfl_sync(kFull, two ? 2 : 1, 0), steps = __shfl_sync(kFull, nsteps, 0);
            const uint32_t tm = __shfl_sync(kFull, tmem, 0);
            // descriptors: 16-byte units, so 16 more a K step of 256 bytes
            const uint64_t dq = mdesc(sQ, 128, 32 * D), dk = mdesc(sK, 128, 16 * D), dv = mdesc(sV, 128, 1024);
            auto wait = [&](uint32_t id, uint32_t ph) {
                ok = ok && __all_sync(kFull, bar_wait(bar(id), ph));
                return ok;
            };
            auto scores = [&](uint32_t st, int tile) {
                const uint64_t a = dq + (uint64_t)tile * (512 * D / 16), b = dk + (uint64_t)st * (PL::kKStage / 16);
                const uint32_t d = tm + (uint32_t)tile * kTileCols + st * kStep;
                // (the queries' low parts first: a sum is cut by what it is when a product joins it)
#pragma unroll
                for (int ks = 0; ks < 2 * D / 16; ks++)
                    mma_ss(el, d, a + 16 * (ks ^ (D / 16)), b + 16 * (ks % (D / 16)), idS, ks > 0);
                commit(el, bar(B_SFULL + 2 * tile + st));
            };
            wait(B_QFULL, 0);
            if (ok && part0 == 0 && lane == 0) {  // the queries of the tiles that vote
                const VoteTiles vt(qlen, a.window, G);
                for (int t = 0; t < tiles; t++) {
                    const int tile = 2 * pair + t;
                    if (tile < vt.first || tile >= vt.end) continue;
                    const size_t at = ((size_t)b * a.Hkv + kv) * a.wtiles + (tile - vt.first);
                    const uint32_t from = vt.from<D>(tile);
                    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                                     a.q_img + at * (512u * D) + from),
                                 "r"(sQ + (uint32_t)t * (512u * D) + from), "r"(vt.bytes<D>(tile))
                                 : "memory");
                }
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            __syncwarp();
            if (steps > 0 && ok && wait(B_KFULL, 0)) {
                tc_after_sync();
                for (int t = 0; t < tiles; t++) scores(0, t);
                commit(el, bar(B_KFREE));
            }
            // a tile's next scores, then its product: the tiles run half a step apart, and
            // neither waits for the other's softmax to get its scores
#pragma unroll 1
            for (int s = 0; s < steps && ok; s++) {
                const uint32_t st = (uint32_t)s & 1u, nx = st ^ 1u;
                const bool more = s + 1 < steps;
                if (more) wait(B_KFULL + nx, (uint32_t)((s + 1) >> 1) & 1u);
                for (int t = 0; t < tiles && ok; t++) {
                    if (more) {
                        // its buffer held the weights of step s - 1, read by that step's product
                        if (s > 0) wait(B_OFULL + t, (uint32_t)(s - 1) & 1u);
                        if (!ok) break;
                        tc_after_sync();
                        scores(nx, t);
                        if (t == tiles - 1) commit(el, bar(B_KFREE + nx));
                    }
                    if (t == 0) wait(B_VFULL + st, (uint32_t)(s >> 1) & 1u);
                    wait(B_PFULL + 2 * t + st, (uint32_t)(s >> 1) & 1u);
                    if (s > 0) wait(B_OFREE + t, (uint32_t)(s - 1) & 1u);
                    if (!ok) break;
                    tc_after_sync();
                    const uint32_t tb = tm + (uint32_t)t * kTileCols, pa = tb + st * kStep;
                    const uint64_t b = dv + (uint64_t)st * (PL::kVStage / 16);
                    // (p_hi v_lo and p_lo v_hi before the large products)
#pragma unroll
                    for (int seg = 2; seg >= 0; seg--)
#pragma unroll
                        for (int ks = 0; ks < kStep / 16; ks++)
                            mma_ts(el, tb + kOCol, pa + 16u * ks + (seg == 2 ? 8u : 0u),
                                   b + (seg == 1 ? PL::kVPart / 16 : 0u) + 16 * ks, idO, seg < 2 || ks > 0);
                    // a record that holds a sixteenth, fifteen times more
                    const uint32_t small = ld_s32(sSmall + 4 * st);
                    if (__any_sync(kFull, small != 0)) {
#pragma unroll 1
                        for (int i = 0; i < 3 * (kAgain - 1) * (kStep / 16); i++) {
                            const int seg = i % 3, ks = i / (3 * (kAgain - 1));
                            if ((small >> (8 * ks)) & 1u)
                                mma_ts(el, tb + kOCol, pa + 16u * ks + (seg == 2 ? 8u : 0u),
                                       b + (seg == 1 ? PL::kVPart / 16 : 0u) + 16 * ks, idO, 1);
                        }
                    }
                    commit(el, bar(B_OFULL + t));
                }
                if (!ok) break;
                commit(el, bar(B_VFREE + st));
            }
            // every MMA has been seen to end: the products by the waits of the rows, and here
            if (steps > 0)
                for (int t = 0; t < tiles && ok; t++) wait(B_OFULL + t, (uint32_t)(steps - 1) & 1u);
            if (!ok) misc[1] = 1;
            if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
            __syncwarp();
        }
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    if (tid == 0 && misc[1]) flag_status(a.status, TQ_STATUS_TIMEOUT);
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// ------------------------------------------------------------------ votes
template <int D>
struct VPlan {
    static constexpr uint32_t kQ = 0;                       // [128 rows][2 D], the image
    static constexpr uint32_t kK = kQ + 512u * D;           // [128 tokens][D]
    static constexpr uint32_t kLut = kK + 256u * D;
    static constexpr uint32_t kLse = kLut + 1024u;
    static constexpr uint32_t kLim = kLse + 4u * kRows;
    static constexpr uint32_t kBars = kLim + 4u * kRows;    // the image, S
    static constexpr uint32_t kMisc = kBars + 16u;
    static constexpr uint32_t kEnd = kMisc + 16u;
    static constexpr int kCtas = D == 128 ? 2 : 4;  // per SM
    static_assert(kCtas * (kEnd + 1024u) <= 233472u, "228 KB per SM, 1 KB of it per CTA");
};

// The maximum and the sum (of 2^(score - maximum + kHead)) of a row whose context was cut.
__device__ __forceinline__ float2 join_stats(const float2* st, int parts) {
    float2 r = make_float2(-INFINITY, 0.f);
#pragma unroll 4
    for (int c = 0; c < parts; c++) r.x = fmaxf(r.x, st[(size_t)c * (2 * kRows)].x);
    if (r.x == -INFINITY) return r;  // no token seen
#pragma unroll 4
    for (int c = 0; c < parts; c++) {
        const float2 s = st[(size_t)c * (2 * kRows)];
        r.y = fmaf(exp2a(s.x - r.x), s.y, r.y);
    }
    return r;
}

// Dims 16 m .. 16 m + 15 of the outputs of one row tile from its parts, one row per thread.
template <int D>
__device__ __forceinline__ void join_rows(const WArgs& a, int b, int kv, int G, int q0, int qfull, int qlen, int L,
                                          int tile, int m) {
    const int pair = tile / 2, R_ = tile * kRows + (int)threadIdx.x, r = R_ - pair * 2 * kRows, rows_b = qlen * G;
    if (pair >= a.pairs || R_ >= rows_b) return;
    const Walk walk(a, L, qfull, rows_b, G, pair * 2 * kRows);
    if (walk.parts == 1) return;  // written by the attention kernel
    const size_t at = (((size_t)b * a.Hkv + kv) * a.pairs + pair) * a.parts;
    const float2* st = a.part_stat + at * (2 * kRows) + r;
    const float2 total = join_stats(st, walk.parts);
    const float4* src = a.part_o + at * (2 * kRows * D / 4) + (4 * m) * (2 * kRows) + r;
    float4 o[4];
#pragma unroll
    for (int j = 0; j < 4; j++) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int c = 0; c < walk.parts; c++, src += 2 * kRows * D / 4) {
        const float f = total.x == -INFINITY ? 0.f : exp2a(st[(size_t)c * (2 * kRows)].x - total.x);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float4 v = src[j * (2 * kRows)];
            o[j].x = fmaf(f, v.x, o[j].x);
            o[j].y = fmaf(f, v.y, o[j].y);
            o[j].z = fmaf(f, v.z, o[j].z);
            o[j].w = fmaf(f, v.w, o[j].w);
        }
    }
    const float inv = total.y > 0.f ? 1.f / total.y : 0.f;
    float4* dst = reinterpret_cast<float4*>(a.out) + ((size_t)(q0 + R_ / G) * a.Hq + kv * G + R_ % G) * (D / 4);
#pragma unroll
    for (int j = 0; j < 4; j++)
        dst[4 * m + j] = make_float4(o[j].x * inv, o[j].y * inv, o[j].z * inv, o[j].w * inv);
}

// A CTA takes every vblocks-th tile of 128 tokens.
template <int D>
__global__ void __launch_bounds__(kRows, VPlan<D>::kCtas) votes_kernel(WArgs a) {
    using R = Rec<D>;
    using PL = VPlan<D>;
    extern __shared__ __align__(1024) unsigned char psm[];
    const uint32_t base = saddr(psm);
    const int tid = threadIdx.x, warp = tid >> 5;
    const bool join = (int)blockIdx.z >= a.B;  // the layers behind those of the votes
    const int b = join ? blockIdx.z - a.B : blockIdx.z, kv = blockIdx.y, G = a.Hq / a.Hkv;
    if (!join && (int)blockIdx.x >= a.vblocks) return;
    // The block of this thread's token in a tile; behind the table: none.
    auto block_of = [&](int tile) {
        const int blk = tile * (kRows / kBlock) + tid / kBlock;
        return blk < a.max_blocks ? (int)ldg_u32(a.block_tables + (size_t)b * a.max_blocks + blk) : -1;
    };
    int blk = block_of(blockIdx.x);
    const int q0 = a.q_start[b], q1 = a.q_start[b + 1];
    if (q0 < 0 || q1 <= q0 || q1 > a.T) return;  // flagged by the attention kernel
    const int qfull = q1 - q0;
    const int qlen = min(qfull, a.max_q_len);
    const int L = a.seq_lens[b];
    if (L < qfull || L > a.max_blocks * kBlock) return;
    if (join) {
        join_rows<D>(a, b, kv, G, q0, qfull, qlen, L, blockIdx.x / (D / 16), blockIdx.x % (D / 16));
        return;
    }
    if (L > a.w_stride) {  // no room for its sums
        if (tid == 0 && kv == 0 && blockIdx.x == 0) flag_status(a.status, TQ_STATUS_BAD_LEN);
        return;
    }
    const int tiles = (L + kRows - 1) / kRows;
    if ((int)blockIdx.x >= tiles) return;
    const VoteTiles vt(qlen, a.window, G);
    const int votes = vt.end - vt.first;
    // What a token needs from memory, in flight while the tile before is worked on.
    bool there;
    uint4 codes[D / 32];
    uint16_t norm_bits;
    float before;
    float* const sums = a.token_weights + ((size_t)b * a.Hkv + kv) * a.w_stride;
    auto bring = [&](int tile) {
        const int t = tile * kRows + tid;
        there = t < L && (uint32_t)blk < (uint32_t)a.num_blocks;
        const unsigned char* rec = a.cache + ((size_t)(there ? blk : 0) * a.Hkv + kv) * R::kBytes;
#pragma unroll
        for (int c = 0; c < D / 32; c++) codes[c] = ldg_u128(rec + (t % kBlock) * R::kCodeRow + 16 * c);
        norm_bits = ldg_u16(rec + R::kKNorm + 2 * (t % kBlock));
        before = there ? sums[t] : 0.f;
    };
    bring(blockIdx.x);
    blk = block_of((int)blockIdx.x + a.vblocks);

    const uint32_t sQ = base + PL::kQ, sK = base + PL::kK, sLut = base + PL::kLut;
    const uint32_t barQ = base + PL::kBars, barS = barQ + 8;
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(psm + PL::kMisc);
    float* lse = reinterpret_cast<float*>(psm + PL::kLse);
    int* lim = reinterpret_cast<int*>(psm + PL::kLim);
    if (tid == 0) {
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(barQ) : "memory");
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(barS) : "memory");
        misc[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + PL::kMisc),
                     "r"(128u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const uint16_t* tab = a.k_tables ? a.k_tables + kv * 16 : nullptr;
    for (int v = tid; v < 256; v += kRows) {
        const uint32_t lo = tab ? tab[v & 15] : a.default_table[v & 15];
        const uint32_t hi = tab ? tab[v >> 4] : a.default_table[v >> 4];
        st_s32(sLut + 4 * v, lo | (hi << 16));
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = misc[0];
    const uint32_t lane_off = (uint32_t)(32 * warp) << 16;
    const size_t at0 = ((size_t)b * a.Hkv + kv) * a.wtiles;
    // The voting queries of tile v (thread 0): one tile's stay, several are loaded in turn, the
    // next ones while the weights of the tile before are summed.
    auto load = [&](int v) {
        if (tid != 0) return;
        const uint32_t from = vt.from<D>(vt.first + v), bytes = vt.bytes<D>(vt.first + v);
        async_proxy_fence();
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(barQ), "r"(bytes) : "memory");
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         sQ + from),
                     "l"(a.q_img + (at0 + v) * (512u * D) + from), "r"(bytes), "r"(barQ)
                     : "memory");
    };
    load(0);
    // log2 of the sum of 2^score of this thread's row of voting tile v; +inf or NaN: no vote
    auto lse_of = [&](int v) {
        const int tile = vt.first + v, pair = tile / 2, R_ = tile * kRows + tid;
        const Walk walk(a, L, qfull, qlen * G, G, pair * 2 * kRows);
        if (walk.parts == 1) return a.lse[(at0 + v) * kRows + tid];
        if (R_ < vt.row0 || R_ >= qlen * G) return INFINITY;
        const size_t at = (((size_t)b * a.Hkv + kv) * a.pairs + pair) * a.parts;
        const float2 s = join_stats(a.part_stat + at * (2 * kRows) + (R_ - pair * 2 * kRows), walk.parts);
        return row_lse(s.x, s.y);
    };
    float mine = lse_of(0);
    uint32_t loads = 0, products = 0;  // phases of the barriers
    bool ok = true;
#pragma unroll 1
    for (int tile = blockIdx.x; tile < tiles && ok; tile += a.vblocks) {
        const int t = tile * kRows + tid;
        // this token's centroids as a row of A; a token that is not there is 0
        const bool here = there;
        const float norm = here ? half_bits_to_float(norm_bits) : 0.f, old = before;
        {
            const uint32_t row = sK + (uint32_t)((tid / 8) * (16 * D) + (tid % 8) * 16);
#pragma unroll
            for (int c = 0; c < D / 8; c++) {
                const uint4 c4 = codes[c / 4];
                const uint32_t w = c % 4 == 0 ? c4.x : c % 4 == 1 ? c4.y : c % 4 == 2 ? c4.z : c4.w;
                uint4 w4 = make_uint4(ld_s32(sLut + 4 * (w & 0xFFu)), ld_s32(sLut + 4 * ((w >> 8) & 0xFFu)),
                                      ld_s32(sLut + 4 * ((w >> 16) & 0xFFu)), ld_s32(sLut + 4 * (w >> 24)));
                if (!here) w4 = make_uint4(0, 0, 0, 0);
                st_s128(row + 128u * c, w4);
            }
        }
        const bool last = tile + a.vblocks >= tiles;
        if (!last) {
            bring(tile + a.vblocks);
            blk = block_of(tile + 2 * a.vblocks);
        }
        float sum = 0.f;
#pragma unroll 1
        for (int v = 0; v < votes; v++) {
            if (votes > 1 || tile == (int)blockIdx.x) {
                lse[tid] = mine;
                // the last position row r sees; a row without a vote, whose scores may not be
                // numbers, sees none
                lim[tid] = mine < INFINITY ? L - qfull + ((vt.first + v) * kRows + tid) / G : -1;
                if (isnan(mine)) misc[1] = v + 1;
                ok = bar_wait(barQ, loads++ & 1u);
            }
            async_proxy_fence();
            tc_before_sync();
            if (!__syncthreads_and(ok)) {
                ok = false;
                break;
            }
            tc_after_sync();
            if (warp == 0) {
                constexpr uint32_t id = idesc_f16(kRows, kRows, 0);
                const uint64_t dk = mdesc(sK, 128, 16 * D), dq = mdesc(sQ, 128, 32 * D);
                const uint32_t el = elect_one(), tm = __shfl_sync(kFull, tmem, 0);
#pragma unroll
                for (int ks = 0; ks < 2 * D / 16; ks++)
                    mma_ss(el, tm, dk + 16 * (ks % (D / 16)), dq + 16 * (ks ^ (D / 16)), id, ks > 0);
                commit(el, barS);
            }
            ok = bar_wait(barS, products++ & 1u);
            if (!__syncthreads_and(ok)) {
                ok = false;
                break;
            }
            tc_after_sync();
            if (votes > 1 && (v + 1 < votes || !last)) {  // the scores have read this tile's queries
                const int next = v + 1 < votes ? v + 1 : 0;
                load(next);
                mine = lse_of(next);
            }
            const int lo = vt.lo(vt.first + v), hi = vt.hi(vt.first + v);
            // this token's weights: 2^(norm * score - lse); no limits where all sixteen rows vote
            // and the first row sees the whole token tile
            const bool whole = tile * kRows + kRows - 1 <= L - qfull + ((vt.first + v) * kRows + lo) / G &&
                               (int)misc[1] != v + 1;
            const float2 n2 = make_float2(norm, norm);
            float2 part = make_float2(0.f, 0.f);
            float x[2][16];
            tmem_ld16_start(tmem + lane_off, x[0]);
#pragma unroll
            for (int c = 0; c < kRows / 16; c++) {
                tmem_ld_wait(x[c & 1]);
                if (c + 1 < kRows / 16) tmem_ld16_start(tmem + lane_off + 16u * (c + 1), x[(c + 1) & 1]);
                if (16 * c >= hi || 16 * c + 16 <= lo) continue;
                const bool mask = !whole || 16 * c < lo || 16 * c + 16 > hi;
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float* xc = x[c & 1] + j;
                    const float2 l2 = *reinterpret_cast<const float2*>(lse + 16 * c + j);
                    float2 y = __ffma2_rn(make_float2(xc[0], xc[1]), n2, make_float2(-l2.x, -l2.y));
                    if (mask) {
                        y.x = t <= lim[16 * c + j] ? y.x : -INFINITY;
                        y.y = t <= lim[16 * c + j + 1] ? y.y : -INFINITY;
                    }
                    part = __fadd2_rn(part, make_float2(exp2a(y.x), exp2a(y.y)));
                }
            }
            sum += part.x + part.y;
            tc_before_sync();
            __syncthreads();
            tc_after_sync();
        }
        if (here && ok) sums[t] = old + sum;
    }
    if (!ok && tid == 0) flag_status(a.status, TQ_STATUS_TIMEOUT);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(128u) : "memory");
}

// Raise a kernel's dynamic shared memory limit, once per device.
struct SmemLimit {
    std::mutex mu;
    bool configured[64] = {};
    cudaError_t raise(const void* kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        std::lock_guard<std::mutex> lk(mu);
        if (dev < 0 || dev >= 64 || !configured[dev]) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (e == cudaSuccess && dev >= 0 && dev < 64) configured[dev] = true;
        }
        return e;
    }
};

template <int D, bool CUT>
cudaError_t launch_rows(const WArgs& a, cudaStream_t stream) {
    static SmemLimit limit;
    cudaError_t e = limit.raise((const void*)prefill_rows_kernel<D, CUT>, (int)APlan<D>::kEnd);
    if (e != cudaSuccess) return e;
    static const bool regs_ok = [] {  // the register split draws on the launch's registers
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, prefill_rows_kernel<D, CUT>) == cudaSuccess && at.numRegs >= kLaunchRegs;
    }();
    if (!regs_ok) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)(a.pairs * a.parts), (unsigned)a.Hkv, (unsigned)a.B);
    prefill_rows_kernel<D, CUT><<<grid, kThreads, APlan<D>::kEnd, stream>>>(a);
    return cudaGetLastError();  // the votes add to the caller's sums: not without this kernel
}

template <int D>
cudaError_t launch_w(const WArgs& a, cudaStream_t stream) {
    static SmemLimit votes_limit;
    cudaError_t e = a.parts > 1 ? launch_rows<D, true>(a, stream) : launch_rows<D, false>(a, stream);
    if (e != cudaSuccess) return e;
    e = votes_limit.raise((const void*)votes_kernel<D>, (int)VPlan<D>::kEnd);
    if (e != cudaSuccess) return e;
    const long long tokens = std::min(a.w_stride, (long long)a.max_blocks * kBlock);
    WArgs v = a;
    // One or two voting tiles: the CTAs that the SMs' shared memory holds at once, each with
    // its set-up and queries once (128 rows on 32768 tokens x 8: 48 -> 35 us).  More of
    // them outweigh the set-up, and a CTA per token tile levels out ragged lengths (5 tiles,
    // 16 sequences x 2: 38 us, the other way 46 us).
    const long long tiles = (tokens + kRows - 1) / kRows;
    const long long ctas = a.wtiles <= 2 ? std::max(1LL, VPlan<D>::kCtas * kSMs / ((long long)a.Hkv * a.B)) : tiles;
    const long long each = (tiles + ctas - 1) / ctas;
    v.vblocks = (int)((tiles + each - 1) / each);
    const int joins = a.parts > 1 ? a.pairs * 2 * (D / 16) : 0;
    const dim3 vgrid((unsigned)std::max(v.vblocks, joins), (unsigned)a.Hkv, (unsigned)(joins ? 2 * a.B : a.B));
    votes_kernel<D><<<vgrid, kRows, VPlan<D>::kEnd, stream>>>(v);
    return cudaGetLastError();
}

}  // namespace

// The voting rows are at most window * G consecutive ones and start anywhere in a tile.
static int prefill_vote_tiles(int max_q_len, int window, int G) {
    const long long rows = (long long)(window > 0 ? std::min(window, max_q_len) : max_q_len) * G;
    return (int)((rows + kRows - 1) / kRows) + (window > 0 && window < max_q_len ? 1 : 0);
}

// Parts of every context: as many as fill the SMs once.  A chunk of few rows has few CTAs (5
// tokens, 32 query / 8 kv heads: eight), whose whole contexts would leave most SMs idle: 900 us
// a call at context 32768 against 98 in 18 parts; 64 tokens x 8 sequences at 8192: 436 us, in
// two parts 322.  Smaller parts in more waves do not pay: a part costs about 10 us by itself,
// and its sums go through memory (the first chunk in 32 parts 115 us, the second in four 331).
namespace {
int row_pairs(int max_q_len, int G) { return (int)(((long long)max_q_len * G + 2 * kRows - 1) / (2 * kRows)); }
int context_parts(int B, int Hkv, int max_q_len, int G) {
    return (int)std::max(1LL, std::min((long long)kMaxParts, kSMs / ((long long)B * Hkv * row_pairs(max_q_len, G))));
}
}  // namespace

// Queries and statistics of the voting tiles, then statistics and sums of the parts.
size_t prefill_weights_bytes(int B, int Hkv, int G, int max_q_len, int window, int head_dim) {
    const size_t tiles = (size_t)B * Hkv * prefill_vote_tiles(max_q_len, window, G);
    const int parts = context_parts(B, Hkv, max_q_len, G);
    const size_t rows = parts > 1 ? (size_t)B * Hkv * row_pairs(max_q_len, G) * parts * (2 * kRows) : 0;
    return tiles * (512 * (size_t)head_dim + kRows * sizeof(float)) +
           rows * (sizeof(float2) + head_dim * sizeof(float));
}

cudaError_t launch_prefill_weights(WArgs& a, void* workspace, int head_dim, cudaStream_t stream) {
    const int G = a.Hq / a.Hkv;
    a.wtiles = prefill_vote_tiles(a.max_q_len, a.window, G);
    a.pairs = row_pairs(a.max_q_len, G);
    a.parts = context_parts(a.B, a.Hkv, a.max_q_len, G);
    const size_t tiles = (size_t)a.B * a.Hkv * a.wtiles;
    a.q_img = static_cast<unsigned char*>(workspace);
    a.lse = reinterpret_cast<float*>(a.q_img + tiles * 512 * head_dim);
    a.part_stat = reinterpret_cast<float2*>(a.lse + tiles * kRows);
    a.part_o = reinterpret_cast<float4*>(a.part_stat + (size_t)a.B * a.Hkv * a.pairs * a.parts * (2 * kRows));
    return head_dim == 128 ? launch_w<128>(a, stream) : launch_w<64>(a, stream);
}

}  // namespace tq
