// tq_weights.cu -- attention weights accumulated per cached token: what a cache that
// evicts by accumulated attention keeps beside its records.
//
// Decode.  A token's weight is p_h,t = 2^(s_h,t - M_h) / l_h with the row's final
// reference M and sum l, which no split knows while it runs.  The split kernels therefore
// keep their base-2 scores s (fp32; 4 bytes per query head and token, at d = 128 and
// four heads per kv head 16 bytes beside the 146 bytes of the record they came from),
// and one kernel after them does the rest: its first CTAs merge the rows that ranges cut
// (as the combine of the plain decode), the others form
//   w[b][kv][t] += sum over the kv head's query heads of p_h,t.
// Scoring the keys again instead would read 66 of the 146 bytes a second time.
//
// Bound by the scores' way through L2 and HBM (33.5 MB out and in, 16.8 MB of sums for 32 x
// 8192 tokens and 8 heads of 4): 13 us of a 105 us call.
#include <algorithm>

#include "tq_kernels.cuh"

namespace tq {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 4;                  // consecutive tokens per thread
constexpr int kTile = kThreads * kPer;   // tokens of a tile
constexpr int kMaxGroup = 64;            // query heads per kv head
constexpr int kBatch = 4;                // heads whose scores are in flight together

__device__ __forceinline__ float ex2(float x) {  // 2^x; -inf gives 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What the launcher works out once.
struct Shape {
    int G;       // query heads per kv head
    Div32 by_R;  // division by the plan's records per range
    int merges;  // CTAs that merge rows
    int chunks;  // CTAs of a (sequence, kv head)
    int turns;   // token tiles of a CTA
};

// The partial results of a query head of sequence b: ranges [first, last], part r's slot.
struct Parts {
    int first, last;  // first == last: not cut, the row is finished
    int item, h, hpi; // TQ4/4 plan
    // head g of kv head kv
    __device__ __forceinline__ Parts(const DecodeArgs& a, const Shape& d, int b, int kv, int g) {
        if (a.bf16) {
            first = 0;
            last = a.bf_splits - 1;
            item = b * a.Hq + kv * d.G + g;
            return;
        }
        hpi = 4 * a.qpi;  // 4 or 8
        const int quad = g >> (a.qpi + 1);
        h = g & (hpi - 1);
        item = (b * a.Hkv + kv) * a.quads + quad;
        first = (int)fast_div32((uint32_t)(item * a.nmax), d.by_R);  // both below 2^30
        last = (int)fast_div32((uint32_t)(item * a.nmax + a.nmax - 1), d.by_R);
    }
    __device__ __forceinline__ size_t slot(const DecodeArgs& a, int r) const {
        if (a.bf16) return (size_t)item * a.bf_splits + r;
        // the range's first item is in slot 0, its last in slot 1: the item is the first one
        // of a range that starts inside it
        return ((size_t)r * 2 + (r * a.R >= item * a.nmax ? 0 : 1)) * hpi + h;
    }
};

// (M, 1 / l) of a row, by a warp (a row without tokens: 1 / l = 0).
__device__ __forceinline__ float2 row_stats(const DecodeArgs& a, const Parts& p, size_t row, int lane) {
    float M = -INFINITY, l = 0.f;
    if (p.first == p.last) {
        const float2 v = a.fin_ml[row];
        M = v.x;
        l = v.y;
    } else {
        // (a part whose sum is not a number takes the row with it, even one without a maximum)
        auto join = [&](float m2, float l2) {
            const float Mn = fmaxf(M, m2);
            const float f = M == -INFINITY ? 0.f : ex2(M - Mn), f2 = m2 == -INFINITY ? 0.f : ex2(m2 - Mn);
            l = fmaf(f2, l2, f * l);
            M = Mn;
        };
        for (int r = p.first + lane; r <= p.last; r += 32) {
            const float2 v = a.ws_ml[p.slot(a, r)];
            join(v.x, v.y);
        }
#pragma unroll
        for (int m = 16; m; m >>= 1) {
            const float Mo = __shfl_xor_sync(kFull, M, m), lo = __shfl_xor_sync(kFull, l, m);
            join(Mo, lo);
        }
    }
    return l > 0.f ? make_float2(M, 1.f / l) : make_float2(0.f, 0.f);
}

template <int D>
__global__ void __launch_bounds__(kThreads) decode_weights_kernel(DecodeArgs a, float* tw, long long stride,
                                                                  Shape d) {
    __shared__ float2 ml[kMaxGroup];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = d.G;
    if ((int)blockIdx.x < d.merges) {  // a warp merges the parts of one row
        const int row = blockIdx.x * kWarps + warp;
        if (row >= a.B * a.Hq) return;
        const int b = row / a.Hq, hh = row % a.Hq;
        const Parts p(a, d, b, hh / G, hh % G);
        if (p.first == p.last) return;
        const float2 st = row_stats(a, p, row, lane);
        constexpr int DPL = D / 32;
        float o[DPL];
#pragma unroll
        for (int j = 0; j < DPL; j++) o[j] = 0.f;
#pragma unroll 4
        for (int r = p.first; r <= p.last; r++) {
            const size_t at = p.slot(a, r);
            const float m = a.ws_ml[at].x;
            const float f = m == -INFINITY ? 0.f : ex2(m - st.x);
#pragma unroll
            for (int j = 0; j < DPL; j++) {
                const float v = a.ws_o[at * D + j * 32 + lane];
                o[j] = fmaf(f, v, o[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < DPL; j++) a.out[(size_t)row * D + j * 32 + lane] = o[j] * st.y;
        return;
    }
    const int bx = (int)blockIdx.x - d.merges;
    const int chunk = bx % d.chunks, bk = bx / d.chunks;
    const int kv = bk % a.Hkv, b = bk / a.Hkv;
    int L = a.seq_lens[b];
    if (L < 0 || L > a.max_blocks * kBlock) L = 0;  // flagged by the decode
    L = min(L, a.max_seq_len);
    const int t0 = chunk * d.turns * kTile;
    if (t0 >= L) return;
    // score rows are whole blocks: the four scores are there, those of tokens past L unused.
    // The first heads' scores and the running sums are on their way while the statistics
    // are merged, and a tile's while the one before is summed.
    const float* s = a.scores + (size_t)(b * a.Hq + kv * G) * a.score_stride;
    float* w = tw + (size_t)bk * stride;
    float4 x[kBatch];
    float old[kPer];
    auto load = [&](int t) {
        if (t >= L) return;
#pragma unroll
        for (int h = 0; h < kBatch; h++)
            if (h < G) x[h] = __ldcs(reinterpret_cast<const float4*>(s + h * a.score_stride + t));
#pragma unroll
        for (int j = 0; j < kPer; j++) old[j] = t + j < L ? w[t + j] : 0.f;
    };
    int t = t0 + kPer * threadIdx.x;
    load(t);
    for (int h = warp; h < G; h += kWarps) {
        const float2 st = row_stats(a, Parts(a, d, b, kv, h), (size_t)b * a.Hq + kv * G + h, lane);
        if (lane == 0) ml[h] = st;
    }
    __syncthreads();
#pragma unroll 1
    for (int turn = 0; turn < d.turns && t < L; turn++, t += kTile) {
        // the heads are summed apart from the running sum, which so is rounded once a call
        float acc[kPer] = {};
#pragma unroll 1
        for (int h0 = 0; h0 < G; h0 += kBatch) {
#pragma unroll
            for (int h = 0; h < kBatch; h++) {
                if (h0 + h >= G) break;
                const float2 v = ml[h0 + h];
                if (v.y == 0.f) continue;  // a row without a sum (no token, or not a number) gives nothing
                acc[0] = fmaf(ex2(x[h].x - v.x), v.y, acc[0]);
                acc[1] = fmaf(ex2(x[h].y - v.x), v.y, acc[1]);
                acc[2] = fmaf(ex2(x[h].z - v.x), v.y, acc[2]);
                acc[3] = fmaf(ex2(x[h].w - v.x), v.y, acc[3]);
            }
#pragma unroll
            for (int h = 0; h < kBatch; h++)
                if (h0 + kBatch + h < G)
                    x[h] = __ldcs(reinterpret_cast<const float4*>(s + (h0 + kBatch + h) * a.score_stride + t));
        }
        float sum[kPer];
#pragma unroll
        for (int j = 0; j < kPer; j++) sum[j] = old[j] + acc[j];
        if (turn + 1 < d.turns) load(t + kTile);
#pragma unroll
        for (int j = 0; j < kPer; j++)
            if (t + j < L) w[t + j] = sum[j];
    }
}

}  // namespace

cudaError_t launch_decode_weights(const DecodeArgs& a, int head_dim, int num_sms, float* token_weights,
                                  long long stride, cudaStream_t stream) {
    Shape d;
    d.G = a.Hq / a.Hkv;
    d.by_R = div32_magic((uint32_t)(a.bf16 ? 1 : a.R));
    const bool cut = a.bf16 ? a.bf_splits > 1 : decode_needs_combine(a);
    d.merges = cut ? (a.B * a.Hq + kWarps - 1) / kWarps : 0;
    // a CTA merges its heads' statistics once, for up to eight tiles of tokens, as long as
    // four CTAs an SM remain (32 x 8192 tokens, 8 heads: 105 us for the call, 107 us with
    // sixteen; of lengths from 410 to 4095: 63 us, 67 us with two)
    const int tiles = (a.max_seq_len + kTile - 1) / kTile;
    const long long rows = (long long)a.B * a.Hkv;
    d.turns = (int)std::min(8LL, std::max(1LL, rows * tiles / (4LL * num_sms)));
    d.chunks = std::max(1, (tiles + d.turns - 1) / d.turns);
    const long long grid = (tiles ? rows * d.chunks : 0) + d.merges;  // < 2^31: the scores fit in memory
    if (grid == 0) return cudaSuccess;
    if (head_dim == 128)
        decode_weights_kernel<128><<<(unsigned)grid, kThreads, 0, stream>>>(a, token_weights, stride, d);
    else
        decode_weights_kernel<64><<<(unsigned)grid, kThreads, 0, stream>>>(a, token_weights, stride, d);
    return cudaGetLastError();
}

}  // namespace tq
