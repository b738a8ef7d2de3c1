// tq_evict.cu -- eviction from the cache by accumulated attention weight: the choice of
// the tokens each kv head keeps, and the move of their records to the front.
//
// Selection.  Per (sequence, kv head) the first `sink` and the last `recent` tokens stay
// and the budget's other K places go to the largest sums among the rest, equal sums to the
// lowest position.  A row is taken by a cluster of CTAs that hold it in shared memory as
// 32-bit keys whose unsigned order is the order of the sums, so HBM sees the row once.
// The K-th largest key is found by radix (11 + 11 + 10 bits): each pass counts the keys
// that share the prefix found so far, the CTAs of the cluster add their counts to the
// first one's through distributed shared memory, and it hands the digit to all.  One more
// pass judges the keys, and the kept positions leave in order.  The row is read once
// (8.4 MB of sums: 1.3 us of HBM); what bounds the call is the chain of short phases, each
// a barrier and a few shared-memory latencies: calls in a row take 16 us for 256 rows of 8192,
// 27 us for 32 rows of 131072, and 12 us (launch and Python) where that is longer.
//
// Compaction.  Kept token j of a (sequence, kv head) moves from slot kept[j] to slot j.
// One warp builds one destination record (16 tokens): it gathers the 16 source tokens'
// fields into registers in the destination's placement and stores whole 16-byte runs.  A
// slot with no token to receive takes its own old bytes, so nothing behind the last kept
// token changes.  In place, kept[j] >= j orders the moves: the CTAs of a cluster load one
// wave of consecutive records, meet at a barrier and store it; a later wave's sources lie
// behind every slot that was stored.
// Bound by HBM in whole sectors: a token's 146 bytes lie in nine 32-byte sectors (its value
// codes alternate with its neighbour's), so a quarter of 32 x 8192 tokens in 8 heads costs
// 266 MB of traffic for 154 MB of tokens: 50 us at 5.3 TB/s.
#include <cooperative_groups.h>

#include <mutex>

#include "tq_kernels.cuh"

namespace tq {
namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------ selection
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kDigits = 3;
constexpr int kHist = 2048;          // bins of the widest digit
constexpr int kSelHold = 40960;      // keys a CTA holds in shared memory (160 KB)
constexpr int kSelSmem = kDigits * kHist * (int)sizeof(uint32_t);  // beside the keys

// Unsigned key in the order of the sums: NaN below everything, -0 equal to +0.
__device__ __forceinline__ uint32_t sum_key(float x) {
    const int u = __float_as_int(x + 0.0f);
    return x == x ? (uint32_t)(u ^ ((u >> 31) | (int)0x80000000)) : 0u;
}

struct SelectArgs {
    const float* w;
    long long stride;
    const int32_t* seq_lens;
    int B, Hkv, max_seq_len, budget, sink, recent;
    int32_t* kept;
    int32_t* kept_lens;
    int32_t* status;
    int hold;  // keys of a CTA's part that fit in its shared memory
};

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(kFull, v, m);
        if (lane >= m) v += o;
    }
    return v;
}
// Sum of v over the threads before this one; `part` holds one value per warp.  `part` may be
// written again after a further barrier.
__device__ __forceinline__ int block_before(int v, int* part, int lane, int warp) {
    const int incl = warp_scan(v, lane);
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    const int p = lane < kSelWarps ? part[lane] : 0;
    const int upto = warp_scan(p, lane);
    return incl - v + __shfl_sync(kFull, upto - p, warp);
}
// Where key i of a CTA's part lies: runs of four keys, the eight runs of a 32-key stretch
// exchanged so that both orders of reading them, runs in a row over the lanes and 32 keys
// in a row per lane, hit all the banks.
__device__ __forceinline__ int key_run(int r) { return r ^ ((r >> 3) & 7); }

__global__ void __launch_bounds__(kSelThreads) select_kernel(SelectArgs a) {
    extern __shared__ __align__(16) uint32_t keys[];  // [hold], then the digits' counts
    __shared__ int s_part[kSelWarps], s_tie[kSelWarps];
    __shared__ int2 s_found;  // (digit, keys above it)
    __shared__ int2 s_total;  // this CTA's (sure, tied) tokens
    uint32_t* hist = keys + a.hold;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int row = (int)blockIdx.x / C, b = row / a.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int L = a.seq_lens[b];
    if (L < 0 || L > a.max_seq_len) {
        if (tid == 0 && rank == 0 && row % a.Hkv == 0) flag_status(a.status, TQ_STATUS_BAD_LEN);
        L = 0;
    }
    const int n = min(L, a.budget);
    int32_t* kept = a.kept + (size_t)row * a.budget;
    if (tid == 0 && rank == 0 && row % a.Hkv == 0) a.kept_lens[b] = n;
    for (int j = n + rank * kSelThreads + tid; j < a.budget; j += C * kSelThreads) kept[j] = -1;
    if (L <= a.budget) {  // everything stays (the whole cluster leaves together)
        for (int j = rank * kSelThreads + tid; j < n; j += C * kSelThreads) kept[j] = j;
        return;
    }
    const int lo = a.sink, hi = L - a.recent;  // the tokens that compete
    int K = a.budget - a.sink - a.recent;      // for this many places, K < hi - lo
    // this CTA's contiguous part of the row, its first `hold` keys in shared memory
    const int per = (L + C - 1) / C;
    const int t0 = min(rank * per, L), cnt = min(per, L - t0);
    const int held = min(cnt, a.hold);
    const float* w = a.w + (size_t)row * a.stride + t0;
    for (int i = tid; i < kDigits * kHist / 4; i += kSelThreads)
        reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
    // four sums at a time, as 16 bytes where the row's alignment allows
    if ((reinterpret_cast<uintptr_t>(w) & 15) == 0) {
#pragma unroll 8
        for (int i = 4 * tid; i + 3 < held; i += 4 * kSelThreads) {
            const float4 x = *reinterpret_cast<const float4*>(w + i);
            *reinterpret_cast<uint4*>(keys + 4 * key_run(i >> 2)) =
                make_uint4(sum_key(x.x), sum_key(x.y), sum_key(x.z), sum_key(x.w));
        }
    } else {
#pragma unroll 4
        for (int i = 4 * tid; i + 3 < held; i += 4 * kSelThreads)
            *reinterpret_cast<uint4*>(keys + 4 * key_run(i >> 2)) =
                make_uint4(sum_key(w[i]), sum_key(w[i + 1]), sum_key(w[i + 2]), sum_key(w[i + 3]));
    }
    if (const int i = (held & ~3) + tid; i < held) keys[4 * key_run(i >> 2) + (i & 3)] = sum_key(w[i]);
    // keys i .. i + 3 of this CTA's part (i a multiple of 4); those past its end are 0
    auto key4 = [&](int i, uint32_t (&k)[4]) {
        if (i + 3 < held) {
            const uint4 v = *reinterpret_cast<const uint4*>(keys + 4 * key_run(i >> 2));
            k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++)
                k[e] = i + e >= cnt ? 0u : i + e < held ? keys[4 * key_run(i >> 2) + e] : sum_key(w[i + e]);
        }
    };
    const int c0 = lo - t0, c1 = min(hi - t0, cnt);  // the competitors of this part
    if (C > 1)
        cluster.sync();  // every CTA's counts are zero (and its keys there)
    else
        __syncthreads();

    uint32_t prefix = 0;  // the digits found so far
    int shift = 32;
#pragma unroll 1
    for (int p = 0; p < kDigits && K > 0; p++) {
        const int bits = p < 2 ? 11 : 10, bins = 1 << bits;
        const int up = shift;
        shift -= bits;
        uint32_t* h = hist + p * kHist;
        const uint32_t h_at = (uint32_t)__cvta_generic_to_shared(h);
        // key k counts if its digits so far are the prefix (`any`: always) and `in` holds
        auto count = [&](uint32_t k, bool any, bool in) {
            const uint32_t at = h_at + 4 * ((k >> shift) & (bins - 1));
            const uint32_t yes = in && (any || (k >> up) == prefix);
            asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %0, 0;\n @p red.shared.add.u32 [%1], 1;\n}\n" ::"r"(yes),
                         "r"(at)
                         : "memory");
        };
        // the competitors of this part that fill runs of four held keys, then the others
        const int f0 = (max(c0, 0) + 3) & ~3, f1 = max(f0, min(c1, held) & ~3);
        if (p == 0) {
#pragma unroll 4
            for (int i = f0 + 4 * tid; i < f1; i += 4 * kSelThreads) {
                const uint4 k = *reinterpret_cast<const uint4*>(keys + 4 * key_run(i >> 2));
                count(k.x, true, true), count(k.y, true, true), count(k.z, true, true), count(k.w, true, true);
            }
        } else {
#pragma unroll 4
            for (int i = f0 + 4 * tid; i < f1; i += 4 * kSelThreads) {
                const uint4 k = *reinterpret_cast<const uint4*>(keys + 4 * key_run(i >> 2));
                count(k.x, false, true), count(k.y, false, true), count(k.z, false, true), count(k.w, false, true);
            }
        }
        if (tid < f0 - max(c0, 0) && max(c0, 0) + tid < c1) {
            uint32_t k[4];
            key4((max(c0, 0) + tid) & ~3, k);
            const int e = (max(c0, 0) + tid) & 3;
            count(e == 0 ? k[0] : e == 1 ? k[1] : e == 2 ? k[2] : k[3], p == 0, true);
        }
        for (int i = f1 + 4 * tid; i < c1; i += 4 * kSelThreads) {
            uint32_t k[4];
            key4(i, k);
#pragma unroll
            for (int e = 0; e < 4; e++) count(k[e], p == 0, i + e < c1);
        }
        __syncthreads();
        // a thread takes four consecutive bins, thread 0 the highest ones; the other CTAs
        // add theirs to the first one's, which finds the digit for all: the bin where the
        // count from the top passes K
        const int bin0 = bins - 4 - 4 * tid;
        if (C > 1) {
            if (rank > 0 && bin0 >= 0) {
                const uint4 v = *reinterpret_cast<const uint4*>(h + bin0);
                uint32_t* far = cluster.map_shared_rank(h, 0) + bin0;
                if (v.x) atomicAdd(far, v.x);
                if (v.y) atomicAdd(far + 1, v.y);
                if (v.z) atomicAdd(far + 2, v.z);
                if (v.w) atomicAdd(far + 3, v.w);
            }
            cluster.sync();
        }
        if (rank == 0) {
            const uint4 c = bin0 >= 0 ? *reinterpret_cast<const uint4*>(h + bin0) : make_uint4(0, 0, 0, 0);
            const int e[4] = {(int)c.w, (int)c.z, (int)c.y, (int)c.x};
            const int mine = e[0] + e[1] + e[2] + e[3];
            int above = block_before(mine, s_part, lane, warp);  // keys in higher bins than this thread's
            if (above < K && above + mine >= K) {
                int2 found = make_int2(-1, 0);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (found.x < 0 && above + e[i] >= K) found = make_int2(bin0 + 3 - i, above);
                    above += e[i];
                }
                for (int r = 0; r < C; r++) *cluster.map_shared_rank(&s_found, r) = found;
            }
        }
        if (C > 1)
            cluster.sync();
        else
            __syncthreads();
        prefix = (prefix << bits) | (uint32_t)s_found.x;
        K -= s_found.y;
    }
    // keys above `prefix` are kept, and the K lowest positions among the equal ones; a lane
    // judges up to 32 keys in a row and keeps the verdicts as bits
    const uint32_t T = K > 0 ? prefix : 0xffffffffu;
    int up_before = 0, eq_before = 0;  // kept and tied tokens of the parts before this one
    const int lk = min(((cnt + kSelThreads - 1) / kSelThreads + 3) & ~3, 32);  // keys of a lane
    const int tile = lk * kSelThreads;
    auto judge = [&](int i0, uint32_t& mu, uint32_t& mq) {
        mu = mq = 0;
#pragma unroll
        for (int s = 0; s < 8; s++) {
            const int i = i0 + 4 * s;
            if (i >= cnt || 4 * s >= lk) break;
            uint32_t k[4];
            key4(i, k);
            uint32_t u = 0, q = 0;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                u |= (k[e] > T ? 1u : 0u) << e;
                q |= (k[e] == T ? 1u : 0u) << e;
            }
            if (i < c0 || i + 3 >= c1) {  // the first and the last tokens stay
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (i + e >= cnt) {
                        u &= ~(1u << e);
                        q &= ~(1u << e);
                    } else if (i + e < c0 || i + e >= c1) {
                        u |= 1u << e;
                        q &= ~(1u << e);
                    }
            }
            mu |= u << (4 * s);
            mq |= q << (4 * s);
        }
        if (K == 0) mq = 0;
    };
    uint32_t mu, mq;
    judge(lk * tid, mu, mq);
    if (C > 1) {
        int sure = __popc(mu), tied = __popc(mq);
        for (int i0 = tile; i0 < cnt; i0 += tile) {
            uint32_t u, q;
            judge(i0 + lk * tid, u, q);
            sure += __popc(u);
            tied += __popc(q);
        }
        if (tid == 0) s_total = make_int2(0, 0);
        __syncthreads();
        sure = __reduce_add_sync(kFull, sure);
        tied = __reduce_add_sync(kFull, tied);
        if (lane == 0) {
            atomicAdd(&s_total.x, sure);
            atomicAdd(&s_total.y, tied);
        }
        cluster.sync();
        int2 v[8];
#pragma unroll
        for (int r = 0; r < 8; r++)
            if (r < rank) v[r] = *cluster.map_shared_rank(&s_total, r);
#pragma unroll
        for (int r = 0; r < 8; r++)
            if (r < rank) up_before += v[r].x, eq_before += v[r].y;
    }
#pragma unroll 1
    for (int i0 = 0; i0 < cnt; i0 += tile) {
        if (i0 > 0) judge(i0 + lk * tid, mu, mq);
        const int su = warp_scan(__popc(mu), lane), sq = warp_scan(__popc(mq), lane);
        if (lane == 31) {
            s_part[warp] = su;
            s_tie[warp] = sq;
        }
        __syncthreads();  // (the keys of this tile have been read)
        const int pu = lane < kSelWarps ? s_part[lane] : 0, pq = lane < kSelWarps ? s_tie[lane] : 0;
        const int au = warp_scan(pu, lane), aq = warp_scan(pq, lane);
        int nu = up_before + __shfl_sync(kFull, au - pu, warp) + su - __popc(mu);
        int nq = eq_before + __shfl_sync(kFull, aq - pq, warp) + sq - __popc(mq);
        // of the equal ones before a token, min(., K) were taken.  A tile's kept positions
        // go through the tile's own key space, so that they leave in whole sectors
        const int first = up_before + min(eq_before, K);
        up_before += __shfl_sync(kFull, au, 31);
        eq_before += __shfl_sync(kFull, aq, 31);
        const int last = up_before + min(eq_before, K);
        const bool staged = i0 + tile <= held || cnt <= held;
        uint32_t* stage = keys + i0 - first;
        for (uint32_t m = mu | mq; m; m &= m - 1) {
            const int e = __ffs(m) - 1;
            const bool sure = mu >> e & 1;
            if (sure || nq < K) {
                const int at = nu + min(nq, K);
                if (staged)
                    stage[at] = (uint32_t)(t0 + i0 + lk * tid + e);
                else
                    kept[at] = t0 + i0 + lk * tid + e;
            }
            nu += sure;
            nq += !sure;
        }
        __syncthreads();
        if (staged)
            for (int at = first + tid; at < last; at += kSelThreads) kept[at] = (int)stage[at];
    }
    if (C > 1) cluster.sync();  // no CTA leaves while another still reads its shared memory
}

// ------------------------------------------------------------------ compaction
constexpr int kMoveWarps = 8;

struct MoveArgs {
    unsigned char* cache;
    int num_blocks, Hkv, B;
    const int32_t* src_tables;
    int src_max;
    const int32_t* seq_lens;
    const int32_t* kept;       // [B][Hkv][budget]
    const int32_t* kept_lens;  // [B]
    int budget;
    const int32_t* dst_tables;  // the source's tables when in place
    int dst_max;
    const float* w;  // null: no sums to move
    float* w_out;
    long long w_stride, out_stride;
    int32_t* status;
    int ctas;  // CTAs per (sequence, kv head)
};

// The 16 source tokens of a destination record: lane l < 16 knows slot l's.
struct Sources {
    int blk, off;  // physical block and slot of this lane's token
    __device__ __forceinline__ const unsigned char* rec(const MoveArgs& a, int slot, int kv, uint32_t bytes,
                                                        int& o) const {
        const int p = __shfl_sync(kFull, blk, slot);
        o = __shfl_sync(kFull, off, slot);
        return a.cache + ((size_t)p * a.Hkv + kv) * bytes;
    }
};

// A TQ4/4 record's fields in registers.  Lane l holds, in the destination's placement:
// key codes, 16-byte runs l, l + 32; value chunks (one token pair's one r) l, l + 32; norm
// of token l; one 8-byte unit of scales (low lanes) or zero points.
template <int D>
struct TqMove {
    using R = Rec<D>;
    static constexpr uint32_t kBytes = R::kBytes;
    static constexpr int kKeyRuns = 16 * (D / 2) / 16 / 32;  // 16-byte runs per lane
    static constexpr int kRunsPerTok = D / 32;
    static constexpr int kWords = D / 32;  // words of a value chunk (D / 8 bytes)
    static constexpr int kUnits = 4 * R::kGroups;
    uint4 k[kKeyRuns];
    uint32_t v[2][kWords];
    uint16_t norm;
    uint2 sz;

    __device__ __forceinline__ void load(const MoveArgs& a, const Sources& s, int kv, int lane) {
        int o;
#pragma unroll
        for (int i = 0; i < kKeyRuns; i++) {
            const int run = lane + 32 * i;
            const unsigned char* p = s.rec(a, run / kRunsPerTok, kv, kBytes, o);
            k[i] = *reinterpret_cast<const uint4*>(p + o * R::kCodeRow + (run % kRunsPerTok) * 16);
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int pair = (lane + 32 * i) / 8, r = lane % 8;
            int oa, ob;
            const unsigned char* pa = s.rec(a, 2 * pair, kv, kBytes, oa);
            const unsigned char* pb = s.rec(a, 2 * pair + 1, kv, kBytes, ob);
            uint32_t wa[kWords], wb[kWords];
            chunk(pa, oa, r, wa);
            chunk(pb, ob, r, wb);
            // the low half of a word is the even token's bytes, the high half the odd one's
            const uint32_t sel = (oa & 1 ? 0x32u : 0x10u) | (ob & 1 ? 0x7600u : 0x5400u);
#pragma unroll
            for (int e = 0; e < kWords; e++) v[i][e] = __byte_perm(wa[e], wb[e], sel);
        }
        {
            const unsigned char* p = s.rec(a, lane & 15, kv, kBytes, o);
            norm = *reinterpret_cast<const uint16_t*>(p + R::kKNorm + 2 * o);
        }
        uint16_t h[4];
        const int unit = lane % kUnits, c = unit / R::kGroups, g = unit % R::kGroups;
        const int area = lane < kUnits ? R::kVScale : R::kVZero;
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const unsigned char* p = s.rec(a, 2 * c + (u & 1) + 8 * (u >> 1), kv, kBytes, o);
            h[u] = *reinterpret_cast<const uint16_t*>(p + area + R::group_pos(o, g));
        }
        sz = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
    }
    static __device__ __forceinline__ void chunk(const unsigned char* rec, int o, int r, uint32_t (&w)[kWords]) {
        const int p = o >> 1;
        const unsigned char* at = rec + R::kVCodes + (8 * p + ((r + 2 * p) & 7)) * R::kPairChunk;
        if constexpr (kWords == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(at);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(at);
            w[0] = x.x, w[1] = x.y;
        }
    }
    __device__ __forceinline__ void store(unsigned char* rec, int lane) const {
#pragma unroll
        for (int i = 0; i < kKeyRuns; i++) *reinterpret_cast<uint4*>(rec + (lane + 32 * i) * 16) = k[i];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int p = (lane + 32 * i) / 8, r = lane % 8;
            unsigned char* at = rec + R::kVCodes + (8 * p + ((r + 2 * p) & 7)) * R::kPairChunk;
            if constexpr (kWords == 4)
                *reinterpret_cast<uint4*>(at) = make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
            else
                *reinterpret_cast<uint2*>(at) = make_uint2(v[i][0], v[i][1]);
        }
        if (lane < 16) *reinterpret_cast<uint16_t*>(rec + R::kKNorm + 2 * lane) = norm;
        if (lane < 2 * kUnits)
            *reinterpret_cast<uint2*>(rec + (lane < kUnits ? R::kVScale : R::kVZero) + 8 * (lane % kUnits)) = sz;
    }
};

// A bf16 record: 32 rows of 2 D bytes, 16-byte chunk j of row r at j ^ (r mod 8).
template <int D>
struct BfMove {
    static constexpr uint32_t kBytes = 64 * D;
    static constexpr int kPerRow = D / 8;             // chunks of a row
    static constexpr int kRuns = 32 * kPerRow / 32;   // chunks per lane
    uint4 x[kRuns];
    __device__ __forceinline__ void load(const MoveArgs& a, const Sources& s, int kv, int lane) {
#pragma unroll
        for (int i = 0; i < kRuns; i++) {
            const int run = lane + 32 * i, row = run / kPerRow, j = run % kPerRow;
            int o;
            const unsigned char* p = s.rec(a, row & 15, kv, kBytes, o);
            x[i] = *reinterpret_cast<const uint4*>(p + ((row & 16) + o) * (2 * D) + 16 * (j ^ (o & 7)));
        }
    }
    __device__ __forceinline__ void store(unsigned char* rec, int lane) const {
#pragma unroll
        for (int i = 0; i < kRuns; i++) {
            const int run = lane + 32 * i, row = run / kPerRow, j = run % kPerRow;
            *reinterpret_cast<uint4*>(rec + row * (2 * D) + 16 * (j ^ (row & 7))) = x[i];
        }
    }
};

template <class M, bool INPLACE>
__global__ void __launch_bounds__(kMoveWarps * 32) move_kernel(MoveArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = (int)(blockIdx.x / (unsigned)a.ctas), cta = (int)(blockIdx.x % (unsigned)a.ctas);
    const int b = row / a.Hkv, kv = row % a.Hkv;
    int L = a.seq_lens[b], n = a.kept_lens[b];
    const bool bad = L < 0 || L > a.src_max * kBlock || (a.w && (L > a.w_stride || L > a.out_stride)) || n < 0 ||
                     n > L || n > a.budget || n > a.dst_max * kBlock;
    if (bad) {  // nothing of this sequence is touched (the whole cluster leaves together)
        if (threadIdx.x == 0 && cta == 0 && kv == 0) flag_status(a.status, TQ_STATUS_BAD_LEN);
        return;
    }
    const int nrec = (n + kBlock - 1) / kBlock;
    const int wave = a.ctas * kMoveWarps;  // records of a wave
    const int32_t* kept = a.kept + (size_t)row * a.budget;
    const int32_t* st = a.src_tables + (size_t)b * a.src_max;
    const int32_t* dt = a.dst_tables + (size_t)b * a.dst_max;
    const float* w = a.w ? a.w + (size_t)row * a.w_stride : nullptr;
    float* w_out = a.w ? a.w_out + (size_t)row * a.out_stride : nullptr;
#pragma unroll 1
    for (int r0 = 0; r0 < nrec; r0 += wave) {
        const int r = r0 + cta * kMoveWarps + warp;
        M m;
        bool go = false;
        unsigned char* dst = nullptr;
        float wv = 0.f;
        bool have = false;  // this lane's slot receives a token
        if (r < nrec) {
            const int db = dt[r];
            go = (uint32_t)db < (uint32_t)a.num_blocks;
            if (!go && lane == 0) flag_status(a.status, TQ_STATUS_BAD_BLOCK);
            const int j = r * kBlock + (lane & 15);
            Sources s{db, lane & 15};  // a slot that receives nothing copies itself
            if (j < n) {
                const int t = kept[j];
                if (t < 0 || t >= L || (INPLACE && t < j)) {
                    flag_status(a.status, TQ_STATUS_BAD_SLOT);
                } else {
                    const int sb = st[t / kBlock];
                    if ((uint32_t)sb < (uint32_t)a.num_blocks) {
                        s.blk = sb;
                        s.off = t % kBlock;
                        have = true;
                        if (w && lane < 16) wv = w[t];
                    } else {
                        flag_status(a.status, TQ_STATUS_BAD_BLOCK);
                    }
                }
            }
            if (go) {
                dst = a.cache + ((size_t)db * a.Hkv + kv) * M::kBytes;
                m.load(a, s, kv, lane);
            }
        }
        if constexpr (INPLACE) cg::this_cluster().sync();
        if (go) {
            m.store(dst, lane);
            if (w && have && lane < 16) w_out[r * kBlock + lane] = wv;
        }
    }
    // the freed places of the sums: behind every source of the last wave's barrier
    if (w)
        for (int t = n + cta * (kMoveWarps * 32) + threadIdx.x; t < L; t += a.ctas * kMoveWarps * 32) w_out[t] = 0.f;
}

template <class M>
cudaError_t launch_m(MoveArgs a, bool in_place, cudaStream_t stream) {
    const int nrec = (a.budget + kBlock - 1) / kBlock;
    const int groups = (nrec + kMoveWarps - 1) / kMoveWarps;
    const long long rows = (long long)a.B * a.Hkv;
    if (!in_place) {
        a.ctas = groups;
        move_kernel<M, false><<<(unsigned)(rows * groups), kMoveWarps * 32, 0, stream>>>(a);
        return cudaGetLastError();
    }
    a.ctas = 1;
    while (a.ctas < 8 && a.ctas < groups) a.ctas *= 2;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)a.ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * a.ctas));
    cfg.blockDim = dim3(kMoveWarps * 32);
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, move_kernel<M, true>, a);
}

}  // namespace

cudaError_t launch_select(const float* w, long long stride, const int32_t* seq_lens, int B, int Hkv, int max_seq_len,
                          int budget, int sink, int recent, int32_t* kept, int32_t* kept_lens, int32_t* status,
                          cudaStream_t stream) {
    SelectArgs a = {w, stride, seq_lens, B, Hkv, max_seq_len, budget, sink, recent, kept, kept_lens, status, 0};
    // the fewest CTAs (up to 8) whose part of a row is judged in one go.  Calls in a row: more
    // are slower where there are rows enough (256 rows x 8192: 16.5 us with one, 26.7 with two),
    // fewer where parts get long (32 rows x 131072: 26.7 us with eight, 28.7 with four, 84 with
    // two).  Two to eight rows would gain by more: x 16384, 16.5 us with one, 12.4 with four; x
    // 8192, 12.4 and 10.7 to 12.3.
    int C = 1;
    while (C < 8 && (max_seq_len + C - 1) / C > 32 * kSelThreads) C *= 2;
    const int per = (max_seq_len + C - 1) / C;
    a.hold = per < kSelHold ? (per + 31) & ~31 : kSelHold;
    const size_t smem = (size_t)a.hold * sizeof(uint32_t) + kSelSmem;
    const long long rows = (long long)B * Hkv;  // rows * C < 2^31: B < 2^16, Hkv <= 2^5, C <= 2^3
    static std::mutex mu;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev < 0 || dev >= 64 || !configured[dev]) {
            e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kSelHold * (int)sizeof(uint32_t) + kSelSmem);
            if (e != cudaSuccess) return e;
            if (dev >= 0 && dev < 64) configured[dev] = true;
        }
    }
    if (C == 1) {
        select_kernel<<<(unsigned)rows, kSelThreads, smem, stream>>>(a);
        return cudaGetLastError();
    }
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)C;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, select_kernel, a);
}

cudaError_t launch_compact(unsigned char* cache, int num_blocks, int Hkv, int head_dim, int bf16,
                           const int32_t* src_tables, int src_max, const int32_t* seq_lens, const int32_t* kept,
                           const int32_t* kept_lens, int B, int budget, const int32_t* dst_tables, int dst_max,
                           const float* w, long long w_stride, float* w_out, long long out_stride, int32_t* status,
                           cudaStream_t stream) {
    MoveArgs a = {cache, num_blocks, Hkv, B, src_tables, src_max, seq_lens, kept, kept_lens, budget, dst_tables,
                  dst_max, w, w_out, w_stride, out_stride, status, 0};
    const bool in_place = dst_tables == nullptr;
    if (in_place) {
        a.dst_tables = src_tables;
        a.dst_max = src_max;
        a.w_out = const_cast<float*>(w);
        a.out_stride = w_stride;
    }
    if (bf16) return head_dim == 128 ? launch_m<BfMove<128>>(a, in_place, stream) : launch_m<BfMove<64>>(a, in_place, stream);
    return head_dim == 128 ? launch_m<TqMove<128>>(a, in_place, stream) : launch_m<TqMove<64>>(a, in_place, stream);
}

}  // namespace tq
