// pa_blocks.cu -- decoding over selected blocks of a long context: bounds of each block's keys,
// and the selection of blocks by a score of the query against them.  (The attention over the
// selected blocks is in pa_sparse.cuh.)
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_masked.h"

namespace pa {

namespace {

// 16 bytes that no other thread reads, kept out of L1: bounds of 58 K tokens of new prompts 21.2 us
// and a selection over 20 contexts of 60-126 K tokens 48.1 us; through L1 22.3 and 51.7.
__device__ __forceinline__ uint4 ld_once(const void* at) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(at));
    return v;
}

// floor(log2 x), -100 at least, of x >= 0 (not NaN).
__device__ __forceinline__ int32_t exponent_of(float x) {
    return max((int32_t)(__float_as_uint(x) >> 23) - 127, -100);
}
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float power_of_two(int32_t e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Pairs of 16-bit values (8-bit caches: widened to fp16): the larger and smaller ones (of a number
// and NaN: the number), and x * 0 + acc, which is NaN from the first infinity or NaN on.
template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (BF16) asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t odd2(uint32_t acc, uint32_t x) {
    uint32_t r;
    if constexpr (BF16) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
    else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
    return r;
}

// 16 bytes of K as pairs.
template <BoundsType T>
__device__ __forceinline__ void pairs(const uint4& x, uint32_t (&v)[T == BoundsType::kFp8 ? 8 : 4]) {
    if constexpr (T == BoundsType::kFp8) {
        e4m3x4_to_f16x2x2(x.x, v[0], v[1]);
        e4m3x4_to_f16x2x2(x.y, v[2], v[3]);
        e4m3x4_to_f16x2x2(x.z, v[4], v[5]);
        e4m3x4_to_f16x2x2(x.w, v[6], v[7]);
    } else {
        v[0] = x.x;
        v[1] = x.y;
        v[2] = x.z;
        v[3] = x.w;
    }
}

constexpr int kBoundsWarps = 4;
// Blocks of a sequence and kv head that a warp takes, one after another.
constexpr int kBoundsRun = 4;

// A warp per kv head and run of blocks: its lanes read a block's rows, 16 bytes each and several
// rows at once, and keep the largest and smallest value of their dims; the halves of the warp join
// by shuffles.  The step is a power of two, so that x / step and its rounding are exact in fp32.
// Bound by HBM for prompts (one read of K, 1/16 of it written), by latency for a step.  A run, since
// what comes before a block's rows (lengths, then table entries) is as long as the rows' own wait:
// 58 K tokens of new prompts, 8 heads of 128 (125 MB): 21.2 us, 5.9 TB/s (through L1, where the rest was
// measured, 22.3; a block at a time 23.2, 16 blocks 40; 26.7 with values compared one by one in fp32).
template <BoundsType T, int D, int BS>
__global__ void __launch_bounds__(32 * kBoundsWarps) key_bounds_kernel(const BoundsParams p) {
    constexpr int kElem = T == BoundsType::kFp8 ? 1 : 2;
    constexpr int kDims = 16 / kElem;                 // dims of a lane
    constexpr int kLanes = D / kDims;                 // lanes per row
    constexpr int kRows = 32 / kLanes;                // rows of one load
    constexpr int kLoads = BS / kRows;
    grid_dependency_wait();
    allow_dependent_launch();
    const int32_t lane = threadIdx.x & 31;
    const int32_t runs = (p.slots + kBoundsRun - 1) / kBoundsRun;
    const int64_t unit = (int64_t)blockIdx.x * kBoundsWarps + (threadIdx.x >> 5);
    const int32_t h = (int32_t)(unit % p.num_kv_heads);
    const int64_t at = unit / p.num_kv_heads;
    const int32_t s = (int32_t)(at / runs), run = (int32_t)(at - (int64_t)s * runs);
    if (s >= p.num_seqs) return;
    const int64_t cap = min((int64_t)p.max_blocks_per_seq * BS, (int64_t)INT32_MAX);
    int32_t n = p.max_new_tokens;
    const int32_t l = p.context_lens[s];
    bool bad = l < 0 || l > cap;
    if (p.query_starts) {
        n = p.query_starts[s + 1] - p.query_starts[s];
        bad |= n < 0 || n > p.max_new_tokens;
        n = min(max(n, 0), p.max_new_tokens);
    }
    if (bad && run == 0 && h == 0 && lane == 0 && p.status) atomicOr(p.status, kDevBadLen);
    const int32_t len = (int32_t)min((int64_t)max(l, 0), cap);
    // this run's blocks: of those that hold a new token
    const int32_t first = max(len - n, 0) / BS + run * kBoundsRun;
    const int32_t count = n == 0 ? 0 : min(len / BS + (len % BS != 0) - first, kBoundsRun);
    int32_t entry = 0;                                // lane i: block i's place in the pool
    if (lane < count) entry = p.block_tables[(size_t)s * p.max_blocks_per_seq + first + lane];
    for (int32_t i = 0; i < count; ++i) {
        const int32_t block = first + i, valid = min(len - block * BS, BS);
        const int32_t phys = __shfl_sync(0xffffffffu, entry, i);
        if (phys < 0 || phys >= p.num_blocks) {
            if (h == 0 && lane == 0 && p.status) atomicOr(p.status, kDevBadBlock);
            continue;
        }
        const int64_t place = (int64_t)phys * p.num_kv_heads + h;
        const uint4* rows = static_cast<const uint4*>(p.key_cache) + place * BS * kLanes;
        uint4 x[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (i * kRows + lane / kLanes < valid) x[i] = ld_once(rows + i * 32 + lane);
        constexpr bool kBf16 = T == BoundsType::kBf16;
        constexpr uint32_t kInf = kBf16 ? 0x7F807F80u : 0x7C007C00u, kSign = 0x80008000u;
        uint32_t top[kDims / 2], bottom[kDims / 2], odd = 0;
#pragma unroll
        for (int d = 0; d < kDims / 2; ++d) {
            top[d] = kInf | kSign;
            bottom[d] = kInf;
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (i * kRows + lane / kLanes < valid) {
                uint32_t v[kDims / 2];
                pairs<T>(x[i], v);
#pragma unroll
                for (int d = 0; d < kDims / 2; ++d) {
                    odd = odd2<kBf16>(odd, v[d]);
                    top[d] = max2<kBf16>(top[d], v[d]);
                    bottom[d] = min2<kBf16>(bottom[d], v[d]);
                }
            }
        }
#pragma unroll
        for (int o = kLanes; o < 32; o <<= 1)
#pragma unroll
            for (int d = 0; d < kDims / 2; ++d) {
                top[d] = max2<kBf16>(top[d], __shfl_xor_sync(0xffffffffu, top[d], o));
                bottom[d] = min2<kBf16>(bottom[d], __shfl_xor_sync(0xffffffffu, bottom[d], o));
            }
        // (rare) an infinity, or NaN?
        bool nan = false;
        if (__any_sync(0xffffffffu, odd != 0)) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                if (i * kRows + lane / kLanes < valid) {
                    uint32_t v[kDims / 2];
                    pairs<T>(x[i], v);
#pragma unroll
                    for (int d = 0; d < kDims / 2; ++d)
                        nan |= (v[d] & 0x7FFFu) > (kInf & 0xFFFFu) || ((v[d] >> 16) & 0x7FFFu) > (kInf & 0xFFFFu);
                }
        }
        float hi[kDims], lo[kDims];
#pragma unroll
        for (int d = 0; d < kDims / 2; ++d) {
            unpack2<kBf16>(top[d], hi[2 * d], hi[2 * d + 1]);
            unpack2<kBf16>(bottom[d], lo[2 * d], lo[2 * d + 1]);
        }
        nan = __any_sync(0xffffffffu, nan);
        // (a dim of NaN alone stays at -inf, inf: it counts as 0; an infinity as the largest number)
        constexpr float kMost = T == BoundsType::kBf16 ? 3.38953139e38f : 65504.f;
        float most = 0.f;
#pragma unroll
        for (int d = 0; d < kDims; ++d) {
            if (hi[d] < lo[d]) hi[d] = lo[d] = 0.f;
            most = fmaxf(most, fmaxf(fabsf(hi[d]), fabsf(lo[d])));
        }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        const int32_t e = min(exponent_of(fminf(most, kMost)), 96) - 6;
        const float inv = power_of_two(-e);
        // row groups 0 and 1 write the upper and the lower bounds
        int8_t* out = p.bounds + place * 2 * D;
        const int32_t part = lane / kLanes;
        if (part < 2) {
            uint32_t w[kDims / 4];
#pragma unroll
            for (int k = 0; k < kDims / 4; ++k) {
                w[k] = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const float y = part ? lo[4 * k + b] : hi[4 * k + b];
                    const int32_t q = __float2int_rn(fminf(fmaxf(y * inv, -127.f), 127.f));
                    w[k] |= ((uint32_t)q & 0xFFu) << (8 * b);
                }
            }
            int8_t* dst = out + part * D + (lane % kLanes) * kDims;
            if constexpr (kDims == 16) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            else *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        }
        if (lane == 0) p.steps[place] = nan ? __int_as_float(0x7fc00000) : power_of_two(e);
    }
}

// ------------------------------------------------------------------ selection
// Context of a sequence, clamped to its table row and the host's bound.
__device__ __forceinline__ int32_t context_of(const SelectParams& p, int32_t s, bool report) {
    const int64_t row = (int64_t)p.max_blocks_per_seq * p.block_size;
    const int32_t cap = (int32_t)min(row, (int64_t)p.max_context_len);
    const int32_t l = p.context_lens[s];
    if (report && (l < 0 || l > cap) && p.status) atomicOr(p.status, kDevBadLen);
    return min(max(l, 0), cap);
}
// Blocks that query token j of a sequence with context `len` sees.
__device__ __forceinline__ int32_t blocks_of(const SelectParams& p, int32_t len, int32_t j) {
    const int32_t seen = max(len - p.q_len + j + 1, 0);
    return seen / p.block_size + (seen % p.block_size != 0);
}

// The score of a block needs of a group's queries only the sums of their positive and of their
// negative values: with p the queries as whole numbers,
//     sum_j sum_d max(p_jd hi_d, p_jd lo_d) = sum_d P_d hi_d + N_d lo_d,
//     P = sum_j max(p_j, 0), N = sum_j min(p_j, 0),
// however many heads.  D / 16 lanes take a (query token, kv head), 16 dims each, and write its
// weights, 16 bits each: P of 16 dims, then N, lane by lane.

// What takes the queries of a group, the largest of magnitude `most`, to whole numbers of at most 64
// (an infinity counts as the largest number, which comes to 64 as well).
template <bool BF16>
__device__ __forceinline__ float weight_scale(float most) {
    constexpr float kBig = BF16 ? 3.38953139e38f : 65504.f;
    return power_of_two(5 - exponent_of(fminf(most, kBig)));
}
__device__ __forceinline__ int32_t weight_of(float v, float scale) {
    return __float2int_rn(fminf(fmaxf(v * scale, -64.f), 64.f));
}

// The weights of dims 16 c .. of a row's group of queries (`q`: the row's queries, dims 16 c on), by
// D / 16 lanes together.
template <bool BF16, int D>
__device__ __forceinline__ void group_weights(const uint4* q, int32_t group, uint32_t (&w)[16]) {
    constexpr int kLanes = D / 16;
    // four heads' rows at once (those past the group: the last one's again, not counted)
    uint4 x[4][2];
    auto load = [&](int32_t g0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int32_t g = min(g0 + k, group - 1);
            x[k][0] = q[g * (D / 8)];
            x[k][1] = q[g * (D / 8) + 1];
        }
    };
    // calls f(i, v) for the 16 values of head k (NaN: 0)
    auto each = [&](int k, auto&& f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint4& y = x[k][i >> 2];
            float a, b;
            unpack2<BF16>((i & 3) == 0 ? y.x : (i & 3) == 1 ? y.y : (i & 3) == 2 ? y.z : y.w, a, b);
            f(2 * i, a == a ? a : 0.f);
            f(2 * i + 1, b == b ? b : 0.f);
        }
    };
    float most = 0.f;
    for (int32_t g0 = 0; g0 < group; g0 += 4) {
        load(g0);
#pragma unroll
        for (int k = 0; k < 4; ++k) each(k, [&](int, float v) { most = fmaxf(most, fabsf(v)); });
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    const float inv = weight_scale<BF16>(most);
    int32_t up[16], down[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) up[i] = down[i] = 0;
    for (int32_t g0 = 0; g0 < group; g0 += 4) {
        if (group > 4) load(g0);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (g0 + k < group)
                each(k, [&](int i, float v) {
                    const int32_t z = weight_of(v, inv);
                    up[i] += max(z, 0);
                    down[i] += min(z, 0);
                });
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[i] = (uint32_t)((up[2 * i] & 0xFFFF) | (up[2 * i + 1] << 16));
        w[8 + i] = (uint32_t)((down[2 * i] & 0xFFFF) | (down[2 * i + 1] << 16));
    }
}

constexpr int kWeightThreads = 128;
template <bool BF16, int D>
__global__ void __launch_bounds__(kWeightThreads) select_weights_kernel(const SelectParams p) {
    constexpr int kLanes = D / 16;
    grid_dependency_wait();
    allow_dependent_launch();      // (after the wait: the scores read all but the weights early)
    const int64_t row = ((int64_t)blockIdx.x * kWeightThreads + threadIdx.x) / kLanes;   // token and head
    const int32_t c = threadIdx.x % kLanes;
    const int64_t rows = (int64_t)p.num_seqs * p.q_len * p.num_kv_heads;
    uint32_t w[16];
    group_weights<BF16, D>(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.query) +
                                                          min(row, rows - 1) * p.group * D + c * 16),
                           p.group, w);
    if (row >= rows) return;
    uint4* out = reinterpret_cast<uint4*>(p.weights + (row * kLanes + c) * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

constexpr int kScoreThreads = 256;
constexpr int kScoreBatch = 4;            // records that a lane has on their way

// Four records of a lane, 16 dims each: upper and lower bounds; the step of the one whose score the
// lane ends up with (0: a block outside the pool).
struct ScoreBatch {
    uint4 x[kScoreBatch][2];
    float step;
};

// Which of four records a lane ends up with.
template <int D>
__device__ __forceinline__ int32_t record_of(int32_t c) {
    return (c / (D / 64)) & 3;
}

// The scores of four records against weights P (wp) and N (wn), D / 16 lanes together (every lane of
// the warp comes here), in an order that unsigned numbers keep: record record_of(c)'s in lane c.
template <int D>
__device__ __forceinline__ uint32_t score_batch(const ScoreBatch& y, const int32_t (&wp)[8], const int32_t (&wn)[8],
                                                int32_t c) {
    int32_t dot[kScoreBatch];
#pragma unroll
    for (int k = 0; k < kScoreBatch; ++k) {
        int32_t a = 0, b = 0;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const uint4 &v = y.x[k][0], &z = y.x[k][1];
            const int32_t hi = (int32_t)(m == 0 ? v.x : m == 1 ? v.y : m == 2 ? v.z : v.w);
            const int32_t lo = (int32_t)(m == 0 ? z.x : m == 1 ? z.y : m == 2 ? z.z : z.w);
            a = __dp2a_lo(wp[2 * m], hi, a);
            b = __dp2a_hi(wp[2 * m + 1], hi, b);
            a = __dp2a_lo(wn[2 * m], lo, a);
            b = __dp2a_hi(wn[2 * m + 1], lo, b);
        }
        dot[k] = a + b;
    }
    // the lanes' sums: half of the lanes go on with records 2, 3, then with the odd one
    constexpr int kHalf = D / 32, kQuarter = D / 64;
    const bool top = c & kHalf, odd = c & kQuarter;
    int32_t a = top ? dot[2] : dot[0], b = top ? dot[3] : dot[1];
    a += __shfl_xor_sync(0xffffffffu, top ? dot[0] : dot[2], kHalf);
    b += __shfl_xor_sync(0xffffffffu, top ? dot[1] : dot[3], kHalf);
    int32_t d = odd ? b : a;
    d += __shfl_xor_sync(0xffffffffu, odd ? a : b, kQuarter);
#pragma unroll
    for (int o = kQuarter / 2; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    const float f = fmaf((float)d, y.step, 0.f);      // (0, not -0, where the step is 0)
    const uint32_t bits = __float_as_uint(f);
    return f != f ? 0xffffffffu : (bits >> 31) ? ~bits : bits | 0x80000000u;
}

// Blocks of a sequence with scores: the last query token's, without the first and last ones.
__device__ __forceinline__ int32_t scored_of(const SelectParams& p, int32_t s) {
    const int32_t blocks = blocks_of(p, context_of(p, s, false), p.q_len - 1);
    return blocks > p.num_selected ? blocks - p.num_first - p.num_last : 0;
}

// Scores of the sequences' blocks, laid end to end (and once more for each further turn of kv
// heads, as many at a time as the CTA has groups of lanes) and cut into equal slices, one per CTA:
// contexts of any lengths keep all CTAs busy to the end.  (20 contexts of 60-126 K tokens, the whole
// selection: 48 us; with a CTA per piece of 64 blocks of a sequence 8 more.)  A lane has 16 dims of a
// head: their weights in registers, and 16 bytes of upper and of lower bounds of four records on
// their way; D / 16 lanes share a record.  Whole-number products, exact sums (below 2^24), one exact
// product with the block's step.  All that the weights do not come with is read before the kernel
// that writes them has finished.  Bound by HBM: 2 D + 4 bytes per block and kv head.  QT query tokens
// share a fetch: with more than two a CTA fetches its chunk again for each further pair, and the
// kernels of pairs spill 124 bytes at 128 registers (those of one token none).
template <int D, int QT>
__global__ void __launch_bounds__(kScoreThreads, 2) block_scores_kernel(const SelectParams p) {
    constexpr int kLanes = D / 16;                           // lanes per record
    constexpr int kGroups = kScoreThreads / kLanes;
    __shared__ int32_t rec_s[kMaxScoreChunk];                // first record of the blocks; -1: none
    allow_dependent_launch();
    const int32_t tid = threadIdx.x, lane = tid & 31;
    const int32_t heads = min(p.num_kv_heads, kGroups);      // kv heads of this CTA at a time
    const int32_t turns = (p.num_kv_heads + heads - 1) / heads;
    const int32_t grp = tid / kLanes, c = tid % kLanes;
    const int32_t sub = grp / heads, subs = kGroups / heads;
    // Sequences s0 .. s0 + 31, one per lane: blocks with scores, and their running sum.
    int32_t own = 0, upto = 0;
    auto sequences = [&](int32_t s0) {
        own = s0 + lane < p.num_seqs ? scored_of(p, s0 + lane) : 0;
        upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        return __shfl_sync(0xffffffffu, upto, 31);
    };
    // this CTA's slice
    int64_t all = 0;
    for (int32_t s0 = 0; s0 < p.num_seqs; s0 += 32) all += sequences(s0);
    const int64_t total = all * turns;
    int64_t at0 = total * blockIdx.x / gridDim.x;
    const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
    bool waited = false;
    while (at0 < end) {
        // the sequence and block of `at0` (every warp for itself)
        const int32_t turn = (int32_t)(at0 / all);
        int64_t before = turn * all;
        int32_t s = 0, b0 = 0, n = 0;
        for (int32_t s0 = 0; s0 < p.num_seqs; s0 += 32) {
            if (p.num_seqs > 32) sequences(s0);
            const uint32_t past = __ballot_sync(0xffffffffu, before + upto > at0);
            if (past) {
                const int32_t l = __ffs(past) - 1;
                s = s0 + l;
                n = __shfl_sync(0xffffffffu, own, l);
                b0 = (int32_t)(at0 - before) - (__shfl_sync(0xffffffffu, upto, l) - n);
                break;
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
        n = (int32_t)min(min((int64_t)(n - b0), end - at0), (int64_t)kMaxScoreChunk);
        at0 += n;
        b0 += p.num_first;
        bool bad = false;
        for (int32_t i = tid; i < n; i += kScoreThreads) {
            const int32_t phys = p.block_tables[(size_t)s * p.max_blocks_per_seq + b0 + i];
            const bool out = phys < 0 || phys >= p.num_blocks;
            bad |= out;
            rec_s[i] = out ? -1 : phys * p.num_kv_heads;     // (a pool has fewer than 2^31 rows)
        }
        __syncthreads();
        const int32_t h = turn * heads + grp % heads;
        const bool mine = sub < subs && h < p.num_kv_heads;
        const int32_t head = mine ? h : 0;
        // the record whose score this lane ends up with, of four
        const int32_t u = record_of<D>(c);
        const int8_t* const at = p.bounds + c * 16;
        // four records of this lane, from place `first` on (past the end: the last one again)
        auto fetch = [&](int32_t first, ScoreBatch& t) {
            int32_t rec[kScoreBatch];
#pragma unroll
            for (int k = 0; k < kScoreBatch; ++k) rec[k] = rec_s[min(first + k * subs, n - 1)];
#pragma unroll
            for (int k = 0; k < kScoreBatch; ++k) {
                const int8_t* src = at + (size_t)(uint32_t)(max(rec[k], 0) + head) * (2 * D);
                t.x[k][0] = ld_once(src);
                t.x[k][1] = ld_once(src + D);
            }
            const int32_t r = u == 0 ? rec[0] : u == 1 ? rec[1] : u == 2 ? rec[2] : rec[3];
            t.step = __ldg(p.steps + (size_t)(uint32_t)(max(r, 0) + head));
            if (r < 0) t.step = 0.f;
        };
        const int32_t stride = kScoreBatch * subs;
        ScoreBatch one, two;
        fetch(sub, one);
        if (!waited) {
            grid_dependency_wait();
            waited = true;
        }
        if (bad && turn == 0 && p.status) atomicOr(p.status, kDevBadBlock);
        for (int32_t j0 = 0; j0 < p.q_len; j0 += QT) {
            int32_t wp[QT][8], wn[QT][8];                    // 16 weights each, two to a register
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                const int64_t row = ((int64_t)s * p.q_len + min(j0 + t, p.q_len - 1)) * p.num_kv_heads + head;
                const int4* src = reinterpret_cast<const int4*>(p.weights + (row * kLanes + c) * 16);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int4 a = src[i], b = src[2 + i];
                    wp[t][4 * i] = a.x, wp[t][4 * i + 1] = a.y, wp[t][4 * i + 2] = a.z, wp[t][4 * i + 3] = a.w;
                    wn[t][4 * i] = b.x, wn[t][4 * i + 1] = b.y, wn[t][4 * i + 2] = b.z, wn[t][4 * i + 3] = b.w;
                }
            }
            uint32_t* const keys =
                p.keys + (((size_t)s * p.q_len + j0) * p.num_kv_heads + head) * p.max_blocks + b0;
            auto score = [&](int32_t first, const ScoreBatch& y) {
                const int32_t i = first + u * subs;
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    const uint32_t key = score_batch<D>(y, wp[t], wn[t], c);
                    if (mine && c % (kLanes / 4) == 0 && i < n && j0 + t < p.q_len)
                        keys[(size_t)t * p.num_kv_heads * p.max_blocks + i] = key;
                }
            };
            // (a warp's groups go through the steps together: its shuffles need every lane)
            if (j0 > 0) fetch(sub, one);
            for (int32_t first = sub; first - sub < n; first += 2 * stride) {
                fetch(first + stride, two);
                score(first, one);
                fetch(first + 2 * stride, one);
                score(first + stride, two);
            }
        }
        __syncthreads();                                     // rec_s is free again
    }
    if (!waited) grid_dependency_wait();
    if (blockIdx.x == 0)
        for (int32_t s = tid; s < p.num_seqs; s += kScoreThreads) (void)context_of(p, s, true);   // reports
}

// (1024, with half the keys each: the selection over 20 contexts of 60-126 K tokens 2.5 us more)
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelRegs = 16;              // keys of a thread that stay in registers
constexpr int kSelBins = 2048;

// Exclusive scan over the CTA's threads; *total receives the sum.  `buf`: 32 ints.
__device__ __forceinline__ int32_t scan_cta(int32_t x, int32_t* buf, int32_t* total) {
    const int32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) buf[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int32_t w = lane < kSelWarps ? buf[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        buf[lane] = w;
    }
    __syncthreads();
    const int32_t before = (warp > 0 ? buf[warp - 1] : 0) + v - x;
    *total = buf[31];
    __syncthreads();
    return before;
}

// The `want` largest of a row's scores, by one CTA.  A histogram over the scores' own range (2048
// bins, so that the counts spread) finds the bin that holds the smallest of them; what is in that
// bin is ranked one against the other, or, where that is more than there are threads, the range is
// narrowed to the bin and divided again, until one value is left, of which the first blocks are
// taken.  What is taken is a bit per block, which puts the list in order.  Bound by latency: the
// passes over at most 16 keys a thread and the scans between them.
struct SelectSmem {
    int32_t buf[32];
    alignas(16) int32_t hist[kSelBins];
    uint32_t range[2];             // the scores' least and greatest
    int32_t found[2];              // the bin, and the scores above it
    int32_t gathered;
    static_assert(2 * kSelThreads <= kSelBins, "the candidates take the histogram's place");
};

// Before select_row, and a barrier.
__device__ __forceinline__ void select_clear(SelectSmem& sm) {
    for (int32_t i = threadIdx.x; i < kSelBins; i += kSelThreads) sm.hist[i] = 0;
    if (threadIdx.x == 0) {
        sm.range[0] = 0xffffffffu;
        sm.range[1] = 0u;
        sm.gathered = 0;
    }
}

// keys[i]: block i's score, of the blocks from num_first on and before the last num_last of the
// row's `blocks`; `bits`: two bits of shared memory per block.
__device__ __forceinline__ void select_row(const SelectParams& p, int32_t blocks, const uint32_t* keys,
                                           uint32_t* bits_smem, SelectSmem& sm, int32_t* out) {
    const int32_t tid = threadIdx.x, lane = tid & 31;
    const int32_t words = (blocks + 31) / 32;
    uint32_t* const take = bits_smem;
    uint32_t* const tie = bits_smem + (p.max_blocks + 31) / 32;
    const int32_t m0 = p.num_first, m1 = blocks - p.num_last;    // scored blocks: m0 .. m1 - 1
    int32_t want = p.num_selected - p.num_first - p.num_last;
    const int32_t rounds = (blocks + kSelThreads - 1) / kSelThreads;
    uint32_t reg[kSelRegs];
#pragma unroll
    for (int r = 0; r < kSelRegs; ++r) {
        const int32_t i = r * kSelThreads + tid;
        reg[r] = i >= m0 && i < m1 ? keys[i] : 0u;
    }
    // calls f(block, key) for this thread's scored blocks
    auto each = [&](auto&& f) {
#pragma unroll
        for (int r = 0; r < kSelRegs; ++r) {
            const int32_t i = r * kSelThreads + tid;
            if (i >= m0 && i < m1) f(i, reg[r]);
        }
        for (int32_t i = kSelRegs * kSelThreads + tid; i < m1; i += kSelThreads)
            if (i >= m0) f(i, keys[i]);
    };
    uint32_t lo = 0xffffffffu, hi = 0u;
    each([&](int32_t, uint32_t k) {
        lo = min(lo, k);
        hi = max(hi, k);
    });
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        atomicMin(&sm.range[0], lo);
        atomicMax(&sm.range[1], hi);
    }
    __syncthreads();
    lo = sm.range[0];
    hi = sm.range[1];
    // Narrow lo .. hi until all of it is taken (`all`), few enough of it are left to be ranked
    // (`rank`), or one value is; `want` of it are taken.
    bool all = want == 0, rank = false;
    if (all) lo = hi = 0xffffffffu;               // (nothing above, nothing within)
    for (bool again = false; !all && !rank && lo < hi; again = true) {
        const int32_t shift = max(0, 21 - __clz(hi - lo));
        if (again) {
            for (int32_t i = tid; i < kSelBins; i += kSelThreads) sm.hist[i] = 0;
            __syncthreads();
        }
        each([&](int32_t, uint32_t k) {
            if (k >= lo && k <= hi) atomicAdd(&sm.hist[(k - lo) >> shift], 1);
        });
        __syncthreads();
        // bins from the top: thread t has the bins that end at kSelBins - 1 - 4 t
        constexpr int kPer = kSelBins / kSelThreads;
        int32_t mine = 0, n[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            n[k] = sm.hist[kSelBins - 1 - (tid * kPer + k)];
            mine += n[k];
        }
        int32_t total, above = scan_cta(mine, sm.buf, &total);
        if (above < want && want <= above + mine) {
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                if (above < want && want <= above + n[k]) {
                    sm.found[0] = kSelBins - 1 - (tid * kPer + k);
                    sm.found[1] = above;
                }
                above += n[k];
            }
        }
        __syncthreads();
        const int32_t bin = sm.found[0], here = sm.hist[bin];
        want -= sm.found[1];
        all = here == want;
        rank = !all && here <= kSelThreads;
        lo += (uint32_t)bin << shift;
        hi = lo + min(hi - lo, (1u << shift) - 1u);      // (lo + a bin may pass 32 bits)
        __syncthreads();
    }
    // the bits: everything above the range, and the range itself if all of it is taken; what is
    // to be ranked goes to a list, what is equal to bits of its own
    uint2* const cand = reinterpret_cast<uint2*>(sm.hist);
    auto mark = [&](int32_t i, uint32_t k, bool scored) {
        const bool here = scored && want > 0 && k >= lo && k <= hi;
        const bool in = i < blocks && (!scored || (want > 0 && k > hi) || (here && all));
        const uint32_t t = __ballot_sync(0xffffffffu, in);
        if (lane == 0 && (i >> 5) < words) take[i >> 5] = t;
        if (!all && !rank) {
            const uint32_t e = __ballot_sync(0xffffffffu, here);
            if (lane == 0 && (i >> 5) < words) tie[i >> 5] = e;
        } else if (here && rank) {
            cand[atomicAdd(&sm.gathered, 1)] = make_uint2(k, (uint32_t)i);
        }
    };
#pragma unroll
    for (int r = 0; r < kSelRegs; ++r) {
        if (r < rounds) {
            const int32_t i = r * kSelThreads + tid;
            mark(i, reg[r], i >= m0 && i < m1);
        }
    }
    for (int32_t r = kSelRegs; r < rounds; ++r) {
        const int32_t i = r * kSelThreads + tid;
        const bool scored = i >= m0 && i < m1;
        mark(i, scored ? keys[i] : 0u, scored);
    }
    __syncthreads();
    if (rank) {
        const int32_t n = sm.gathered;
        if (tid < n) {
            const uint2 me = cand[tid];
            int32_t better = 0;
            for (int32_t i = 0; i < n; ++i) {
                const uint2 x = cand[i];
                better += x.x > me.x || (x.x == me.x && x.y < me.y);
            }
            if (better < want) atomicOr(&take[me.y >> 5], 1u << (me.y & 31));
        }
        __syncthreads();
    }
    // of the ties, the first `want`; then the list, word by word
    int32_t ties = 0, at = 0;
    for (int32_t w0 = 0; w0 < words; w0 += kSelThreads) {
        const int32_t w = w0 + tid;
        uint32_t bits = w < words ? take[w] : 0u;
        int32_t total;
        if (!all && !rank) {
            uint32_t e = w < words ? tie[w] : 0u;
            const int32_t before = ties + scan_cta(__popc(e), sm.buf, &total);
            ties += total;
            for (int32_t left = want - before; e && left > 0; --left) {
                bits |= e & (0u - e);
                e &= e - 1u;
            }
        }
        int32_t to = at + scan_cta(__popc(bits), sm.buf, &total);
        at += total;
        for (; bits; bits &= bits - 1u) out[to++] = 32 * w + __ffs(bits) - 1;
    }
}

// CTA (query token, kv head): the selection from scores in memory.
__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(const SelectParams p) {
    extern __shared__ uint32_t sel_smem[];
    __shared__ SelectSmem sm;
    // (the kernel that writes the weights has waited for all that comes before this call)
    const int64_t row = (int64_t)blockIdx.x * p.num_kv_heads + blockIdx.y;
    const int32_t s = (int32_t)(blockIdx.x / p.q_len), j = (int32_t)(blockIdx.x % p.q_len);
    const int32_t blocks = blocks_of(p, context_of(p, s, false), j);
    select_clear(sm);
    __syncthreads();
    grid_dependency_wait();
    allow_dependent_launch();
    int32_t* out = p.selected + row * p.num_selected;
    if (blocks <= p.num_selected) {
        for (int32_t i = threadIdx.x; i < p.num_selected; i += kSelThreads) out[i] = i < blocks ? i : -1;
        return;
    }
    select_row(p, blocks, p.keys + row * p.max_blocks, sel_smem, sm, out);
}

// Short contexts: the same in one launch, CTA (query token, kv head).  The first warp takes the
// weights, four dims to a lane, while the others' first records come; D / 16 lanes score four blocks
// at a time into shared memory.
template <bool BF16, int D>
__global__ void __launch_bounds__(kSelThreads) select_short_kernel(const SelectParams p) {
    constexpr int kLanes = D / 16, kGroups = kSelThreads / kLanes;
    extern __shared__ uint32_t sel_smem[];      // two bits per block, then the scores
    __shared__ SelectSmem sm;
    __shared__ __align__(16) uint32_t weights[kLanes][16];
    select_clear(sm);
    grid_dependency_wait();
    allow_dependent_launch();
    const int32_t tid = threadIdx.x, lane = tid & 31, c = tid % kLanes, grp = tid / kLanes, h = blockIdx.y;
    const int64_t row = (int64_t)blockIdx.x * p.num_kv_heads + h;
    const int32_t s = (int32_t)(blockIdx.x / p.q_len), j = (int32_t)(blockIdx.x % p.q_len);
    // (the first blocks' table entries, the queries and the length are on their way together; an
    // entry past the context is not used)
    const int32_t first = p.num_first, u = record_of<D>(c);
    const int32_t* const table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    int32_t phys[kScoreBatch];
    auto entries = [&](int32_t i0) {
#pragma unroll
        for (int k = 0; k < kScoreBatch; ++k)
            phys[k] = table[min(first + i0 + k * kGroups + grp, p.max_blocks_per_seq - 1)];
    };
    auto fetch = [&](ScoreBatch& y) {           // (a block outside the pool: the first one's, times 0)
#pragma unroll
        for (int k = 0; k < kScoreBatch; ++k) {
            const bool out_of = phys[k] < 0 || phys[k] >= p.num_blocks;
            const size_t rec = (size_t)(out_of ? 0 : phys[k]) * p.num_kv_heads + h;
            const int8_t* src = p.bounds + rec * 2 * D + c * 16;
            y.x[k][0] = __ldg(reinterpret_cast<const uint4*>(src));
            y.x[k][1] = __ldg(reinterpret_cast<const uint4*>(src + D));
            if (k == u) {
                y.step = __ldg(p.steps + rec);
                if (out_of) y.step = 0.f;
            }
        }
    };
    entries(0);
    const int32_t blocks = blocks_of(p, context_of(p, s, tid == 0 && h == 0 && j == 0), j);
    int32_t* out = p.selected + row * p.num_selected;
    if (blocks <= p.num_selected) {
        for (int32_t i = tid; i < p.num_selected; i += kSelThreads) out[i] = i < blocks ? i : -1;
        return;
    }
    const int32_t n = blocks - p.num_first - p.num_last;
    ScoreBatch y;
    fetch(y);
    if (tid < 32) {
        // dims 4 lane .. of the group's heads, four heads at a time
        const bool here = 4 * lane < D;
        const uint2* q = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.query) + row * p.group * D) +
                         (here ? lane : 0);
        float v[4][4], most = 0.f;
        auto load = [&](int32_t g0) {
            uint2 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = q[min(g0 + k, p.group - 1) * (D / 4)];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                unpack2<BF16>(x[k].x, v[k][0], v[k][1]);
                unpack2<BF16>(x[k].y, v[k][2], v[k][3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[k][i] = v[k][i] == v[k][i] ? v[k][i] : 0.f;      // (NaN: 0)
            }
        };
        for (int32_t g0 = 0; g0 < p.group; g0 += 4) {
            load(g0);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) most = fmaxf(most, fabsf(v[k][i]));
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        const float inv = weight_scale<BF16>(most);
        int32_t up[4] = {0, 0, 0, 0}, down[4] = {0, 0, 0, 0};
        for (int32_t g0 = 0; g0 < p.group; g0 += 4) {
            if (p.group > 4) load(g0);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int32_t z = g0 + k < p.group ? weight_of(v[k][i], inv) : 0;
                    up[i] += max(z, 0);
                    down[i] += min(z, 0);
                }
        }
        if (here) {
            uint32_t* const w = &weights[lane / 4][2 * (lane & 3)];
            w[0] = (uint32_t)((up[0] & 0xFFFF) | (up[1] << 16));
            w[1] = (uint32_t)((up[2] & 0xFFFF) | (up[3] << 16));
            w[8] = (uint32_t)((down[0] & 0xFFFF) | (down[1] << 16));
            w[9] = (uint32_t)((down[2] & 0xFFFF) | (down[3] << 16));
        }
    }
    __syncthreads();
    int32_t wp[8], wn[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int4 a = reinterpret_cast<const int4*>(weights[c])[i], b = reinterpret_cast<const int4*>(weights[c])[2 + i];
        wp[4 * i] = a.x, wp[4 * i + 1] = a.y, wp[4 * i + 2] = a.z, wp[4 * i + 3] = a.w;
        wn[4 * i] = b.x, wn[4 * i + 1] = b.y, wn[4 * i + 2] = b.z, wn[4 * i + 3] = b.w;
    }
    uint32_t* const keys = sel_smem + 2 * ((p.max_blocks + 31) / 32);
    bool bad = false;
    for (int32_t i0 = 0; i0 < n; i0 += kScoreBatch * kGroups) {
        if (i0 > 0) fetch(y);
#pragma unroll
        for (int k = 0; k < kScoreBatch; ++k)
            bad |= (phys[k] < 0 || phys[k] >= p.num_blocks) && i0 + k * kGroups + grp < n;
        entries(i0 + kScoreBatch * kGroups);
        const uint32_t key = score_batch<D>(y, wp, wn, c);
        const int32_t i = i0 + u * kGroups + grp;
        if (c % (kLanes / 4) == 0 && i < n) keys[first + i] = key;
    }
    if (bad && p.status) atomicOr(p.status, kDevBadBlock);
    __syncthreads();
    select_row(p, blocks, keys, sel_smem, sm, out);
}

template <class Arg>
cudaError_t launch_pdl(dim3 grid, dim3 block, size_t smem, cudaStream_t stream, void (*kern)(Arg), const Arg& arg) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, arg);
}

template <BoundsType T>
cudaError_t launch_bounds_of(const BoundsParams& p, cudaStream_t stream) {
    using Kern = void (*)(BoundsParams);
    const Kern kern = p.head_size == 128
                          ? (p.block_size == 16 ? (Kern)key_bounds_kernel<T, 128, 16> : (Kern)key_bounds_kernel<T, 128, 32>)
                          : (p.block_size == 16 ? (Kern)key_bounds_kernel<T, 64, 16> : (Kern)key_bounds_kernel<T, 64, 32>);
    const int64_t units = (int64_t)p.num_seqs * ((p.slots + kBoundsRun - 1) / kBoundsRun) * p.num_kv_heads;
    return launch_pdl(dim3((unsigned)((units + kBoundsWarps - 1) / kBoundsWarps)), dim3(32 * kBoundsWarps), 0, stream,
                      kern, p);
}

}  // namespace

cudaError_t launch_key_bounds(const BoundsParams& p, BoundsType type, cudaStream_t stream) {
    switch (type) {
        case BoundsType::kF16: return launch_bounds_of<BoundsType::kF16>(p, stream);
        case BoundsType::kBf16: return launch_bounds_of<BoundsType::kBf16>(p, stream);
        default: return launch_bounds_of<BoundsType::kFp8>(p, stream);
    }
}

cudaError_t launch_select_blocks(const SelectParams& p, bool bf16, cudaStream_t stream) {
    using Kern = void (*)(SelectParams);
    const bool wide = p.head_size == 128;
    const dim3 rows((unsigned)(p.num_seqs * p.q_len), (unsigned)p.num_kv_heads);
    const size_t bits = 2 * sizeof(uint32_t) * (size_t)((p.max_blocks + 31) / 32);
    if (!p.keys) {
        const Kern kern = bf16 ? (wide ? (Kern)select_short_kernel<true, 128> : (Kern)select_short_kernel<true, 64>)
                               : (wide ? (Kern)select_short_kernel<false, 128> : (Kern)select_short_kernel<false, 64>);
        // (lists with room for every block need no scores)
        const size_t smem = p.max_blocks > p.num_selected ? bits + sizeof(uint32_t) * (size_t)p.max_blocks : 0;
        return launch_pdl(rows, dim3(kSelThreads), smem, stream, kern, p);
    }
    const bool one = p.q_len == 1;
    const Kern weights = bf16 ? (wide ? (Kern)select_weights_kernel<true, 128> : (Kern)select_weights_kernel<true, 64>)
                              : (wide ? (Kern)select_weights_kernel<false, 128> : (Kern)select_weights_kernel<false, 64>);
    const Kern scores = wide ? (one ? (Kern)block_scores_kernel<128, 1> : (Kern)block_scores_kernel<128, 2>)
                             : (one ? (Kern)block_scores_kernel<64, 1> : (Kern)block_scores_kernel<64, 2>);
    const int64_t lanes = (int64_t)p.num_seqs * p.q_len * p.num_kv_heads * (p.head_size / 16);
    cudaError_t e = launch_pdl(dim3((unsigned)((lanes + kWeightThreads - 1) / kWeightThreads)), dim3(kWeightThreads), 0,
                               stream, weights, p);
    if (e != cudaSuccess) return e;
    const int32_t heads = std::min(p.num_kv_heads, kScoreThreads / (p.head_size / 16));
    // two CTAs to an SM, but none with fewer than 32 blocks of the longest contexts
    const int64_t most = (int64_t)p.num_seqs * ((p.num_kv_heads + heads - 1) / heads) * p.max_blocks;
    e = launch_pdl(dim3((unsigned)std::max<int64_t>(std::min<int64_t>(2 * p.sms, most / 32), 1)), dim3(kScoreThreads), 0,
                   stream, scores, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(rows, dim3(kSelThreads), bits, stream, select_blocks_kernel, p);
}

}  // namespace pa
