// pa_blocks.cu -- decoding over selected blocks of a long context: bounds of each block's keys,
// and the selection of blocks by a score of the query against them.  (The attention over the
// selected blocks is in pa_sparse.cu.)
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_masked.h"

namespace pa {

namespace {

// floor(log2 x), -100 at least, of x >= 0 (not NaN).
__device__ __forceinline__ int32_t exponent_of(float x) {
    return max((int32_t)(__float_as_uint(x) >> 23) - 127, -100);
}
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float power_of_two(int32_t e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// 16 bytes of K as floats.
template <BoundsType T>
__device__ __forceinline__ void widen(const uint4& x, float (&v)[T == BoundsType::kFp8 ? 16 : 8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (T == BoundsType::kFp8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t lo, hi;
            e4m3x4_to_f16x2x2(w[i], lo, hi);
            unpack2<false>(lo, v[4 * i], v[4 * i + 1]);
            unpack2<false>(hi, v[4 * i + 2], v[4 * i + 3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack2<T == BoundsType::kBf16>(w[i], v[2 * i], v[2 * i + 1]);
    }
}

constexpr int kBoundsWarps = 4;

// A warp per (block, kv head): its lanes read the block's rows, 16 bytes each and several rows
// at once, and keep the largest and smallest value of their dims; the halves of the warp join by
// shuffles.  The step is a power of two, so that x / step and its rounding are exact in fp32.
// Bound by HBM for prompts (one read of K, 1/16 of it written), by latency for a step.
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
    const int64_t unit = (int64_t)blockIdx.x * kBoundsWarps + (threadIdx.x >> 5);
    const int32_t h = (int32_t)(unit % p.num_kv_heads);
    const int64_t at = unit / p.num_kv_heads;
    const int32_t s = (int32_t)(at / p.slots), j = (int32_t)(at - (int64_t)s * p.slots);
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
    if (bad && j == 0 && h == 0 && lane == 0 && p.status) atomicOr(p.status, kDevBadLen);
    const int32_t len = (int32_t)min((int64_t)max(l, 0), cap);
    const int32_t block = max(len - n, 0) / BS + j;   // the j-th block that holds a new token
    const int32_t valid = min(len - block * BS, BS);
    if (n == 0 || valid <= 0) return;
    const int32_t phys = p.block_tables[(size_t)s * p.max_blocks_per_seq + block];
    if (phys < 0 || phys >= p.num_blocks) {
        if (h == 0 && lane == 0 && p.status) atomicOr(p.status, kDevBadBlock);
        return;
    }
    const int64_t place = (int64_t)phys * p.num_kv_heads + h;
    const uint4* rows = static_cast<const uint4*>(p.key_cache) + place * BS * kLanes;
    uint4 x[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        if (i * kRows + lane / kLanes < valid) x[i] = rows[i * 32 + lane];
    float hi[kDims], lo[kDims];
    bool nan = false;
#pragma unroll
    for (int d = 0; d < kDims; ++d) {
        hi[d] = -INFINITY;
        lo[d] = INFINITY;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        if (i * kRows + lane / kLanes < valid) {
            float v[kDims];
            widen<T>(x[i], v);
#pragma unroll
            for (int d = 0; d < kDims; ++d) {
                nan |= v[d] != v[d];
                hi[d] = fmaxf(hi[d], v[d]);
                lo[d] = fminf(lo[d], v[d]);
            }
        }
    }
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1)
#pragma unroll
        for (int d = 0; d < kDims; ++d) {
            hi[d] = fmaxf(hi[d], __shfl_xor_sync(0xffffffffu, hi[d], o));
            lo[d] = fminf(lo[d], __shfl_xor_sync(0xffffffffu, lo[d], o));
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

constexpr int kScoreThreads = 256;
constexpr int kScoreBatch = 4;            // records that a lane has on their way

// Two signed 16-bit by two signed 8-bit products, added: the lower (upper) bytes of b.
__device__ __forceinline__ int32_t dp2_lo(int32_t a, int32_t b, int32_t c) { return __dp2a_lo(a, b, c); }
__device__ __forceinline__ int32_t dp2_hi(int32_t a, int32_t b, int32_t c) { return __dp2a_hi(a, b, c); }

// Scores of a chunk of one sequence's blocks: CTA (sequence, chunk, kv heads by the groups of
// lanes that it has).  The heads of a kv head's group are quantised with one power-of-two step
// to whole numbers of at most 64 and added, the positive ones against the upper bounds, the
// negative ones against the lower: sum_j sum_d max(q hi, q lo) = sum_d P hi + N lo, however
// many heads.  A group of lanes has a head's weights (16-bit) in registers and 16 bytes of a
// record (2 D bytes) each; whole-number products, exact sums (below 2^24), one exact product
// with the block's step.  Bound by HBM: 2 D + 4 bytes per block and kv head.
template <bool BF16, int D, int QT>
__global__ void __launch_bounds__(kScoreThreads) block_scores_kernel(const SelectParams p) {
    constexpr int kLanes = 2 * D / 16;                       // lanes per record
    constexpr int kGroups = kScoreThreads / kLanes;
    __shared__ int32_t phys_s[kMaxScoreChunk];
    grid_dependency_wait();
    allow_dependent_launch();
    const int32_t s = blockIdx.x, tid = threadIdx.x;
    const int32_t len = context_of(p, s, blockIdx.y == 0 && blockIdx.z == 0 && tid == 0);
    // blocks to score: the last query token's, without the first and last ones
    const int32_t blocks = blocks_of(p, len, p.q_len - 1);
    const int32_t b0 = max((int32_t)blockIdx.y * p.chunk, p.num_first);
    const int32_t b1 = min(((int32_t)blockIdx.y + 1) * p.chunk, blocks - p.num_last);
    if (blocks <= p.num_selected || b0 >= b1) return;
    const int32_t heads = min(p.num_kv_heads, kGroups);      // kv heads of this CTA at a time
    for (int32_t i = tid; i < b1 - b0; i += kScoreThreads) {
        int32_t phys = p.block_tables[(size_t)s * p.max_blocks_per_seq + b0 + i];
        if (phys < 0 || phys >= p.num_blocks) {
            if (p.status && blockIdx.z == 0) atomicOr(p.status, kDevBadBlock);
            phys = -1;
        }
        phys_s[i] = phys;
    }
    const int32_t grp = tid / kLanes, c = tid % kLanes;
    const int32_t h = (int32_t)blockIdx.z * heads + grp % heads, sub = grp / heads, subs = kGroups / heads;
    const bool mine = sub < subs && h < p.num_kv_heads;
    const bool low = c >= kLanes / 2;                        // this lane has lower bounds
    const int32_t d0 = (c % (kLanes / 2)) * 16;
    __syncthreads();
    for (int32_t j0 = 0; j0 < p.q_len; j0 += QT) {
        int32_t w[QT][8];                                    // 16 weights, two to a register
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const int32_t j = min(j0 + t, p.q_len - 1);
            const uint4* q = reinterpret_cast<const uint4*>(
                static_cast<const uint16_t*>(p.query) +
                (((size_t)s * p.q_len + j) * p.num_q_heads + (size_t)(mine ? h : 0) * p.group) * D + d0);
            constexpr float kBig = BF16 ? 3.38953139e38f : 65504.f;
            auto dims = [&](int32_t g, float (&v)[16]) {
                const uint4 a = q[g * (D / 8)], b = q[g * (D / 8) + 1];
                const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    unpack2<BF16>(x[i], v[2 * i], v[2 * i + 1]);
                    // (NaN counts as 0, an infinity as the largest number)
                    v[2 * i] = v[2 * i] == v[2 * i] ? fminf(fmaxf(v[2 * i], -kBig), kBig) : 0.f;
                    v[2 * i + 1] = v[2 * i + 1] == v[2 * i + 1] ? fminf(fmaxf(v[2 * i + 1], -kBig), kBig) : 0.f;
                }
            };
            float most = 0.f;
            for (int32_t g = 0; g < p.group; ++g) {
                float v[16];
                dims(g, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(v[i]));
            }
#pragma unroll
            for (int o = 1; o < kLanes / 2; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            const float inv = power_of_two(5 - exponent_of(most));
            int32_t sum[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[i] = 0;
            for (int32_t g = 0; g < p.group; ++g) {
                float v[16];
                dims(g, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int32_t x = __float2int_rn(v[i] * inv);
                    sum[i] += low ? min(x, 0) : max(x, 0);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) w[t][i] = (sum[2 * i] & 0xFFFF) | (sum[2 * i + 1] << 16);
        }
        // (a warp's groups go through the batches together: its shuffles need every lane)
        for (int32_t first = 0; first < b1 - b0; first += kScoreBatch * subs) {
            uint4 x[kScoreBatch];
            // the record whose score this lane ends up with
            const int32_t u = (c / (kLanes / 4)) & 3;
            float step = 0.f;
#pragma unroll
            for (int k = 0; k < kScoreBatch; ++k) {
                const int32_t i = first + k * subs + sub;
                x[k] = make_uint4(0u, 0u, 0u, 0u);
                if (mine && i < b1 - b0 && phys_s[i] >= 0) {
                    const size_t rec = (size_t)phys_s[i] * p.num_kv_heads + h;
                    x[k] = __ldg(reinterpret_cast<const uint4*>(p.bounds + rec * 2 * D) + c);
                    if (k == u) step = __ldg(p.steps + rec);
                }
            }
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                int32_t dot[kScoreBatch];
#pragma unroll
                for (int k = 0; k < kScoreBatch; ++k) {
                    int32_t a = dp2_lo(w[t][0], (int32_t)x[k].x, 0), b = dp2_hi(w[t][1], (int32_t)x[k].x, 0);
                    a = dp2_lo(w[t][2], (int32_t)x[k].y, a);
                    b = dp2_hi(w[t][3], (int32_t)x[k].y, b);
                    a = dp2_lo(w[t][4], (int32_t)x[k].z, a);
                    b = dp2_hi(w[t][5], (int32_t)x[k].z, b);
                    a = dp2_lo(w[t][6], (int32_t)x[k].w, a);
                    b = dp2_hi(w[t][7], (int32_t)x[k].w, b);
                    dot[k] = a + b;
                }
                // the lanes' sums: half of the lanes go on with records 2, 3, then with the odd one
                constexpr int kHalf = kLanes / 2, kQuarter = kLanes / 4;
                const bool up = c & kHalf, odd = c & kQuarter;
                int32_t a = up ? dot[2] : dot[0], b = up ? dot[3] : dot[1];
                a += __shfl_xor_sync(0xffffffffu, up ? dot[0] : dot[2], kHalf);
                b += __shfl_xor_sync(0xffffffffu, up ? dot[1] : dot[3], kHalf);
                int32_t y = odd ? b : a;
                y += __shfl_xor_sync(0xffffffffu, odd ? a : b, kQuarter);
#pragma unroll
                for (int o = kQuarter / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                const int32_t i = first + u * subs + sub;
                if (mine && c % kQuarter == 0 && i < b1 - b0 && j0 + t < p.q_len) {
                    const float score = (float)y * step;
                    const uint32_t bits = __float_as_uint(score);
                    const uint32_t key = score != score ? 0xffffffffu : (bits >> 31) ? ~bits : bits | 0x80000000u;
                    p.keys[(((size_t)s * p.q_len + j0 + t) * p.num_kv_heads + h) * p.max_blocks + b0 + i] = key;
                }
            }
        }
    }
}

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

// CTA (query token, kv head): the `want` largest of its row's scores, by histograms over the
// range that still holds the smallest of them: each pass divides it by 2048, starting from the
// scores' own range, so that the counts spread.  What is taken is a bit per block, which puts
// the list in order; of equal scores the first ones are taken.  Bound by latency: about three
// passes over at most 16 keys a thread, with the scans between them.
__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(const SelectParams p) {
    extern __shared__ uint32_t sel_smem[];
    __shared__ int32_t buf[32];
    __shared__ int32_t hist[kSelBins];
    __shared__ uint32_t range[2];             // the scores' least and greatest
    __shared__ int32_t found[2];              // the bin, and the scores above it
    grid_dependency_wait();
    allow_dependent_launch();
    const int32_t tid = threadIdx.x, lane = tid & 31;
    const int64_t row = (int64_t)blockIdx.x * p.num_kv_heads + blockIdx.y;
    const int32_t s = (int32_t)(blockIdx.x / p.q_len), j = (int32_t)(blockIdx.x % p.q_len);
    const int32_t blocks = blocks_of(p, context_of(p, s, false), j);
    int32_t* out = p.selected + row * p.num_selected;
    if (blocks <= p.num_selected) {
        for (int32_t i = tid; i < p.num_selected; i += kSelThreads) out[i] = i < blocks ? i : -1;
        return;
    }
    const int32_t words = (blocks + 31) / 32;
    uint32_t* const take = sel_smem;
    uint32_t* const tie = sel_smem + (p.max_blocks + 31) / 32;
    const uint32_t* keys = p.keys + row * p.max_blocks;
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
    if (tid == 0) {
        range[0] = 0xffffffffu;
        range[1] = 0u;
    }
    __syncthreads();
    each([&](int32_t, uint32_t k) {
        lo = min(lo, k);
        hi = max(hi, k);
    });
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        atomicMin(&range[0], lo);
        atomicMax(&range[1], hi);
    }
    __syncthreads();
    lo = range[0];
    hi = range[1];
    // narrow lo .. hi until all of it is taken, or one value is left; `want` of it are
    bool all = want == 0;
    if (all) lo = hi = 0xffffffffu;               // (nothing above, nothing within)
    while (!all && lo < hi) {
        const int32_t shift = max(0, 21 - __clz(hi - lo));
        for (int32_t i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        each([&](int32_t, uint32_t k) {
            if (k >= lo && k <= hi) atomicAdd(&hist[(k - lo) >> shift], 1);
        });
        __syncthreads();
        // bins from the top: thread t has the bins that end at kSelBins - 1 - 4 t
        constexpr int kPer = kSelBins / kSelThreads;
        int32_t mine = 0, n[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            n[k] = hist[kSelBins - 1 - (tid * kPer + k)];
            mine += n[k];
        }
        int32_t total, above = scan_cta(mine, buf, &total);
        if (above < want && want <= above + mine) {
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                if (above < want && want <= above + n[k]) {
                    found[0] = kSelBins - 1 - (tid * kPer + k);
                    found[1] = above;
                }
                above += n[k];
            }
        }
        __syncthreads();
        const int32_t bin = found[0];
        want -= found[1];
        all = hist[bin] == want;
        lo += (uint32_t)bin << shift;
        hi = lo + min(hi - lo, (1u << shift) - 1u);      // (lo + a bin may pass 32 bits)
        __syncthreads();
    }
    // the bits: everything above the range, and the range itself if all of it is taken
    auto mark = [&](int32_t i, uint32_t k, bool scored) {
        const bool here = scored && k >= lo && k <= hi && !(want == 0);
        const bool in = i < blocks && (!scored || (want > 0 ? k > hi : false) || (here && all));
        const uint32_t t = __ballot_sync(0xffffffffu, in), e = __ballot_sync(0xffffffffu, here && !all);
        if (lane == 0 && (i >> 5) < words) {
            take[i >> 5] = t;
            tie[i >> 5] = e;
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
    // of the ties, the first `want`; then the list, word by word
    int32_t ties = 0, at = 0;
    for (int32_t w0 = 0; w0 < words; w0 += kSelThreads) {
        const int32_t w = w0 + tid;
        uint32_t bits = w < words ? take[w] : 0u;
        int32_t total;
        if (!all) {
            uint32_t e = w < words ? tie[w] : 0u;
            const int32_t before = ties + scan_cta(__popc(e), buf, &total);
            ties += total;
            for (int32_t left = want - before; e && left > 0; --left) {
                bits |= e & (0u - e);
                e &= e - 1u;
            }
        }
        int32_t to = at + scan_cta(__popc(bits), buf, &total);
        at += total;
        for (; bits; bits &= bits - 1u) out[to++] = 32 * w + __ffs(bits) - 1;
    }
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
    const int64_t units = (int64_t)p.num_seqs * p.slots * p.num_kv_heads;
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
    const bool one = p.q_len == 1, wide = p.head_size == 128;
    const Kern kern =
        bf16 ? (wide ? (one ? (Kern)block_scores_kernel<true, 128, 1> : (Kern)block_scores_kernel<true, 128, 4>)
                     : (one ? (Kern)block_scores_kernel<true, 64, 1> : (Kern)block_scores_kernel<true, 64, 4>))
             : (wide ? (one ? (Kern)block_scores_kernel<false, 128, 1> : (Kern)block_scores_kernel<false, 128, 4>)
                     : (one ? (Kern)block_scores_kernel<false, 64, 1> : (Kern)block_scores_kernel<false, 64, 4>));
    if (p.max_blocks > p.num_selected) {
        const int32_t groups = kScoreThreads / (2 * p.head_size / 16);
        const int32_t heads = std::min(p.num_kv_heads, groups);
        cudaError_t e = launch_pdl(dim3((unsigned)p.num_seqs, (unsigned)((p.max_blocks + p.chunk - 1) / p.chunk),
                                        (unsigned)((p.num_kv_heads + heads - 1) / heads)),
                                   dim3(kScoreThreads), 0, stream, kern, p);
        if (e != cudaSuccess) return e;
    }
    const size_t smem = 2 * sizeof(uint32_t) * (size_t)((p.max_blocks + 31) / 32);
    return launch_pdl(dim3((unsigned)(p.num_seqs * p.q_len), (unsigned)p.num_kv_heads), dim3(kSelThreads), smem,
                      stream, select_blocks_kernel, p);
}

}  // namespace pa
