// pa_chunk_aux.cu -- the kernels around the chunk attention: the plan that cuts a ragged
// batch into work items, rotary positions fused with the write into the paged pools, and
// the moving of blocks when a pool is compacted.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "pa_chunk_device.cuh"
#include "pa_device.cuh"

namespace pa {

namespace {

constexpr int32_t kBadSlot = 1, kBadBlock = 2, kBadLen = 4;

// Block-wide exclusive scan of x over blockDim.x (a multiple of 32) threads; *total
// receives the sum.  `buf` holds 32 ints of shared memory.
__device__ __forceinline__ int32_t block_scan(int32_t x, int32_t* buf, int32_t* total) {
    const int32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int32_t v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) buf[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int32_t w = lane < nw ? buf[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        buf[lane] = w;
    }
    __syncthreads();
    const int32_t excl = (warp > 0 ? buf[warp - 1] : 0) + v - x;
    *total = buf[31];
    __syncthreads();
    return excl;
}

constexpr int kPlanThreads = 512;
constexpr int kBuckets = 256;
// Batches up to these sizes keep what the plan's passes read again in shared memory.
constexpr int kPlanSeqs = 512, kPlanTiles = 2048;

// Lists the row tiles of a ragged batch and settles how the attention kernel shares them
// out (see PfHeader).  Whole units are claimed longest first, which leaves the shortest for
// the end.  Where that would still leave the longest CTA over an equal share by more than
// what joining partial results costs (few or long units), the work is cut into equal shares
// instead, whatever the units' ends.  Both sides, whole / cut (us a call, calls back to back;
// 32 query and 8 kv heads of 128, bf16, 16-token blocks): prompts of 2048, 4096 and 8192 tokens
// 48 / 54, 106 / 126 and 360 / 411; chunks of 640 and 760 beside 61 single tokens, all behind
// 200-4000, 126 / 156; 16 chunks of 200 behind 1 K 76 / 91; 2 of 700 behind 4 K 112 / 88; 1 of
// 512 behind 16 K 192 / 110; 8 of 64 behind 8 K 104 / 79; 40 of 32 behind 8 K 264 / 230; 64
// query heads, 4 chunks of 24 behind 50-62 K 665 / 190.  The rule takes the better side of each
// of these.  It looks at the first four rounds of units only, so a short fifth one goes unseen:
// 77 chunks of 32 behind 8 K (616 units on 152 CTAs) are taken whole, 448 / 417.
__global__ void __launch_bounds__(kPlanThreads) prefill_plan_kernel(const PrefillParams p) {
    __shared__ int32_t buf[32];
    __shared__ int32_t hist[kBuckets], first[kBuckets];
    __shared__ int32_t longest, whole;
    __shared__ int4 seq_s[kPlanSeqs];
    __shared__ int32_t tiles_s[kPlanTiles];
    allow_dependent_launch();
    grid_dependency_wait();
    const int32_t tid = threadIdx.x, span = 2 * p.tpt;
    if (tid < kBuckets) hist[tid] = 0;
    if (tid == 0) longest = whole = 0;
    // the sequences: chunk, context, first row tile; bad metadata is clamped and reported
    int32_t row_tiles = 0;
    for (int32_t base = 0; base < p.num_seqs; base += kPlanThreads) {
        const int32_t s = base + tid;
        const PfChunk c = chunk_of(p, s, true);
        int32_t sum;
        const int32_t at = row_tiles + block_scan(c.row_tiles, buf, &sum);
        if (s < p.num_seqs) {
            const int4 q = make_int4(c.start, c.count, c.len, at);
            p.seqs[s] = q;
            if (s < kPlanSeqs) seq_s[s] = q;
        }
        // chunks that overlap could ask for more row tiles than there is room for
        row_tiles = min(row_tiles + sum, p.max_row_tiles + 1);
    }
    if (row_tiles > p.max_row_tiles) {
        if (tid == 0 && p.status) atomicOr(p.status, kBadLen);
        row_tiles = p.max_row_tiles;
    }
    __syncthreads();
    // row tile i: its sequence (the last whose first row tile is at or before i), and the
    // tiles it needs, up to the last token its last row sees
    auto seq_at = [&](int32_t s) { return p.num_seqs <= kPlanSeqs ? seq_s[s] : p.seqs[s]; };
    auto tiles_of = [&](int32_t i, int32_t s) {
        const int4 q = seq_at(s);
        const int32_t last = min((i - q.w + 1) * span, q.y);
        return (max(q.z - q.y + last, 0) + kPfTok - 1) / kPfTok;
    };
    long long cost = 0;
    for (int32_t base = 0; base < row_tiles; base += kPlanThreads) {
        const int32_t i = base + tid;
        int32_t n = 0;
        if (i < row_tiles) {
            int32_t a = 0, b = p.num_seqs;
            while (b - a > 1) {
                const int32_t m = (a + b) >> 1;
                if (seq_at(m).w <= i) a = m;
                else b = m;
            }
            p.seq_of[i] = a;
            n = tiles_of(i, a);
            if (i < kPlanTiles) tiles_s[i] = n;
            if (n > 0) atomicMax(&longest, n);
            n += kPfItemCost;
        }
        int32_t sum;      // (512 row tiles of at most 2^21 each; a longer context counts as that)
        const int32_t at = block_scan(min(n, 1 << 21), buf, &sum);
        if (i < row_tiles) p.before[i] = cost + at;
        cost += sum;
    }
    if (tid == 0) p.before[row_tiles] = cost;
    __syncthreads();
    const long long units = (long long)row_tiles * p.num_kv_heads, all = cost * p.num_kv_heads;
    // shares: all CTAs, unless that makes them too short to be worth it
    const long long shares = max(1ll, min((long long)p.grid, max(units, all / kPfMinShare)));
    // Row tiles by length, longest first, and from that what whole units would take: with m
    // CTAs some CTA gets j of the first (j - 1) m + 1 units, all at least as long as the last.
    const int32_t scale = longest + 1;
    auto tiles_at = [&](int32_t i) { return i < kPlanTiles ? tiles_s[i] : tiles_of(i, p.seq_of[i]); };
    auto bucket = [&](int32_t n) {
        return kBuckets - 1 - min(kBuckets - 1, (int32_t)((int64_t)n * kBuckets / scale));
    };
    for (int32_t i = tid; i < row_tiles; i += kPlanThreads) atomicAdd(&hist[bucket(tiles_at(i))], 1);
    __syncthreads();
    {
        int32_t sum;
        const int32_t h = tid < kBuckets ? hist[tid] : 0;
        const int32_t at = block_scan(h, buf, &sum);
        if (tid < kBuckets) {
            first[tid] = at;
            const int32_t most = (int32_t)(((int64_t)(kBuckets - tid) * scale + kBuckets - 1) / kBuckets) - 1;
            for (int32_t j = 1; j <= 4; ++j) {
                const long long k = (long long)(j - 1) * p.grid;
                if ((long long)at * p.num_kv_heads <= k && k < (long long)(at + h) * p.num_kv_heads)
                    atomicMax(&whole, j * (min(most, longest) + kPfItemCost));
            }
        }
        __syncthreads();
    }
    const bool cut = longest > 1 && (whole - kPfCutCost) * shares > all;
    // Trees of more than one row tile behind long contexts: two row tiles of a sequence read the same
    // K and V, and laid end to end they would read it far apart in time, from memory both times.  So
    // two neighbouring CTAs take the shares of a pair of row tiles, each its own, and keep in step:
    // the second read comes from L2.  (A row tile left over leaves a CTA idle meanwhile; pairs are
    // taken where that costs no more than a tenth.)  4 trees of 50-63 tokens, 8 heads to a kv head,
    // behind 56-60 K: 370 us end to end, 330 in pairs; 415 and 361-380 at the power cap.
    long long paired = 0;
    int32_t lines = row_tiles;
    auto pair_cost = [&](int32_t i) {          // of the pair that begins at row tile i, 0: none does
        if (i >= row_tiles) return 0;
        const int32_t s = p.seq_of[i];
        if ((i - seq_at(s).w) & 1) return 0;
        const bool two = i + 1 < row_tiles && p.seq_of[i + 1] == s;
        return min(tiles_of(two ? i + 1 : i, s) + kPfItemCost, 1 << 21);
    };
    if (cut && p.tree_mask && p.grid > 1) {
        __syncthreads();                       // seq_of
        for (int32_t base = 0; base < row_tiles; base += kPlanThreads) {
            int32_t sum;
            (void)block_scan(pair_cost(base + tid), buf, &sum);
            paired += sum;
        }
    }
    const bool pairs = paired > 0 && 20 * paired <= 11 * cost;
    if (pairs) {
        long long before = 0;
        lines = 0;
        for (int32_t base = 0; base < row_tiles; base += kPlanThreads) {
            const int32_t i = base + tid, n = pair_cost(i);
            int32_t sum, count;
            const int32_t at = block_scan(n, buf, &sum);
            const int32_t place = lines + block_scan(n > 0 ? 1 : 0, buf, &count);
            if (n > 0) {
                p.before[place] = before + at;
                p.order[place] = i;
            }
            before += sum;
            lines += count;
        }
        if (tid == 0) p.before[lines] = before;
    }
    if (!cut) {
        for (int32_t i = tid; i < row_tiles; i += kPlanThreads)
            p.order[atomicAdd(&first[bucket(tiles_at(i))], 1)] = i;
    } else {
        for (int32_t i = tid; i < 2 * p.grid; i += kPlanThreads) p.arrive[i] = 0;
    }
    if (tid == 0) {
        p.hdr->counter = 0;
        p.hdr->total_units = (uint32_t)units;
        p.hdr->cut = cut ? 1 : 0;
        const long long cost2 = paired * p.num_kv_heads, units2 = (long long)lines * p.num_kv_heads;
        p.hdr->shares = (uint32_t)(pairs ? max(1ll, min(p.grid / 2ll, max(units2, cost2 / kPfMinShare))) : shares);
        p.hdr->cost = pairs ? cost2 : all;
        p.hdr->lines = (uint32_t)lines;
        p.hdr->pairs = pairs ? 1 : 0;
    }
}

// ------------------------------------------------------------------ rotary + cache write
// Threads per token and 32-byte units a thread has in flight.  8200 tokens of 32 + 8 heads of
// 128 (202 MB moved, slots at random): 64 threads with 2 units 34.7 us, 128 with 4 41, 32
// with 3 36.7, against 30.1 us at the measured copy bandwidth.  More threads leave fewer
// tokens per SM to cover the wait for a token's positions and angles.
constexpr int kRopeThreads = 64;
constexpr int kRopeUnits = 2;

// A position's step in turns, as a 64-bit fraction: inv_freq / 2 pi modulo 1.  inv_freq is
// m 2^e with an integer m below 2^24; m times the first 96 bits of 1 / 2 pi is shifted into
// place.  Within 2^-64 of a turn (|inv_freq| < 2^24).
__device__ __forceinline__ unsigned long long turn_step(float inv_freq) {
    const uint32_t bits = __float_as_uint(inv_freq), ex = (bits >> 23) & 255u;
    const uint32_t m = ex ? (bits & 0x7FFFFFu) | 0x800000u : bits & 0x7FFFFFu;
    const int32_t shift = 32 + 150 - (int32_t)(ex ? ex : 1u);      // of the product, to the right
    const unsigned long long p0 = (unsigned long long)m * 0x7F09D5F4u;
    const unsigned long long p1 = (unsigned long long)m * 0x9391054Au + (p0 >> 32);
    const unsigned long long p2 = (unsigned long long)m * 0x28BE60DBu + (p1 >> 32);
    // words of the product, lowest first: (uint32)p0, (uint32)p1, p2 (two words)
    const unsigned long long low = (p1 << 32) | (uint32_t)p0, high = p2;
    unsigned long long f;
    if (shift >= 128) f = 0;
    else if (shift >= 64) f = high >> (shift - 64);
    else if (shift > 0) f = (high << (64 - shift)) | (low >> shift);
    else f = low << (-shift & 63);
    return (bits >> 31) ? 0ull - f : f;
}

// Rotates the query and key rows of new tokens and writes K and V into the pools.
//
// Pair i of a row turns by the angle positions[axis(i)][token] * inv_freq[i].  In turns,
// that product is taken in 64-bit fixed point: the step is a 64-bit fraction of a turn, its
// product with the integer position wraps modulo one turn exactly, and what is left is
// rounded once, to fp32, so that far positions lose nothing: 2^31 steps are off by 2^-33
// turns.
//
// A CTA takes a token.  Its rows are cut into 32-byte units (two 16-byte pieces: 8 pairs,
// or 16 dimensions that do not turn), and a thread has the same unit of every few heads, so
// that its pairs' cosines and sines are read once; the first heads' units are on their way
// while those are computed, one thread per pair, into shared memory.
template <bool BF16, bool KV8>
__global__ void __launch_bounds__(kRopeThreads) rope_and_cache_kernel(const RopeParams p) {
    __shared__ __align__(16) float2 turn[kMaxRopePairs];
    allow_dependent_launch();   // what follows waits for this kernel before it reads the pools
    grid_dependency_wait();
    const int64_t i = blockIdx.x;
    const int32_t half = p.rot_dim / 2, tid = threadIdx.x;
    int32_t slot = p.slot_mapping[i];
    if ((int64_t)slot >= (int64_t)p.num_blocks * p.block_size) {
        if (tid == 0 && p.status) atomicOr(p.status, kBadSlot);
        slot = -1;
    }
    const int64_t block = slot / p.block_size, offset = slot - block * p.block_size;
    const int32_t units = p.head_size / 16, hq = p.num_q_heads, hk = p.num_kv_heads;
    // this thread's unit c of heads h0, h0 + step, ..: first the query's, then the key's and
    // the value's (a padding token's are not written)
    const int32_t step = kRopeThreads / units, h0 = tid / units, c = tid - h0 * units;
    const int32_t heads = h0 < step ? (slot < 0 ? hq : hq + 2 * hk) : 0;
    const bool turns = c < p.rot_dim / 16, apart = turns && !p.interleaved;
    struct Place {
        int32_t kind, head;      // 0 query, 1 key, 2 value
        int32_t d0, d1;          // first dimensions of the unit's pieces
    };
    auto place = [&](int32_t h) {
        Place q;
        q.kind = h < hq ? 0 : h < hq + hk ? 1 : 2;
        q.head = q.kind == 0 ? h : q.kind == 1 ? h - hq : h - hq - hk;
        const bool a = apart && q.kind != 2;
        q.d0 = a ? 8 * c : 16 * c;
        q.d1 = a ? half + 8 * c : 16 * c + 8;
        return q;
    };
    uint4 xa[kRopeUnits], xb[kRopeUnits];
    auto load = [&](int32_t first) {
#pragma unroll
        for (int k = 0; k < kRopeUnits; ++k) {
            const int32_t h = first + k * step;
            if (h >= heads) break;
            const Place q = place(h);
            const uint16_t* src = q.kind == 0   ? static_cast<const uint16_t*>(p.query) + i * p.q_stride
                                  : q.kind == 1 ? static_cast<const uint16_t*>(p.key) + i * p.k_stride
                                                : static_cast<const uint16_t*>(p.value) + i * p.v_stride;
            src += q.head * p.head_size;
            xa[k] = *reinterpret_cast<const uint4*>(src + q.d0);
            xb[k] = *reinterpret_cast<const uint4*>(src + q.d1);
        }
    };
    load(h0);
    for (int32_t e = tid; e < half; e += kRopeThreads) {
        const unsigned long long pos = (unsigned long long)p.positions[(int64_t)p.axis[e] * p.num_tokens + i];
        // the upper half, as a signed number of half turns in [-1, 1)
        const float x = (float)(int32_t)((turn_step(p.inv_freq[e]) * pos) >> 32) * 4.656612873077392578125e-10f;
        float sn, cs;
        sincospif(x, &sn, &cs);
        turn[e] = make_float2(cs, sn);
    }
    __syncthreads();
    float4 w[4];                 // (cos, sin) of this thread's eight pairs
    if (turns) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = reinterpret_cast<const float4*>(&turn[8 * c])[j];
    }
    for (int32_t first = h0; first < heads; first += kRopeUnits * step) {
        if (first != h0) load(first);
#pragma unroll
        for (int k = 0; k < kRopeUnits; ++k) {
            const int32_t h = first + k * step;
            if (h >= heads) break;
            const Place q = place(h);
            const bool rot = turns && q.kind != 2;
            uint4 ya = xa[k], yb = xb[k];      // a unit that does not turn goes out as it came in
            float a[8], b[8];
            if (rot || (KV8 && q.kind != 0)) {
                const uint32_t wa[4] = {xa[k].x, xa[k].y, xa[k].z, xa[k].w};
                const uint32_t wb[4] = {xb[k].x, xb[k].y, xb[k].z, xb[k].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    unpack2<BF16>(wa[j], a[2 * j], a[2 * j + 1]);
                    unpack2<BF16>(wb[j], b[2 * j], b[2 * j + 1]);
                }
            }
            if (rot) {
                if (!p.interleaved) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = a[2 * j], y = b[2 * j], z = a[2 * j + 1], v = b[2 * j + 1];
                        a[2 * j] = x * w[j].x - y * w[j].y;
                        b[2 * j] = x * w[j].y + y * w[j].x;
                        a[2 * j + 1] = z * w[j].z - v * w[j].w;
                        b[2 * j + 1] = z * w[j].w + v * w[j].z;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float* r = j < 2 ? a + 4 * j : b + 4 * (j - 2);
                        const float x = r[0], y = r[1], z = r[2], v = r[3];
                        r[0] = x * w[j].x - y * w[j].y;
                        r[1] = x * w[j].y + y * w[j].x;
                        r[2] = z * w[j].z - v * w[j].w;
                        r[3] = z * w[j].w + v * w[j].z;
                    }
                }
                ya = make_uint4(pack2<BF16>(a[0], a[1]), pack2<BF16>(a[2], a[3]), pack2<BF16>(a[4], a[5]),
                                pack2<BF16>(a[6], a[7]));
                yb = make_uint4(pack2<BF16>(b[0], b[1]), pack2<BF16>(b[2], b[3]), pack2<BF16>(b[4], b[5]),
                                pack2<BF16>(b[6], b[7]));
            }
            const int64_t row = q.kind == 0 ? i * hq + q.head : (block * hk + q.head) * p.block_size + offset;
            if (KV8 && q.kind != 0) {
                // e4m3(x * (1 / scale)): fp32 product, nearest-even, saturated
                uint8_t* dst = static_cast<uint8_t*>(q.kind == 1 ? p.key_cache : p.value_cache) + row * p.head_size;
                const float inv = q.kind == 1 ? p.k_inv : p.v_inv;
                uint32_t qa[4], qb[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    qa[j] = f32x2_to_e4m3x2(__fmul_rn(a[2 * j], inv), __fmul_rn(a[2 * j + 1], inv));
                    qb[j] = f32x2_to_e4m3x2(__fmul_rn(b[2 * j], inv), __fmul_rn(b[2 * j + 1], inv));
                }
                *reinterpret_cast<uint2*>(dst + q.d0) = make_uint2(qa[0] | (qa[1] << 16), qa[2] | (qa[3] << 16));
                *reinterpret_cast<uint2*>(dst + q.d1) = make_uint2(qb[0] | (qb[1] << 16), qb[2] | (qb[3] << 16));
            } else {
                uint16_t* dst =
                    static_cast<uint16_t*>(q.kind == 0 ? p.query_out : q.kind == 1 ? p.key_cache : p.value_cache) +
                    row * p.head_size;
                *reinterpret_cast<uint4*>(dst + q.d0) = ya;
                *reinterpret_cast<uint4*>(dst + q.d1) = yb;
            }
        }
    }
}

// ------------------------------------------------------------------ block moves
constexpr int kMoveThreads = 256;
constexpr int kMoveTableCtas = 8;

// Copies block `from` to block `to` in both pools of every layer, and rewrites the block
// tables' entries.  CTA (i, y): pair i of pool y (2 * layer, + 1 for V), or, past the
// pairs and for y = 0, a share of the table entries: each entry looks itself up among the
// pairs, which ascend by `from`.  Bound by HBM: 201 blocks of 32 KB in both pools of 32 layers
// (843 MB read and written) take 123.5 us, 6.83 TB/s; every CTA has 32 KB on their way.
__global__ void __launch_bounds__(kMoveThreads) move_blocks_kernel(const __grid_constant__ MoveParams p) {
    const int32_t i = blockIdx.x;
    if (i >= p.num_pairs) {
        if (blockIdx.y != 0 || !p.block_tables) return;
        for (int64_t e = (int64_t)(i - p.num_pairs) * kMoveThreads + threadIdx.x; e < p.num_entries;
             e += (int64_t)kMoveTableCtas * kMoveThreads) {
            const int32_t b = p.block_tables[e];
            if (b < 0 || b >= p.num_blocks) continue;
            int32_t lo = 0, hi = p.num_pairs;
            while (lo < hi) {
                const int32_t m = (lo + hi) >> 1;
                if (p.pairs[2 * m] < b) lo = m + 1;
                else hi = m;
            }
            if (lo < p.num_pairs && p.pairs[2 * lo] == b) {
                const int32_t to = p.pairs[2 * lo + 1];
                if (to >= 0 && to < p.num_blocks) p.block_tables[e] = to;
            }
        }
        return;
    }
    const int32_t from = p.pairs[2 * i], to = p.pairs[2 * i + 1];
    const bool bad = from < 0 || from >= p.num_blocks || to < 0 || to >= p.num_blocks;
    if (p.report && blockIdx.y == 0 && threadIdx.x == 0 && p.status &&
        (bad || (i > 0 && p.pairs[2 * i - 2] >= from)))
        atomicOr(p.status, kBadBlock);
    const int32_t layer = blockIdx.y >> 1;
    if (bad || layer >= p.num_layers) return;
    uint4* const pool = static_cast<uint4*>((blockIdx.y & 1) ? p.value[layer] : p.key[layer]);
    const uint4* src = pool + (int64_t)from * p.vecs_per_block;
    uint4* dst = pool + (int64_t)to * p.vecs_per_block;
    int64_t e = threadIdx.x;
    // eight 16-byte loads in flight per thread
    for (; e + 7 * kMoveThreads < p.vecs_per_block; e += 8 * kMoveThreads) {
        uint4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = __ldcs(src + e + k * kMoveThreads);
#pragma unroll
        for (int k = 0; k < 8; ++k) __stcs(dst + e + k * kMoveThreads, x[k]);
    }
    for (; e < p.vecs_per_block; e += kMoveThreads) dst[e] = src[e];
}

// Launches `kern` as a programmatic dependent of the kernel before it on `stream`.
template <class Arg>
cudaError_t launch_pdl(dim3 grid, dim3 block, cudaStream_t stream, void (*kern)(Arg), const Arg& arg) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, arg);
}

}  // namespace

cudaError_t launch_prefill_plan(const PrefillParams& p, cudaStream_t stream) {
    return launch_pdl<PrefillParams>(dim3(1), dim3(kPlanThreads), stream,
                                     prefill_plan_kernel, p);
}

cudaError_t launch_rope_and_cache(const RopeParams& p, bool bf16, bool kv8, cudaStream_t stream) {
    if (p.num_tokens <= 0) return cudaSuccess;
    using Kern = void (*)(RopeParams);
    const Kern kern = kv8 ? (bf16 ? (Kern)rope_and_cache_kernel<true, true> : (Kern)rope_and_cache_kernel<false, true>)
                          : (bf16 ? (Kern)rope_and_cache_kernel<true, false> : (Kern)rope_and_cache_kernel<false, false>);
    return launch_pdl<RopeParams>(dim3((unsigned)p.num_tokens), dim3(kRopeThreads), stream, kern, p);
}

cudaError_t launch_move_blocks(const MoveParams& p, cudaStream_t stream) {
    // An ordinary launch: the tables it rewrites may be read early by a kernel after it.
    move_blocks_kernel<<<dim3((unsigned)p.num_pairs + (p.block_tables ? kMoveTableCtas : 0u),
                              (unsigned)std::max(2 * p.num_layers, 1)),
                         kMoveThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pa
