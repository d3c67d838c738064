// pa_prefill.cuh -- attention of a ragged chunk of new tokens over the paged cache, on the
// 5th-generation tensor cores (tcgen05, tensor memory).
//
// What it computes: sequence s brings C_s new tokens (rows query_starts[s] ..
// query_starts[s+1]-1 of query and out), already in the pools; token j of them sits at
// position L_s - C_s + j and attends to every token before and at it:
//     out[i][h] = sum_t softmax_t(scale q[i][h] . k_t) v_t,   t < L_s - C_s + j + 1.
//
// One work item is (row tile, kv head, partition of the context).  A row tile is two
// streams of 128 query rows each; row r of a stream is new token r / group and query head
// kvh * group + r % group, so that the heads of a group share every K/V tile.  Per tile of
// 128 tokens and stream:
//     S = Q K^T   M = 128 rows, N = 128 tokens, Q and K in shared memory, S in tensor memory
//     P = 2^(S scale - ref)  two threads per row, written back over S as 16-bit pairs
//     O += P V    M = 128 rows, N = head dims, P read from tensor memory, V MN-major
// The MMA thread issues PV of one stream and its next QK^T back to back, stream by stream,
// so the tensor pipe works on one stream while the other's softmax runs.  A row's
// reference moves (and O is rescaled in tensor memory) only when 64 of its weights add up to
// 2^8 times the weight of the score that set it: this is seen on the sum, which is needed
// anyway, held in fp32, and takes no maximum.
//
// Weights enter PV as one 16-bit term: rounding them costs at most half a step of the
// 16-bit type relative to each weight (2^-8 bf16, 2^-11 fp16), as much as rounding the
// output itself; a second term would cost half of PV's matrix rate again.  fp16 weights are
// taken 2^7 larger, up to 2^15: what is lost below fp16's normal range is then at most
// 2^-32 of the row's largest weight per token, so that a long tail of small weights behind
// one large one is not rounded away.
//
// Rows must not see what they are masked from, and a weight of 0 times an infinite or NaN
// value would be NaN.  Only tiles that some row sees in part can hold such values; there
// the fixing warps zero the V rows past the context, replace non-finite V elements by 0,
// and note for each head dim the first token with +inf, -inf and NaN; the rows that do see
// that token get the value added at the end.
//
// Elsewhere an infinite value goes through the product, or through the join of partitions,
// with a weight that may have vanished in its type: 0 times infinity is NaN, where the weight
// of the formula is never 0.  An output element that is NaN while its row's weights are not is
// therefore settled from V itself, by a second look at the rows that the token sees; outputs
// are only checked for that otherwise (nine prompts of head size 64: 51.0-51.8 us, 49.4-49.7
// without the check and what it leads to; other cases within 0.5 %).
//
// Warps: 0-7 and 8-15 softmax and epilogue of streams 0 and 1, two threads per row; 16
// producer (claims items, TMA of Q and K); 17 MMA issuer; 18 TMA of V; 19 waits for tiles;
// 20-23 fix V tiles (16-bit caches), or widen the fp8 K/V tiles to fp16 and fix them.  Every
// wait is bounded; the warps of a stream decide together whether to stop.
//
// What bounds it, and what it measured.  Long prompts: the tensor pipe.  A pair of tiles is
// 2,048 cycles of products and takes about 2,740 (issue gaps at the streams' turns); 8192
// tokens of 32 query and 8 kv heads of 128, bf16, take 345 us (1,590 TFLOP/s) until the power
// cap sets in and 360-371 back to back.  Few new tokens behind long contexts (4 x 24 tokens, 64
// heads, 50-62 K): 190-200 us, 4.5-4.8 TB/s, at the power cap too; 256 single tokens behind
// 200-4000: 342 us, 6.2 TB/s of K/V.  Head size 64: neither pipe is full (products 23 % of the
// cycles, exponentials 24 %, issue slots 48 %); a pair of tiles with 1,024 cycles of products and
// as many of exponentials takes 2,500, the softmax warps' own chain of wait, load, weights, store
// and arrival: 51 us for nine prompts of 40-1500 tokens with 16 heads, 292 for one of 8192 with
// 32.  fp8 caches: the widening, 1,300 cycles a tile for its four warps, and the lead that three
// stages leave (365 us where fp16 products alone take 211); single tokens pay it in full: the
// 256 take 402 us, more than over a 16-bit cache.
#pragma once

#include "pa_chunk_device.cuh"
#include "pa_decode.cuh"

namespace pa {
namespace pf {

constexpr int kWarpLoad = 16, kWarpMma = 17, kWarpLoadV = 18, kWarpReady = 19, kWarpFix0 = 20;
constexpr int kThreads = 768;
constexpr int kStreamThreads = 256;    // two warpgroups of softmax per stream
// Named barriers: 1-8 the two warps that share 32 rows, 9 and 10 the warps of a stream
constexpr int kBarRows = 1, kBarStream = 9;
constexpr int32_t kNoToken = 0x7fffffff;
// Longest context that is looked at again for infinite values: with one at its end, a call over
// a context of 60 K tokens takes 6 ms and one of 2^22 tokens 0.42 s, and waits run out after 2 s.
constexpr int32_t kSettleTokens = 1 << 22;
// Registers per thread: 80 at launch, re-divided among the six warpgroups.
constexpr int kRegLaunch = 80, kRegSoft = 88, kRegAux = 72, kRegFix = 56;
static_assert(4 * kRegSoft + kRegAux + kRegFix <= 6 * kRegLaunch, "register split");

// BF16: type of the MMA operands (fp16 for fp8 caches); QBF16: type of query and out.
template <bool BF16_, bool QBF16_, int D_, int BS_, bool KV8_>
struct Cfg {
    static constexpr bool kBf16 = BF16_, kQBf16 = QBF16_, kKv8 = KV8_;
    static constexpr int D = D_, BS = BS_;
    static constexpr int BLOCKS = kPfTok / BS_;
    static constexpr int HALVES = D_ / 64;                   // 128-byte swizzle spans per row
    static constexpr uint32_t HALF = kPfTok * 128;           // one span of 128 rows
    static constexpr uint32_t TILE = HALVES * HALF;          // a 16-bit tile of K, V or Q
    static constexpr uint32_t TILE8 = kPfTok * 128;          // an fp8 tile (head_size 128)
    // K and V tiles alternate in one ring, as large as shared memory admits
    static constexpr int NST = KV8_ ? 3 : (D_ == 128 ? 4 : 8);
    static constexpr int N8 = KV8_ ? 3 : 0;                  // fp8 tiles on their way
    static constexpr uint32_t COL_S = 0, COL_O = 2 * kPfTok; // tensor-memory columns
    // log2 of the weight of the score that sets a reference, and the sum of 64 weights that
    // moves it (2^8 of those): no weight is larger
    static constexpr float kLift = BF16_ ? 0.f : 7.f, kMost = BF16_ ? 256.f : 32768.f;
    static_assert(!KV8_ || (D_ == 128 && !BF16_), "fp8 tiles are widened to fp16");
};

struct Unit {
    int32_t seq;          // -1: no more items
    int32_t kvh, len, q_start, q_len, tok0, tile0;
    int32_t cnt[2];       // tiles each stream takes
    int32_t nt;           // tiles of the item
    int32_t both;         // the streams share the first one's rows and take turns at the tiles
    int32_t single;       // the unit has rows for one stream only
    int32_t fix0;         // tiles at or past this one (within the item) are fixed
    int32_t nparts, part; // the unit's partitions, and which of them this is
    int32_t first;        // the share (CTA) that holds partition 0
};

template <class C>
struct alignas(1024) Smem {
    uint8_t q[2][C::TILE];
    uint8_t kv[C::NST][C::TILE];
    uint8_t kv8[C::N8 ? C::N8 : 1][C::N8 ? C::TILE8 : 16];
    // A tile lands on kv_full; a V tile of a 16-bit cache that has to be fixed lands on
    // kv_raw, and the fixing warps arrive on kv_fixed.  Each of the three counts only its
    // own tiles of the stage: a warp that skips tiles could not tell a barrier two phases
    // behind from one that is ready.
    uint64_t kv_full[C::NST], kv_raw[C::NST], kv_fixed[C::NST], kv_empty[C::NST];
    uint64_t kv8_full[C::N8 ? C::N8 : 1], kv8_empty[C::N8 ? C::N8 : 1];
    uint64_t q_full, q_ready, q_empty, item_ready, k_ready;
    uint64_t s_full[2], p_full[2], o_full[2], o_free[2];
    uint64_t x_full[2], x_again[2];    // by item parity: streams that share rows meet
    float red[2][2][kPfRows];          // [stream][half][row]: maxima
    // by item parity: weight sums [stream][half][row] and references
    float xsum[2][2][2][kPfRows], xref[2][2][kPfRows];
    uint64_t u_full[2], u_empty[2], drain;
    Unit unit[2];
    // first token with +inf / -inf / NaN of each head dim among an item's fixed tiles
    int32_t nonfinite[2][3][C::D];
    int32_t any_nonfinite[2];
    int32_t last_part[2], last_seq[2];
    uint32_t tmem_base;
    volatile int32_t abort;
};

template <class C>
constexpr size_t smem_bytes() {
    return sizeof(Smem<C>) + 1024;
}

// The lower and upper words of a shared-memory descriptor of 128-byte swizzled rows.  The
// upper one is a constant and the steps of a product change only the lower one, which keeps
// the issue loop short: the tensor pipe takes a product step every 64 cycles.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
    return ((saddr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

// D (TMEM) (+)= A (shared) x B (shared); one thread issues it.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}
// D (TMEM) (+)= A (TMEM) x B (shared).
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}

// True in one lane of the (converged) warp, always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// Two fp32 values per instruction (the .x2 forms of sm_100 and later).
__device__ __forceinline__ uint64_t pack_f32(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack_f32(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 32 consecutive 32-bit tensor-memory columns of this thread's lane (no wait).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// Waits for this thread's tensor-memory loads; x, loaded before, is not used before that.
__device__ __forceinline__ void tmem_arrived(float (&x)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]),
                   "+f"(x[5]), "+f"(x[6]), "+f"(x[7]), "+f"(x[8]), "+f"(x[9]),
                   "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]),
                   "+f"(x[15]), "+f"(x[16]), "+f"(x[17]), "+f"(x[18]), "+f"(x[19]),
                   "+f"(x[20]), "+f"(x[21]), "+f"(x[22]), "+f"(x[23]), "+f"(x[24]),
                   "+f"(x[25]), "+f"(x[26]), "+f"(x[27]), "+f"(x[28]), "+f"(x[29]),
                   "+f"(x[30]), "+f"(x[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
    tmem_wait_ld();
    return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(v))
                 : "memory");
    tmem_wait_st();
}

// 3-D tiled TMA load (Q: head dims, heads, tokens).
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int32_t x, int32_t y,
                                            int32_t z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_2d_keep(void* dst, const CUtensorMap* map, int32_t x,
                                                 int32_t y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// Eight 32-bit words to global memory, 32-byte aligned.
__device__ __forceinline__ void st_v8(void* dst, const uint32_t (&y)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(y[0]), "r"(y[1]),
                 "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                 : "memory");
}

// Is either of the two 16-bit values infinite or NaN?  x * 0 is NaN for exactly those, and
// stays so in the half of acc that it is added to.
template <bool kBf16>
__device__ __forceinline__ uint32_t taint(uint32_t acc, uint32_t x) {
    uint32_t r;
    if constexpr (kBf16)
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
    else
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
    return r;
}

// Which of the 16 values at `at` (16-byte aligned) are infinite or NaN: bit c of `inf` is
// +inf, bit 16 + c -inf, bit c of `nan` NaN.
template <bool kBf16>
__device__ __forceinline__ void odd_values(const uint16_t* at, uint32_t& inf, uint32_t& nan) {
    constexpr uint32_t kExp = kBf16 ? 0x7F80u : 0x7C00u;
    uint32_t acc = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 x = reinterpret_cast<const uint4*>(at)[i];
        acc = taint<kBf16>(acc, x.x);
        acc = taint<kBf16>(acc, x.y);
        acc = taint<kBf16>(acc, x.z);
        acc = taint<kBf16>(acc, x.w);
    }
    if ((acc & kExp) != kExp && ((acc >> 16) & kExp) != kExp) return;
#pragma unroll 1
    for (int c = 0; c < 16; ++c) {
        const uint32_t v = at[c];
        if ((v & 0x7FFFu) == kExp) inf |= 1u << (c + ((v >> 15) ? 16 : 0));
        else if ((v & kExp) == kExp) nan |= 1u << c;
    }
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const PrefillParams p) {
    extern __shared__ uint8_t smem_raw[];
    Smem<C>& sm = *reinterpret_cast<Smem<C>*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int D = C::D;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NST; ++i) {
            mbar_init(&sm.kv_full[i], C::kKv8 ? 4 : 1);   // the widening warps, or TMA
            mbar_init(&sm.kv_empty[i], 1);
            mbar_init(&sm.kv_raw[i], 1);
            mbar_init(&sm.kv_fixed[i], 4);
        }
        for (int i = 0; i < C::N8; ++i) {
            mbar_init(&sm.kv8_full[i], 1);
            mbar_init(&sm.kv8_empty[i], 4);
        }
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_ready, 4);
        mbar_init(&sm.q_empty, 1);
        mbar_init(&sm.item_ready, 1);
        mbar_init(&sm.k_ready, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i], 9);     // 8 softmax warps and the readiness warp
            mbar_init(&sm.o_full[i], 1);
            mbar_init(&sm.o_free[i], 16);    // 8 warps twice, or 16
            mbar_init(&sm.x_full[i], 16);
            mbar_init(&sm.x_again[i], 16);
            mbar_init(&sm.u_full[i], 1);
            mbar_init(&sm.u_empty[i], 23);   // V, MMA, readiness, 16 softmax warps, 4 fixing warps
            sm.any_nonfinite[i] = 1;         // the producer clears the tables first
        }
        mbar_init(&sm.drain, 1);
        sm.abort = 0;
        fence_barrier_init();
        prefetch_tensor_map(&qmap);
        prefetch_tensor_map(&kmap);
        prefetch_tensor_map(&vmap);
    }
    if (warp == kWarpMma) {
        tmem_alloc(&sm.tmem_base, 512);
        tmem_relinquish();
    }
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tmem = sm.tmem_base;
    grid_dependency_wait();   // the plan kernel, and with it everything before it, has finished

    const int32_t Hkv = p.num_kv_heads, G = p.group;
    auto fail = [&]() {
        flag_error(p.status, PA_DEVERR_TIMEOUT_);
        sm.abort = 1;
    };

    if (warp >= kWarpLoad && warp < kWarpFix0) {
        warpgroup_reg_release<kRegAux>();
        // ---------------------------------------------------------------- loads
        // Block-table entries of an item, 32 at a time, one per lane; an entry outside the
        // pool becomes a row past the tensor map (TMA reads zeros).
        auto entries = [&](int32_t seq, int32_t first, int32_t end) {
            int32_t phys = p.num_blocks;
            if (first + lane < end) {
                phys = p.block_tables[(size_t)seq * p.max_blocks_per_seq + first + lane];
                if (phys < 0 || phys >= p.num_blocks) {
                    flag_error(p.status, PA_DEVERR_BAD_BLOCK_);
                    phys = p.num_blocks;
                }
            }
            return phys;
        };
        // The K (V) tiles of an item, ring places n0, n0 + 2, ..; one lane issues the copies,
        // all from values the whole warp agrees on (copies issued lane by lane took 90 cycles
        // each, and bounded the kernel).  `phase`: bit s, parity of this warp's next copy on
        // stage s; V tiles from fix0 on land on kv_raw (16-bit caches).
        constexpr uint32_t kRing = C::kKv8 ? C::N8 : C::NST;
        auto load_tiles = [&](const CUtensorMap* map, uint32_t n0, int32_t nt, int32_t seq, int32_t kvh,
                              int32_t tile0, int32_t len, int32_t fix0, uint32_t& full_phase,
                              uint32_t& raw_phase) {
            const int32_t nb0 = tile0 * C::BLOCKS;
            const int32_t nb1 = min(nb0 + nt * C::BLOCKS, (len + C::BS - 1) / C::BS);
            int32_t chunk = 0, cur = entries(seq, nb0, nb1), nxt = entries(seq, nb0 + 32, nb1);
            uint32_t n = n0;
#pragma unroll 1
            for (int32_t j = 0; j < nt; ++j, n += 2) {
                const int32_t tb = j * C::BLOCKS;
                if ((tb >> 5) != chunk) {
                    chunk = tb >> 5;
                    cur = nxt;
                    nxt = entries(seq, nb0 + 32 * (chunk + 1), nb1);
                }
                const uint32_t st = n % kRing;
                const bool raw = !C::kKv8 && j >= fix0;
                uint64_t* const full = C::kKv8 ? &sm.kv8_full[st] : raw ? &sm.kv_raw[st] : &sm.kv_full[st];
                if (!mbar_wait_warp(C::kKv8 ? &sm.kv8_empty[st] : &sm.kv_empty[st], ((n / kRing) & 1) ^ 1))
                    return false;
                int32_t y[C::BLOCKS];
#pragma unroll
                for (int b = 0; b < C::BLOCKS; ++b)
                    y[b] = (__shfl_sync(0xffffffffu, cur, (tb & 31) + b) * Hkv + kvh) * C::BS;
                if (elect_one()) {
                    mbar_arrive_expect_tx(full, C::kKv8 ? C::TILE8 : C::TILE);
                    uint8_t* const dst = C::kKv8 ? sm.kv8[st] : sm.kv[st];
#pragma unroll
                    for (int b = 0; b < C::BLOCKS; ++b)
#pragma unroll
                        for (int h = 0; h < (C::kKv8 ? 1 : C::HALVES); ++h)
                            tma_load_2d_keep(dst + h * C::HALF + b * C::BS * 128, map, h * 64, y[b], full);
                }
                __syncwarp();
                if (raw) raw_phase ^= 1u << st;
                else full_phase ^= 1u << st;
            }
            return true;
        };
        // After an abort, copies may still be landing: waits (bounded) for this warp's last
        // ones, at ring places before `end`.  (The fp8 ring is odd, so its stages change
        // hands, and a wait there may run to its limit.)
        auto settle_copies = [&](uint32_t full_phase, uint32_t raw_phase, uint32_t end) {
            if (lane != 0 || !sm.abort) return;
            for (uint32_t k = 2; k <= 2 * kRing && k <= end; k += 2) {
                const uint32_t n = end - k, st = n % kRing;
                if (C::kKv8) {
                    (void)mbar_wait(&sm.kv8_full[st], (n / kRing) & 1);
                } else {
                    (void)mbar_wait(&sm.kv_full[st], ((full_phase >> st) & 1) ^ 1);
                    (void)mbar_wait(&sm.kv_raw[st], ((raw_phase >> st) & 1) ^ 1);
                }
            }
        };
        if (warp == kWarpLoad) {
            // ---------------------------------------- items, Q and K tiles
            PfHeader hdr = {};
            int4 mine = make_int4(0, 0, 0, 0);   // direct: sequence `lane`, as the plan lists it
            if (!p.direct) {
                hdr = *p.hdr;
            } else {
                const PfChunk c = chunk_of(p, lane, lane < p.num_seqs && blockIdx.x == 0);
                int32_t tiles = c.row_tiles, before = tiles;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int32_t y = __shfl_up_sync(0xffffffffu, before, o);
                    if (lane >= o) before += y;
                }
                mine = make_int4(c.start, c.count, c.len, before - tiles);
                int32_t all = __shfl_sync(0xffffffffu, before, 31);
                if (all > p.max_row_tiles) {   // chunks that overlap
                    if (lane == 0 && blockIdx.x == 0) flag_error(p.status, PA_DEVERR_BAD_LEN_);
                    all = p.max_row_tiles;
                }
                hdr.total_units = (uint32_t)(all * Hkv);
            }
            const int64_t shares = hdr.shares;
            // cut 0: the unit to take next; cut 1: the cost at which this share goes on, and
            // where it ends
            int32_t w = (int32_t)blockIdx.x;
            auto share_at = [&](int64_t b) { return b * hdr.cost / shares; };
            int64_t at = 0, end = 0;
            int32_t here = 0;
            if (hdr.cut && w < (int32_t)hdr.shares) {
                at = share_at(w);
                end = share_at(w + 1);
            }
            uint32_t kt = 0, nq = 0;   // ring places and Q loads used
            uint32_t full_phase = 0, raw_phase = 0;
            bool ok = true;
            for (uint32_t it = 0; ok; ++it) {
                const uint32_t us = it & 1;
                ok = mbar_wait_warp(&sm.u_empty[us], ((it >> 1) & 1) ^ 1);
                if (!ok) break;
                // the next unit: row tile and kv head, and (cut 1) the tiles of this share
                Unit u;
                u.seq = -1;
                u.cnt[0] = u.cnt[1] = u.nt = u.both = u.single = 0;
                u.nparts = 1;
                u.part = u.first = 0;
                int32_t claimed = 0, rt = -1, tile0 = 0, tile1 = kNoToken;
                if (warp_sees_abort(sm.abort)) {
                } else if (!hdr.cut) {
                    if (w < (int32_t)hdr.total_units) {
                        if (p.direct) claimed = (int32_t)hdr.total_units;
                        else if (lane == 0) claimed = (int32_t)(gridDim.x + atomicAdd(&p.hdr->counter, 1u));
                        rt = p.direct ? w / Hkv : p.order[w / Hkv];
                        u.kvh = w % Hkv;
                    }
                } else {
                    // (a share may be used up by the beginning of a unit that belongs to the
                    // next one)
                    if (at < end) do {
                        // row tile: the last one whose units begin at or before `at`
                        int32_t a = here;
                        if (it == 0) {
                            int32_t b = (int32_t)(hdr.total_units / (uint32_t)Hkv);
                            while (b - a > 1) {
                                const int32_t m = (a + b) >> 1;
                                if (p.before[m] * Hkv <= at) a = m;
                                else b = m;
                            }
                        } else if (p.before[a + 1] * Hkv <= at) {
                            ++a;
                        }
                        here = a;
                        const int64_t len = p.before[a + 1] - p.before[a];   // a unit's cost
                        const int64_t in = at - p.before[a] * Hkv;
                        const int32_t kvh = (int32_t)(in / len);
                        const int64_t begin = p.before[a] * Hkv + kvh * len;
                        const int64_t body = begin + kPfItemCost;            // its first tile
                        if (end <= body && end < begin + len) {
                            at = end;                                        // the next share's
                            break;
                        }
                        // shares that begin inside the unit's tiles: lo, lo + 1, .. hi
                        const int64_t lo = ((body + 1) * shares + hdr.cost - 1) / hdr.cost;
                        const int64_t hi = ((begin + len) * shares - 1) / hdr.cost;
                        rt = a;
                        u.kvh = kvh;
                        u.nparts = (int32_t)max(hi - lo + 1, (int64_t)0) + 1;
                        u.first = (int32_t)(u.nparts > 1 ? lo - 1 : w);
                        u.part = w - u.first;
                        tile0 = at > body ? (int32_t)(at - body) : 0;
                        tile1 = end < begin + len ? (int32_t)(end - body) : kNoToken;
                        at = min(begin + len, end);
                    } while (false);
                }
                if (rt >= 0) {
                    int4 q;
                    if (p.direct) {
                        // the last sequence whose first row tile is at or before this one
                        u.seq = 31 - __clz(__ballot_sync(0xffffffffu, lane < p.num_seqs && mine.w <= rt));
                        q.x = __shfl_sync(0xffffffffu, mine.x, u.seq);
                        q.y = __shfl_sync(0xffffffffu, mine.y, u.seq);
                        q.z = __shfl_sync(0xffffffffu, mine.z, u.seq);
                        q.w = __shfl_sync(0xffffffffu, mine.w, u.seq);
                    } else {
                        u.seq = p.seq_of[rt];
                        q = p.seqs[u.seq];
                    }
                    u.q_start = q.x;
                    u.q_len = q.y;
                    u.len = q.z;
                    u.tok0 = (rt - q.w) * 2 * p.tpt;
                    u.tile0 = tile0;
                    // tiles a stream needs: up to the last token its last row sees
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int32_t a = u.tok0 + i * p.tpt, b = min(a + p.tpt, u.q_len);
                        const int32_t n = a < u.q_len ? max(u.len - u.q_len + b, 0) : 0;
                        u.cnt[i] = max(min((n + kPfTok - 1) / kPfTok, tile1) - tile0, 0);
                    }
                    u.nt = max(u.cnt[0], u.cnt[1]);
                    u.single = u.tok0 + p.tpt >= u.q_len;
                    // rows for one stream only: both take them, and every other tile each
                    // (not with the fp8 ring, whose three stages hold too few tiles ahead)
                    if (!C::kKv8 && u.single && u.nt > 1) {
                        u.both = 1;
                        u.cnt[0] = (u.nt + 1) / 2;
                        u.cnt[1] = u.nt / 2;
                    }
                    // first tile that some row does not see whole
                    u.fix0 = max(u.len - u.q_len + u.tok0 + 1, 0) / kPfTok - tile0;
                }
                // no one reads the table of two items ago any more
                if (sm.any_nonfinite[us]) {
                    __syncwarp();
                    for (int i = lane; i < 3 * D; i += 32) (&sm.nonfinite[us][0][0])[i] = kNoToken;
                    if (lane == 0) sm.any_nonfinite[us] = 0;
                }
                __syncwarp();
                if (lane == 0) {
                    sm.unit[us] = u;
                    mbar_arrive(&sm.u_full[us]);
                }
                if (u.seq < 0) {
                    if (lane == 0) allow_dependent_launch();
                    break;
                }
                const int32_t nt = u.nt;
                if (nt > 0) {
                    if (lane == 0) {
                        ok = mbar_wait(&sm.q_empty, (nq & 1) ^ 1);
                        if (ok) {
                            const uint32_t rows = (uint32_t)(p.tpt * G);
                            mbar_arrive_expect_tx(&sm.q_full, ((u.cnt[0] > 0) + (u.cnt[1] > 0)) * rows *
                                                                  C::HALVES * 128u);
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (u.cnt[i] > 0)
                                    for (int h = 0; h < C::HALVES; ++h)
                                        tma_load_3d(sm.q[i] + h * C::HALF, &qmap, h * 64, u.kvh * G,
                                                    u.q_start + u.tok0 + (u.both ? 0 : i * p.tpt),
                                                    &sm.q_full);
                        }
                    }
                    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                    if (ok) ++nq;
                }
                if (ok && nt > 0)
                    ok = load_tiles(&kmap, kt, nt, u.seq, u.kvh, u.tile0, u.len, nt, full_phase, raw_phase);
                kt += 2 * nt;
                if (!hdr.cut) w = __shfl_sync(0xffffffffu, claimed, 0);
            }
            if (!ok && lane == 0) fail();
            settle_copies(full_phase, raw_phase, kt);
            if (lane == 0 && sm.abort && nq > 0) (void)mbar_wait(&sm.q_full, (nq - 1) & 1);
            __syncwarp();
        } else if (warp == kWarpLoadV) {
            // ---------------------------------------- V tiles
            uint32_t kt = 0, full_phase = 0, raw_phase = 0;
            bool ok = true;
            for (uint32_t it = 0; ok; ++it) {
                const uint32_t us = it & 1;
                ok = mbar_wait_warp(&sm.u_full[us], (it >> 1) & 1);
                if (!ok) break;
                const int32_t seq = __shfl_sync(0xffffffffu, sm.unit[us].seq, 0);
                const int32_t kvh = __shfl_sync(0xffffffffu, sm.unit[us].kvh, 0);
                const int32_t tile0 = __shfl_sync(0xffffffffu, sm.unit[us].tile0, 0);
                const int32_t len = __shfl_sync(0xffffffffu, sm.unit[us].len, 0);
                const int32_t fix0 = __shfl_sync(0xffffffffu, sm.unit[us].fix0, 0);
                const int32_t nt = __shfl_sync(0xffffffffu, sm.unit[us].nt, 0);
                if (lane == 0) mbar_arrive(&sm.u_empty[us]);
                if (seq < 0) break;
                if (nt > 0)
                    ok = load_tiles(&vmap, kt + 1, nt, seq, kvh, tile0, len, fix0, full_phase, raw_phase);
                kt += 2 * nt;
            }
            if (!ok && lane == 0) fail();
            settle_copies(full_phase, raw_phase, kt + 1);
            __syncwarp();
        } else if (warp == kWarpReady) {
            // ------------------------------------------------------------ readiness
            // Waits in the MMA warp's stead for everything but the weights: for Q, the first
            // K tile, then per tile its V, the next K and (first tile) the stream's O, and
            // adds its arrival to the weights'.  A wait costs the MMA warp 130-200 cycles even
            // when it is over; now it has one per stream and tile.
            uint32_t st = 0, q_phase = 0;             // next stage of the ring; parity of q
            uint32_t full_phase = 0, fix_phase = 0;   // bit s: parity of stage s's next such tile
            uint32_t p_phase = 0x3, o_phase = 0;      // bit i: parities of stream i (P: the last one)
            bool ok = true;
            auto next = [](uint32_t x) { return x + 1 == C::NST ? 0u : x + 1; };
            auto wait_kv = [&](uint32_t x, bool fixed) {
                const uint32_t phase = fixed ? fix_phase : full_phase;
                const bool here = mbar_wait_warp(fixed ? &sm.kv_fixed[x] : &sm.kv_full[x], (phase >> x) & 1);
                if (fixed) fix_phase ^= 1u << x;
                else full_phase ^= 1u << x;
                return here;
            };
#pragma unroll 1
            for (uint32_t it = 0; ok; ++it) {
                const uint32_t us = it & 1;
                ok = mbar_wait_warp(&sm.u_full[us], (it >> 1) & 1);
                if (!ok) break;
                const int32_t seq = sm.unit[us].seq, fix0 = sm.unit[us].fix0, nt = sm.unit[us].nt;
                const int32_t cnt0 = sm.unit[us].cnt[0], cnt1 = sm.unit[us].cnt[1];
                const bool both = sm.unit[us].both;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.u_empty[us]);
                if (seq < 0) break;
                if (nt == 0) continue;
                ok = mbar_wait_warp(C::kKv8 && C::kQBf16 ? &sm.q_ready : &sm.q_full, q_phase);
                q_phase ^= 1;
                if (ok) ok = wait_kv(st, false);
                if (ok && both) ok = wait_kv(next(next(st)), false);
                if (!ok) break;
                if (lane == 0) mbar_arrive(&sm.item_ready);
                // a stream's next K tile comes `ahead` tiles after the one it works on
                const int32_t ahead = both ? 2 : 1;
#pragma unroll 1
                for (int32_t j = 0; j < nt && ok; ++j) {
                    const uint32_t vs = next(st), kn = next(vs);
                    ok = wait_kv(vs, !C::kKv8 && j >= fix0);
                    if (!C::kKv8 && ok && j + ahead < nt) ok = wait_kv(both ? next(next(kn)) : kn, false);
#pragma unroll 1
                    for (uint32_t i = 0; i < 2 && ok; ++i) {
                        if (both ? (j & 1) != (int32_t)i : j >= (i ? cnt1 : cnt0)) continue;
                        if (j < ahead) {
                            ok = mbar_wait_warp(&sm.o_free[i], ((o_phase >> i) & 1) ^ 1);
                            o_phase ^= 1u << i;
                        }
                        // (the arrival belongs to this tile's phase: the last one is over)
                        if (ok) ok = mbar_wait_warp(&sm.p_full[i], (p_phase >> i) & 1);
                        p_phase ^= 1u << i;
                        if (ok && lane == 0) mbar_arrive(&sm.p_full[i]);
                    }
                    // (a widened K tile comes later: its stage is the last V tile's)
                    if (C::kKv8 && ok && j + 1 < nt) {
                        ok = wait_kv(kn, false);
                        if (ok && lane == 0) mbar_arrive(&sm.k_ready);
                    }
                    st = kn;
                }
            }
            if (!ok && lane == 0) fail();
            __syncwarp();
        } else {
            // ------------------------------------------------------------ MMA issuer
            // The whole warp runs the loop and one elected lane issues: with every value the
            // same in all lanes, descriptors stay in uniform registers, and a product step
            // issues faster than the tensor pipe takes it (64 cycles).
            constexpr uint32_t kIdQK = mma_idesc_f16(C::kBf16, 0, 0, kPfRows, kPfTok);
            constexpr uint32_t kIdPV = mma_idesc_f16(C::kBf16, 0, 1, kPfRows, D);
            const uint32_t q_lo = desc_lo(smem_u32(sm.q[0]), 16);
            const uint32_t k_lo = desc_lo(smem_u32(sm.kv[0]), 16);
            const uint32_t v_lo = desc_lo(smem_u32(sm.kv[0]), C::HALF);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            uint32_t st = 0, i_phase = 0, k_phase = 0;   // next stage of the ring; parities
            uint32_t p_phase = 0;                     // bit i: parity of stream i
            bool ok = true;
            auto next = [](uint32_t x) { return x + 1 == C::NST ? 0u : x + 1; };
            // (one lane) S of stream i = Q K^T with the K tile of stage x
            auto qk = [&](uint32_t i, uint32_t x) {
                const uint32_t a = q_lo + i * (C::TILE >> 4), b = k_lo + x * (C::TILE >> 4);
                const uint32_t d = tm + C::COL_S + i * kPfTok;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 2) * C::HALF + (k & 3) * 32) >> 4;
                    mma_ss(d, a + off, b + off, kIdQK, k > 0);
                }
                mma_commit(&sm.s_full[i]);
            };
            // (one lane) O of stream i += P V with the V tile of stage x; P of either half of
            // the tokens sits where that half's scores were
            auto pv = [&](uint32_t i, uint32_t x, uint32_t more) {
                const uint32_t a = tm + C::COL_S + i * kPfTok, b = v_lo + x * (C::TILE >> 4);
                const uint32_t d = tm + C::COL_O + i * D;
#pragma unroll
                for (int k = 0; k < kPfTok / 16; ++k)
                    mma_ts(d, a + 8 * (k & 3) + (k >> 2) * (kPfTok / 2), b + k * (2048 >> 4), kIdPV,
                           k > 0 ? 1u : more);
            };
#pragma unroll 1
            for (uint32_t it = 0; ok; ++it) {
                const uint32_t us = it & 1;
                ok = mbar_wait_warp(&sm.u_full[us], (it >> 1) & 1);
                if (!ok) break;
                const int32_t seq = __shfl_sync(0xffffffffu, sm.unit[us].seq, 0);
                const int32_t cnt0 = __shfl_sync(0xffffffffu, sm.unit[us].cnt[0], 0);
                const int32_t cnt1 = __shfl_sync(0xffffffffu, sm.unit[us].cnt[1], 0);
                const int32_t nt = __shfl_sync(0xffffffffu, sm.unit[us].nt, 0);
                const int32_t both = __shfl_sync(0xffffffffu, sm.unit[us].both, 0);
                if (lane == 0) mbar_arrive(&sm.u_empty[us]);
                if (seq < 0) break;
                if (nt == 0) continue;
                ok = mbar_wait_warp(&sm.item_ready, i_phase);
                i_phase ^= 1;
                if (!ok) break;
                // tile j's K sits in stage ks, its V in the next one
                uint32_t ks = st;
                tmem_fence_after_sync();
                const int32_t ahead = both ? 2 : 1;   // tiles to a stream's next one
                if (elect_one()) {
                    const uint32_t k1 = both ? next(next(ks)) : ks;
                    if (cnt0 > 0) qk(0, ks);
                    if (cnt1 > 0) qk(1, k1);
                    mma_commit(&sm.kv_empty[ks]);
                    if (both) mma_commit(&sm.kv_empty[k1]);
                    if (nt <= ahead) mma_commit(&sm.q_empty);
                }
                // per tile: PV of each stream and its next QK^T, with nothing to wait for in
                // between
#pragma unroll 1
                for (int32_t j = 0; j < nt; ++j) {
                    const uint32_t vs = next(ks), kn = next(vs);   // V of tile j, K of the next
                    const uint32_t kq = both ? next(next(kn)) : kn;   // the next scores' K
                    const uint32_t last = both ? (uint32_t)j & 1u : j < cnt1 ? 1 : 0;
                    bool k_here = false;
#pragma unroll 1
                    for (uint32_t i = both ? last : j < cnt0 ? 0 : 1; i <= last; ++i) {
                        const bool more = both ? j + 2 < nt : j + 1 < (i ? cnt1 : cnt0);
                        ok = mbar_wait_warp(&sm.p_full[i], (p_phase >> i) & 1);
                        if (!ok) break;
                        tmem_fence_after_sync();
                        // (one lane) what follows PV: the stages given back, the next scores
                        auto go_on = [&]() {
                            if (i == last) mma_commit(&sm.kv_empty[vs]);
                            if (more) qk(i, kq);
                            if (i == last) {
                                if (j + ahead < nt) mma_commit(&sm.kv_empty[kq]);
                                if (j + ahead + 1 == nt) mma_commit(&sm.q_empty);
                            }
                        };
                        if (elect_one()) {
                            pv(i, vs, j >= ahead ? 1u : 0u);
                            if (!more) mma_commit(&sm.o_full[i]);
                            if (!C::kKv8) go_on();
                        }
                        if (C::kKv8) {
                            // (the V stage is given back after the wait for K: a K tile that
                            // needs the stage cannot become ready, and complete the barrier's
                            // next phase, while this one is still waited for)
                            if (more && !k_here) {
                                ok = mbar_wait_warp(&sm.k_ready, k_phase);
                                k_phase ^= 1;
                                k_here = true;
                                if (!ok) break;
                                tmem_fence_after_sync();
                            }
                            if (elect_one()) go_on();
                        }
                        p_phase ^= 1u << i;
                    }
                    if (!ok) break;
                    ks = kn;
                }
                st = ks;
            }
            if (!ok && lane == 0) fail();
            // every MMA of this warp has completed before tensor memory is freed
            if (elect_one()) mma_commit(&sm.drain);
            (void)mbar_wait_warp(&sm.drain, 0);
            __syncwarp();
        }
    } else if (warp >= kWarpFix0) {
        // ---------------------------------------------------------- fixing / widening warps
        warpgroup_reg_release<kRegFix>();
        const int fw = warp - kWarpFix0, tid = fw * 32 + lane;
        uint32_t kt = 0, nq = 0;
        uint32_t raw_phase = 0;   // bit s: parity of stage s's next tile to fix
        bool ok = true;
        for (uint32_t it = 0; ok; ++it) {
            const uint32_t us = it & 1;
            ok = mbar_wait_warp(&sm.u_full[us], (it >> 1) & 1);
            if (!ok) break;
            const int32_t seq = sm.unit[us].seq, fix0 = sm.unit[us].fix0;
            const int32_t cnt0 = sm.unit[us].cnt[0], cnt1 = sm.unit[us].cnt[1];
            const int32_t len = sm.unit[us].len, tile0 = sm.unit[us].tile0, nt = sm.unit[us].nt;
            __syncwarp();
            // (the slot is released by the softmax warps at the item's end as well, so the
            // table of non-finite values stays this item's until then)
            if (lane == 0) mbar_arrive(&sm.u_empty[us]);
            if (seq < 0) break;
            if (nt == 0) continue;
            auto note = [&](int d, int32_t tok, int cls) {
                atomicMin(&sm.nonfinite[us][cls][d], tok);
                sm.any_nonfinite[us] = 1;
            };
            // V row `row` of a 16-bit tile in `buf`: zeroed past the context; else its
            // infinite and NaN elements noted and replaced by 0
            auto fix_row = [&](uint8_t* buf, int row, int32_t tok) {
                if (tok >= len) {
#pragma unroll
                    for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            *reinterpret_cast<uint4*>(buf + h * C::HALF + row * 128 +
                                                      (((c + row) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                    return;
                }
                uint32_t acc = 0;
#pragma unroll
                for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const uint4 x = *reinterpret_cast<const uint4*>(buf + h * C::HALF + row * 128 +
                                                                        (((c + row) & 7) << 4));
                        acc = taint<C::kBf16>(acc, x.x);
                        acc = taint<C::kBf16>(acc, x.y);
                        acc = taint<C::kBf16>(acc, x.z);
                        acc = taint<C::kBf16>(acc, x.w);
                    }
                constexpr uint32_t kExp = C::kBf16 ? 0x7F80u : 0x7C00u;
                if ((acc & kExp) != kExp && ((acc >> 16) & kExp) != kExp) return;
#pragma unroll 1
                for (int d = 0; d < D; ++d) {
                    uint16_t* x = reinterpret_cast<uint16_t*>(
                        buf + (d >> 6) * C::HALF + row * 128 + ((((d >> 3) & 7) ^ (row & 7)) << 4) + (d & 7) * 2);
                    const uint32_t v = *x;
                    if ((v & kExp) == kExp) {
                        note(d, tok, (v & 0x7FFFu) != kExp ? 2 : (v >> 15));
                        *x = 0;
                    }
                }
            };
            if constexpr (!C::kKv8) {
                for (int32_t j = max(fix0, 0); j < nt && ok; ++j) {
                    const uint32_t n = kt + 2 * j + 1, vs = n % C::NST;
                    ok = mbar_wait_warp(&sm.kv_raw[vs], (raw_phase >> vs) & 1);
                    if (!ok) break;
                    raw_phase ^= 1u << vs;
                    fix_row(sm.kv[vs], tid, (tile0 + j) * kPfTok + tid);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.kv_fixed[vs]);
                }
                kt += 2 * nt;
            } else {
                if constexpr (C::kQBf16) {
                    // bf16 queries as fp16 (|q| <= 65504), in place
                    ok = mbar_wait_warp(&sm.q_full, nq & 1);
                    if (!ok) break;
                    for (int i = 0; i < 2; ++i) {
                        if ((i ? cnt1 : cnt0) == 0) continue;
                        uint4* q = reinterpret_cast<uint4*>(sm.q[i]);
#pragma unroll 4
                        for (int c = tid; c < (int)(C::TILE / 16); c += 128) {
                            uint4 x = q[c];
                            uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float a, b;
                                unpack2<true>(w[k], a, b);
                                w[k] = pack2<false>(a, b);
                            }
                            q[c] = x;
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.q_ready);
                    ++nq;
                }
                for (int32_t t = 0; t < 2 * nt && ok; ++t, ++kt) {
                    const uint32_t s8 = kt % C::N8, st = kt % C::NST;
                    ok = mbar_wait_warp(&sm.kv8_full[s8], (kt / C::N8) & 1) &&
                         mbar_wait_warp(&sm.kv_empty[st], ((kt / C::NST) & 1) ^ 1);
                    if (!ok) break;
                    const bool fix = (t & 1) && (t >> 1) >= fix0;
                    uint8_t* const dst = sm.kv[st];
                    // 16 elements per step: lanes 0..7 of a row take its eight 16-byte pieces;
                    // four steps' reads go ahead of their writes, which the compiler could not
                    // move past one another
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        uint4 x4[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = (4 * g + i) * 16 + (tid >> 3), c = tid & 7;
                            x4[i] = *reinterpret_cast<const uint4*>(sm.kv8[s8] + row * 128 + ((c ^ (row & 7)) << 4));
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = (4 * g + i) * 16 + (tid >> 3), c = tid & 7;
                            uint4 x = x4[i];
                            if (fix) {
                                const int32_t tok = (tile0 + (t >> 1)) * kPfTok + row;
                                uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    if (tok >= len) w[k] = 0;
                                    // a byte of E4M3 is NaN when its low seven bits are all set
                                    const uint32_t nan = ((w[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                                    if (nan) {
#pragma unroll 1
                                        for (int b = 0; b < 4; ++b)
                                            if ((nan >> (8 * b)) & 0x80u) {
                                                note(16 * c + 4 * k + b, tok, 2);
                                                w[k] &= ~(0xFFu << (8 * b));
                                            }
                                    }
                                }
                            }
                            uint4 lo, hi;
                            e4m3x4_to_f16x2x2(x.x, lo.x, lo.y);
                            e4m3x4_to_f16x2x2(x.y, lo.z, lo.w);
                            e4m3x4_to_f16x2x2(x.z, hi.x, hi.y);
                            e4m3x4_to_f16x2x2(x.w, hi.z, hi.w);
                            // pieces of the second half go out in the other order, so that
                            // eight lanes always write to eight different bank groups
                            uint8_t* const r = dst + (c >> 2) * C::HALF + row * 128;
                            const int c0 = (2 * c) & 7, odd = c >> 2;
                            *reinterpret_cast<uint4*>(r + (((c0 + odd) ^ (row & 7)) << 4)) = odd ? hi : lo;
                            *reinterpret_cast<uint4*>(r + (((c0 + 1 - odd) ^ (row & 7)) << 4)) = odd ? lo : hi;
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.kv8_empty[s8]);
                        mbar_arrive(&sm.kv_full[st]);
                    }
                }
            }
        }
        if (!ok && lane == 0) fail();
    } else {
        // ---------------------------------------------------------- softmax and epilogue
        // Two threads per query row: thread `row` of warpgroup `half` takes tokens 64 half ..
        // of every tile and the same half of the head dims of O.
        warpgroup_reg_alloc<kRegSoft>();
        constexpr int kCols = kPfTok / 2, kDims = D / 2;
        const int si = warp >> 3, half = (warp >> 2) & 1, sw = warp & 3;
        const int row = sw * 32 + lane;                 // query row of the stream = TMEM lane
        const uint32_t taddr = tmem + ((uint32_t)(sw * 32) << 16);
        const uint32_t ts = taddr + C::COL_S + si * kPfTok + half * kCols;
        const uint32_t to = taddr + C::COL_O + si * D + half * kDims;
        const int bar = kBarStream + si, row_bar = kBarRows + si * 4 + sw;
        const int32_t qtok = row / G;                   // new token of this row, within the stream
        const uint64_t scale2 = pack_f32(p.scale_log2, p.scale_log2);
        const float hidden = p.scale_log2 < 0.f ? INFINITY : -INFINITY;   // -inf once scaled
        uint32_t ns = 0, no = 0;                        // scores seen, outputs taken
        uint32_t x_phase = 0, xa_phase = 0;             // bit us: parities of the streams' meetings
        bool failed = false;
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
#pragma unroll 1
        for (uint32_t it = 0;; ++it) {
            const uint32_t us = it & 1;
            bool ok = mbar_wait_warp(&sm.u_full[us], (it >> 1) & 1);
            // the warps of a stream stop together
            if (consumers_any(!ok, kStreamThreads, bar)) {
                failed = true;
                break;
            }
            // (the slot stays this item's until these warps release it, so what only the
            // epilogue needs is read there)
            const Unit& un = sm.unit[us];
            if (un.seq < 0) break;
            const int32_t cnt = un.cnt[si];
            const bool both = !C::kKv8 && un.both;
            // tokens this row sees, and the fewest any row of the stream sees
            const int32_t whole = un.len - un.q_len + un.tok0 + (both ? 0 : si * p.tpt) + 1;
            const int32_t limit = min(whole + qtok, un.len);
            // first token of the half tile
            int32_t t0 = (un.tile0 + (both ? si : 0)) * kPfTok + half * kCols;
            const int32_t t_step = both ? 2 * kPfTok : kPfTok;
            float ref = -INFINITY, sum = 0.f;
#pragma unroll 1
            for (int32_t j = 0; j < cnt; ++j, t0 += t_step) {
                ok = mbar_wait_warp(&sm.s_full[si], ns & 1);
                ++ns;
                tmem_fence_after_sync();
                const bool masked = t0 + kCols > whole;
                const int32_t seen = limit - t0;
                // 32 of the row's 64 scores, loaded before, masked
                auto scores = [&](int h, float (&x)[32]) {
                    tmem_arrived(x);
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) x[c] = 32 * h + c < seen ? x[c] : hidden;
                    }
                };
                // The largest scores of the rows that have to move (`over`, in either thread)
                // become their references, and O is rescaled.  Other rows of the two warps go
                // through this unchanged: a row's bits do not depend on its neighbours, some of
                // which hold no query.
                auto raise = [&](bool over) {
                    float m = -INFINITY;
#pragma unroll 1
                    for (int h = 0; h < kCols / 32; ++h) {
                        float x[32];
                        tmem_ld32(ts + 32 * h, x);
                        scores(h, x);
#pragma unroll
                        for (int c = 0; c < 32; ++c) m = fmaxf(m, x[c] * p.scale_log2);
                    }
                    sm.red[si][half][row] = over ? m : -INFINITY;
                    failed = consumers_any(!ok, 64, row_bar);
                    m = fmaxf(sm.red[si][half][row], sm.red[si][half ^ 1][row]) - C::kLift;
                    const float next = fmaxf(ref, m);
                    const float a = ref == next ? 1.f : fast_exp2(ref - next);
                    sum *= a;
                    ref = next;
                    if (j > 0 && __any_sync(0xffffffffu, a != 1.f) && !failed) {
                        // (the wait for S has also seen the previous tile's PV complete)
#pragma unroll 1
                        for (int h = 0; h < kDims / 32; ++h) {
                            float o[32];
                            tmem_ld32(to + 32 * h, o);
                            tmem_arrived(o);
#pragma unroll
                            for (int c = 0; c < 32; ++c) o[c] *= a;
                            tmem_st32(to + 32 * h, reinterpret_cast<const uint32_t*>(o));
                        }
                    }
                };
                if (j == 0) {
                    raise(true);
                    if (failed) break;
                }
                // Weights against the present reference and their sum, in one go.  A weight
                // that is too large makes the sum too large: then the references are raised
                // and the weights taken once more (the scores stay in tensor memory until P
                // overwrites them).
                uint32_t w[kCols / 2];
                float tile_sum;
#pragma unroll 1
                for (bool again = j == 0;; again = true) {
                    const float nref = ref == -INFINITY ? 0.f : -ref;
                    const uint64_t nref2 = pack_f32(nref, nref);
                    uint64_t s2[2] = {0ull, 0ull};
                    // (the second half's scores are on their way while the first's weights
                    // are taken)
                    float x[kCols / 32][32];
                    tmem_ld32(ts, x[0]);
#pragma unroll
                    for (int h = 0; h < kCols / 32; ++h) {
                        scores(h, x[h]);
                        if (h + 1 < kCols / 32) tmem_ld32(ts + 32 * (h + 1), x[h + 1]);
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            float a, b;
                            unpack_f32(fma_x2(pack_f32(x[h][2 * c], x[h][2 * c + 1]), scale2, nref2), a, b);
                            a = fast_exp2(a);
                            b = fast_exp2(b);
                            s2[c & 1] = add_x2(s2[c & 1], pack_f32(a, b));
                            w[16 * h + c] = pack2<C::kBf16>(a, b);
                        }
                    }
                    float a, b;
                    unpack_f32(add_x2(s2[0], s2[1]), a, b);
                    tile_sum = a + b;
                    if (again) break;
                    const bool over = tile_sum > C::kMost || (ref == -INFINITY && seen > 0);
                    if (!consumers_any(!ok || over, 64, row_bar)) break;
                    raise(over);   // rare
                    if (failed) break;
                }
                if (failed) break;
                sum += tile_sum;
                tmem_st32(ts, w);
                tmem_wait_st();
                tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full[si]);
            }
            // ---- the item's rows
            ok = !failed;
            if (cnt > 0 && ok) {
                ok = mbar_wait_warp(&sm.o_full[si], no & 1);
                ++no;
                tmem_fence_after_sync();
            }
            sm.xsum[us][si][half][row] = sum;
            if (half == 0) sm.xref[us][si][row] = ref;
            // (streams that share their rows meet here, with a bounded wait: each may have
            // given up on its own)
            auto meet = [&](uint64_t* at, uint32_t& phase) {
                tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(at);
                const bool here = mbar_wait_warp(at, (phase >> us) & 1);
                phase ^= 1u << us;
                tmem_fence_after_sync();
                return here;
            };
            if (both && ok) ok = meet(&sm.x_full[us], x_phase);
            if (consumers_any(!ok, kStreamThreads, bar)) {
                failed = true;
                break;
            }
            sum += sm.xsum[us][si][half ^ 1][row];   // (two terms: the same sum in both halves)
            const Unit u = un;
            const int32_t tok = u.tok0 + (both ? 0 : si * p.tpt) + qtok;
            const bool mine = qtok < p.tpt && tok < u.q_len;
            const bool nonfinite = sm.any_nonfinite[us] != 0;
            // Shared rows: O and the weight sums of the two streams, each against its own
            // reference, become one, w0 O0 + w1 O1.
            float w0 = 1.f, w1 = 0.f;
            bool top_here = true;      // the weight of this stream's O is 1
            if (both) {
                const float theirs = sm.xref[us][si ^ 1][row], top = fmaxf(ref, theirs);
                const float other = sm.xsum[us][si ^ 1][0][row] + sm.xsum[us][si ^ 1][1][row];
                const float a = state_weight(ref, top), b = state_weight(theirs, top);
                // (the same order of terms in either stream)
                sum = si ? fmaf(a, sum, b * other) : fmaf(b, other, a * sum);
                w0 = si ? b : a;
                w1 = si ? a : b;
                top_here = si ? ref > theirs : ref >= theirs;
                ref = top;
            }
            // infinite and NaN values that were kept out of the products, for the rows that
            // see them
            if (nonfinite && cnt > 0) {
#pragma unroll 1
                for (int d = 0; d < kDims; ++d) {
                    float o = tmem_ld1(to + d);
                    const int32_t* const first = &sm.nonfinite[us][0][half * kDims + d];
                    if (top_here && first[0] < limit) o += INFINITY;
                    if (top_here && first[D] < limit) o -= INFINITY;
                    if (top_here && first[2 * D] < limit) o = __int_as_float(0x7fc00000);
                    tmem_st1(to + d, o);
                }
            }
            int dims = kDims, dim0 = half * kDims;
            uint32_t o_at = to, o_other = 0;
            if (both) {
                if (nonfinite) {
                    ok = meet(&sm.x_again[us], xa_phase);
                    if (consumers_any(!ok, kStreamThreads, bar)) {
                        failed = true;
                        break;
                    }
                }
                // each of the four warpgroups has a quarter of the head dims
                dims = D / 4;
                dim0 = (2 * si + half) * (D / 4);
                o_at = taddr + C::COL_O + dim0;
                o_other = o_at + D;
            }
            // 16 head dims of O (0 where the stream had no tile)
            auto load_o = [&](int h, float (&o)[16]) {
                if (cnt > 0) {
                    tmem_ld16(o_at + 16 * h, o);
                    tmem_wait_ld();
                    if (both) {
                        float o1[16];
                        tmem_ld16(o_other + 16 * h, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; ++c) o[c] = fmaf(w0, o[c], w1 * o1[c]);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 16; ++c) o[c] = 0.f;
                }
            };
            // 16 outputs from head dim d on, packed, of rows among which some are infinite or NaN:
            // where one is NaN in a row whose sum of weights is not, the V rows that the row sees
            // say whether it is +inf or -inf.
            auto settle = [&](int d, uint32_t (&y)[8], int32_t seq, bool has_sum) {
                constexpr uint32_t kExp = C::kQBf16 ? 0x7F80u : 0x7C00u;
                uint32_t odd = 0, inf = 0, nan = 0;
                if (has_sum && mine && limit <= kSettleTokens) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        odd |= (y[k] & 0x7FFFu) > kExp ? 1u << (2 * k) : 0u;
                        odd |= ((y[k] >> 16) & 0x7FFFu) > kExp ? 2u << (2 * k) : 0u;
                    }
                }
                const uint32_t any = __reduce_or_sync(0xffffffffu, odd);
                if (any == 0) return;
                auto look = [&](int32_t t) {
                    const int32_t block = p.block_tables[(size_t)seq * p.max_blocks_per_seq + t / C::BS];
                    if (block < 0 || block >= p.num_blocks) return;
                    const int64_t vrow = ((int64_t)block * Hkv + u.kvh) * C::BS + t % C::BS;
                    odd_values<C::kBf16>(static_cast<const uint16_t*>(p.value_cache) + vrow * D + d, inf, nan);
                };
                // the tokens that all these rows see, the warp together, then each row's own
                const int32_t all = __reduce_min_sync(0xffffffffu, odd ? limit : kNoToken);
#pragma unroll 1
                for (int32_t t = 0; t < all; t += 32) {
                    if (t + lane < all) look(t + lane);
                    if ((__reduce_or_sync(0xffffffffu, nan) & any) == any) break;
                }
                inf = __reduce_or_sync(0xffffffffu, inf);
                nan = __reduce_or_sync(0xffffffffu, nan);
#pragma unroll 1
                for (int32_t t = all; odd && t < limit; ++t) look(t);
                __syncwarp();
                odd &= ~nan & (inf ^ (inf >> 16));
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    if ((odd >> c) & 1u) {
                        const uint32_t v = kExp | ((inf >> c) & 1u ? 0u : 0x8000u);
                        y[c / 2] = c & 1 ? (y[c / 2] & 0xFFFFu) | (v << 16) : (y[c / 2] & 0xFFFF0000u) | v;
                    }
            };
            auto store_row = [&](int d, const float (&o)[16], float f, int32_t seq) {
                uint32_t y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = pack2<C::kQBf16>(o[2 * k] * f, o[2 * k + 1] * f);
                if constexpr (!C::kKv8) {      // (e4m3 has no infinity: NaN it is)
                    uint32_t z0 = 0, z1 = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        z0 = taint<C::kQBf16>(z0, y[k]);
                        z1 = taint<C::kQBf16>(z1, y[k + 4]);
                    }
                    if (__any_sync(0xffffffffu, mine && (z0 | z1) != 0)) settle(d, y, seq, f == f);
                }
                if (!mine) return;
                const size_t orow =
                    ((size_t)(u.q_start + tok) * p.num_q_heads + (size_t)u.kvh * G + row % G) * D;
                uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + orow + d);
                // (a warp's lanes write to as many rows, and what counts is the number of stores:
                // 16 bytes at a time, a prompt of 8192 tokens took 353 us instead of 345)
                if (wide) {
                    st_v8(dst, y);
                } else {
                    dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
                    dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
                }
            };
            // these warps are done with the item's O and its slot
            auto release = [&]() {
                tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (both) {
                        mbar_arrive(&sm.o_free[0]);
                        mbar_arrive(&sm.o_free[1]);
                    } else if (cnt > 0) {
                        mbar_arrive(&sm.o_free[si]);
                        mbar_arrive(&sm.o_free[si]);
                    }
                    mbar_arrive(&sm.u_empty[us]);
                }
            };
            if (u.nparts == 1) {
                const float f = sum == 0.f ? 0.f : p.out_scale / sum;
#pragma unroll 1
                for (int h = 0; h < dims / 16; ++h) {
                    float o[16];
                    load_o(h, o);
                    store_row(dim0 + 16 * h, o, f, un.seq);
                }
                release();
            } else {
                // Partial rows, [dim][row] so that a warp's accesses are contiguous.  (A
                // share's place 1 is for a unit that goes on, 0 for one that came to it;
                // rows of one stream only are its first stream's, whoever works on them.)
                const int sj = u.single ? 0 : si;
                const bool takes_part = both || !u.single || si == 0;
                auto place = [&](int part) {
                    return ((size_t)(2 * (u.first + part) + (part == 0)) * 2 + sj) * kPfRows;
                };
                auto cell = [&](size_t at, int d) { return at * D + (size_t)d * kPfRows + row; };
                if (takes_part) {
                    const size_t at = place(u.part);
#pragma unroll 1
                    for (int h = 0; h < dims / 16; ++h) {
                        float o[16];
                        load_o(h, o);
#pragma unroll
                        for (int c = 0; c < 16; ++c) p.part_acc[cell(at, dim0 + 16 * h + c)] = o[c];
                    }
                    if (half == 0 && !(both && si)) p.part_ml[at + row] = make_float2(ref, sum);
                }
                release();
                if (takes_part) {
                    // The stream that finishes the row tile's last partition joins them,
                    // always in the order of the partitions.  Shared rows count once for each
                    // stream, so a partition of a single stream's rows is worth two.
                    __threadfence();
                    named_bar_sync(bar, kStreamThreads);
                    if (row == 0 && half == 0) {
                        const int32_t worth = u.single && !both ? 2 : 1;
                        const int32_t full = u.single ? 2 * u.nparts : u.nparts;
                        sm.last_seq[si] = u.seq;
                        sm.last_part[si] = atomicAdd(&p.arrive[2 * u.first + sj], worth) == full - worth;
                    }
                    named_bar_sync(bar, kStreamThreads);
                    if (sm.last_part[si]) {
                        __threadfence();
                        float M = -INFINITY;
#pragma unroll 1
                        for (int q = 0; q < u.nparts; ++q) M = fmaxf(M, __ldcg(&p.part_ml[place(q) + row]).x);
                        float den = 0.f;
#pragma unroll 1
                        for (int q = 0; q < u.nparts; ++q) {
                            const float2 ml = __ldcg(&p.part_ml[place(q) + row]);
                            den += state_weight(ml.x, M) * ml.y;
                        }
                        const float f = den == 0.f ? 0.f : p.out_scale / den;
                        // (three partitions' values are on their way together: one at a time, joining six of them
                        // took 20 us)
#pragma unroll 1
                        for (int h = 0; h < kDims / 16; ++h) {
                            const int d = half * kDims + 16 * h;
                            float o[16];
#pragma unroll
                            for (int c = 0; c < 16; ++c) o[c] = 0.f;
#pragma unroll 1
                            for (int q = 0; q < u.nparts; q += 3) {
                                float v[3][16], wq[3];
#pragma unroll
                                for (int t = 0; t < 3; ++t) {
                                    const size_t pr = place(min(q + t, u.nparts - 1));
                                    const bool in = mine && q + t < u.nparts;
                                    wq[t] = in ? __ldcg(&p.part_ml[pr + row]).x : -INFINITY;
#pragma unroll
                                    for (int c = 0; c < 16; ++c)
                                        v[t][c] = in ? __ldcg(&p.part_acc[cell(pr, d + c)]) : 0.f;
                                }
#pragma unroll
                                for (int t = 0; t < 3; ++t) {
                                    const float weight = state_weight(wq[t], M);
#pragma unroll
                                    for (int c = 0; c < 16; ++c) o[c] = fmaf(weight, v[t][c], o[c]);
                                }
                            }
                            store_row(d, o, f, sm.last_seq[si]);
                        }
                    }
                }
            }
        }
        if (failed && lane == 0) fail();
    }

    __syncthreads();
    if (warp == kWarpMma) {
        tmem_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace pf
}  // namespace pa
