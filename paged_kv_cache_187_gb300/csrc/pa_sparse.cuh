// pa_sparse.cuh -- attention over selected blocks of the paged cache: for each query token and kv
// head (a row) the softmax over the tokens of its selected blocks.
//
// Rows are short (64 blocks of 16 tokens are 512 KB of K and V) and mostly of one length, and a call
// has a few of them or some hundreds; what it costs beside the bytes is latency: launches, dependent
// loads (list -> block table -> tiles) and the round trips where the parts of a row meet.  So there
// is one launch and no plan, and a row belongs to a cluster of 1 to 16 CTAs: each translates its
// piece of the list (pa_sparse_device.cuh) and streams its tiles through a ring in shared memory by
// TMA, the consumers being the decode's (pa_decode.cuh: tiles of one or two blocks, online softmax
// on mma.sync for grouped heads and 8-bit caches, on CUDA cores for single ones; a tile or a CTA's
// whole part may hold scores of -inf alone, from infinite keys, whose weights are 0: kLow); the parts
// meet in shared memory, where every CTA joins its share of the row's elements out of the others'.
//
// Measured (device time a call, calls back to back; 8 kv heads of 128, floors at the measured copy
// bandwidth in brackets).  One sequence, 64 blocks of 16 tokens a row, 32 query heads: 7.1-7.6 us [0.6];
// with the decode over tables that a kernel of its own made, 20.4.  48 sequences, 128 blocks: 64
// [59.3], where the decode's partitions took 83, and slices of one size for every CTA, cut through
// the rows and joined through memory, 71: CTAs with the same bytes finish up to 13 us apart, and
// every joint is a round trip of 3-6 us.  Below the launch's 3 us and the first tile's 3 what bounds
// it is HBM from some 300 CTAs on, and the bytes that the CTAs have on their way below that.
#pragma once

#include <algorithm>
#include <atomic>

#include "pa_decode_family.cuh"
#include "pa_masked.h"
#include "pa_sparse_device.cuh"

namespace pa {

__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

template <class C>
struct alignas(1024) SparseSmem {
    // a ring of K and V tiles; once they are all consumed, the consumers' states in its place
    union {
        uint8_t kv[C::NSTAGE][2][C::TILE_BYTES];
        struct {
            float sums[C::HCAP * C::D];
            float states[C::NCONS > 1 ? C::NCONS - 1 : 1][C::NSTATE * 32];
        };
    };
    alignas(128) uint8_t q[C::HCAP * C::D * 2];
    alignas(16) float pbuf[C::kMma ? 1 : C::NCONS][C::kMma ? 1 : C::HCAP][C::kMma ? 1 : C::BS];
    alignas(16) float2 ml[C::HCAP];           // (reference, weight sum) of this CTA's part
    uint64_t full[C::NSTAGE], empty[C::NSTAGE], qfull, listed;
    uint32_t issued[C::NSTAGE], consumed[C::NSTAGE];
    int32_t blocks[kSparseEntries + C::TB - 1];
    int32_t tokens, q_read;
    volatile int32_t abort;
};
template <class C>
constexpr size_t sparse_smem_bytes() {
    return sizeof(SparseSmem<C>) + 1024;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Every thread of every CTA of the cluster; what was written before is seen after.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// A consumer's state (unnormalised sums, references, weight sums) into shared memory, [head][dim].
template <class C>
__device__ __forceinline__ void stage_state(const MmaConsumer<C>& cons, float* ostage, float2* ml, int nrows, int lane) {
    using M = MmaConsumer<C>;
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float v = cons.l[nt][j];
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            const int h = nt * 8 + 2 * lane + j;
            if (lane < 4 && h < nrows) ml[h] = make_float2(cons.m[nt][j], v);
        }
#pragma unroll
    for (int i = 0; i < M::KS; ++i)
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int h = nt * 8 + 2 * (lane & 3) + (r & 1);
                ostage[h * C::D + M::out_dim(i, lane, r)] = cons.acc[i][nt][r];
            }
}
template <class C>
__device__ __forceinline__ void stage_state(const CoreConsumer<C>& cons, float* ostage, float2* ml, int nrows, int lane) {
    constexpr int DPL = C::D / 32;
#pragma unroll
    for (int h = 0; h < C::HCAP; ++h) {
        float v = cons.l[h];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        if (lane == 0 && h < nrows) ml[h] = make_float2(cons.m[h], v);
#pragma unroll
        for (int j = 0; j < DPL; ++j) ostage[h * C::D + lane * DPL + j] = cons.acc[h][j];
    }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::MIN_CTAS)
    sparse_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const DecodeParams p, const SparseParams sp) {
    extern __shared__ uint8_t smem_raw[];
    SparseSmem<C>& sm = *reinterpret_cast<SparseSmem<C>*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t parts = sp.cluster;
    const int32_t rank = parts > 1 ? (int32_t)cluster_rank() : 0;
    const int32_t row = (int32_t)blockIdx.x / parts;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NSTAGE; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
            sm.issued[i] = 0;
            sm.consumed[i] = 0;
        }
        mbar_init(&sm.qfull, 1);
        mbar_init(&sm.listed, 1);
        sm.abort = sm.q_read = 0;
        fence_barrier_init();
        prefetch_tensor_map(&kmap);
        prefetch_tensor_map(&vmap);
    }
    if (threadIdx.x < C::HCAP) sm.ml[threadIdx.x] = make_float2(-INFINITY, 0.f);
    __syncthreads();
    grid_dependency_wait();
    auto timed_out = [&]() {
        if (lane == 0) {
            flag_error(p.status, PA_DEVERR_TIMEOUT_);
            sm.abort = 1;
        }
    };
    // Elements 8 i .. of the row's outputs, of their sums and the sum of the weights (0: nothing is
    // seen; NaN: some score is)
    auto store_eight = [&](int32_t i, float den, const float (&y)[8]) {
        const float f = den == 0.f ? 0.f : p.out_scale / den;
        uint4 o;
        o.x = pack2<C::kBf16>(y[0] * f, y[1] * f);
        o.y = pack2<C::kBf16>(y[2] * f, y[3] * f);
        o.z = pack2<C::kBf16>(y[4] * f, y[5] * f);
        o.w = pack2<C::kBf16>(y[6] * f, y[7] * f);
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (size_t)row * p.group * C::D)[i] = o;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            const uint32_t qbytes = (uint32_t)(p.group * C::D * 2);
            mbar_arrive_expect_tx(&sm.qfull, qbytes);
            bulk_load(sm.q, reinterpret_cast<const uint8_t*>(p.q) + (size_t)row * p.group * C::D * 2, qbytes,
                      &sm.qfull);
        }
        // this CTA's piece of the list, kSparseEntries entries at a time
        const int32_t K = sp.num_selected;
        const int32_t per = ((K + parts - 1) / parts + C::TB - 1) / C::TB * C::TB;
        const int32_t e0 = min(rank * per, K), e1 = min(e0 + per, K);
        int32_t tokens = 0;
        auto tell = [&]() {
            if (lane == 0) {
                sm.tokens = tokens;
                mbar_arrive(&sm.listed);
            }
        };
        if (e1 - e0 > kSparseEntries) {      // the consumers have to know how many tokens there are
            for (int32_t c0 = e0; c0 < e1; c0 += kSparseEntries)
                tokens += walk_list(sp, row, c0, min(c0 + kSparseEntries, e1), 0, [](int32_t, int32_t) {}).tokens;
            tell();
        }
        // (blocks that several query tokens read may stay in L2)
        const uint64_t policy = sp.q_len > 1 ? l2_evict_normal_policy() : l2_evict_first_policy();
        bool out = false, ok = true;
        uint32_t stage = 0, ephase = 1;
        int32_t have = 0;                    // blocks of a tile that the next piece completes
        for (int32_t c0 = e0; ok && c0 < e1; c0 += kSparseEntries) {
            const int32_t c1 = min(c0 + kSparseEntries, e1);
            const SparseList list = walk_list(sp, row, c0, c1, p.num_blocks,
                                              [&](int32_t i, int32_t b) { sm.blocks[have + i] = b; });
            __syncwarp();
            if (e1 - e0 <= kSparseEntries) {
                tokens = list.tokens;
                tell();
            }
            const int32_t n = have + list.count;
            const int32_t ntiles = c1 == e1 ? (n + C::TB - 1) / C::TB : n / C::TB;
            for (int32_t i = 0; i < ntiles && ok; ++i) {
                if (lane == 0) {
                    ok = mbar_wait(&sm.empty[stage], ephase);
                    if (ok) {
                        mbar_arrive_expect_tx(&sm.full[stage], 2u * C::TILE_BYTES);
#pragma unroll
                        for (int bi = 0; bi < C::TB; ++bi) {
                            // (a tile's block past the list: a row past the tensor map, zeros)
                            const int32_t e = i * C::TB + bi;
                            const int32_t b = e < n ? sm.blocks[e] : p.num_blocks;
                            out |= e < n && b == p.num_blocks;
                            const int32_t y = b * C::PBS;
                            const uint32_t off = bi * C::PBS * 128;
#pragma unroll
                            for (int hf = 0; hf < C::HALVES; ++hf) {
                                tma_load_2d(sm.kv[stage][0] + hf * C::HALF_BYTES + off, &kmap, hf * 64, y,
                                            &sm.full[stage], policy);
                                tma_load_2d(sm.kv[stage][1] + hf * C::HALF_BYTES + off, &vmap, hf * 64, y,
                                            &sm.full[stage], policy);
                            }
                        }
                        sm.issued[stage] += 1;
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                if (++stage == C::NSTAGE) {
                    stage = 0;
                    ephase ^= 1;
                }
            }
            // (blocks left over go to the front)
            __syncwarp();
            const int32_t rest = max(n - ntiles * C::TB, 0);
            const int32_t b = lane < rest ? sm.blocks[ntiles * C::TB + lane] : 0;
            __syncwarp();
            if (lane < rest) sm.blocks[lane] = b;
            have = rest;
        }
        // (at the start, the next call's CTAs took the places that are left, unevenly: 48 sequences 71
        // instead of 64 us)
        if (lane == 0) allow_dependent_launch();
        if (e0 >= e1) tell();
        if (!ok) timed_out();
        if (out) flag_error(p.status, PA_DEVERR_BAD_BLOCK_);
    } else {
        // ------------------------------------------------------------ consumers
        using Consumer = typename std::conditional<C::kMma, MmaConsumer<C>, CoreConsumer<C>>::type;
        const int c = warp - 1;
        constexpr int TS = C::NCONS;
        Consumer cons;
        bool stop = !mbar_wait_warp(&sm.qfull, 0) || !mbar_wait_warp(&sm.listed, 0);
        cons.reset();
        if (!stop) {
            cons.load_q(sm.q, p.group, lane);
            if (c == 0 && lane == 0) sm.q_read = 1;
            const int32_t tokens = sm.tokens, ntiles = (tokens + C::BS - 1) / C::BS;
            for (int32_t t = c; t < ntiles; t += TS) {
                const uint32_t stage = (uint32_t)t % C::NSTAGE, fphase = ((uint32_t)t / C::NSTAGE) & 1;
                stop = warp_sees_abort(sm.abort) || !mbar_wait_warp(&sm.full[stage], fphase);
                if (stop) break;
                const int valid = min(C::BS, tokens - t * C::BS);
                if constexpr (C::kMma)
                    cons.tile(sm.kv[stage][0], sm.kv[stage][1], valid, t * C::BS, p.scale_log2, lane, nullptr);
                else
                    cons.tile(sm.kv[stage][0], sm.kv[stage][1], valid, t * C::BS, p.scale_log2, lane, sm.pbuf[c]);
                __syncwarp();
                if (lane == 0) {
                    sm.consumed[stage] += 1;
                    mbar_arrive(&sm.empty[stage]);
                }
            }
        }
        if (stop) timed_out();
        // the consumers' states meet in the first one (no tile is read any more, or, after an
        // abort, nothing of this is used)
        if constexpr (TS > 1) {
            stop = consumers_any(stop, 32 * TS);
            if (c > 0 && !stop) cons.export_state(sm.states[c - 1], lane);
            named_bar_sync(1, 32 * TS);
        }
        if (c == 0 && !stop) {
            for (int o = 0; o < TS - 1; ++o) cons.merge_state(sm.states[o], lane);
            stage_state<C>(cons, sm.sums, sm.ml, p.group, lane);
            __syncwarp();
            if (parts == 1 && !warp_sees_abort(sm.abort)) {
                for (int32_t i = lane; i < p.group * C::D / 8; i += 32) {
                    const float4* x = reinterpret_cast<const float4*>(sm.sums + 8 * i);
                    const float4 a = x[0], b = x[1];
                    store_eight(i, sm.ml[i / (C::D / 8)].y, {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w});
                }
            }
        }
    }
    if (parts > 1) {
        // The row's parts meet: each CTA takes every parts-th piece of eight elements.
        __syncwarp();
        cluster_sync();
        const uint32_t acc0 = smem_u32(sm.sums), ml0 = smem_u32(sm.ml);
        if (!sm.abort) {
            for (int32_t i = (int32_t)threadIdx.x * parts + rank; i < p.group * C::D / 8; i += C::THREADS * parts) {
                const int32_t h = i / (C::D / 8);
                // (a running join, eight parts' values on their way together)
                float M = -INFINITY, den = 0.f, y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                for (int32_t q0 = 0; q0 < parts; q0 += 8) {
                    float2 ml[8];
                    float4 x[8][2];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        ml[q] = make_float2(-INFINITY, 0.f);
                        x[q][0] = x[q][1] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (q0 + q < parts) {
                            ml[q] = ld_cluster2(map_to_rank(ml0 + h * 8, q0 + q));
                            const uint32_t a = map_to_rank(acc0 + i * 32, q0 + q);
                            x[q][0] = ld_cluster4(a);
                            x[q][1] = ld_cluster4(a + 16);
                        }
                    }
                    float next = M;
#pragma unroll
                    for (int q = 0; q < 8; ++q) next = fmaxf(next, ml[q].x);
                    const float keep = state_weight(M, next);
                    M = next;
                    den *= keep;
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[k] *= keep;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float w = state_weight(ml[q].x, M);
                        den += w * ml[q].y;
                        y[0] += w * x[q][0].x, y[1] += w * x[q][0].y, y[2] += w * x[q][0].z, y[3] += w * x[q][0].w;
                        y[4] += w * x[q][1].x, y[5] += w * x[q][1].y, y[6] += w * x[q][1].z, y[7] += w * x[q][1].w;
                    }
                }
                store_eight(i, den, y);
            }
        }
        __syncwarp();
        cluster_sync();          // (the others may still be reading here)
    }
    // On a timeout, copies may still be landing: wait (bounded) for those never consumed.
    __syncthreads();
    if (threadIdx.x == 0 && sm.abort) {
        for (int i = 0; i < C::NSTAGE; ++i)
            if (sm.issued[i] > sm.consumed[i]) (void)mbar_wait(&sm.full[i], sm.consumed[i] & 1);
        if (!sm.q_read) (void)mbar_wait(&sm.qfull, 0);
    }
}

// A short ring, so that more CTAs fit an SM: about half of the decode's stages (8-bit caches: two
// consumers and four stages; three and three took 115 us where these take 80).
template <int NSTAGE, int NCONS>
constexpr int short_stages() {
    return std::max((NSTAGE / 2 + NCONS - 1) / NCONS * NCONS, 2);
}

// Launches the attention with `ctas` CTAs, or (ctas 0) tells the CTAs per SM that it can have.
template <int D, int BS, bool BF16, bool MMA, int HCAP, bool KV8, int TB>
cudaError_t launch_sparse_one(const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeParams& p,
                              const SparseParams& sp, int32_t ctas, cudaStream_t stream, int32_t* per_sm) {
    constexpr int kTile = BS * TB;
    constexpr int kCons = consumers_for<MMA, kTile, KV8>();
    constexpr int kStages = stages_for<D * (KV8 ? 1 : 2) / 2, kTile, kCons>();
    using C0 = DecodeCfg<D, kTile, BF16, MMA, HCAP, kStages, 1, kCons, KV8, false, 0, BS>;
    using C = DecodeCfg<D, kTile, BF16, MMA, HCAP, kStages, 1, kCons, KV8, false, decode_min_ctas<C0>(), BS, true>;
    constexpr int kShortCons = KV8 ? 2 : kCons, kShort = KV8 ? 4 : short_stages<kStages, kCons>();
    using CS = DecodeCfg<D, kTile, BF16, MMA, HCAP, kShort, 1, kShortCons, KV8, false, decode_min_ctas<C0>(), BS, true>;
    using Kern = void (*)(CUtensorMap, CUtensorMap, DecodeParams, SparseParams);
    const Kern kerns[2] = {sparse_kernel<C>, sparse_kernel<CS>};
    constexpr size_t smems[2] = {sparse_smem_bytes<C>(), sparse_smem_bytes<CS>()};
    constexpr int threads[2] = {C::THREADS, CS::THREADS};
    const int kind = sp.short_ring ? 1 : 0;
    static PerDeviceOnce configured;
    static std::atomic<int32_t> known[2][PerDeviceOnce::kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = static_cast<cudaError_t>(configured.run(dev, [&] {
        cudaError_t e1 = cudaSuccess;
        for (int i = 0; i < 2 && e1 == cudaSuccess; ++i) {
            e1 = cudaFuncSetAttribute(kerns[i], cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smems[i]);
            // (clusters of 16)
            if (e1 == cudaSuccess) e1 = cudaFuncSetAttribute(kerns[i], cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        }
        return e1;
    }));
    if (e != cudaSuccess) return e;
    if (ctas == 0) {
        const bool cached = dev >= 0 && dev < PerDeviceOnce::kMaxDevices;
        int n = cached ? known[kind][dev].load() : 0;
        if (n == 0) {
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kerns[kind], threads[kind], smems[kind]);
            if (e != cudaSuccess) return e;
            if (cached) known[kind][dev].store(n);
        }
        *per_sm = n;
        return cudaSuccess;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads[kind]);
    cfg.dynamicSmemBytes = smems[kind];
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)sp.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = sp.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kerns[kind], kmap, vmap, p, sp);
}

// The instantiations of one type over 16-bit caches: single query heads on the CUDA cores, groups
// on the tensor cores, as the decode (8-bit caches: pa_sparse_fp8.cu).
template <bool BF16>
cudaError_t launch_sparse_16(const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeParams& p,
                             const SparseParams& sp, int32_t head_size, int32_t ctas, cudaStream_t stream,
                             int32_t* per_sm) {
#define PA_CASE(D_, BS_)                                                                                       \
    if (head_size == D_ && sp.block_size == BS_) {                                                             \
        if (p.group == 1) return launch_sparse_one<D_, BS_, BF16, false, 1, false, 1>(kmap, vmap, p, sp, ctas, stream, per_sm); \
        if (p.group <= 8) return launch_sparse_one<D_, BS_, BF16, true, 8, false, 1>(kmap, vmap, p, sp, ctas, stream, per_sm);  \
        return launch_sparse_one<D_, BS_, BF16, true, 16, false, 1>(kmap, vmap, p, sp, ctas, stream, per_sm);  \
    }
    PA_CASE(128, 16)
    PA_CASE(128, 32)
    PA_CASE(64, 16)
    PA_CASE(64, 32)
#undef PA_CASE
    return cudaErrorInvalidValue;
}

}  // namespace pa
