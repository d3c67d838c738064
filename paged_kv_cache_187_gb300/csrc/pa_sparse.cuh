// pa_sparse.cuh -- attention over selected blocks of the paged cache: for each query token and kv
// head (a row) the softmax over the tokens of its selected blocks.
//
// The consumers are the decode's (pa_decode.cuh: tiles of one or two blocks, online softmax on
// mma.sync for grouped heads and 8-bit caches, on CUDA cores for single ones, partial states joined
// by the last part to finish); what differs is where the work comes from.  Rows are short and many
// of one length, so instead of whole rows or partitions of one size, handed out as they are asked
// for, all rows' tiles are laid end to end and cut into equal slices, one per CTA: every CTA streams
// the same number of bytes without a pause, and a row is cut in two or three pieces at most where
// there are more rows than CTAs.  (48 x 8 rows of 2048 tokens, 402 MB: 83 us with partitions, see
// below for the slices.)  The slices follow from the context lengths alone, so no plan is made: each
// CTA sums the lengths while the kernel before it still runs.
#pragma once

#include <atomic>

#include "pa_decode_family.cuh"
#include "pa_masked.h"

namespace pa {

__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::MIN_CTAS)
    sparse_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                         const DecodeParams p, const SparseParams sp) {
    extern __shared__ uint8_t smem_raw[];
    DecodeSmem<C>& sm = *reinterpret_cast<DecodeSmem<C>*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NSTAGE; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
            sm.issued[i] = 0;
            sm.consumed[i] = 0;
        }
        mbar_init(&sm.xfree, 1);
        for (int i = 0; i < C::NQ; ++i) {
            mbar_init(&sm.qfull[i], 1);
            mbar_init(&sm.qempty[i], C::NCONS);
            sm.qissued[i] = 0;
            sm.qconsumed[i] = 0;
        }
        sm.abort = 0;
        fence_barrier_init();
        prefetch_tensor_map(&kmap);
        prefetch_tensor_map(&vmap);
    }
    __syncthreads();

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        const int32_t Hkv = sp.num_kv_heads, QL = sp.q_len, S = sp.num_seqs;
        const int32_t cap = (int32_t)min((int64_t)sp.max_blocks_per_seq * C::PBS, (int64_t)INT32_MAX);
        auto len_of = [&](int32_t s) { return min(max(sp.context_lens[s], 0), cap); };
        // tiles of a row of query token j, at most: what the context holds, up to the list's length
        auto tiles_of = [&](int32_t len, int32_t j) {
            const int32_t seen = max(len - QL + j + 1, 0);
            const int32_t blocks = min(seen / C::PBS + (seen % C::PBS != 0), sp.num_selected);
            return (blocks + C::TB - 1) / C::TB;
        };
        auto cost_of = [&](int32_t s) {      // of a sequence's rows
            int64_t sum = 0;
            if (s < S) {
                const int32_t len = len_of(s);
                for (int32_t j = 0; j < QL; ++j) sum += tiles_of(len, j) + kSparseRowCost;
            }
            return sum * Hkv;
        };
        // Sequences s0 .. s0 + 31, one per lane: cost, and running sum.
        int64_t own = 0, upto = 0;
        auto sequences = [&](int32_t s0) {
            own = upto = cost_of(s0 + lane);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            return __shfl_sync(0xffffffffu, upto, 31);
        };
        int64_t total = 0;
        for (int32_t s0 = 0; s0 < S; s0 += 32) total += sequences(s0);
        const int64_t G = gridDim.x;
        const int64_t lo = total * (int64_t)blockIdx.x / G, hi = total * ((int64_t)blockIdx.x + 1) / G;
        auto cta_at = [&](int64_t x) { return (int32_t)(((x + 1) * G - 1) / total); };
        // the row that `lo` is in: sequence, query token, kv head, and where its costs begin
        int32_t s = 0, j = 0, h = 0, len = 0, T = 0;
        int64_t base = 0;
        {
            int64_t before = 0;
            for (int32_t s0 = 0; s0 < S; s0 += 32) {
                if (S > 32) sequences(s0);
                const uint32_t past = __ballot_sync(0xffffffffu, before + upto > lo);
                if (past) {
                    const int32_t l = __ffs(past) - 1;
                    s = s0 + l;
                    base = before + __shfl_sync(0xffffffffu, upto, l) - __shfl_sync(0xffffffffu, own, l);
                    break;
                }
                before += __shfl_sync(0xffffffffu, upto, 31);
            }
            len = len_of(s);
            for (j = 0; j < QL; ++j) {
                T = tiles_of(len, j);
                const int64_t c = (int64_t)(T + kSparseRowCost) * Hkv;
                if (base + c > lo) break;
                base += c;
            }
            h = (int32_t)((lo - base) / (T + kSparseRowCost));
            base += (int64_t)h * (T + kSparseRowCost);
        }
        // what the tables kernel writes (and with it everything before it)
        grid_dependency_wait();
        // The next unit of this slice, in *u (seq -1: none): the row at the cursor, or one after it,
        // with the tiles that this slice has of it.  A row belongs to the slices that hold its tiles;
        // one without tiles to the slice where it begins.
        auto next_unit = [&](UnitDesc& u) {
            u.seq = -1;
            u.kvh = u.tok0 = u.tok1 = u.row0 = u.len = 0;
            u.pslot = -1;
            u.pbase = 0;
            u.nparts = 1;
            u.nrows = p.group;
            u.pad[0] = u.pad[1] = 0;
            while (base < hi) {
                const int64_t first = base + kSparseRowCost;
                const int32_t t0 = (int32_t)min(max(lo - first, (int64_t)0), (int64_t)T);
                const int32_t t1 = (int32_t)min(max(hi - first, (int64_t)0), (int64_t)T);
                const bool here = t1 > t0 || (T == 0 && base >= lo);
                if (here) {
                    const int32_t row = (s * QL + j) * Hkv + h;
                    u.seq = row;
                    u.tok0 = t0 * C::BS;
                    u.tok1 = t1 * C::BS;       // (at most: the row's tokens are not known yet)
                    if (T > 0 && (t0 > 0 || t1 < T)) {
                        const int32_t a = cta_at(first), b = cta_at(first + T - 1);
                        u.nparts = b - a + 1;
                        u.pbase = a + row;     // (slots: a CTA's and its row's number, added)
                        u.pslot = (int32_t)blockIdx.x + row;
                    }
                }
                // the cursor goes on
                base += T + kSparseRowCost;
                if (++h == Hkv) {
                    h = 0;
                    if (++j == QL) {
                        j = 0;
                        if (++s < S) len = len_of(s);
                    }
                    T = tiles_of(len, j);
                }
                if (here) return;
            }
        };
        // Table entries b0 .. b0 + 31 of a row, one per lane; those outside the pool become a row
        // past the tensor map (TMA reads zeros).
        auto load_blocks = [&](int32_t row, int32_t b0, int32_t n) {
            int32_t phys = p.num_blocks;
            if (lane < n) {
                phys = sp.tables[(size_t)row * sp.num_selected + b0 + lane];
                if (phys < 0 || phys >= p.num_blocks) {
                    flag_error(p.status, PA_DEVERR_BAD_BLOCK_);
                    phys = p.num_blocks;
                }
            }
            return phys;
        };
        // the row's tokens, and its first blocks here (all of them in the table are written up to
        // the row's count; entries past it are not used)
        auto row_len = [&](const UnitDesc& u) { return u.seq >= 0 ? sp.lens[u.seq] : 0; };
        auto first_blocks = [&](const UnitDesc& u, int32_t n_tok) {
            const int32_t b0 = u.tok0 / C::PBS;
            const int32_t b1 = (min(u.tok1, n_tok) + C::PBS - 1) / C::PBS;
            return u.seq >= 0 ? load_blocks(u.seq, b0, min(32, b1 - b0)) : 0;
        };
        const uint64_t policy = QL > 1 ? l2_evict_normal_policy() : l2_evict_first_policy();
        const uint32_t qbytes = (uint32_t)(p.group * C::D * 2);
        UnitDesc u, next;
        next_unit(u);
        int32_t tokens = row_len(u), phys0 = first_blocks(u, tokens);
        uint32_t stage = 0, ephase = 1;
        for (uint32_t it = 0;; ++it) {
            if (warp_sees_abort(sm.abort)) u.seq = -1;
            u.tok1 = max(min(u.tok1, tokens), u.tok0);
            const uint32_t qs = it % C::NQ, qphase = ((it / C::NQ) & 1) ^ 1;
            bool ok = true;
            if (lane == 0) {
                ok = mbar_wait(&sm.qempty[qs], qphase);
                if (ok) {
                    sm.unit[qs] = u;
                    if (u.seq < 0) {
                        mbar_arrive(&sm.qfull[qs]);
                    } else {
                        mbar_arrive_expect_tx(&sm.qfull[qs], qbytes);
                        bulk_load(sm.qbuf[qs],
                                  reinterpret_cast<const uint8_t*>(p.q) + (size_t)u.seq * p.group * C::D * 2, qbytes,
                                  &sm.qfull[qs]);
                        sm.qissued[qs] += 1;
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (!ok) {
                if (lane == 0) {
                    flag_error(p.status, PA_DEVERR_TIMEOUT_);
                    sm.abort = 1;
                }
                break;
            }
            if (u.seq < 0) {
                if (lane == 0) allow_dependent_launch();
                break;
            }
            // the unit after this one, its length and first blocks on their way meanwhile
            next_unit(next);
            const int32_t next_tokens = row_len(next);
            int32_t next_phys = 0;
            bool have_next = false;
            const int32_t nb0 = u.tok0 / C::PBS, nb1 = (u.tok1 + C::PBS - 1) / C::PBS;
            const int32_t ntiles = (u.tok1 - u.tok0 + C::BS - 1) / C::BS;
            int32_t phys = phys0;
            for (int32_t i = 0; i < ntiles && ok; ++i) {
                const int32_t e = (i * C::TB) & 31;
                if (e == 0 && i > 0) phys = load_blocks(u.seq, nb0 + i * C::TB, min(32, nb1 - nb0 - i * C::TB));
                if (i == 1) {
                    next_phys = first_blocks(next, next_tokens);
                    have_next = true;
                }
                int32_t pb[C::TB];
#pragma unroll
                for (int bi = 0; bi < C::TB; ++bi) pb[bi] = __shfl_sync(0xffffffffu, phys, e + bi);
                if (lane == 0) {
                    ok = mbar_wait(&sm.empty[stage], ephase);
                    if (ok) {
                        mbar_arrive_expect_tx(&sm.full[stage], 2u * C::TILE_BYTES);
#pragma unroll
                        for (int bi = 0; bi < C::TB; ++bi) {
                            const int32_t y = pb[bi] * C::PBS;
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
                if (!ok) break;
                if (++stage == C::NSTAGE) {
                    stage = 0;
                    ephase ^= 1;
                }
            }
            if (!ok) {
                if (lane == 0) {
                    flag_error(p.status, PA_DEVERR_TIMEOUT_);
                    sm.abort = 1;
                }
                break;
            }
            if (!have_next) next_phys = first_blocks(next, next_tokens);
            u = next;
            tokens = next_tokens;
            phys0 = next_phys;
        }
    } else {
        // ------------------------------------------------------------ consumers (as the decode's)
        grid_dependency_wait();
        using Consumer = typename std::conditional<C::kMma, MmaConsumer<C>, CoreConsumer<C>>::type;
        const int c = warp - 1;
        constexpr int TS = C::NCONS;
        auto all_agree = [&](bool v) {
            if constexpr (C::NCONS > 1) return consumers_any(v, 32 * C::NCONS);
            else return __any_sync(0xffffffffu, v);
        };
        auto timed_out = [&]() {
            if (lane == 0) {
                flag_error(p.status, PA_DEVERR_TIMEOUT_);
                sm.abort = 1;
            }
        };
        Consumer cons;
        uint32_t gtile = 0;   // tiles of all earlier units
        for (uint32_t it = 0;; ++it) {
            const uint32_t qs = it % C::NQ, qphase = (it / C::NQ) & 1;
            bool stop = !mbar_wait_warp(&sm.qfull[qs], qphase);
            if (stop) timed_out();
            stop = stop || warp_sees_abort(sm.abort);
            const UnitDesc u = sm.unit[qs];
            if (stop || u.seq < 0) {
                (void)all_agree(true);   // the unit barrier below, from a consumer that stops
                break;
            }
            cons.load_q(sm.qbuf[qs], u.nrows, lane);
            __syncwarp();
            if (lane == 0) {
                if (c == 0) sm.qconsumed[qs] += 1;
                mbar_arrive(&sm.qempty[qs]);
            }
            cons.reset();
            const int32_t b0 = u.tok0 / C::BS;
            const int32_t ntiles = (u.tok1 + C::BS - 1) / C::BS - b0;
            // tile k (over all units) goes to consumer k % TS; the last tile's consumer leads
            const int gmod = (int)(gtile % (uint32_t)TS);
            const int lead = (gmod + ntiles - 1 + TS) % TS;
            for (int32_t t = (c - gmod + TS) % TS; t < ntiles; t += TS) {
                const uint32_t k = gtile + (uint32_t)t;
                const uint32_t stage = k % C::NSTAGE, fphase = (k / C::NSTAGE) & 1;
                if (warp_sees_abort(sm.abort)) {
                    stop = true;
                    break;
                }
                if (!mbar_wait_warp(&sm.full[stage], fphase)) {
                    timed_out();
                    stop = true;
                    break;
                }
                const int tile0 = (b0 + t) * C::BS;
                const int valid = min(C::BS, u.tok1 - tile0);
                if constexpr (C::kMma)
                    cons.tile(sm.kv[stage][0], sm.kv[stage][1], valid, tile0, p.scale_log2, lane, nullptr);
                else
                    cons.tile(sm.kv[stage][0], sm.kv[stage][1], valid, tile0, p.scale_log2, lane, sm.pbuf[c]);
                __syncwarp();
                if (lane == 0) {
                    sm.consumed[stage] += 1;
                    mbar_arrive(&sm.empty[stage]);
                }
            }
            gtile += (uint32_t)ntiles;
            if (TS > 1 && !stop && c != lead) {
                if (it > 0 && !mbar_wait_warp(&sm.xfree, (it - 1) & 1)) {
                    timed_out();
                    stop = true;
                } else {
                    cons.export_state(sm.xbuf[(c - lead - 1 + TS) % TS], lane);
                }
            }
            if (all_agree(stop)) break;   // the unit barrier (also: the states are in shared memory)
            if (c == lead) {
                for (int o = 0; o < TS - 1; ++o) cons.merge_state(sm.xbuf[o], lane);
                if (TS > 1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.xfree);
                }
                if (!warp_sees_abort(sm.abort)) cons.finish(sm.ostage, p, u, lane);
            }
        }
    }

    // On a timeout, copies may still be landing: wait (bounded) for those never consumed.
    __syncthreads();
    if (threadIdx.x == 0 && sm.abort) {
        for (int i = 0; i < C::NSTAGE; ++i)
            if (sm.issued[i] > sm.consumed[i]) (void)mbar_wait(&sm.full[i], sm.consumed[i] & 1);
        for (int i = 0; i < C::NQ; ++i)
            if (sm.qissued[i] > sm.qconsumed[i]) (void)mbar_wait(&sm.qfull[i], sm.qconsumed[i] & 1);
    }
}

// Launches the kernel with `ctas` CTAs, or (ctas 0) tells the CTAs per SM that it can have.
template <int D, int BS, bool BF16, bool MMA, int HCAP, bool KV8, int TB>
cudaError_t launch_sparse_one(const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeParams& p,
                              const SparseParams& sp, int32_t ctas, cudaStream_t stream, int32_t* per_sm) {
    constexpr int kTile = BS * TB;
    constexpr int kCons = consumers_for<MMA, kTile, KV8>();
    constexpr int kStages = stages_for<D * (KV8 ? 1 : 2) / 2, kTile, kCons>();
    using C0 = DecodeCfg<D, kTile, BF16, MMA, HCAP, kStages, 2, kCons, KV8, false, 0, BS>;
    using C = DecodeCfg<D, kTile, BF16, MMA, HCAP, kStages, 2, kCons, KV8, false, decode_min_ctas<C0>(), BS>;
    constexpr size_t smem = decode_smem_bytes<C>();
    auto kern = sparse_decode_kernel<C>;
    static PerDeviceOnce configured;
    static std::atomic<int32_t> known[PerDeviceOnce::kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = static_cast<cudaError_t>(configured.run(dev, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    }));
    if (e != cudaSuccess) return e;
    if (ctas == 0) {
        int n = dev >= 0 && dev < PerDeviceOnce::kMaxDevices ? known[dev].load() : 0;
        if (n == 0) {
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, C::THREADS, smem);
            if (e != cudaSuccess) return e;
            if (dev >= 0 && dev < PerDeviceOnce::kMaxDevices) known[dev].store(n);
        }
        *per_sm = n;
        return cudaSuccess;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, kmap, vmap, p, sp);
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
