// gemm_act.cu -- the bf16 product with bias, activation and residual in its epilogue (sm_100a):
//   h[t][f] = sum_k A[t][k] B[f][k] + bias[f],   D = act(h) + residual,   pre = h in bf16
//
// On SM pairs (tcgen05.mma.cta_group::2, kind::f16, fp32 accumulators in TMEM).  The features are the MMA's M side, 256
// per tile, 128 per CTA; the rows are its N side, up to 256 per tile in steps of 32.  So few rows cost few MMA cycles, a
// TMEM lane is a feature and the epilogue's bias a register, and the 32 lanes of a warp hold 32 neighbours of one output
// row: bias, activation, residual and stores are done from registers, with no staging in shared memory.
//
// Warps: 0 TMA producer (6 stages of 64 products, 192 KiB per CTA), 1 MMA issuer in the pair's leader, in the other CTA it
// forwards "accumulator read"; 2-17 epilogue.  The accumulator is double-buffered (2 x 256 TMEM columns).  The tensor
// core truncates as it accumulates, so an accumulator holds at most 512 products with fp32 output and 1024 with bf16
// output (errors of 5e-7 and 1e-6), and the epilogue joins such runs in registers, rounded to nearest, while the next
// one is under way; the activations and stores of one tile run under the products of the next.
//
// SPLIT > 1: where there are fewer tiles than pairs, a cluster of SPLIT pairs takes one tile, each pair a part of K.  The
// pairs' sums meet in shared memory: each pair finishes a part of the rows, for which the others send it theirs
// through the cluster's network, into the ring that the products no longer need, and adds them in the order of the
// parts.  No workspace, no atomics, no waiting on memory.
//
// Every mbarrier wait is bounded by the caller's budget; on expiry the CTA raises the timeout flag, drains its copies
// and MMAs (bounded again) and frees its TMEM.
#include <algorithm>

#include "act.cuh"
#include "nvfp4_device.cuh"
#include "sm100_ptx.cuh"

namespace nvfp4 {

using namespace ptx;

constexpr int kGaStages = 6;
constexpr int kGaK = 64;                                 // products per stage
constexpr int kGaOpBytes = 128 * kGaK * 2;               // an operand's 128 features or rows
constexpr int kGaStageBytes = 2 * kGaOpBytes;
constexpr int kGaRing = kGaStages * kGaStageBytes;       // 192 KiB
constexpr int kGaEpiWarps = 16;
constexpr int kGaThreads = 64 + 32 * kGaEpiWarps;
constexpr int kGaRunK = 512, kGaRunBf16 = 4096;          // products per accumulator with fp32, bf16 output
constexpr int kGaBand = 8;                               // row tiles swept together along the features (L2 reuse)
constexpr uint64_t kGaDrainNs = 2000000000ull;           // teardown waits, whatever the caller's budget

struct GemmActParams {
    const float* bias;
    const void* residual;
    uint16_t* pre;
    void* d;
    int64_t ldr, ldpre, ldd;
    int32_t M, N;
    int32_t stages, run;    // of K, and of an accumulator
    int32_t np, nq, wq;     // feature tiles, row tiles and their width
    int32_t act, out_fp32, res_fp32;
    int32_t pairs;          // D, pre and the residual can be taken two features at a time
    uint32_t* flags;
    uint64_t budget_ns;
};

struct GemmActSmem {        // behind the stages
    uint64_t full[kGaStages];      // leader: a stage's bytes of both CTAs
    uint64_t empty[kGaStages];     // both: the MMAs that read the stage are done
    uint64_t tfull[2];             // both: accumulator ready
    uint64_t tempty[2];            // leader: both CTAs' epilogues have read it
    uint64_t edrained[2];          // the other CTA: its epilogue has read it
    uint64_t done;
    uint32_t tmem, abort, peer_abort, issued;
    uint32_t consumed, runs;       // leader: stages and accumulators that the MMA issuer has committed
    uint32_t stage_tx[kGaStages];  // bytes per CTA of the last use of each stage
};
constexpr int kGaSmem = kGaRing + (int)sizeof(GemmActSmem) + 1024;
static_assert(kGaSmem <= 232448, "shared memory");

struct GemmActMaps {
    CUtensorMap p, q[3];    // features; rows in boxes of 32, 64 and 128
};

struct GaTile {
    int p0, q0, qn, n;      // first feature, first row, valid rows, the MMA's N
};
__device__ __forceinline__ GaTile ga_tile(const GemmActParams& p, int t) {
    GaTile r;
    const int band = t / (kGaBand * p.np), in_band = t - band * (kGaBand * p.np);
    const int rows = min(kGaBand, p.nq - band * kGaBand);
    const int pt = in_band / rows;
    r.p0 = 256 * pt;
    r.q0 = (band * kGaBand + in_band - pt * rows) * p.wq;
    r.qn = min(p.wq, p.M - r.q0);
    r.n = (r.qn + 31) & ~31;
    return r;
}

// arrivals in both CTAs of the pair whose leader has cluster rank `leader`
__device__ __forceinline__ void commit_pair(uint32_t bar, uint32_t leader) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)(3u << leader))
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "f"(r[0]), "f"(r[1]),
                 "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster_f32(uint32_t cluster_addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

// ---------------------------------------------------------------------------------------
// epilogue: 16 rows of one feature per lane, from sums to their places
//
// bf16 words hold two features of a row, so neighbouring lanes trade: a lane packs its feature of rows i and i + 1,
// and of its own word and its neighbour's the even lane keeps row i's halves, the odd one row i + 1's.
// ---------------------------------------------------------------------------------------
template <int ACT>
__device__ __forceinline__ void act16(float* v, bool wide) {
    if (wide) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = act::wide<ACT>(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; i += 2) act::pair<ACT>(v[i], v[i + 1]);
    }
}
__device__ __forceinline__ void act16(int act, float* v, bool wide) {
    switch (act) {
        case kActRelu: act16<kActRelu>(v, wide); break;
        case kActRelu2: act16<kActRelu2>(v, wide); break;
        case kActGelu: act16<kActGelu>(v, wide); break;
        case kActSilu: act16<kActSilu>(v, wide); break;
    }
}
// the trade, its own inverse: halves {own row i, own row i + 1} <-> {feature even, feature odd} of row i + odd
__device__ __forceinline__ uint32_t traded(uint32_t w, uint32_t select) {
    return __byte_perm(w, __shfl_xor_sync(0xFFFFFFFFu, w, 1), select);
}
// 16 rows of bf16 words from row0 + odd on, two features a lane
__device__ __forceinline__ void put_words(uint16_t* at, int64_t ld, const float* v, uint32_t select) {
#pragma unroll
    for (int i = 0; i < 16; i += 2, at += 2 * ld) *reinterpret_cast<uint32_t*>(at) = traded(f32x2_to_bf16x2(v[i], v[i + 1]), select);
}

// v: sums of rows row0 .. row0 + 15 of feature f.  All of the rows and of the warp's 32 features exist, and leading
// dimensions are even.
__device__ __forceinline__ void finish16(float* v, const GemmActParams& p, int row0, int f, float bias) {
    const int odd = threadIdx.x & 1, fe = f - odd;
    const uint32_t select = odd ? 0x3276u : 0x5410u;
    // the residual first: its loads are under way during the rest
    float w[16];
    if (p.residual) {
        if (p.res_fp32) {
            const float* r = reinterpret_cast<const float*>(p.residual) + row0 * p.ldr + f;
#pragma unroll
            for (int i = 0; i < 16; ++i, r += p.ldr) w[i] = *r;
        } else {
            const uint16_t* r = reinterpret_cast<const uint16_t*>(p.residual) + (row0 + odd) * p.ldr + fe;
#pragma unroll
            for (int i = 0; i < 8; ++i, r += 2 * p.ldr) w[i] = __uint_as_float(*reinterpret_cast<const uint32_t*>(r));
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += bias;
    if (p.pre) put_words(p.pre + (row0 + odd) * p.ldpre + fe, p.ldpre, v, select);
    act16(p.act, v, p.out_fp32);
    if (p.residual) {
        if (p.res_fp32) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] += w[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t u = traded(__float_as_uint(w[i]), select);
                v[2 * i] += bf16_lo(u);
                v[2 * i + 1] += bf16_hi(u);
            }
        }
    }
    if (p.out_fp32) {
        float* at = reinterpret_cast<float*>(p.d) + row0 * p.ldd + f;
#pragma unroll
        for (int i = 0; i < 16; ++i, at += p.ldd) *at = v[i];
    } else {
        put_words(reinterpret_cast<uint16_t*>(p.d) + (row0 + odd) * p.ldd + fe, p.ldd, v, select);
    }
}

// The same at the edges of the output, or where a leading dimension is odd: the first n rows, element by element
__device__ __noinline__ void finish_edge(float v0, float v1, float v2, float v3, const GemmActParams& p, int64_t row0, int n, int f, float bias) {
    float v[4] = {v0 + bias, v1 + bias, v2 + bias, v3 + bias};
    if (f >= p.N) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= n) break;
        const int64_t row = row0 + i;
        if (p.pre) p.pre[row * p.ldpre + f] = (uint16_t)f32x2_to_bf16x2(v[i], 0.0f);
        float y;
        if (p.out_fp32) {
            y = act::wide(p.act, v[i]);
        } else {
            float z = y = v[i];
            switch (p.act) {
                case kActRelu: act::pair<kActRelu>(y, z); break;
                case kActRelu2: act::pair<kActRelu2>(y, z); break;
                case kActGelu: act::pair<kActGelu>(y, z); break;
                case kActSilu: act::pair<kActSilu>(y, z); break;
            }
        }
        if (p.residual)
            y += p.res_fp32 ? reinterpret_cast<const float*>(p.residual)[row * p.ldr + f]
                            : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p.residual)[row * p.ldr + f] << 16);
        if (p.out_fp32) reinterpret_cast<float*>(p.d)[row * p.ldd + f] = y;
        else reinterpret_cast<uint16_t*>(p.d)[row * p.ldd + f] = (uint16_t)f32x2_to_bf16x2(y, 0.0f);
    }
}

// ---------------------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------------------
template <int SPLIT>
__global__ void __launch_bounds__(kGaThreads, 1) gemm_act_kernel(const __grid_constant__ GemmActMaps maps, const __grid_constant__ GemmActParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    GemmActSmem& sm = *reinterpret_cast<GemmActSmem*>(smem + kGaRing);
    volatile uint32_t* abort_flag = &sm.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_rank(), rank = crank & 1u, leader = crank & ~1u;
    const int part = (int)(crank >> 1);                            // of K
    const int unit = blockIdx.x / (2 * SPLIT), units = gridDim.x / (2 * SPLIT);
    const int tiles = p.np * p.nq;
    const int s0 = (int)((int64_t)p.stages * part / SPLIT), s1 = (int)((int64_t)p.stages * (part + 1) / SPLIT);

    if (threadIdx.x == 8 * 32) {
        for (int s = 0; s < kGaStages; ++s) {
            mbar_init(smem_u32(&sm.full[s]), 1);
            mbar_init(smem_u32(&sm.empty[s]), 1);
            sm.stage_tx[s] = 0;
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&sm.tfull[b]), 1);
            mbar_init(smem_u32(&sm.tempty[b]), kGaEpiWarps + 1);   // and the other CTA's forwarded arrival
            mbar_init(smem_u32(&sm.edrained[b]), kGaEpiWarps);
        }
        mbar_init(smem_u32(&sm.done), 1);
        sm.abort = 0u;
        sm.peer_abort = 0u;
        sm.issued = 0u;
        sm.consumed = 0u;
        sm.runs = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&maps.p);
        prefetch_map(&maps.q[2]);
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    cluster_arrive();   // this CTA's barriers and TMEM are there
    // what comes before overlaps the end of the kernel before, what follows touches memory that it may have written
    griddep_wait();
    griddep_launch();
    cluster_wait();     // and the others'
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const int run = p.run;   // stages per accumulator

    if (warp == 0) {
        // ------------------------------- producer (both CTAs) --------------------------------
        if (elect_one()) {
            int g = 0, s = 0;              // stages issued, the next one's slot
            uint32_t parity = 1;           // of the slot's `empty`: at first there is no use to wait for
            const uint32_t base = smem_u32(smem), empty = smem_u32(&sm.empty[0]), full = smem_u32(&sm.full[0]),
                           leader_full = map_rank(full, leader);
            bool ok = true;
            for (int t = unit; ok && t < tiles; t += units) {
                const GaTile c = ga_tile(p, t);
                const int half = c.n >> 1, p0 = c.p0 + (int)rank * 128, q0 = c.q0 + (int)rank * half;
                const int qbox = half <= 32 ? 0 : half <= 64 ? 1 : 2;
                const uint32_t tx = (uint32_t)(kGaOpBytes + (4096 << qbox));
                for (int k = s0; k < s1; ++k) {
                    if (!mbar_wait(empty + 8u * s, parity, abort_flag, p.flags, p.budget_ns)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_expect_tx(full + 8u * s, 2u * tx);
                    sm.stage_tx[s] = tx;
                    const uint32_t dst = base + (uint32_t)(s * kGaStageBytes), bar = leader_full + 8u * s;
                    ++g;
                    if (++s == kGaStages) {
                        s = 0;
                        parity ^= 1u;
                    }
                    tma_load_2d_pair(dst, &maps.p, k * kGaK, p0, bar);
                    tma_load_2d_pair(dst + kGaOpBytes, &maps.q[qbox], k * kGaK, q0, bar);
                }
            }
            sm.issued = (uint32_t)g;   // read by the drain, after the cluster barrier
            // the releases of the last stages, which the leader's MMAs signal in both CTAs, land before the end
            for (int k = max(0, g - kGaStages); ok && k < g; ++k)
                ok = mbar_wait(empty + 8u * (k % kGaStages), (uint32_t)(k / kGaStages) & 1u, abort_flag, p.flags, p.budget_ns);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            // ------------------------------- MMA issuer (leader) -----------------------------
            if (elect_one()) {
                const uint32_t base = smem_u32(smem);
                const uint64_t pdesc = desc_k_major(base), qdesc = desc_k_major(base + kGaOpBytes);
                constexpr uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(256 >> 4) << 24);
                int it = 0, s = 0;
                uint32_t parity = 0, consumed = 0;   // of the slot's `full`; stages committed
                const uint32_t full = smem_u32(&sm.full[0]), empty = smem_u32(&sm.empty[0]);
                bool ok = true;
                for (int t = unit; ok && t < tiles; t += units) {
                    const GaTile c = ga_tile(p, t);
                    const uint32_t idesc = idesc0 | ((uint32_t)(c.n >> 3) << 17);
                    for (int k = s0; k < s1; ++it) {
                        const int end = min(s1, k + run);
                        const int buf = it & 1;
                        if (!mbar_wait<true>(smem_u32(&sm.tempty[buf]), ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag, p.flags, p.budget_ns)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t acc = tmem + 256u * buf;
                        uint32_t add = 0;   // an accumulator's first MMA stores
                        for (; k < end; ++k) {
                            if (!mbar_wait(full + 8u * s, parity, abort_flag, p.flags, p.budget_ns)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            const uint64_t off = (uint64_t)((uint32_t)(s * kGaStageBytes) >> 4);
#pragma unroll
                            for (int j = 0; j < kGaK / 16; ++j)   // products past K are zero
                                mma_bf16_pair(acc, pdesc + off + 2 * j, qdesc + off + 2 * j, idesc, j ? 1u : add);
                            add = 1;
                            commit_pair(empty + 8u * s, leader);
                            ++consumed;
                            if (++s == kGaStages) {
                                s = 0;
                                parity ^= 1u;
                            }
                        }
                        if (!ok) break;
                        commit_pair(smem_u32(&sm.tfull[buf]), leader);
                    }
                }
                mma_commit_local(smem_u32(&sm.done));
                mbar_wait(smem_u32(&sm.done), 0u, abort_flag, p.flags, kGaDrainNs, false);
                sm.consumed = consumed;
                sm.runs = (uint32_t)it;
            }
            __syncwarp();
        } else {
            // this CTA's read accumulators as one remote arrival each
            int it = 0;
            bool ok = true;
            for (int t = unit; ok && t < tiles; t += units) {
                for (int k = s0; k < s1; k += run, ++it) {
                    // a cluster's one tile: its last accumulator is read behind barriers that this warp takes part in
                    if (SPLIT > 1 && k + run >= s1) break;
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&sm.edrained[it & 1]), (uint32_t)(it >> 1) & 1u, abort_flag,
                                                           p.flags, p.budget_ns))) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_remote(map_rank(smem_u32(&sm.tempty[it & 1]), leader));
                    __syncwarp();
                }
            }
        }
    }
    // ------------------------------- epilogue (both CTAs) ------------------------------------
    // Warps 2-17: the warp's TMEM lanes are 32 q .. 32 q + 31, its columns 16 from c0 and from every 64 further.
    // Sums that take several runs (or parts) are joined in registers and put back where the last run stood, so that
    // the tile is finished from TMEM, 16 columns at a time: with the 64 sums of a warp still in registers, those of
    // the epilogue do not fit, and what is spilled goes to L2 with the output (8192 x 20480 x 5120: 1235 us).
    const bool epilogue = warp >= 2;
    const int q = warp & 3, c0 = ((warp - 2) >> 2) * 16;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    int it = 0;
    bool ok = true;
    // with SPLIT > 1 every warp comes by once, for the cluster's barriers
    for (int t = unit; (epilogue || SPLIT > 1) && ok && t < tiles; t += units) {
        const GaTile c = ga_tile(p, t);
        const auto ready = [&]() {   // the next accumulator is complete
            const bool full = mbar_wait(smem_u32(&sm.tfull[it & 1]), (uint32_t)(it >> 1) & 1u, abort_flag, p.flags, p.budget_ns);
            if (!__all_sync(0xFFFFFFFFu, full)) return false;
            tc_fence_after();
            return true;
        };
        const auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(rank == 0 ? &sm.tempty[it & 1] : &sm.edrained[it & 1]));
            ++it;
        };
        if (SPLIT > 1 || s1 - s0 > run) {
            float acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0.0f;
            if (epilogue)
                for (int k = s0; k < s1; k += run) {
                    if (!(ok = ready())) break;
#pragma unroll
                    for (int h = 0; h < 8; ++h) {
                        const int at = c0 + 64 * (h >> 1) + 8 * (h & 1);
                        if (at >= c.qn) break;
                        float v[8];
                        tmem_ld8(lanes + 256u * (it & 1) + (uint32_t)at, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[8 * h + i] += v[i];
                    }
                    if (k + run < s1) release();
                }
            if constexpr (SPLIT > 1) {
                // chunk (c0 / 16) + 4 h of 16 rows is finished by part (c0 / 16 + h) % SPLIT, in whose shared memory the
                // others' sums of it stand at [sender][h * 4 / SPLIT + c0 / 16 / SPLIT][row][feature]
                constexpr uint32_t kChunk = 16 * 128 * 4;
                const int group = c0 >> 4;
                const uint32_t mine = (uint32_t)(q * 32 + lane) * 4u;
                const auto place = [&](int owner, int sender, int h) {
                    const int slot = sender < owner ? sender : sender - 1;
                    return smem_u32(smem) + (uint32_t)(slot * (16 / SPLIT) + h * (4 / SPLIT) + group / SPLIT) * kChunk + mine;
                };
                __syncwarp();
                cluster_arrive();
                cluster_wait();      // the products of all parts are done: the rings are free
                if (epilogue && ok) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int owner = (group + h) % SPLIT;
                        if (c0 + 64 * h >= c.qn || owner == part) continue;
                        const uint32_t at = map_rank(place(owner, part, h), (uint32_t)(2 * owner) + rank);
#pragma unroll
                        for (int i = 0; i < 16; ++i) st_cluster_f32(at + 512u * i, acc[16 * h + i]);
                    }
                }
                __syncwarp();
                cluster_arrive();
                cluster_wait();      // and what each part finishes is there
                if (epilogue && ok) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        if (c0 + 64 * h >= c.qn || (group + h) % SPLIT != part) continue;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float sum = 0.0f;
#pragma unroll
                            for (int s = 0; s < SPLIT; ++s) {   // in the order of the parts
                                float v = acc[16 * h + i];
                                if (s != part) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(place(part, s, h) + 512u * i));
                                sum = s == 0 ? v : sum + v;
                            }
                            acc[16 * h + i] = sum;
                        }
                    }
                }
            }
            if (epilogue && ok) {
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    const int at = c0 + 64 * (h >> 1) + 8 * (h & 1);
                    if (at >= c.qn) break;
                    tmem_st8(lanes + 256u * (it & 1) + (uint32_t)at, acc + 8 * h);
                }
                tmem_st_wait();
            }
        } else {
            ok = ready();
        }
        if (!epilogue || !ok) continue;
        const int f = c.p0 + (int)rank * 128 + q * 32 + lane;
        const float bias = p.bias && f < p.N ? p.bias[f] : 0.0f;
        const bool whole = p.pairs && f - lane + 32 <= p.N;
#pragma unroll 1
        for (int h = 0; h < 4; ++h) {
            const int at = c0 + 64 * h;
            if (at >= c.qn) break;
            if (SPLIT > 1 && ((c0 >> 4) + h) % SPLIT != part) continue;
            float v[16];
            tmem_ld16(lanes + 256u * (it & 1) + (uint32_t)at, v);
            tmem_ld_wait();
            if (whole && at + 16 <= c.qn) {
                finish16(v, p, c.q0 + at, f, bias);
            } else {
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    if (at + i < c.qn) finish_edge(v[i], v[i + 1], v[i + 2], v[i + 3], p, c.q0 + at + i, c.qn - (at + i), f, bias);
            }
        }
        release();
    }

    // Each warp hands an abort that it has seen to the pair's leader.  No arrival may land in a CTA that has ended: those that
    // the MMAs signal are waited for by the producers and the epilogues, after an abort by the drain; those
    // that the other CTA's warp 1 makes on the leader's barriers are ordered before its end by a release here, as is what the drain
    // reads.  The epilogue arrives without one, since it makes no such arrival and would wait for its stores.
    const bool aborted = __any_sync(0xFFFFFFFFu, *abort_flag != 0u);
    if (aborted && rank == 1 && lane == 0) st_cluster_u32(map_rank(smem_u32(&sm.peer_abort), leader), 1u);
    __syncwarp();
    tc_fence_before();
    if (aborted || warp < 2)
        cluster_arrive();   // both producers have stopped and published what they issued
    else
        cluster_arrive_relaxed();
    cluster_wait();
    if (warp == 0 && lane == 0 && (sm.abort || sm.peer_abort)) {
        // Drain after an abort: every copy lands before its CTA exits.  Copies of both CTAs land on the leader's barriers.  A
        // producer is at most a ring ahead of the MMAs, so only the last uses of its stages can be outstanding; a stage that only
        // the other CTA issued has its arrival made here, one that only the leader issued has the other's bytes cancelled.
        const uint32_t consumed = ld_cluster_u32(map_rank(smem_u32(&sm.consumed), leader)), runs = ld_cluster_u32(map_rank(smem_u32(&sm.runs), leader));
        for (int k = max(0, (int)consumed - kGaStages); k < (int)consumed; ++k)
            mbar_wait(smem_u32(&sm.empty[k % kGaStages]), (uint32_t)(k / kGaStages) & 1u, abort_flag, p.flags, kGaDrainNs, false);
        for (int i = max(0, (int)runs - 2); i < (int)runs; ++i)
            mbar_wait(smem_u32(&sm.tfull[i & 1]), (uint32_t)(i >> 1) & 1u, abort_flag, p.flags, kGaDrainNs, false);
        if (rank == 0) {
            const int gl = (int)sm.issued, gp = (int)ld_cluster_u32(map_rank(smem_u32(&sm.issued), leader + 1)), gm = max(gl, gp);
            for (int k = max(0, gm - kGaStages); k < gm; ++k) {
                const int s = k % kGaStages;
                const uint32_t bar = smem_u32(&sm.full[s]);
                const uint32_t tx = k < gl ? sm.stage_tx[s] : ld_cluster_u32(map_rank(smem_u32(&sm.stage_tx[s]), leader + 1));
                if (k >= gl) mbar_expect_tx(bar, tx);
                else if (k >= gp) mbar_complete_tx(bar, tx);
                mbar_wait(bar, (uint32_t)(k / kGaStages) & 1u, abort_flag, p.flags, kGaDrainNs, false);
            }
        }
    }
    __syncwarp();
    cluster_arrive_relaxed();
    cluster_wait();   // all are done with TMEM, barriers and each other's shared memory
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ---------------------------------------------------------------------------------------
// few rows: the weights are read once and the rows cost nothing against them
//
// A CTA takes 16 features; its warps cut K into chunks of 64 and join their sums through shared memory, so that a few
// hundred features are spread over most SMs, with no tensor maps, TMEM or clusters to set up.  The products run on mma.sync
// m16n8k16 (features x groups of 8 rows): the work is bound by memory, and the fragments come straight from global
// memory in 16-byte loads.  For that the K positions within a chunk are permuted, the same way for both operands: lane
// (g, t) holds 8 consecutive products of feature g (and g + 8) and of row g, which serve as its fragment slots of
// two MMAs.
// ---------------------------------------------------------------------------------------
constexpr int kGfRun = 512;   // products that a warp accumulates on the tensor core before they are joined in fp32

struct GemmActFewParams {
    const uint16_t* a;
    const uint16_t* b;
    int64_t lda, ldb;
    int32_t K;
    GemmActParams e;          // the epilogue's
};

__device__ __forceinline__ uint4 gf_stream(const uint16_t* p) {   // weights: read once
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ void gf_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NG: groups of 8 rows in one pass over the weights; with more rows there are more passes (their weights then come from L2)
template <int NG, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 32 / WARPS) gemm_act_few_kernel(const GemmActFewParams p) {
    __shared__ float part[WARPS][NG * 8][17];   // [warp][row][feature], padded
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int f0 = blockIdx.x * 16, N = p.e.N;
    // features past the end read the last one
    const uint16_t* w0 = p.b + (int64_t)min(f0 + g, N - 1) * p.ldb + 8 * t;
    const uint16_t* w1 = p.b + (int64_t)min(f0 + g + 8, N - 1) * p.ldb + 8 * t;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int lo = 0; lo < p.e.M; lo += 8 * NG) {
        const int rows = min(8 * NG, p.e.M - lo), groups = (rows + 7) >> 3;
        const uint16_t* x = p.a + (int64_t)(lo + g) * p.lda + 8 * t;   // row g of each group
        // runs of kGfRun products, joined in the warp's own part of shared memory (registers are full)
#pragma unroll 1
        for (int k = 64 * warp, run = 0; run == 0 || k < p.K; ++run) {
            const int end = min(p.K, k + kGfRun * WARPS);
            float acc[NG][4] = {};
#pragma unroll 1
            for (; k < end; k += 64 * WARPS) {
                const bool in0 = k + 8 * t < p.K, in1 = k + 32 + 8 * t < p.K;
                const uint4 a00 = in0 ? gf_stream(w0 + k) : zero, a01 = in1 ? gf_stream(w0 + k + 32) : zero;
                const uint4 a10 = in0 ? gf_stream(w1 + k) : zero, a11 = in1 ? gf_stream(w1 + k + 32) : zero;
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    if (i >= groups) break;
                    const bool row = 8 * i + g < rows;
                    const uint16_t* xi = x + (int64_t)(8 * i) * p.lda + k;
                    const uint4 b0 = row && in0 ? __ldg(reinterpret_cast<const uint4*>(xi)) : zero;
                    const uint4 b1 = row && in1 ? __ldg(reinterpret_cast<const uint4*>(xi + 32)) : zero;
                    gf_mma(acc[i], a00.x, a10.x, a00.y, a10.y, b0.x, b0.y);
                    gf_mma(acc[i], a00.z, a10.z, a00.w, a10.w, b0.z, b0.w);
                    gf_mma(acc[i], a01.x, a11.x, a01.y, a11.y, b1.x, b1.y);
                    gf_mma(acc[i], a01.z, a11.z, a01.w, a11.w, b1.z, b1.w);
                }
            }
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                if (i >= groups) break;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float& s = part[warp][8 * i + 2 * t + (j & 1)][g + 4 * (j & 2)];
                    s = run == 0 ? acc[i][j] : s + acc[i][j];
                }
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * rows; i += 32 * WARPS) {
            const int f = f0 + (i & 15), r = i >> 4, row = lo + r;
            if (f >= N) continue;
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) s += part[w][r][i & 15];
            if (p.e.bias) s += p.e.bias[f];
            if (p.e.pre) p.e.pre[(int64_t)row * p.e.ldpre + f] = (uint16_t)f32x2_to_bf16x2(s, 0.0f);
            s = act::wide(p.e.act, s);
            if (p.e.residual) {
                const int64_t at = (int64_t)row * p.e.ldr + f;
                s += p.e.res_fp32 ? reinterpret_cast<const float*>(p.e.residual)[at]
                                  : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p.e.residual)[at] << 16);
            }
            const int64_t at = (int64_t)row * p.e.ldd + f;
            if (p.e.out_fp32) reinterpret_cast<float*>(p.e.d)[at] = s;
            else reinterpret_cast<uint16_t*>(p.e.d)[at] = (uint16_t)f32x2_to_bf16x2(s, 0.0f);
        }
        __syncthreads();   // the next pass writes `part` again
    }
}

// ---------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------
constexpr int kGfRows = 16;      // rows up to which the kernel for few is taken
constexpr int kGfLongK = 2048;   // a K from which 16 warps cut it, where one wave of CTAs holds the launch

template <int SPLIT>
static cudaError_t launch_pairs(const GemmActMaps& maps, const GemmActParams& p, int clusters, cudaStream_t s) {
    static std::atomic<uint64_t> attr{0};
    auto kern = gemm_act_kernel<SPLIT>;
    if (cudaError_t e = host::ensure_smem(reinterpret_cast<const void*>(kern), kGaSmem, attr)) return e;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 2 * SPLIT;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(2 * SPLIT * clusters));
    cfg.blockDim = dim3(kGaThreads);
    cfg.dynamicSmemBytes = kGaSmem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

struct GaPlan {
    int split, wq;
};
// The row tiles' width and the parts of K: the least of waves x (stages x a stage's cycles + a tile's fixed ones)
static GaPlan ga_plan(int64_t M, int64_t N, int64_t stages, int sms) {
    const int64_t np = (N + 255) / 256;
    const int fit[3] = {sms / 2, sms / 4 - 1, sms / 8 - 1};   // clusters of 2, 4 and 8 CTAs at once
    GaPlan best{1, 256};
    double least = 1e300;
    for (int i = 0; i < 3; ++i) {
        const int split = 1 << i;
        if (split > stages || fit[i] < 1) break;
        for (int w = 256; w >= 32; w -= 32) {
            const int64_t nq = (M + w - 1) / w;
            const int wq = (int)(((M + nq - 1) / nq + 31) / 32 * 32);
            if (wq != w && w < 256) continue;   // an even cut of that many tiles has been seen
            const double waves = (double)((np * nq + fit[i] - 1) / fit[i]);
            const double cycles = std::max(320.0, 256.0 + wq) * (double)((stages + split - 1) / split) + (split > 1 ? 2500.0 : 1000.0);
            if (waves * cycles < least) {
                least = waves * cycles;
                best = GaPlan{split, wq};
            }
        }
    }
    return best;
}

cudaError_t launch_gemm_act(const GemmAct& g, cudaStream_t s) {
    GemmActParams p{};
    p.bias = g.bias;
    p.residual = g.residual;
    p.pre = g.pre;
    p.d = g.d;
    p.ldr = g.ldr;
    p.ldpre = g.ldpre;
    p.ldd = g.ldd;
    p.M = (int32_t)g.M;
    p.N = (int32_t)g.N;
    p.act = g.act;
    p.out_fp32 = g.out_fp32;
    p.res_fp32 = g.res_fp32;
    p.pairs = (g.out_fp32 || g.ldd % 2 == 0) && (!g.pre || g.ldpre % 2 == 0) && (!g.residual || g.ldr % 2 == 0);
    p.flags = g.flags;
    p.budget_ns = g.budget_ns;
    if (g.M <= kGfRows) {
        const GemmActFewParams f{g.a, g.b, g.lda, g.ldb, (int32_t)g.K, p};
        const unsigned blocks = (unsigned)((g.N + 15) / 16);
        const bool long_k = g.K >= kGfLongK && blocks <= 2u * host::sm_count();
        if (g.M <= 8) {
            if (long_k) gemm_act_few_kernel<1, 16><<<blocks, 512, 0, s>>>(f);
            else gemm_act_few_kernel<1, 8><<<blocks, 256, 0, s>>>(f);
        } else {
            if (long_k) gemm_act_few_kernel<2, 16><<<blocks, 512, 0, s>>>(f);
            else gemm_act_few_kernel<2, 8><<<blocks, 256, 0, s>>>(f);
        }
        return cudaGetLastError();
    }
    const int sms = host::sm_count();
    const int64_t stages = (g.K + kGaK - 1) / kGaK;
    const GaPlan plan = ga_plan(g.M, g.N, stages, sms);
    p.stages = (int32_t)stages;
    // even runs: a tile is finished under the first run of the next one
    const int64_t part = (stages + plan.split - 1) / plan.split, most = (g.out_fp32 ? kGaRunK : kGaRunBf16) / kGaK;
    const int64_t runs = (part + most - 1) / most;
    p.run = (int32_t)((part + runs - 1) / runs);
    p.wq = plan.wq;
    p.np = (int32_t)((g.N + 255) / 256);
    p.nq = (int32_t)((g.M + plan.wq - 1) / plan.wq);
    GemmActMaps maps;
    const int64_t bdims[2] = {g.K, g.N}, bstrides[1] = {g.ldb}, adims[2] = {g.K, g.M}, astrides[1] = {g.lda};
    const uint32_t bbox[2] = {64, 128};
    if (!host::bf16_map(&maps.p, g.b, 2, bdims, bstrides, bbox)) return cudaErrorInvalidValue;
    for (int i = 0; i < 3; ++i) {
        const uint32_t abox[2] = {64, 32u << i};
        if (!host::bf16_map(&maps.q[i], g.a, 2, adims, astrides, abox)) return cudaErrorInvalidValue;
    }
    const int64_t tiles = (int64_t)p.np * p.nq;
    switch (plan.split) {
        case 1: return launch_pairs<1>(maps, p, (int)std::min<int64_t>(tiles, sms / 2), s);
        case 2: return launch_pairs<2>(maps, p, (int)tiles, s);
        default: return launch_pairs<4>(maps, p, (int)tiles, s);
    }
}

// ---------------------------------------------------------------------------------------
// the activation's and the bias' gradient: dh = dy act'(h) in bf16, db[f] (+)= sum over the rows of dy act'(h)
//
// A CTA takes 64 features (8 lanes of 8) of a run of rows; its threads' sums over their rows are joined in shared memory, and the
// runs' by a second kernel, in a fixed order.
// ---------------------------------------------------------------------------------------
constexpr int kAbThreads = 256;

template <int ACT>
__global__ void __launch_bounds__(kAbThreads) act_bwd_kernel(const ActBwd p, int rows_per) {
    __shared__ float part[kAbThreads / 8][64 + 1];
    const int c = threadIdx.x & 7, r = threadIdx.x >> 3;
    const int64_t col = (int64_t)blockIdx.x * 64 + 8 * c;
    const int64_t t0 = (int64_t)blockIdx.y * rows_per, t1 = min(p.rows, t0 + rows_per);
    float sum[8] = {};
    if (col < p.n)
        for (int64_t t = t0 + r; t < t1; t += kAbThreads / 8) {
            const uint4 g4 = *reinterpret_cast<const uint4*>(p.dy + t * p.lddy + col);   // dh may be dy
            uint4 h4 = make_uint4(0, 0, 0, 0);
            if (ACT != kActNone) h4 = __ldg(reinterpret_cast<const uint4*>(p.pre + t * p.ldpre + col));
            const uint32_t g[4] = {g4.x, g4.y, g4.z, g4.w}, h[4] = {h4.x, h4.y, h4.z, h4.w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x = bf16_lo(h[i]), y = bf16_hi(h[i]);
                act::slope_pair<ACT>(x, y);
                x *= bf16_lo(g[i]);
                y *= bf16_hi(g[i]);
                sum[2 * i] += x;
                sum[2 * i + 1] += y;
                o[i] = f32x2_to_bf16x2(x, y);
            }
            if (p.dh) *reinterpret_cast<uint4*>(p.dh + t * p.lddh + col) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    if (!p.dbias) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) part[r][8 * c + i] = sum[i];
    __syncthreads();
    if (threadIdx.x < 64 && (int64_t)blockIdx.x * 64 + threadIdx.x < p.n) {
        float s = 0.0f;
        for (int i = 0; i < kAbThreads / 8; ++i) s += part[i][threadIdx.x];
        p.scratch[(int64_t)blockIdx.y * p.n + (int64_t)blockIdx.x * 64 + threadIdx.x] = s;
    }
}

__global__ void __launch_bounds__(256) act_bwd_join_kernel(const ActBwd p, int runs) {
    const int64_t f = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (f >= p.n) return;
    float s = p.accumulate ? p.dbias[f] : 0.0f;
    for (int i = 0; i < runs; ++i) s += p.scratch[(int64_t)i * p.n + f];
    p.dbias[f] = s;
}

cudaError_t launch_act_bwd(const ActBwd& p, cudaStream_t s) {
    const int64_t cols = (p.n + 63) / 64;
    const int64_t want = std::max<int64_t>(1, 8 * host::sm_count() / cols);   // CTAs in all
    const int64_t runs = std::min<int64_t>({(int64_t)kActBwdRuns, want, (p.rows + 31) / 32});
    const int rows_per = (int)((p.rows + runs - 1) / runs);
    const int used = (int)((p.rows + rows_per - 1) / rows_per);
    const dim3 grid((unsigned)cols, (unsigned)used);
    switch (p.act) {
        case kActNone: act_bwd_kernel<kActNone><<<grid, kAbThreads, 0, s>>>(p, rows_per); break;
        case kActRelu: act_bwd_kernel<kActRelu><<<grid, kAbThreads, 0, s>>>(p, rows_per); break;
        case kActRelu2: act_bwd_kernel<kActRelu2><<<grid, kAbThreads, 0, s>>>(p, rows_per); break;
        case kActGelu: act_bwd_kernel<kActGelu><<<grid, kAbThreads, 0, s>>>(p, rows_per); break;
        case kActSilu: act_bwd_kernel<kActSilu><<<grid, kAbThreads, 0, s>>>(p, rows_per); break;
    }
    if (cudaError_t e = cudaGetLastError()) return e;
    if (!p.dbias) return cudaSuccess;
    act_bwd_join_kernel<<<(unsigned)((p.n + 255) / 256), 256, 0, s>>>(p, used);
    return cudaGetLastError();
}

}  // namespace nvfp4
