// gemm_act.cu -- the bf16 product with bias, activation and residual in its epilogue (sm_100a):
//   h[t][f] = sum_k A[t][k] B[f][k] + bias[f],   D = act(h) + residual,   pre = h in bf16
// and the gradients of activation and bias.
//
// Three kernels for the product: SM pairs for many rows, one CTA per tile where there are few or small tiles, one without
// tensor memory for up to 16 rows (the rules stand at ga_plan and kGfRows).
//
// SM pairs (tcgen05.mma.cta_group::2, kind::f16, fp32 accumulators in TMEM).  The features are the MMA's M side, 256
// per tile, 128 per CTA; the rows are its N side, up to 256 per tile in steps of 32.  So few rows cost few MMA cycles, a
// TMEM lane is a feature and the epilogue's bias a register, and the 32 lanes of a warp hold 32 neighbours of one output
// row: bias, activation, residual and stores are done from registers, with no staging in shared memory.
//
// Warps: 0 TMA producer (6 stages of 64 products, 192 KiB per CTA), 1 MMA issuer in the pair's leader, in the other CTA it
// forwards "accumulator read"; 2-17 epilogue.  The accumulator is double-buffered (2 x 256 TMEM columns).  The tensor
// core truncates as it accumulates (5e-7 after 512 products, 2e-6 after 2048, 9e-6 after 8192, relative), so an accumulator
// holds at most 512 products with fp32 output and 4096 with bf16, whose half step is 2e-3 at least; the epilogue joins such
// runs, rounded to nearest, while the next one is under way.  Runs are cut evenly, since a tile is finished under the first
// run of the next one: with 1024 products the MMAs waited for the epilogue (8192 x 20480 x 5120, gelu, pre: 1261 us, now
// 1145 to 1160; the product alone 1088 to 1105, cuBLAS' 1080).
//
// Either operand may have K outermost (a layer's gradients take weights, gradients and activations as they lie): its tiles
// are then MN-major blocks of 64 x 64, by instantiations of their own (KOUT).  Input gradient 587 x 96 x 5120 8.3 us, 4096 x 5120 x
// 5120 146 (1.47 PFLOP/s); weight gradient of 256 x 256 over 16384 rows 15.6.
//
// Where there are fewer tiles than SMs, a cluster takes one tile and each pair (or CTA) of it a part of K.  The sums
// meet in shared memory: no workspace, no atomics, no waiting on memory (tile_epilogue).
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

// Operands with K outermost: 64 features or rows of 64 products are a block of 64 x 64, the MMA's MN-major layout (zeros past the ends)
constexpr uint32_t kGaKnBlock = 8192, kGaKnStep = 2048 >> 4;
__host__ __device__ constexpr uint32_t ga_row_bytes(bool a_km, int rows) {   // of a stage
    return a_km ? kGaKnBlock * (uint32_t)((rows + 63) / 64) : 2u * kGaK * (uint32_t)rows;
}

struct GemmActParams {
    const float* bias;
    const void* residual;
    uint16_t* pre;
    void* d;
    int64_t ldr, ldpre, ldd;
    int32_t M, N;
    int32_t stages, run;    // of K, and of an accumulator
    int32_t np, nq, wq;     // feature tiles, row tiles and their width
    int32_t split, per;     // parts of K; chunks of 16 rows that a part finishes at most
    int32_t part_stages, longer;   // of a part, and how many have one more
    int32_t ring;           // one CTA per tile: stages of the ring
    uint32_t tmem_cols;
    int32_t act, out_fp32, res_fp32;
    int32_t pairs;          // D, pre and the residual can be taken two features at a time
    int32_t b_kn, a_km;     // B is [K][N], A is [K][M]
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
constexpr int kGaClusterStages = 4;                      // where an inbox takes the room of two
constexpr int kInbox = 96 * 1024;                        // of a part's CTA: the sums of up to 3 (pairs) or 7 others
constexpr int kGaSmem = kGaRing + (int)sizeof(GemmActSmem) + 1024;
constexpr int kGaClusterSmem = kGaClusterStages * kGaStageBytes + kInbox + (int)sizeof(GemmActSmem) + 1024;
static_assert(kGaSmem <= 232448 && kGaClusterSmem <= 232448, "shared memory");

struct GemmActMaps {
    CUtensorMap p, q;       // features in boxes of 128; rows in boxes of a tile's (a pair's: half)
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
// In a loop that moves the values along, 8 at a time: a launch of few tiles runs each of these instructions once or twice, and
// fetches them for that.
template <int ACT>
__device__ __forceinline__ void act16(float* v) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = v[j];
#pragma unroll
        for (int j = 0; j < 8; j += 2) act::pair<ACT>(w[j], w[j + 1]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = v[j + 8];
            v[j + 8] = w[j];
        }
    }
}
__device__ __forceinline__ void act16(int act, float* v) {
    switch (act) {
        case kActRelu: act16<kActRelu>(v); break;
        case kActRelu2: act16<kActRelu2>(v); break;
        case kActGelu: act16<kActGelu>(v); break;
        case kActSilu: act16<kActSilu>(v); break;
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

// v: sums of rows row0 .. row0 + 15 of feature f, the first n of which exist.  whole: all 16 do and all of the warp's 32
// features, and leading dimensions are even; else each lane takes its own feature, element by element.
__device__ __forceinline__ void finish16(float* v, const GemmActParams& p, int row0, int n, int f, float bias, bool whole) {
    const int odd = threadIdx.x & 1, fe = f - odd;
    const uint32_t select = odd ? 0x3276u : 0x5410u;
    const bool in = f < p.N;
    // the residual first: its loads are under way during the rest
    float w[16];
    const bool words = whole && !p.res_fp32;
    if (p.residual) {
        if (words) {
            const uint16_t* r = reinterpret_cast<const uint16_t*>(p.residual) + (row0 + odd) * p.ldr + fe;
#pragma unroll
            for (int i = 0; i < 8; ++i, r += 2 * p.ldr) w[i] = __uint_as_float(*reinterpret_cast<const uint32_t*>(r));
        } else if (whole) {
            const float* r = reinterpret_cast<const float*>(p.residual) + row0 * p.ldr + f;
#pragma unroll
            for (int i = 0; i < 16; ++i, r += p.ldr) w[i] = *r;
        } else if (p.res_fp32) {
            const float* r = reinterpret_cast<const float*>(p.residual) + row0 * p.ldr + f;
#pragma unroll
            for (int i = 0; i < 16; ++i, r += p.ldr) w[i] = in && i < n ? *r : 0.0f;
        } else {
            const uint16_t* r = reinterpret_cast<const uint16_t*>(p.residual) + row0 * p.ldr + f;
#pragma unroll
            for (int i = 0; i < 16; ++i, r += p.ldr) w[i] = in && i < n ? __uint_as_float((uint32_t)*r << 16) : 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += bias;
    if (p.pre) {
        if (whole) {
            put_words(p.pre + (row0 + odd) * p.ldpre + fe, p.ldpre, v, select);
        } else {
            uint16_t* at = p.pre + row0 * p.ldpre + f;
#pragma unroll
            for (int i = 0; i < 16; ++i, at += p.ldpre)
                if (in && i < n) *at = (uint16_t)f32x2_to_bf16x2(v[i], 0.0f);
        }
    }
    act16(p.act, v);
    if (p.residual) {
        if (words) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t u = traded(__float_as_uint(w[i]), select);
                v[2 * i] += bf16_lo(u);
                v[2 * i + 1] += bf16_hi(u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] += w[i];
        }
    }
    if (p.out_fp32) {
        float* at = reinterpret_cast<float*>(p.d) + row0 * p.ldd + f;
        if (whole) {
#pragma unroll
            for (int i = 0; i < 16; ++i, at += p.ldd) *at = v[i];
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i, at += p.ldd)
                if (in && i < n) *at = v[i];
        }
    } else if (whole) {
        put_words(reinterpret_cast<uint16_t*>(p.d) + (row0 + odd) * p.ldd + fe, p.ldd, v, select);
    } else {
        uint16_t* at = reinterpret_cast<uint16_t*>(p.d) + row0 * p.ldd + f;
#pragma unroll
        for (int i = 0; i < 16; ++i, at += p.ldd)
            if (in && i < n) *at = (uint16_t)f32x2_to_bf16x2(v[i], 0.0f);
    }
}

// ---------------------------------------------------------------------------------------
// A tile's epilogue, for the warps of both kernels below.  The warp's TMEM lanes start at `lanes`, its columns (rows of
// the output) are the chunks of 16 numbered group, group + G, ...
//
// Sums of several runs are joined in registers and put back where the last run stood, so that the tile is finished from
// TMEM, 16 columns at a time: with 64 sums of a lane still in registers, those of the epilogue do not fit, and what is
// spilled goes to L2 with the output (8192 x 20480 x 5120: 1235 us, without 1107).
//
// CLUSTER: the tile's K is cut into `split` parts.  Chunk c is finished by part c % split, to which the others send their
// sums of it, through the cluster's network, to [sender][c / split][row][feature] at `inbox`; they are added in the order of the
// parts.  Every warp of the cluster comes by, for the barriers: one that each has arrived at when it began (no
// sums before their CTA runs), one behind the sends.
// ---------------------------------------------------------------------------------------
constexpr uint32_t kChunkBytes = 16 * 128 * 4;
struct EpilogueTile {
    int q0, qn, f;           // first row, rows, this lane's feature
    int group, runs;         // the warp's first chunk; accumulators of the tile
    int split, part, per;    // per: chunks of a part at most
    uint32_t rank_step, rank0;   // part s stands at cluster rank s * rank_step + rank0
    uint32_t inbox;          // shared::cta address, plus 4 bytes for each feature before this lane's
    uint32_t lanes, buf_cols;
};
template <int G, bool CLUSTER, class Ready, class Release>
__device__ __forceinline__ bool tile_epilogue(const GemmActParams& p, const EpilogueTile& e, bool works, int& it, const Ready& ready, const Release& release) {
    bool ok = true;
    if (works) {
        if (e.runs > 1) {
            float acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0.0f;
            for (int r = 0; r < e.runs; ++r) {
                if (!(ok = ready())) break;
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    const int at = 16 * (e.group + G * (h >> 1)) + 8 * (h & 1);
                    if (at >= e.qn) break;
                    float v[8];
                    tmem_ld8(e.lanes + e.buf_cols * (it & 1) + (uint32_t)at, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[8 * h + i] += v[i];
                }
                if (r + 1 < e.runs) release();
            }
            if (ok) {
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    const int at = 16 * (e.group + G * (h >> 1)) + 8 * (h & 1);
                    if (at >= e.qn) break;
                    tmem_st8(e.lanes + e.buf_cols * (it & 1) + (uint32_t)at, acc + 8 * h);
                }
                tmem_st_wait();
            }
        } else {
            ok = ready();
        }
    }
    const uint32_t from = e.lanes + e.buf_cols * (it & 1);
    if constexpr (CLUSTER) {
        __syncwarp();
        cluster_wait();
        if (works && ok) {
            int owner = e.group, row = 0;   // c % split, c / split
#pragma unroll 1
            for (int c = e.group; 16 * c < e.qn; c += G, owner += G) {
                while (owner >= e.split) {
                    owner -= e.split;
                    ++row;
                }
                if (owner == e.part) continue;
                float v[16];
                tmem_ld16(from + (uint32_t)(16 * c), v);
                const int slot = e.part < owner ? e.part : e.part - 1;
                const uint32_t at = map_rank(e.inbox + (uint32_t)(slot * e.per + row) * kChunkBytes, (uint32_t)owner * e.rank_step + e.rank0);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) st_cluster_f32(at + 512u * i, v[i]);
            }
        }
        tc_fence_before();
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        tc_fence_after();
    }
    if (!works || !ok) return ok;
    const float bias = p.bias && e.f < p.N ? p.bias[e.f] : 0.0f;
    const bool whole = p.pairs && (e.f & ~31) + 32 <= p.N;
    // in a cluster the part's own chunks, part, part + split, ..., are dealt out anew over the warps of a lane quarter
    const int step = CLUSTER ? G * e.split : G;
    int row = e.group;
#pragma unroll 1
    for (int c = CLUSTER ? e.part + e.group * e.split : e.group; 16 * c < e.qn; c += step, row += G) {
        float v[16];
        tmem_ld16(from + (uint32_t)(16 * c), v);
        tmem_ld_wait();
        if constexpr (CLUSTER) {
            float own[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                own[i] = v[i];
                v[i] = e.part == 0 ? own[i] : 0.0f;
            }
#pragma unroll 1
            for (int slot = 0; slot < e.split - 1; ++slot) {
                const uint32_t at = e.inbox + (uint32_t)(slot * e.per + row) * kChunkBytes;
                float w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(w[i]) : "r"(at + 512u * i));
                const bool mine = slot + 1 == e.part;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    v[i] += w[i];
                    if (mine) v[i] += own[i];
                }
            }
        }
        finish16(v, p, e.q0 + 16 * c, e.qn - 16 * c, e.f, bias, whole && 16 * c + 16 <= e.qn);
    }
    return true;
}

// ---------------------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------------------
// KOUT: operands with K outermost, by p.b_kn and p.a_km (looked up in every call, they cost 8192 x 20480 x 5120 10 us of 1137)
template <bool CLUSTER, bool KOUT>
__global__ void __launch_bounds__(kGaThreads, 1) gemm_act_kernel(const __grid_constant__ GemmActMaps maps, const __grid_constant__ GemmActParams p) {
    extern __shared__ uint8_t smem_raw[];
    const bool b_kn = KOUT && p.b_kn, a_km = KOUT && p.a_km;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // in a cluster of several pairs: four stages, and the inbox behind them
    constexpr int kStages = CLUSTER ? kGaClusterStages : kGaStages;
    GemmActSmem& sm = *reinterpret_cast<GemmActSmem*>(smem + kStages * kGaStageBytes + (CLUSTER ? kInbox : 0));
    volatile uint32_t* abort_flag = &sm.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_rank(), rank = crank & 1u, leader = crank & ~1u;
    const int split = CLUSTER ? p.split : 1, part = CLUSTER ? (int)(crank >> 1) : 0;   // of K
    const int unit = CLUSTER ? (int)blockIdx.x / (2 * split) : (int)blockIdx.x >> 1, units = CLUSTER ? (int)gridDim.x / (2 * split) : (int)gridDim.x >> 1;
    const int tiles = p.np * p.nq;
    const int s0 = CLUSTER ? part * p.part_stages + min(part, p.longer) : 0, s1 = CLUSTER ? s0 + p.part_stages + (part < p.longer) : p.stages;

    if (threadIdx.x == 8 * 32) {
        for (int s = 0; s < kStages; ++s) {
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
        prefetch_map(&maps.q);
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
    if (CLUSTER) cluster_arrive_relaxed();   // for the epilogue
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
                const uint32_t tx = (uint32_t)kGaOpBytes + ga_row_bytes(a_km, p.wq >> 1);   // rows of the box past the tile's are not used
                for (int k = s0; k < s1; ++k) {
                    if (!mbar_wait(empty + 8u * s, parity, abort_flag, p.flags, p.budget_ns)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_expect_tx(full + 8u * s, 2u * tx);
                    sm.stage_tx[s] = tx;
                    const uint32_t dst = base + (uint32_t)(s * kGaStageBytes), bar = leader_full + 8u * s;
                    ++g;
                    if (++s == kStages) {
                        s = 0;
                        parity ^= 1u;
                    }
                    if (b_kn) {
                        tma_load_2d_pair(dst, &maps.p, p0, k * kGaK, bar);
                        tma_load_2d_pair(dst + kGaKnBlock, &maps.p, p0 + 64, k * kGaK, bar);
                    } else {
                        tma_load_2d_pair(dst, &maps.p, k * kGaK, p0, bar);
                    }
                    if (a_km) {
                        tma_load_2d_pair(dst + kGaOpBytes, &maps.q, q0, k * kGaK, bar);
                        if (p.wq > 128) tma_load_2d_pair(dst + kGaOpBytes + kGaKnBlock, &maps.q, q0 + 64, k * kGaK, bar);
                    } else {
                        tma_load_2d_pair(dst + kGaOpBytes, &maps.q, k * kGaK, q0, bar);
                    }
                }
            }
            sm.issued = (uint32_t)g;   // read by the drain, after the cluster barrier
            // the releases of the last stages, which the leader's MMAs signal in both CTAs, land before the end
            for (int k = max(0, g - kStages); ok && k < g; ++k)
                ok = mbar_wait(empty + 8u * (k % kStages), (uint32_t)(k / kStages) & 1u, abort_flag, p.flags, p.budget_ns);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            // ------------------------------- MMA issuer (leader) -----------------------------
            if (elect_one()) {
                const uint32_t base = smem_u32(smem);
                const uint64_t pdesc = b_kn ? desc_mn_major(base, kGaKnBlock) : desc_k_major(base);
                const uint64_t qdesc = a_km ? desc_mn_major(base + kGaOpBytes, kGaKnBlock) : desc_k_major(base + kGaOpBytes);
                const uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_kn << 15) | ((uint32_t)a_km << 16) | ((uint32_t)(256 >> 4) << 24);
                const uint32_t pstep = b_kn ? kGaKnStep : 2, qstep = a_km ? kGaKnStep : 2;   // 16 products further
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
                                mma_bf16_pair(acc, pdesc + off + pstep * j, qdesc + off + qstep * j, idesc, j ? 1u : add);
                            add = 1;
                            commit_pair(empty + 8u * s, leader);
                            ++consumed;
                            if (++s == kStages) {
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
                    if (CLUSTER && k + run >= s1) break;
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
    // Warps 2-17, four to a TMEM lane quarter
    const bool epilogue = warp >= 2;
    const int q = warp & 3;
    EpilogueTile e;
    e.group = (warp - 2) >> 2;
    e.runs = 1;
    for (int k = s0 + run; k < s1; k += run) ++e.runs;
    e.split = split;
    e.part = part;
    e.per = p.per;
    e.rank_step = 2;
    e.rank0 = rank;
    e.inbox = smem_u32(smem) + kStages * kGaStageBytes + (uint32_t)(q * 32 + lane) * 4u;
    e.lanes = tmem + ((uint32_t)(q * 32) << 16);
    e.buf_cols = 256;
    int it = 0;
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
    for (int t = unit; (epilogue || CLUSTER) && t < tiles; t += units) {   // a cluster: one tile
        const GaTile c = ga_tile(p, t);
        e.q0 = c.q0;
        e.qn = c.qn;
        e.f = c.p0 + (int)rank * 128 + q * 32 + lane;
        if (!tile_epilogue<4, CLUSTER>(p, e, epilogue, it, ready, release)) break;
        if (!CLUSTER) release();
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
        for (int k = max(0, (int)consumed - kStages); k < (int)consumed; ++k)
            mbar_wait(smem_u32(&sm.empty[k % kStages]), (uint32_t)(k / kStages) & 1u, abort_flag, p.flags, kGaDrainNs, false);
        for (int i = max(0, (int)runs - 2); i < (int)runs; ++i)
            mbar_wait(smem_u32(&sm.tfull[i & 1]), (uint32_t)(i >> 1) & 1u, abort_flag, p.flags, kGaDrainNs, false);
        if (rank == 0) {
            const int gl = (int)sm.issued, gp = (int)ld_cluster_u32(map_rank(smem_u32(&sm.issued), leader + 1)), gm = max(gl, gp);
            for (int k = max(0, gm - kStages); k < gm; ++k) {
                const int s = k % kStages;
                const uint32_t bar = smem_u32(&sm.full[s]);
                const uint32_t tx = k < gl ? sm.stage_tx[s] : ld_cluster_u32(map_rank(smem_u32(&sm.stage_tx[s]), leader + 1));
                if (k >= gl) mbar_expect_tx(bar, tx);
                else if (k >= gp) mbar_complete_tx(bar, tx);
                mbar_wait(bar, (uint32_t)(k / kStages) & 1u, abort_flag, p.flags, kGaDrainNs, false);
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
// tiles too few or too small for the SM pairs: one CTA per tile of 128 features x up to 128 rows, two CTAs per SM
//
// What bounds such a product is how fast an SM takes in operands (64 bytes a cycle from L2: 300 cycles for a stage of 128
// features and 32 rows, whose MMAs take 64), and the fixed cost of a launch.  So the tiles are small, a cluster of up to 8
// CTAs cuts K, every SM takes a share, and there is as little set-up as possible: no pairs, no cluster barriers unless K is cut,
// the first loads issued before the CTA's other warps are ready.
// Warps: 0 producer, 1 MMA issuer, 2-9 epilogue.
// ---------------------------------------------------------------------------------------
constexpr int kGmRing = 96 * 1024;
constexpr int kGmMaxStages = 5;
constexpr int kGmEpiWarps = 8;
constexpr int kGmThreads = 64 + 32 * kGmEpiWarps;
constexpr int kGmMaxRows = 128, kGmMaxSplit = 8;
struct GemmMidSmem {
    uint64_t full[kGmMaxStages], empty[kGmMaxStages], tfull[2], tempty[2], done;
    uint32_t tmem, abort;
};
constexpr int kGmSmem = kGmRing + (int)sizeof(GemmMidSmem) + 1024;
constexpr int kGmClusterSmem = kGmSmem + kInbox;
static_assert(2 * (kGmSmem + 1024) <= 232448 && kGmClusterSmem <= 232448, "two CTAs per SM, one of a cluster");

__device__ __forceinline__ uint32_t cluster_x() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void mma_bf16_single(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit_single(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// KOUT: operands with K outermost, by p.b_kn and p.a_km (333 x 1288 x 5120 takes 0.4 us longer where they are looked up)
template <bool CLUSTER, bool KOUT>
__global__ void __launch_bounds__(kGmThreads, CLUSTER ? 1 : 2) gemm_act_mid_kernel(const __grid_constant__ GemmActMaps maps, const __grid_constant__ GemmActParams p) {
    extern __shared__ uint8_t smem_raw[];
    const bool b_kn = KOUT && p.b_kn, a_km = KOUT && p.a_km;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    GemmMidSmem& sm = *reinterpret_cast<GemmMidSmem*>(smem + kGmRing + (CLUSTER ? kInbox : 0));
    volatile uint32_t* abort_flag = &sm.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = CLUSTER ? p.split : 1, part = CLUSTER ? (int)cluster_rank() : 0;
    // neighbours share the features' rows of B
    const int q0 = (int)(CLUSTER ? cluster_x() : blockIdx.x) * p.wq, p0 = 128 * (int)blockIdx.y, qn = min(p.wq, p.M - q0);
    const int s0 = CLUSTER ? part * p.part_stages + min(part, p.longer) : 0, s1 = CLUSTER ? s0 + p.part_stages + (part < p.longer) : p.stages;
    const int run = p.run;
    const int n = (qn + 15) & ~15;                       // the MMA's N
    const uint32_t stage_bytes = (uint32_t)kGaOpBytes + ga_row_bytes(a_km, p.wq);
    const int ring = p.ring;
    const uint32_t base = smem_u32(smem), full = smem_u32(&sm.full[0]), empty = smem_u32(&sm.empty[0]);
    const uint32_t cols = p.tmem_cols;                   // two accumulators (one, where one run serves)

    int g = s0, s = 0;                                   // the producer's next stage, its slot
    const auto load = [&]() {
        mbar_expect_tx(full + 8u * s, stage_bytes);
        if (b_kn) {
            tma_load_2d(base + s * stage_bytes, &maps.p, p0, g * kGaK, full + 8u * s);
            tma_load_2d(base + s * stage_bytes + kGaKnBlock, &maps.p, p0 + 64, g * kGaK, full + 8u * s);
        } else {
            tma_load_2d(base + s * stage_bytes, &maps.p, g * kGaK, p0, full + 8u * s);
        }
        if (a_km) {
            tma_load_2d(base + s * stage_bytes + kGaOpBytes, &maps.q, q0, g * kGaK, full + 8u * s);
            if (p.wq > 64) tma_load_2d(base + s * stage_bytes + kGaOpBytes + kGaKnBlock, &maps.q, q0 + 64, g * kGaK, full + 8u * s);
        } else {
            tma_load_2d(base + s * stage_bytes + kGaOpBytes, &maps.q, g * kGaK, q0, full + 8u * s);
        }
        ++g;
        if (++s == ring) s = 0;
    };
    if (warp == 0) {
        if (lane == 0) {
            for (int i = 0; i < ring; ++i) {
                mbar_init(full + 8u * i, 1);
                mbar_init(empty + 8u * i, 1);
            }
            for (int b = 0; b < 2; ++b) {
                mbar_init(smem_u32(&sm.tfull[b]), 1);
                mbar_init(smem_u32(&sm.tempty[b]), kGmEpiWarps);
            }
            mbar_init(smem_u32(&sm.done), 1);
            sm.abort = 0u;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            fence_async_smem();
            griddep_wait();
            for (int i = 0; i < ring && g < s1; ++i) load();
        }
        __syncwarp();
    } else if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    griddep_wait();
    griddep_launch();
    __syncthreads();
    if (CLUSTER) cluster_arrive_relaxed();   // for the epilogue
    tc_fence_after();
    const uint32_t tmem = sm.tmem, buf_cols = cols >> 1;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t parity = 0;     // of the slots' first release
            bool ok = true;
            while (ok && g < s1) {
                const bool wrap = s + 1 == ring;
                ok = mbar_wait(empty + 8u * s, parity, abort_flag, p.flags, p.budget_ns);
                if (!ok) break;
                load();
                if (wrap) parity ^= 1u;
            }
            // every copy lands, and every release of the MMAs, before the CTA ends
            const int issued = g - s0;
            for (int k = max(0, issued - ring); k < issued; ++k) {
                const uint32_t ph = (uint32_t)(k / ring) & 1u;
                mbar_wait(full + 8u * (k % ring), ph, abort_flag, p.flags, kGaDrainNs, false);
                if (ok) ok = mbar_wait(empty + 8u * (k % ring), ph, abort_flag, p.flags, p.budget_ns);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {
            const uint64_t pdesc = b_kn ? desc_mn_major(base, kGaKnBlock) : desc_k_major(base);
                const uint64_t qdesc = a_km ? desc_mn_major(base + kGaOpBytes, kGaKnBlock) : desc_k_major(base + kGaOpBytes);
            const uint32_t pstep = b_kn ? kGaKnStep : 2, qstep = a_km ? kGaKnStep : 2;   // 16 products further
            const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_kn << 15) | ((uint32_t)a_km << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
            int it = 0, slot = 0;
            uint32_t parity = 0;
            bool ok = true;
            for (int k = s0; ok && k < s1; ++it) {
                const int end = min(s1, k + run);
                if (!mbar_wait(smem_u32(&sm.tempty[it & 1]), ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag, p.flags, p.budget_ns)) break;
                tc_fence_after();
                const uint32_t acc = tmem + buf_cols * (it & 1);
                uint32_t add = 0;
                for (; k < end; ++k) {
                    ok = mbar_wait(full + 8u * slot, parity, abort_flag, p.flags, p.budget_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t off = (uint64_t)((slot * stage_bytes) >> 4);
#pragma unroll
                    for (int j = 0; j < kGaK / 16; ++j) mma_bf16_single(acc, pdesc + off + pstep * j, qdesc + off + qstep * j, idesc, j ? 1u : add);
                    add = 1;
                    commit_single(empty + 8u * slot);
                    if (++slot == ring) {
                        slot = 0;
                        parity ^= 1u;
                    }
                }
                if (ok) commit_single(smem_u32(&sm.tfull[it & 1]));
            }
            commit_single(smem_u32(&sm.done));
            mbar_wait(smem_u32(&sm.done), 0u, abort_flag, p.flags, kGaDrainNs, false);
        }
        __syncwarp();
    }
    // epilogue: warps 2-9, two to a TMEM lane quarter
    const int q = warp & 3;
    EpilogueTile e;
    e.q0 = q0;
    e.qn = qn;
    e.f = p0 + q * 32 + lane;
    e.group = (warp - 2) >> 2;
    e.runs = 1;
    for (int k = s0 + run; k < s1; k += run) ++e.runs;
    e.split = split;
    e.part = part;
    e.per = p.per;
    e.rank_step = 1;
    e.rank0 = 0;
    e.inbox = base + kGmRing + (uint32_t)(q * 32 + lane) * 4u;
    e.lanes = tmem + ((uint32_t)(q * 32) << 16);
    e.buf_cols = buf_cols;
    int it = 0;
    const auto ready = [&]() {
        const bool done = mbar_wait(smem_u32(&sm.tfull[it & 1]), (uint32_t)(it >> 1) & 1u, abort_flag, p.flags, p.budget_ns);
        if (!__all_sync(0xFFFFFFFFu, done)) return false;
        tc_fence_after();
        return true;
    };
    const auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.tempty[it & 1]));
        ++it;
    };
    if (warp >= 2 || CLUSTER) tile_epilogue<2, CLUSTER>(p, e, warp >= 2, it, ready, release);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
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

// the products of one chunk's fragments with the rows' own at k: `x` is row g of the first group
template <int NG>
__device__ __forceinline__ void gf_chunk(const GemmActFewParams& p, float (&acc)[NG][4], const uint16_t* x, int k, int g, bool in0, bool in1,
                                         const uint4& a00, const uint4& a01, const uint4& a10, const uint4& a11) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        const bool row = 8 * i + g < p.e.M;
        const uint16_t* xi = x + (int64_t)(8 * i) * p.lda + k;
        const uint4 b0 = row && in0 ? __ldg(reinterpret_cast<const uint4*>(xi)) : zero;
        const uint4 b1 = row && in1 ? __ldg(reinterpret_cast<const uint4*>(xi + 32)) : zero;
        gf_mma(acc[i], a00.x, a10.x, a00.y, a10.y, b0.x, b0.y);
        gf_mma(acc[i], a00.z, a10.z, a00.w, a10.w, b0.z, b0.w);
        gf_mma(acc[i], a01.x, a11.x, a01.y, a11.y, b1.x, b1.y);
        gf_mma(acc[i], a01.z, a11.z, a01.w, a11.w, b1.z, b1.w);
    }
}
// the warps' sums (part[warp][row][feature], padded) joined, and the outputs of 16 features from f0 on
template <int NG, int WARPS>
__device__ __forceinline__ void gf_finish(const GemmActParams& e, const float (&part)[WARPS][NG * 8][17], int f0) {
    for (int i = threadIdx.x; i < 16 * e.M; i += 32 * WARPS) {
        const int f = f0 + (i & 15), row = i >> 4;
        if (f >= e.N) continue;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) s += part[w][row][i & 15];
        if (e.bias) s += e.bias[f];
        if (e.pre) e.pre[(int64_t)row * e.ldpre + f] = (uint16_t)f32x2_to_bf16x2(s, 0.0f);
        s = act::one(e.act, s);
        if (e.residual) {
            const int64_t at = (int64_t)row * e.ldr + f;
            s += e.res_fp32 ? reinterpret_cast<const float*>(e.residual)[at]
                            : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(e.residual)[at] << 16);
        }
        const int64_t at = (int64_t)row * e.ldd + f;
        if (e.out_fp32) reinterpret_cast<float*>(e.d)[at] = s;
        else reinterpret_cast<uint16_t*>(e.d)[at] = (uint16_t)f32x2_to_bf16x2(s, 0.0f);
    }
}

// NG: groups of 8 rows; PER_SM: CTAs of an SM.  With three of 8 warps a thread has the registers for two chunks of weights in flight
template <int NG, int WARPS, int PER_SM>
__global__ void __launch_bounds__(32 * WARPS, PER_SM) gemm_act_few_kernel(const GemmActFewParams p) {
    __shared__ float part[WARPS][NG * 8][17];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int f0 = blockIdx.x * 16, N = p.e.N;
    // features past the end read the last one
    const uint16_t* w0 = p.b + (int64_t)min(f0 + g, N - 1) * p.ldb + 8 * t;
    const uint16_t* w1 = p.b + (int64_t)min(f0 + g + 8, N - 1) * p.ldb + 8 * t;
    const uint16_t* x = p.a + (int64_t)g * p.lda + 8 * t;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    // runs of kGfRun products, joined in the warp's own part of shared memory (registers are full)
#pragma unroll 1
    for (int k = 64 * warp, run = 0; run == 0 || k < p.K; ++run) {
        const int end = min(p.K, k + kGfRun * WARPS);
        float acc[NG][4] = {};
#pragma unroll(PER_SM * WARPS <= 24 ? 2 : 1)
        for (; k < end; k += 64 * WARPS) {
            const bool in0 = k + 8 * t < p.K, in1 = k + 32 + 8 * t < p.K;
            const uint4 a00 = in0 ? gf_stream(w0 + k) : zero, a01 = in1 ? gf_stream(w0 + k + 32) : zero;
            const uint4 a10 = in0 ? gf_stream(w1 + k) : zero, a11 = in1 ? gf_stream(w1 + k + 32) : zero;
            gf_chunk<NG>(p, acc, x, k, g, in0, in1, a00, a01, a10, a11);
        }
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float& s = part[warp][8 * i + 2 * t + (j & 1)][g + 4 * (j & 2)];
                s = run == 0 ? acc[i][j] : s + acc[i][j];
            }
    }
    __syncthreads();
    gf_finish<NG, WARPS>(p.e, part, f0);
}

// ---------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------
constexpr int kGfRows = 16;      // rows up to which the kernel for few is taken (B [N][K])
constexpr int kGfLongK = 2048;   // a K from which 16 warps cut it, where one wave of CTAs holds the launch

template <class Kernel>
static cudaError_t launch_ga(Kernel kern, int bytes, std::atomic<uint64_t>& attr, int cluster, int threads, int64_t blocks,
                             unsigned rows, const GemmActMaps& maps, const GemmActParams& p, cudaStream_t s) {
    if (cudaError_t e = host::ensure_smem(reinterpret_cast<const void*>(kern), bytes, attr)) return e;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks, rows);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

// The kernel, the row tiles' width w and the parts of K, by an estimate of the time in ns, whose terms are fitted to
// measurements of every width and split at 20 shapes from 17 x 256 x 64 to 1024 x 5120 x 5120:
//   a stage of 64 products takes a CTA the time its operands need, (128 + w) * 128 bytes at 122 bytes a ns, a pair of CTAs
//   180 + 0.26 w, or 1.465 w for the MMAs; all SMs together take 12000 bytes a ns from L2, and memory gives 6000, 75 to
//   one SM (operands of more than 100 MB do not stay in L2);
//   a launch takes 2900 + 19 w (one CTA per tile), 3800 + 150 split + 14 w (K cut over CTAs), 5000 + 8 w (pairs) or 4600 + 26 w (K
//   cut over pairs) besides; clusters that do not fit at once have cost 20 us a wave.
// Estimate / measured of what it chooses (us): 64 x 1280 x 5120 7.7 / 7.9 (one CTA per tile, 5 parts; one pair 18.3), 333 x 1288 x
// 5120 12.7 / 12.6 (3 parts; in 4, 0.1 less in a sweep; pairs in 3 parts 14.1), 500 x 5120 x 5120 29.5 / 28.7 (pairs), 1000 x 1280 x
// 5120 21.1 / 18.6 (pairs in 2 parts), 2000 x 2568 x 1288 19.6 / 22.6 (pairs), 2088 x 376 x 504 5.7 / 5.6 (one CTA per tile; pairs 7.6),
// 64 x 20480 x 5120 52.6 / 41.4 (one CTA per tile, 160 of them, counted as two whole waves; pairs 53).
// With K outermost the terms are the same, and the estimate is short: whole blocks of 64 are loaded (w = 48 loads 64), and
// clusters of 8 CTAs may not all fit at once.  16384 rows of 256 x 256 11.6 / 16.1, 8192 of 1000 x 1000 23.3 / 48.3, 3974 of 208 x
// 2384 11.9 / 13.9.
struct GaPlan {
    bool single;     // one CTA per tile
    int split, wq;
};
static int even(int64_t rows, int64_t tiles, int step) { return (int)(((rows + tiles - 1) / tiles + step - 1) / step * step); }
static GaPlan ga_plan(int64_t M, int64_t N, int64_t stages, int sms) {
    GaPlan best{false, 1, 256};
    double least = 1e300;
    const auto take = [&](bool single, int split, int wq, double ns) {
        if (ns < least) {
            least = ns;
            best = GaPlan{single, split, wq};
        }
    };
    const int64_t np2 = (N + 255) / 256, np1 = (N + 127) / 128;
    const double bytes = 128.0 * (double)(M + N) * (double)stages, memory_ns = bytes / 6000.0;
    const bool resident = bytes < 100e6;
    int64_t seen = 0;
    for (int w = 256; w >= 32; w -= 32) {
        const int64_t nq = (M + w - 1) / w, tiles = np2 * nq;
        if (nq == seen) continue;   // the same even cut
        seen = nq;
        const int wq = even(M, nq, 32);
        const double per_sm = 128.0 * (128 + wq / 2);
        for (int split = 1; split <= 4 && split <= stages; ++split) {
            const int64_t fit = split == 1 ? sms / 2 : sms / (2 * split) - (split > 2 ? 2 : 1);   // clusters at once
            if (fit < 1 || (split > 1 && tiles > fit)) break;
            const double part = (double)((stages + split - 1) / split);
            const auto wave = [&](int64_t now) {
                const double stage = std::max({180.0 + 0.26 * wq, 1.465 * wq, (double)(now * 2 * split) * per_sm / 12000.0, resident ? 0.0 : per_sm / 75.0});
                return std::max(part * stage, memory_ns * (double)now / (double)tiles);
            };
            const int64_t full = tiles / fit, rest = tiles % fit;
            take(false, split, wq, (full ? (double)full * wave(fit) : 0.0) + (rest ? wave(rest) : 0.0) +
                                       (split > 1 ? 4600.0 + 26.0 * wq : 5000.0 + 8.0 * wq));
        }
    }
    seen = 0;
    for (int w = kGmMaxRows; w >= 16; w -= 16) {
        const int64_t nq = (M + w - 1) / w;
        if (nq == seen) continue;
        if (np1 * nq > 4 * sms) break;
        seen = nq;
        const int wq = even(M, nq, 16);
        const double per_sm = 128.0 * (128 + wq);
        for (int split = 1; split <= kGmMaxSplit && split <= stages; ++split) {
            const int64_t ctas = np1 * nq * split;
            if (split > 1 && ctas > sms - sms / 16) break;
            const double waves = (double)((ctas + sms - 1) / sms), now = (double)std::min<int64_t>(ctas, sms);
            const double stage = std::max({per_sm / 122.0, now * per_sm / 12000.0, resident ? 0.0 : per_sm / 75.0 / std::min(waves, 2.0)});
            take(true, split, wq, std::max(waves * (double)((stages + split - 1) / split) * stage, memory_ns) +
                                      (split > 1 ? 3800.0 + 150.0 * split + 14.0 * wq : 2900.0 + 19.0 * wq));
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
    p.b_kn = g.b_kn;
    p.a_km = g.a_km;   // only with b_kn
    if (g.M <= kGfRows && !g.b_kn && !g.a_km) {
        const GemmActFewParams f{g.a, g.b, g.lda, g.ldb, (int32_t)g.K, p};
        const unsigned blocks = (unsigned)((g.N + 15) / 16);
        const bool long_k = g.K >= kGfLongK && blocks <= 2u * host::sm_count();
        if (g.M <= 8) {
            // Three CTAs per SM, unless four need fewer waves, one or two: 1 x 20480 x 5120 35.2 us, with four 38.5; 1 x 10240 x 5120 21.4,
            // 23.8; 1 x 5120 x 20480 36.5, 41.8; but 1 x 8192 x 4096 (512 CTAs) 16.6, 13.7 and 1 x 16384 x 2048 15.5, 13.9.
            const unsigned sms = (unsigned)host::sm_count(), four = (blocks + 4 * sms - 1) / (4 * sms), three = (blocks + 3 * sms - 1) / (3 * sms);
            if (long_k) gemm_act_few_kernel<1, 16, 2><<<blocks, 512, 0, s>>>(f);
            else if (four <= 2 && four < three) gemm_act_few_kernel<1, 8, 4><<<blocks, 256, 0, s>>>(f);
            else gemm_act_few_kernel<1, 8, 3><<<blocks, 256, 0, s>>>(f);
        } else {
            if (long_k) gemm_act_few_kernel<2, 16, 2><<<blocks, 512, 0, s>>>(f);
            else gemm_act_few_kernel<2, 8, 4><<<blocks, 256, 0, s>>>(f);
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
    p.split = plan.split;
    p.per = ((plan.wq + 15) / 16 + plan.split - 1) / plan.split;
    p.part_stages = (int32_t)(stages / plan.split);
    p.longer = (int32_t)(stages % plan.split);
    p.np = (int32_t)((g.N + (plan.single ? 127 : 255)) / (plan.single ? 128 : 256));
    p.nq = (int32_t)((g.M + plan.wq - 1) / plan.wq);
    GemmActMaps maps;
    const int64_t bdims[2] = {g.b_kn ? g.N : g.K, g.b_kn ? g.K : g.N}, bstrides[1] = {g.ldb}, adims[2] = {g.a_km ? g.M : g.K, g.a_km ? g.K : g.M}, astrides[1] = {g.lda};
    const uint32_t bbox[2] = {64, g.b_kn ? (uint32_t)kGaK : 128u}, abox[2] = {64, g.a_km ? (uint32_t)kGaK : (uint32_t)(plan.single ? plan.wq : plan.wq / 2)};
    if (!host::bf16_map(&maps.p, g.b, 2, bdims, bstrides, bbox) || !host::bf16_map(&maps.q, g.a, 2, adims, astrides, abox))
        return cudaErrorInvalidValue;
    const int64_t tiles = (int64_t)p.np * p.nq;
    static std::atomic<uint64_t> attr[8];
    const int split = plan.split;
    if (plan.single) {
        p.ring = std::min(kGmMaxStages, kGmRing / (kGaOpBytes + (int)ga_row_bytes(g.a_km, plan.wq)));
        p.tmem_cols = 64;   // two accumulators
        while ((int)p.tmem_cols < 2 * plan.wq) p.tmem_cols <<= 1;
        if (split > 1)
            return g.b_kn ? launch_ga(gemm_act_mid_kernel<true, true>, kGmClusterSmem, attr[4], split, kGmThreads, p.nq * split, p.np, maps, p, s)
                          : launch_ga(gemm_act_mid_kernel<true, false>, kGmClusterSmem, attr[0], split, kGmThreads, p.nq * split, p.np, maps, p, s);
        return g.b_kn ? launch_ga(gemm_act_mid_kernel<false, true>, kGmSmem, attr[5], 1, kGmThreads, p.nq, p.np, maps, p, s)
                      : launch_ga(gemm_act_mid_kernel<false, false>, kGmSmem, attr[1], 1, kGmThreads, p.nq, p.np, maps, p, s);
    }
    if (split > 1)
        return g.b_kn ? launch_ga(gemm_act_kernel<true, true>, kGaClusterSmem, attr[6], 2 * split, kGaThreads, 2 * tiles * split, 1, maps, p, s)
                      : launch_ga(gemm_act_kernel<true, false>, kGaClusterSmem, attr[2], 2 * split, kGaThreads, 2 * tiles * split, 1, maps, p, s);
    const int64_t blocks = 2 * std::min<int64_t>(tiles, sms / 2);
    return g.b_kn ? launch_ga(gemm_act_kernel<false, true>, kGaSmem, attr[7], 2, kGaThreads, blocks, 1, maps, p, s)
                  : launch_ga(gemm_act_kernel<false, false>, kGaSmem, attr[3], 2, kGaThreads, blocks, 1, maps, p, s);
}

// ---------------------------------------------------------------------------------------
// the activation's and the bias' gradient: dh = dy act'(h) in bf16, db[f] (+)= sum over the rows of dy act'(h)
//
// A CTA takes 64 features (8 lanes of 8) of a run of rows; its threads' sums over their rows are joined in shared memory, and the
// runs' by a second kernel, in a fixed order.  Bound by memory (squared ReLU) and by the erf's arithmetic: 8192 x 20480, with the bias'
// gradient, 157 us (6.4 TB/s) with squared ReLU, 220 with GeLU; one row at a time 202 and 297, four rows (whose registers leave an SM
// 2 or 3 CTAs) 164 to 178 and 211 to 224.
// ---------------------------------------------------------------------------------------
constexpr int kAbThreads = 256, kAbPerSm = 4;

template <int ACT>
__global__ void __launch_bounds__(kAbThreads, kAbPerSm) act_bwd_kernel(const ActBwd p, int rows_per) {
    __shared__ float part[kAbThreads / 8][64 + 1];
    const int c = threadIdx.x & 7, r = threadIdx.x >> 3;
    const int64_t col = (int64_t)blockIdx.x * 64 + 8 * c;
    const int64_t t0 = (int64_t)blockIdx.y * rows_per, t1 = min(p.rows, t0 + rows_per);
    float sum[8] = {};
    if (p.dbias) ptx::griddep_launch();
    // the loads of two rows go out before the first is used; dh may be dy, whose rows a thread reads before it writes them
    constexpr int kStep = kAbThreads / 8, kRows = 2;
    if (col < p.n)
        for (int64_t t = t0 + r; t < t1; t += kRows * kStep) {
            uint4 g4[kRows], h4[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u)
                if (t + u * kStep < t1) {
                    g4[u] = *reinterpret_cast<const uint4*>(p.dy + (t + u * kStep) * p.lddy + col);
                    if (ACT != kActNone) h4[u] = __ldg(reinterpret_cast<const uint4*>(p.pre + (t + u * kStep) * p.ldpre + col));
                }
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                if (t + u * kStep >= t1) break;
                if (ACT == kActNone) h4[u] = make_uint4(0, 0, 0, 0);
                const uint32_t g[4] = {g4[u].x, g4[u].y, g4[u].z, g4[u].w}, h[4] = {h4[u].x, h4[u].y, h4[u].z, h4[u].w};
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
                if (p.dh) *reinterpret_cast<uint4*>(p.dh + (t + u * kStep) * p.lddh + col) = make_uint4(o[0], o[1], o[2], o[3]);
            }
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
    ptx::griddep_wait();
    if (f >= p.n) return;
    float s = p.accumulate ? p.dbias[f] : 0.0f;
#pragma unroll 8
    for (int i = 0; i < runs; ++i) s += p.scratch[(int64_t)i * p.n + f];
    p.dbias[f] = s;
}

cudaError_t launch_act_bwd(const ActBwd& p, cudaStream_t s) {
    const int64_t cols = (p.n + 63) / 64;
    // as few runs as fill whole waves of CTAs (kAbPerSm of an SM) to nine tenths, or those that fill them best
    const int64_t wave = (int64_t)kAbPerSm * host::sm_count(), most = std::min<int64_t>(kActBwdRuns, (p.rows + 31) / 32);
    int64_t runs = 1;
    double best = 0.0;
    for (int64_t r = 1; r <= most && best < 0.9; ++r) {
        const int64_t waves = (cols * r + wave - 1) / wave;
        const double full = (double)(cols * r) / (double)(waves * wave);
        if (full > best) {
            best = full;
            runs = r;
        }
    }
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
    cudaLaunchAttribute pdl{};
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((p.n + 255) / 256));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = &pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, act_bwd_join_kernel, p, used);
}

}  // namespace nvfp4
