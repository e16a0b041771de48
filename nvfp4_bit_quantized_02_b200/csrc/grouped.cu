// grouped.cu -- bf16 products grouped by expert on the 5th-generation tensor cores (sm_100a):
//   fprop   D[t] = A[t] . W_e^T      W_e [N][K], rows t of expert e
//   dgrad   D[t] = A[t] . W_e        W_e [K][N]
//   wgrad   D_e (+)= sum_t A[t]^T B[t]   over the rows t of expert e
//
// One kernel, three instantiations, on SM pairs (clusters of two CTAs, tcgen05.mma.cta_group::2,
// kind::f16, fp32 accumulators in TMEM).  The operand whose elements lie next to one another in a
// row of the output is the MMA's M side ("P": the weights of fprop and dgrad, B of wgrad), 256
// features per tile, 128 per CTA; the other is its N side ("Q": the token rows, A's features of
// wgrad), up to 256 output rows per tile in steps of 32.  So
//   - a ragged run of rows costs MMA time for its rows rounded up to 32, not to a tile's 256;
//   - a TMEM lane is an output feature and a TMEM column an output row: the 32 lanes of an epilogue
//     warp hold 32 neighbours of one output row, and plain stores are whole 64-byte (bf16) or
//     128-byte (fp32) pieces.  No staging in shared memory, no output box that could touch another
//     expert's rows: a row past the run is a predicate.
// Operands whose reduction index is contiguous (fprop's both, dgrad's A) are K-major in shared
// memory; the others (dgrad's W_e, both of wgrad) are MN-major, read by TMA as they lie: no
// transposed copies.
//
// Warps: 0 TMA producer (a ring of 192 KiB per CTA: Shape below); 1 MMA issuer in the leader CTA, in the
// peer it forwards "accumulator drained"; 2-17 epilogue; 18 (wgrad) clears the rows of a run's last
// stage that belong to the next expert.
// The accumulator is double-buffered (2 x 256 TMEM columns).  Where a tile is one accumulator, half of
// the epilogue warps take the even ones and half the odd ones, 16 columns in turn.  The tensor core
// truncates as it accumulates (measured on N(0, 1) operands, relative to the result: 5e-7 after 512
// products, 2e-6 after 2048, 9e-6 after 8192, 4e-5 after 32768; positive operands, 6e-3 after 2^20), so
// an accumulator holds at most 512 products with fp32 output and 1024 with bf16, whose half step is 2e-3
// at least, and the epilogue joins such runs in registers, rounded to nearest, while the next run is under
// way: all 16 warps, 16 columns in turn, 64 at most.  fp32 runs of 512 cost wgrad of the shapes below 3 %
// over one accumulator.  bf16 runs of 1024 cost 0 to 3 %: fprop of those shapes 157.7 us in one, 158.3 in
// runs of 1024; 8 experts of 4096 x 5120 x 5120 called without a pause 1201 and 1240; runs of 512 are
// 2 % slower again.  The 64 sums leave no register to spare (five warps share a scheduler's 16384): read
// 16 columns at a time they spill, and wgrad takes 3 us more.
//
// The offsets stay on the device: every CTA reads them, takes their running maximum clamped to
// [0, rows], and numbers the tiles of all experts; a pair walks tiles pair, pair + pairs, ...
// Every mbarrier wait is bounded by the caller's budget; on expiry the CTA raises the timeout flag,
// drains its copies and MMAs (bounded again) and frees its TMEM.
//
// Measured on 16384 rows x 16 experts of 5120 x 1280, even counts, beside cuBLAS' batched product of the
// same shapes (us; a call after a pause / one of thousands in a row, where the 1000 W limit holds the SMs
// at ~1.5 GHz), in one run:
//   fprop 157 / 192, cuBLAS 164 / 200; dgrad 160 / 198, cuBLAS 152 / 187; wgrad 192 / 232, cuBLAS 186 / 227.
// One expert of 8192 x 5120 x 5120: fprop 280 / 331 (1.53 PFLOP/s), cuBLAS 281 / 335.  The tensor pipe is
// active in 86 % of fprop's cycles, 77 % of dgrad's and 62 % of wgrad's, which writes 419 MB of fp32 (without
// its stores it took a quarter less).  With uneven counts (log-normal, sigma 0.6) the tiles of the longest
// expert count: dealt out by number, the busiest pair has 1.06 of the mean in fprop, 1.03 in dgrad and 1.06
// to 1.20 in wgrad.  Without effect: the last wave's tiles cut into row parts, the reduction begun at
// another stage for each tile, stores with an evict-first policy or spread out by sleeps, bands of 2 to 16
// tiles, 4 or 5 stages of 64 products, longer suspended waits.
// The producer's and the MMA issuer's loops are one elected lane's and kept short: a stage of 64 products
// takes them 320 cycles, less than 256 rows' MMAs (512); at 465 they bound every narrower tile (256 rows x
// 5120 x 1280 25.0 us, now 19.2).
#include <algorithm>

#include "nvfp4_device.cuh"
#include "sm100_ptx.cuh"

namespace nvfp4 {

using namespace ptx;

enum : int { kFprop = 0, kDgrad = 1, kWgrad = 2 };

constexpr int kMaxStages = 6;
constexpr int kRingBytes = 192 * 1024;                   // every instantiation's stages together
constexpr int kEpiWarps = 16;
constexpr int kRunK = 512;                               // products per accumulator with fp32 output
constexpr int kRunBf16 = 1024;                           // and with bf16 output
constexpr int kWidths = 5;                               // Q rows per tile: 256, 224, ... 128 (the plan below)
constexpr int kBand = 8;                                 // Q tiles of an expert swept together (L2 reuse)
constexpr uint64_t kGDrainBudgetNs = 2000000000ull;      // teardown waits, whatever the caller's budget

struct GroupedParams {
    const int32_t* offsets;
    void* d;
    int64_t ldd, stride_d;
    int32_t rows, experts;
    int32_t P, Q;           // features of the P side; wgrad: features of the Q side
    int32_t K;              // fprop, dgrad: the reduction
    int32_t expert_step;    // 1: expert e reads slice e of the weights' map, 0: always slice 0
    int32_t out_fp32, accumulate;
    int32_t deep;           // dgrad: K is a multiple of 64, Q's boxes hold two blocks of products
    uint32_t* flags;
    uint64_t budget_ns;
};

struct GroupedSmem {        // behind the stages
    uint64_t full[kMaxStages];     // leader: a stage's bytes of both CTAs
    uint64_t empty[kMaxStages];    // both: the MMAs that read the stage are done
    uint64_t tail[kMaxStages];     // each CTA: its bytes of a stage whose rows have to be cleared (wgrad)
    uint64_t tfull[2];             // both: accumulator ready
    uint64_t tempty[2];            // leader: both CTAs' epilogues have read it
    uint64_t edrained[2];          // peer: its epilogue has read it
    uint64_t done;
    uint32_t tmem, abort, peer_abort, issued, tails;
    uint32_t consumed, runs;       // leader: stages and accumulators that the MMA issuer has committed
    uint32_t stage_tx[kMaxStages]; // bytes per CTA of the last use of each stage, 0: a tail
    int32_t best;                  // the chosen width's number
    uint32_t cost[kWidths];        // fp32 patterns, the last three bits the width's number
    int32_t row[kMaxExperts + 4];              // expert e owns rows [row[e], row[e + 1])
    int32_t tile[kWidths][kMaxExperts + 4];    // and Q tiles [tile[w][e], tile[w][e + 1]) at width w
};
constexpr int kGroupedSmem = kRingBytes + (int)sizeof(GroupedSmem) + 1024;
static_assert(kGroupedSmem <= 232448, "shared memory");

// A stage is one TMA load per operand and CTA, since the TMA engine's rate, not L2's, bounds the
// loads, and each load has a fixed cost (fprop at 8192 x 5120 x 5120: 1519 TFLOP/s with one 128-row
// box for Q, 1171 with four of 32).  That cost is higher for the 4-dimensional MN-major boxes, so
// they are taken deeper: loads alone, 16384 rows x 16 experts x 5120 x 1280, take dgrad 121 us in
// stages of 128 products and 147 in stages of 64, wgrad 153 and 177 (the whole kernels were 2 and 4 %
// faster).  K-major boxes gain little (119 and 122) and lose the finer ring (fprop 4 % slower).
template <int MODE>
struct Shape {
    static constexpr bool kPmn = MODE != kFprop;         // P is MN-major
    static constexpr bool kQmn = MODE == kWgrad;
    static constexpr int kThreads = MODE == kWgrad ? 608 : 576;
    static constexpr int kK = MODE == kFprop ? 64 : 128;   // products per stage
    static constexpr int kOpBytes = 256 * kK;            // an operand's 128 features or rows
    static constexpr int kStageBytes = 2 * kOpBytes;
    static constexpr int kStages = kRingBytes / kStageBytes;
    static constexpr int kBlock = 128 * kK;              // an MN-major block: 64 features x kK products
    static_assert(kStages <= kMaxStages && kRunK % kK == 0, "ring");
};

// The maps of a launch.
// K-major Q: boxes of 32, 64 and 128 rows (q[0..2]), the smallest that holds a tile's rows; the
// same with two blocks of 64 products (q_deep, where K is a multiple of 64) for dgrad's stages.
// MN-major operands: a row's features cut into blocks of 64, so that one box holds two blocks (wide);
// where a tile's 128 features are not all there, or do not start at a block, two boxes of one
// block each, which end at the tensor's width (p, q[0]).
struct Maps {
    CUtensorMap p, p_wide, q[3], q_deep[3];
};

// One output tile
struct Tile {
    int e, p0;          // expert, first feature
    int q0, qn;         // first output row (wgrad: of D_e) and how many are valid
    int n;              // the MMA's N: qn rounded up to 32
    int k0, klen;       // the reduction: first index and length
    int stages;         // that it takes
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Quotients of the plan, which stands between a launch and its first load: from fp32, set right by
// the remainder, in a few instructions rather than an integer division's.
__device__ __forceinline__ int tiles_of(int len, int width, float inv) {   // ceil(len / width)
    const int q = (int)((float)len * inv), r = len - q * width;            // the floor, or off by 1 (len <= 2^30)
    return q + (r > 0) + (r > width) - (r <= -width);
}
__device__ __forceinline__ int even_width(int len, int tiles, int width) {   // len over tiles, a multiple of 32
    int c = (int)ceilf(__fdividef((float)len, 32.0f * (float)tiles));
    c += (int64_t)c * tiles * 32 < len;
    c -= (int64_t)(c - 1) * tiles * 32 >= len;
    return min(32 * c, width);   // tiles * width >= len > (tiles - 1) * width
}

// Walks the tiles of one pair: pair, pair + pairs, ...  An expert's tiles go along P row by row of Q
// tiles, so that a last, partial P tile (little to write) comes to every pair in turn; with more than
// kBand rows, in bands of kBand Q tiles, within a band along P with Q fastest.
// What can be read again from shared memory is: the epilogue has no registers to spare.
template <int MODE>
struct Walk {
    const GroupedParams& p;
    const GroupedSmem& sm;
    int t, step;             // the next tile, their distance
    int e = 0;               // the tile's expert
    __device__ __forceinline__ Walk(const GroupedParams& p_, const GroupedSmem& sm_, int pair, int pairs)
        : p(p_), sm(sm_), t(pair), step(pairs) {}
    // the next tile, if there is one
    __device__ __forceinline__ bool next(Tile& r) {
        const int w = sm.best;
        const int32_t* tile = sm.tile[w];
        const int np = ceil_div(p.P, 256);
        if (t >= tile[p.experts] * np) return false;
        while (t >= tile[e + 1] * np) ++e;
        const int lo = sm.row[e], len = sm.row[e + 1] - lo;
        const int nq = tile[e + 1] - tile[e], i = t - tile[e] * np;
        const int wq = even_width(MODE == kWgrad ? p.Q : len, nq, 256 - 32 * w);
        t += step;
        int pt, qt;
        if (nq <= kBand) {
            qt = (int)__fdividef((float)i, (float)np);   // at most 7, so off by 1 at most
            qt -= qt * np > i;
            qt += (qt + 1) * np <= i;
            pt = i - qt * np;
        } else {
            const int band = i / (kBand * np), in_band = i - band * (kBand * np);
            const int rows = min(kBand, nq - band * kBand);
            pt = in_band / rows;
            qt = band * kBand + (in_band - pt * rows);
        }
        r.e = e;
        r.p0 = pt * 256;
        r.q0 = qt * wq;
        r.qn = min(wq, (MODE == kWgrad ? p.Q : len) - r.q0);
        r.n = (r.qn + 31) & ~31;
        if (MODE == kWgrad) {
            r.k0 = lo;
            r.klen = len;
        } else {
            r.q0 += lo;
            r.k0 = 0;
            r.klen = p.K;
        }
        r.stages = ceil_div(r.klen, Shape<MODE>::kK);
        return true;
    }
};

// Warp w < kWidths: the offsets' running maximum (warp 0 writes sm.row), and, for Q tiles of a width
// of 256 - 32 w, the experts' first ones and the cost: waves of tiles over the pairs times a tile's
// operand rows (256 features and its own rows, evenly cut), since a stage takes the time its operands
// need from L2.  wgrad's Q tiles cut features, the same for every expert (8192 rows, one expert of
// 1000 x 1000: 54.8 us, with tiles of 256 67.5).
// All of it stands between a launch and its first load, hence one pass without integer divisions: a
// launch of one small tile takes 4.9 us, and took 6.8 with two passes, a drain at every end and barriers
// there that wait for the stores.
template <int MODE>
__device__ __forceinline__ void plan(GroupedSmem& sm, const GroupedParams& p, int pairs) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int width = 256 - 32 * warp;
    const float inv = __frcp_rn((float)width);
    int carry = 0, tiles = 0, rows = 0;   // tiles: before this chunk; rows: this lane's
    bool bad = false;
    for (int i = lane; i - lane <= p.experts; i += 32) {   // lane: the run that ends at offset i
        const bool in = i <= p.experts;
        const int o = in ? ld_global_s32(p.offsets + i) : 0;
        int v = in ? min(max(o, 0), p.rows) : 0;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, v, s);
            if (lane >= s) v = max(v, u);
        }
        v = max(v, carry);
        bad |= in && o != v;
        int len = v - __shfl_up_sync(0xFFFFFFFFu, v, 1);
        if (lane == 0) len = i == 0 ? 0 : v - carry;
        int n = 0;
        if (in && i > 0 && (len > 0 || (MODE == kWgrad && !p.accumulate))) {
            if (MODE == kWgrad) len = p.Q;
            n = tiles_of(len, width, inv);
            rows += n * 32 * (int)ceilf(__fdividef((float)len, 32.0f * (float)n));
        }
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, n, s);
            if (lane >= s) n += u;
        }
        if (in) {
            sm.tile[warp][i] = tiles + n;
            if (warp == 0) sm.row[i] = v;
        }
        tiles += __shfl_sync(0xFFFFFFFFu, n, 31);
        carry = __shfl_sync(0xFFFFFFFFu, v, 31);
    }
    if (warp == 0 && bad && blockIdx.x == 0) atomicOr(p.flags, kFlagOffsets);
    rows = __reduce_add_sync(0xFFFFFFFFu, rows);
    const float cost = ceilf(__fdividef((float)tiles * ceil_div(p.P, 256), (float)pairs)) *
                       (256.0f + __fdividef((float)rows, fmaxf((float)tiles, 1.0f)));
    if (lane == 0) sm.cost[warp] = (__float_as_uint(cost) & ~7u) | (uint32_t)warp;
}

// Stores (wgrad: or adds) 16 output rows of one feature per lane: the first `n` are the tile's.  `at` is
// the first row's offset in D.
template <int MODE>
__device__ __forceinline__ void put_fp32(const float* v, const GroupedParams& p, int64_t at, int f, int n) {
    float* d = reinterpret_cast<float*>(p.d) + at + f;
    if (f >= p.P) return;
    if (MODE == kWgrad && p.accumulate) {
#pragma unroll
        for (int i = 0; i < 16; ++i, d += p.ldd)   // once per element and call: no order to depend on, no load to wait for
            if (i < n) atomicAdd(d, v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i, d += p.ldd)
            if (i < n) *d = v[i];
    }
}
__device__ __forceinline__ void put_bf16(const float* v, const GroupedParams& p, int64_t at, int f, int n) {
    // neighbouring lanes trade one value of two rows, so that each stores two features of one row
    const int odd = threadIdx.x & 1;
    uint16_t* d = reinterpret_cast<uint16_t*>(p.d) + at + odd * p.ldd + (f - odd);
#pragma unroll
    for (int i = 0; i < 16; i += 2, d += 2 * p.ldd) {
        const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[i] : v[i + 1], 1);
        const uint32_t w = odd ? f32x2_to_bf16x2(other, v[i + 1]) : f32x2_to_bf16x2(v[i], other);
        if (i + odd < n && f < p.P) *reinterpret_cast<uint32_t*>(d) = w;
    }
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Shape<MODE>::kThreads, 1)
    grouped_kernel(const __grid_constant__ Maps maps, const GroupedParams p) {
    using S = Shape<MODE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    GroupedSmem& sm = *reinterpret_cast<GroupedSmem*>(smem + kRingBytes);
    volatile uint32_t* abort_flag = &sm.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 8 * 32) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(smem_u32(&sm.full[s]), MODE == kWgrad ? 2 : 1);
            mbar_init(smem_u32(&sm.empty[s]), 1);
            mbar_init(smem_u32(&sm.tail[s]), 1);
            sm.stage_tx[s] = 0;
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&sm.tfull[b]), 1);
            mbar_init(smem_u32(&sm.tempty[b]), kEpiWarps + 1);   // and the peer's forwarded arrival
            mbar_init(smem_u32(&sm.edrained[b]), kEpiWarps);
        }
        mbar_init(smem_u32(&sm.done), 1);
        sm.abort = 0u;
        sm.peer_abort = 0u;
        sm.issued = 0u;
        sm.tails = 0u;
        sm.consumed = 0u;
        sm.runs = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(S::kPmn ? &maps.p_wide : &maps.p);
        prefetch_map(S::kQmn ? &maps.q_deep[0] : &maps.q[2]);
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    cluster_arrive();   // this CTA's barriers and TMEM are there
    // a launch behind another kernel of the stream: what comes before overlaps that kernel's end, what
    // follows touches memory that it may have written
    griddep_wait();
    griddep_launch();
    if (warp < kWidths) plan<MODE>(sm, p, pairs);
    __syncthreads();
    if (warp == 0) {   // the width: the least cost, of the first with it
        const uint32_t best = __reduce_min_sync(0xFFFFFFFFu, lane < kWidths ? sm.cost[lane] : ~0u) & 7u;
        if (lane == 0) sm.best = (int)best;
    }
    __syncthreads();
    cluster_wait();   // the peer's too
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const int run = (p.out_fp32 ? kRunK : kRunBf16) / S::kK;   // stages per accumulator

    if (warp == 0) {
        // ------------------------------- producer (both CTAs) --------------------------------
        if (elect_one()) {
            Walk<MODE> walk(p, sm, pair, pairs);
            Tile c;
            int g = 0, tails = 0, s = 0;   // stages issued, the next one's slot
            uint32_t parity = 1;           // of the slot's `empty`: at first there is no use to wait for
            const uint32_t base = smem_u32(smem), empty = smem_u32(&sm.empty[0]), full = smem_u32(&sm.full[0]),
                           leader_full = map_rank(full, 0);
            bool ok = true;
            while (ok && walk.next(c)) {
                const int p0 = c.p0 + (int)rank * 128, half = c.n >> 1, q0 = c.q0 + (int)rank * half;
                // K-major Q: the box that holds the half's rows; MN-major: whether one wide box serves
                const int qbox = half <= 32 ? 0 : half <= 64 ? 1 : 2;
                const bool pwide = S::kPmn && p0 + 128 <= p.P, qwide = S::kQmn && half == 128 && q0 + 128 <= p.Q;
                const uint32_t tx = (uint32_t)(S::kOpBytes + (S::kQmn ? (half <= 64 ? S::kBlock : S::kOpBytes) : (64 * S::kK) << qbox));
                const int z = c.e * p.expert_step;
                for (int k = 0; k < c.klen; k += S::kK) {
                    if (!mbar_wait(empty + 8u * s, parity, abort_flag, p.flags, p.budget_ns)) {
                        ok = false;
                        break;
                    }
                    uint32_t bar = leader_full + 8u * s;
                    const bool tail = MODE == kWgrad && (min(S::kK, c.klen - k) & 15) != 0;
                    if (tail) {
                        bar = smem_u32(&sm.tail[tails % S::kStages]);
                        mbar_expect_tx(bar, tx);
                        ++tails;
                    } else if (rank == 0) {
                        mbar_expect_tx(full + 8u * s, 2u * tx);
                        if (MODE == kWgrad) mbar_arrive(full + 8u * s);
                    }
                    sm.stage_tx[s] = tail ? 0u : tx;
                    const uint32_t dst = base + (uint32_t)(s * S::kStageBytes), dq = dst + S::kOpBytes;
                    ++g;
                    if (++s == S::kStages) {
                        s = 0;
                        parity ^= 1u;
                    }
                    const int kk = c.k0 + k;
                    if (!S::kPmn) {
                        tma_load_3d_pair(dst, &maps.p, kk, p0, z, bar);
                    } else if (pwide) {
                        tma_load_4d_pair(dst, &maps.p_wide, 0, kk, p0 >> 6, z, bar);
                    } else {
                        tma_load_3d_pair(dst, &maps.p, p0, kk, z, bar);
                        tma_load_3d_pair(dst + S::kBlock, &maps.p, p0 + 64, kk, z, bar);
                    }
                    if (MODE == kFprop) {
                        tma_load_2d_pair(dq, &maps.q[qbox], kk, q0, bar);
                    } else if (MODE == kDgrad) {
                        if (p.deep) {
                            tma_load_3d_pair(dq, &maps.q_deep[qbox], 0, q0, kk >> 6, bar);
                        } else {   // products past K read as zero
                            tma_load_2d_pair(dq, &maps.q[qbox], kk, q0, bar);
                            tma_load_2d_pair(dq + (4096 << qbox), &maps.q[qbox], kk + 64, q0, bar);
                        }
                    } else if (qwide) {
                        tma_load_4d_pair(dq, &maps.q_deep[0], 0, kk, q0 >> 6, 0, bar);
                    } else {
                        tma_load_3d_pair(dq, &maps.q[0], q0, kk, 0, bar);
                        if (half > 64) tma_load_3d_pair(dq + S::kBlock, &maps.q[0], q0 + 64, kk, 0, bar);
                    }
                }
            }
            sm.issued = (uint32_t)g;   // read by the drain, after the cluster barrier
            sm.tails = (uint32_t)tails;
            // the releases of the last stages, which the leader's MMAs signal in both CTAs, land before the end
            for (int k = max(0, g - S::kStages); ok && k < g; ++k)
                ok = mbar_wait(empty + 8u * (k % S::kStages), (uint32_t)(k / S::kStages) & 1u, abort_flag, p.flags, p.budget_ns);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // ------------------------------- MMA issuer (leader) -----------------------------
            if (elect_one()) {
                const uint32_t base = smem_u32(smem);
                const uint64_t pdesc = S::kPmn ? desc_mn_major(base, S::kBlock) : desc_k_major(base);
                const uint64_t qdesc = S::kQmn ? desc_mn_major(base + S::kOpBytes, S::kBlock) : desc_k_major(base + S::kOpBytes);
                // 16 products further: 16 rows MN-major, 32 bytes K-major (of rows of 64 products: the next
                // 64 are the next block, of the tile's box rows)
                constexpr uint32_t mn_step = 2048 >> 4, k_step = 32 >> 4;
                // fp32 accumulator, bf16 operands, transpose bits of the MN-major ones, M = 256
                constexpr uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | (S::kPmn ? 1u << 15 : 0u) |
                                            (S::kQmn ? 1u << 16 : 0u) | ((uint32_t)(256 >> 4) << 24);
                Walk<MODE> walk(p, sm, pair, pairs);
                Tile c;
                int it = 0, s = 0;
                uint32_t parity = 0, consumed = 0;   // of the slot's `full`; stages committed
                const uint32_t full = smem_u32(&sm.full[0]), empty = smem_u32(&sm.empty[0]);
                bool ok = true;
                while (ok && walk.next(c)) {
                    const uint32_t idesc = idesc0 | ((uint32_t)(c.n >> 3) << 17);
                    const uint32_t qblock = (uint32_t)((c.n >> 1) <= 32 ? 4096 : (c.n >> 1) <= 64 ? 8192 : 16384) >> 4;
                    for (int k = 0; k < c.stages; ++it) {
                        const int end = min(c.stages, k + min(run, c.stages - k));
                        const int buf = it & 1;
                        if (!mbar_wait<true>(smem_u32(&sm.tempty[buf]), ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag, p.flags, p.budget_ns)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t acc = tmem + 256u * buf;
                        uint32_t add = 0;   // an accumulator's first MMA stores
                        for (; k < end; ++k) {
                            if (!mbar_wait<MODE == kWgrad>(full + 8u * s, parity, abort_flag, p.flags, p.budget_ns)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            const uint64_t off = (uint64_t)((uint32_t)(s * S::kStageBytes) >> 4);
                            const uint64_t pd = pdesc + off, qd = qdesc + off;
                            const auto mma = [&](int j) {
                                mma_bf16_pair(acc, pd + (S::kPmn ? mn_step : k_step) * j,
                                              qd + (S::kQmn ? mn_step * j : (j >> 2) * qblock + k_step * (j & 3)), idesc, j ? 1u : add);
                            };
                            const int left = c.klen - S::kK * k;
                            if (left >= S::kK) {
#pragma unroll
                                for (int j = 0; j < S::kK / 16; ++j) mma(j);
                            } else {
#pragma unroll
                                for (int j = 0; j < S::kK / 16; ++j)
                                    if (16 * j < left) mma(j);
                            }
                            add = 1;
                            mma_commit_pair(empty + 8u * s);
                            ++consumed;
                            if (++s == S::kStages) {
                                s = 0;
                                parity ^= 1u;
                            }
                        }
                        if (!ok) break;
                        mma_commit_pair(smem_u32(&sm.tfull[buf]));
                    }
                }
                mma_commit_local(smem_u32(&sm.done));
                mbar_wait(smem_u32(&sm.done), 0u, abort_flag, p.flags, kGDrainBudgetNs, false);
                sm.consumed = consumed;
                sm.runs = (uint32_t)it;
            }
            __syncwarp();
        } else {
            // the peer's drained accumulators as one remote arrival each
            Walk<MODE> walk(p, sm, pair, pairs);
            Tile c;
            int it = 0;
            bool ok = true;
            while (ok && walk.next(c)) {
                const int stages = c.stages;
                for (int k = 0; k < stages; k += min(run, stages), ++it) {
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&sm.edrained[it & 1]), (uint32_t)(it >> 1) & 1u, abort_flag,
                                                           p.flags, p.budget_ns))) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_remote(map_rank(smem_u32(&sm.tempty[it & 1]), 0));
                    __syncwarp();
                }
            }
        }
    } else if (warp < 2 + kEpiWarps) {
        // ------------------------------- epilogue (both CTAs) --------------------------------
        const int q = warp & 3, group = (warp - 2) >> 2;   // the warp's TMEM lanes; four warps a group
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        Walk<MODE> walk(p, sm, pair, pairs);
        Tile c;
        int it = 0;
        bool ok = true;
        while (ok && walk.next(c)) {
            const int stages = c.stages;
            const int f = c.p0 + (int)rank * 128 + q * 32 + lane;
            const int64_t at = (MODE == kWgrad ? c.e * p.stride_d : 0) + (int64_t)c.q0 * p.ldd;
            const auto ready = [&](int i) {   // accumulator i of this pair is complete
                const bool full = mbar_wait(smem_u32(&sm.tfull[i & 1]), (uint32_t)(i >> 1) & 1u, abort_flag, p.flags, p.budget_ns);
                if (!__all_sync(0xFFFFFFFFu, full)) return false;
                tc_fence_after();
                return true;
            };
            const auto release = [&](int i) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(rank == 0 ? &sm.tempty[i & 1] : &sm.edrained[i & 1]));
            };
            if (stages <= run) {
                // One run (none: zeros).  Half of the warps take the even accumulators, half the odd ones,
                // so that the stores of one tile and the reads of the next overlap: 128 columns a warp,
                // 16 at a time from TMEM to their place.
                if (stages > 0 && !(ok = ready(it))) break;
                if ((group >> 1) == (it & 1)) {
                    const int c0 = (group & 1) * 16;
                    int h = c0;
#pragma unroll 1
                    for (; h < c.qn; h += 32) {
                        float v[16] = {};
                        if (stages > 0) {
                            tmem_ld16(tmem + lanes + 256u * (it & 1) + (uint32_t)h, v);
                            tmem_ld_wait();
                            if (h + 32 >= c.qn) release(it);
                        }
                        if (MODE == kWgrad || p.out_fp32)
                            put_fp32<MODE>(v, p, at + h * p.ldd, f, c.qn - h);
                        else
                            put_bf16(v, p, at + h * p.ldd, f, c.qn - h);
                    }
                    if (h == c0 && stages > 0) release(it);   // none of its own
                } else if (stages > 0) {
                    release(it);
                }
                it += stages > 0 ? 1 : 0;
                continue;
            }
            const int c0 = group * 16;   // and every 64 further
            float acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0.0f;
            for (int k = 0; k < stages; k += run, ++it) {
                if (!(ok = ready(it))) break;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    if (c0 + 64 * h < c.qn) {
#pragma unroll
                        for (int j = 0; j < 16; j += 8) {
                            float v[8];
                            tmem_ld8(tmem + lanes + 256u * (it & 1) + (uint32_t)(c0 + 64 * h + j), v);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 8; ++i) acc[16 * h + j + i] += v[i];
                        }
                    }
                }
                release(it);
            }
            if (!ok) continue;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                if (c0 + 64 * h >= c.qn) break;
                if (MODE == kWgrad || p.out_fp32)
                    put_fp32<MODE>(acc + 16 * h, p, at + (c0 + 64 * h) * p.ldd, f, c.qn - (c0 + 64 * h));
                else
                    put_bf16(acc + 16 * h, p, at + (c0 + 64 * h) * p.ldd, f, c.qn - (c0 + 64 * h));
            }
        }
    } else {
        // ------------------------------- tails (wgrad, both CTAs) ----------------------------
        // A run's last stage holds rows of the next expert behind its own.  MMAs stop at the 16 rows
        // that hold the last one; the rest of those 16 is cleared, in both operands (0 x NaN).
        Walk<MODE> walk(p, sm, pair, pairs);
        Tile c;
        // From one tail to the next may be the whole launch: a budget for each stage between them.
        int g = 0, tails = 0, waited = 0;
        while (walk.next(c)) {
            g += c.stages;
            const int last = c.klen % S::kK;
            if (!(last & 15)) continue;
            const uint64_t budget = min(p.budget_ns, (uint64_t)1 << 40) * (uint32_t)(g - waited);
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&sm.tail[tails % S::kStages]), (uint32_t)(tails / S::kStages) & 1u,
                                                   abort_flag, p.flags, budget)))
                break;
            ++tails;
            waited = g;
            const int s = (g - 1) % S::kStages;
            // a lane clears 16 bytes of each row of one of the stage's four blocks
            const uint32_t box = smem_u32(smem + s * S::kStageBytes) + (uint32_t)(lane >> 3) * (uint32_t)S::kBlock + (uint32_t)(lane & 7) * 16u;
            for (int r = last; r & 15; ++r)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(box + (uint32_t)r * 128u), "r"(0) : "memory");
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_release_cluster(map_rank(smem_u32(&sm.full[s]), 0));
        }
    }

    // Each warp hands an abort that it has seen (its own at least) to the leader.  No arrival may land in
    // a CTA that has ended.  Those that the MMAs signal are waited for: by the producers and the epilogues,
    // after an abort by the drain.  Those that the peer makes on the leader's barriers (warp 1's for a
    // pair's last accumulators are waited for by nobody) are ordered before the leader's end by a release
    // here, as is what the drain reads.  Only the epilogue arrives without one, since it makes no such
    // arrival and a release would wait for its stores of the output, which the next kernel waits for anyway.
    const bool aborted = __any_sync(0xFFFFFFFFu, *abort_flag != 0u);
    if (aborted && rank == 1 && lane == 0) st_cluster_u32(map_rank(smem_u32(&sm.peer_abort), 0), 1u);
    __syncwarp();
    tc_fence_before();
    if (aborted || warp < 2 || warp >= 2 + kEpiWarps)
        cluster_arrive();   // both producers have stopped and published what they issued
    else
        cluster_arrive_relaxed();
    cluster_wait();
    if (warp == 0 && lane == 0 && (sm.abort || sm.peer_abort)) {
        // Drain after an abort: every copy lands before its CTA exits.  (Without one it has: the leader's
        // MMA warp has waited for each stage of both CTAs, each CTA's tail warp for its tails.)  Tails land
        // on the CTA's own barriers; the other stages of both CTAs on the leader's.  A producer is at most
        // a ring ahead of the MMAs, so only the last uses of its stages can be outstanding.  The counts
        // may differ: a stage that only the peer issued has its arrivals made here, one that only the
        // leader issued has the peer's bytes cancelled.
        const int tails = (int)sm.tails;
        for (int j = max(0, tails - S::kStages); j < tails; ++j)
            mbar_wait(smem_u32(&sm.tail[j % S::kStages]), (uint32_t)(j / S::kStages) & 1u, abort_flag, p.flags, kGDrainBudgetNs, false);
        // what the MMA issuer has committed signals both CTAs
        const int consumed = (int)ld_cluster_u32(map_rank(smem_u32(&sm.consumed), 0)), runs = (int)ld_cluster_u32(map_rank(smem_u32(&sm.runs), 0));
        for (int k = max(0, consumed - S::kStages); k < consumed; ++k)
            mbar_wait(smem_u32(&sm.empty[k % S::kStages]), (uint32_t)(k / S::kStages) & 1u, abort_flag, p.flags, kGDrainBudgetNs, false);
        for (int i = max(0, runs - 2); i < runs; ++i)
            mbar_wait(smem_u32(&sm.tfull[i & 1]), (uint32_t)(i >> 1) & 1u, abort_flag, p.flags, kGDrainBudgetNs, false);
        if (rank == 0) {
            const int gl = (int)sm.issued, gp = (int)ld_cluster_u32(map_rank(smem_u32(&sm.issued), 1)), gm = max(gl, gp);
            for (int k = max(0, gm - S::kStages); k < gm; ++k) {
                const int s = k % S::kStages;
                const uint32_t bar = smem_u32(&sm.full[s]);
                const uint32_t tx = k < gl ? sm.stage_tx[s] : ld_cluster_u32(map_rank(smem_u32(&sm.stage_tx[s]), 1));
                if (tx == 0) continue;
                if (k >= gl) {
                    mbar_expect_tx(bar, tx);
                    if (MODE == kWgrad) mbar_arrive(bar);
                } else if (k >= gp) {
                    mbar_complete_tx(bar, tx);
                }
                mbar_wait(bar, (uint32_t)(k / S::kStages) & 1u, abort_flag, p.flags, kGDrainBudgetNs, false);
            }
        }
    }
    __syncwarp();
    cluster_arrive_relaxed();
    cluster_wait();   // both CTAs are done with TMEM, barriers and each other's shared memory
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <int MODE>
static cudaError_t launch(const Maps& maps, const GroupedParams& p, int64_t most_tiles, cudaStream_t s) {
    static std::atomic<uint64_t> attr{0};
    auto kern = grouped_kernel<MODE>;
    if (cudaError_t e = host::ensure_smem(reinterpret_cast<const void*>(kern), kGroupedSmem, attr)) return e;
    const int64_t pairs = std::min<int64_t>(std::max<int64_t>(most_tiles, 1), host::sm_count() / 2);
    cudaLaunchAttribute attr_pdl{};
    attr_pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr_pdl.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(Shape<MODE>::kThreads);
    cfg.dynamicSmemBytes = kGroupedSmem;
    cfg.stream = s;
    cfg.attrs = &attr_pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

// MN-major operand [slices][rows][cols] (row stride ld, slice stride `stride`): one-block boxes up to
// the width, and two-block boxes over the whole blocks (valid where there are any); `depth` products
static bool mn_maps(CUtensorMap* narrow, CUtensorMap* wide, const void* x, int64_t cols, int64_t rows, int64_t ld,
                    int64_t slices, int64_t stride, uint32_t depth) {
    const int64_t dims[4] = {cols, rows, slices, 0}, strides[3] = {ld, stride, 0};
    const uint32_t box[4] = {64, depth, 1, 0};
    if (!host::bf16_map(narrow, x, 3, dims, strides, box)) return false;
    *wide = *narrow;
    if (cols < 128) return true;
    const int64_t wdims[4] = {64, rows, cols / 64, slices}, wstrides[3] = {ld, 64, stride};
    const uint32_t wbox[4] = {64, depth, 2, 1};
    return host::bf16_map(wide, x, 4, wdims, wstrides, wbox);
}

constexpr int kFewManyN = 4096, kFewOneN = 2048;   // features from which the pair kernel has tiles enough

cudaError_t launch_gemm_grouped(const GroupedGemm& g, cudaStream_t s) {
    // A few rows only stream the weights: the kernel without set-up (grouped_few.cu), whose passes over an
    // expert's weights take 16 rows each.  How the rows lie over several experts is known on the device
    // alone, so there the rule looks at N.  16 experts of N x K, rows spread evenly, then all with one
    // expert, that kernel and the pair kernel in us:
    //   8 rows:  2048 x 1280 10.5 and 11.1, 3.7 and 7.8; 2560 x 5120 39.4 and 49.5, 11.5 and 19.0;
    //            4096 x 1408 19.7 and 19.0, 5.6 and 8.3
    //   16 rows: 2048 x 1280 19.2 and 17.8, 5.0 and 7.7; 2560 x 5120 69.6 and 78.6, 14.3 and 18.9;
    //            4096 x 1408 34.9 and 33.2, 8.6 and 8.3
    //   64 rows: 1280 x 5120 spread 40 and 50; 2048 x 1280 19.6 and 17.8, 12.8 and 8.1; 2048 x 2048 26.6 and
    //            25.9, 16.4 and 10.3; 2816 x 2048 34.1 and 35.5, 16.9 and 10.3; 2560 x 5120 70.8 and 79.1,
    //            37.7 and 19.4; 4096 x 1408 35.8 and 33.7, 16.6 and 8.7
    // So below 4096 features it gains up to a quarter where rows are spread and the pair kernel's tiles are
    // few and long, and loses up to half where more than 24 of them lie with one expert, a tenth at 2048 x
    // 1280 spread.  A rule from the number of tiles, the pairs and K would be closer; this one is not.
    // With one expert in all the passes are known: 24 rows of 4096 x 4096 16.1 and 17.3, 32 rows 17.8
    // and 17.4, 2048 x 512 3.8 and 5.4, 5.4 and 5.4; where the pair kernel has few and long tiles, 1280 x
    // 5120, 48 rows 17.0 and 18.6.
    const int64_t most = g.experts > 1 ? (g.N < kFewManyN ? kFewMaxRows : 8) : (g.N < kFewOneN && g.K >= kFewLongK ? kFewMaxRows : 24);
    if (!g.b_kn && g.rows <= most && g.experts <= kFewMaxExperts) return launch_gemm_grouped_few(g, s);
    GroupedParams p{};
    p.offsets = g.offsets;
    p.d = g.d;
    p.ldd = g.ldd;
    p.rows = (int32_t)g.rows;
    p.experts = g.experts;
    p.P = (int32_t)g.N;
    p.K = (int32_t)g.K;
    p.out_fp32 = g.out_fp32;
    p.flags = g.flags;
    p.budget_ns = g.budget_ns;
    // one weight for all experts (stride 0) is one slice of the map
    const bool many = g.experts > 1 && g.stride_b > 0;
    p.expert_step = many ? 1 : 0;
    const int64_t slices = many ? g.experts : 1, stride = many ? g.stride_b : 8;
    Maps maps;
    if (g.b_kn) {
        if (!mn_maps(&maps.p, &maps.p_wide, g.b, g.N, g.K, g.ldb, slices, stride, Shape<kDgrad>::kK)) return cudaErrorInvalidValue;
    } else {
        const int64_t dims[3] = {g.K, g.N, slices}, strides[2] = {g.ldb, stride};
        const uint32_t box[3] = {64, 128, 1};
        if (!host::bf16_map(&maps.p, g.b, 3, dims, strides, box)) return cudaErrorInvalidValue;
        maps.p_wide = maps.p;
    }
    for (int i = 0; i < 3; ++i) {
        const int64_t dims[2] = {g.K, g.rows}, strides[1] = {g.lda};
        const uint32_t box[2] = {64, 32u << i};
        if (!host::bf16_map(&maps.q[i], g.a, 2, dims, strides, box)) return cudaErrorInvalidValue;
        maps.q_deep[i] = maps.q[i];
        if (g.b_kn && g.K % 64 == 0) {
            const int64_t ddims[3] = {64, g.rows, g.K / 64}, dstrides[2] = {g.lda, 64};
            const uint32_t dbox[3] = {64, 32u << i, 2};
            if (!host::bf16_map(&maps.q_deep[i], g.a, 3, ddims, dstrides, dbox)) return cudaErrorInvalidValue;
            p.deep = 1;
        }
    }
    const int64_t tiles = ((g.N + 255) / 256) * (g.rows / 128 + std::min<int64_t>(g.rows, g.experts));
    return g.b_kn ? launch<kDgrad>(maps, p, tiles, s) : launch<kFprop>(maps, p, tiles, s);
}

cudaError_t launch_wgrad_grouped(const GroupedWgrad& g, cudaStream_t s) {
    GroupedParams p{};
    p.offsets = g.offsets;
    p.d = g.d;
    p.ldd = g.ldd;
    p.stride_d = g.stride_d;
    p.rows = (int32_t)g.rows;
    p.experts = g.experts;
    p.P = (int32_t)g.N;
    p.Q = (int32_t)g.M;
    p.out_fp32 = 1;
    p.accumulate = g.accumulate;
    p.flags = g.flags;
    p.budget_ns = g.budget_ns;
    // without rows nothing is read: the maps then stand over the output, which is there
    const int64_t rows = std::max<int64_t>(g.rows, 1);
    const void* b = g.rows ? (const void*)g.b : (const void*)g.d;
    const void* a = g.rows ? (const void*)g.a : (const void*)g.d;
    Maps maps;
    if (!mn_maps(&maps.p, &maps.p_wide, b, g.N, rows, g.ldb, 1, 8, Shape<kWgrad>::kK) ||
        !mn_maps(&maps.q[0], &maps.q_deep[0], a, g.M, rows, g.lda, 1, 8, Shape<kWgrad>::kK))
        return cudaErrorInvalidValue;
    maps.q[1] = maps.q[2] = maps.q_deep[1] = maps.q_deep[2] = maps.q[0];   // unused
    const int64_t tiles = ((g.N + 255) / 256) * ((g.M + 127) / 128) * g.experts;
    return launch<kWgrad>(maps, p, tiles, s);
}

}  // namespace nvfp4
