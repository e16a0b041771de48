// nvfp4_internal.h -- declarations shared by the CUDA translation units of libnvfp4.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace nvfp4 {

// workspace layout (256 bytes, caller-owned device memory)
struct Workspace {
    uint32_t flags;       // kFlag* bits, sticky until nvfp4_poll
    uint32_t amax_a;      // fp32 bits: plain amax of the last quantize call
    uint32_t amax_b;      // fp32 bits: amax after the RHT
    uint32_t pad[61];
};
static_assert(sizeof(Workspace) == 256, "workspace is 256 bytes");

constexpr uint32_t kFlagNonFinite = 1u;
constexpr uint32_t kFlagTimeout = 2u;
constexpr uint32_t kFlagOffsets = 4u;   // expert offsets out of order or range

// the 16 RHT signs as bf16-pair masks (0x80008000 for a -1 sign), a by-value kernel parameter
struct SignMasks {
    uint32_t m[16];
};
inline SignMasks sign_masks(uint32_t signs) {
    SignMasks s;
    for (int j = 0; j < 16; ++j) s.m[j] = ((signs >> j) & 1u) ? 0x80008000u : 0u;
    return s;
}

// parameters of the tile quantizer (one read of x, up to two forms)
struct QuantParams {
    const uint16_t* x;
    int64_t rows, cols, ld;
    int32_t block16;  // 1: 16x16 tiles (both forms share the tile scale)
    // ROW form: K = cols
    uint8_t* codes_row;
    uint8_t* scales_row;
    uint8_t* tiles_row;
    float* st_row;
    const uint32_t* amax_row;
    int64_t nkt_row;
    int32_t sr_row;
    uint32_t stream_row;
    // COL form: K = rows (the transposed operand)
    uint8_t* codes_col;
    uint8_t* scales_col;
    uint8_t* tiles_col;
    float* st_col;
    const uint32_t* amax_col;
    int64_t nkt_col;
    int32_t sr_col;
    int32_t rht_col;
    uint32_t stream_col;
    uint32_t signs;
    uint64_t sr_seed;
    uint32_t* flags;  // workspace flags (timeout of a tile copy)
    // filled by launch_quantize_tiles (constant-bank operands in the kernel):
    uint32_t sign_mask2[16];  // RHT sign j as a bf16-pair mask: 0x80008000 when sign j is -1, else 0
    uint32_t key0[10];        // Philox4x32-10 round keys of sr_seed (Weyl sequence of its two words)
    uint32_t key1[10];
    // SR bit indexing of a token shard: x holds rows [row_offset, row_offset + rows) of a
    // rows_total-row tensor, and SR fields are indexed in the forms of that whole tensor
    int64_t row_offset;
    int64_t rows_total;
};

// parameters of the MXFP4 tile quantizer (one form per call)
struct MxParams {
    const uint16_t* x;
    int64_t rows, cols, ld;    // the bf16 source [rows][ld]
    // the row form (K = cols) and the column form (K = rows); a call fills the forms it launches
    uint8_t* codes;            // row form's codes [rows][cols/2]
    uint8_t* scales;           // its UE8M0 scales in 128x4 tiles
    int64_t nkt;               // ceil(cols / 128): 128x4 scale tiles per 128 form rows
    uint32_t stream_id;        // its SR stream
    uint8_t* codes_col;        // column form's codes [cols][rows/2]
    uint8_t* scales_col;
    int64_t nkt_col;           // ceil(rows / 128)
    uint32_t stream_col;
    int32_t sr;                // 1: stochastic rounding (both forms)
    uint32_t* flags;           // workspace flags (timeout of a tile copy)
    uint32_t key0[10];         // Philox4x32-10 round keys of the SR seed
    uint32_t key1[10];
};

cudaError_t launch_quantize_mx(const MxParams& p, bool row_form, bool column_form, uint64_t sr_seed, cudaStream_t s);

cudaError_t launch_amax_plain(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, uint32_t* amax,
                              uint32_t* flags, cudaStream_t s);
cudaError_t launch_amax_rht(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, uint32_t signs,
                            uint32_t* amax_plain, uint32_t* amax_rht, uint32_t* flags, cudaStream_t s);
cudaError_t launch_quantize_tiles(const QuantParams& p, cudaStream_t s);
cudaError_t launch_transpose_2d(const uint8_t* codes, const uint8_t* tiles, int64_t R, int64_t K, uint8_t* codes_t,
                                uint8_t* scales_t, uint8_t* tiles_t, const float* st_in, float* st_out,
                                cudaStream_t s);
cudaError_t launch_gemm_nvf4(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_st, int64_t M,
                             const uint8_t* b_codes, const uint8_t* b_scales, const float* b_st, int64_t N, int64_t K,
                             void* d, int64_t ldd, bool out_fp32, uint32_t* flags, uint64_t budget_ns,
                             cudaStream_t stream);
cudaError_t launch_gemm_nvf4_reduce_scatter(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_st, int64_t M,
                                            const uint8_t* b_codes, const uint8_t* b_scales, const float* b_st, int64_t N,
                                            int64_t K, float* const* shards, int n_owners, int64_t owner_rows, int64_t ldd,
                                            uint32_t* flags, uint64_t budget_ns, cudaStream_t stream);
cudaError_t launch_gemm_nvf4_amax(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_st, int64_t M,
                                  const uint8_t* b_codes, const uint8_t* b_scales, const float* b_st, int64_t N, int64_t K,
                                  void* d, int64_t ldd, uint32_t* amax_out, uint32_t rht_signs, uint32_t* flags,
                                  uint64_t budget_ns, cudaStream_t stream);
cudaError_t launch_gemm_mxf4(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M, const uint8_t* b_codes,
                             const uint8_t* b_scales, int64_t N, int64_t K, void* d, int64_t ldd, bool out_fp32,
                             uint32_t* flags, uint64_t budget_ns, cudaStream_t stream);
cudaError_t launch_gemm_bf16(const uint16_t* a, int64_t lda, const uint16_t* b, int64_t ldb, int64_t M, int64_t N,
                             int64_t K, void* d, int64_t ldd, bool out_fp32, uint32_t* flags, uint64_t budget_ns,
                             cudaStream_t stream);
cudaError_t launch_transpose_bf16(const uint16_t* x, int64_t rows, int64_t cols, int64_t ldx, uint16_t* xt, int64_t ldt,
                                  cudaStream_t s);
cudaError_t launch_gelu_fwd(const uint16_t* h, uint16_t* g, int64_t n, cudaStream_t s);
cudaError_t launch_gelu_bwd(const uint16_t* h, const uint16_t* dg, uint16_t* dh, int64_t n, cudaStream_t s);
cudaError_t launch_gelu_amax(bool bwd, const uint16_t* h, const uint16_t* dg, uint16_t* out, int64_t rows,
                             int64_t cols, uint32_t signs, uint32_t* amax_plain, uint32_t* amax_rht, uint32_t* flags,
                             cudaStream_t s);

// Products grouped by expert.  offsets: device int32 [experts + 1]; expert e owns the rows from the
// running maximum (clamped to [0, rows]) of offsets[0..e] up to that of offsets[0..e+1].
constexpr int kMaxExperts = 1024;
struct GroupedGemm {        // D[t] = A[t] . B_e^T (b_kn = 0, B_e [N][K]) or A[t] . B_e (b_kn = 1, B_e [K][N])
    const uint16_t* a;
    const uint16_t* b;
    void* d;
    const int32_t* offsets;
    int64_t lda, ldb, stride_b, ldd;
    int64_t rows, N, K;
    int experts;
    bool b_kn, out_fp32;
    uint32_t* flags;
    uint64_t budget_ns;
};
struct GroupedWgrad {       // D_e[m][n] (+)= sum over e's rows t of A[t][m] B[t][n]
    const uint16_t* a;
    const uint16_t* b;
    float* d;
    const int32_t* offsets;
    int64_t lda, ldb, ldd, stride_d;
    int64_t rows, M, N;
    int experts;
    bool accumulate;
    uint32_t* flags;
    uint64_t budget_ns;
};
cudaError_t launch_gemm_grouped(const GroupedGemm& g, cudaStream_t s);
constexpr int kFewMaxRows = 64, kFewMaxExperts = 256, kFewLongK = 2048;
cudaError_t launch_gemm_grouped_few(const GroupedGemm& g, cudaStream_t s);   // within those, b_kn = 0
cudaError_t launch_wgrad_grouped(const GroupedWgrad& g, cudaStream_t s);

// AdamW: one tensor of a launch (80 bytes: a launch's table fits the 32764 bytes of kernel parameters)
constexpr int kAdamMaxTensors = 384;
constexpr uint32_t kStreamMoment1 = 4u, kStreamMoment2 = 5u;
struct AdamwEntry {
    float* p;
    const void* g;
    uint16_t* w;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    uint32_t* amax;
    int64_t n;
    uint32_t first_chunk;   // set by the launcher
    int32_t index_g;        // the tensor's index in the call << 1 | (gradient is bf16)
};
struct AdamwDynamic {       // nvfp4_adamw_dynamic
    float keep, step_size, v_fix, grad_scale;
    uint64_t sr_seed, reserved;
};
struct AdamwScalars {
    float keep, step_size, v_fix, grad_scale;
    float beta1, one_beta1, beta2, one_beta2, eps;
    int32_t sr;
    uint64_t sr_seed;
    const AdamwDynamic* dynamic;
};
cudaError_t launch_adamw(const AdamwEntry* entries, int count, bool fp8, const AdamwScalars& sc, uint32_t* flags,
                         cudaStream_t s);

// host-side Philox4x32-10 (same algorithm as the device one) for the RHT sign draw
uint32_t rht_signs_host(uint64_t seed);

}  // namespace nvfp4
