// kernels.hpp -- internal launch functions of libe2m1lut.so (not part of the C ABI).
// Arguments are validated by the C entry points in api.hip before these run.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace e2m1 {

// Compute units of the current device (cached per device).
int device_cu_count();

hipError_t launch_fill_zero_u16(uint16_t* dst, int64_t count, hipStream_t stream);

hipError_t launch_decode(const uint8_t* packed, const uint8_t* scales, uint16_t* out,
                         int64_t nblocks, hipStream_t stream);

hipError_t launch_mxfp4_quantize(const uint16_t* x, uint8_t* packed, uint8_t* scales, int64_t nblocks,
                                 hipStream_t stream);

hipError_t launch_nvfp4_quantize(const uint16_t* x, const float* global_scale, uint8_t* packed,
                                 uint8_t* block_scale, int64_t nblocks, hipStream_t stream);

hipError_t launch_gemv(const uint8_t* packed, const uint8_t* scales, const uint16_t* x, void* y,
                       bool out_bf16, int batch, int64_t n, int64_t k, hipStream_t stream);

// One batch-1 product of a grouped launch (host-side descriptor).
struct GemvMatrix {
    const uint8_t* packed;
    const uint8_t* scales;
    const uint16_t* x;
    void* y;
    int64_t n, k;
};
constexpr int kGemvGroupMax = 64;   // E2M1_GEMV_MAX_GROUPS
// count <= kGemvGroupMax matrices with n >= 1 and k >= 32 (validated by the caller).
hipError_t launch_gemv_group(const GemvMatrix* mats, int count, bool out_bf16, hipStream_t stream);

hipError_t launch_gemm(const uint8_t* packed, const uint8_t* scales, const uint16_t* x, void* y, bool out_bf16,
                       int64_t m, int64_t n, int64_t k, hipStream_t stream);

hipError_t launch_nm_spmm(const uint16_t* values, const uint32_t* meta, const uint16_t* x, void* y, bool out_bf16,
                          int64_t batch, int64_t rows, int64_t k, int nn, int mm, hipStream_t stream);

// bf16 (or fp32) rows -> int8 codes and one scale per row; k % 16 == 0, k >= 16.
hipError_t launch_int8_quantize(const void* x, bool bf16, int8_t* q, float* scale, int64_t rows, int64_t k,
                                hipStream_t stream);
// residual (and then residual_out) may be null
hipError_t launch_rmsnorm_int8_quantize(const void* x, const void* residual, const void* weight, bool bf16, float eps,
                                        void* residual_out, int8_t* q, float* scale, int64_t rows, int64_t k,
                                        hipStream_t stream);
hipError_t launch_silu_mul_int8_quantize(const void* gate_up, bool bf16, int8_t* q, float* scale, int64_t rows,
                                         int64_t inter, hipStream_t stream);

hipError_t launch_int8_gemm(const int8_t* x, const float* x_scale, const int8_t* w, const float* w_scale,
                            const float* bias, void* y, bool out_bf16, int64_t m, int64_t n, int64_t k,
                            hipStream_t stream);

// A paged MXFP4 cache of keys and values: codes [pages, heads, page, head_dim / 2], scales [.., head_dim / 32].
struct CacheView {
    uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    int64_t slots;       // pages * page size
    int heads, head_dim; // head_dim 64 or 128
    int page_bits;       // log2 of the page size
};

// Rows k [tokens, heads, head_dim] and v (row strides in elements) -> the cache's slots; err_flag may be null.
hipError_t launch_cache_write(const void* k, const void* v, bool bf16, int64_t k_stride, int64_t v_stride,
                              const int64_t* slots, const CacheView& c, int64_t tokens, int32_t* err_flag,
                              hipStream_t stream);

struct NormRope {
    const void* qkv;
    int64_t stride;
    const void *q_weight, *k_weight;   // each may be null: that norm is left out
    float eps;
    const float* cos_sin;              // [max_pos, rot]
    int64_t max_pos;
    int rot;                           // a multiple of 16, 0: no rotation
    bool interleaved;
    const int64_t *positions, *slots;
    uint16_t* q_out;
    int heads;
};
hipError_t launch_norm_rope_write(const NormRope& a, bool bf16, const CacheView& c, int64_t tokens, int32_t* err_flag,
                                  hipStream_t stream);

hipError_t launch_cache_read(const CacheView& c, const int64_t* slots, uint16_t* k_out, uint16_t* v_out, int64_t tokens,
                             int32_t* err_flag, hipStream_t stream);

struct Attention {
    const uint16_t* q;
    int64_t q_stride;
    const int32_t *page_table, *kv_lens, *q_offsets;
    const float* sinks;   // may be null
    float scale;
    bool causal;
    int64_t window;       // 0: none
    uint16_t* out;
    int64_t tokens, seqs;
    int heads;
    int64_t table_width;
    int32_t* err_flag;
};
size_t attention_workspace_bytes(int64_t tokens, int64_t seqs, int64_t heads, int64_t kv_heads, int64_t head_dim);
hipError_t launch_attention(const Attention& a, const CacheView& c, void* workspace, size_t workspace_bytes,
                            hipStream_t stream);

hipError_t launch_ternary(const uint32_t* packed, const float* row_scale, const float* x, float* y,
                          int64_t n, int64_t k, hipStream_t stream);

// Device workspace launch_ternary_gemm uses for (batch, k); 0 where it takes the one-launch kernels.
size_t ternary_gemm_workspace_bytes(int64_t batch, int64_t k);
hipError_t launch_ternary_gemm(const uint32_t* packed, const float* row_scale, const float* x, float* y,
                               int64_t batch, int64_t n, int64_t k, void* workspace, hipStream_t stream);

hipError_t launch_ternary_wl(const uint32_t* const mats[4], const float* scale, const float* x_re,
                             const float* x_im, float* y_re, float* y_im, int64_t n, int64_t k,
                             hipStream_t stream);

hipError_t launch_nvfp4_gather(const uint8_t* table, const uint8_t* block_scale,
                               const float* global_scale, const int64_t* ids, uint16_t* out,
                               int64_t vocab, int64_t hidden, int64_t ntok, int32_t* err_flag,
                               hipStream_t stream);

size_t moe_workspace_bytes(int64_t tokens, int64_t hidden, int64_t inter, int64_t experts,
                           int64_t topk);

hipError_t launch_moe(const uint16_t* x, const uint8_t* w13, const uint8_t* w13s,
                      const uint8_t* w2, const uint8_t* w2s, const int32_t* ids,
                      const float* weights, uint16_t* out, void* workspace, int64_t tokens,
                      int64_t hidden, int64_t inter, int64_t experts, int64_t topk,
                      hipStream_t stream);

}  // namespace e2m1

// Which form int8_gemm takes for a product on a device of `cus` compute units: the place of its shape in the table for
// rows of whole 128-byte lines or in the other one, one more for 256 x 256 tiles whose last round is halved. Host only;
// exported for the tests, which have to reach every form.
extern "C" int e2m1_int8_gemm_variant(int64_t m, int64_t n, int64_t k, int whole_lines, int cus);

// Which form mxfp4_attention takes for rows that see up to `length` tokens: 10 * tiles of 16 rows a wave + waves of a
// worker, + 100 for whole segments, + 200 for cut ones, + 1000 where their joins go by worker, + 2000 where a workgroup
// joins a row. Host only; exported for the tests, which have to reach every form.
extern "C" int e2m1_mxfp4_attention_form(int64_t tokens, int64_t seqs, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                         int64_t length);
