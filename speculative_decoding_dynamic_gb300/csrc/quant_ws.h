// Launchers of the 8-bit KV cache, the 4-bit LM head, the 8-bit product and
// norm, the token log-probabilities and the distillation loss. Not part of the
// public ABI.
#pragma once

#include "eagle_ws.h"

namespace eagle {

// The 8-bit KV cache (eagle_kvq_cfg, checked): strides of codes in bytes, of
// scales in elements.
struct KvqDims {
    int B, Hq, Hkv, layers, max_len, block;
    int64_t seq_stride, layer_stride, kv_stride, pos_stride;
    int64_t s_seq, s_layer, s_kv, s_blk;
};
constexpr int kKvqHeadDim = 128;
cudaError_t launch_kvq_store(const KvqDims& kv, int layer, int T, const void* k, const void* v, int64_t row_stride,
                             const int32_t* row_start, const int32_t* start, const int32_t* count, void* codes,
                             float* scales, int* status, cudaStream_t stream);
cudaError_t launch_kvq_compact(const KvqDims& kv, void* codes, float* scales, const int32_t* prefix_len,
                               const int32_t* accept_len, const int32_t* slots, int slots_stride, int32_t* new_len,
                               int* status, cudaStream_t stream);
size_t kvq_attention_ws_bytes(const KvqDims& kv, int T);
cudaError_t launch_kvq_attention(const KvqDims& kv, int T, const void* q, const void* codes, const float* scales,
                                 int layer, const int32_t* prefix_len, const uint32_t* mask, const int32_t* n_tree,
                                 void* out, void* ws, cudaStream_t stream);

// LM-head logits [M, V] of hidden [M, H] (bf16) and 4-bit weights.
constexpr int kLmQuantMaxHidden = 8192;  // eight hidden rows of it fit in shared memory beside the ring
cudaError_t launch_lmhead_quant(int M, int V, int H, int group, const void* hidden, const void* codes,
                                const void* scales, int out_dtype, void* out, int* status, cudaStream_t stream);
cudaError_t launch_lmhead_quant_pack(int V, int H, int group, const void* weight, void* codes, void* scales,
                                     cudaStream_t stream);

struct LogprobArgs {
    int n, per_seq, rows_per_seq, V, n_alt;  // n = n_seq * per_seq entries
    float temperature;
    const void* logits;
    const int32_t *slots, *tokens;
    float *logprob, *entropy, *alt_logprobs;
    int32_t *rank, *alt_ids;
    int* status;
};
cudaError_t launch_token_logprobs(const LogprobArgs& a, int dtype, cudaStream_t stream);

// Rows of e4m3 codes with a power-of-two scale (a byte, E8M0) for each 128 entries.
constexpr int kFp8Block = 128;
constexpr int kFp8MaxNormDim = 16384;  // a row's entries in the registers of 1024 threads
inline int fp8_scale_stride(int dim) { return ((dim - 1) / (4 * kFp8Block) + 1) * 4; }  // dim >= 1, up to the largest int
struct RmsnormFp8Args {
    int rows, dim, scale_stride;
    int64_t row_stride;  // elements
    const void *x, *residual, *weight;
    void* sum;
    float eps, inv_dim, inv_dim_lo;  // 1 / dim as a sum of two
    void* codes;
    uint8_t* scales;
    int* status;
};
cudaError_t launch_rmsnorm_fp8(const RmsnormFp8Args& a, int dtype, cudaStream_t stream);
cudaError_t launch_fp8_pack(int N, int K, int scale_stride, const void* weight, void* codes, uint8_t* scales,
                            cudaStream_t stream);
// out [M, N] = x [M, K] w [N, K]^T, both of codes and scales.
cudaError_t launch_linear_fp8(int M, int N, int K, const void* x, const uint8_t* x_scales, const void* w,
                              const uint8_t* w_scales, int out_dtype, void* out, int* status, cudaStream_t stream);

// The same for one row of x or two, without the tensor cores.
cudaError_t launch_linear_fp8_rows(int M, int N, int K, const void* x, const uint8_t* x_scales, const void* w,
                                   const uint8_t* w_scales, int out_dtype, void* out, cudaStream_t stream);

constexpr int kDistillMaxTop = 256;  // a teacher's list: one thread of a CTA for each entry
struct DistillArgs {
    int rows, V, n_top;
    float temperature;
    const void* logits;
    const int32_t* ids;
    const float *teacher, *teacher_lse, *row_weight;
    float* loss;
    void* grad;
    int* status;
};
cudaError_t launch_distill(const DistillArgs& a, int dtype, cudaStream_t stream);

}  // namespace eagle
