// Launchers of the 8-bit KV cache, the 4-bit LM head and the token
// log-probabilities. Not part of the public ABI.
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

}  // namespace eagle
