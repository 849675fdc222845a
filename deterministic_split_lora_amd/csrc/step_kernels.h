// Internal interface between the C entry points of the operators around the
// adapters (abi_step.hip) and their kernel files: MX4 (microscaled 4-bit
// floating point), the norm / gate / residual step and sampling.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lora {

constexpr int kMxBlock = 32;                 // elements that share one E8M0 scale
constexpr int kNormMaxC = 32768;             // widest row of the block norm

struct Mx4QuantParams {
    const uint16_t* x;              // quantise: bf16 in
    uint16_t* x_out;                // dequantise: bf16 out
    int64_t ld_x;
    uint8_t* q;
    int64_t ld_q;                   // bytes
    uint8_t* scales;
    int64_t ld_s;                   // bytes
    int64_t M;
    int32_t K;
};

hipError_t launch_mx4_quantize(const Mx4QuantParams& p, hipStream_t st);
hipError_t launch_mx4_dequantize(const Mx4QuantParams& p, hipStream_t st);

struct Mx4LinearParams {
    const void* x;                  // bf16 [M][ld_x], or packed codes [M][ld_x bytes]
    int64_t ld_x;                   // elements (bf16) or bytes (codes)
    const uint8_t* xs;              // scales of x (codes only)
    int64_t ld_xs;
    const uint8_t* wq;              // [N][ld_wq bytes]
    int64_t ld_wq;
    const uint8_t* ws;              // [N][ld_ws bytes]
    int64_t ld_ws;
    uint16_t* y;                    // bf16 [M][ld_y]
    int64_t ld_y;
    float* partial;                 // workspace of the split schedule
    int64_t M;
    int64_t N;
    int32_t k_chunk;                // K / split_k, a multiple of 32
    int32_t split_k;
};

// Bytes of workspace launch_mx4_linear may take for these sizes (0: none), with
// either kind of x and any alignment of the scales.
int64_t mx4_linear_workspace(int64_t M, int64_t N, int32_t k_chunk, int32_t split_k);
hipError_t launch_mx4_linear(const Mx4LinearParams& p, bool x_is_mx4, hipStream_t st);

struct NormParams {
    const uint16_t* y;              // may be null: no block output
    int64_t ld_y;
    const uint16_t* post_w;         // may be null: 1
    const uint16_t* post_b;         // may be null: 0
    const uint16_t* gate;           // may be null: 1
    int64_t ld_gate;
    int64_t gate_group;             // rows of y per row of gate
    const uint16_t* r;
    int64_t ld_r;
    uint16_t* r_out;
    int64_t ld_ro;
    const uint16_t* pre_w;
    const uint16_t* pre_b;
    uint16_t* x_out;                // may be null: no pre-norm
    int64_t ld_xo;
    int64_t M;
    int32_t C;
    int32_t post;                   // lora_norm_kind
    int32_t pre;
    float res_scale;
    float eps;
};

hipError_t launch_block_norm(const NormParams& p, hipStream_t st);

struct SampleParams {
    const void* logits;
    int64_t ld;
    const float* temperature;       // each may be null: 1, off, off, off
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* u;
    int32_t* tokens;
    float* logprobs;                // may be null
    int32_t V;
    int64_t B;
};

hipError_t launch_sample(const SampleParams& p, bool bf16, hipStream_t st);

struct VerifyParams {
    const void* target;             // [B * (n + 1)][ld_t]
    const void* draft;              // [B * n][ld_d], may be null: drafts of certainty
    int64_t ld_t;
    int64_t ld_d;
    const int32_t* drafted;         // [B][n]
    const float* u;                 // [B][n + 1]
    const float* temperature;       // each may be null: 1, off, off, off
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    int32_t* tokens;                // [B][n + 1]
    int32_t* accepted;              // [B]
    float* logprobs;                // [B][n + 1], may be null
    void* workspace;
    int32_t V;
    int32_t n;
    int64_t B;
};

constexpr int kMaxDrafts = 63;               // of a sequence: a lane each, and one for the row behind them

// Bytes of workspace, and threads of the largest launch.
int64_t verify_workspace(int64_t B, int64_t n);
int64_t verify_threads(int64_t B, int64_t n, int64_t V);
hipError_t launch_verify(const VerifyParams& p, bool bf16, hipStream_t st);

constexpr int kKvBlock = 16;                 // tokens that share a scale in the cache

// The paged cache and the batch's tables (kv_cache.h has the layouts).
struct KvCacheView {
    uint8_t* k;
    uint8_t* v;
    uint8_t* k_scales;
    uint8_t* v_scales;
    int64_t ld_k;                   // bytes from page to page
    int64_t ld_v;
    int64_t ld_ks;
    int64_t ld_vs;
    const int32_t* page_table;      // [n_seqs][ld_table], max_pages used
    int64_t ld_table;
    int64_t max_pages;
    const int32_t* seq_lens;        // [n_seqs]
    const int32_t* cu_tokens;       // [n_seqs + 1]
    int64_t n_seqs;
    int32_t n_pages;
    int32_t page_size;              // a power of two, 16 at least
    int32_t page_shift;
    int32_t heads;                  // of keys and values
};

struct KvAppendParams {
    KvCacheView cache;
    const uint16_t* q;              // may be null: no queries
    int64_t ld_q;
    uint16_t* q_out;
    int64_t ld_qo;
    const uint16_t* k;
    int64_t ld_k;
    const uint16_t* v;
    int64_t ld_v;
    const uint16_t* q_norm;         // each may be null: no norm
    const uint16_t* k_norm;
    const float* rope;              // may be null: no rotation
    int64_t ld_rope;
    int64_t rope_rows;
    int64_t T;
    int32_t rope_dim;
    int32_t pairs;
    int32_t q_heads;
    int32_t D;
    float eps;
};

hipError_t launch_kv_append(const KvAppendParams& p, hipStream_t st);

struct KvAttentionParams {
    KvCacheView cache;
    const uint16_t* q;
    int64_t ld_q;
    uint16_t* out;
    int64_t ld_out;
    float* lse;                     // may be null
    int64_t ld_lse;
    float* partial;                 // workspace of several chunks
    int64_t T;
    int64_t max_len;
    int64_t chunk;                  // keys of a chunk, a multiple of kKvChunkUnit
    int64_t max_new;
    int32_t q_heads;
    int32_t D;
    int32_t causal;
    int32_t window;                 // 0: none
    float scale;
};

constexpr int kKvChunkUnit = 256;

// The chunk that these sizes get by default.
int64_t kv_attention_chunk(int64_t max_new, int32_t q_heads, int32_t kv_heads, int32_t D, int64_t max_len);
// Bytes of workspace (0: one chunk) and blocks of a launch with these sizes.
int64_t kv_attention_workspace(int64_t T, int32_t q_heads, int32_t D, int64_t max_len, int64_t chunk);
int64_t kv_attention_blocks(int64_t T, int64_t n_seqs, int64_t max_new, int32_t q_heads, int32_t kv_heads, int32_t D,
                            int64_t max_len, int64_t chunk);
hipError_t launch_kv_attention(const KvAttentionParams& p, hipStream_t st);

}  // namespace lora
