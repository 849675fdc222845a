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

}  // namespace lora
