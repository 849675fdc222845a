// C entry points of the operators around the adapters (declared in
// include/lora_det.h): MX4 quantisation and products, the block norm, sampling.
// As in abi.hip, every scalar and pointer is checked on the host before any HIP
// call, and nothing here allocates, frees or synchronises.
#include "../../include/lora_det.h"
#include "step_kernels.h"

using namespace lora;

namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxGrid = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxGridY = 65535;
constexpr int64_t kMaxColumns = int64_t{1} << 25;      // of a product
constexpr int64_t kMaxTiles = int64_t{1} << 22;        // 64 x 128 tiles of a product's y
constexpr int64_t kMaxDraws = int64_t{1} << 21;        // rows of one sampling call
constexpr int64_t kMaxPitch = int64_t{1} << 23;        // bytes; 256 rows stay below 2^32
constexpr int64_t kMaxVocabulary = int64_t{1} << 22;   // a row's weight stays below 2^53

bool aligned(const void* p, unsigned n)
{
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

int launch_status(hipError_t e)
{
    return e == hipSuccess ? LORA_OK : LORA_ERR_LAUNCH;
}

// One MX4 operand: codes and scales of rows of K values.
int check_mx4(const uint8_t* q, int64_t ld_q, const uint8_t* s, int64_t ld_s, int64_t K)
{
    if (ld_q < K / 2 || ld_s < K / kMxBlock)
        return LORA_ERR_SHAPE;
    if (ld_q > kMaxPitch)
        return LORA_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || ld_q % 16 || !aligned(s, 4) || ld_s % 4)
        return LORA_ERR_ALIGN;
    return LORA_OK;
}

int check_mx4_convert(const uint16_t* x, int64_t ld_x, const uint8_t* q, int64_t ld_q, const uint8_t* s,
                      int64_t ld_s, int64_t M, int64_t K)
{
    if (M < 0 || M > kMaxDim || K <= 0 || K > kMaxDim)
        return LORA_ERR_SHAPE;
    if (K % kMxBlock)
        return LORA_ERR_UNSUPPORTED;
    if (M * ((K + 2047) / 2048) > kMaxGrid)
        return LORA_ERR_SHAPE;
    if (M == 0)
        return LORA_OK;
    if (!x || !q || !s)
        return LORA_ERR_NULL;
    if (ld_x < K)
        return LORA_ERR_SHAPE;
    const int st = check_mx4(q, ld_q, s, ld_s, K);
    if (st != LORA_OK)
        return st;
    return aligned(x, 16) && ld_x % 8 == 0 ? LORA_OK : LORA_ERR_ALIGN;
}

Mx4QuantParams convert_params(const uint8_t* q, int64_t ld_q, const uint8_t* s, int64_t ld_s, int64_t ld_x, int64_t M,
                              int64_t K)
{
    Mx4QuantParams p{};
    p.q = const_cast<uint8_t*>(q);
    p.ld_q = ld_q;
    p.scales = const_cast<uint8_t*>(s);
    p.ld_s = ld_s;
    p.ld_x = ld_x;
    p.M = M;
    p.K = (int32_t)K;
    return p;
}

// Sizes of the products; 0 rows or columns are valid and leave nothing to do.
int check_linear_sizes(int64_t M, int64_t K, int64_t N, int32_t split_k)
{
    if (M < 0 || M > kMaxDim || N < 0 || N > kMaxDim || K <= 0 || K > kMaxDim)
        return LORA_ERR_SHAPE;
    if (split_k != 1 && split_k != 2 && split_k != 4 && split_k != 8 && split_k != 16)
        return LORA_ERR_UNSUPPORTED;
    if (K % (kMxBlock * (int64_t)split_k) || N % 8)
        return LORA_ERR_UNSUPPORTED;
    // what a launch holds: fewer than 2^32 threads
    if ((M + 63) / 64 > kMaxGridY || N > kMaxColumns || ((M + 63) / 64) * ((N + 127) / 128) > kMaxTiles)
        return LORA_ERR_SHAPE;
    return LORA_OK;
}

// The checks and the launch behind both products.
int linear(const void* x, int64_t ld_x, const uint8_t* xs, int64_t ld_xs, const uint8_t* wq, int64_t ld_wq,
           const uint8_t* ws, int64_t ld_ws, uint16_t* y, int64_t ld_y, int64_t M, int64_t K, int64_t N,
           int32_t split_k, void* workspace, size_t workspace_bytes, void* stream, bool x_is_mx4)
{
    int st = check_linear_sizes(M, K, N, split_k);
    if (st != LORA_OK || M == 0 || N == 0)
        return st;
    if (!x || !wq || !ws || !y || (x_is_mx4 && !xs))
        return LORA_ERR_NULL;
    if (ld_y < N || (!x_is_mx4 && ld_x < K))
        return LORA_ERR_SHAPE;
    if ((!x_is_mx4 && ld_x > kMaxPitch / 2) || ld_ws > kMaxPitch || ld_xs > kMaxPitch)
        return LORA_ERR_UNSUPPORTED;
    if (x_is_mx4 && (st = check_mx4(static_cast<const uint8_t*>(x), ld_x, xs, ld_xs, K)) != LORA_OK)
        return st;
    if ((st = check_mx4(wq, ld_wq, ws, ld_ws, K)) != LORA_OK)
        return st;
    if (!aligned(x, 16) || !aligned(y, 16) || ld_y % 8 || (!x_is_mx4 && ld_x % 8) || !aligned(workspace, 16))
        return LORA_ERR_ALIGN;
    const size_t need = mx4_linear_workspace(M, N, (int32_t)(K / split_k), split_k);
    if (need > workspace_bytes)
        return LORA_ERR_WORKSPACE;
    if (need && !workspace)
        return LORA_ERR_NULL;
    Mx4LinearParams p{};
    p.x = x;
    p.ld_x = ld_x;
    p.xs = xs;
    p.ld_xs = ld_xs;
    p.wq = wq;
    p.ld_wq = ld_wq;
    p.ws = ws;
    p.ld_ws = ld_ws;
    p.y = y;
    p.ld_y = ld_y;
    p.partial = static_cast<float*>(workspace);
    p.M = M;
    p.N = N;
    p.k_chunk = (int32_t)(K / split_k);
    p.split_k = split_k;
    return launch_status(launch_mx4_linear(p, x_is_mx4, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {
#pragma GCC visibility push(default)

int lora_mx4_quantize(const uint16_t* x, int64_t ld_x, uint8_t* q, int64_t ld_q, uint8_t* scales, int64_t ld_s,
                      int64_t M, int64_t K, void* stream)
{
    const int st = check_mx4_convert(x, ld_x, q, ld_q, scales, ld_s, M, K);
    if (st != LORA_OK || M == 0)
        return st;
    Mx4QuantParams p = convert_params(q, ld_q, scales, ld_s, ld_x, M, K);
    p.x = x;
    return launch_status(launch_mx4_quantize(p, static_cast<hipStream_t>(stream)));
}

int lora_mx4_dequantize(const uint8_t* q, int64_t ld_q, const uint8_t* scales, int64_t ld_s, uint16_t* x,
                        int64_t ld_x, int64_t M, int64_t K, void* stream)
{
    const int st = check_mx4_convert(x, ld_x, q, ld_q, scales, ld_s, M, K);
    if (st != LORA_OK || M == 0)
        return st;
    Mx4QuantParams p = convert_params(q, ld_q, scales, ld_s, ld_x, M, K);
    p.x_out = x;
    return launch_status(launch_mx4_dequantize(p, static_cast<hipStream_t>(stream)));
}

size_t lora_mx4_linear_workspace_bytes(int64_t M, int64_t K, int64_t N, int32_t split_k)
{
    if (check_linear_sizes(M, K, N, split_k) != LORA_OK || M == 0 || N == 0)
        return 0;
    return mx4_linear_workspace(M, N, (int32_t)(K / split_k), split_k);
}

int lora_mx4_linear(const uint16_t* x, int64_t ld_x, const uint8_t* wq, int64_t ld_wq, const uint8_t* ws,
                    int64_t ld_ws, uint16_t* y, int64_t ld_y, int64_t M, int64_t K, int64_t N, int32_t split_k,
                    void* workspace, size_t workspace_bytes, void* stream)
{
    return linear(x, ld_x, nullptr, 0, wq, ld_wq, ws, ld_ws, y, ld_y, M, K, N, split_k, workspace,
                  workspace_bytes, stream, false);
}

int lora_mx4_linear_q(const uint8_t* xq, int64_t ld_xq, const uint8_t* xs, int64_t ld_xs, const uint8_t* wq,
                      int64_t ld_wq, const uint8_t* ws, int64_t ld_ws, uint16_t* y, int64_t ld_y, int64_t M,
                      int64_t K, int64_t N, int32_t split_k, void* workspace, size_t workspace_bytes, void* stream)
{
    return linear(xq, ld_xq, xs, ld_xs, wq, ld_wq, ws, ld_ws, y, ld_y, M, K, N, split_k, workspace,
                  workspace_bytes, stream, true);
}

int lora_block_norm(const uint16_t* y, int64_t ld_y, int32_t post, const uint16_t* post_w, const uint16_t* post_b,
                    const uint16_t* gate, int64_t ld_gate, int64_t gate_group, const uint16_t* r, int64_t ld_r,
                    float res_scale, uint16_t* r_out, int64_t ld_ro, int32_t pre, const uint16_t* pre_w,
                    const uint16_t* pre_b, uint16_t* x_out, int64_t ld_xo, int64_t M, int64_t C, float eps,
                    void* stream)
{
    if (M < 0 || M > kMaxDim || C < 0)
        return LORA_ERR_SHAPE;
    if (C < 8 || C > kNormMaxC || C % 8 || post < LORA_NORM_NONE || post > LORA_NORM_LAYER ||
        pre < LORA_NORM_NONE || pre > LORA_NORM_LAYER)
        return LORA_ERR_UNSUPPORTED;
    if (M == 0)
        return LORA_OK;
    if (!r || !r_out || (pre != LORA_NORM_NONE && !x_out) || (!y && post != LORA_NORM_NONE))
        return LORA_ERR_NULL;
    // a pointer without the step that uses it is a caller's mistake
    if ((pre == LORA_NORM_NONE && (x_out || pre_w || pre_b)) || (post == LORA_NORM_NONE && (post_w || post_b)) ||
        (!y && gate))
        return LORA_ERR_UNSUPPORTED;
    if (ld_r < C || ld_ro < C || (y && ld_y < C) || (x_out && ld_xo < C) || (gate && (gate_group < 1 || ld_gate < C)))
        return LORA_ERR_SHAPE;
    const void* ptrs[] = {y, post_w, post_b, gate, r, r_out, pre_w, pre_b, x_out};
    for (const void* q : ptrs)
        if (!aligned(q, 16))
            return LORA_ERR_ALIGN;
    if (ld_r % 8 || ld_ro % 8 || (y && ld_y % 8) || (x_out && ld_xo % 8) || (gate && ld_gate % 8))
        return LORA_ERR_ALIGN;
    NormParams p{};
    p.y = y;
    p.ld_y = ld_y;
    p.post_w = post_w;
    p.post_b = post_b;
    p.gate = gate;
    p.ld_gate = ld_gate;
    p.gate_group = gate ? gate_group : 1;
    p.r = r;
    p.ld_r = ld_r;
    p.r_out = r_out;
    p.ld_ro = ld_ro;
    p.pre_w = pre_w;
    p.pre_b = pre_b;
    p.x_out = x_out;
    p.ld_xo = ld_xo;
    p.M = M;
    p.C = (int32_t)C;
    p.post = post;
    p.pre = pre;
    p.res_scale = res_scale;
    p.eps = eps;
    return launch_status(launch_block_norm(p, static_cast<hipStream_t>(stream)));
}

int lora_sample(const void* logits, int32_t logits_type, int64_t ld, int64_t B, int64_t V, const float* temperature,
                const int32_t* top_k, const float* top_p, const float* min_p, const float* u, int32_t* tokens,
                float* logprobs, void* stream)
{
    if (B < 0 || B > kMaxDraws || V < 1)
        return LORA_ERR_SHAPE;
    if (V > kMaxVocabulary || (logits_type != LORA_LOGITS_BF16 && logits_type != LORA_LOGITS_F32))
        return LORA_ERR_UNSUPPORTED;
    if (B == 0)
        return LORA_OK;
    if (!logits || !u || !tokens)
        return LORA_ERR_NULL;
    if (ld < V)
        return LORA_ERR_SHAPE;
    const bool bf16 = logits_type == LORA_LOGITS_BF16;
    const void* ptrs[] = {temperature, top_k, top_p, min_p, u, tokens, logprobs};
    for (const void* q : ptrs)
        if (!aligned(q, 4))
            return LORA_ERR_ALIGN;
    if (!aligned(logits, bf16 ? 2 : 4))
        return LORA_ERR_ALIGN;
    SampleParams p{};
    p.logits = logits;
    p.ld = ld;
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.u = u;
    p.tokens = tokens;
    p.logprobs = logprobs;
    p.V = (int32_t)V;
    p.B = B;
    return launch_status(launch_sample(p, bf16, static_cast<hipStream_t>(stream)));
}

#pragma GCC visibility pop
}  // extern "C"
