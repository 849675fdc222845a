// C entry points of the paged cache (declared in include/lora_det.h): appending to
// it and attention over it.  As in abi.hip, every scalar and pointer is checked on
// the host before any HIP call, and nothing here allocates, frees or synchronises.
#include "../../include/lora_det.h"
#include "step_kernels.h"

#include <math.h>

using namespace lora;

namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxThreads = (int64_t{1} << 32) - 1;    // of a launch
constexpr int64_t kMaxLen = int64_t{1} << 30;
constexpr int64_t kMaxHeads = 65536;
constexpr int64_t kMaxSeqs = 65536;
constexpr int32_t kMaxPageSize = 32768;
constexpr int kWaveGroup = 256;                            // threads of an attention block

bool aligned(const void* p, unsigned n)
{
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

bool head_dim_ok(int32_t D)
{
    return D == 64 || D == 128 || D == 256;
}

int launch_status(hipError_t e)
{
    return e == hipSuccess ? LORA_OK : LORA_ERR_LAUNCH;
}

// Everything of the cache that needs no step; no sequences are valid too.
int check_cache(const lora_kv_cache* c)
{
    if (!c)
        return LORA_ERR_NULL;
    if (c->n_seqs < 0 || c->n_seqs > kMaxSeqs || c->heads < 1 || c->heads > kMaxHeads || c->n_pages < 1 ||
        c->n_pages > kMaxDim || c->max_pages < 1 || c->max_pages > kMaxDim)
        return LORA_ERR_SHAPE;
    if (!head_dim_ok(c->head_dim) || c->page_size < kKvBlock || c->page_size > kMaxPageSize ||
        (c->page_size & (c->page_size - 1)))
        return LORA_ERR_UNSUPPORTED;
    return LORA_OK;
}

int check_cache_arrays(const lora_kv_cache* c)
{
    if (!c->k || !c->v || !c->k_scales || !c->v_scales || !c->page_table || !c->seq_lens || !c->cu_tokens)
        return LORA_ERR_NULL;
    const int64_t blocks = (int64_t)c->heads * (c->page_size / kKvBlock), codes = blocks * kKvBlock * c->head_dim;
    if (c->ld_k < codes || c->ld_v < codes || c->ld_ks < blocks || c->ld_vs < blocks || c->ld_table < c->max_pages)
        return LORA_ERR_SHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->ld_k % 16 || c->ld_v % 16 || !aligned(c->page_table, 4) ||
        !aligned(c->seq_lens, 4) || !aligned(c->cu_tokens, 4))
        return LORA_ERR_ALIGN;
    return LORA_OK;
}

KvCacheView view(const lora_kv_cache* c)
{
    KvCacheView v{};
    v.k = c->k;
    v.v = c->v;
    v.k_scales = c->k_scales;
    v.v_scales = c->v_scales;
    v.ld_k = c->ld_k;
    v.ld_v = c->ld_v;
    v.ld_ks = c->ld_ks;
    v.ld_vs = c->ld_vs;
    v.page_table = c->page_table;
    v.ld_table = c->ld_table;
    v.max_pages = c->max_pages;
    v.seq_lens = c->seq_lens;
    v.cu_tokens = c->cu_tokens;
    v.n_seqs = c->n_seqs;
    v.n_pages = (int32_t)c->n_pages;
    v.page_size = c->page_size;
    v.page_shift = __builtin_ctz((unsigned)c->page_size);
    v.heads = c->heads;
    return v;
}

// Sizes of an attention step that say how much workspace it takes.
int check_attention_sizes(int64_t T, int32_t q_heads, int32_t heads, int32_t D, int64_t max_new, int64_t max_len,
                          int64_t chunk)
{
    if (T < 0 || T > kMaxDim || heads < 1 || heads > kMaxHeads || q_heads < heads || q_heads > kMaxHeads ||
        T * q_heads > kMaxDim || max_new < 1 || max_new > kMaxDim / q_heads || max_len < 1 || chunk < 0)
        return LORA_ERR_SHAPE;
    if (q_heads % heads || !head_dim_ok(D) || chunk % kKvChunkUnit || max_len > kMaxLen)
        return LORA_ERR_UNSUPPORTED;
    return LORA_OK;
}

// The chunk of a step whose sizes are sound: the default for 0, and no longer than the
// caller's max_len needs, so that sums of both stay small.
int64_t chunk_of(int64_t chunk, int64_t max_new, int32_t q_heads, int32_t heads, int32_t D, int64_t max_len)
{
    if (chunk == 0)
        return kv_attention_chunk(max_new, q_heads, heads, D, max_len);
    const int64_t whole = (max_len + kKvChunkUnit - 1) / kKvChunkUnit * kKvChunkUnit;
    return chunk < whole ? chunk : whole;
}

}  // namespace

extern "C" {
#pragma GCC visibility push(default)

int lora_kv_append(const lora_kv_cache* cache, const uint16_t* q, int64_t ld_q, uint16_t* q_out, int64_t ld_qo,
                   int32_t q_heads, const uint16_t* k, int64_t ld_k, const uint16_t* v, int64_t ld_v, int64_t T,
                   const uint16_t* q_norm, const uint16_t* k_norm, float eps, const float* rope, int64_t ld_rope,
                   int64_t rope_rows, int32_t rope_dim, int32_t pairs, void* stream)
{
    int st = check_cache(cache);
    if (st != LORA_OK)
        return st;
    const int64_t D = cache->head_dim;
    if (T < 0 || T > kMaxDim || (q && (q_heads < 1 || q_heads > kMaxHeads)))
        return LORA_ERR_SHAPE;
    if ((pairs != 0 && pairs != 1) || (rope && (rope_dim < 16 || rope_dim > D || rope_dim % 16)) ||
        (T > 0 && !q && q_norm) || (!q != !q_out))
        return LORA_ERR_UNSUPPORTED;
    const int64_t blocks = (T / kKvBlock + 2 * cache->n_seqs) * cache->heads + (q ? T : 0);
    if (blocks * 2 * D > kMaxThreads)
        return LORA_ERR_SHAPE;
    if (T == 0 || cache->n_seqs == 0)
        return LORA_OK;
    if (!k || !v)
        return LORA_ERR_NULL;
    if ((st = check_cache_arrays(cache)) != LORA_OK)
        return st;
    if (ld_k < cache->heads * D || ld_v < cache->heads * D || (q && (ld_q < q_heads * D || ld_qo < q_heads * D)) ||
        (rope && (ld_rope < rope_dim || rope_rows < 0)))
        return LORA_ERR_SHAPE;
    const void* ptrs[] = {q, q_out, k, v, q_norm, k_norm, rope};
    for (const void* x : ptrs)
        if (!aligned(x, 16))
            return LORA_ERR_ALIGN;
    if (ld_k % 8 || ld_v % 8 || (q && (ld_q % 8 || ld_qo % 8)) || (rope && ld_rope % 4))
        return LORA_ERR_ALIGN;
    KvAppendParams p{};
    p.cache = view(cache);
    p.q = q;
    p.ld_q = ld_q;
    p.q_out = q_out;
    p.ld_qo = ld_qo;
    p.k = k;
    p.ld_k = ld_k;
    p.v = v;
    p.ld_v = ld_v;
    p.q_norm = q_norm;
    p.k_norm = k_norm;
    p.rope = rope;
    p.ld_rope = ld_rope;
    p.rope_rows = rope_rows;
    p.T = T;
    p.rope_dim = rope ? rope_dim : 0;
    p.pairs = pairs;
    p.q_heads = q ? q_heads : 0;
    p.D = (int32_t)D;
    p.eps = eps;
    return launch_status(launch_kv_append(p, static_cast<hipStream_t>(stream)));
}

int64_t lora_kv_attention_chunk(int64_t max_new, int32_t q_heads, int32_t heads, int32_t head_dim, int64_t max_len)
{
    if (check_attention_sizes(0, q_heads, heads, head_dim, max_new, max_len, 0) != LORA_OK)
        return 0;
    return kv_attention_chunk(max_new, q_heads, heads, head_dim, max_len);
}

size_t lora_kv_attention_workspace_bytes(int64_t T, int32_t q_heads, int32_t heads, int32_t head_dim, int64_t max_new,
                                         int64_t max_len, int64_t chunk)
{
    if (check_attention_sizes(T, q_heads, heads, head_dim, max_new, max_len, chunk) != LORA_OK || T == 0)
        return 0;
    chunk = chunk_of(chunk, max_new, q_heads, heads, head_dim, max_len);
    if (max_len <= chunk)
        return 0;
    if (T * q_heads > kMaxThreads / kWaveGroup || T * q_heads * ((max_len + chunk - 1) / chunk) > kMaxThreads)
        return 0;                            // more than a launch takes
    return (size_t)kv_attention_workspace(T, q_heads, head_dim, max_len, chunk);
}

int lora_kv_attention(const lora_kv_cache* cache, const uint16_t* q, int64_t ld_q, uint16_t* out, int64_t ld_out,
                      float* lse, int64_t ld_lse, int64_t T, int32_t q_heads, int64_t max_new, int64_t max_len,
                      float scale, int32_t causal, int64_t window, int64_t chunk, void* workspace,
                      size_t workspace_bytes, void* stream)
{
    int st = check_cache(cache);
    if (st != LORA_OK)
        return st;
    const int32_t D = cache->head_dim, H = cache->heads;
    if ((st = check_attention_sizes(T, q_heads, H, D, max_new, max_len, chunk)) != LORA_OK)
        return st;
    if (window < 0 || window > kMaxDim)
        return LORA_ERR_SHAPE;
    if ((causal != 0 && causal != 1) || (window && !causal) || !(scale > 0.0f) || !(scale < INFINITY))
        return LORA_ERR_UNSUPPORTED;
    if (T == 0 || cache->n_seqs == 0)
        return LORA_OK;
    if (!q || !out)
        return LORA_ERR_NULL;
    if ((st = check_cache_arrays(cache)) != LORA_OK)
        return st;
    const int64_t columns = (int64_t)q_heads * D;
    if (ld_q < columns || ld_out < columns || (lse && ld_lse < q_heads))
        return LORA_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16) || ld_q % 8 || ld_out % 8)
        return LORA_ERR_ALIGN;
    chunk = chunk_of(chunk, max_new, q_heads, H, D, max_len);    // by the caller's max_len, as the workspace's size
    const int64_t capacity = cache->max_pages * cache->page_size;
    max_len = max_len < capacity ? max_len : capacity;
    if (kv_attention_blocks(T, cache->n_seqs, max_new, q_heads, H, D, max_len, chunk) > kMaxThreads / kWaveGroup ||
        (max_len > chunk && T * q_heads > kMaxThreads / kWaveGroup))
        return LORA_ERR_SHAPE;
    const int64_t need = kv_attention_workspace(T, q_heads, D, max_len, chunk);
    if (need && !workspace)
        return LORA_ERR_NULL;
    if ((size_t)need > workspace_bytes)
        return LORA_ERR_WORKSPACE;
    KvAttentionParams p{};
    p.cache = view(cache);
    p.q = q;
    p.ld_q = ld_q;
    p.out = out;
    p.ld_out = ld_out;
    p.lse = lse;
    p.ld_lse = ld_lse;
    p.partial = need ? static_cast<float*>(workspace) : nullptr;
    p.T = T;
    p.max_len = max_len;
    p.chunk = chunk;
    p.max_new = max_new;
    p.q_heads = q_heads;
    p.D = D;
    p.causal = causal;
    p.window = (int32_t)window;
    p.scale = scale;
    return launch_status(launch_kv_attention(p, static_cast<hipStream_t>(stream)));
}

#pragma GCC visibility pop
}  // extern "C"
