// Attention over the paged cache in 8 bits.
//
// One pass over the keys with the running maximum and sum of the softmax.  The queries
// of a sequence that share a key head form rows, r = token * G + member
// of the group; a wave has tiles of 16 rows as the columns of its matrix products:
//   S^T = K Q^T     a step's 64 keys x 16 rows, four products of 16 keys
//   O^T += V^T P^T  D x 16 rows, reduced over the step's 64 keys
// With e the exponent of a block's value scale, the weight of a key in the second is
//   P = 2^(S + e - m),  m = max(S + e)      (base 2)
// so V enters as its codes, exactly, in fp16, and P too: times 2^15, of 11 bits down to
// 2^-29 of the largest, with steps of 2^-39 of it below.  (P as bf16, with the scale in
// V, put the output 0.0019-0.0022 from the formula, where its own rounding alone is
// 0.0016-0.0017, as it is now; prompts took 3-4% less time, few rows the same.  P as two
// bf16 parts took 30% more for prompts and 2-7% for few rows.)  The sum of the softmax,
// l = sum 2^(S - m), is taken before that rounding and in fp32, as m and O are.
// Key rows are dealt to the products so that lane group g (16 lanes) gets the S
// of the step's block g, all 16 tokens: these are the P it then supplies, and the
// tokens of the 16 bytes of V that it loads.  No value changes lanes but for the
// row's maximum and sum.  Codes of K become bf16 (exactly) on the way from the load to
// the product, times their block's scale.
//
// Measured on MI355X, 8 key heads of 128 unless said otherwise.  Few rows, by the cache's
// bytes: 61 sequences of up to 16384, 64 heads, 280 us (4.6 TB/s; 250, 5.2 TB/s, in chunks
// of 2048); one of 131071 48 us (5.5 TB/s, of which the last-level cache has a part; 58 when
// it has none); one of 1025 9.5 (two launches); 32 x 5 drafts, heads of 64, 39.  Many rows,
// by the matrix cores and the vector unit together: prompts of 8191 and 5119 tokens 850-880
// us (870-900 TFLOP/s; a large library product of bf16 reaches 1450; 930-955 us in six
// passes on their own), 512 tokens against 32768 312-364 by card (750-870).
// Heads of 256, 4 key heads: a token against 1025 12 us, against 131071 50; 61 of up to
// 16384, 32 heads, 323 (263 in chunks of 2048); 32 x 5 drafts against up to 6000 121 (88; the
// codes alone would take 51); 512 tokens against 32768, 16 heads, 500, prompts of 8191 and
// 5119 tokens 1390 (550 TFLOP/s).
#include "kv_cache.h"

#include <math.h>
#include <type_traits>

namespace lora {

namespace {

constexpr int kStep = 64;                    // keys a wave takes at a time
constexpr int kWaves = 4;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

constexpr int kUp = 15;                      // P and O are held times 2^15
constexpr float kDown = 1.0f / (1 << kUp);

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));    // converted to nearest, ties to even

// Eight codes times a power of two.
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi, float scale)
{
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Eight codes, exactly.
__device__ __forceinline__ f16x8 widen_f16(uint32_t lo, uint32_t hi)
{
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A maximum large enough that no rounding of the exponents makes a P larger than 2^kUp.
__device__ __forceinline__ float above(float m)
{
    return fmaf(fabsf(m), 0x1p-22f, m);      // NaN of -inf, which the next maximum drops
}

// What takes a sum of P of a block with this scale byte to its part of l.
__device__ __forceinline__ float back_of(int byte)
{
    return __builtin_amdgcn_ldexpf(1.0f, 127 - kUp - byte);
}

// Of each byte that is a NaN code the top bit, of others 0.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t codes)
{
    return ((codes & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

__device__ __forceinline__ float group_max(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}

__device__ __forceinline__ float group_sum(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// A logit's place under a maximum that may be -inf (no key yet).
__device__ __forceinline__ float shift_of(float m)
{
    return m == -INFINITY ? 0.0f : m;
}

struct Work {
    int64_t b;                               // sequence
    int64_t row0;                            // first row of the tile
    int rows;                                // rows of the tile, 0: nothing to do
    KvSequence s;
};

// Rows of the sequences lie in tiles of R; tiles of a sequence begin at a slot that
// grows with it.
template <int R>
__device__ __forceinline__ Work find_work(const KvAttentionParams& p, int64_t slot, int64_t slots, int G)
{
    auto at = [&](int64_t j, int64_t cu) { return cu * G / R + j; };
    Work w{};
    const KvFound found = kv_find(p.cache, p.T, slot, slots, at);
    w.b = found.b;
    w.s = found.s;
    w.row0 = (slot - at(w.b, w.s.first)) * R;
    const int64_t left = w.s.n * G - w.row0;
    w.rows = w.row0 >= 0 && left > 0 ? (int)min(left, (int64_t)R) : 0;
    return w;
}

// The keys that a row sees: lo .. hi.
struct Seen {
    int32_t lo, hi;
};

__device__ __forceinline__ Seen seen_by(const KvAttentionParams& p, const KvSequence& s, int64_t token)
{
    const int64_t end = min(s.len, p.max_len);
    const int64_t pos = s.len - s.n + token;
    const int64_t hi = p.causal ? min(pos, end - 1) : end - 1;
    const int64_t lo = p.window ? max(pos - p.window + 1, (int64_t)0) : 0;
    return {(int32_t)lo, (int32_t)max(hi, (int64_t)-1)};
}

__host__ __device__ constexpr int64_t partial_floats(int D) { return D + 4; }

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// Four values of a finished row from column c on, and with the first its lse.
__device__ __forceinline__ void write_row(const KvAttentionParams& p, int64_t at, int h, int c, const f32x4& x, float top,
                                          float total, int D)
{
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    *reinterpret_cast<bf16x4*>(p.out + at * p.ld_out + (int64_t)h * D + c) =
        bf16x4{(__bf16)(x[0] * inv), (__bf16)(x[1] * inv), (__bf16)(x[2] * inv), (__bf16)(x[3] * inv)};
    if (p.lse && c == 0)
        p.lse[at * p.ld_lse + h] = total == 0.0f ? -INFINITY : (top + log2f(total)) * kLn2;
}

// Few rows (single tokens, drafts): bound by the cache's bytes.  The waves share the
// tile's rows and deal out the steps of the chunk.  K of a wave's next step is asked
// for as soon as this step's S are there, V as soon as it is multiplied, so one of
// them is always on its way without registers of its own.
// A sequence has `tiles` workgroups a head and chunk, enough for max_new tokens; where it has
// more they go round again.
// Two tiles of heads of 128 (386 registers) and one of heads of 256 (403) leave one wave a
// SIMD, half of what the others have; nothing is spilled.
template <int D, int NT>
__global__ void __launch_bounds__(kWaves * 64, D * NT <= 128 ? 2 : 1) k_attention(KvAttentionParams p, uint32_t tiles)
{
    constexpr int R = 16 * NT;
    constexpr int kLoads = D / 64;           // 16-byte loads of a key by its 4 lanes
    constexpr int kOut = D / 16;             // tiles of 16 d
    __shared__ float ml[kWaves][R][2];
    __shared__ __align__(16) float ow[kWaves][16][D + 4];
    const int H = p.cache.heads, G = p.q_heads / H;
    const int lane = threadIdx.x & 63, li = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = (int)(blockIdx.x % (uint32_t)H);
    const uint32_t slot = blockIdx.x / (uint32_t)H, of_chunk = tiles * (uint32_t)p.cache.n_seqs;
    const int64_t chunk = slot / of_chunk;
    Work w{};
    w.b = slot % of_chunk / tiles;
    w.s = kv_sequence(p.cache, w.b, p.T);
    const bool several = p.partial != nullptr;
    // rows of all sequences fit 31 bits
    const int all_rows = (int)w.s.n * G;
#pragma unroll 1
    for (int row0 = (int)(slot % tiles) * R; row0 < all_rows; row0 += (int)tiles * R) {
        w.row0 = row0;
        w.rows = min(all_rows - row0, R);
        const int first_token = row0 / G, last_token = (row0 + w.rows - 1) / G;
        const Seen first = seen_by(p, w.s, first_token), last = seen_by(p, w.s, last_token);
        const int64_t begin = max(chunk * p.chunk, (int64_t)first.lo / kStep * kStep);
        const int64_t end = min((chunk + 1) * p.chunk, (int64_t)last.hi + 1);
        if (several && begin >= end)
            continue;

        const int P = p.cache.page_size;
        // this lane's row of the S products is a key of block li / 4, its V is of block g
        int page_k = -1, page_v = -1;            // of the step that is loaded next
        u32x4 kc[4][kLoads], vc[kOut];
        float ks = 1.0f;
        int vs = 127;                            // the scale byte of V's block
        auto pages_of = [&](int step) {
            page_k = kv_page(p.cache, w.b, (int64_t)step * kStep + li / 4 * kKvBlock);
            page_v = kv_page(p.cache, w.b, (int64_t)step * kStep + g * kKvBlock);
        };
        auto load_k = [&](int step) {
            const int64_t i = max(page_k, 0);
            const int at = head * P + ((step * kStep + li / 4 * kKvBlock) & (P - 1));    // in tokens of all heads
            const uint8_t* src = p.cache.k + i * p.cache.ld_k + (int64_t)(at + li % 4) * D + 16 * g;
            ks = pow2_of_scale(p.cache.k_scales[i * p.cache.ld_ks + at / kKvBlock]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < kLoads; ++j)
                    kc[t][j] = *(const global_u32x4*)(src + 4 * t * D + 64 * j);
        };
        auto load_v = [&](int step) {
            const int64_t i = max(page_v, 0);
            const int at = head * P + ((step * kStep + g * kKvBlock) & (P - 1));
            const uint8_t* src = p.cache.v + i * p.cache.ld_v + (int64_t)at * D + 16 * li;
            vs = p.cache.v_scales[i * p.cache.ld_vs + at / kKvBlock];
#pragma unroll
            for (int d = 0; d < kOut; ++d)
                vc[d] = *(const global_u32x4*)(src + 16 * 16 * d);
        };
        // steps are dealt by their number, wherever the first one lies
        const int s1 = (int)((end + kStep - 1) / kStep);
        int step = (int)(begin / kStep);
        step += (wave - step % kWaves + kWaves) % kWaves;
        if (step < s1) {
            pages_of(step);
            load_k(step);
            load_v(step);
        }

        // the rows of this lane's columns
        Seen seen[NT];
        bf16x8 q[NT][2 * kLoads];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = n * 16 + li;
            const bool in = r < w.rows;
            const int row = (int)w.row0 + (in ? r : 0), token = row / G, q_head = head * G + row - token * G;
            seen[n] = seen_by(p, w.s, token);
            if (!in)
                seen[n].hi = -1;
            const uint16_t* src = p.q + (w.s.first + token) * p.ld_q + (int64_t)q_head * D + 16 * g;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                q[n][2 * j] = load_bf16x8(src + 64 * j);
                q[n][2 * j + 1] = load_bf16x8(src + 64 * j + 8);
            }
        }

        f32x4 o[NT][kOut];
        float m[NT], l[NT];                      // l: of this lane's keys
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n] = -INFINITY;
            l[n] = 0.0f;
#pragma unroll
            for (int d = 0; d < kOut; ++d)
                o[n][d] = f32x4{0, 0, 0, 0};
        }
        const float sl = p.scale * kLog2e;

#pragma unroll 1
        for (; step < s1; step += kWaves) {
            const int p0 = step * kStep, pv = p0 + g * kKvBlock;
            const bool missing = page_v < 0, more = step + kWaves < s1;
            if (more)
                pages_of(step + kWaves);
            f32x4 s[NT][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    s[n][t] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < kLoads; ++j) {
                    const bf16x8 k0 = widen(kc[t][j][0], kc[t][j][1], ks), k1 = widen(kc[t][j][2], kc[t][j][3], ks);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        s[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, q[n][2 * j], s[n][t], 0, 0, 0);
                        s[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, q[n][2 * j + 1], s[n][t], 0, 0, 0);
                    }
                }
            }
            if (more)
                load_k(step + kWaves);

            // every row of the tile sees every key of most steps
            const bool edge = p0 < last.lo || p0 + kStep - 1 > first.hi || __any(missing);
            uint32_t bad = 0;
            if (edge) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = pv + 4 * t + i;
                            const bool in = !missing && key >= seen[n].lo && key <= seen[n].hi;
                            s[n][t][i] = in ? s[n][t][i] : -INFINITY;
                        }
                // a block that no row sees may hold anything
                const bool unseen = missing || pv > last.hi || pv + kKvBlock <= first.lo;
#pragma unroll
                for (int d = 0; d < kOut; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        vc[d][i] = unseen ? 0u : vc[d][i];
                        bad |= nan_bytes(vc[d][i]);
                    }
            }
            const float e = (float)(vs - 127), back = back_of(vs);
            f16x8 prob[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float top = -INFINITY;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        top = fmaxf(top, s[n][t][i]);
                const float mn = fmaxf(m[n], above(group_max(fmaf(top, sl, e))));
                const float shift = shift_of(mn), up = e + (float)kUp - shift, f = __builtin_amdgcn_exp2f(m[n] - shift);
                m[n] = mn;
                float sum = 0.0f;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = __builtin_amdgcn_exp2f(fmaf(s[n][t][i], sl, up));
                        sum += x;
                        prob[n][t / 2][4 * (t % 2) + i] = (_Float16)x;
                    }
                l[n] = fmaf(sum, back, l[n] * f);
#pragma unroll
                for (int d = 0; d < kOut; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[n][d][i] *= f;
            }
            if (edge && __any(bad != 0)) {
                // a value that is NaN reaches the rows that see its key, and no others
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    bf16x8 sees[2];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = pv + 4 * t + i;
                            const bool in = !missing && key >= seen[n].lo && key <= seen[n].hi;
                            sees[t / 2][4 * (t % 2) + i] = in ? (__bf16)1.0f : (__bf16)0.0f;
                        }
#pragma unroll
                    for (int d = 0; d < kOut; ++d) {
                        f32x4 hit = {0, 0, 0, 0};
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            // a code of 2^-3 where there is a NaN
                            const bf16x8 one =
                                widen(nan_bytes(vc[d][2 * u]) >> 2, nan_bytes(vc[d][2 * u + 1]) >> 2, 1.0f);
                            hit = __builtin_amdgcn_mfma_f32_16x16x32_bf16(one, sees[u], hit, 0, 0, 0);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[n][d][i] = hit[i] > 0.0f ? __builtin_nanf("") : o[n][d][i];
                    }
                }
#pragma unroll
                for (int d = 0; d < kOut; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        vc[d][i] &= ~((nan_bytes(vc[d][i]) >> 7) * 0xFFu);
            }
#pragma unroll
            for (int d = 0; d < kOut; ++d) {
                const f16x8 v0 = widen_f16(vc[d][0], vc[d][1]), v1 = widen_f16(vc[d][2], vc[d][3]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    o[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, prob[n][0], o[n][d], 0, 0, 0);
                    o[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, prob[n][1], o[n][d], 0, 0, 0);
                }
            }
            if (more)
                load_v(step + kWaves);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
            l[n] = group_sum(l[n]);

        // the waves' shares are joined in ascending order
#pragma unroll
        for (int n = 0; n < NT; ++n)
            if (g == 0) {
                ml[wave][n * 16 + li][0] = m[n];
                ml[wave][n * 16 + li][1] = l[n];
            }
        // unrolled, so that o stays in registers
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            __syncthreads();
#pragma unroll
            for (int d = 0; d < kOut; ++d)
                *reinterpret_cast<f32x4*>(&ow[wave][li][16 * d + 4 * g]) = o[n][d];
            __syncthreads();
            // 16 threads a row, each D / 16 values next to one another by fours
            const int r = threadIdx.x >> 4, c0 = (threadIdx.x & 15) * 4, row = n * 16 + r;
            if (row < w.rows) {
                float top = -INFINITY;
#pragma unroll
                for (int v = 0; v < kWaves; ++v)
                    top = fmaxf(top, ml[v][row][0]);
                const float shift = shift_of(top);
                float total = 0.0f, f[kWaves];
#pragma unroll
                for (int v = 0; v < kWaves; ++v) {
                    f[v] = exp2f(ml[v][row][0] - shift);
                    total += ml[v][row][1] * f[v];
                }
                const int rr = (int)w.row0 + row, token = rr / G, h = head * G + rr - token * G;
                const int64_t at = w.s.first + token;
#pragma unroll
                for (int c = 0; c < D; c += 64) {
                    f32x4 x = {0, 0, 0, 0};
#pragma unroll
                    for (int v = 0; v < kWaves; ++v) {
                        const f32x4 y = *reinterpret_cast<const f32x4*>(&ow[v][r][c + c0]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[i] += y[i] * (f[v] * kDown);
                    }
                    if (several) {
                        float* dst = p.partial + ((chunk * p.T + at) * p.q_heads + h) * partial_floats(D);
                        *reinterpret_cast<f32x4*>(dst + 4 + c + c0) = x;
                        if (c + c0 == 0) {
                            dst[0] = top;
                            dst[1] = total;
                        }
                    } else {
                        write_row(p, at, h, c + c0, x, top, total, D);
                    }
                }
            }
        }
        __syncthreads();                         // before the next tile's shares
    }
}

// ---------------------------------------------------------------------------
// Many rows (prompts): bound by the matrix cores.  A workgroup has 128 rows, a wave
// 32 of them; K and V of a step are widened to 16 bits on their way to LDS, once for
// all waves, and lie there in the order of the operands:
//   S^T = K Q^T       32x32x16 products, 32 keys x 32 rows
//   O^T += V^T P^T    32x32x16 products, 32 d x 32 rows
// A lane half gets the S of keys 4h .. 4h+3 and 8 + 4h .. 8 + 4h+3 of each block of 16,
// and V's tokens lie in that order, so P goes from one product to the other as it is.
// While a wave takes the softmax of a step it multiplies the next one (S), which does
// not depend on it; two workgroups a CU fill each other's gaps.  By counters the matrix
// cores are busy 41% of the time, the vector unit 52%, LDS 33% (no conflicts); a wave waits
// for data 27% and for an instruction slot 27% of its time.  Heads of 128 fill the 256
// registers of two waves a SIMD (6 are spilled before the loop and read behind it); heads
// of 256 fill 512 at one (13 spilled, of which a turn of the loop reads six), with 135 KB
// of LDS and so one workgroup a CU: that is why they reach 550 TFLOP/s, not 890.
// ---------------------------------------------------------------------------
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTileRows = kWaves * 32;

template <int D>
struct TileLds {
    u32x4 k[2][D / 16][2][kStep];            // bf16: 8 d of a key, for each lane half
    u32x4 v[2][kStep / kKvBlock][2][D];      // fp16: 8 keys of a d, for each lane half
    float v_exponent[2][kStep / kKvBlock];   // of the blocks' scales, written with K
    float v_back[2][kStep / kKvBlock];       // back_of them
    uint32_t nan_step[2];                    // the last step with a value that is NaN
    uint16_t nan[2][kStep / kKvBlock][D];    // then: which keys' value of a d is
};

__device__ __forceinline__ float half_max(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v),
                                                    false, false);
    const uint32_t a = r[0], b = r[1];       // a bit cast takes a vector's first element
    return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}

__device__ __forceinline__ float half_sum(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v),
                                                    false, false);
    const uint32_t a = r[0], b = r[1];
    return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
}

template <int D>
__global__ void __launch_bounds__(kWaves * 64, D == 256 ? 1 : 2) k_attention_tile(KvAttentionParams p, uint32_t slots)
{
    constexpr int kKeys = kStep;
    constexpr int kTiles = kKeys / 32;       // tiles of 32 keys
    constexpr int kBlocks = kKeys / kKvBlock;
    constexpr int kDeep = D / 16;            // products of 16 d
    constexpr int kOut = D / 32;             // tiles of 32 d
    constexpr int kPieces = D / 64;          // 16-byte pieces of K, and of V, a thread brings to LDS
    __shared__ __align__(16) TileLds<D> lds;
    const int H = p.cache.heads, G = p.q_heads / H;
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = (int)(blockIdx.x % (uint32_t)H);
    const uint32_t tile = blockIdx.x / (uint32_t)H;
    // a prompt's last rows see the most keys: they begin first
    const int64_t slot = slots - 1 - tile % slots, chunk = tile / slots;

    const Work w = find_work<kTileRows>(p, slot, slots, G);
    if (w.rows == 0)
        return;
    const int first_token = (int)w.row0 / G, last_token = ((int)w.row0 + w.rows - 1) / G;
    const Seen first = seen_by(p, w.s, first_token), last = seen_by(p, w.s, last_token);
    const int64_t begin = max(chunk * p.chunk, (int64_t)first.lo / kKeys * kKeys);
    const int64_t end = min((chunk + 1) * p.chunk, (int64_t)last.hi + 1);
    const bool several = p.partial != nullptr;
    if (several && begin >= end)
        return;

    const int row = wave * 32 + r;
    const bool in = row < w.rows;
    const int at = (int)w.row0 + (in ? row : 0), token = at / G, q_head = head * G + at - token * G;
    Seen seen = seen_by(p, w.s, token);
    if (!in)
        seen.hi = -1;
    bf16x8 q[kDeep];
    {
        const uint16_t* src = p.q + (w.s.first + token) * p.ld_q + (int64_t)q_head * D + 8 * h;
#pragma unroll
        for (int j = 0; j < kDeep; ++j)
            q[j] = load_bf16x8(src + 16 * j);
    }

    f32x16 o[kOut];
#pragma unroll
    for (int d = 0; d < kOut; ++d)
        o[d] = f32x16{};
    float m = -INFINITY, l = 0.0f;           // l: of this lane's keys
    const float sl = p.scale * kLog2e;
    const int P = p.cache.page_size;

    // A wave brings its block of a step to LDS: a thread 16 d of a key, and the keys of a d.
    static_assert(kBlocks == kWaves, "");
    const int k_key = lane % kKvBlock, k_piece = lane / kKvBlock;
    // the sequence's row of the table, read by scalar loads
    typedef __attribute__((address_space(4))) const int32_t constant_i32;
    constant_i32* pages = (constant_i32*)(p.cache.page_table + __builtin_amdgcn_readfirstlane((int)w.b) * p.cache.ld_table);
    const int shift = p.cache.page_shift, n_pages = p.cache.n_pages;
    const int max_page = (int)min(p.cache.max_pages, (int64_t)1 << 30);
    auto page_of = [&](int key) {
        const int i = key >> shift, page = pages[min(i, max_page - 1)];
        return i < max_page && page >= 0 && page < n_pages ? page : -1;
    };
    // The page of this wave's block of a step; `gone`: the step's blocks without one, a bit each.
    auto page_at = [&](int step, uint32_t& gone) {
        const int page = page_of(step * kKeys + wave * kKvBlock);
        gone = page < 0 ? 15u : 0u;
        if (P < kKeys) {
            gone = 0;
#pragma unroll
            for (int u = 0; u < kBlocks; ++u)
                gone |= (page_of(step * kKeys + u * kKvBlock) < 0 ? 1u : 0u) << u;
        }
        return page;
    };
    // every row of the tile sees every key of most steps
    auto whole = [&](int step) { return step * kKeys >= last.lo && step * kKeys + kKeys - 1 <= first.hi; };

    u32x4 kr[kPieces], vr[kPieces];
    uint32_t kscale, vscale;
    auto load_k = [&](int step, int page) __attribute__((always_inline)) {
        const int64_t g = max(page, 0);
        const int at = head * P + ((step * kKeys + wave * kKvBlock) & (P - 1));    // in tokens of all heads
        const uint8_t* src = p.cache.k + (g * p.cache.ld_k + (int64_t)at * D);
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
            kr[j] = *(const global_u32x4*)(src + (k_key * D + 16 * k_piece + 64 * j));
        kscale = p.cache.k_scales[g * p.cache.ld_ks + at / kKvBlock];
        vscale = p.cache.v_scales[g * p.cache.ld_vs + at / kKvBlock];
    };
    auto load_v = [&](int step, int page) __attribute__((always_inline)) {
        const int64_t g = max(page, 0);
        const int at = head * P + ((step * kKeys + wave * kKvBlock) & (P - 1));
        const uint8_t* src = p.cache.v + (g * p.cache.ld_v + (int64_t)at * D);
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
            vr[j] = *(const global_u32x4*)(src + (lane * 16 + 1024 * j));
    };
    auto store_k = [&](int buf) __attribute__((always_inline)) {
        const float s = pow2_of_scale(kscale);
        lds.v_exponent[buf][wave] = (float)((int)vscale - 127);
        lds.v_back[buf][wave] = back_of((int)vscale);
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            auto& to = lds.k[buf][k_piece + 4 * j];
            to[0][wave * kKvBlock + k_key] = __builtin_bit_cast(u32x4, widen(kr[j][0], kr[j][1], s));
            to[1][wave * kKvBlock + k_key] = __builtin_bit_cast(u32x4, widen(kr[j][2], kr[j][3], s));
        }
    };
    // gaps: some rows do not see all keys of the step
    auto store_v = [&](bool gaps, int buf, int step, int page) __attribute__((always_inline)) {
        if (gaps) {
            // a block that no row sees may hold anything
            const int key = step * kKeys + wave * kKvBlock;
            const bool unseen = page < 0 || key > last.hi || key + kKvBlock <= first.lo;
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                uint32_t bad = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t c = unseen ? 0u : vr[j][i], b = nan_bytes(c) >> 7;
                    vr[j][i] = c & ~(b * 0xFFu);
                    bad |= ((b | b >> 7 | b >> 14 | b >> 21) & 15u) << (4 * i);
                }
                lds.nan[buf][wave][lane + 64 * j] = (uint16_t)bad;
                if (bad)
                    lds.nan_step[buf] = (uint32_t)step;
            }
        }
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            lds.v[buf][wave][0][lane + 64 * j] = __builtin_bit_cast(u32x4, widen_f16(vr[j][0], vr[j][2]));
            lds.v[buf][wave][1][lane + 64 * j] = __builtin_bit_cast(u32x4, widen_f16(vr[j][1], vr[j][3]));
        }
    };

    typedef f32x16 Logits[kTiles];
    typedef f16x8 Probs[kBlocks];
    auto product = [&](int buf, Logits& out) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            out[t] = f32x16{};
#pragma unroll
        for (int j = 0; j < kDeep; ++j)
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                const bf16x8 k = __builtin_bit_cast(bf16x8, lds.k[buf][j][h][32 * t + r]);
                out[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q[j], out[t], 0, 0, 0);
            }
    };
    auto output = [&](int buf, const Probs& prob) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < kBlocks; ++u)
#pragma unroll
            for (int d = 0; d < kOut; ++d) {
                const f16x8 v = __builtin_bit_cast(f16x8, lds.v[buf][u][h][32 * d + r]);
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, prob[u], o[d], 0, 0, 0);
            }
    };
    // a value that is NaN reaches the rows that see its key, and no others
    auto spread_nan = [&](int buf, int step) __attribute__((always_inline)) {
        const int from = min(max(seen.lo - step * kKeys, 0), kKeys), to = min(max(seen.hi + 1 - step * kKeys, 0), kKeys);
        const uint64_t sees =
            (to < 64 ? (uint64_t(1) << to) - 1 : ~uint64_t(0)) & (from < 64 ? ~uint64_t(0) << from : 0);
#pragma unroll
        for (int d = 0; d < kOut; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                uint64_t bad = 0;
#pragma unroll
                for (int u = 0; u < kBlocks; ++u)
                    bad |= (uint64_t)lds.nan[buf][u][32 * d + 8 * (i / 4) + 4 * h + i % 4] << (16 * u);
                o[d][i] = bad & sees ? __builtin_nanf("") : o[d][i];
            }
    };

    const int s0 = (int)(begin / kKeys), s1 = (int)((end + kKeys - 1) / kKeys);
    int page_v = -1, page_k = -1;            // of the next step, the one behind it
    uint32_t gone = 0, gone_next = 0, gone_far = 0;    // of this step, the next, the one behind it
    // of the step's V, the same in every lane: no registers of the vector unit
    float e[kBlocks], back[kBlocks];
    auto of_wave = [](float x) { return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x))); };
    auto exponents = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < kBlocks; ++u) {
            e[u] = of_wave(lds.v_exponent[buf][u]);
            back[u] = of_wave(lds.v_back[buf][u]);
        }
    };
    Logits s_even, s_odd;                    // of the even and odd steps from the first on
    if (threadIdx.x < 2)
        lds.nan_step[threadIdx.x] = 0xFFFFFFFFu;
    if (s0 < s1) {
        const int page = page_at(s0, gone);
        page_v = page_at(s0 + 1, gone_next);
        page_k = page_at(s0 + 2, gone_far);
        load_k(s0, page);
        load_v(s0, page);
        store_k(s0 & 1);
        load_k(s0 + 1, page_v);
        __syncthreads();
        store_v(!whole(s0) || gone, s0 & 1, s0, page);
        store_k((s0 + 1) & 1);
        load_v(s0 + 1, page_v);
        load_k(s0 + 2, page_k);
        __syncthreads();
        product(s0 & 1, s_even);
        exponents(s0 & 1);
        __syncthreads();                     // K of the first step is read: its place is free
    }
    // One step: its S are in s, those of the next go to s_next.  V of the next step and K of the
    // one behind it have been loaded during the step before.
    auto take = [&](int step, Logits& s, Logits& s_next) __attribute__((always_inline)) {
        const int buf = step & 1;
        const bool gaps = !whole(step) || gone;
        if (gaps) {
            const int key0 = step * kKeys + 4 * h;
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int key = key0 + 32 * t + 8 * (i / 4) + i % 4;
                    const bool sees = key >= seen.lo && key <= seen.hi && !(gone >> (2 * t + i / 8) & 1);
                    s[t][i] = sees ? s[t][i] : -INFINITY;
                }
        }
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < kBlocks; ++u) {
            float of_block = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                of_block = fmaxf(of_block, s[u / 2][u % 2 * 8 + i]);
            top = fmaxf(top, fmaf(of_block, sl, e[u]));
        }
        const float mn = fmaxf(m, above(half_max(top)));
        if (__any(mn > m)) {
            const float f = __builtin_amdgcn_exp2f(m - shift_of(mn));
            l *= f;
            m = mn;
#pragma unroll
            for (int d = 0; d < kOut; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[d][i] *= f;
        }
        const float shift = shift_of(m) - (float)kUp;
        // a wave with products to give comes before the others' vector work: 820 -> 805 us
        // for prompts of 8191 and 5119 tokens, 32 heads
        __builtin_amdgcn_s_setprio(1);
        product(buf ^ 1, s_next);
        Probs prob;
#pragma unroll
        for (int u = 0; u < kBlocks; ++u) {
            const float up = e[u] - shift;
            float sum = 0.0f;                // of the P before their rounding, which lse would show
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = __builtin_amdgcn_exp2f(fmaf(s[u / 2][u % 2 * 8 + i], sl, up));
                sum = i ? sum + x : x;
                prob[u][i] = (_Float16)x;
            }
            l = fmaf(sum, back[u], l);
        }
        store_k(buf);
        output(buf, prob);
        __builtin_amdgcn_s_setprio(0);
        if (gaps && lds.nan_step[buf] == (uint32_t)step)
            spread_nan(buf, step);
        store_v(!whole(step + 1) || gone_next, buf ^ 1, step + 1, page_v);
        page_v = page_k;
        load_v(step + 2, page_v);
        gone = gone_next;
        gone_next = gone_far;
        page_k = page_at(step + 3, gone_far);
        load_k(step + 3, page_k);
        exponents(buf ^ 1);                  // K of the next step is there, and they with it
        __syncthreads();
    };
    // two steps a turn, so that nothing moves from the registers of a step to those of another
#pragma unroll 1
    for (int step = s0; step < s1; step += 2) {
        take(step, s_even, s_odd);
        if (step + 1 < s1)
            take(step + 1, s_odd, s_even);
    }
    l = half_sum(l);
    if (!in)
        return;
    const int64_t out_row = w.s.first + token;
    float* dst = p.partial + ((chunk * p.T + out_row) * p.q_heads + q_head) * partial_floats(D);
    if (several && h == 0) {
        dst[0] = m;
        dst[1] = l;
    }
#pragma unroll
    for (int d = 0; d < kOut; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 x = {o[d][4 * i] * kDown, o[d][4 * i + 1] * kDown, o[d][4 * i + 2] * kDown, o[d][4 * i + 3] * kDown};
            const int c = 32 * d + 8 * i + 4 * h;
            if (several)
                *reinterpret_cast<f32x4*>(dst + 4 + c) = x;
            else
                write_row(p, out_row, q_head, c, x, m, l, D);
        }
}

// Joins the chunks of a row: kGroups groups of D / 4 threads take its chunks in turn, by
// their number, and are joined in ascending order, so that the chunks of a token far into
// a long cache are read together.  A block has heads of one token.
template <int D>
__global__ void __launch_bounds__(256) k_join(KvAttentionParams p)
{
    constexpr int kGroups = 4, kThreads = D / 4, kHeads = 256 / (kThreads * kGroups);
    __shared__ __align__(16) float part[kHeads][kGroups][D];
    __shared__ float ml[kHeads][kGroups][2];
    const uint32_t blocks = ((uint32_t)p.q_heads + kHeads - 1) / kHeads;
    const int64_t at = blockIdx.x / blocks;
    const int group = threadIdx.x / kThreads % kGroups, c = threadIdx.x % kThreads * 4;
    const int my = threadIdx.x / (kThreads * kGroups), h = (int)(blockIdx.x % blocks) * kHeads + my;
    const KvSequence s = kv_find(p.cache, p.T, at, p.T, [](int64_t, int64_t cu) { return cu; }).s;
    if (s.n == 0 || at < s.first)
        return;
    const Seen seen = seen_by(p, s, at - s.first);
    const int c0 = (int)(seen.lo / p.chunk), c1 = seen.hi < seen.lo ? c0 : (int)(seen.hi / p.chunk) + 1;
    const int64_t pitch = p.T * p.q_heads * partial_floats(D);
    const float* src = p.partial + (at * p.q_heads + h) * partial_floats(D);
    float top = -INFINITY, total = 0.0f;
    f32x4 x = {0, 0, 0, 0};
    const int last = h < p.q_heads ? c1 : 0;
#pragma unroll 4
    for (int i = c0 + (group - c0 % kGroups + kGroups) % kGroups; i < last; i += kGroups) {
        const float mi = src[i * pitch], li = src[i * pitch + 1];
        const f32x4 y = *reinterpret_cast<const f32x4*>(src + i * pitch + 4 + c);
        const float now = fmaxf(top, mi), shift = shift_of(now);
        const float f = __builtin_amdgcn_exp2f(top - shift), fi = __builtin_amdgcn_exp2f(mi - shift);
        top = now;
        total = total * f + li * fi;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[e] = x[e] * f + y[e] * fi;
    }
    *reinterpret_cast<f32x4*>(&part[my][group][c]) = x;
    if (c == 0) {
        ml[my][group][0] = top;
        ml[my][group][1] = total;
    }
    __syncthreads();
    if (group > 0 || h >= p.q_heads)
        return;
    for (int i = 0; i < kGroups; ++i)
        top = fmaxf(top, ml[my][i][0]);
    const float shift = shift_of(top);
    total = 0.0f;
    x = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const float f = __builtin_amdgcn_exp2f(ml[my][i][0] - shift);
        const f32x4 y = *reinterpret_cast<const f32x4*>(&part[my][i][c]);
        total += ml[my][i][1] * f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[e] += y[e] * f;
    }
    write_row(p, at, h, c, x, top, total, D);
}

// Rows of a tile that these sizes get; up to 64 rows a sequence the waves split the keys.
// (Two tiles of 16 rows of 256 would not fit the registers.)
int tile_rows(int64_t max_new, int G, int D)
{
    const int64_t rows = max_new * G;
    return rows <= 16 || (rows <= 64 && D == 256) ? 16 : rows <= 64 ? 32 : kTileRows;
}

bool few_rows(int R) { return R <= 32; }

// Workgroups of a head and chunk: few rows have so many for each sequence, tiles of many
// rows lie behind one another over all of them.
int64_t tile_slots(int64_t T, int64_t n_seqs, int64_t max_new, int R, int G)
{
    return few_rows(R) ? n_seqs * ((max_new * G + R - 1) / R) : T * G / R + n_seqs;
}

template <int D>
hipError_t launch(const KvAttentionParams& p, hipStream_t st)
{
    const int G = p.q_heads / p.cache.heads, R = tile_rows(p.max_new, G, D);
    const int64_t slots = tile_slots(p.T, p.cache.n_seqs, p.max_new, R, G);
    const uint32_t tiles = (uint32_t)((p.max_new * G + R - 1) / R);
    const int64_t chunks = (p.max_len + p.chunk - 1) / p.chunk;
    const dim3 grid((unsigned)(slots * p.cache.heads * chunks)), threads(kWaves * 64);
    if (R == 16)
        hipLaunchKernelGGL((k_attention<D, 1>), grid, threads, 0, st, p, tiles);
    else if (R == 32)
        hipLaunchKernelGGL((k_attention<D == 256 ? 64 : D, 2>), grid, threads, 0, st, p, tiles);
    else
        hipLaunchKernelGGL(k_attention_tile<D>, grid, threads, 0, st, p, (uint32_t)slots);
    if (p.partial)
        hipLaunchKernelGGL(k_join<D>, dim3((unsigned)(p.T * ((p.q_heads * D + 255) / 256))), dim3(256), 0, st, p);
    return hipGetLastError();
}

}  // namespace

// About one workgroup a CU for one sequence.  Shorter chunks cost a batch more than they
// give a sequence alone: 512 keys instead of 256 take one of 1025 from 9.5 to 10.8 us
// (so up to 2048 it keeps 256; one of 2049 to 8192 would gain 0.9 to 1.8 us by it too, from
// 11.2-11.6), but 61 of up to 16384 from 333 to 280 (2048: 250), 32 drafts of 5 tokens
// from 49 to 39 (2048: 33); from 12000 on 512 is the faster for one as well (12.0 against
// 13.8); one of 131071 takes 56 with 512, 48 with 2048 or 4096, 74 with 8192.
int64_t kv_attention_chunk(int64_t max_new, int32_t q_heads, int32_t kv_heads, int32_t D, int64_t max_len)
{
    const int G = q_heads / kv_heads, R = tile_rows(max_new, G, D);
    const int64_t tiles = (max_new * G + R - 1) / R * kv_heads;
    // tiles of many rows run two to a CU
    const int64_t wanted = few_rows(R) ? 256 : 512, splits = tiles < wanted ? wanted / tiles : 1;
    const int64_t chunk = (max_len + splits - 1) / splits, least = max_len > 2048 ? 2 * kKvChunkUnit : kKvChunkUnit;
    return ((chunk > least ? chunk : least) + kKvChunkUnit - 1) / kKvChunkUnit * kKvChunkUnit;
}

int64_t kv_attention_workspace(int64_t T, int32_t q_heads, int32_t D, int64_t max_len, int64_t chunk)
{
    const int64_t chunks = (max_len + chunk - 1) / chunk;
    return chunks > 1 ? chunks * T * q_heads * partial_floats(D) * 4 : 0;
}

int64_t kv_attention_blocks(int64_t T, int64_t n_seqs, int64_t max_new, int32_t q_heads, int32_t kv_heads, int32_t D,
                            int64_t max_len, int64_t chunk)
{
    const int G = q_heads / kv_heads;
    return tile_slots(T, n_seqs, max_new, tile_rows(max_new, G, D), G) * kv_heads * ((max_len + chunk - 1) / chunk);
}

hipError_t launch_kv_attention(const KvAttentionParams& p, hipStream_t st)
{
    return p.D == 64 ? launch<64>(p, st) : p.D == 128 ? launch<128>(p, st) : launch<256>(p, st);
}

}  // namespace lora
