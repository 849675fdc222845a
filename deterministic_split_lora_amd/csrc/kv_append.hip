// Appends a step's keys and values to the paged cache: the norms of queries and
// keys per head, the rotation by their position, the rounding to 8 bits.
//
//   n = t / sqrt(mean(t^2) + eps) * w              (queries, keys; mean per head)
//   (a, b) -> (a cos - b sin, b cos + a sin)       for the pairs of the rotated part
//   q_out = bf16(n rotated),  k = e4m3(n rotated 2^-e),  v = e4m3(v 2^-e)
// e is the block's exponent: the least, within limits, at which the
// largest value of the block's tokens is no more than 448.  A block that goes on
// keeps its exponent unless the new tokens need a larger one; then its earlier
// codes are rounded again, in place.  (A power of two: their exponent moves, and
// only codes that become subnormal lose anything.)  It does not fall again when the
// tokens that raised it are taken back: what their codes were is not kept.
//
// Every fp32 operation rounds on its own and the sum of squares is taken in fp64,
// where its order leaves no trace: which code a value gets does not depend on how
// the work is laid out.
//
// One launch: a workgroup takes a block of a head with all of its new tokens, keys
// in one half and values in the other, so nobody else writes there and no atomics
// are needed; further workgroups take a token's queries.  A thread holds 16 values
// that rotate among themselves.
//
// Measured on MI355X, with the queries: 8190 tokens of 64 + 2 x 8 heads of 128, normed,
// 78-84 us (364 MB, 4.3-4.6 TB/s: the rate of a large copy); 251 single tokens of 32 + 2 x 8
// heads 12 (105 registers: about 1024 of the 2259 workgroups run at a time, so this is three
// rounds of what one token takes, most of whose lanes have only V's old codes to move); one
// token 5.2 (three rounds of loads that wait for one another, and the launch).
#include "kv_cache.h"

#include <math.h>

namespace lora {

namespace {

// keep every value normal and finite in fp32 and bf16: larger ones than 448 2^119 saturate
constexpr int kMinExponent = -100, kMaxExponent = 119;
constexpr float kMaxCode = 448.0f;

// Which 16 values of a head a thread holds: two runs of 8, and the row of 8
// angles that rotates them (-1: none).  In halves a run rotates with the one half
// the rotated part further on, in pairs each value with its neighbour.
struct Share {
    int c0, c1, angle;
};

__device__ __forceinline__ Share share_of(int a, int rope_dim, bool pairs)
{
    const int turned = rope_dim / 16;        // threads with rotated values
    if (pairs)
        return {16 * a, 16 * a + 8, a < turned ? 8 * a : -1};
    if (a < turned)
        return {8 * a, 8 * a + rope_dim / 2, 8 * a};
    return {rope_dim + 16 * (a - turned), rope_dim + 16 * (a - turned) + 8, -1};
}

__device__ __forceinline__ void load16(const uint16_t* p, const Share& s, float (&x)[16])
{
    const u32x4 lo = *(const global_u32x4*)(p + s.c0), hi = *(const global_u32x4*)(p + s.c1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __builtin_bit_cast(float, lo[i] << 16);
        x[2 * i + 1] = __builtin_bit_cast(float, lo[i] & 0xFFFF0000u);
        x[8 + 2 * i] = __builtin_bit_cast(float, hi[i] << 16);
        x[8 + 2 * i + 1] = __builtin_bit_cast(float, hi[i] & 0xFFFF0000u);
    }
}

// LANES neighbouring lanes hold a head; g: the norm's weights.
template <int LANES>
__device__ __forceinline__ void head_norm(float (&x)[16], const float (&g)[16], float eps)
{
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        sum = fma((double)x[i], (double)x[i], sum);
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1)
        sum += __shfl_xor(sum, d);
    const float inv = 1.0f / sqrtf((float)(sum * (1.0 / (16 * LANES))) + eps);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        x[i] = x[i] * inv * g[i];
}

// The cosines and sines of a thread's values.
struct Angles {
    float c[8], n[8];
};

// A position outside the table rotates by NaN.
__device__ __forceinline__ Angles angles_of(const KvAppendParams& p, const Share& s, int64_t pos)
{
    Angles a;
    if (pos >= 0 && pos < p.rope_rows) {
        const float* row = p.rope + pos * p.ld_rope + s.angle;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4 vc = *(const global_u32x4*)(row + 4 * h);
            const u32x4 vn = *(const global_u32x4*)(row + p.rope_dim / 2 + 4 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t bc = vc[i], bn = vn[i];
                a.c[4 * h + i] = __builtin_bit_cast(float, bc);
                a.n[4 * h + i] = __builtin_bit_cast(float, bn);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            a.c[i] = a.n[i] = __builtin_nanf("");
    }
    return a;
}

__device__ __forceinline__ void rotate(float (&x)[16], const Angles& r, bool pairs)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int ia = pairs ? 2 * i : i, ib = pairs ? 2 * i + 1 : i + 8;
        const float a = x[ia], b = x[ib];
        x[ia] = a * r.c[i] - b * r.n[i];
        x[ib] = b * r.c[i] + a * r.n[i];
    }
}

__device__ __forceinline__ float pow2(int e)
{
    return __builtin_amdgcn_ldexpf(1.0f, e);
}

__device__ __forceinline__ float clamp_code(float x)
{
    return x != x ? x : fminf(fmaxf(x, -kMaxCode), kMaxCode);
}

// Codes of four values times `up`.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float up)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_code(a * up), clamp_code(b * up), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp_code(c * up), clamp_code(d * up), r, true);
}

// Codes of four codes times 2^-shift.
__device__ __forceinline__ uint32_t encode_again(uint32_t codes, float down)
{
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
    return encode4(lo[0], lo[1], hi[0], hi[1], down);
}

// The exponent that values up to amax (finite) need: amax 2^-e <= 448 = 1.75 2^8.
__device__ __forceinline__ int exponent_of(float amax)
{
    const uint32_t bits = __builtin_bit_cast(uint32_t, amax);
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u);
    return min(max(e, kMinExponent), kMaxExponent);
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Slots of blocks that a batch may write, over all sequences: n tokens from any
// position on touch at most n / 16 + 2 blocks.
__host__ __device__ int64_t block_slots(int64_t T, int64_t n_seqs)
{
    return T / kKvBlock + 2 * n_seqs;
}

// Keys (threads 0 .. D-1) and values (D .. 2D-1) of a sequence's new tokens in one of its blocks.
template <int D>
__device__ void append_block(const KvAppendParams& p, int64_t b, const KvSequence& s, int64_t block, int head)
{
    constexpr int LANES = D / 16;
    constexpr int kWaves = 2 * D / 64;
    __shared__ uint32_t amax[kWaves];
    __shared__ __align__(16) uint8_t turned[D * kKvBlock];
    const KvCacheView& c = p.cache;
    const int64_t pos0 = s.len - s.n, from = max(pos0, (int64_t)0);
    const int64_t p0 = max(from, block * kKvBlock), p1 = min(s.len, (block + 1) * kKvBlock);
    if (s.n == 0 || block < 0 || p0 >= p1)
        return;
    const int first = (int)(p0 - block * kKvBlock), last = (int)(p1 - block * kKvBlock);   // new: [first, last)
    const int within = (int)(block & (c.page_size / kKvBlock - 1));

    const bool is_v = threadIdx.x >= D;
    const int i = is_v ? threadIdx.x - D : threadIdx.x;
    const int t = i / LANES, a = i % LANES;
    const bool fresh = t >= first && t < last;
    const Share sh = share_of(a, is_v ? 0 : p.rope_dim, is_v || p.pairs);
    const int64_t pos = block * kKvBlock + t;
    // what does not wait for the page is asked for with it
    float x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
        x[j] = 0.0f;
    if (fresh)
        load16((is_v ? p.v + (s.first + (pos - pos0)) * p.ld_v : p.k + (s.first + (pos - pos0)) * p.ld_k) + head * D,
               sh, x);
    const bool norm = !is_v && p.k_norm, turn = !is_v && p.rope && fresh && sh.angle >= 0;
    float g[16];
    Angles angles;
    if (norm)
        load16(p.k_norm, sh, g);
    if (turn)
        angles = angles_of(p, sh, pos);
    const int32_t page = kv_page(c, b, block * kKvBlock);
    if (page < 0)
        return;
    uint8_t* scale = (is_v ? c.v_scales + (int64_t)page * c.ld_vs : c.k_scales + (int64_t)page * c.ld_ks) +
                     (int64_t)head * (c.page_size / kKvBlock) + within;
    const int had = first > 0 ? *scale : 0;
    uint8_t* base = (is_v ? c.v + (int64_t)page * c.ld_v : c.k + (int64_t)page * c.ld_k) +
                    ((int64_t)head * c.page_size + within * kKvBlock) * D;
    // of the values all tokens of a d lie together, so old ones are read with them
    u32x4 before = {0, 0, 0, 0};
    if (is_v && last - first < kKvBlock)
        before = *(const global_u32x4*)(base + i * kKvBlock);
    if (norm)
        head_norm<LANES>(x, g, p.eps);
    if (turn)
        rotate(x, angles, p.pairs);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint32_t m = __builtin_bit_cast(uint32_t, x[j]) & 0x7FFFFFFFu;
        top = max(top, m < 0x7F800000u ? m : 0u);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if ((threadIdx.x & 63) == 0)
        amax[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves / 2; ++w)
        top = max(top, amax[(is_v ? kWaves / 2 : 0) + w]);
    const int need = exponent_of(__builtin_bit_cast(float, top)) + 127;
    const int now = first > 0 ? max(need, had) : need;
    const bool again = first > 0 && now > had;
    const float up = pow2(127 - now), down = pow2(max(had - now, -120));
    uint32_t code[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        code[j] = encode4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3], up);
    if (i == 0)
        *scale = (uint8_t)now;
    if (is_v) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            turned[(16 * a + j) * kKvBlock + t] = (uint8_t)(code[j / 4] >> (8 * (j % 4)));
    }
    __syncthreads();
    if (is_v) {
        u32x4 now4 = *reinterpret_cast<const u32x4*>(turned + i * kKvBlock);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t old = before[j], earlier = again ? encode_again(old, down) : old;
            uint32_t r = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int token = 4 * j + e;
                const uint32_t from4 = token < first ? earlier : token < last ? now4[j] : old;
                r |= from4 & (0xFFu << (8 * e));
            }
            now4[j] = r;
        }
        *reinterpret_cast<u32x4*>(base + i * kKvBlock) = now4;
    } else if (fresh || (again && t < first)) {
        u32x2* k0 = reinterpret_cast<u32x2*>(base + t * D + sh.c0);
        u32x2* k1 = reinterpret_cast<u32x2*>(base + t * D + sh.c1);
        u32x2 n0 = {code[0], code[1]}, n1 = {code[2], code[3]};
        if (!fresh) {
            const u32x2 o0 = *k0, o1 = *k1;
            n0 = u32x2{encode_again(o0[0], down), encode_again(o0[1], down)};
            n1 = u32x2{encode_again(o1[0], down), encode_again(o1[1], down)};
        }
        *k0 = n0;
        *k1 = n1;
    }
}

template <int D>
__device__ void append_queries(const KvAppendParams& p, int64_t token)
{
    constexpr int LANES = D / 16;
    const KvCacheView& c = p.cache;
    const KvSequence s = kv_find(c, p.T, token, p.T, [](int64_t, int64_t cu) { return cu; }).s;
    if (s.n == 0 || token < s.first)
        return;
    const int64_t pos = s.len - s.n + (token - s.first);
    const Share sh = share_of(threadIdx.x % LANES, p.rope_dim, p.pairs);
    float g[16];
    Angles angles;
    const bool turn = p.rope && sh.angle >= 0;
    if (p.q_norm)
        load16(p.q_norm, sh, g);
    if (turn)
        angles = angles_of(p, sh, pos);
    // whole heads a round, so that lanes of a head stay together
    for (int h = threadIdx.x / LANES; h < p.q_heads; h += 2 * D / LANES) {
        float x[16];
        load16(p.q + token * p.ld_q + (int64_t)h * D, sh, x);
        if (p.q_norm)
            head_norm<LANES>(x, g, p.eps);
        if (turn)
            rotate(x, angles, p.pairs);
        uint16_t* out = p.q_out + token * p.ld_qo + (int64_t)h * D;
        u16x8 lo, hi;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = __builtin_bit_cast(uint16_t, (__bf16)x[i]);
            hi[i] = __builtin_bit_cast(uint16_t, (__bf16)x[8 + i]);
        }
        *reinterpret_cast<u16x8*>(out + sh.c0) = lo;
        *reinterpret_cast<u16x8*>(out + sh.c1) = hi;
    }
}

// DIRECT: a workgroup a sequence and head, for one block usually; else one for each block
// that may be written.  (In one kernel the loop's registers halve the other way's waves:
// 8190 tokens 80 -> 92 us.)
template <int D, bool DIRECT>
__global__ void __launch_bounds__(2 * D) k_kv_append(KvAppendParams p, int64_t blocks)
{
    const int64_t w = blockIdx.x;
    if (w >= blocks) {
        append_queries<D>(p, w - blocks);
        return;
    }
    const int64_t slot = (uint32_t)w / (uint32_t)p.cache.heads;
    const int head = (int)((uint32_t)w % (uint32_t)p.cache.heads);
    if constexpr (DIRECT) {
        const KvSequence q = kv_sequence(p.cache, slot, p.T);
        const int64_t stop = q.n ? (q.len + kKvBlock - 1) / kKvBlock : 0;
#pragma unroll 1
        for (int64_t block = max(q.len - q.n, (int64_t)0) / kKvBlock; block < stop; ++block) {
            append_block<D>(p, slot, q, block, head);
            __syncthreads();                 // before the next one's values
        }
    } else {
        const KvFound f = kv_find(p.cache, p.T, slot, block_slots(p.T, p.cache.n_seqs),
                                  [](int64_t j, int64_t cu) { return cu / kKvBlock + 2 * j; });
        if (f.b >= 0)
            append_block<D>(p, f.b, f.s,
                            max(f.s.len - f.s.n, (int64_t)0) / kKvBlock + (slot - (f.s.first / kKvBlock + 2 * f.b)), head);
    }
}

template <int D>
hipError_t launch(const KvAppendParams& p, hipStream_t st)
{
    // as many new tokens as sequences: a step of single tokens, nearly always; half of the
    // slots would find nothing to do (251 tokens, 8 heads 14.1 -> 12.5 us)
    const bool direct = p.T == p.cache.n_seqs;
    const int64_t blocks = (direct ? p.T : block_slots(p.T, p.cache.n_seqs)) * p.cache.heads;
    const dim3 grid((unsigned)(blocks + (p.q ? p.T : 0)));
    if (direct)
        hipLaunchKernelGGL((k_kv_append<D, true>), grid, dim3(2 * D), 0, st, p, blocks);
    else
        hipLaunchKernelGGL((k_kv_append<D, false>), grid, dim3(2 * D), 0, st, p, blocks);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvAppendParams& p, hipStream_t st)
{
    return p.D == 64 ? launch<64>(p, st) : p.D == 128 ? launch<128>(p, st) : launch<256>(p, st);
}

}  // namespace lora
