// Products with MX4 weights:  y = x W^T  for bf16 x and for MX4 x.
//
// Arithmetic, the same in every kernel of this file so that schedules agree
// bit for bit.  K is cut into split_k chunks.  A chunk's sum is one chain of
// matrix-core steps over its blocks in ascending k, four blocks (128 k) at a
// time, from zero, in fp32; block g of the four belongs to the lanes of group g
// (li = lane % 16, g = lane / 16).  Chunk sums are added in ascending order and
// the total is rounded once to bf16.  Blocks past the chunk's end enter as
// zeros.
//   bf16 x: a step is four V_MFMA_F32_16X16X32_BF16; the s-th takes elements
//     8s .. 8s+7 of each block, the codes converted to bf16 (exactly) on the way.
//   MX4 x: a step is one V_MFMA_SCALE_F32_16X16X128_F8F6F4, which takes both
//     operands' codes and scales as they are stored.
// The "row" operand is W, so a lane's accumulator holds four consecutive output
// columns of one token.
#include "mx4_tile.h"

namespace lora {

namespace {

constexpr int kStepK = 128;

__device__ __forceinline__ MxOperand load_mx(const uint8_t* q, const uint8_t* s, int64_t k, bool ok)
{
    MxOperand o;
    o.q = ok ? *(const global_u32x4*)(q + k / 2) : u32x4{0, 0, 0, 0};
    o.s = ok ? s[k / kMxBlock] : 127u;
    return o;
}

// Few tokens: a workgroup owns 16 RT tokens x 16 CT columns (times the column
// groups G), its wave (g, s) the chain of chunk s; the chains meet in LDS.
template <bool XMX, int RT, int CT>
__global__ void __launch_bounds__(1024) k_mx4_linear_rows(Mx4LinearParams p, int groups)
{
    extern __shared__ float lds[];
    const int lane = threadIdx.x & 63;
    const int li = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int S = p.split_k;
    const int chunk = wave % S, group = wave / S;
    const int64_t n0 = ((int64_t)blockIdx.x * groups + group) * (16 * CT);
    const int64_t m0 = (int64_t)blockIdx.y * (16 * RT);

    f32x4 acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c)
            acc[r][c] = f32x4{0, 0, 0, 0};

    const uint8_t* wq[CT];
    const uint8_t* ws[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int64_t n = min(n0 + 16 * c + li, p.N - 1);
        wq[c] = p.wq + n * p.ld_wq;
        ws[c] = p.ws + n * p.ld_ws;
    }
    const uint8_t* xq[RT];
    const uint8_t* xs[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int64_t m = min(m0 + 16 * r + li, p.M - 1);
        xq[r] = static_cast<const uint8_t*>(p.x) + m * p.ld_x * (XMX ? 1 : 2);
        xs[r] = XMX ? p.xs + m * p.ld_xs : nullptr;
    }
    const int64_t kc = (int64_t)chunk * p.k_chunk;
    for (int t = 0; t < p.k_chunk; t += kStepK) {
        const bool ok = t + g * kMxBlock < p.k_chunk;
        const int64_t k = kc + t + g * kMxBlock;
        MxOperand w[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c)
            w[c] = load_mx(wq[c], ws[c], k, ok);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            if constexpr (XMX) {
                const MxOperand x = load_mx(xq[r], xs[r], k, ok);
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    acc[r][c] = mfma_mx4(w[c], x, acc[r][c]);
            } else {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const bf16x8 x = ok ? load_bf16x8(reinterpret_cast<const uint16_t*>(xq[r]) + k + 8 * s)
                                        : bf16x8_zero();
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        acc[r][c] = mfma_16x16x32(mx4_to_bf16(w[c].q[s], mx_scale_f32(w[c].s)), x, acc[r][c]);
                }
            }
        }
    }

    // chains to LDS: [group][chunk][r][c][lane][4], then a thread adds its
    // output's chunks in ascending order
    constexpr int kTile = 256;
    float* mine = lds + ((int64_t)group * S + chunk) * (RT * CT * kTile);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c)
            *reinterpret_cast<f32x4*>(mine + (r * CT + c) * kTile + lane * 4) = acc[r][c];
    __syncthreads();
    const int quads = groups * RT * CT * 64;
    for (int i = threadIdx.x; i < quads; i += blockDim.x) {
        const int l = i & 63, tile = (i >> 6) % (RT * CT), grp = (i >> 6) / (RT * CT);
        const float* src = lds + ((int64_t)grp * S * (RT * CT) + tile) * kTile + l * 4;
        f32x4 sum = *reinterpret_cast<const f32x4*>(src);
        for (int s = 1; s < S; ++s) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(src + s * (RT * CT * kTile));
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum[e] += v[e];
        }
        const int64_t m = m0 + 16 * (tile / CT) + (l & 15);
        const int64_t n = ((int64_t)blockIdx.x * groups + grp) * (16 * CT) + 16 * (tile % CT) + 4 * (l >> 4);
        if (m < p.M && n < p.N) {
            const uint32_t lo = f32_to_bf16_bits(sum[0]) | (uint32_t)f32_to_bf16_bits(sum[1]) << 16;
            const uint32_t hi = f32_to_bf16_bits(sum[2]) | (uint32_t)f32_to_bf16_bits(sum[3]) << 16;
            *reinterpret_cast<u32x2*>(p.y + m * p.ld_y + n) = u32x2{lo, hi};
        }
    }
}

template <bool XMX, int RT, int CT>
hipError_t launch_rows(const Mx4LinearParams& p, hipStream_t st)
{
    const int groups = p.split_k < 4 ? 4 / p.split_k : 1;
    const int64_t cols = 16 * CT * groups;
    const dim3 grid((unsigned)((p.N + cols - 1) / cols), (unsigned)((p.M + 16 * RT - 1) / (16 * RT)));
    const size_t lds = (size_t)groups * p.split_k * RT * CT * 1024;
    hipLaunchKernelGGL((k_mx4_linear_rows<XMX, RT, CT>), grid, dim3(64 * groups * p.split_k), lds, st, p, groups);
    return hipGetLastError();
}

}  // namespace

int64_t mx4_linear_workspace(int64_t M, int64_t N, int32_t k_chunk, int32_t split_k, bool x_is_mx4)
{
    (void)M; (void)N; (void)k_chunk; (void)split_k; (void)x_is_mx4;
    return 0;
}

hipError_t launch_mx4_linear(const Mx4LinearParams& p, bool x_is_mx4, hipStream_t st)
{
    if (p.M > 64 && p.k_chunk * (int64_t)p.split_k >= 512) {
        if (p.split_k > 1)
            return x_is_mx4 ? launch_tile<true, 128, 256, true>(p, st) : launch_tile<false, 128, 256, true>(p, st);
        return x_is_mx4 ? launch_tile<true, 256, 256, false>(p, st) : launch_tile<false, 128, 256, false>(p, st);
    }
    if (p.M <= 16)
        return x_is_mx4 ? launch_rows<true, 1, 1>(p, st) : launch_rows<false, 1, 1>(p, st);
    if (p.M <= 32)
        return x_is_mx4 ? launch_rows<true, 2, 1>(p, st) : launch_rows<false, 2, 1>(p, st);
    return x_is_mx4 ? launch_rows<true, 4, 1>(p, st) : launch_rows<false, 4, 1>(p, st);
}

}  // namespace lora
