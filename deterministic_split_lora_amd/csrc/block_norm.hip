// The step between two blocks of a network, one pass over each row:
//     t  = post_norm(y)                     RMS or layer norm, or y itself
//     r' = res_scale r + gate t             fp32; stored as bf16
//     x  = pre_norm(r')                     from the fp32 r', stored as bf16
// with norm(v) = v rsqrt(mean(v^2) + eps) w (+ b), v centred first for a layer
// norm.  Bound by memory: y, r (and a gate per token) are read once, r' and x
// written once; the row stays in registers between its two reductions.
//
// A workgroup owns a row; a thread holds VPT groups of 8 consecutive elements.
// A sum is: a thread's elements in order, the wave's 64 lanes by a butterfly,
// then the waves in ascending order.  Threads and VPT follow from C alone, so a
// row's bits do not depend on the other rows.  As many threads as the row has
// groups (up to 1024), because a single token's latency is two reductions:
// measured on MI355X, 1 x 8192 in 4.1 us, 4096 x 8192 with a gate per token in
// 66 us (335 MB, 5.1 TB/s, a large copy's rate).  Between the variants' widths part
// of a workgroup has no columns: without a gate, 8192 x 2048 24 us, 8192 x 2560 51
// (3.3 TB/s), 8192 x 4096 54 (5.0), 8192 x 5120 74 (4.6), 8192 x 8192 101 (5.3).
#include "device.h"
#include "step_kernels.h"

namespace lora {

namespace {

constexpr int kNormNone = 0, kNormLayer = 2;   // lora_norm_kind

template <int WAVES>
__device__ __forceinline__ float row_sum(float v, float* buf)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v += __shfl_xor(v, d);
    if constexpr (WAVES > 1) {
        if ((threadIdx.x & 63) == 0)
            buf[threadIdx.x >> 6] = v;
        __syncthreads();
        v = buf[0];
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
            v += buf[w];
    }
    return v;
}

__device__ __forceinline__ void unpack8(u32x4 u, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __builtin_bit_cast(float, u[i] << 16);
        f[2 * i + 1] = __builtin_bit_cast(float, u[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ u32x4 pack8(const float (&f)[8])
{
    u32x4 u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = f32_to_bf16_bits(f[2 * i]) | (uint32_t)f32_to_bf16_bits(f[2 * i + 1]) << 16;
    return u;
}

__device__ __forceinline__ u32x4 load16(const uint16_t* p)
{
    return *(const global_u32x4*)(p);
}

// v <- norm(v) over the row, in place; buf: 2 * WAVES floats of this call's own.
template <int VPT, int WAVES>
__device__ __forceinline__ void normalise(float (&v)[VPT][8], const NormParams& p, int kind, const uint16_t* w,
                                          const uint16_t* b, float* buf)
{
    const float inv_c = 1.0f / (float)p.C;
    if (kind == kNormLayer) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s += v[i][e];
        const float mean = row_sum<WAVES>(s, buf) * inv_c;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[i][e] -= mean;
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if ((int)(threadIdx.x + i * WAVES * 64) * 8 < p.C) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                q = fmaf(v[i][e], v[i][e], q);
        }
    const float rs = rsqrtf(row_sum<WAVES>(q, buf + WAVES) * inv_c + p.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (threadIdx.x + i * WAVES * 64) * 8;
        if (c < p.C) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[i][e] *= rs;
            if (w) {
                unpack8(load16(w + c), f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[i][e] *= f[e];
            }
            if (b) {
                unpack8(load16(b + c), f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[i][e] += f[e];
            }
        }
    }
}

template <int VPT, int WAVES>
__device__ __forceinline__ void norm_row(const NormParams& p, int64_t row, float* buf)
{
    float v[VPT][8];
    u32x4 rr[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (threadIdx.x + i * WAVES * 64) * 8;
        const bool in = c < p.C;
        rr[i] = in ? load16(p.r + row * p.ld_r + c) : u32x4{0, 0, 0, 0};
        unpack8(in && p.y ? load16(p.y + row * p.ld_y + c) : u32x4{0, 0, 0, 0}, v[i]);
    }
    if (p.y && p.post != kNormNone)
        normalise<VPT, WAVES>(v, p, p.post, p.post_w, p.post_b, buf);
    const uint16_t* gate = p.gate ? p.gate + (row / p.gate_group) * p.ld_gate : nullptr;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (threadIdx.x + i * WAVES * 64) * 8;
        const bool in = c < p.C;
        if (p.y && gate && in) {
            float f[8];
            unpack8(load16(gate + c), f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[i][e] *= f[e];
        }
        float f[8];
        unpack8(rr[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[i][e] = in ? (p.y ? fmaf(p.res_scale, f[e], v[i][e]) : p.res_scale * f[e]) : 0.0f;
        if (in)
            *reinterpret_cast<u32x4*>(p.r_out + row * p.ld_ro + c) = pack8(v[i]);
    }
    if (!p.x_out)
        return;
    normalise<VPT, WAVES>(v, p, p.pre, p.pre_w, p.pre_b, buf + 2 * WAVES);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (threadIdx.x + i * WAVES * 64) * 8;
        if (c < p.C)
            *reinterpret_cast<u32x4*>(p.x_out + row * p.ld_xo + c) = pack8(v[i]);
    }
}

// A launch holds fewer than 2^32 threads: beyond kMaxRows a workgroup takes
// further rows.
constexpr int64_t kMaxRows = int64_t{1} << 20;

template <int VPT, int WAVES>
__global__ void __launch_bounds__(WAVES * 64) k_block_norm(NormParams p)
{
    __shared__ float buf[4 * WAVES];
    norm_row<VPT, WAVES>(p, blockIdx.x, buf);
    for (int64_t row = (int64_t)blockIdx.x + kMaxRows; row < p.M; row += kMaxRows) {
        __syncthreads();                     // the row before's sums have been read
        norm_row<VPT, WAVES>(p, row, buf);
    }
}

}  // namespace

hipError_t launch_block_norm(const NormParams& p, hipStream_t st)
{
    const dim3 grid((unsigned)(p.M < kMaxRows ? p.M : kMaxRows));
    if (p.C <= 512)
        hipLaunchKernelGGL((k_block_norm<1, 1>), grid, dim3(64), 0, st, p);
    else if (p.C <= 2048)
        hipLaunchKernelGGL((k_block_norm<1, 4>), grid, dim3(256), 0, st, p);
    else if (p.C <= 8192)
        hipLaunchKernelGGL((k_block_norm<1, 16>), grid, dim3(1024), 0, st, p);
    else if (p.C <= 16384)
        hipLaunchKernelGGL((k_block_norm<2, 16>), grid, dim3(1024), 0, st, p);
    else
        hipLaunchKernelGGL((k_block_norm<4, 16>), grid, dim3(1024), 0, st, p);
    return hipGetLastError();
}

}  // namespace lora
