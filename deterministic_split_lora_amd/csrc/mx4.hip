// MX4 quantisation and its inverse.
//
// Quantise: a block of 32 values v takes the scale 2^e with
// e = max(floor(log2 max|v|) - 2, -127), so that the largest magnitude lies in
// [4, 8) 2^e, and each value becomes the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6
// times 2^e (ties to the code with the even last bit, magnitudes above 6
// become 6).  Division by a power of two is exact, so the only rounding is the
// conversion's own.  A block with a NaN or an infinity gets the NaN scale.
//
// Both directions are bound by memory (2 bytes of bf16 and 17/32 of a byte of
// codes and scales an element).  A lane holds 8 elements, one 16-byte access
// on the bf16 side and one word of codes; four neighbouring lanes are a block.
// A wave takes up to kSegment elements of one row, all its loads first.  Measured
// on MI355X: 4099 x 14336 quantised in 30.2 us (4.9 TB/s) and dequantised in
// 23.4 us (6.4 TB/s, the codes partly from the last-level cache); 32 x 4096 in
// 3.2 and 3.0 us, a launch each.
#include "mx4.h"

namespace lora {

namespace {

constexpr int kLaneElems = 8;
constexpr int kPass = kWave * kLaneElems;    // elements of one wave pass
constexpr int kPasses = 4;
constexpr int kSegment = kPass * kPasses;
constexpr int kQuantWaves = 4;
constexpr int64_t kMaxBlocks = int64_t{1} << 20;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
}

// f(row, this lane's first element) for each part of a row that this wave has.
template <class F>
__device__ __forceinline__ void wave_segments(const Mx4QuantParams& p, F f)
{
    const uint32_t segs = ((uint32_t)p.K + kSegment - 1) / kSegment;
    int64_t item = (int64_t)blockIdx.x * kQuantWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (; item < p.M * segs; item += (int64_t)gridDim.x * kQuantWaves) {
        const int64_t row = item / segs;
        f(row, (int)(item - row * segs) * kSegment + (int)(threadIdx.x & 63) * kLaneElems);
    }
}

__device__ __forceinline__ void quantize_segment(const Mx4QuantParams& p, int64_t row, int k0)
{
    u32x4 v[kPasses];
    const uint16_t* xr = p.x + row * p.ld_x;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int k = k0 + i * kPass;
        v[i] = k < p.K ? *(const global_u32x4*)(xr + k) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int k = k0 + i * kPass;
        // largest magnitude of the block, as bf16 bits (they order like the values)
        uint32_t m = max_u16x2(max_u16x2(v[i][0] & 0x7FFF7FFFu, v[i][1] & 0x7FFF7FFFu),
                               max_u16x2(v[i][2] & 0x7FFF7FFFu, v[i][3] & 0x7FFF7FFFu));
        m = max_u16x2(m, (uint32_t)__shfl_xor((int)m, 1));
        m = max_u16x2(m, (uint32_t)__shfl_xor((int)m, 2));
        const uint32_t top = max(m & 0xFFFFu, m >> 16) >> 7;        // its exponent field
        const bool bad = top == 255;
        const uint32_t b = bad ? 255u : (top > 2 ? top - 2 : 0u);
        const float scale = mx_scale_f32(bad ? 127u : b);
        const uint32_t w = bf16_to_mx4(v[i], scale);
        if (k < p.K) {
            *reinterpret_cast<uint32_t*>(p.q + row * p.ld_q + k / 2) = bad ? 0u : w;
            if (k % kMxBlock == 0)
                p.scales[row * p.ld_s + k / kMxBlock] = (uint8_t)b;
        }
    }
}

__device__ __forceinline__ void dequantize_segment(const Mx4QuantParams& p, int64_t row, int k0)
{
    uint32_t w[kPasses], b[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int k = k0 + i * kPass;
        w[i] = k < p.K ? *reinterpret_cast<const uint32_t*>(p.q + row * p.ld_q + k / 2) : 0u;
        b[i] = k < p.K ? p.scales[row * p.ld_s + k / kMxBlock] : 0u;
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int k = k0 + i * kPass;
        if (k < p.K)
            *reinterpret_cast<u32x4*>(p.x_out + row * p.ld_x + k) =
                __builtin_bit_cast(u32x4, mx4_to_bf16(w[i], mx_scale_f32(b[i])));
    }
}

__global__ void __launch_bounds__(kQuantWaves * kWave) k_mx4_quantize(Mx4QuantParams p)
{
    wave_segments(p, [&](int64_t row, int k0) { quantize_segment(p, row, k0); });
}

__global__ void __launch_bounds__(kQuantWaves * kWave) k_mx4_dequantize(Mx4QuantParams p)
{
    wave_segments(p, [&](int64_t row, int k0) { dequantize_segment(p, row, k0); });
}

// A launch holds fewer than 2^32 threads; waves take further parts beyond that.
unsigned quant_grid(const Mx4QuantParams& p)
{
    const int64_t segs = ((int64_t)p.K + kSegment - 1) / kSegment;
    const int64_t blocks = (p.M * segs + kQuantWaves - 1) / kQuantWaves;
    return (unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks);
}

}  // namespace

hipError_t launch_mx4_quantize(const Mx4QuantParams& p, hipStream_t st)
{
    k_mx4_quantize<<<dim3(quant_grid(p)), dim3(kQuantWaves * kWave), 0, st>>>(p);
    return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const Mx4QuantParams& p, hipStream_t st)
{
    k_mx4_dequantize<<<dim3(quant_grid(p)), dim3(kQuantWaves * kWave), 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace lora
