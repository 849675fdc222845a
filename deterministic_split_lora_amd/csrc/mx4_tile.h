// Large products with MX4 weights: a workgroup of eight waves owns a TM x TN
// tile of y, wave (wm, wn) of 2 x 4 a (TM / 2) x (TN / 4) part of it.  Included by
// mx4_linear.hip, which states the arithmetic.
//
// Steps of 128 k go through a ring of NS stages in LDS, filled by loads that
// write LDS themselves.  At step j a wave waits until its own loads of stage j
// have landed, meets the others at the one barrier of the step (then all of
// stage j is there and stage j - 1 is read out), starts the loads of step
// j + NS - 1 into the buffer of stage j - 1, and multiplies stage j.
//
// LDS layout: 16-byte pieces of a row, in an order that depends on the row, so
// that the 16 rows a matrix-core operand reads at one k fall on different
// banks.  The order is applied to the global address each lane loads from
// (the loads fill LDS in lane order).  Scales: one word (four blocks) of every
// row a slot, kSlots words deep, read by the byte; a row's scale bytes are
// contiguous over the chunks, so words are loaded once each, in order.
#pragma once

#include "mx4.h"

namespace lora {

constexpr int kTileWaves = 8;
constexpr int kSlots = 8;                    // scale words of a row in flight

typedef __attribute__((address_space(3))) uint8_t lds_u8;

// 64 lanes x 16 (4) bytes from per-lane addresses to LDS at `to` + 16 (4) lane.
// These write no registers, so the compiler need not know when they land; the
// kernel waits for them by count (wait_loads).
__device__ __forceinline__ void load_to_lds16(const uint8_t* from, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(to) : "memory");
}

__device__ __forceinline__ void load_to_lds4(const uint8_t* from, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(from), "s"(to) : "memory");
}

// Waits until at most N of this wave's loads are outstanding and its LDS reads
// are done, then meets the workgroup.
template <int N>
__device__ __forceinline__ void wait_loads_and_meet()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Where 16-byte piece c of a row goes: rows of 64 bytes (4 pieces) and of 256
// bytes (16 pieces).
__device__ __forceinline__ int swizzle4(int row)
{
    return ((row >> 1) & 3) ^ ((row >> 3) & 1);
}

__device__ __forceinline__ int swizzle16(int row)
{
    return row & 15;
}

template <bool XMX, int TM, int TN>
struct TileShape {
    static constexpr int kXBytes = XMX ? 64 : 256;           // of a row and step
    static constexpr int kXStage = TM * kXBytes;
    static constexpr int kWStage = TN * 64;
    static constexpr int kStage = kXStage + kWStage;
    static constexpr int kXLoads = kXStage / (kTileWaves * 1024);
    static constexpr int kWLoads = kWStage / (kTileWaves * 1024);
    static constexpr int kScaleRows = TN + (XMX ? TM : 0);   // W's rows first
    static constexpr int kScaleWaves = kScaleRows / 64;
    static constexpr int kRows = TM / 32, kCols = TN / 64;   // 16 x 16 tiles of a wave
    static constexpr int kBudget = 160 * 1024 - kSlots * kScaleRows * 4;
    static constexpr int kStages = kBudget / kStage < 4 ? kBudget / kStage : 4;
    static constexpr int kLds = kStages * kStage + kSlots * kScaleRows * 4;
    static_assert(kXLoads >= 1 && kWLoads >= 1 && kStages >= 2, "tile too small or too large");
};

template <bool XMX, int TM, int TN, bool SPLIT>
__global__ void __launch_bounds__(kTileWaves * 64, 2) k_mx4_linear_tile(Mx4LinearParams p)
{
    using T = TileShape<XMX, TM, TN>;
    __shared__ __align__(16) uint8_t lds[T::kLds];
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8*)lds;
    const int lane = threadIdx.x & 63;
    const int li = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 2, wn = wave & 3;

    // Tile of this workgroup.  Workgroups go round the XCDs one by one; each XCD
    // gets a contiguous run of the tiles, in strips of eight tile rows walked
    // column by column, so that tiles in flight together share x and W in its L2.
    const int tiles_m = (int)((p.M + TM - 1) / TM), tiles_n = (int)((p.N + TN - 1) / TN);
    const int total = tiles_m * tiles_n;
    constexpr int kXcds = 8, kStrip = 8;
    const int xcd = (int)blockIdx.x % kXcds, pos = (int)blockIdx.x / kXcds;
    const int per = total / kXcds, extra = total % kXcds;
    const int id = xcd * per + min(xcd, extra) + pos;
    const int strip = id / (kStrip * tiles_n);
    const int in_strip = id - strip * kStrip * tiles_n;
    const int strip_rows = min(kStrip, tiles_m - strip * kStrip);
    const int64_t m0 = (int64_t)(strip * kStrip + in_strip % strip_rows) * TM;
    const int64_t n0 = (int64_t)(in_strip / strip_rows) * TN;

    // per-lane sources: a piece's place in LDS is its load's place in the
    // stage, load i of wave w filling 1024 bytes from (i * 8 + w) * 1024
    const uint8_t* xsrc[T::kXLoads];
    int xblock[T::kXLoads];
#pragma unroll
    for (int i = 0; i < T::kXLoads; ++i) {
        constexpr int P = T::kXBytes / 16;
        const int piece = (i * kTileWaves + wave) * 64 + lane;
        const int row = piece / P;
        const int c = (piece % P) ^ (XMX ? swizzle4(row) : swizzle16(row));
        const int64_t m = min(m0 + row, p.M - 1);
        xblock[i] = XMX ? c : c >> 2;
        xsrc[i] = static_cast<const uint8_t*>(p.x) + m * p.ld_x * (XMX ? 1 : 2) + c * 16;
    }
    const uint8_t* wsrc[T::kWLoads];
    int wblock[T::kWLoads];
#pragma unroll
    for (int i = 0; i < T::kWLoads; ++i) {
        const int piece = (i * kTileWaves + wave) * 64 + lane;
        const int row = piece / 4;
        const int c = (piece % 4) ^ swizzle4(row);
        const int64_t n = min(n0 + row, p.N - 1);
        wblock[i] = c;
        wsrc[i] = p.wq + n * p.ld_wq + c * 16;
    }
    const uint8_t* ssrc = nullptr;
    {
        const int row = wave * 64 + lane;
        if (row < TN)
            ssrc = p.ws + min(n0 + row, p.N - 1) * p.ld_ws;
        else if (XMX && row < TN + TM)
            ssrc = p.xs + min(m0 + row - TN, p.M - 1) * p.ld_xs;
    }

    const int chunk_steps = (p.k_chunk + 127) / 128;
    const int steps = chunk_steps * p.split_k;
    const int last_word = (p.k_chunk / kMxBlock * p.split_k - 1) >> 2;
    int words = 0;                           // scale words whose loads have been started

    // the step whose loads come next: its number within the chunk and its k
    int next_t = 0;
    int64_t next_k = 0;
    int next_stage = 0;
    auto start_loads = [&]() {
        const uint32_t base = lds0 + next_stage * T::kStage;
        const int left = p.k_chunk - next_t * 128;           // k left in the chunk
#pragma unroll
        for (int i = 0; i < T::kXLoads; ++i) {
            // blocks past the chunk's end load the step's first block instead
            const int64_t back = xblock[i] * kMxBlock < left ? 0 : xblock[i] * (XMX ? 16 : 64);
            load_to_lds16(xsrc[i] + (XMX ? next_k / 2 : next_k * 2) - back,
                          __builtin_amdgcn_readfirstlane(base + (i * kTileWaves + wave) * 1024));
        }
#pragma unroll
        for (int i = 0; i < T::kWLoads; ++i) {
            const int64_t back = wblock[i] * kMxBlock < left ? 0 : wblock[i] * 16;
            load_to_lds16(wsrc[i] + next_k / 2 - back,
                          __builtin_amdgcn_readfirstlane(base + T::kXStage + (i * kTileWaves + wave) * 1024));
        }
        const int need = min((int)((next_k / kMxBlock + 3) >> 2), last_word);
        if (words <= need) {                 // at most one more word a step
            if (wave < T::kScaleWaves)
                load_to_lds4(ssrc + words * 4,
                             __builtin_amdgcn_readfirstlane(lds0 + T::kStages * T::kStage +
                                                            ((words % kSlots) * T::kScaleRows + wave * 64) * 4));
            ++words;
        }
        next_k += min(left, 128);
        next_t = next_t + 1 == chunk_steps ? 0 : next_t + 1;
        next_stage = next_stage + 1 == T::kStages ? 0 : next_stage + 1;
    };

    f32x4 acc[T::kRows][T::kCols], tot[SPLIT ? T::kRows : 1][T::kCols];
#pragma unroll
    for (int r = 0; r < T::kRows; ++r)
#pragma unroll
        for (int c = 0; c < T::kCols; ++c)
            acc[r][c] = f32x4{0, 0, 0, 0};

    for (int j = 0; j < T::kStages - 1; ++j)
        if (j < steps)
            start_loads();

    int t = 0, chunk = 0, stage = 0;
    int64_t k = 0;
    for (int j = 0; j < steps; ++j) {
        // the loads of the steps after j may still be on their way
        constexpr int kStepLoads = T::kXLoads + T::kWLoads;
        if (j + T::kStages - 2 < steps)
            wait_loads_and_meet<(T::kStages - 2) * kStepLoads>();
        else
            wait_loads_and_meet<0>();
        if (j + T::kStages - 1 < steps)
            start_loads();

        const uint8_t* xs = lds + stage * T::kStage;
        const uint8_t* ws = xs + T::kXStage;
        const int left = p.k_chunk - t * 128;
        // the scale of one block, of row 0 (rows are 4 bytes apart)
        auto scale_bytes = [&](int block) {
            return lds + T::kStages * T::kStage + ((block >> 2) % kSlots) * (T::kScaleRows * 4) + (block & 3);
        };

        if constexpr (XMX) {
            const bool ok = g * kMxBlock < left;
            const int block = (int)(k / kMxBlock) + g;
            const uint8_t* sc = scale_bytes(block);
            MxOperand w[T::kCols];
#pragma unroll
            for (int c = 0; c < T::kCols; ++c) {
                const int row = wn * (TN / 4) + 16 * c + li;
                w[c].q = *reinterpret_cast<const u32x4*>(ws + row * 64 + ((g ^ swizzle4(row)) * 16));
                w[c].s = sc[row * 4];
                if (!ok)
                    w[c] = MxOperand{u32x4{0, 0, 0, 0}, 127};
            }
#pragma unroll
            for (int r = 0; r < T::kRows; ++r) {
                const int row = wm * (TM / 2) + 16 * r + li;
                MxOperand x;
                x.q = *reinterpret_cast<const u32x4*>(xs + row * 64 + ((g ^ swizzle4(row)) * 16));
                x.s = sc[(TN + row) * 4];
                if (!ok)
                    x = MxOperand{u32x4{0, 0, 0, 0}, 127};
#pragma unroll
                for (int c = 0; c < T::kCols; ++c)
                    acc[r][c] = mfma_mx4(w[c], x, acc[r][c]);
            }
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (s * kMxBlock >= left)
                    break;
                const uint8_t* sc = scale_bytes((int)(k / kMxBlock) + s);
                bf16x8 wb[T::kCols];
#pragma unroll
                for (int c = 0; c < T::kCols; ++c) {
                    const int row = wn * (TN / 4) + 16 * c + li;
                    const uint32_t q = *reinterpret_cast<const uint32_t*>(ws + row * 64 + ((s ^ swizzle4(row)) * 16) + 4 * g);
                    wb[c] = mx4_to_bf16(q, mx_scale_f32(sc[row * 4]));
                }
#pragma unroll
                for (int r = 0; r < T::kRows; ++r) {
                    const int row = wm * (TM / 2) + 16 * r + li;
                    const u32x4 x = *reinterpret_cast<const u32x4*>(xs + row * 256 + (((4 * s + g) ^ swizzle16(row)) * 16));
#pragma unroll
                    for (int c = 0; c < T::kCols; ++c)
                        acc[r][c] = mfma_16x16x32(wb[c], __builtin_bit_cast(bf16x8, x), acc[r][c]);
                }
            }
        }

        k += min(left, 128);
        stage = stage + 1 == T::kStages ? 0 : stage + 1;
        if (++t == chunk_steps) {
            t = 0;
            if constexpr (SPLIT) {
#pragma unroll
                for (int r = 0; r < T::kRows; ++r)
#pragma unroll
                    for (int c = 0; c < T::kCols; ++c) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            tot[r][c][e] = chunk == 0 ? acc[r][c][e] : tot[r][c][e] + acc[r][c][e];
                        acc[r][c] = f32x4{0, 0, 0, 0};
                    }
                ++chunk;
            }
        }
    }

#pragma unroll
    for (int r = 0; r < T::kRows; ++r) {
        const int64_t m = m0 + wm * (TM / 2) + 16 * r + li;
#pragma unroll
        for (int c = 0; c < T::kCols; ++c) {
            const int64_t n = n0 + wn * (TN / 4) + 16 * c + 4 * g;
            const f32x4 v = SPLIT ? tot[SPLIT ? r : 0][c] : acc[r][c];
            if (m < p.M && n < p.N) {
                const uint32_t lo = f32_to_bf16_bits(v[0]) | (uint32_t)f32_to_bf16_bits(v[1]) << 16;
                const uint32_t hi = f32_to_bf16_bits(v[2]) | (uint32_t)f32_to_bf16_bits(v[3]) << 16;
                *reinterpret_cast<u32x2*>(p.y + m * p.ld_y + n) = u32x2{lo, hi};
            }
        }
    }
}

template <bool XMX, int TM, int TN, bool SPLIT>
hipError_t launch_tile(const Mx4LinearParams& p, hipStream_t st)
{
    const int64_t tiles = ((p.M + TM - 1) / TM) * ((p.N + TN - 1) / TN);
    hipLaunchKernelGGL((k_mx4_linear_tile<XMX, TM, TN, SPLIT>), dim3((unsigned)tiles), dim3(kTileWaves * 64), 0, st,
                       p);
    return hipGetLastError();
}

}  // namespace lora
