// Products with MX4 weights:  y = x W^T  for bf16 x and for MX4 x.
//
// Arithmetic, the same in every kernel of this file so that schedules agree
// bit for bit.  K is cut into split_k chunks.  A chunk's sum is one chain of
// matrix-core steps in ascending k, from zero, in fp32.  Chunk sums are added in
// ascending order and the total is rounded once to bf16.
//   bf16 x: a step is one V_MFMA_F32_16X16X32_BF16 over a block of 32, lane
//     group g (li = lane % 16, g = lane / 16) holding elements 8g .. 8g+7 of it;
//     W's codes are converted to bf16 (exactly) on the way.
//   MX4 x: a step is one V_MFMA_SCALE_F32_16X16X128_F8F6F4 over four blocks, lane
//     group g holding block g; both operands' codes and scales enter as they are
//     stored.  Blocks past the chunk's end enter as zeros.
// The "row" operand is W, so a lane's accumulator holds four consecutive output
// columns of one token.
#include "mx4_tile.h"

namespace lora {

namespace {

constexpr int kStepK = 128;                  // k of one step's loads
constexpr int kScaleSteps = 16;              // steps whose scales are loaded together
constexpr int kRowsThreads = 1024;           // at most, of a workgroup of few rows: 16 chunks

__device__ __forceinline__ MxOperand mx_operand(u32x4 q, uint32_t s, bool ok)
{
    return ok ? MxOperand{q, s} : MxOperand{u32x4{0, 0, 0, 0}, 127};
}

// Four words at a word-aligned address.
typedef uint32_t u32x4_word_aligned __attribute__((ext_vector_type(4), aligned(4)));

// A wave-uniform base and a lane's 32-bit offset from it.
template <class T>
__device__ __forceinline__ T load_at(const uint8_t* base, uint32_t offset)
{
    typedef __attribute__((address_space(1))) const uint8_t global_u8;
    typedef __attribute__((address_space(1))) const T global_t;
    return *(global_t*)((global_u8*)base + offset);
}

// Few tokens: a workgroup owns 16 RT tokens x 16 columns (times the column
// groups), its wave (group, s) the chain of chunk s; the chains meet in LDS.
// Bound by how many loads are in flight: W's come D steps of 128 k ahead, those
// of x (which the other workgroups read too, so that it is near) DX ahead, and a
// wave never meets the others before its chain is done.  Every load is 64
// contiguous bytes a row: 16 bytes a lane, x of one block, W of four blocks, one a
// lane group, whose words the lane groups then exchange (bf16 x).  So do the
// scales, 64 blocks at a time, which a wave keeps in its part of LDS: read four
// bytes a row and step they would come from L2 every time, a line each.  Measured
// on MI355X: 1 x 4096 x 6144 in 8 chunks 6.7 us, MX4 x 16 x 8192 x 8192 in 8
// chunks 10.8 us (36 MB, 3.4 TB/s).
template <bool XMX, int RT, int D, int DX>
__global__ void __launch_bounds__(kRowsThreads) k_mx4_linear_rows(Mx4LinearParams p, int groups)
{
    static_assert(D % DX == 0 && kScaleSteps % D == 0, "the rings turn together");
    extern __shared__ float lds[];
    const int lane = threadIdx.x & 63;
    const int li = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int S = p.split_k;
    const int chunk = wave % S, group = wave / S;             // wave = group * S + chunk
    const int64_t n0 = ((int64_t)blockIdx.x * groups + group) * 16;
    const int64_t m0 = (int64_t)blockIdx.y * (16 * RT);

    f32x4 acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        acc[r] = f32x4{0, 0, 0, 0};

    const int64_t kc = (int64_t)chunk * p.k_chunk;
    const int steps = (p.k_chunk + kStepK - 1) / kStepK, last = steps - 1;
    const int rem = (p.k_chunk - last * kStepK) / kMxBlock;    // blocks of the last step
    // in the last step a lane group without a block reads the step's first one
    const uint32_t back = g < rem ? 0u : 16u * g;

    // first row of the tiles (a group past the last column repeats the last row)
    const int64_t nb = min(n0, p.N - 1);
    const uint8_t* wq0 = p.wq + nb * p.ld_wq + kc / 2;
    const uint8_t* ws0 = p.ws + nb * p.ld_ws;
    const uint8_t* xq0 = static_cast<const uint8_t*>(p.x) + (XMX ? m0 * p.ld_x + kc / 2 : 2 * (m0 * p.ld_x + kc));
    const uint8_t* xs0 = XMX ? p.xs + m0 * p.ld_xs : nullptr;
    const int sb0 = (int)(kc / kMxBlock);                      // the chunk's first scale byte
    const int last_word = (p.k_chunk / kMxBlock * S - 1) >> 2;
    const int64_t n_li = min(nb + li, p.N - 1) - nb;
    const uint32_t wo = (uint32_t)(n_li * p.ld_wq) + 16 * g, wso = (uint32_t)(n_li * p.ld_ws);
    uint32_t xo[RT], xso[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int64_t m = min(m0 + 16 * r + li, p.M - 1) - m0;
        xo[r] = (uint32_t)(m * p.ld_x) * (XMX ? 1 : 2) + 16 * g;
        xso[r] = XMX ? (uint32_t)(m * p.ld_xs) : 0;
    }

    u32x4 w[D], x[DX][RT][XMX ? 1 : 4];

    // This wave's scales, W's tile first: [tile][16 rows][kScaleSteps words], a
    // word the four blocks of a step.
    constexpr int kTile = 256, kScaleTiles = XMX ? 1 + RT : 1;
    constexpr int kWaveLds = (RT > kScaleTiles ? RT : kScaleTiles) * kTile;
    uint32_t* sc = reinterpret_cast<uint32_t*>(lds) + wave * kWaveLds;
    const int shift = 8 * (sb0 & 3);
    // Loaded a run of steps ahead and put into LDS when the run begins: a load that
    // is waited for makes all earlier ones be waited for, so it has to be older
    // than W's loads in flight (MX4 x, 1 x 4096 x 6144: 6.1 us; loaded where they
    // are put, 6.4).
    uint32_t sv[kScaleTiles][5];
    auto load_scales = [&](int j) {
        // lane group g has words 4g .. 4g+3 of the rows, if there are so many steps
        if (j + 4 * g >= steps)
            return;
        const int word = ((sb0 + 4 * j) >> 2) + 4 * g;
        const bool inside = word + 4 <= last_word;
#pragma unroll
        for (int i = 0; i < kScaleTiles; ++i) {
            const uint8_t* s0 = i == 0 ? ws0 : xs0;
            const uint32_t off = i == 0 ? wso : xso[i == 0 ? 0 : i - 1];
            if (inside) {
                const u32x4 q = load_at<u32x4_word_aligned>(s0, off + 4 * word);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sv[i][e] = q[e];
                sv[i][4] = shift ? load_at<uint32_t>(s0, off + 4 * word + 16) : 0;
            } else {
#pragma unroll
                for (int e = 0; e < 5; ++e)
                    sv[i][e] = load_at<uint32_t>(s0, off + 4 * min(word + e, last_word));
            }
        }
    };
    auto put_scales = [&]() {
#pragma unroll
        for (int i = 0; i < kScaleTiles; ++i) {
            u32x4 q;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                q[e] = __builtin_amdgcn_alignbit(sv[i][e + 1], sv[i][e], shift);
            *reinterpret_cast<u32x4*>(sc + i * kTile + li * kScaleSteps + 4 * g) = q;
        }
    };
    auto load_w = [&](u32x4& b, int j) { b = load_at<u32x4>(wq0 + j * 64, wo - (j == last ? back : 0)); };
    auto load_x = [&](u32x4 (&b)[RT][XMX ? 1 : 4], int j) {
        const uint32_t less = j == last ? back : 0;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            if constexpr (XMX) {
                b[r][0] = load_at<u32x4>(xq0 + j * 64, xo[r] - less);
            } else {
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    b[r][s] = load_at<u32x4>(xq0 + j * 256 + (j < last || s < rem ? 64 * s : 0), xo[r]);
            }
        }
    };
    auto scales = [&](int tile, int j) { return sc[tile * kTile + li * kScaleSteps + j % kScaleSteps]; };
    auto multiply = [&](u32x4& a, u32x4 (&b)[RT][XMX ? 1 : 4], int j) {
        if constexpr (XMX) {
            const bool ok = j < last || g < rem;
            const MxOperand wm = mx_operand(a, scales(0, j) >> (8 * g), ok);
#pragma unroll
            for (int r = 0; r < RT; ++r)
                acc[r] = mfma_mx4(wm, mx_operand(b[r][0], scales(1 + r, j) >> (8 * g), ok), acc[r]);
        } else {
            transpose_groups(a);
            const uint32_t s4 = scales(0, j);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (j == last && s >= rem)
                    break;
                const bf16x8 wb = mx4_to_bf16(a[s], mx_scale_f32((s4 >> (8 * s)) & 255u));
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    acc[r] = mfma_16x16x32(wb, __builtin_bit_cast(bf16x8, b[r][s]), acc[r]);
            }
        }
    };

    load_scales(0);
    // loads past the last step repeat it, so that how many are in flight is
    // known wherever one is waited for
#pragma unroll
    for (int d = 0; d < D; ++d) {
        load_w(w[d], min(d, last));
        if (d < DX)
            load_x(x[d], min(d, last));
    }
    int j = 0;
    for (; j + D < steps; j += D) {
        if (j % kScaleSteps == 0) {
            put_scales();
            load_scales(j + kScaleSteps);
        }
#pragma unroll
        for (int d = 0; d < D; ++d) {
            multiply(w[d], x[d % DX], j + d);
            load_w(w[d], min(j + D + d, last));
            load_x(x[d % DX], min(j + DX + d, last));
        }
    }
    if (j % kScaleSteps == 0)
        put_scales();
#pragma unroll
    for (int d = 0; d < D; ++d) {
        if (j + d < steps)
            multiply(w[d], x[d % DX], j + d);
        if (d + DX < D)
            load_x(x[d % DX], min(j + DX + d, last));
    }

    // chains to LDS: [group][chunk][r][lane][4], then a thread adds its
    // output's chunks in ascending order
    float* mine = lds + wave * kWaveLds;     // wave = group * S + chunk
#pragma unroll
    for (int r = 0; r < RT; ++r)
        *reinterpret_cast<f32x4*>(mine + r * kTile + lane * 4) = acc[r];
    __syncthreads();
    const int quads = groups * RT * 64;
    for (int i = threadIdx.x; i < quads; i += blockDim.x) {
        const int l = i & 63, tile = (i >> 6) % RT, grp = (i >> 6) / RT;
        const float* src = lds + grp * S * kWaveLds + tile * kTile + l * 4;
        f32x4 sum = *reinterpret_cast<const f32x4*>(src);
        for (int s = 1; s < S; ++s) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(src + s * kWaveLds);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum[e] += v[e];
        }
        const int64_t m = m0 + 16 * tile + (l & 15);
        const int64_t n = ((int64_t)blockIdx.x * groups + grp) * 16 + 4 * (l >> 4);
        if (m < p.M && n < p.N) {
            const uint32_t lo = f32_to_bf16_bits(sum[0]) | (uint32_t)f32_to_bf16_bits(sum[1]) << 16;
            const uint32_t hi = f32_to_bf16_bits(sum[2]) | (uint32_t)f32_to_bf16_bits(sum[3]) << 16;
            *reinterpret_cast<u32x2*>(p.y + m * p.ld_y + n) = u32x2{lo, hi};
        }
    }
}

template <bool XMX, int RT, int D, int DX>
hipError_t launch_rows(const Mx4LinearParams& p, hipStream_t st)
{
    const int groups = p.split_k < 4 ? 4 / p.split_k : 1;
    const int64_t cols = 16 * groups;
    const dim3 grid((unsigned)((p.N + cols - 1) / cols), (unsigned)((p.M + 16 * RT - 1) / (16 * RT)));
    const int tiles = XMX ? 1 + RT : RT;
    const size_t lds = (size_t)groups * p.split_k * tiles * 1024;
    hipLaunchKernelGGL((k_mx4_linear_rows<XMX, RT, D, DX>), grid, dim3(64 * groups * p.split_k), lds, st, p, groups);
    return hipGetLastError();
}

// Second launch of the split schedule: the chunks' sums, added in ascending
// order, eight columns a thread.
__global__ void __launch_bounds__(256) k_mx4_linear_join(Mx4LinearParams p)
{
    const int64_t per_row = p.N / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = i / per_row, n = (i - m * per_row) * 8;
    if (m >= p.M)
        return;
    const float* src = p.partial + m * p.N + n;
    f32x4 a = *reinterpret_cast<const f32x4*>(src), b = *reinterpret_cast<const f32x4*>(src + 4);
    for (int s = 1; s < p.split_k; ++s) {
        src += p.M * p.N;
        const f32x4 u = *reinterpret_cast<const f32x4*>(src), v = *reinterpret_cast<const f32x4*>(src + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            a[e] += u[e];
            b[e] += v[e];
        }
    }
    u16x8 out;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        out[e] = f32_to_bf16_bits(a[e]);
        out[4 + e] = f32_to_bf16_bits(b[e]);
    }
    *reinterpret_cast<u16x8*>(p.y + m * p.ld_y + n) = out;
}

template <bool XMX, int TM, int TN>
hipError_t launch_split_tile(const Mx4LinearParams& p, int unit, hipStream_t st)
{
    const hipError_t e = launch_tile<XMX, TM, TN, kPartial>(p, unit, st);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(k_mx4_linear_join, dim3((unsigned)((p.M * (p.N / 8) + 255) / 256)), dim3(256), 0, st, p);
    return hipGetLastError();
}

// The bytes of a row's scales that the tile kernel loads together: 16 where rows
// are aligned to them and every chunk starts at a word of scales, otherwise 4.
int scale_unit(const Mx4LinearParams& p, bool mx)
{
    const uintptr_t rows = reinterpret_cast<uintptr_t>(p.ws) | (uintptr_t)p.ld_ws |
                           (mx ? reinterpret_cast<uintptr_t>(p.xs) | (uintptr_t)p.ld_xs : 0);
    return rows % 16 == 0 && (p.split_k == 1 || p.k_chunk % 128 == 0) ? 16 : 4;
}

// Which kernel a call takes: the one of least estimated time.  The estimates, in
// ns, come from measurements on MI355X:
//   rows    a chain's steps of 128 k follow one another, and a CU shares its waves'
//           loads: by tiles of 16 tokens, one step alone / per CU
//   tiles   a workgroup a CU (two of the small tiles), steps of 128 k one after
//           another; a step costs more where scales come 4 bytes at a time
//   split   the small tiles, a chunk a workgroup, then the joining launch, which
//           moves 8 bytes an output and chunk
// e.g. bf16 x, 200 x 4096 x 6144, split_k 4: 64 x 128 tiles 24.9 us, split 26.8, rows
// 85, 128 x 256 tiles 54; 33 x 14336 x 4096, split_k 8: split 17.5, rows 35.2, 64 x
// 128 tiles 68; with 4-byte scales 2048 x 11008 x 6144, split_k 4: 128 x 128 tiles
// 290, 64 x 128 338, split 413.
// Over 294 calls (K 2720 .. 14336, M 33 .. 4096, N 4096 .. 8192, split_k 1 .. 8,
// either unit of scales, either x) the kernel chosen took 0.4% longer than the
// fastest one on average and 12% at most, and nine of ten estimates of it were
// within 28%.
enum Schedule { kRows, kSplit, kTileSmall, kTileMiddle, kTileLarge };

constexpr int64_t kCus = 256;

int64_t ceil_div(int64_t a, int64_t b)
{
    return (a + b - 1) / b;
}

Schedule schedule_for(int64_t M, int64_t N, int32_t k_chunk, int32_t split_k, bool mx, int unit)
{
    const int64_t chunk_steps = ceil_div(k_chunk, kStepK), steps = chunk_steps * split_k;
    const bool narrow = unit == 4;
    // rows: blocks of up to 64 tokens
    const int64_t alone[2][4] = {{600, 1050, 1600, 2250}, {300, 430, 680, 680}};
    const int64_t shared[2][4] = {{180, 300, 400, 540}, {100, 125, 190, 190}};
    const int64_t tiles = M < 64 ? ceil_div(M, 16) : 4;
    const int64_t waves = ceil_div(M, 64) * ceil_div(N, 16) * split_k;
    const int64_t one = chunk_steps * alone[mx][tiles - 1];
    const int64_t all = ceil_div(waves, kCus) * chunk_steps * shared[mx][tiles - 1];
    Schedule best = kRows;
    int64_t least = 2000 + (one > all ? one : all);
    auto consider = [&](Schedule s, int64_t ns) {
        if (ns < least) {
            least = ns;
            best = s;
        }
    };
    auto rounds = [&](int64_t tm, int64_t tn) { return ceil_div(ceil_div(M, tm) * ceil_div(N, tn), kCus); };
    // the small tiles: two of them share a CU
    const int64_t small_tiles = ceil_div(M, mx ? 128 : 64) * ceil_div(N, 128);
    auto small = [&](int64_t copies) {
        const int64_t n = small_tiles * copies, rest = n % (2 * kCus);
        const int64_t alone1 = mx ? 520 : 770, paired = mx ? (narrow ? 1250 : 900) : (narrow ? 1320 : 1100);
        return n / (2 * kCus) * paired + (rest > kCus ? paired : rest > 0 ? alone1 : 0);
    };
    consider(kTileSmall, 2000 + small(1) * steps);
    const int64_t middle = mx ? (narrow ? 900 : 790) : narrow ? 1700 : split_k > 1 ? 1750 : 1650;
    if (split_k == 1 || !narrow)
        consider(kTileMiddle, 2000 + rounds(128, 256) * steps * middle);
    else if (!mx)                            // the middle tile is 128 x 128 then
        consider(kTileMiddle, 2000 + rounds(128, 128) * steps * 1100);
    if (mx && split_k == 1)
        consider(kTileLarge, 2000 + rounds(256, 256) * steps * (narrow ? 1250 : 1200));
    if (split_k > 1)
        consider(kSplit, 6500 + small(split_k) * chunk_steps + M * N * split_k * 8 / 4500);
    return best;
}

}  // namespace

int64_t mx4_linear_workspace(int64_t M, int64_t N, int32_t k_chunk, int32_t split_k)
{
    for (int i = 0; i < 4; ++i)
        if (schedule_for(M, N, k_chunk, split_k, i & 1, i & 2 ? 16 : 4) == kSplit)
            return M * N * split_k * (int64_t)sizeof(float);
    return 0;
}

hipError_t launch_mx4_linear(const Mx4LinearParams& p, bool x_is_mx4, hipStream_t st)
{
    const bool one = p.split_k == 1;
    const int unit = scale_unit(p, x_is_mx4);
    switch (schedule_for(p.M, p.N, p.k_chunk, p.split_k, x_is_mx4, unit)) {
    case kSplit:
        return x_is_mx4 ? launch_split_tile<true, 128, 128>(p, unit, st)
                        : launch_split_tile<false, 64, 128>(p, unit, st);
    case kTileSmall:
        if (x_is_mx4)
            return one ? launch_tile<true, 128, 128, kOneChunk>(p, unit, st)
                       : launch_tile<true, 128, 128, kAllChunks>(p, unit, st);
        return one ? launch_tile<false, 64, 128, kOneChunk>(p, unit, st)
                   : launch_tile<false, 64, 128, kAllChunks>(p, unit, st);
    case kTileMiddle:
        if (one)
            return x_is_mx4 ? launch_tile<true, 128, 256, kOneChunk>(p, unit, st)
                            : launch_tile<false, 128, 256, kOneChunk>(p, unit, st);
        // totals beside the sums and ragged chunks: 256 columns have no registers left
        // (for MX4 x, 128 are the small tile)
        if (unit == 4)
            return launch_tile_unit<false, 128, 128, kAllChunks, 4>(p, st);
        return x_is_mx4 ? launch_tile_unit<true, 128, 256, kAllChunks, 16>(p, st)
                        : launch_tile_unit<false, 128, 256, kAllChunks, 16>(p, st);
    case kTileLarge:
        return launch_tile<true, 256, 256, kOneChunk>(p, unit, st);
    default:
        break;
    }
    if (x_is_mx4) {
        // eight steps ahead where a chain has more than four: 16 x 8192 x 8192 in 8
        // chunks 11.9 us against 15.1; in 16 chunks of four steps 13.7 against 19.4
        if (p.M <= 16)
            return p.k_chunk > 4 * kStepK ? launch_rows<true, 1, 8, 4>(p, st)
                                          : launch_rows<true, 1, 4, 4>(p, st);
        if (p.M <= 32)
            return launch_rows<true, 2, 4, 2>(p, st);
        return launch_rows<true, 4, 2, 2>(p, st);
    }
    if (p.M <= 16)
        return launch_rows<false, 1, 4, 2>(p, st);
    if (p.M <= 32)
        return launch_rows<false, 2, 4, 2>(p, st);
    if (p.M <= 48)
        return launch_rows<false, 3, 4, 1>(p, st);
    return launch_rows<false, 4, 4, 1>(p, st);
}

}  // namespace lora
