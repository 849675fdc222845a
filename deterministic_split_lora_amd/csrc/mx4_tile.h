// Large products with MX4 weights: a workgroup of eight waves owns a TM x TN
// tile of y, wave (wm, wn) of 2 x 4 a (TM / 2) x (TN / 4) part of it.  Included by
// mx4_linear.hip, which states the arithmetic.
//
// Steps of 128 k go through a ring of NS stages in LDS, filled by loads that
// write LDS themselves.  A wave reads its operands from LDS a part of a step
// ahead of their products (half of its rows, MX4 x; one block of 32, bf16 x), so
// that the matrix cores do not wait for LDS.  Once step j's last operands are in
// registers it waits until its own loads of stage j + 1 have landed and meets
// the others at the one barrier of the step: then all of stage j + 1 is there
// and stage j is read out, so the loads of step j + NS start into its place.
//
// Measured on MI355X, the product alone: bf16 x, 128 x 256 tiles, 4096 x 4096 x
// 14336 404 us (1.19 PFLOP/s; the matrix cores busy for 55% of the time, LDS for
// 21%); MX4 x, 256 x 256 tiles, 4096 x 8192 x 28672 559 us (3.4 PFLOP/s; 39%, and
// LDS 30%, a quarter of it bank conflicts).  With loads, LDS reads and barrier taken
// out of a copy, 309 and 361 us remained.
//
// LDS layout: 16-byte pieces of a row, in an order that depends on the row, so
// that the 16 rows a matrix-core operand reads at one k fall on different
// banks.  The order is applied to the global address each lane loads from
// (the loads fill LDS in lane order).  Scales: a row's scale bytes are contiguous
// over the chunks and are loaded once each, in order, kUnit bytes of every row at
// a time, into a ring of kScaleRing bytes a row.  kUnit is 16, and a step's four
// scales are read as one word, where rows are 16-byte aligned and chunks
// multiples of 128; otherwise it is 4 and they are read by the byte (the two
// products above then take 445 and 651 us; 4096 x 4096 x 14336 in 4 chunks 532
// instead of 421, with MX4 x 277 instead of 194).
#pragma once

#include "mx4.h"

namespace lora {

constexpr int kTileWaves = 8;
constexpr int kScaleRing = 32;               // scale bytes of a row in LDS: two aligned runs of 16

// What a workgroup does with the chunks of split_k.
enum TileMode {
    kOneChunk,                               // there is one
    kAllChunks,                              // sums them one after another
    kPartial                                 // computes one and stores its sum to the workspace
};

typedef __attribute__((address_space(3))) uint8_t lds_u8;

// Loads of 64 lanes straight to LDS, 16 (4) bytes a lane in lane order.  They
// write no registers, so the compiler need not know when they land; the kernel
// waits for them by count (wait_loads_and_meet).
// They take the LDS address from m0, which the compiler reserves for its own use;
// it is named as written all the same, so that no value of its is kept there over
// them, and the compiler's remark on that is off.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"

// From `base` plus a lane's offset to LDS at `to` + AT.
template <int AT>
__device__ __forceinline__ void load_to_lds16(const uint8_t* base, uint32_t offset, uint32_t to)
{
    asm volatile("s_add_u32 m0, %1, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %2" ::"v"(offset), "s"(to), "s"(base),
                 "n"(AT)
                 : "memory", "scc", "m0");
}

template <int BYTES>
__device__ __forceinline__ void load_scales_to_lds(const uint8_t* from, uint32_t to)
{
    if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(to)
                     : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(from), "s"(to)
                     : "memory", "m0");
}
#pragma clang diagnostic pop

// Waits until at most N of this wave's loads are outstanding and its LDS reads
// are done, then meets the workgroup.
template <int N>
__device__ __forceinline__ void wait_loads_and_meet()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// What piece number c of a row is combined with to give its place: rows of 64
// bytes (4 pieces) and of 256 bytes (16 pieces).  A 16-byte read of 64 lanes is
// served 16 lanes at a time, and these are lanes 0-3, 12-15 and 20-27, then 4-11,
// 16-19 and 28-31 (and the same of the upper half): with rows in the lanes of a
// group and pieces in the groups, each 16 then have 16 places mod 256 bytes.
__device__ __forceinline__ int swizzle4(int row)
{
    return (4 - (row >> 2)) & 3;
}

__device__ __forceinline__ int swizzle16(int row)
{
    return row & 15;
}

template <int N>
struct Flag {
    static constexpr int value = N;
};

// f(Flag<0>()) ... f(Flag<N - 1>())
template <int N, class F>
__device__ __forceinline__ void unrolled(F f)
{
    if constexpr (N > 0) {
        unrolled<N - 1>(f);
        f(Flag<N - 1>());
    }
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
    static_assert(kScaleWaves <= kTileWaves, "a wave loads the scales of at most 64 rows");
    static constexpr int kRows = TM / 32, kCols = TN / 64;   // 16 x 16 tiles of a wave
    static constexpr int kBudget = 160 * 1024 - kScaleRing * kScaleRows;
    // three stages where that lets two workgroups share a CU: 128 x 8192 x 8192 in
    // 4 chunks 28.9 us against 35.7 with four stages and one workgroup
    static constexpr int kMost = !XMX && TM == 64 ? 3 : 4;
    static constexpr int kStages = kBudget / kStage < kMost ? kBudget / kStage : kMost;
    static constexpr int kLds = kStages * kStage + kScaleRing * kScaleRows;
    static_assert(kXLoads >= 1 && kWLoads >= 1 && kStages >= 2, "tile too small or too large");
};

template <bool XMX, int TM, int TN, TileMode MODE, int kUnit>
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

    // Sources: load i of wave w fills 1024 bytes of a stage from (i * 8 + w) * 1024,
    // x's rows, then W's.  A lane's offset from its tile's first row, and the one
    // of a chunk's ragged last step, where blocks past the chunk's end load the
    // step's first block instead.
    const int rem = p.k_chunk % 128 / kMxBlock;                // blocks of that step, 0: there is none
    uint32_t xoff[2][T::kXLoads], woff[2][T::kWLoads];
#pragma unroll
    for (int i = 0; i < T::kXLoads; ++i) {
        constexpr int P = T::kXBytes / 16;
        const int piece = (i * kTileWaves + wave) * 64 + lane;
        const int row = piece / P;
        const int c = (piece % P) ^ (XMX ? swizzle4(row) : swizzle16(row));
        const uint32_t m = (uint32_t)(min(m0 + row, p.M - 1) - m0);
        xoff[0][i] = m * (uint32_t)(p.ld_x * (XMX ? 1 : 2)) + c * 16;
        xoff[1][i] = xoff[0][i] - ((XMX ? c : c >> 2) < rem ? 0 : XMX ? c * 16 : c / 4 * 64);
    }
#pragma unroll
    for (int i = 0; i < T::kWLoads; ++i) {
        const int piece = (i * kTileWaves + wave) * 64 + lane;
        const int row = piece / 4;
        const int c = (piece % 4) ^ swizzle4(row);
        const uint32_t n = (uint32_t)(min(n0 + row, p.N - 1) - n0);
        woff[0][i] = n * (uint32_t)p.ld_wq + c * 16;
        woff[1][i] = woff[0][i] - (c < rem ? 0 : c * 16);
    }
    const uint8_t* ssrc = p.ws;              // this lane's row of scales
    {
        const int row = wave * 64 + lane;
        if (row < TN)
            ssrc = p.ws + min(n0 + row, p.N - 1) * p.ld_ws;
        else if (XMX && row < TN + TM)
            ssrc = p.xs + min(m0 + row - TN, p.M - 1) * p.ld_xs;
    }

    const int chunk_steps = (p.k_chunk + 127) / 128, whole_steps = p.k_chunk / 128;
    const int chunks = MODE == kAllChunks ? p.split_k : 1;
    const int steps = chunk_steps * chunks;
    const uint32_t b_first = MODE == kPartial ? blockIdx.y * (uint32_t)(p.k_chunk / kMxBlock) : 0;
    const uint32_t last_unit = ((uint32_t)(p.k_chunk / kMxBlock * p.split_k) - 1) / kUnit;

    uint32_t units = b_first / kUnit;        // scale units whose loads have been started
    auto load_unit = [&]() {
        if (wave < T::kScaleWaves)
            load_scales_to_lds<kUnit>(ssrc + (uint64_t)units * kUnit,
                                      lds0 + T::kStages * T::kStage +
                                          (units % (kScaleRing / kUnit) * T::kScaleRows + wave * 64) * kUnit);
        ++units;
    };
    // loads of one step into the stage at `slot`; ld_* is the step whose loads
    // come next
    uint32_t slot = 0, ld_block = b_first;
    int ld_t = 0;
    const uint8_t* xbase = static_cast<const uint8_t*>(p.x) + m0 * p.ld_x * (XMX ? 1 : 2) +
                           (uint64_t)b_first * (XMX ? 16 : 64);
    const uint8_t* wbase = p.wq + n0 * p.ld_wq + (uint64_t)b_first * 16;
    constexpr int kStepLoads = T::kXLoads + T::kWLoads;
    // load i of kStepLoads of the step, into the stage at `at`
    auto load_piece = [&](auto i, uint32_t at) {
        constexpr int I = decltype(i)::value;
        const uint32_t to = lds0 + at + wave * 1024;
        const bool ragged = ld_t == whole_steps;
        if constexpr (I < T::kXLoads)
            load_to_lds16<I * kTileWaves * 1024>(xbase, ragged ? xoff[1][I] : xoff[0][I], to);
        else
            load_to_lds16<I * kTileWaves * 1024>(wbase, ragged ? woff[1][I - T::kXLoads] : woff[0][I - T::kXLoads], to);
    };
    // after the last of them
    auto end_loads = [&]() {
        // a step's four scale bytes end at most one unit past the step before's
        if (units <= min((ld_block + 3) / kUnit, last_unit))
            load_unit();
        const int blocks = ld_t == whole_steps ? rem : 4;
        ld_block += blocks;
        xbase += blocks * (XMX ? 16 : 64);
        wbase += blocks * 16;
        ld_t = ld_t + 1 == chunk_steps ? 0 : ld_t + 1;
    };
    auto next_slot = [&]() { slot = slot + T::kStage == T::kStages * T::kStage ? 0 : slot + T::kStage; };

    constexpr bool SPLIT = MODE == kAllChunks;
    f32x4 acc[T::kRows][T::kCols], tot[SPLIT ? T::kRows : 1][T::kCols];
#pragma unroll
    for (int r = 0; r < T::kRows; ++r)
#pragma unroll
        for (int c = 0; c < T::kCols; ++c)
            acc[r][c] = f32x4{0, 0, 0, 0};

    // a chunk that starts inside a unit may need two for its first step
    if (MODE == kPartial && units < last_unit)
        load_unit();
    for (int j = 0; j < T::kStages; ++j) {
        if (j < steps) {
            unrolled<kStepLoads>([&](auto i) { load_piece(i, slot); });
            end_loads();
        }
        next_slot();
    }
    // Of the loads in flight, those of later steps may stay so.  Scale units, which
    // not every step has, are not counted among them.
    if (T::kStages <= steps)
        wait_loads_and_meet<(T::kStages - 1) * kStepLoads>();
    else
        wait_loads_and_meet<0>();

    // On to the next step, once stage j + 1 has landed everywhere and stage j is
    // read out: its place, the value, takes the loads of step j + NS.  What is read
    // from here on is stage j + 1, at `slot`, whose first block is rd_block.
    uint32_t rd_block = b_first;
    auto next_step = [&](auto tail, auto drain) {
        wait_loads_and_meet<decltype(drain)::value ? 0 : (T::kStages - 2) * kStepLoads>();
        const uint32_t freed = slot;
        next_slot();
        rd_block += decltype(tail)::value ? rem : 4;
        return freed;
    };
    // the scale of one block, of row 0 (rows are kUnit bytes apart)
    auto scale_bytes = [&](uint32_t block) {
        return lds + T::kStages * T::kStage + block / kUnit % (kScaleRing / kUnit) * (T::kScaleRows * kUnit) +
               block % kUnit;
    };
    const int wrow = wn * (TN / 4) + li, xrow = wm * (TM / 2) + li;
    // rows 16 apart have the same order of pieces
    const uint32_t wat = T::kXStage + wrow * 64, wsw = swizzle4(wrow);
    const uint32_t xat = xrow * T::kXBytes, xsw = XMX ? swizzle4(xrow) : swizzle16(xrow);

    // what a wave has in registers between steps
    constexpr int kHalf = T::kRows / 2;
    MxOperand w[T::kCols], xa[kHalf], xb[kHalf];               // MX4 x
    u32x4 wq[T::kCols], even[T::kRows], odd[T::kRows];         // bf16 x
    uint32_t ws4[T::kCols];
    bf16x8 wb[2][T::kCols];

    auto read_w = [&](int c) {
        w[c].q = *reinterpret_cast<const u32x4*>(lds + slot + wat + (g ^ wsw) * 16 + c * 1024);
        w[c].s = scale_bytes(rd_block + g)[(wrow + 16 * c) * kUnit];
    };
    auto read_x = [&](MxOperand (&x)[kHalf], int first) {
#pragma unroll
        for (int r = 0; r < kHalf; ++r) {
            x[r].q = *reinterpret_cast<const u32x4*>(lds + slot + xat + (g ^ xsw) * 16 +
                                                     (first + r) * 1024);
            x[r].s = scale_bytes(rd_block + g)[(TN + xrow + 16 * (first + r)) * kUnit];
        }
    };
    // bf16 x: W's codes of a step, block g in lane group g, and its scales
    auto read_codes = [&](u32x4 (&q)[T::kCols], uint32_t (&s)[T::kCols]) {
#pragma unroll
        for (int c = 0; c < T::kCols; ++c) {
            q[c] = *reinterpret_cast<const u32x4*>(lds + slot + wat + (g ^ wsw) * 16 + c * 1024);
            const int row = (wrow + 16 * c) * kUnit;
            if constexpr (kUnit == 16) {
                s[c] = *reinterpret_cast<const uint32_t*>(scale_bytes(rd_block) + row);
            } else {
                s[c] = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[c] |= (uint32_t)scale_bytes(rd_block + e)[row] << (8 * e);
            }
        }
    };
    auto read_block = [&](u32x4 (&x)[T::kRows], uint32_t s) {
#pragma unroll
        for (int r = 0; r < T::kRows; ++r)
            x[r] = *reinterpret_cast<const u32x4*>(lds + slot + xat + ((4 * s + g) ^ xsw) * 16 +
                                                   r * 4096);
    };
    // blocks past the chunk's end enter as zeros
    auto clear = [&](auto& o) {
        for (auto& v : o)
            if (g >= rem)
                v = MxOperand{u32x4{0, 0, 0, 0}, 127};
    };
    auto convert = [&](bf16x8 (&to)[T::kCols], int s) {
#pragma unroll
        for (int c = 0; c < T::kCols; ++c)
            to[c] = mx4_to_bf16(wq[c][s], mx_scale_f32((ws4[c] >> (8 * s)) & 255u));
    };
    auto row_products = [&](bf16x8 (&wv)[T::kCols], u32x4 (&x)[T::kRows], int r) {
#pragma unroll
        for (int c = 0; c < T::kCols; ++c)
            acc[r][c] = mfma_16x16x32(wv[c], __builtin_bit_cast(bf16x8, x[r]), acc[r][c]);
    };
    // the products of block s and, between them (the vector unit is free while a
    // matrix instruction runs), the conversion of block s + 1's W, if there are
    // registers for both
    constexpr bool kBetween = !SPLIT || T::kRows <= 2;
    auto products = [&](u32x4 (&x)[T::kRows], auto s) {
        constexpr int S0 = decltype(s)::value;
        if constexpr (!kBetween)
            convert(wb[0], S0);
#pragma unroll
        for (int r = 0; r < T::kRows; ++r)
            row_products(wb[kBetween ? S0 % 2 : 0], x, r);
        if constexpr (kBetween) {
            convert(wb[(S0 + 1) % 2], S0 + 1);
#pragma unroll
            for (int i = 0; i < T::kRows * T::kCols; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);              // matrix
                __builtin_amdgcn_sched_group_barrier(0x002, 6 / T::kRows + 1, 0);   // vector
            }
        }
    };
    auto take_codes = [&](u32x4 (&q)[T::kCols], uint32_t (&s)[T::kCols]) {
#pragma unroll
        for (int c = 0; c < T::kCols; ++c) {
            wq[c] = q[c];
            ws4[c] = s[c];
            transpose_groups(wq[c]);
        }
    };
    // One step.  The order of reads, loads and products written here is the order
    // they run in (what a chunk's ragged last step does more is branched around).
    // drain: no more loads start, and those in flight are no longer NS steps'.
    auto step = [&](auto tail, auto drain) {
        constexpr bool TAIL = decltype(tail)::value != 0, DRAIN = decltype(drain)::value != 0;
        if constexpr (XMX) {
            read_x(xb, kHalf);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (TAIL) {
                clear(w);
                clear(xa);
            }
#pragma unroll
            for (int c = 0; c < T::kCols; ++c)
#pragma unroll
                for (int r = 0; r < kHalf; ++r)
                    acc[r][c] = mfma_mx4(w[c], xa[r], acc[r][c]);
            __builtin_amdgcn_sched_barrier(0);
            const uint32_t freed = next_step(tail, drain);
            if constexpr (!DRAIN) {
                unrolled<kStepLoads>([&](auto i) { load_piece(i, freed); });
                end_loads();
            }
            read_x(xa, 0);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (TAIL)
                clear(xb);
            // a column's W is read for the next step as soon as its last product
            // has started
#pragma unroll
            for (int c = 0; c < T::kCols; ++c) {
#pragma unroll
                for (int r = 0; r < kHalf; ++r)
                    acc[kHalf + r][c] = mfma_mx4(w[c], xb[r], acc[kHalf + r][c]);
                __builtin_amdgcn_sched_barrier(0);
                read_w(c);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            read_block(odd, 1);
            __builtin_amdgcn_sched_barrier(0);
            products(even, Flag<0>());
            __builtin_amdgcn_sched_barrier(0);
            read_block(even, 2);
            __builtin_amdgcn_sched_barrier(0);
            if (!TAIL || rem > 1)
                products(odd, Flag<1>());
            __builtin_amdgcn_sched_barrier(0);
            read_block(odd, 3);
            __builtin_amdgcn_sched_barrier(0);
            if (!TAIL || rem > 2)
                products(even, Flag<2>());
            __builtin_amdgcn_sched_barrier(0);
            const uint32_t freed = next_step(tail, drain);
            u32x4 q[T::kCols];
            uint32_t s4[T::kCols];
            read_codes(q, s4);
            read_block(even, 0);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (!TAIL && !kBetween)
                convert(wb[1], 3);
            unrolled<T::kRows>([&](auto r) {
                if constexpr (!TAIL)
                    row_products(wb[1], odd, r.value);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (!DRAIN)
                    unrolled<kStepLoads>([&](auto i) {
                        if constexpr (i.value * T::kRows / kStepLoads == r.value)
                            load_piece(i, freed);
                    });
                __builtin_amdgcn_sched_barrier(0);
            });
            if constexpr (!DRAIN)
                end_loads();
            take_codes(q, s4);
            if constexpr (kBetween)
                convert(wb[0], 0);
        }
    };

    if constexpr (XMX) {
#pragma unroll
        for (int c = 0; c < T::kCols; ++c)
            read_w(c);
        read_x(xa, 0);
    } else {
        u32x4 q[T::kCols];
        uint32_t s4[T::kCols];
        read_codes(q, s4);
        take_codes(q, s4);
        convert(wb[0], 0);
        read_block(even, 0);
    }
    int full = steps - T::kStages;           // steps that start loads
    for (int chunk = 0; chunk < chunks; ++chunk) {
        const int n = max(0, min(full, whole_steps));
        for (int t = 0; t < n; ++t)
            step(Flag<0>(), Flag<0>());
        for (int t = n; t < whole_steps; ++t)
            step(Flag<0>(), Flag<1>());
        // several chunks whose scales come by the word are multiples of 128
        if constexpr (MODE == kOneChunk || kUnit == 4)
            if (rem) {
                if (full >= chunk_steps)
                    step(Flag<1>(), Flag<0>());
                else
                    step(Flag<1>(), Flag<1>());
            }
        full -= chunk_steps;
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
        }
    }

#pragma unroll
    for (int r = 0; r < T::kRows; ++r) {
        const int64_t m = m0 + wm * (TM / 2) + 16 * r + li;
#pragma unroll
        for (int c = 0; c < T::kCols; ++c) {
            const int64_t n = n0 + wn * (TN / 4) + 16 * c + 4 * g;
            const f32x4 v = SPLIT ? tot[SPLIT ? r : 0][c] : acc[r][c];
            if (m >= p.M || n >= p.N)
                continue;
            if constexpr (MODE == kPartial) {
                *reinterpret_cast<f32x4*>(p.partial + ((int64_t)blockIdx.y * p.M + m) * p.N + n) = v;
            } else {
                const uint32_t lo = f32_to_bf16_bits(v[0]) | (uint32_t)f32_to_bf16_bits(v[1]) << 16;
                const uint32_t hi = f32_to_bf16_bits(v[2]) | (uint32_t)f32_to_bf16_bits(v[3]) << 16;
                *reinterpret_cast<u32x2*>(p.y + m * p.ld_y + n) = u32x2{lo, hi};
            }
        }
    }
}

template <bool XMX, int TM, int TN, TileMode MODE, int kUnit>
hipError_t launch_tile_unit(const Mx4LinearParams& p, hipStream_t st)
{
    const int64_t tiles = ((p.M + TM - 1) / TM) * ((p.N + TN - 1) / TN);
    const dim3 grid((unsigned)tiles, MODE == kPartial ? (unsigned)p.split_k : 1u), block(kTileWaves * 64);
    hipLaunchKernelGGL((k_mx4_linear_tile<XMX, TM, TN, MODE, kUnit>), grid, block, 0, st, p);
    return hipGetLastError();
}

// By the bytes of scales that are loaded together (scale_unit).
template <bool XMX, int TM, int TN, TileMode MODE>
hipError_t launch_tile(const Mx4LinearParams& p, int unit, hipStream_t st)
{
    return unit == 16 ? launch_tile_unit<XMX, TM, TN, MODE, 16>(p, st) : launch_tile_unit<XMX, TM, TN, MODE, 4>(p, st);
}

}  // namespace lora
