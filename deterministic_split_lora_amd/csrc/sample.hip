// One token per row of logits: temperature, top-k, top-p, min-p and a draw
// from a given random number.
//
// A logit l of weight  w = rint(2^31 exp((l - max) / T))  is a whole number, so
// every sum below is a 64-bit integer sum: exact, hence the same in any order,
// for any work split and next to any other rows.
//
// Tokens are ordered by (logit descending, index ascending).  Each of top-k,
// top-p and min-p keeps a prefix of that order, so their intersection is a
// prefix too and is given by its last element.
//
// One workgroup owns a row: it reads it once for the maximum and once or twice
// more for what its settings need.  A batch is bound by memory, which every pass
// reads again.  Measured on MI355X, 256 x 128259 fp32 and the bytes read by the
// counters: greedy 22 us (132 MB), no cuts 46 (270 MB), top-k 50 47 (264 MB), min-p
// 67, top-p 75-77 (402 MB, 5.2 TB/s; the vector unit is busy for 57% of the time
// there and for 47% without cuts).  A row alone waits for one CU's passes: 1 x
// 32000 bf16 4.9 greedy, 11 no cuts, 13.5 top-k 50, 16 min-p, 19 top-p; 1 x 128259
// fp32 11, 26, 21, 40, 51.
//
// Where a list of the usual paths overflows, sample_any takes the row, in six
// to eleven more passes: 256 x 128259 447-560 us, 1 x 128259 305-424, 1 x 32000 97-130.
// That is so
//   with top-k, where more than kFew logits are no less than the k-th largest of
//     the threads' maxima: of independent logits from a k of 650 to 700 on (at 400
//     comparing the gathered ones takes 142 us already, at 600 231); of logits that
//     fall with the index, as in vocabularies ordered by frequency, for 200; and for
//     any k where more than kFew are left beside masks of a finite value that cover
//     all logits of some thread (3000 beside -1e9); also where k is above the number
//     of threads with logits, V / 8 (bf16) or V / 4, and V above kFew;
//   with top-p or min-p, where the bin that is cut holds more than kList logits:
//     flat rows (normal logits of unit spread, 128259 of them, at temperature 4).
#include "device.h"
#include "step_kernels.h"

#include <float.h>

namespace lora {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 2048;
constexpr int kSegs = 2048;                  // segments of a row whose sums are kept
constexpr float kOne = 2147483648.0f;        // 2^31, the weight of the largest logit

struct Row {
    const void* logits;
    bool bf16;
    int V;
    float inv_t;
    float lmax;
    // (l - lmax) inv_t as (half l - half_max) inv_half_t: half is 0.5 where the
    // temperature is above 1, so that a difference past the largest float keeps its
    // value where it counts (exact, a power of two; 1 below, where it weighs nothing)
    float half, half_max, inv_half_t;
};

// The logit of column i; NaN counts as masked (-inf), -0 as +0 (they tie).
__device__ __forceinline__ float logit(const Row& r, int i)
{
    const float l = r.bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(r.logits)[i])
                           : static_cast<const float*>(r.logits)[i];
    return l != l ? -INFINITY : l + 0.0f;
}

// Orders like the logit (-0 with +0).
__device__ __forceinline__ uint32_t order_key(float l)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, l + 0.0f);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ uint32_t weight(const Row& r, float l)
{
    if (l == r.lmax)
        return 1u << 31;
    const float z = fmaf(l, r.half, -r.half_max) * r.inv_half_t;
    // a masked logit, or one whose exponent is not a number (infinite maximum at
    // an infinite temperature), has no weight
    return l == -INFINITY || !(z == z) ? 0u : __float2uint_rn(expf(z) * kOne);
}

struct Acc {
    uint32_t n;                              // elements
    uint64_t w;                              // their weight
};

// Sums within a wave go through the vector unit's lane moves, a few cycles each;
// a shuffle through LDS takes over a hundred, and a row alone on its CU waits for
// every one (1 x 32000 top-k 15.0 -> 13.3 us).  Every lane of the wave has to be active.

// v of the lane that the move CTRL reads, 0 where there is none.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t moved(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint64_t moved(uint64_t v)
{
    return (uint64_t)moved<CTRL, ROWS>((uint32_t)(v >> 32)) << 32 | moved<CTRL, ROWS>((uint32_t)v);
}

constexpr int kRowShift = 0x110;             // + d: the lane d below, in the same 16
constexpr int kLane15 = 0x142, kLane31 = 0x143;   // last lane of the 16, 32 before
constexpr int kXor1 = 0xB1, kXor2 = 0x4E;    // within four lanes
constexpr int kMirror8 = 0x141, kMirror16 = 0x140;

// Inclusive sum over the wave, in lane order.
__device__ __forceinline__ uint64_t wave_scan(uint64_t v)
{
    v += moved<kRowShift + 1>(v);
    v += moved<kRowShift + 2>(v);
    v += moved<kRowShift + 4>(v);
    v += moved<kRowShift + 8>(v);
    v += moved<kLane15, 0xA>(v);             // to the second and fourth 16
    v += moved<kLane31, 0xC>(v);             // to the upper 32
    return v;
}

// op over each aligned group of `share` lanes (a power of two, at most 64, the
// same in the whole wave); every lane gets it.  Where a mirror stands for a
// distance of 4 or 8, the lanes it mixes up already hold the same value.
template <class Op>
__device__ __forceinline__ uint64_t wave_join(uint64_t v, int share, Op op)
{
    if (share > 1)
        v = op(v, moved<kXor1>(v));
    if (share > 2)
        v = op(v, moved<kXor2>(v));
    if (share > 4)
        v = op(v, moved<kMirror8>(v));
    if (share > 8)
        v = op(v, moved<kMirror16>(v));
    if (share > 16) {
        const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false);
        v = op((uint64_t)hi[0] << 32 | lo[0], (uint64_t)hi[1] << 32 | lo[1]);
    }
    if (share > 32) {
        const auto lo = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
        const auto hi = __builtin_amdgcn_permlane32_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false);
        v = op((uint64_t)hi[0] << 32 | lo[0], (uint64_t)hi[1] << 32 | lo[1]);
    }
    return v;
}

__device__ __forceinline__ uint64_t wave_sum(uint64_t v, int share = 64)
{
    return wave_join(v, share, [](uint64_t a, uint64_t b) { return a + b; });
}

__device__ __forceinline__ uint64_t wave_max(uint64_t v)
{
    return wave_join(v, 64, [](uint64_t a, uint64_t b) { return max(a, b); });
}

// Inclusive sum over the workgroup of one value a thread, in thread order.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* buf)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = wave_scan(v);
    __syncthreads();
    if (lane == 63)
        buf[wave] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves - 1; ++i)
        v += i < wave ? buf[i] : 0;
    return v;
}

struct Shared {
    uint32_t hist_n[kBins];
    unsigned long long hist_w[kBins];
    unsigned long long seg[kSegs];
    uint64_t scan[2 * kWaves];
    uint64_t pick_sum;
    uint64_t pick_n;
    int pick;
};

// A radix select over the logits' bits, 11, 11 and 10 at a time, with a
// histogram of counts and weights in LDS.  Finds the element of the order at which a running sum (of counts when BY_N,
// of weights otherwise) over the elements before it is still below `target`
// (> 0), and the next element's is not: its key, the number of elements and the
// weight before its key.  Only elements with a weight take part.
template <bool BY_N>
__device__ void select(const Row& r, Shared& s, uint64_t target, uint32_t* key_out, uint32_t* n_out, uint64_t* w_out,
                       uint32_t* ties_out)
{
    uint32_t prefix = 0, n_before = 0, ties = 0;
    uint64_t w_before = 0;
    int shift = 32;
    const int bits[3] = {11, 11, 10};
    for (int pass = 0; pass < 3; ++pass) {
        const uint32_t high = shift == 32 ? 0u : prefix >> shift;
        const int low = shift - bits[pass];
        for (int i = threadIdx.x; i < kBins; i += kThreads) {
            s.hist_n[i] = 0;
            s.hist_w[i] = 0;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < r.V; i += kThreads) {
            const float l = logit(r, i);
            const uint32_t k = order_key(l);
            const uint32_t w = weight(r, l);
            if (w && (shift == 32 || k >> shift == high)) {
                const uint32_t bin = (k >> low) & ((1u << bits[pass]) - 1);
                atomicAdd(&s.hist_n[bin], 1u);
                atomicAdd(&s.hist_w[bin], (unsigned long long)w);
            }
        }
        __syncthreads();
        // bins from the top: thread t has bins kBins-1-2t and kBins-2-2t
        const int b0 = kBins - 1 - 2 * threadIdx.x, b1 = b0 - 1;
        const uint64_t n0 = s.hist_n[b0], n1 = s.hist_n[b1], w0 = s.hist_w[b0], w1 = s.hist_w[b1];
        const uint64_t sn = block_scan(n0 + n1, s.scan) - n0 - n1 + n_before;
        const uint64_t sw = block_scan(w0 + w1, s.scan) - w0 - w1 + w_before;
        const uint64_t at = BY_N ? sn : sw, c0 = BY_N ? n0 : w0, c1 = BY_N ? n1 : w1;
        if (at < target && at + c0 >= target && c0) {
            s.pick = b0;
            s.pick_n = sn;
            s.pick_sum = sw;
        } else if (at + c0 < target && at + c0 + c1 >= target && c1) {
            s.pick = b1;
            s.pick_n = sn + n0;
            s.pick_sum = sw + w0;
        }
        __syncthreads();
        prefix |= (uint32_t)s.pick << low;
        n_before = (uint32_t)s.pick_n;
        w_before = s.pick_sum;
        ties = s.hist_n[s.pick];
        shift = low;
        __syncthreads();
    }
    *key_out = prefix;
    *n_out = n_before;
    *w_out = w_before;
    *ties_out = ties;
}

// The lowest index at which the running sum of value(i) over columns 0..i exceeds
// t (t below the total).
template <class F>
__device__ int locate(const Row& r, Shared& s, uint64_t t, F value)
{
    const int seg_len = ((r.V + kSegs - 1) / kSegs + 63) / 64 * 64;
    const int segs = (r.V + seg_len - 1) / seg_len;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < kSegs; i += kThreads)
        s.seg[i] = 0;
    __syncthreads();
    for (int g = wave; g < segs; g += kWaves) {
        uint64_t sum = 0;
        const int end = min(r.V, (g + 1) * seg_len);
        for (int i = g * seg_len + lane; i < end; i += 64)
            sum += value(i);
        sum = wave_sum(sum);
        if (lane == 0)
            s.seg[g] = sum;
    }
    __syncthreads();
    const uint64_t a = s.seg[2 * threadIdx.x], b = s.seg[2 * threadIdx.x + 1];
    const uint64_t before = block_scan(a + b, s.scan) - a - b;
    if (before <= t && before + a > t) {
        s.pick = 2 * threadIdx.x;
        s.pick_sum = before;
    } else if (before + a <= t && before + a + b > t) {
        s.pick = 2 * threadIdx.x + 1;
        s.pick_sum = before + a;
    }
    __syncthreads();
    if (wave == 0) {
        uint64_t run = s.pick_sum;
        const int first = s.pick * seg_len, end = min(r.V, first + seg_len);
        for (int base = first; base < end; base += 64) {
            const int i = base + lane;
            uint64_t v = i < end ? value(i) : 0;
            v = wave_scan(v);
            const uint64_t hit = __ballot(run + v > t);
            if (hit) {
                if (lane == 0)
                    s.pick = base + __builtin_ctzll(hit);
                break;
            }
            run += __shfl((unsigned long long)v, 63);
        }
    }
    __syncthreads();
    const int i = s.pick;
    __syncthreads();
    return i;
}

// One row's settings, as the definition reads them.
struct Settings {
    int k;                                   // 0: off
    float top_p;                             // 1: off
    uint32_t floor_w;                        // 0: off
    float u;
};

// The weight a token's predecessors have to stay below.
__device__ __forceinline__ uint64_t top_p_mass(float top_p, uint64_t total)
{
    return top_p > 0.0f ? max((uint64_t)ceil((double)top_p * (double)total), (uint64_t)1) : 1;
}

__device__ __forceinline__ uint64_t target(float u, uint64_t total)
{
    const double want = u > 0.0f ? (double)u * (double)total : 0.0;
    return want >= (double)total ? total - 1 : (uint64_t)want;
}

__device__ __forceinline__ void answer(const SampleParams& p, int64_t row, int token, uint32_t w, uint64_t total)
{
    p.tokens[row] = token;
    if (p.logprobs)
        p.logprobs[row] = logf((float)((double)w / (double)total));
}

// Any row, by passes over it: the way for what the paths below do not take
// (more ties than their lists hold, top-k above kThreads, infinite maxima or
// inverse temperatures, temperatures of 1e37 and more).
__device__ void sample_any(const SampleParams& p, const Settings& c, const Row& r, Shared& s, int64_t row)
{
    // the kept prefix: keys above `key`, and of those equal to it the first `quota`
    uint32_t key = 0, quota = 0xFFFFFFFFu, ties = 0;
    const int k = c.k;
    const float top_p = c.top_p;
    uint64_t total = 0;
    bool cut = false;
    if (k > 0 && k < r.V) {
        uint32_t nb;
        uint64_t wb;
        // fewer than k elements with a weight: all of them stay
        uint64_t mine = 0;
        for (int i = threadIdx.x; i < r.V; i += kThreads)
            mine += weight(r, logit(r, i)) != 0;
        const uint64_t upto = block_scan(mine, s.scan);
        if (threadIdx.x == kThreads - 1)
            s.pick_n = upto;
        __syncthreads();
        const uint64_t positive = s.pick_n;
        __syncthreads();
        if ((uint64_t)k < positive) {
            select<true>(r, s, (uint64_t)k, &key, &nb, &wb, &ties);
            quota = (uint32_t)k - nb;
            cut = true;
        }
    }
    // top-p needs the weight kept so far
    auto in_prefix = [&](float l) { return !cut || order_key(l) > key; };
    if (top_p < 1.0f) {
        uint64_t mine = 0;
        uint32_t wk = 0;
        for (int i = threadIdx.x; i < r.V; i += kThreads) {
            const float l = logit(r, i);
            const uint32_t w = weight(r, l);
            if (in_prefix(l))
                mine += w;
            else if (order_key(l) == key)
                wk = w;
        }
        const uint64_t upto = block_scan(mine, s.scan);
        if (threadIdx.x == kThreads - 1)
            s.pick_sum = upto;
        if (wk)
            s.pick_n = wk;                   // every writer has the same value
        __syncthreads();
        total = s.pick_sum + (cut ? (uint64_t)quota * s.pick_n : 0);
        __syncthreads();
        const uint64_t mass = top_p_mass(top_p, total);
        uint32_t kp, nb, tp;
        uint64_t wb;
        select<false>(r, s, mass, &kp, &nb, &wb, &tp);
        const uint32_t u = kp ^ ((kp >> 31) ? 0x80000000u : 0xFFFFFFFFu);
        const uint64_t wt = weight(r, __builtin_bit_cast(float, u));
        const uint32_t qp = (uint32_t)((mass - wb + wt - 1) / wt);
        if (!cut || kp > key) {
            key = kp;
            quota = qp;
            ties = tp;
        } else if (kp == key) {
            quota = min(quota, qp);
        }
        cut = true;
    }
    // of the tied elements the first `quota`: up to and including column `last`
    int last = r.V;
    if (cut && quota < ties)
        last = locate(r, s, quota - 1, [&](int i) { return (uint64_t)(order_key(logit(r, i)) == key); });
    const uint32_t floor_w = c.floor_w;
    auto kept = [&](int i) -> uint64_t {
        const float l = logit(r, i);
        const uint32_t w = weight(r, l), o = order_key(l);
        const bool in = !cut || o > key || (o == key && i <= last);
        return in && w >= floor_w ? w : 0u;
    };
    uint64_t mine = 0;
    for (int i = threadIdx.x; i < r.V; i += kThreads)
        mine += kept(i);
    const uint64_t upto = block_scan(mine, s.scan);
    if (threadIdx.x == kThreads - 1)
        s.pick_sum = upto;
    __syncthreads();
    total = s.pick_sum;
    __syncthreads();
    const int token = locate(r, s, target(c.u, total), kept);
    if (threadIdx.x == 0)
        answer(p, row, token, (uint32_t)kept(token), total);
}

// ---------------------------------------------------------------------------
// The usual rows.  The row is read in aligned 16-byte groups of kVec logits;
// wave w has the w-th contiguous run of groups, so that sums over a wave's
// elements are sums over a range of indices.
// ---------------------------------------------------------------------------
constexpr int kHist = 512;                   // bins over the weights' range, per wave
constexpr int kList = 4096;                  // elements of the bins at the threshold
constexpr int kFew = 1024;                   // elements compared with one another
constexpr float kRange = 22.0f;              // rint(2^31 exp(-z)) is 0 from z = 32 ln 2 = 22.2 on
constexpr float kBinsPerUnit = (kHist - 2) / kRange;

struct Fast {
    unsigned long long hist[kWaves][kHist];
    unsigned long long list[kList];          // place() of an element, its weight, its sub-bin
    uint32_t list_w[kList];
    int16_t list_sub[kList];
    unsigned long long sub[kThreads];
    unsigned long long few[kFew];            // place() of an element
    uint32_t few_w[kFew];
    unsigned long long range[kWaves];
    uint64_t scan[2 * kWaves];
    float red[2 * kWaves];
    uint32_t n;
    uint32_t few_n;
    uint64_t last;
    uint64_t all, sum;
    int pick;
};

union Lds {
    Shared any;
    Fast fast;
    __device__ Lds() {}
};

template <bool BF16>
struct Groups {
    static constexpr int kVec = BF16 ? 8 : 4;
    const char* base;                        // 16-byte aligned, at or before the row's start
    int off;                                 // elements between them
    int V;
    int n;                                   // groups
    int run;                                 // groups of a wave, a multiple of 64

    __device__ Groups(const void* logits, int v)
    {
        const uintptr_t a = reinterpret_cast<uintptr_t>(logits);
        base = reinterpret_cast<const char*>(a & ~(uintptr_t)15);
        off = (int)(a & 15) / (BF16 ? 2 : 4);
        V = v;
        n = (v + off + kVec - 1) / kVec;
        run = ((n + kWaves - 1) / kWaves + 63) / 64 * 64;
    }

    __device__ int first(int group) const { return group * kVec - off; }

    // A group's 16 bytes, which lie in the row.
    __device__ __forceinline__ u32x4 load(int group) const
    {
        return *(const global_u32x4*)(base + (int64_t)group * 16);
    }

    // The same of any group, element by element, with -inf outside the row (never
    // read there).
    __device__ __forceinline__ u32x4 load_edge(int group) const
    {
        u32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const int i = first(group) + e;
            const bool in = i >= 0 && i < V;
            if constexpr (BF16) {
                const uint32_t b = in ? reinterpret_cast<const uint16_t*>(base)[(int64_t)group * kVec + e] : 0xFF80u;
                v[e / 2] |= b << (16 * (e % 2));
            } else {
                v[e] = in ? reinterpret_cast<const uint32_t*>(base)[(int64_t)group * kVec + e] : 0xFF800000u;
            }
        }
        return v;
    }

    __device__ bool whole(int group) const { return first(group) >= 0 && first(group) + kVec <= V; }

    // Its logits as they are: a NaN compares false, is no maximum and has no
    // weight, and order_key takes -0 as +0.
    static __device__ __forceinline__ void logits(u32x4 v, float (&l)[kVec])
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t b = v[e];
            if constexpr (BF16) {
                l[2 * e] = __builtin_bit_cast(float, b << 16);
                l[2 * e + 1] = __builtin_bit_cast(float, b & 0xFFFF0000u);
            } else {
                l[e] = __builtin_bit_cast(float, b);
            }
        }
    }

    // f(logits, first column) over the groups of this wave's run, with the loads of
    // the next kAhead in flight; the row's first and last group may be cut and come last.
    // Written out kAhead times, so that each load has its registers: moved on from set
    // to set, 256 x 128259 greedy took 27.5 us instead of 25.1.
    template <class F>
    __device__ __forceinline__ void each_group(F f) const
    {
        constexpr int kAhead = 4;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
        const int begin = max(wave * run, whole(0) ? 0 : 1);
        const int end = min((wave + 1) * run, whole(n - 1) ? n : n - 1);
        if (begin < end) {
            u32x4 v[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) // past the run: its last group again
                v[a] = load(min(begin + lane + a * 64, end - 1));
#pragma unroll 1
            for (int g0 = begin + lane; g0 - lane < end; g0 += kAhead * 64) {
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    const int g = g0 + a * 64;
                    float l[kVec];
                    logits(v[a], l);
                    if (g < end)
                        f(l, first(g));
                    v[a] = load(min(g + kAhead * 64, end - 1));
                }
            }
        }
        // lane 0 has the first group, lane 1 the last, if they are cut
        const int cut = lane == 0 ? 0 : n - 1;
        if (lane < (n > 1 ? 2 : 1) && !whole(cut) && cut / run == wave) {
            float l[kVec];
            logits(load_edge(cut), l);
            f(l, first(cut));
        }
    }

    // f(logit, column) over its elements
    template <class F>
    __device__ __forceinline__ void each(F f) const
    {
        each_group([&](float (&l)[kVec], int i0) {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                f(l[e], i0 + e);
        });
    }

    // Puts the elements with take(logit) into a list by put(slot, logit, column);
    // *n counts them.  A lane takes its slots once a group.
    template <class T, class P>
    __device__ __forceinline__ void gather(uint32_t* n, T take, P put) const
    {
        each_group([&](float (&l)[kVec], int i0) {
            uint32_t hits = 0;
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                hits |= (uint32_t)take(l[e]) << e;
            if (hits) {
                uint32_t slot = atomicAdd(n, (uint32_t)__builtin_popcount(hits));
#pragma unroll 1
                for (; hits; hits &= hits - 1) {
                    const int e = __builtin_ctz(hits);
                    float v = l[0];
#pragma unroll
                    for (int j = 1; j < kVec; ++j)
                        v = e == j ? l[j] : v;
                    put(slot++, v, i0 + e);
                }
            }
        });
    }
};

// Where the maximum and the inverse temperature are finite: the exponent of a
// logit and the weight it gives.
__device__ __forceinline__ float exponent(const Row& r, float l)
{
    return (l - r.lmax) * r.inv_t;
}

__device__ __forceinline__ uint32_t weight_of_exponent(float z)
{
    return __float2uint_rn(expf(z) * kOne);
}

__device__ __forceinline__ uint32_t weight_finite(const Row& r, float l)
{
    return weight_of_exponent(exponent(r, l));
}

// Place among the bins, whose number is its whole part: 0 at the maximum, rising
// as the logit falls; kHist - 1 and above for what surely has no weight.
// Monotonous, being rounded products and differences.
__device__ __forceinline__ float bin_place(float z)
{
    return -z * kBinsPerUnit;
}

__device__ __forceinline__ int bin_of(float place)
{
    return (int)fminf(place, (float)(kHist - 1));
}

// An element's place in the order, as a number that falls along it.
__device__ __forceinline__ uint64_t place(uint32_t key, int column)
{
    return (uint64_t)key << 32 | ~(uint32_t)column;
}

__device__ __forceinline__ uint32_t place_column(uint64_t place)
{
    return ~(uint32_t)place;
}

__device__ __forceinline__ float block_reduce_max(float v, float* buf)
{
    v = __builtin_bit_cast(float, (uint32_t)wave_join(__builtin_bit_cast(uint32_t, v), 64, [](uint64_t a, uint64_t b) {
        return (uint64_t)__builtin_bit_cast(
            uint32_t, fmaxf(__builtin_bit_cast(float, (uint32_t)a), __builtin_bit_cast(float, (uint32_t)b)));
    }));
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        buf[threadIdx.x >> 6] = v;
    __syncthreads();
    v = buf[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i)
        v = fmaxf(v, buf[i]);
    return v;
}

__device__ __forceinline__ uint64_t block_sum(uint64_t v, uint64_t* buf)
{
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        buf[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i)
        v += buf[i];
    return v;
}

// s.few[0, n) are compared with one another: few_share(n) neighbouring threads
// stand for each element, and share the others among them.
__device__ __forceinline__ int few_share(int n)
{
    int share = kThreads;
    while (share > 1 && (kThreads / share) < n)
        share >>= 1;
    return share;
}

template <class F>
__device__ __forceinline__ void over_few(int n, int share, F f)
{
#pragma unroll 4
    for (int j = threadIdx.x % share; j < n; j += share)
        f(j);
}

// Sum over the `share` neighbouring threads that stand for one element.
__device__ __forceinline__ uint64_t share_sum(uint64_t v, int share, uint64_t* wide)
{
    v = wave_sum(v, min(share, 64));
    if (share > 64) {                        // uniform: few elements, several waves each
        __syncthreads();
        if ((threadIdx.x & 63) == 0)
            wide[threadIdx.x >> 6] = v;
        __syncthreads();
        const int waves = share >> 6, first = (threadIdx.x >> 6) / waves * waves;
        v = 0;
        for (int i = 0; i < waves; ++i)
            v += wide[first + i];
    }
    return v;
}

// Top-k rows: the k-th largest of the threads' own maxima bounds the k-th
// largest logit from below.  The logits in its bin and above are gathered and
// compared with one another.  False if they are more than kFew, as with a large k,
// or where the large logits are neighbours or the bins are stretched by a finite
// mask.
template <bool BF16>
__device__ bool sample_top_k(const SampleParams& p, const Settings& c, const Row& r, const Groups<BF16>& G, Fast& s,
                             int64_t row, float mine)
{
    // bins over the maxima's range; a thread without logits has none.  `per` stays
    // finite for any range, so that the maximum's own place is 0
    const float lowest = -block_reduce_max(mine == -INFINITY ? -INFINITY : -mine, s.red);
    if (!(r.lmax - lowest < INFINITY))
        return false;
    const float per = lowest < r.lmax ? fminf((kThreads - 1) / (r.lmax - lowest), FLT_MAX) : 0.0f;
    auto at = [&](float l) { return (r.lmax - l) * per; };
    uint32_t* count = reinterpret_cast<uint32_t*>(s.sub);
    count[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        s.n = 0;
        s.pick = kThreads - 1;               // fewer maxima than k: every bin
    }
    __syncthreads();
    if (mine != -INFINITY)
        atomicAdd(&count[(int)fminf(at(mine), (float)(kThreads - 1))], 1u);
    __syncthreads();
    const uint64_t own = count[threadIdx.x];
    const uint64_t upto = block_scan(own, s.scan);
    const bool enough = upto >= (uint64_t)c.k && upto - own < (uint64_t)c.k;
    if (enough)
        s.pick = threadIdx.x;
    __syncthreads();
    // with fewer than k maxima the k-th logit may lie below all of them, as far as
    // the type reaches: every logit's place is 0
    const bool all = block_sum(own, s.scan) < (uint64_t)c.k;
    const float take_per = all ? 0.0f : per, end_place = all ? 1.0f : (float)(s.pick + 1);
    G.gather(
        &s.n, [&](float l) { return (r.lmax - l) * take_per < end_place; },    // so is not -inf (NaN or infinite)
        [&](uint32_t slot, float l, int i) {
            if (slot < kFew) {
                s.few[slot] = place(order_key(l), i);
                s.few_w[slot] = weight_finite(r, l);
            }
        });
    __syncthreads();
    const int n = (int)s.n;
    if (n > kFew)
        return false;
    const int share = few_share(n), me = threadIdx.x / share;
    const uint64_t mine_at = me < n ? s.few[me] : 0;
    const uint32_t w = me < n ? s.few_w[me] : 0;
    uint64_t rank = 0, before = 0;
    if (me < n)
        over_few(n, share, [&](int j) {
            const bool first = s.few[j] > mine_at;
            rank += first;
            before += first ? s.few_w[j] : 0u;
        });
    rank = share_sum(rank, share, s.scan);
    __syncthreads();
    before = share_sum(before, share, s.scan);
    const bool lead = me < n && threadIdx.x % share == 0;
    uint64_t total = block_sum(lead && rank < (uint64_t)c.k ? w : 0, s.scan);
    const bool keep = me < n && rank < (uint64_t)c.k && w >= max(c.floor_w, 1u) &&
                      (c.top_p >= 1.0f || before < top_p_mass(c.top_p, total));
    total = block_sum(lead && keep ? w : 0, s.scan);
    if (lead)
        s.few_w[me] = keep ? w : 0;
    __syncthreads();
    uint64_t below = 0;                      // kept weight at lower indices
    const uint32_t idx = place_column(mine_at);
    if (keep)
        over_few(n, share, [&](int j) { below += place_column(s.few[j]) < idx ? s.few_w[j] : 0u; });
    below = share_sum(below, share, s.scan);
    const uint64_t t = target(c.u, total);
    if (lead && keep && below <= t && t < below + w)
        answer(p, row, (int)idx, w, total);
    return true;
}

// The other rows: a histogram of the weights for each wave's range of indices
// gives the row's weight and the bin where top-p (and min-p) cuts; only that
// bin's elements are looked at one by one.  False if they are too many.
template <bool BF16>
__device__ bool sample_mass(const SampleParams& p, const Settings& c, const Row& r, const Groups<BF16>& G, Fast& s,
                            int64_t row)
{
    constexpr int kVec = Groups<BF16>::kVec;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool cut = c.top_p < 1.0f || c.floor_w > 0;
    // the kept prefix ends with `last`; floor_w applies on top
    uint64_t last = 0;
    uint64_t total = 0;
    if (!cut) {
        uint64_t sum = 0;
        G.each([&](float l, int) { sum += weight_finite(r, l); });
        sum = wave_sum(sum);
        if (lane == 0)
            s.range[wave] = sum;
        __syncthreads();
    } else {
        for (int i = lane; i < kHist; i += 64)
            s.hist[wave][i] = 0;
        if (threadIdx.x == 0) {
            s.n = 0;
        }
        G.each([&](float l, int) {
            const float z = exponent(r, l);
            const uint32_t w = weight_of_exponent(z);
            if (w)
                atomicAdd(&s.hist[wave][bin_of(bin_place(z))], (unsigned long long)w);
        });
        __syncthreads();
        // the bin where top-p cuts
        uint64_t own = 0;
        if (threadIdx.x < kHist)
#pragma unroll
            for (int i = 0; i < kWaves; ++i)
                own += s.hist[i][threadIdx.x];
        const uint64_t upto = block_scan(own, s.scan);
        if (threadIdx.x == kThreads - 1)
            s.all = upto;
        __syncthreads();
        const uint64_t all = s.all;
        const uint64_t mass = c.top_p < 1.0f ? top_p_mass(c.top_p, all) : all;
        if (upto >= mass && upto - own < mass) {
            s.pick = threadIdx.x;
            s.sum = upto - own;
        }
        __syncthreads();
        // the bins that are looked at one by one: that one, and where min-p cuts
        // the one of its logarithm with a neighbour on both sides (rounding)
        const int pick = s.pick;
        const uint64_t pick_before = s.sum;
        int from = pick, to = pick;
        if (c.floor_w) {
            // w >= floor_w from 2^31 exp(-z) >= floor_w - 1/2 on
            const int f = (int)fminf(-logf(((float)c.floor_w - 0.5f) / kOne) * kBinsPerUnit, (float)(kHist - 1));
            if (pick >= f - 1) {
                from = max(min(pick, f - 1), 0);
                to = min(pick, f + 1);
            }
        }
        // bins below `from` are kept whole, bins above `to` not at all; sub-bins of
        // the one where top-p cuts
        const float first_place = (float)from, end_place = to >= kHist - 1 ? INFINITY : (float)(to + 1);
        auto sub_bin = [&](float at) {       // exact, so monotonous; of other bins: outside
            return at >= (float)pick && (at < (float)(pick + 1) || pick == kHist - 1)
                       ? (int)fminf((at - (float)pick) * kThreads, (float)(kThreads - 1))
                       : -1;
        };
        s.sub[threadIdx.x] = 0;
        if (threadIdx.x < kWaves)
            s.range[threadIdx.x] = 0;
        __syncthreads();
        G.gather(
            &s.n,
            [&](float l) {                   // so is not -inf
                const float at = bin_place(exponent(r, l));
                return at >= first_place && at < end_place;
            },
            [&](uint32_t slot, float l, int i) {
                if (slot < kList) {
                    const float z = exponent(r, l);
                    const uint32_t w = weight_of_exponent(z);
                    const int sub = sub_bin(bin_place(z));
                    s.list[slot] = place(order_key(l), i);
                    s.list_w[slot] = w;
                    s.list_sub[slot] = (int16_t)sub;
                    if (sub >= 0)
                        atomicAdd(&s.sub[sub], (unsigned long long)w);
                }
            });
        __syncthreads();
        const int n = (int)s.n;
        if (n > kList)
            return false;
        if (c.top_p < 1.0f && pick <= to) {
            const uint64_t o = s.sub[threadIdx.x];
            const uint64_t up = block_scan(o, s.scan) + pick_before;
            if (up >= mass && up - o < mass) {
                s.pick = threadIdx.x;
                s.sum = up - o;
            }
            if (threadIdx.x == 0)
                s.few_n = 0;
            __syncthreads();
            const int sub = s.pick;
            const uint64_t sub_before = s.sum;
#pragma unroll 1
            for (int i = threadIdx.x; i < n; i += kThreads)
                if (s.list_sub[i] == sub) {
                    const uint32_t at = atomicAdd(&s.few_n, 1u);
                    if (at < kFew) {
                        s.few[at] = s.list[i];
                        s.few_w[at] = s.list_w[i];
                    }
                }
            __syncthreads();
            const int m = (int)s.few_n;
            if (m > kFew)
                return false;
            const int share = few_share(m), me = threadIdx.x / share;
            uint64_t before = 0;
            const uint64_t mine_at = me < m ? s.few[me] : 0;
            if (me < m)
                over_few(m, share, [&](int j) { before += s.few[j] > mine_at ? s.few_w[j] : 0u; });
            before = share_sum(before, share, s.scan) + sub_before;
            // the last one kept: its predecessors stay below the mass, with it they reach it
            if (me < m && threadIdx.x % share == 0 && before < mass && before + s.few_w[me] >= mass)
                s.last = mine_at;
            __syncthreads();
            last = s.last;
        }
        // kept weight of each range of indices
        uint64_t sum = 0;
        for (int i = lane; i < from; i += 64)
            sum += s.hist[wave][i];
        if (sum)
            atomicAdd(&s.range[wave], (unsigned long long)sum);
#pragma unroll 1
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const uint64_t at = s.list[i];
            const uint32_t w = s.list_w[i];
            if (w >= c.floor_w && at >= last)
                atomicAdd(&s.range[((int)place_column(at) + G.off) / kVec / G.run], (unsigned long long)w);
        }
        __syncthreads();
    }
    // the range the number falls into, then the place in it
#pragma unroll
    for (int i = 0; i < kWaves; ++i)
        total += s.range[i];
    const uint64_t t = target(c.u, total);
    uint64_t before = 0;
    int range = 0;
    for (; range < kWaves - 1; ++range) {
        if (before + s.range[range] > t)
            break;
        before += s.range[range];
    }
    const int per = (G.run + kThreads - 1) / kThreads;
    const int first = range * G.run + threadIdx.x * per;
    const int stop = min(min(first + per, (range + 1) * G.run), G.n);
    auto kept = [&](float l, int i) -> uint32_t {
        const uint32_t w = weight_finite(r, l);
        return w >= c.floor_w && place(order_key(l), i) >= last ? w : 0u;
    };
    uint64_t own = 0;
    for (int g = first; g < stop; ++g) {
        float l[kVec];
        G.logits(G.whole(g) ? G.load(g) : G.load_edge(g), l);
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            own += kept(l[e], G.first(g) + e);
    }
    uint64_t at = block_scan(own, s.scan) - own + before;
    if (at <= t && t < at + own) {
        for (int g = first; g < stop; ++g) {
            float l[kVec];
            G.logits(G.whole(g) ? G.load(g) : G.load_edge(g), l);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const uint32_t w = kept(l[e], G.first(g) + e);
                if (at <= t && t < at + w)
                    answer(p, row, G.first(g) + e, w, total);
                at += w;
            }
        }
    }
    return true;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_sample(SampleParams p)
{
    __shared__ Lds lds;
    Fast& s = lds.fast;
    const int64_t row = blockIdx.x;
    Row r;
    r.bf16 = BF16;
    r.V = p.V;
    r.logits = static_cast<const char*>(p.logits) + row * p.ld * (BF16 ? 2 : 4);
    const float T = p.temperature ? p.temperature[row] : 1.0f;
    const bool greedy = !(T > 0.0f);
    r.inv_t = greedy ? 1.0f : 1.0f / T;
    Settings c;
    c.k = p.top_k ? p.top_k[row] : 0;
    c.k = c.k > 0 && c.k < p.V ? c.k : 0;
    c.top_p = p.top_p ? fminf(p.top_p[row], 1.0f) : 1.0f;      // NaN: 1
    const float min_p = p.min_p ? p.min_p[row] : 0.0f;
    c.floor_w = min_p > 0.0f ? (uint32_t)fmin(ceil((double)min_p * (double)kOne), (double)kOne) : 0u;
    c.u = p.u[row];

    const Groups<BF16> G(r.logits, r.V);
    if (greedy) {                            // the first of the order
        float best = -INFINITY;
        int at = 0;
        G.each([&](float l, int i) {
            at = l > best || (l == best && i < at) ? i : at;
            best = fmaxf(best, l);
        });
        uint64_t top = best == -INFINITY ? 0 : place(order_key(best), at);
        top = wave_max(top);
        if ((threadIdx.x & 63) == 0)
            s.scan[threadIdx.x >> 6] = top;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kWaves; ++i)
                top = max(top, s.scan[i]);
            p.tokens[row] = top ? (int)place_column(top) : -1;
            if (p.logprobs)
                p.logprobs[row] = top ? 0.0f : -INFINITY;
        }
        return;
    }
    float mine = -INFINITY;
    G.each([&](float l, int) { mine = fmaxf(mine, l); });
    r.lmax = block_reduce_max(mine, s.red);
    if (r.lmax == -INFINITY) {               // every logit masked
        if (threadIdx.x == 0) {
            p.tokens[row] = -1;
            if (p.logprobs)
                p.logprobs[row] = -INFINITY;
        }
        return;
    }
    r.half = r.inv_t < 1.0f ? 0.5f : 1.0f;
    r.half_max = r.half * r.lmax;
    r.inv_half_t = r.inv_t / r.half;
    // also that a difference of logits past the largest float weighs nothing: from
    // 1 / T = 22.2 / 3.4e38 on
    const bool finite = r.lmax < INFINITY && r.inv_t > 1e-37f && r.inv_t < INFINITY;
    bool done = false;
    if (finite && c.k > 0 && c.k <= kThreads)
        done = sample_top_k<BF16>(p, c, r, G, s, row, mine);
    else if (finite && c.k == 0)
        done = sample_mass<BF16>(p, c, r, G, s, row);
    if (!done) {
        __syncthreads();
        sample_any(p, c, r, lds.any, row);
    }
}

}  // namespace

hipError_t launch_sample(const SampleParams& p, bool bf16, hipStream_t st)
{
    if (bf16)
        hipLaunchKernelGGL(k_sample<true>, dim3((unsigned)p.B), dim3(kThreads), 0, st, p);
    else
        hipLaunchKernelGGL(k_sample<false>, dim3((unsigned)p.B), dim3(kThreads), 0, st, p);
    return hipGetLastError();
}

}  // namespace lora
