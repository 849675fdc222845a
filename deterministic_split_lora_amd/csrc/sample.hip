// One token per row of logits: temperature, top-k, top-p, min-p and a draw
// from a given random number.
//
// A logit l of weight  w = rint(2^31 exp((l - max) / T))  is a whole number, so
// every sum below is a 64-bit integer sum: exact, hence the same in any order,
// for any work split and next to any other rows.
//
// Tokens are ordered by (logit descending, index ascending).  Each of top-k,
// top-p and min-p keeps a prefix of that order, so their intersection is a
// prefix too and is given by its last element: a threshold key and how many of
// the elements with that very key are kept (the lowest indices).  Thresholds
// are found by a radix select over the logits' bits, 11, 11 and 10 at a time,
// with a histogram of counts and weights in LDS.
//
// One workgroup owns a row.
#include "device.h"
#include "step_kernels.h"

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
};

// The logit of column i; NaN counts as masked (-inf), -0 as +0 (they tie).
__device__ __forceinline__ float logit(const Row& r, int i)
{
    const float l = r.bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(r.logits)[i])
                           : static_cast<const float*>(r.logits)[i];
    return l != l ? -INFINITY : l + 0.0f;
}

__device__ __forceinline__ uint32_t order_key(float l)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, l);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ uint32_t weight(const Row& r, float l)
{
    if (l == r.lmax)
        return 1u << 31;
    const float z = (l - r.lmax) * r.inv_t;
    // a masked logit, or one whose exponent is not a number (infinite maximum at
    // an infinite temperature), has no weight
    return l == -INFINITY || !(z == z) ? 0u : __float2uint_rn(expf(z) * kOne);
}

struct Acc {
    uint32_t n;                              // elements
    uint64_t w;                              // their weight
};

// Inclusive sum over the workgroup of one value a thread, in thread order.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* buf)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t u = __shfl_up((unsigned long long)v, d);
        if (lane >= d)
            v += u;
    }
    __syncthreads();
    if (lane == 63)
        buf[wave] = v;
    __syncthreads();
    for (int i = 0; i < wave; ++i)
        v += buf[i];
    return v;
}

struct Shared {
    uint32_t hist_n[kBins];
    unsigned long long hist_w[kBins];
    unsigned long long seg[kSegs];
    uint64_t scan[2 * kWaves];
    float red[kWaves];
    uint64_t pick_sum;
    uint64_t pick_n;
    int pick;
};

// Finds the element of the order at which a running sum (of counts when BY_N,
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
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
            sum += __shfl_xor((unsigned long long)sum, d);
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
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const uint64_t u = __shfl_up((unsigned long long)v, d);
                if (lane >= d)
                    v += u;
            }
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

__global__ void __launch_bounds__(kThreads) k_sample(SampleParams p, bool bf16)
{
    __shared__ Shared s;
    const int64_t row = blockIdx.x;
    Row r;
    r.bf16 = bf16;
    r.V = p.V;
    r.logits = static_cast<const char*>(p.logits) + row * p.ld * (bf16 ? 2 : 4);
    const float T = p.temperature ? p.temperature[row] : 1.0f;
    const bool greedy = !(T > 0.0f);
    r.inv_t = greedy ? 1.0f : 1.0f / T;

    float m = -INFINITY;
    for (int i = threadIdx.x; i < r.V; i += kThreads)
        m = fmaxf(m, logit(r, i));
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        m = fmaxf(m, __shfl_xor(m, d));
    if ((threadIdx.x & 63) == 0)
        s.red[threadIdx.x >> 6] = m;
    __syncthreads();
    for (int i = 0; i < kWaves; ++i)
        m = fmaxf(m, s.red[i]);
    r.lmax = m;
    if (m == -INFINITY) {                    // every logit masked
        if (threadIdx.x == 0) {
            p.tokens[row] = -1;
            if (p.logprobs)
                p.logprobs[row] = -INFINITY;
        }
        return;
    }

    // the kept prefix: keys above `key`, and of those equal to it the first `quota`
    uint32_t key = 0, quota = 0xFFFFFFFFu, ties = 0;
    const int k = greedy ? 1 : (p.top_k ? p.top_k[row] : 0);
    const float top_p = greedy || !p.top_p ? 1.0f : p.top_p[row];
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
    if (!(top_p >= 1.0f) && top_p == top_p) {
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
        const uint64_t mass = max((uint64_t)ceil((double)top_p * (double)total), (uint64_t)1);
        if (!(top_p > 0.0f) || mass <= total) {
            uint32_t kp, nb, tp;
            uint64_t wb;
            select<false>(r, s, top_p > 0.0f ? mass : 1, &kp, &nb, &wb, &tp);
            const uint32_t u = kp ^ ((kp >> 31) ? 0x80000000u : 0xFFFFFFFFu);
            const uint64_t wt = weight(r, __builtin_bit_cast(float, u));
            const uint64_t need = top_p > 0.0f ? mass : 1;
            const uint32_t qp = (uint32_t)((need - wb + wt - 1) / wt);
            if (!cut || kp > key) {
                key = kp;
                quota = qp;
                ties = tp;
            } else if (kp == key) {
                quota = min(quota, qp);
            }
            cut = true;
        }
    }
    // of the tied elements the first `quota`: up to and including column `last`
    int last = r.V;
    if (cut && quota < ties)
        last = locate(r, s, quota - 1, [&](int i) { return (uint64_t)(order_key(logit(r, i)) == key); });
    const float min_p = greedy || !p.min_p ? 0.0f : p.min_p[row];
    const uint32_t floor_w =
        min_p > 0.0f ? (uint32_t)fmin(ceil((double)min_p * (double)kOne), (double)kOne) : 0u;
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
    const float u = p.u[row];
    const double want = u > 0.0f ? (double)u * (double)total : 0.0;
    const uint64_t t = want >= (double)total ? total - 1 : (uint64_t)want;
    const int token = locate(r, s, t, kept);
    if (threadIdx.x == 0) {
        p.tokens[row] = token;
        if (p.logprobs)
            p.logprobs[row] = logf((float)((double)kept(token) / (double)total));
    }
}

}  // namespace

hipError_t launch_sample(const SampleParams& p, bool bf16, hipStream_t st)
{
    hipLaunchKernelGGL(k_sample, dim3((unsigned)p.B), dim3(kThreads), 0, st, p, bf16);
    return hipGetLastError();
}

}  // namespace lora
