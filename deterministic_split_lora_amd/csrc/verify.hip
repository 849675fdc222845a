// Verification of drafted tokens against the target's distributions.
//
// A drafted token x that came with probability q(x) is kept with probability
// min(1, p(x) / q(x)); the first that is not is replaced by a draw from
// max(p - q, 0): the tokens then have the target's distribution p.  Probabilities
// are whole numbers, P = rint(2^40 p), so that every sum is exact (below 2^53) and
// no split of the work can change a token.
//
// Three launches.  The rows' maxima, cuts and weights: a workgroup a row, the same
// steps as a draw (sample_row.h), all rows at once, since which ones count is only
// known from them; with its cuts a row leaves what it gives its drafted token.  Then
// the sums of max(P - Q, 0) over segments of the one row a sequence draws from, and the
// draw itself from its segment; each of these works out the accepted tokens anew, a
// lane a token, which is cheaper than a launch.
#include "sample_row.h"

namespace lora {

namespace {

constexpr double kUnit = 1099511627776.0;    // 2^40, the probability 1
constexpr int kSegment = 2048;               // columns of a segment
constexpr int kSumThreads = 256;

// What is left of a row once its cuts are known.
struct Cut {
    uint64_t total;                          // kept weight, 0: every logit masked
    uint64_t last;                           // place of the last element kept, or a lower one
    double given;                            // P or Q of the drafted token
    float lmax;
    uint32_t weight;                         // kept weight of the drafted token
};

__device__ __forceinline__ RowSettings settings_of(const VerifyParams& p, int64_t i)
{
    return {p.temperature ? p.temperature[i] : 1.0f, p.top_k ? p.top_k[i] : 0, p.top_p ? p.top_p[i] : 1.0f,
            p.min_p ? p.min_p[i] : 0.0f, 0.0f};
}

// A row's distribution.
struct Dist {
    Row r;
    uint64_t total, last;
    double unit;                             // 2^40 / total
    uint32_t floor_w;
    bool greedy;

    // Kept weight of column i with logit l.
    __device__ __forceinline__ uint32_t kept(float l, int i) const
    {
        const uint64_t at = place(order_key(l), i);
        if (greedy)
            return at == last && total ? 1u : 0u;
        const uint32_t w = weight(r, l);
        return w >= floor_w && at >= last && total ? w : 0u;
    }
    __device__ __forceinline__ double probability(uint32_t w) const { return rint((double)w * unit); }
};

__device__ __forceinline__ Dist dist_from(uint64_t total, uint64_t last, float lmax, const RowSettings& set)
{
    Dist d{};
    set_inverse(d.r, set.temperature);
    set_maximum(d.r, lmax);
    d.total = total;
    d.last = last;
    d.unit = total ? kUnit / (double)total : 0.0;
    d.floor_w = weight_floor(set.min_p);
    d.greedy = !(set.temperature > 0.0f);
    return d;
}

struct ToWorkspace {
    static constexpr bool kDraw = false;
    Cut* cut;
    RowSettings set;
    int x;                                   // the drafted token, -1: none
    float logit_x;

    __device__ __forceinline__ void kept(float lmax, uint64_t total, uint64_t last) const
    {
        const Dist d = dist_from(total, last, lmax, set);
        const uint32_t w = x >= 0 ? d.kept(logit_x, x) : 0;
        *cut = {total, last, d.probability(w), lmax, w};
    }
    __device__ __forceinline__ void first(uint64_t top) const { kept(0.0f, top ? 1 : 0, top); }
    __device__ __forceinline__ void none() const { kept(0.0f, 0, 0); }
};

// Where a sequence's drafts end: the first number that is no token.  The whole wave.
__device__ __forceinline__ int drafts_of(const VerifyParams& p, int64_t i)
{
    const int lane = threadIdx.x & 63;
    const int32_t x = lane < p.n ? p.drafted[i * p.n + lane] : -1;
    return __builtin_ctzll(__ballot(x < 0 || x >= p.V));
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_verify_rows(VerifyParams p)
{
    __shared__ Lds lds;
    const int64_t rows = p.B * (p.n + 1), row = blockIdx.x;
    const bool draft = row >= rows;
    const int64_t at = draft ? row - rows : row;
    const int per = draft ? p.n : p.n + 1;
    const int64_t i = at / per;
    const int j = (int)(at - i * per), n = drafts_of(p, i);
    if (draft ? j >= n : j > n)              // behind the sequence's drafts
        return;
    Row r;
    r.logits = static_cast<const char*>(draft ? p.draft : p.target) + at * (draft ? p.ld_d : p.ld_t) * (BF16 ? 2 : 4);
    r.bf16 = BF16;
    const int x = j < n ? p.drafted[i * p.n + j] : -1;
    const RowSettings set = settings_of(p, i);
    sample_row<BF16>(ToWorkspace{static_cast<Cut*>(p.workspace) + row, set, x, x >= 0 ? logit(r, x) : 0.0f}, r.logits, p.V,
                     set, lds);
}

__device__ __forceinline__ Dist dist_of(const VerifyParams& p, bool bf16, bool draft, int64_t i, int j,
                                        const RowSettings& set)
{
    const int64_t at = draft ? i * p.n + j : i * (p.n + 1) + j;
    const Cut& cut = static_cast<const Cut*>(p.workspace)[draft ? p.B * (p.n + 1) + at : at];
    Dist d = dist_from(cut.total, cut.last, cut.lmax, set);
    d.r.logits = static_cast<const char*>(draft ? p.draft : p.target) + at * (draft ? p.ld_d : p.ld_t) * (bf16 ? 2 : 4);
    d.r.bf16 = bf16;
    d.r.V = p.V;
    return d;
}

struct Verdict {
    int accepted;
    bool rejected;                           // a token, not the drafts' end, is what follows
    float logprob;                           // of this lane's token, if it is accepted
};

__device__ __forceinline__ float log_of(uint32_t w, uint64_t total)
{
    return logf((float)((double)w / (double)total));
}

// The accepted tokens of sequence i; the whole wave, lane j tests x_j.  All it reads is asked
// for at once; what lies behind the drafts' end was not written and is not looked at.
__device__ __forceinline__ Verdict verdict_of(const VerifyParams& p, int64_t i)
{
    const int lane = threadIdx.x & 63;
    const Cut* cuts = static_cast<const Cut*>(p.workspace);
    const int j = min(lane, max(p.n - 1, 0));
    const float u = p.u[i * (p.n + 1) + j];
    const Cut& t = cuts[i * (p.n + 1) + j];
    const double P = t.given;
    const uint32_t w = t.weight;
    const uint64_t total = t.total;
    const double Q = p.draft ? cuts[p.B * (p.n + 1) + i * p.n + j].given : kUnit;
    const int n = drafts_of(p, i);
    const bool ok = lane < n && (u > 0.0f ? (double)u * Q : 0.0) < P;
    Verdict v;
    v.logprob = ok ? log_of(w, total) : 0.0f;
    v.accepted = __builtin_ctzll(~__ballot(ok));               // lane 63 tests nothing
    v.rejected = v.accepted < n;
    return v;
}

// The numbers that sequence i's next token is drawn from.
struct Source {
    Dist t, d;
    bool rejected, with_draft;
    int x;

    // Of column i: the target's weight, and max(P - Q, 0) where a token was rejected.
    __device__ __forceinline__ void at(float lt, float ld, int i, uint32_t& w, uint64_t& rest) const
    {
        w = t.kept(lt, i);
        rest = 0;
        if (rejected && w) {
            const double q = with_draft ? d.probability(d.kept(ld, i)) : i == x ? kUnit : 0.0;
            const double diff = t.probability(w) - q;
            rest = diff > 0.0 ? (uint64_t)diff : 0;
        }
    }
};

__device__ __forceinline__ Source source_of(const VerifyParams& p, bool bf16, int64_t i, const Verdict& v,
                                            const RowSettings& set)
{
    Source s;
    s.t = dist_of(p, bf16, false, i, v.accepted, set);
    s.rejected = v.rejected;
    s.with_draft = v.rejected && p.draft;
    s.x = v.rejected ? p.drafted[i * p.n + v.accepted] : -1;
    s.d = s.t;
    if (s.with_draft)
        s.d = dist_of(p, bf16, true, i, v.accepted, set);
    return s;
}

__host__ __device__ int64_t cuts(int64_t B, int64_t n) { return B * (2 * n + 1); }

struct Sums {
    unsigned long long w, rest;
};

// Segments of a sequence whose sums are kept at most: a larger vocabulary has larger ones.
constexpr int kMaxSegments = 256;

__host__ __device__ int segment_length(int64_t V)
{
    const int64_t even = (V + kMaxSegments - 1) / kMaxSegments;
    return (int)(even > kSegment ? even : kSegment);
}

__host__ __device__ int segments(int64_t V) { return (int)((V + segment_length(V) - 1) / segment_length(V)); }

__device__ __forceinline__ Sums* sums_of(const VerifyParams& p)
{
    return reinterpret_cast<Sums*>(static_cast<Cut*>(p.workspace) + cuts(p.B, p.n));
}

template <bool BF16>
__global__ void __launch_bounds__(kSumThreads) k_verify_sums(VerifyParams p, int segs)
{
    __shared__ uint64_t part[2][kSumThreads / 64];
    const int64_t i = blockIdx.x / (uint32_t)segs;
    const int seg = (int)(blockIdx.x % (uint32_t)segs), len = segment_length(p.V);
    const RowSettings set = settings_of(p, i);
    const Source s = source_of(p, BF16, i, verdict_of(p, i), set);
    const int end = min(p.V, (seg + 1) * len);
    uint64_t sw = 0, sr = 0;
#pragma unroll 8
    for (int c = seg * len + threadIdx.x; c < end; c += kSumThreads) {
        uint32_t w;
        uint64_t rest;
        s.at(logit(s.t.r, c), s.with_draft ? logit(s.d.r, c) : 0.0f, c, w, rest);
        sw += w;
        sr += rest;
    }
    sw = wave_sum(sw);
    sr = wave_sum(sr);
    if ((threadIdx.x & 63) == 0) {
        part[0][threadIdx.x >> 6] = sw;
        part[1][threadIdx.x >> 6] = sr;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        sw = sr = 0;
        for (int w = 0; w < kSumThreads / 64; ++w) {
            sw += part[0][w];
            sr += part[1][w];
        }
        sums_of(p)[blockIdx.x] = {sw, sr};
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_verify_draw(VerifyParams p, int segs)
{
    __shared__ uint64_t scan[kWaves];
    __shared__ uint64_t pick_sum, sum;
    __shared__ int pick;
    const int64_t i = blockIdx.x;
    const RowSettings set = settings_of(p, i);
    const Verdict v = verdict_of(p, i);
    const Source s = source_of(p, BF16, i, v, set);
    // sums of the segments, a thread each
    static_assert(kMaxSegments <= kThreads, "");
    Sums mine{0, 0};
    if ((int)threadIdx.x < segs)
        mine = sums_of(p)[i * segs + threadIdx.x];
    uint64_t upto_w = block_scan(mine.w, scan);
    uint64_t upto_r = block_scan(mine.rest, scan);
    if (threadIdx.x == kThreads - 1) {
        pick_sum = upto_w;
        sum = upto_r;
    }
    __syncthreads();
    const uint64_t total_w = pick_sum, total_r = sum;
    const bool by_rest = total_r > 0;
    const uint64_t total = by_rest ? total_r : total_w;
    __syncthreads();
    int token = -1;
    uint32_t weight_at = 0;
    if (total) {
        const uint64_t t = target(p.u[i * (p.n + 1) + p.n], total);
        const uint64_t upto = by_rest ? upto_r : upto_w, own = by_rest ? mine.rest : mine.w;
        if (upto > t && upto - own <= t) {
            pick = threadIdx.x;
            pick_sum = upto - own;
        }
        __syncthreads();
        const int len = segment_length(p.V), per = (len + kThreads - 1) / kThreads;
        const int first = pick * len + threadIdx.x * per;
        const int end = min(min(first + per, (pick + 1) * len), p.V);
        const uint64_t before = pick_sum;
        uint64_t here = 0;
        for (int c = first; c < end; ++c) {
            uint32_t w;
            uint64_t rest;
            s.at(logit(s.t.r, c), s.with_draft ? logit(s.d.r, c) : 0.0f, c, w, rest);
            here += by_rest ? rest : w;
        }
        uint64_t at = block_scan(here, scan) - here + before;
        __syncthreads();
        if (at <= t && t < at + here) {
            for (int c = first; c < end; ++c) {
                uint32_t w;
                uint64_t rest;
                s.at(logit(s.t.r, c), s.with_draft ? logit(s.d.r, c) : 0.0f, c, w, rest);
                const uint64_t x = by_rest ? rest : w;
                if (at <= t && t < at + x) {
                    pick = c;
                    sum = w;
                }
                at += x;
            }
        }
        __syncthreads();
        token = pick;
        weight_at = (uint32_t)sum;
    }
    if ((int)threadIdx.x > p.n)
        return;
    const int j = threadIdx.x;
    const int64_t out = i * (p.n + 1) + j;
    p.tokens[out] = j < v.accepted ? p.drafted[i * p.n + j] : j == v.accepted ? token : -1;
    if (p.logprobs)
        p.logprobs[out] = j < v.accepted ? v.logprob
                          : j == v.accepted && token >= 0 ? log_of(weight_at, s.t.total) : -INFINITY;
    if (j == 0)
        p.accepted[i] = v.accepted;
}

template <bool BF16>
void launch(const VerifyParams& p, hipStream_t st)
{
    const int segs = segments(p.V);
    const int64_t rows = p.B * (p.n + 1) + (p.draft ? p.B * p.n : 0);
    hipLaunchKernelGGL(k_verify_rows<BF16>, dim3((unsigned)rows), dim3(kThreads), 0, st, p);
    hipLaunchKernelGGL(k_verify_sums<BF16>, dim3((unsigned)(p.B * segs)), dim3(kSumThreads), 0, st, p, segs);
    hipLaunchKernelGGL(k_verify_draw<BF16>, dim3((unsigned)p.B), dim3(kThreads), 0, st, p, segs);
}

}  // namespace

int64_t verify_workspace(int64_t B, int64_t n)
{
    return cuts(B, n) * (int64_t)sizeof(Cut) + B * kMaxSegments * (int64_t)sizeof(Sums);
}

int64_t verify_threads(int64_t B, int64_t n, int64_t V)
{
    const int64_t rows = cuts(B, n) * kThreads, sums = B * segments(V) * kSumThreads;
    return rows > sums ? rows : sums;
}

hipError_t launch_verify(const VerifyParams& p, bool bf16, hipStream_t st)
{
    bf16 ? launch<true>(p, st) : launch<false>(p, st);
    return hipGetLastError();
}

}  // namespace lora
