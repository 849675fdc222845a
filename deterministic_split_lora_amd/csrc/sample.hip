// One token per row of logits: temperature, top-k, top-p, min-p and a draw
// from a given random number (sample_row.h has the steps).
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
#include "sample_row.h"

namespace lora {

namespace {

// The draw's results.
struct Drawn {
    static constexpr bool kDraw = true;
    const SampleParams& p;
    int64_t row;

    __device__ __forceinline__ void write(int token, float logprob) const
    {
        p.tokens[row] = token;
        if (p.logprobs)
            p.logprobs[row] = logprob;
    }
    __device__ __forceinline__ void token(int token, uint32_t w, uint64_t total) const
    {
        write(token, logf((float)((double)w / (double)total)));
    }
    __device__ __forceinline__ void first(uint64_t top) const
    {
        write(top ? (int)place_column(top) : -1, top ? 0.0f : -INFINITY);
    }
    __device__ __forceinline__ void none() const { write(-1, -INFINITY); }
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_sample(SampleParams p)
{
    __shared__ Lds lds;
    const int64_t row = blockIdx.x;
    const RowSettings set{p.temperature ? p.temperature[row] : 1.0f, p.top_k ? p.top_k[row] : 0,
                          p.top_p ? p.top_p[row] : 1.0f, p.min_p ? p.min_p[row] : 0.0f, p.u[row]};
    sample_row<BF16>(Drawn{p, row}, static_cast<const char*>(p.logits) + row * p.ld * (BF16 ? 2 : 4), p.V, set, lds);
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
