// k_token.hip -- log probabilities of given tokens with entropy and the top alternatives from
// logits (zo_token_logprobs), and the mean negative log probability of groups of rows
// (zo_group_loss).
//
// One pass over a row keeps, per thread, the running maximum m and the sums
//   s = sum_v e^{x_v - m},   t = sum_v e^{x_v - m} (x_v - m);
// a larger maximum m' rescales them by r = e^{m - m'}: s <- s r, t <- (t + s (m - m')) r, and
// two partial rows merge the same way.  Then lse = m + log s, logp = (x_t - m) - log s and the
// entropy is log s - t / s, all in fp32.
#include <float.h>
#include <math.h>

#include "zo_lm.hpp"

namespace zo {
namespace {

constexpr int kTokenThreads = 256;

template <class T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen<float>(float v) { return v; }
template <>
__device__ __forceinline__ float widen<uint16_t>(uint16_t v) { return bf16lo_to_f32(v); }

// A 64-bit key that orders values (all NaN equal and above +inf, -0 equal to +0), then lower
// indices first.
__device__ __forceinline__ uint64_t top_key(float x, uint32_t idx)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    if (x != x) o = 0xFFFFFFFFu;
    return ((uint64_t)o << 32) | (uint64_t)(0xFFFFFFFFu - idx);
}

template <class T>
__global__ __launch_bounds__(kTokenThreads) void k_token(
    const T *logits, uint32_t vocab, uint64_t stride, const int64_t *targets, float *logp,
    float *entropy, uint32_t top_k, int64_t *top_ids, float *top_logp)
{
    const uint64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const int64_t tgt = targets ? targets[row] : 0;
    if (targets && tgt == kIgnoreToken) {
        if (tid == 0) {
            logp[row] = 0.0f;
            if (entropy) entropy[row] = 0.0f;
        }
        for (uint32_t i = tid; i < top_k; i += kTokenThreads) {
            top_ids[row * top_k + i] = -1;
            top_logp[row * top_k + i] = 0.0f;
        }
        return;
    }
    const T *p = logits + row * stride;
    SoftStats st = SoftStats::empty();
    for (uint32_t v = tid; v < vocab; v += kTokenThreads) {
        const float x = widen(p[v]);
        st.raise(x);
        st.add(x);
    }
    st.wave_merge();
    __shared__ SoftStats parts[kTokenThreads / kWave];
    __shared__ uint64_t keys[kTokenThreads / kWave];
    if ((tid & (kWave - 1)) == 0) parts[tid / kWave] = st;
    __syncthreads();
    st = parts[0];
    for (int w = 1; w < kTokenThreads / kWave; ++w) st.merge(parts[w]);
    const float logs = logf(st.s);
    if (tid == 0) {
        if (targets) {
            float lp = __builtin_nanf("");
            if (tgt >= 0 && tgt < (int64_t)vocab) lp = (widen(p[tgt]) - st.m) - logs;
            logp[row] = lp;
        }
        if (entropy) entropy[row] = logs - st.t / st.s;
    }
    uint64_t below = ~(uint64_t)0;
    for (uint32_t i = 0; i < top_k; ++i) {
        uint64_t best = 0;
        for (uint32_t v = tid; v < vocab; v += kTokenThreads) {
            const uint64_t k = top_key(widen(p[v]), v);
            if (k < below && k > best) best = k;
        }
        for (int o = kWave / 2; o; o >>= 1) {
            const uint64_t k = __shfl_xor(best, o);
            best = k > best ? k : best;
        }
        __syncthreads();
        if ((tid & (kWave - 1)) == 0) keys[tid / kWave] = best;
        __syncthreads();
        for (int w = 0; w < kTokenThreads / kWave; ++w) best = keys[w] > best ? keys[w] : best;
        if (tid == 0) {
            const uint32_t id = 0xFFFFFFFFu - (uint32_t)best;
            top_ids[row * top_k + i] = id;
            top_logp[row * top_k + i] = (widen(p[id]) - st.m) - logs;
        }
        below = best;
    }
}

constexpr int kGroupThreads = 256;

__global__ __launch_bounds__(kGroupThreads) void k_group_loss(
    const float *logp, const int64_t *targets, const int64_t *starts, uint64_t rows, double *loss)
{
    const uint32_t g = blockIdx.x;
    const int tid = threadIdx.x;
    const uint64_t lo = clamp_row(starts[g], rows), hi = clamp_row(starts[g + 1], rows);
    double sum = 0.0;
    uint64_t count = 0;
    for (uint64_t r = lo + tid; r < hi; r += kGroupThreads)
        if (!targets || targets[r] != kIgnoreToken) {
            sum += (double)logp[r];
            ++count;
        }
    for (int o = kWave / 2; o; o >>= 1) {
        sum += __shfl_xor(sum, o);
        count += __shfl_xor(count, o);
    }
    __shared__ double ps[kGroupThreads / kWave];
    __shared__ uint64_t pc[kGroupThreads / kWave];
    if ((tid & (kWave - 1)) == 0) {
        ps[tid / kWave] = sum;
        pc[tid / kWave] = count;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kGroupThreads / kWave; ++w) {
            sum += ps[w];
            count += pc[w];
        }
        loss[g] = -sum / (double)count;   // 0 / 0: a group without counted rows has no loss
    }
}

}  // namespace

hipError_t launch_token_logprobs(const void *logits, bool bf16, uint64_t rows, uint32_t vocab,
                                 uint64_t stride, const int64_t *targets, float *logp,
                                 float *entropy, uint32_t top_k, int64_t *top_ids,
                                 float *top_logp, hipStream_t stream)
{
    if (bf16)
        k_token<uint16_t><<<(uint32_t)rows, kTokenThreads, 0, stream>>>(
            static_cast<const uint16_t *>(logits), vocab, stride, targets, logp, entropy, top_k,
            top_ids, top_logp);
    else
        k_token<float><<<(uint32_t)rows, kTokenThreads, 0, stream>>>(
            static_cast<const float *>(logits), vocab, stride, targets, logp, entropy, top_k,
            top_ids, top_logp);
    return hipGetLastError();
}

hipError_t launch_group_loss(const float *logp, const int64_t *targets, const int64_t *starts,
                             uint32_t n_groups, uint64_t rows, double *loss, hipStream_t stream)
{
    k_group_loss<<<n_groups, kGroupThreads, 0, stream>>>(logp, targets, starts, rows, loss);
    return hipGetLastError();
}

}  // namespace zo
