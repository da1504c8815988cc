// k_token.hip -- log probabilities of given tokens with entropy and the top alternatives from
// logits (zo_token_logprobs), and the mean negative log probability of groups of rows
// (zo_group_loss).
//
// One pass over a row keeps, per thread, the running maximum m and the sums
//   s = sum_v e^{x_v - m},   t = sum_v e^{x_v - m} (x_v - m);
// a larger maximum m' rescales them by r = e^{m - m'}: s <- s r, t <- (t + s (m - m')) r, and
// two partial rows merge the same way.  Then lse = m + log s, logp = (x_t - m) - log s and the
// entropy is log s - t / s, all in fp32.
#include <math.h>

#include <type_traits>

#include "zo_lm.hpp"

namespace zo {
namespace {

template <class T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen<float>(float v) { return v; }
template <>
__device__ __forceinline__ float widen<uint16_t>(uint16_t v) { return bf16lo_to_f32(v); }

// A 64-bit key that orders values (all NaN equal and above +inf, -0 equal to +0), then lower
// indices first.  Never 0 nor ~0, which stand for no key and for the bound above all keys.
__device__ __forceinline__ uint64_t top_key(float x, uint32_t idx)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    if (x != x) o = 0xFFFFFFFEu;        // a NaN again in key_value
    return ((uint64_t)o << 32) | (uint64_t)(0xFFFFFFFFu - idx);
}

// The value of a key (of -0: +0).
__device__ __forceinline__ float key_value(uint64_t key)
{
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// One row: elements [0, head) up to a 16-byte boundary, then `pieces` of 16 bytes, then the
// rest.
template <class T>
struct Row {
    static constexpr uint32_t kPiece = 16 / sizeof(T);
    const T *p;
    uint32_t vocab, head, pieces;

    __device__ __forceinline__ Row(const T *row, uint32_t v) : p(row), vocab(v)
    {
        head = (uint32_t)(-(intptr_t)row & 15) / sizeof(T);
        head = head < vocab ? head : vocab;
        pieces = (vocab - head) / kPiece;
    }
    __device__ __forceinline__ uint32_t rest() const { return head + pieces * kPiece; }
    // kOnce: not looked at again, so not kept in the caches.
    template <bool kOnce = false>
    __device__ __forceinline__ u32x4 piece(uint32_t i) const
    {
        const u32x4 *at = reinterpret_cast<const u32x4 *>(p + head + (uint64_t)i * kPiece);
        if constexpr (kOnce) return __builtin_nontemporal_load(at);
        else return *at;
    }
    static __device__ __forceinline__ float value(const u32x4 &v, int i)
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(v[i]);
        else return i & 1 ? bf16hi_to_f32(v[i >> 1]) : bf16lo_to_f32(v[i >> 1]);
    }
    // -inf in every value.
    static __device__ __forceinline__ u32x4 nothing()
    {
        const uint32_t w = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
        return u32x4{w, w, w, w};
    }
};


// The place of each of 64 keys (one per lane, 0: none) among them, largest first.
__device__ __forceinline__ uint32_t rank_in_wave(uint64_t key, const uint64_t *keys)
{
    uint32_t r = 0;
#pragma unroll 8
    for (int i = 0; i < kWave; ++i) r += keys[i] > key ? 1u : 0u;
    return r;
}

// The k-th largest of 64 keys, or 1 if fewer than k are there: a lower bound of the k-th
// largest of everything those keys are maxima of.
__device__ __forceinline__ uint64_t bound_of(const uint64_t *keys, uint32_t k)
{
    const uint64_t key = keys[threadIdx.x & (kWave - 1)];
    const uint32_t r = rank_in_wave(key, keys);
    const uint64_t who = __ballot(key != 0 && r == k - 1);
    return who ? keys[__ffsll((unsigned long long)who) - 1] : 1;
}

// One workgroup per row, one pass over it: each thread loads four pieces, takes their largest
// value first (it rescales the sums at most once per four pieces) and adds up.  Many rows are
// bound by VALU issue (98% of the cycles) close to HBM's rate, once they are read past the caches
// (16384 bf16 rows of 50272: 257 us, 6.4 TB/s): a value costs 11.3 issue slots (widen, half a
// max3, scale and subtract, an exponential of four, add, bound, multiply-add); with one more,
// sums against e, it took 268 us.  Few rows are bound by the latency of a round of loads and of the search.  Rows whose statistics leave
// BinaryStats' reach are passed over again in SoftStats (3.3 times the time, if all do).
//
// Alternatives.  The maxima of 64 parts of the row (one per kThreads / 64 threads) are at hand
// from the pass; the k-th largest of them bounds the k-th largest value from below, so only
// the pieces of threads whose own maximum reaches that bound are looked through again (the
// row is in L2 by then), for a few more than k candidates, which are ranked by counting.  Keys hold
// value and index, so ties neither widen the search nor leave the order open.  Rows where
// that does not hold (NaN, only -inf, or more candidates than fit) take k passes of a search
// for the largest key below the last.
template <class T, int kThreads, bool kOnce>
__global__ __launch_bounds__(kThreads) void k_token(
    const T *logits, uint32_t vocab, uint64_t stride, const int64_t *targets, float *logp,
    float *entropy, uint32_t top_k, int64_t *top_ids, float *top_logp)
{
    constexpr int kWaves = kThreads / kWave;
    // pieces a thread loads before it uses them; where a row has a workgroup's latency to itself,
    // fewer leave less of the last, short round (one row of 50272 bf16, top 20: 13.0 us; 14.5
    // with four, 15.1 with eight)
    constexpr int kUnroll = kThreads == 1024 ? 2 : 4;
    constexpr uint32_t kNone = 0xFFFFFFFFu, kHead = 0xFFFFFFFEu, kRest = 0xFFFFFFFDu;
    // keys that the search for the alternatives can hold: rows of one value everywhere bring up
    // to 32 pieces per thread of a part
    constexpr uint32_t kCandidates = kThreads == 64 ? 512 : 2048;
    const uint64_t at = blockIdx.x;
    const int tid = threadIdx.x;
    const int64_t tgt = targets ? targets[at] : 0;
    if (targets && tgt == kIgnoreToken) {
        if (tid == 0) {
            logp[at] = 0.0f;
            if (entropy) entropy[at] = 0.0f;
        }
        for (uint32_t i = tid; i < top_k; i += kThreads) {
            top_ids[at * top_k + i] = -1;
            top_logp[at * top_k + i] = 0.0f;
        }
        return;
    }
    const Row<T> row(logits + at * stride, vocab);
    constexpr int kPiece = Row<T>::kPiece;
    float target = __builtin_nanf("");
    if (tid == 0 && targets && tgt >= 0 && tgt < (int64_t)vocab) target = widen(row.p[tgt]);
    BinaryStats st = BinaryStats::empty();
    float best = -INFINITY;     // largest value of this thread, and where it was first seen
    uint32_t where = kNone;
    const auto one = [&](float x, uint32_t place) {
        st.raise(x);
        st.add(x);
        if (x > best || where == kNone) {
            best = fmaxf(x, best);
            where = place;
        }
    };
    if ((uint32_t)tid < row.head) one(widen(row.p[tid]), kHead);
    for (uint32_t i = tid; i < row.pieces; i += kUnroll * kThreads) {
        u32x4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            v[u] = i + u * kThreads < row.pieces ? row.template piece<kOnce>(i + u * kThreads)
                                                 : Row<T>::nothing();
        float x[kUnroll * kPiece];
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < kUnroll * kPiece; ++j) {
            x[j] = Row<T>::value(v[j / kPiece], j % kPiece);
            top = fmaxf(top, x[j]);
        }
        if (top > best || where == kNone) {
            best = top;
            where = i;
        }
        st.raise(top);
#pragma unroll
        for (int j = 0; j < kUnroll * kPiece; ++j) st.add(x[j]);
    }
    if (row.rest() + tid < vocab) one(widen(row.p[row.rest() + tid]), kRest);

    __shared__ float parts[kWaves][3];
    const auto leave = [&](SoftStats own) {
        own.wave_merge();
        if ((tid & (kWave - 1)) == 0) {
            parts[tid / kWave][0] = own.m;
            parts[tid / kWave][1] = own.s;
            parts[tid / kWave][2] = own.t;
        }
    };
    const auto join = [&] {
        SoftStats a = {parts[0][0], parts[0][1], parts[0][2]};
        for (int w = 1; w < kWaves; ++w) a.merge({parts[w][0], parts[w][1], parts[w][2]});
        return a;
    };
    leave(st.natural());
    // The first largest element of each part, exactly: by the threads that hold its value.
    __shared__ uint64_t tops[kWave];
    __shared__ uint32_t found, flagged;
    if (top_k) {
        float part = best;
#pragma unroll
        for (int o = 1; o < kThreads / kWave; o <<= 1) part = fmaxf(part, __shfl_xor(part, o));
        uint64_t key = 0;
        if (best < part) {
        } else if (where == kHead) {
            key = top_key(best, tid);
        } else if (where == kRest) {
            key = top_key(best, row.rest() + tid);
        } else if (where != kNone) {
#pragma unroll
            for (int u = kUnroll - 1; u >= 0; --u) {
                const uint32_t i = where + u * kThreads;
                if (i >= row.pieces) continue;
                const u32x4 v = row.piece(i);
#pragma unroll
                for (int j = kPiece - 1; j >= 0; --j)
                    if (Row<T>::value(v, j) == best) key = top_key(best, row.head + i * kPiece + j);
            }
        }
#pragma unroll
        for (int o = 1; o < kThreads / kWave; o <<= 1) {
            const uint64_t other = __shfl_xor(key, o);
            key = other > key ? other : key;
        }
        if (tid % (kThreads / kWave) == 0) tops[tid / (kThreads / kWave)] = key;
        if (tid == 0) found = flagged = 0;
    }
    __syncthreads();
    SoftStats all = join();
    if (!BinaryStats::holds(all)) {
        SoftStats own = SoftStats::empty();
        for (uint32_t v = tid; v < vocab; v += kThreads) {
            const float x = widen(row.p[v]);
            own.raise(x);
            own.add(x);
        }
        __syncthreads();
        leave(own);
        __syncthreads();
        all = join();
    }
    const float logs = logf(all.s);
    if (tid == 0) {
        if (targets) logp[at] = (target - all.m) - logs;
        if (entropy) entropy[at] = logs - all.t / all.s;
    }
    if (!top_k) return;

    const auto give = [&](uint32_t place, uint64_t k) {
        top_ids[at * top_k + place] = 0xFFFFFFFFu - (uint32_t)k;
        top_logp[at * top_k + place] = (key_value(k) - all.m) - logs;
    };
    __shared__ uint64_t list[kCandidates];
    const bool plain = all.s == all.s && all.m > -INFINITY;
    if (plain) {
        const uint64_t bound = bound_of(tops, top_k);
        const auto take = [&](float x, uint32_t idx) {
            const uint64_t k = top_key(x, idx);
            if (k < bound) return;
            const uint32_t n = atomicAdd(&found, 1u);
            if (n < kCandidates) list[n] = k;
        };
        __shared__ uint16_t flags[kThreads];
        if (where != kNone && top_key(best, 0) >= bound) {
            flags[atomicAdd(&flagged, 1u)] = (uint16_t)tid;
            if ((uint32_t)tid < row.head) take(widen(row.p[tid]), tid);
            if (row.rest() + tid < vocab) take(widen(row.p[row.rest() + tid]), row.rest() + tid);
        }
        __syncthreads();
        // all threads share the flagged ones' pieces, so that their loads are in flight at once
        const uint32_t per = (row.pieces + kThreads - 1) / kThreads, items = flagged * per;
        for (uint32_t w = tid; w < items; w += kThreads) {
            const uint32_t i = flags[w / per] + w % per * kThreads;
            if (i >= row.pieces) continue;
            const u32x4 v = row.piece(i);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) take(Row<T>::value(v, j), row.head + i * kPiece + j);
        }
        __syncthreads();
        uint32_t n = found;
        if (n <= kCandidates) {
            if (n > 2 * kWave) {
                // many in one place of the row: bound them once more by the list's own parts
                __syncthreads();
                if (tid < kWave) {
                    uint64_t k = 0;
                    for (uint32_t i = tid; i < n; i += kWave) k = list[i] > k ? list[i] : k;
                    tops[tid] = k;
                }
                if (tid == 0) found = 0;
                __syncthreads();
                const uint64_t again = bound_of(tops, top_k);
                uint64_t mine[kCandidates / kThreads];
#pragma unroll
                for (uint32_t i = 0; i < kCandidates / kThreads; ++i)
                    mine[i] = i * kThreads + tid < n ? list[i * kThreads + tid] : 0;
                __syncthreads();
#pragma unroll
                for (uint32_t i = 0; i < kCandidates / kThreads; ++i)
                    if (mine[i] >= again && mine[i]) list[atomicAdd(&found, 1u)] = mine[i];
                __syncthreads();
                n = found;
            }
            for (uint32_t i = tid; i < n; i += kThreads) {
                const uint64_t k = list[i];
                uint32_t place = 0;
                for (uint32_t j = 0; j < n; ++j) place += list[j] > k ? 1u : 0u;
                if (place < top_k) give(place, k);
            }
            return;
        }
    }
    uint64_t below = ~(uint64_t)0;
    for (uint32_t i = 0; i < top_k; ++i) {
        uint64_t k = 0;
        for (uint32_t v = tid; v < vocab; v += kThreads) {
            const uint64_t c = top_key(widen(row.p[v]), v);
            if (c < below && c > k) k = c;
        }
        for (int o = kWave / 2; o; o >>= 1) {
            const uint64_t c = __shfl_xor(k, o);
            k = c > k ? c : k;
        }
        __syncthreads();
        if ((tid & (kWave - 1)) == 0) tops[tid / kWave] = k;
        __syncthreads();
        for (int w = 0; w < kWaves; ++w) k = tops[w] > k ? tops[w] : k;
        if (tid == 0) give(i, k);
        below = k;
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
    // Few long rows (up to two per CU): all of a row's loads should be in flight at once, so
    // 1024 threads take it.  Many rows hide each other's latency, and the search for
    // alternatives, serial within a row, should hold up few threads while the pass needs enough
    // of them.  Measured at 8192 rows, no / 32 alternatives, with 64, 256 and 512 threads:
    // 8 KB a row 17/35, 29/50, 56/88 us; 16 KB 27/66, 30/59, 56/95; 32 KB 57/144, 53/96, 60/121;
    // 64 KB 94/312, 92/162, 88/145.
    // Logits that the last cache does not hold are read past the caches, unless the search
    // wants their rows again: 4096 bf16 rows of 50272 (412 MB) just written 96 -> 79 us, else
    // 80 -> 74, 16384 rows 282 -> 257; 2048 rows (206 MB) just written 35 -> 41, so smaller ones
    // are not.  With alternatives 2051 fp32 rows of 32003, half ignored, 34 -> 36.
    const auto launch = [&](auto *p, auto threads, auto once) {
        using E = std::remove_cv_t<std::remove_pointer_t<decltype(p)>>;
        constexpr int kThreads = decltype(threads)::value;
        const auto from = [](auto *base, uint64_t i) { return base ? base + i : base; };
        // a launch holds fewer than 2^32 threads
        constexpr uint64_t kRows = kLaunchThreads / kThreads;
        hipError_t e = hipSuccess;
        for (uint64_t r = 0; r < rows && e == hipSuccess; r += kRows) {
            const uint32_t n = (uint32_t)(rows - r < kRows ? rows - r : kRows);
            k_token<E, kThreads, decltype(once)::value><<<n, kThreads, 0, stream>>>(
                p + r * stride, vocab, stride, from(targets, r), from(logp, r), from(entropy, r), top_k,
                from(top_ids, r * top_k), from(top_logp, r * top_k));
            e = hipGetLastError();
        }
        return e;
    };
    const auto typed = [&](auto *p) {
        const uint64_t bytes = (uint64_t)vocab * sizeof(*p);
        const std::false_type kept;
        const std::true_type once;
        if (rows <= 512 && bytes >= 32768) return launch(p, std::integral_constant<int, 1024>(), kept);
        if (top_k && bytes >= 65536) return launch(p, std::integral_constant<int, 512>(), kept);
        const std::integral_constant<int, 64> wave;
        const std::integral_constant<int, 256> waves;
        if (top_k || rows * bytes <= kLastCache)
            return bytes <= 12288 ? launch(p, wave, kept) : launch(p, waves, kept);
        return bytes <= 12288 ? launch(p, wave, once) : launch(p, waves, once);
    };
    return bf16 ? typed(static_cast<const uint16_t *>(logits)) : typed(static_cast<const float *>(logits));
}

hipError_t launch_group_loss(const float *logp, const int64_t *targets, const int64_t *starts,
                             uint32_t n_groups, uint64_t rows, double *loss, hipStream_t stream)
{
    constexpr uint32_t kGroups = kLaunchThreads / kGroupThreads;
    hipError_t e = hipSuccess;
    for (uint64_t g = 0; g < n_groups && e == hipSuccess; g += kGroups) {
        const uint32_t n = n_groups - g < kGroups ? (uint32_t)(n_groups - g) : kGroups;
        k_group_loss<<<n, kGroupThreads, 0, stream>>>(logp, targets, starts + g, rows, loss + g);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace zo
