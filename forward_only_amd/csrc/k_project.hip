// k_project.hip -- the products of zo_adapter_project, y = x w^T + bias + scale (x A_g^T) B_g^T, each
// group of rows with its own low-rank adapter, moved along its own probe while it is read, and of
// zo_head_logprobs, softmax statistics of every row over all features, with the product itself
// kept in registers.
#include "zo_product.hpp"

namespace zo {
namespace {

// ---- joining the head's partial statistics ----------------------------------------------

// The places of the rows that count, in order, and zeros for the others' outputs; how many are in
// each of `pieces` pieces of so many places.  One workgroup, eight rows of a thread in flight at
// once.
__global__ __launch_bounds__(1024) void k_counted(const int64_t *targets, uint64_t rows,
                                                  uint32_t *list, uint32_t *count, float *logp,
                                                  float *entropy, uint64_t piece, uint32_t pieces,
                                                  uint32_t *counts)
{
    constexpr int kAtOnce = 8;
    __shared__ uint32_t waves[kAtOnce][16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t at = 0;
    for (uint64_t r0 = 0; r0 < rows; r0 += 1024 * kAtOnce) {
        int64_t t[kAtOnce];
        uint64_t votes[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const uint64_t r = r0 + i * 1024 + tid;
            t[i] = targets[r < rows ? r : 0];
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            votes[i] = __ballot(r0 + i * 1024 + tid < rows && t[i] != kIgnoreToken);
            if (lane == 0) waves[i][wave] = __popcll(votes[i]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            uint32_t before = at;
            for (int w = 0; w < 16; ++w) {
                if (w < wave) before += waves[i][w];
                at += waves[i][w];
            }
            const uint64_t r = r0 + i * 1024 + tid;
            if (votes[i] >> lane & 1) {
                list[before + __popcll(votes[i] & (((uint64_t)1 << lane) - 1))] = (uint32_t)r;
            } else if (r < rows) {
                if (logp) logp[r] = 0.0f;
                if (entropy) entropy[r] = 0.0f;
            }
        }
        __syncthreads();
    }
    if (tid == 0) *count = at;
    for (uint32_t i = tid; i < pieces; i += 1024)
        counts[i] = at <= i * piece ? 0 : (uint32_t)(at - i * piece < piece ? at - i * piece : piece);
}

// Joins the parts of each place: kOf places per workgroup of 1024 threads.  Eight read whole
// sectors; one, when there are few rows, has its parts in one or two rounds of loads.
template <int kOf>
__global__ __launch_bounds__(1024) void k_head_join(const float *m, const float *s, const float *t,
                                                    const float *tl, uint32_t parts, uint64_t base,
                                                    uint64_t rows, const uint32_t *list,
                                                    const uint32_t *count, const int64_t *targets,
                                                    uint32_t features, float *logp, float *entropy,
                                                    float2 *norms)
{
    const uint64_t n = places(base, rows, count);
    const int of = threadIdx.x % kOf, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t at = (uint64_t)blockIdx.x * kOf + of;
    if ((uint64_t)blockIdx.x * kOf >= n) return;
    SoftStats st = SoftStats::empty();
    if (at < n)
        for (uint32_t p = threadIdx.x / kOf; p < parts; p += 1024 / kOf)
            st.merge({m[(uint64_t)p * rows + at], s[(uint64_t)p * rows + at],
                      t[(uint64_t)p * rows + at]});
    st.wave_merge(32, kOf);
    __shared__ float all[16][kOf][3];
    if (lane < kOf) {
        all[wave][of][0] = st.m;
        all[wave][of][1] = st.s;
        all[wave][of][2] = st.t;
    }
    __syncthreads();
    if (wave) return;
    st = SoftStats::empty();
#pragma unroll
    for (int w = lane / kOf; w < 16; w += kWave / kOf) st.merge({all[w][of][0], all[w][of][1], all[w][of][2]});
    st.wave_merge(32, kOf);
    if (lane >= kOf || at >= n) return;
    const uint64_t row = list ? list[base + at] : base + at;
    const int64_t tgt = targets ? targets[row] : 0;
    const bool ignore = targets && tgt == kIgnoreToken;
    const float logs = logf(st.s);
    const bool known = tgt >= 0 && tgt < (int64_t)features;
    if (logp) logp[row] = ignore ? 0.0f : known ? (tl[at] - st.m) - logs : __builtin_nanf("");
    if (norms) norms[base + at] = make_float2(st.m, known ? logs : __builtin_nanf(""));
    if (entropy) entropy[row] = ignore ? 0.0f : logs - st.t / st.s;
}

// ---- launches ---------------------------------------------------------------------------

// x A_g^T of all groups, and every row's group behind them; nothing where there are no groups.
template <class T>
hipError_t shrink(const AdapterArgs &a, const typename T::elem *px, uint64_t x_stride,
                  const typename T::elem *pa, float *u, hipStream_t stream)
{
    if (a.n_groups == 0) return hipSuccess;
    int32_t *group = reinterpret_cast<int32_t *>(u + a.rows * a.rank);
    // 32 rows per workgroup where the groups are long enough to fill them and still every CU
    // gets one
    const auto launch = [&](auto kXF, auto kAF) {
        constexpr int kX = decltype(kXF)::value, kA = decltype(kAF)::value;
        k_shrink<T, kX, kA><<<(uint32_t)(a.rows / (16 * kX) + a.n_groups), shrink_waves<kX>() * 64,
                              shrink_lds<kX, kA>(), stream>>>(a, px, x_stride, pa, u, group);
    };
    typedef std::integral_constant<int, 1> One;
    typedef std::integral_constant<int, 2> Two;
    const bool long_groups = a.rows / 32 >= kBigSlots && a.rows / a.n_groups >= 32;
    if (a.rank <= 16)
        long_groups ? launch(Two{}, One{}) : launch(One{}, One{});
    else
        long_groups ? launch(Two{}, Two{}) : launch(One{}, Two{});
    return hipGetLastError();
}

template <class T>
hipError_t project(const AdapterArgs &a, const void *x, uint64_t x_stride, const void *w,
                   const void *bias, const void *adapters, float *u, float *slices, void *y,
                   uint64_t y_stride, hipStream_t stream)
{
    typedef typename T::elem E;
    const E *px = static_cast<const E *>(x), *pa = static_cast<const E *>(adapters);
    const hipError_t e = shrink<T>(a, px, x_stride, pa, u, stream);
    if (e != hipSuccess) return e;
    const int32_t *group = reinterpret_cast<int32_t *>(u + a.rows * a.rank);
    const ProductArgs p = {0, a.rows, x_stride, a.d_in, a.d_out, slices};
    const EndProject<T> end = {a, u, group, pa, static_cast<const E *>(bias), static_cast<E *>(y), y_stride};
    const E *pw = static_cast<const E *>(w);
    return by_shape<T>(product_shape(a.rows, a.d_out, a.d_in, T::kBf16), p, px, pw, nullptr, nullptr, end, stream);
}

template <class T>
hipError_t head(const HeadArgs &h, const void *x, const void *w, hipStream_t stream)
{
    typedef typename T::elem E;
    const HeadSpace sp = head_space(h.rows, h.k, h.features, T::kBf16, h.workspace);
    const bool small = sp.shape == Shape::few;
    uint32_t *list = nullptr, *count = nullptr;
    if (h.targets && !small) {
        list = sp.list;
        count = sp.count;
        const hipError_t e = launch_counted(h.targets, h.rows, list, count, h.logp, h.entropy, stream);
        if (e != hipSuccess) return e;
    }
    const E *px = static_cast<const E *>(x), *pw = static_cast<const E *>(w);
    for (uint64_t base = 0; base < h.rows; base += kHeadPlaces) {
        const uint64_t rows = h.rows - base < kHeadPlaces ? h.rows - base : kHeadPlaces;
        const ProductArgs p = {base, rows, h.x_stride, h.k, h.features, sp.slices};
        const EndHead end = {h.features, base, rows, h.targets, list, count, sp.m, sp.s, sp.t, sp.tl};
        hipError_t e = by_shape<T>(sp.shape, p, px, pw, list, count, end, stream);
        if (e != hipSuccess) return e;
        e = launch_head_join({sp.m, sp.s, sp.t, sp.tl, sp.parts, base, rows, list, count, h.targets, h.features, h.logp,
                              h.entropy, nullptr}, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class T>
hipError_t prepare()
{
    const auto raise = [](auto *kernel, int bytes) {
        return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                   hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    };
    const hipError_t all[] = {
        raise(&k_big<T, EndProject<T>>, 2 * 512 * 128),
        raise(&k_big<T, EndSlice>, 2 * 512 * 128),
        raise(&k_big<T, EndHead>, 2 * 512 * 128),
        raise(&k_shrink<T, 1, 1>, shrink_lds<1, 1>()),
        raise(&k_shrink<T, 1, 2>, shrink_lds<1, 2>()),
        raise(&k_shrink<T, 2, 1>, shrink_lds<2, 1>()),
        raise(&k_shrink<T, 2, 2>, shrink_lds<2, 2>()),
        raise(&k_few<T, 1, 2, false, EndProject<T>>, few_lds<1, 2>()),
        raise(&k_few<T, 1, 2, true, EndProject<T>>, few_lds<1, 2>()),
        raise(&k_few<T, 2, 2, false, EndProject<T>>, few_lds<2, 2>()),
        raise(&k_few<T, 2, 2, true, EndProject<T>>, few_lds<2, 2>()),
        raise(&k_few<T, 2, 4, false, EndProject<T>>, few_lds<2, 4>()),
        raise(&k_few<T, 2, 4, true, EndProject<T>>, few_lds<2, 4>()),
        raise(&k_few<T, 3, 2, false, EndProject<T>>, few_lds<3, 2>()),
        raise(&k_few<T, 3, 2, true, EndProject<T>>, few_lds<3, 2>()),
        raise(&k_few<T, 4, 2, false, EndProject<T>>, few_lds<4, 2>()),
        raise(&k_few<T, 4, 2, true, EndProject<T>>, few_lds<4, 2>()),
        raise(&k_few<T, 1, 2, false, EndHead>, few_lds<1, 2>()),
        raise(&k_few<T, 1, 2, true, EndHead>, few_lds<1, 2>()),
        raise(&k_few<T, 2, 2, false, EndHead>, few_lds<2, 2>()),
        raise(&k_few<T, 2, 2, true, EndHead>, few_lds<2, 2>()),
        raise(&k_few<T, 2, 4, false, EndHead>, few_lds<2, 4>()),
        raise(&k_few<T, 2, 4, true, EndHead>, few_lds<2, 4>()),
        raise(&k_few<T, 3, 2, false, EndHead>, few_lds<3, 2>()),
        raise(&k_few<T, 3, 2, true, EndHead>, few_lds<3, 2>()),
        raise(&k_few<T, 4, 2, false, EndHead>, few_lds<4, 2>()),
        raise(&k_few<T, 4, 2, true, EndHead>, few_lds<4, 2>())};
    for (const hipError_t e : all)
        if (e != hipSuccess) return e;
    return hipSuccess;
}

}  // namespace

hipError_t launch_counted(const int64_t *targets, uint64_t rows, uint32_t *list, uint32_t *count, float *logp,
                          float *entropy, hipStream_t stream, uint64_t piece, uint32_t pieces, uint32_t *counts)
{
    k_counted<<<1, 1024, 0, stream>>>(targets, rows, list, count, logp, entropy, piece, pieces, counts);
    return hipGetLastError();
}

hipError_t launch_head_join(const HeadJoin &j, hipStream_t stream)
{
    const auto join = [&](auto of) {
        constexpr int kOf = decltype(of)::value;
        k_head_join<kOf><<<(uint32_t)((j.rows + kOf - 1) / kOf), 1024, 0, stream>>>(
            j.m, j.s, j.t, j.tl, j.parts, j.base, j.rows, j.list, j.count, j.targets, j.features, j.logp, j.entropy,
            static_cast<float2 *>(j.norms));
    };
    if (j.rows <= 256)
        join(std::integral_constant<int, 1>{});
    else
        join(std::integral_constant<int, 8>{});
    return hipGetLastError();
}

hipError_t prepare_products()
{
    const hipError_t e = prepare<Bf16>();
    return e == hipSuccess ? prepare<Fp32>() : e;
}

hipError_t launch_adapter_project(const AdapterArgs &a, bool bf16, const void *x, uint64_t x_stride,
                                  const void *w, const void *bias, const void *adapters, float *u,
                                  float *slices, void *y, uint64_t y_stride, hipStream_t stream)
{
    return bf16 ? project<Bf16>(a, x, x_stride, w, bias, adapters, u, slices, y, y_stride, stream)
                : project<Fp32>(a, x, x_stride, w, bias, adapters, u, slices, y, y_stride, stream);
}

hipError_t launch_adapter_shrink(const AdapterArgs &a, bool bf16, const void *x, uint64_t x_stride,
                                 const void *adapters, float *u, hipStream_t stream)
{
    const auto typed = [&](auto t) {
        typedef typename decltype(t)::elem E;
        return shrink<decltype(t)>(a, static_cast<const E *>(x), x_stride, static_cast<const E *>(adapters), u, stream);
    };
    return bf16 ? typed(Bf16()) : typed(Fp32());
}

hipError_t launch_head_logprobs(const HeadArgs &h, bool bf16, const void *x, const void *w,
                                hipStream_t stream)
{
    return bf16 ? head<Bf16>(h, x, w, stream) : head<Fp32>(h, x, w, stream);
}

}  // namespace zo
