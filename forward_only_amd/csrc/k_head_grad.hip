// k_head_grad.hip -- log probabilities of given tokens from hidden states h [rows, d] and the
// unembedding matrix W [features, d], with the gradients of -sum_r g_r logp_r (zo_head_grad).
//
//   l = h W^T,  p = softmax(l),  D[r][v] = g_r (p[r][v] - [v = t_r]),  dh = D W,  dW = D^T h
//
// The logits are formed twice and never stored: once for each row's largest and sum
// (zo_head_logprobs), and, when these are known, once more in pieces of the features, of which D
// is left, rounded to the type, as it is and turned over.  Each piece then adds to dh, in fp32, and
// gives its rows of dW.  Rows that do not count are left out: the others stand one after
// another in the workspace, as they are and turned over.  All four products take their operands
// along the neighbouring values that they sum over, so the pieces of W are turned over, too.
#include "zo_product.hpp"

namespace zo {
namespace {

// y[c][r] = x[row(r)][c] for `rows` places r (as many as *count, if given) and `cols` columns c, zeros
// from there to the next multiple of 8 places; kCopy: also copy[r] = x[row(r)].  y's rows lie
// `pitch` apart, a multiple of 8.  A workgroup takes 64 x 64 values through LDS.  What bounds it is
// reading and writing them.
template <class T, bool kCopy>
__global__ __launch_bounds__(256) void k_turn(const typename T::elem *x, uint64_t stride, uint64_t rows,
                                              const uint32_t *count, const uint32_t *list, uint32_t cols,
                                              typename T::elem *y, uint64_t pitch, typename T::elem *copy)
{
    typedef typename T::elem E;
    constexpr int kPiece = T::kPiece, kRowPieces = 64 / kPiece, kPitch = 64 + 4 / (int)sizeof(E);
    __shared__ E tile[64 * kPitch];
    const uint64_t have = places(0, rows, count);
    const uint64_t r0 = (uint64_t)blockIdx.x * 64;
    const uint32_t c0 = blockIdx.y * 64;
    if (r0 >= (have + 7) / 8 * 8) return;
#pragma unroll
    for (int i = threadIdx.x; i < 64 * kRowPieces; i += 256) {
        const int r = i / kRowPieces, c = i % kRowPieces * kPiece;
        u32x4 v = {0, 0, 0, 0};
        if (r0 + r < have && c0 + c < cols) {
            const uint64_t row = list ? list[r0 + r] : r0 + r;
            v = piece_at<T>(x + row * stride + c0 + c);
            if constexpr (kCopy) *reinterpret_cast<u32x4 *>(copy + (r0 + r) * cols + c0 + c) = v;
        }
        const E *e = reinterpret_cast<const E *>(&v);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) tile[r * kPitch + c + j] = e[j];
    }
    __syncthreads();
#pragma unroll
    for (int i = threadIdx.x; i < 64 * kRowPieces; i += 256) {
        const int c = i / kRowPieces, r = i % kRowPieces * kPiece;
        if (c0 + c >= cols || r0 + r >= (have + 7) / 8 * 8) continue;
        u32x4 v;
        E *e = reinterpret_cast<E *>(&v);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) e[j] = tile[(r + j) * kPitch + c];
        *reinterpret_cast<u32x4 *>(y + (uint64_t)(c0 + c) * pitch + r0 + r) = v;
    }
}

// The ending that leaves D of a piece of the features, rounded to the type: d [place][pitch_d] with
// zeros behind the features, dt [feature][pitch_t] with zeros from the last place to the next multiple of 8.
// Either may be nullptr.
template <class T>
struct EndGrad {
    static constexpr bool kSlices = false;
    typedef typename T::elem E;
    uint32_t first, features;      // of this piece
    uint64_t rows;
    const int64_t *targets;
    const uint32_t *list, *count;
    const float2 *norms;
    const float *row_grad;
    E *d, *dt;
    uint64_t pitch_d, pitch_t;

    template <class Tl>
    __device__ __forceinline__ void add_rows(Tl &, int, uint32_t, uint64_t) const {}
    __device__ __forceinline__ uint32_t begin(uint64_t) const { return 0; }
    template <class Tl>
    __device__ __forceinline__ void finish(Tl &tile, uint32_t, uint32_t f0, uint64_t r0, u32x4 *) const
    {
        store(tile, f0, r0);
    }
    static __device__ __forceinline__ void store1(float *p, float v) { *p = v; }
    static __device__ __forceinline__ void store1(uint16_t *p, float v) { *p = (uint16_t)pack_bf16x2(v, 0.0f); }

    template <class Tl>
    __device__ __forceinline__ void store(Tl &tile, uint32_t f0, uint64_t r0) const
    {
        constexpr int kMF = Tl::kMF, kMR = Tl::kMR;
        const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
        const uint64_t have = places(0, rows, count), padded = (have + 7) / 8 * 8;
#pragma unroll
        for (int n = 0; n < kMR; ++n) {
            const uint64_t at = r0 + 16 * n + l16;
            if (at >= padded) continue;
            const bool in = at < have;
            const uint64_t row = in ? list[at] : 0;
            const float2 norm = in ? norms[at] : make_float2(0.0f, 0.0f);
            const float g = in ? (row_grad ? row_grad[row] : 1.0f) : 0.0f;
            const int64_t tgt = in ? targets[row] - first : -1;
#pragma unroll
            for (int m = 0; m < kMF; ++m) {
                const uint32_t f = f0 + 16 * m + 4 * q;
                f32x4 v;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = fast_exp((tile.acc[m][n][i] - norm.x) - norm.y);
                    v[i] = g * (p - (tgt == (int64_t)(f + i) ? 1.0f : 0.0f));
                    if (!in || f + i >= features) v[i] = 0.0f;
                }
                if (d && in && f < pitch_d) EndProject<T>::store4(d + at * pitch_d + f, v);
                if (dt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (f + i < features) store1(dt + (uint64_t)(f + i) * pitch_t + at, v[i]);
            }
        }
    }
};

// The ending that adds a piece's part of dh in fp32.
struct EndSum {
    static constexpr bool kSlices = false;
    uint32_t features;
    uint64_t rows;
    const uint32_t *count;
    float *sum;                    // [place][features]
    bool more;                     // parts are there already

    template <class Tl>
    __device__ __forceinline__ void add_rows(Tl &, int, uint32_t, uint64_t) const {}
    __device__ __forceinline__ uint32_t begin(uint64_t) const { return 0; }
    template <class Tl>
    __device__ __forceinline__ void finish(Tl &tile, uint32_t, uint32_t f0, uint64_t r0, u32x4 *) const
    {
        store(tile, f0, r0);
    }
    template <class Tl>
    __device__ __forceinline__ void store(Tl &tile, uint32_t f0, uint64_t r0) const
    {
        const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
        const uint64_t have = places(0, rows, count);
#pragma unroll
        for (int n = 0; n < Tl::kMR; ++n) {
            const uint64_t at = r0 + 16 * n + l16;
            if (at >= have) continue;
#pragma unroll
            for (int m = 0; m < Tl::kMF; ++m) {
                const uint32_t f = f0 + 16 * m + 4 * q;
                if (f >= features) continue;
                f32x4 *to = reinterpret_cast<f32x4 *>(sum + at * features + f);
                *to = more ? *to + tile.acc[m][n] : tile.acc[m][n];
            }
        }
    }
};

// dh of the counted rows from the sums, rounded once; zeros for the others.
template <class T>
__global__ __launch_bounds__(256) void k_hidden_grad(const float *sum, const int64_t *targets, const uint32_t *list,
                                                     const uint32_t *count, uint64_t rows, uint32_t d,
                                                     typename T::elem *out)
{
    const uint64_t have = places(0, rows, count), each = (rows + gridDim.x - 1) / gridDim.x;
    const uint64_t hi = (blockIdx.x + 1) * each < rows ? (blockIdx.x + 1) * each : rows;
    for (uint64_t at = blockIdx.x * each; at < hi; ++at) {
        if (at < have) {
            const f32x4 *from = reinterpret_cast<const f32x4 *>(sum + at * d);
            typename T::elem *to = out + (uint64_t)list[at] * d;
            for (uint32_t i = threadIdx.x; i < d / 4; i += 256) EndProject<T>::store4(to + 4 * i, from[i]);
        }
        if (targets[at] == kIgnoreToken) {
            typename T::elem *to = out + at * d;
            for (uint32_t i = threadIdx.x; i < d / 4; i += 256) EndProject<T>::store4(to + 4 * i, f32x4{0, 0, 0, 0});
        }
    }
}

__global__ __launch_bounds__(256) void k_zeros(u32x4 *p, uint64_t n)
{
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (uint64_t)gridDim.x * 256) p[i] = u32x4{0, 0, 0, 0};
}

template <class T>
hipError_t head_grad(const HeadGradArgs &h, const void *hidden, const void *weight, hipStream_t stream)
{
    typedef typename T::elem E;
    const HeadGradSpace s = head_grad_space(h.rows, h.d, h.features, T::kBf16, h.workspace);
    E *x = static_cast<E *>(s.x), *xt = static_cast<E *>(s.xt), *wt = static_cast<E *>(s.wt);
    E *d = static_cast<E *>(s.d), *dt = static_cast<E *>(s.dt);
    const E *w = static_cast<const E *>(weight);
    if (h.rows == 0) {
        if (h.weight_grad)
            k_zeros<<<2048, 256, 0, stream>>>(static_cast<u32x4 *>(h.weight_grad), (uint64_t)h.features * h.d / T::kPiece);
        return hipGetLastError();
    }
    hipError_t e = launch_counted(h.targets, h.rows, s.list, s.count, h.logp, nullptr, stream);
    if (e != hipSuccess) return e;
    const auto grid = [](uint64_t rows, uint32_t cols) { return dim3((uint32_t)((rows + 63) / 64), (cols + 63) / 64); };
    k_turn<T, true><<<grid(h.rows, h.d), 256, 0, stream>>>(static_cast<const E *>(hidden), h.x_stride, h.rows, s.count,
                                                           s.list, h.d, xt, s.pitch, x);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    HeadArgs stats = {h.rows, h.d, h.d, h.features, h.targets, h.logp, nullptr, s.head};
    stats.list = s.list;
    stats.count = s.count;
    stats.norms = s.norms;
    e = launch_head_logprobs(stats, T::kBf16, x, w, stream);
    if (e != hipSuccess || (!h.hidden_grad && !h.weight_grad)) return e;
    for (uint32_t i = 0; i < s.pieces; ++i) {
        const uint32_t first = i * s.piece;
        const uint32_t n = h.features - first < s.piece ? h.features - first : s.piece;
        const uint32_t pitch = (n + 7) / 8 * 8;
        const ProductArgs logits = {0, h.rows, h.d, h.d, n, s.slices};
        const EndGrad<T> end = {first, n, h.rows, h.targets, s.list, s.count, static_cast<const float2 *>(s.norms), h.row_grad,
                                h.hidden_grad ? d : nullptr, h.weight_grad ? dt : nullptr, pitch, s.pitch};
        e = by_shape<T>(product_shape(h.rows, n, h.d, T::kBf16), logits, x, w + (uint64_t)first * h.d, nullptr, s.count, end, stream);
        if (e != hipSuccess) return e;
        if (h.hidden_grad) {
            k_turn<T, false><<<grid(n, h.d), 256, 0, stream>>>(w + (uint64_t)first * h.d, h.d, n, nullptr, nullptr, h.d, wt,
                                                               pitch, nullptr);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
            const ProductArgs p = {0, h.rows, pitch, pitch, h.d, s.slices};
            const EndSum sum = {h.d, h.rows, s.count, s.sum, i > 0};
            e = by_shape<T>(product_shape(h.rows, h.d, pitch, T::kBf16), p, d, wt, nullptr, s.count, sum, stream);
            if (e != hipSuccess) return e;
        }
        if (h.weight_grad) {
            const ProductArgs p = {0, n, s.pitch, (uint32_t)s.pitch, h.d, s.slices, s.count};
            AdapterArgs none = {};
            none.rows = n;
            none.d_in = (uint32_t)s.pitch;
            none.d_out = h.d;
            const EndProject<T> out = {none, nullptr, nullptr, nullptr, nullptr,
                                       static_cast<E *>(h.weight_grad) + (uint64_t)first * h.d, h.d};
            e = by_shape<T>(product_shape(n, h.d, (uint32_t)s.pitch, T::kBf16), p, dt, xt, nullptr, nullptr, out, stream);
            if (e != hipSuccess) return e;
        }
    }
    if (h.hidden_grad) {
        k_hidden_grad<T><<<(uint32_t)(h.rows < 4096 ? h.rows : 4096), 256, 0, stream>>>(
            s.sum, h.targets, s.list, s.count, h.rows, h.d, static_cast<E *>(h.hidden_grad));
        e = hipGetLastError();
    }
    return e;
}

template <class T, class End>
hipError_t raise_end()
{
    const auto raise = [](auto *kernel, int bytes) {
        return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    };
    const hipError_t all[] = {
        raise(&k_big<T, End>, 2 * 512 * 128), raise(&k_big<T, EndSlice>, 2 * 512 * 128),
        raise(&k_few<T, 1, 2, false, End>, few_lds<1, 2>()), raise(&k_few<T, 1, 2, true, End>, few_lds<1, 2>()),
        raise(&k_few<T, 2, 2, false, End>, few_lds<2, 2>()), raise(&k_few<T, 2, 2, true, End>, few_lds<2, 2>()),
        raise(&k_few<T, 2, 4, false, End>, few_lds<2, 4>()), raise(&k_few<T, 2, 4, true, End>, few_lds<2, 4>()),
        raise(&k_few<T, 3, 2, false, End>, few_lds<3, 2>()), raise(&k_few<T, 3, 2, true, End>, few_lds<3, 2>()),
        raise(&k_few<T, 4, 2, false, End>, few_lds<4, 2>()), raise(&k_few<T, 4, 2, true, End>, few_lds<4, 2>())};
    for (const hipError_t e : all)
        if (e != hipSuccess) return e;
    return hipSuccess;
}

}  // namespace

hipError_t prepare_head_grad()
{
    const hipError_t all[] = {raise_end<Bf16, EndGrad<Bf16>>(), raise_end<Bf16, EndSum>(), raise_end<Bf16, EndProject<Bf16>>(),
                              raise_end<Fp32, EndGrad<Fp32>>(), raise_end<Fp32, EndSum>(), raise_end<Fp32, EndProject<Fp32>>()};
    for (const hipError_t e : all)
        if (e != hipSuccess) return e;
    return hipSuccess;
}

hipError_t launch_head_grad(const HeadGradArgs &h, bool bf16, const void *x, const void *w, hipStream_t stream)
{
    return bf16 ? head_grad<Bf16>(h, x, w, stream) : head_grad<Fp32>(h, x, w, stream);
}

}  // namespace zo
