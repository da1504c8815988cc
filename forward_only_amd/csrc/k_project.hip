// k_project.hip -- products of rows with a weight matrix on MFMA, x [rows, k] times w
// [features, k] transposed, with two endings:
//   zo_adapter_project  y = x w^T + bias + scale (x A_g^T) B_g^T, each group of rows with its
//                       own low-rank adapter, moved along its own probe while it is read;
//   zo_head_logprobs    softmax statistics of every row over all features, with the product
//                       itself kept in registers.
//
// Tiles.  A workgroup computes kF features x kR rows.  Features are the MFMA's M dimension and
// rows its N dimension, so that a lane holds several features of one row: a softmax over
// features is mostly in-lane and a store of y writes neighbouring features.  Operands are read
// in 16-byte pieces of one row (8 bf16 or 4 fp32 along k); for fp32 the four values of a piece
// feed four successive 16x16x4 products, which pairs the same k of both operands.
#include <math.h>

#include <type_traits>

#include "zo_lm.hpp"

namespace zo {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 16 zero bytes: what lanes past the end of k read.
__device__ const u32x4 kZeros = {0, 0, 0, 0};

struct Bf16 {
    typedef uint16_t elem;
    static constexpr bool kBf16 = true;
    static constexpr int kPiece = 8;    // elements per 16-byte piece
    static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ float widen(uint16_t v) { return bf16lo_to_f32(v); }
    static __device__ __forceinline__ void load4(const uint16_t *p, float *v)
    {
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
        v[0] = bf16lo_to_f32(w.x);
        v[1] = bf16hi_to_f32(w.x);
        v[2] = bf16lo_to_f32(w.y);
        v[3] = bf16hi_to_f32(w.y);
    }
    static __device__ __forceinline__ float value(u32x4 v, int i)
    {
        return i & 1 ? bf16hi_to_f32(v[i >> 1]) : bf16lo_to_f32(v[i >> 1]);
    }
    // The piece moved by +/-alpha, sign by bit (set: +), rounded as zo_perturb rounds it.
    static __device__ __forceinline__ u32x4 move(u32x4 v, uint32_t signs, float alpha)
    {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = (signs >> (2 * i)) & 1u ? alpha : -alpha;
            const float b = (signs >> (2 * i + 1)) & 1u ? alpha : -alpha;
            o[i] = pack_bf16x2(bf16lo_to_f32(v[i]) + a, bf16hi_to_f32(v[i]) + b);
        }
        return o;
    }
    // Eight fp32 values as an operand: the bf16 of each and the bf16 of what that leaves, so
    // that 16 bits of each value take part in a product.
    struct Wide {
        u32x4 hi, lo;
    };
    static __device__ __forceinline__ Wide wide(const float *v)
    {
        Wide w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w.hi[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            w.lo[i] = pack_bf16x2(v[2 * i] - bf16lo_to_f32(w.hi[i]),
                                  v[2 * i + 1] - bf16hi_to_f32(w.hi[i]));
        }
        return w;
    }
    static __device__ __forceinline__ f32x4 mma(u32x4 a, const Wide &b, f32x4 c)
    {
        return mma(a, b.hi, mma(a, b.lo, c));
    }
};

struct Fp32 {
    typedef float elem;
    static constexpr bool kBf16 = false;
    static constexpr int kPiece = 4;
    static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]),
                                                     c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ float widen(float v) { return v; }
    static __device__ __forceinline__ void load4(const float *p, float *v)
    {
        const f32x4 w = *reinterpret_cast<const f32x4 *>(p);
        for (int i = 0; i < 4; ++i) v[i] = w[i];
    }
    static __device__ __forceinline__ float value(u32x4 v, int i) { return __uint_as_float(v[i]); }
    static __device__ __forceinline__ u32x4 move(u32x4 v, uint32_t signs, float alpha)
    {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = __float_as_uint(__uint_as_float(v[i]) + ((signs >> i) & 1u ? alpha : -alpha));
        return o;
    }
    typedef u32x4 Wide;
    static __device__ __forceinline__ Wide wide(const float *v)
    {
        return Wide{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                    __float_as_uint(v[3])};
    }
};

template <class T>
__device__ __forceinline__ u32x4 piece_at(const typename T::elem *p)
{
    return *reinterpret_cast<const u32x4 *>(p);
}

// ---- operands through LDS ---------------------------------------------------------------

typedef const __attribute__((address_space(1))) void *gptr_t;
typedef __attribute__((address_space(3))) void *lptr_t;
constexpr int kNonTemporal = 2;     // cache policy of a load

// Wait until at most kLoads vector-memory loads are outstanding, and for all LDS reads if kLds.
template <int kLoads, bool kLds>
__device__ __forceinline__ void wait_for()
{
    __builtin_amdgcn_s_waitcnt((kLoads & 15) | (7 << 4) | ((kLds ? 0 : 15) << 8) | ((kLoads >> 4) << 14));
}

// A barrier that no LDS or global access moves across.
__device__ __forceinline__ void turn_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

// One wave's own operands: kRows16 blocks of 16 rows, 128 bytes of k a step, kStages steps under
// way.  A fragment wants neighbouring lanes in different rows; loaded like that straight into
// registers, a lane's 16 bytes take a cycle of the address unit each (13 bytes a cycle were
// measured).  Loads to LDS take eight rows of 128 bytes instead, and the fragment is read from
// there.  The wave waits for its own loads alone, so there is no barrier.
//
// Staged row i holds its piece c at place c ^ (i / 2 % 8): sixteen rows read at one c then cover
// all banks once.
//
// The first kOnce blocks are loaded past the caches.
template <class T, int kRows16, int kStages, int kOnce = 0>
struct Feed {
    static constexpr int kPieces = 8, kLoads = 2 * kRows16;
    static constexpr uint32_t kStep = kPieces * T::kPiece;
    static constexpr int kStage = kRows16 * 16 * kPieces;       // pieces of one stage
    u32x4 *lds;
    uint32_t k, piece;
    const typename T::elem *src[kLoads];

    // row(i): where row i of the blocks begins.
    template <class Row>
    __device__ __forceinline__ Feed(u32x4 *own, uint32_t of_k, Row row) : lds(own), k(of_k)
    {
        const int lane = threadIdx.x & 63;
        piece = (uint32_t)((lane & 7) ^ (lane >> 4)) * T::kPiece;   // + 4 in the odd eights of rows
#pragma unroll
        for (int j = 0; j < kLoads; ++j) src[j] = row(j * 8 + (lane >> 3));
    }
    __device__ __forceinline__ uint32_t steps() const { return (k + kStep - 1) / kStep; }
    __device__ __forceinline__ void issue(uint32_t step, uint32_t stage) const
    {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const uint64_t at = (uint64_t)step * kStep + (j % 2 ? piece ^ (4 * T::kPiece) : piece);
            const void *g = at < k ? static_cast<const void *>(src[j] + at) : &kZeros;
            u32x4 *to = lds + stage * kStage + j * 8 * kPieces;
            if (j < 2 * kOnce)
                __builtin_amdgcn_global_load_lds((gptr_t)g, (lptr_t)to, 16, 0, kNonTemporal);
            else
                __builtin_amdgcn_global_load_lds((gptr_t)g, (lptr_t)to, 16, 0, 0);
        }
    }
    // Fragment c (of two) of block b.
    __device__ __forceinline__ u32x4 fragment(uint32_t stage, int b, int c) const
    {
        const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
        return lds[stage * kStage + (b * 16 + l16) * kPieces + ((4 * c + q) ^ (l16 >> 1))];
    }
};

// ---- the adapters ---------------------------------------------------------------------

// What a group of rows adds to the projection.
struct Group {
    uint64_t lo, hi;       // its rows
    bool none;             // no adapter
    bool bad;              // an index outside its table: the group's rows become NaN
    uint64_t base;         // first parameter of its adapter
    const uint8_t *bits;   // its probe's packed row, or nullptr
    float alpha;
};

// Group g < n_groups, by loads that do not wait for each other.
__device__ __forceinline__ Group group_of(const AdapterArgs &a, uint32_t g)
{
    const int64_t lo = a.starts[g], hi = a.starts[g + 1];
    const int32_t id = a.ids[g];
    const int32_t probe = a.probes ? a.probes[g] : -1;
    const float alpha = a.probes ? a.alphas[g] : 0.0f;
    Group r;
    r.lo = clamp_row(lo, a.rows);
    r.hi = clamp_row(hi, a.rows);
    r.bad = id != -1 && (id < -1 || (uint32_t)id >= a.n_adapters || probe < -1 ||
                         (probe >= 0 && (uint32_t)probe >= a.n_probes));
    r.none = id == -1 || r.bad;
    r.base = r.none ? 0 : (uint64_t)(uint32_t)id * a.rank * ((uint64_t)a.d_in + a.d_out);
    r.bits = probe >= 0 && !r.none ? a.bits + (uint64_t)probe * a.bits_stride : nullptr;
    r.alpha = alpha;
    return r;
}

// The last group whose `value` is at most `at` (else the first), for values that do not fall
// from group to group: all lanes look at once, 64 groups a round.
template <class Value>
__device__ __forceinline__ uint32_t last_group(uint32_t n_groups, uint64_t at, Value value)
{
    const uint32_t lane = threadIdx.x & 63;
    uint32_t g = 0, n = n_groups;
    while (n > 1) {
        const uint32_t step = (n + 63) / 64, i = lane * step;
        const uint64_t below = __ballot(i < n && value(g + (i < n ? i : 0)) <= at);
        if (!below) break;
        const uint32_t skip = (__popcll(below) - 1) * step;
        g += skip;
        n = n - skip < step ? n - skip : step;
    }
    return __builtin_amdgcn_readfirstlane(g);
}

// u[row][j] = x[row] . A_g[j], fp32, and group[row] = g: one workgroup per 16 kXF rows of a
// group, which owns the slots of that many rows from start_g / (16 kXF) + g on, at least as
// many as its rows fill.  The waves share k and feed themselves; their sums meet in LDS.  16
// kAF rows of A are taken at a time.  What bounds it is the latency of the first loads when
// requests bring single rows (16 rows and eight waves), else reading x once and A once per
// workgroup (32 rows and four waves).
constexpr int kShrinkStages = 3;
template <int kXF>
constexpr int shrink_waves() { return kXF == 1 ? 8 : 4; }
template <int kXF, int kAF>
constexpr uint32_t shrink_lds() { return shrink_waves<kXF>() * kShrinkStages * (kXF + kAF) * 16 * 128; }

template <class T, int kXF, int kAF>
__global__ __launch_bounds__(shrink_waves<kXF>() * 64) void k_shrink(
    AdapterArgs a, const typename T::elem *x, uint64_t x_stride, const typename T::elem *adapters,
    float *u, int32_t *group)
{
    typedef Feed<T, kXF + kAF, kShrinkStages> F;
    constexpr int kRows = 16 * kXF, kShares = shrink_waves<kXF>();
    extern __shared__ u32x4 stage[];            // [wave][stage][x, A], then [wave] of sums
    const uint64_t slot = blockIdx.x;
    const uint32_t g = last_group(a.n_groups, slot,
                                  [&](uint32_t i) { return clamp_row(a.starts[i], a.rows) / kRows + i; });
    const Group gr = group_of(a, g);
    const uint64_t start = gr.lo, end = gr.hi;
    if (slot < start / kRows + g) return;
    const uint64_t row0 = start + (slot - (start / kRows + g)) * kRows;
    if (row0 >= end) return;
    if (threadIdx.x < kRows && row0 + threadIdx.x < end) group[row0 + threadIdx.x] = (int32_t)g;
    if (gr.none) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    float *sums = reinterpret_cast<float *>(stage);
    for (uint32_t j0 = 0; j0 < a.rank; j0 += 16 * kAF) {
        const auto row_of_a = [&](int i) { return j0 + i < a.rank ? j0 + i : a.rank - 1; };
        const F feed(stage + wave * kShrinkStages * F::kStage, a.d_in, [&](int i) {
            if (i < kRows) return x + (row0 + i < end ? row0 + i : end - 1) * x_stride;
            return adapters + gr.base + (uint64_t)row_of_a(i - kRows) * a.d_in;
        });
        f32x4 acc[kAF][kXF];
#pragma unroll
        for (int h = 0; h < kAF; ++h)
#pragma unroll
            for (int n = 0; n < kXF; ++n) acc[h][n] = f32x4{0, 0, 0, 0};
        uint64_t e0[kAF];
#pragma unroll
        for (int h = 0; h < kAF; ++h) e0[h] = gr.base + (uint64_t)row_of_a(16 * h + l16) * a.d_in;
        const uint32_t steps = feed.steps();
        const auto take = [&](auto moved) {
            constexpr bool kMoved = decltype(moved)::value;
            uint8_t sg[2][kAF];
            const auto signs = [&](uint32_t step) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int h = 0; h < kAF; ++h) {
                        const uint64_t k = (uint64_t)step * F::kStep + (4 * c + q) * T::kPiece;
                        sg[c][h] = gr.bits[(e0[h] + (k < a.d_in ? k : 0)) >> 3];
                    }
            };
            if constexpr (kMoved) signs(wave);
#pragma unroll
            for (int i = 0; i < kShrinkStages - 1; ++i) feed.issue(wave + i * kShares, i);
            uint32_t at = 0, to = kShrinkStages - 1;
            for (uint32_t s = wave; s < steps; s += kShares) {
                wait_for<F::kLoads * (kShrinkStages - 2), true>();
                asm volatile("" ::: "memory");
                u32x4 fa[2][kAF], fx[2][kXF];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int n = 0; n < kXF; ++n) fx[c][n] = feed.fragment(at, n, c);
#pragma unroll
                    for (int h = 0; h < kAF; ++h) fa[c][h] = feed.fragment(at, kXF + h, c);
                }
                if constexpr (kMoved) {
                    // past the end of k the moved zeros, +-alpha, meet zeros of x
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int h = 0; h < kAF; ++h)
                            fa[c][h] = T::move(fa[c][h], sg[c][h] >> ((4 * c + q) * T::kPiece & 7), gr.alpha);
                    signs(s + kShares);         // before the loads that the next wait leaves out
                }
                feed.issue(s + (kShrinkStages - 1) * kShares, to);
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int h = 0; h < kAF; ++h)
#pragma unroll
                        for (int n = 0; n < kXF; ++n) acc[h][n] = T::mma(fa[c][h], fx[c][n], acc[h][n]);
                at = at + 1 == kShrinkStages ? 0 : at + 1;
                to = to + 1 == kShrinkStages ? 0 : to + 1;
            }
        };
        if (gr.bits)
            take(std::true_type{});
        else
            take(std::false_type{});
        wait_for<0, true>();
        __syncthreads();                        // the stages are free
        constexpr int kPitch = 16 * kAF + 1;
#pragma unroll
        for (int h = 0; h < kAF; ++h)
#pragma unroll
            for (int n = 0; n < kXF; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sums[(wave * kRows + 16 * n + l16) * kPitch + 16 * h + 4 * q + i] = acc[h][n][i];
        __syncthreads();
        for (int o = threadIdx.x; o < kRows * 16 * kAF; o += kShares * 64) {
            const int r = o / (16 * kAF), c = o % (16 * kAF);
            if (row0 + r >= end || j0 + c >= a.rank) continue;
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kShares; ++w) sum += sums[(w * kRows + r) * kPitch + c];
            u[(row0 + r) * a.rank + j0 + c] = sum;
        }
        __syncthreads();
    }
}

// ---- the product ----------------------------------------------------------------------

struct ProductArgs {
    uint64_t base, rows;   // places [base, base + rows) of the rows, or of the list's rows
    uint64_t x_stride;
    uint32_t k, features;
    float *slices;         // workspace of the sliced tiles, or nullptr: none are sliced
};

// How many of `rows` places from `base` on there are when only *count places hold a row.
__device__ __forceinline__ uint64_t places(uint64_t base, uint64_t rows, const uint32_t *count)
{
    if (!count) return rows;
    const uint64_t n = *count;
    return n <= base ? 0 : (n - base < rows ? n - base : rows);
}

// Accumulators of one wave: kMF x kMR fragments of 16 features x 16 rows.  Lane l holds row
// l % 16 of a fragment; its value i belongs to feature 4 (l / 16) + i.
template <int kMFOf, int kMROf>
struct Tile {
    static constexpr int kMF = kMFOf, kMR = kMROf;
    f32x4 acc[kMF][kMR];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int m = 0; m < kMF; ++m)
#pragma unroll
            for (int n = 0; n < kMR; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
    }
};

// Ending of zo_adapter_project.
template <class T>
struct EndProject {
    static constexpr bool kSlices = false;
    static constexpr uint32_t kRowwise = 4;
    AdapterArgs a;
    const float *u;
    const int32_t *group;
    const typename T::elem *adapters, *bias;
    typename T::elem *y;
    uint64_t y_stride;

    // The last group that starts at or before row r0 (else the first).
    __device__ __forceinline__ uint32_t begin(uint64_t r0) const
    {
        return last_group(a.n_groups, r0, [&](uint32_t i) { return clamp_row(a.starts[i], a.rows); });
    }

    // Many rows: the groups that meet the tile one after another, on MFMA.  `lds`: 8 KiB of
    // this wave's own.
    template <class Tl>
    __device__ __forceinline__ void finish(Tl &t, uint32_t g, uint32_t f0, uint64_t r0, u32x4 *lds) const
    {
        if constexpr (Tl::kMF == 2) {
            // A wave's tile that more than kRowwise groups meet takes the rows' way instead, which
            // does not go through them one by one (32 rows a wave; rank 16, groups of 1, 4 and 8
            // rows: bf16 520 rows, 768 to 768 52 -> 24, 22 -> 18 and 19 us either way; fp32
            // 64 -> 43, 35 -> 32 and 32 either way).
            const uint64_t r1 = r0 + 16 * Tl::kMR < a.rows ? r0 + 16 * Tl::kMR : a.rows;
            if (r0 < r1 && begin(r1 - 1) - g > kRowwise) {
#pragma unroll
                for (int n = 0; n < Tl::kMR; ++n) add_rows(t, n, f0, r0 + 16 * n);
            } else {
                add_groups(t, g, f0, r0);
            }
        } else {
            add_groups(t, g, f0, r0);
        }
        store_rows(t, f0, r0, lds);
    }

    // Rows that each may have an adapter of their own: every lane the products of its row, so
    // that one round of loads serves all groups.
    template <class Tl>
    __device__ __forceinline__ void add_rows(Tl &t, int n, uint32_t f0, uint64_t r0) const
    {
        constexpr int kMF = Tl::kMF;
        const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
        const uint64_t row = r0 + l16;
        if (row >= a.rows) return;
        const int32_t g = group[row];
        if (g < 0 || (uint32_t)g >= a.n_groups) return;
        const Group gr = group_of(a, (uint32_t)g);
        if (gr.bad) {
#pragma unroll
            for (int m = 0; m < kMF; ++m) t.acc[m][n] += __builtin_nanf("");
        }
        if (gr.none) return;
        const uint64_t first = gr.base + (uint64_t)a.rank * a.d_in;
        for (uint32_t j = 0; j < a.rank; j += 8) {
            const f32x4 *pu = reinterpret_cast<const f32x4 *>(u + row * a.rank + j);
            const f32x4 ua = pu[0], ub = pu[1];
            u32x4 fb[kMF][4][8 / T::kPiece];
            uint8_t sg[kMF][4];
#pragma unroll
            for (int m = 0; m < kMF; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t f = f0 + 16 * m + 4 * q + i;
                    const uint64_t at = first + (uint64_t)(f < a.d_out ? f : a.d_out - 1) * a.rank + j;
#pragma unroll
                    for (int h = 0; h < 8 / T::kPiece; ++h) fb[m][i][h] = piece_at<T>(adapters + at + h * T::kPiece);
                    sg[m][i] = *(gr.bits ? gr.bits + (at >> 3) : reinterpret_cast<const uint8_t *>(&kZeros));
                }
#pragma unroll
            for (int m = 0; m < kMF; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float s = 0.0f;
#pragma unroll
                    for (int h = 0; h < 8 / T::kPiece; ++h) {
                        const u32x4 v = gr.bits ? T::move(fb[m][i][h], sg[m][i] >> (h * T::kPiece), gr.alpha)
                                                : fb[m][i][h];
#pragma unroll
                        for (int k = 0; k < T::kPiece; ++k) {
                            const int c = h * T::kPiece + k;
                            s = fmaf(T::value(v, k), c < 4 ? ua[c & 3] : ub[c & 3], s);
                        }
                    }
                    t.acc[m][n][i] += a.scale * s;
                }
        }
    }

    template <class Tl>
    __device__ __forceinline__ void add_groups(Tl &t, uint32_t g, uint32_t f0, uint64_t r0) const
    {
        constexpr int kMF = Tl::kMF, kMR = Tl::kMR;
        const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
        const uint64_t r1 = r0 + 16 * kMR < a.rows ? r0 + 16 * kMR : a.rows;
        for (; g < a.n_groups; ++g) {
            const Group gr = group_of(a, g);
            const uint64_t s = gr.lo, e = gr.hi;
            if (s >= r1) break;
            if (e <= r0 || e <= s) continue;
            if (gr.bad) {
#pragma unroll
                for (int n = 0; n < kMR; ++n) {
                    const uint64_t row = r0 + 16 * n + l16;
                    const float nan = row >= s && row < e ? __builtin_nanf("") : 0.0f;
#pragma unroll
                    for (int m = 0; m < kMF; ++m) t.acc[m][n] += nan;
                }
            }
            if (gr.none) continue;
            // The product is formed apart and added to the group's own rows, so that a NaN in
            // its adapter does not reach the others through 0 * NaN.
            const uint64_t first = gr.base + (uint64_t)a.rank * a.d_in;
            for (uint32_t j0 = 0; j0 < a.rank; j0 += 4 * T::kPiece) {
                const uint32_t j = j0 + q * T::kPiece;
                typename T::Wide v[kMR];
#pragma unroll
                for (int n = 0; n < kMR; ++n) {
                    const uint64_t row = r0 + 16 * n + l16;
                    const bool in = row >= s && row < e && j < a.rank;
                    const f32x4 *pu = reinterpret_cast<const f32x4 *>(u + (in ? row * a.rank + j : s * a.rank));
                    float z[T::kPiece];
#pragma unroll
                    for (int i = 0; i < T::kPiece; i += 4) {
                        f32x4 w = pu[i / 4];
                        if (!in) w = f32x4{0, 0, 0, 0};
#pragma unroll
                        for (int k = 0; k < 4; ++k) z[i + k] = a.scale * w[k];
                    }
                    v[n] = T::wide(z);
                }
                // Loads without branches between them, four at once (eight would spill); lanes
                // past the rank meet zeros of u, lanes past the features are not stored.
                constexpr int kAtOnce = kMF < 4 ? kMF : 4;
#pragma unroll
                for (int m0 = 0; m0 < kMF; m0 += kAtOnce) {
                    asm volatile("" ::: "memory");
                    u32x4 fb[kAtOnce];
                    uint8_t sg[kAtOnce];
#pragma unroll
                    for (int m = 0; m < kAtOnce; ++m) {
                        const uint32_t f = f0 + 16 * (m0 + m) + l16;
                        const uint64_t at = first + (uint64_t)(f < a.d_out ? f : a.d_out - 1) * a.rank +
                                            (j < a.rank ? j : 0);
                        fb[m] = piece_at<T>(adapters + at);
                        sg[m] = *(gr.bits ? gr.bits + (at >> 3) : reinterpret_cast<const uint8_t *>(&kZeros));
                    }
#pragma unroll
                    for (int m = 0; m < kAtOnce; ++m) {
                        if (gr.bits) fb[m] = T::move(fb[m], sg[m] >> (j & 7), gr.alpha);
#pragma unroll
                        for (int n = 0; n < kMR; ++n) {
                            const uint64_t row = r0 + 16 * n + l16;
                            if (r0 + 16 * n + 16 <= s || r0 + 16 * n >= e) continue;
                            const bool in = row >= s && row < e;
                            f32x4 zero = {};
                            const f32x4 add = T::mma(fb[m], v[n], zero);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                t.acc[m0 + m][n][i] = in ? t.acc[m0 + m][n][i] + add[i] : t.acc[m0 + m][n][i];
                        }
                    }
                }
            }
        }
    }

    template <class Tl>
    __device__ __forceinline__ void store(Tl &t, uint32_t f0, uint64_t r0) const
    {
        constexpr int kMF = Tl::kMF, kMR = Tl::kMR;
        const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
        const uint64_t lo = clamp_row(a.starts[0], a.rows);
        const uint64_t hi = clamp_row(a.starts[a.n_groups], a.rows);
#pragma unroll
        for (int n = 0; n < kMR; ++n) {
            const uint64_t row = r0 + 16 * n + l16;
            if (row < lo || row >= hi) continue;
#pragma unroll
            for (int m = 0; m < kMF; ++m) {
                const uint32_t f = f0 + 16 * m + 4 * q;
                if (f >= a.d_out) continue;
                f32x4 v;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = t.acc[m][n][i];
                    if (bias) v[i] += T::widen(bias[f + i]);
                }
                store4(y + row * y_stride + f, v);
            }
        }
    }
    // The same through LDS, 16 rows at a time: a lane then stores 16 bytes next to its
    // neighbours', whole lines of y instead of 8 bytes of each of 16 rows.  Row i keeps its
    // piece c at place c ^ i.
    template <class Tl>
    __device__ __forceinline__ void store_rows(Tl &t, uint32_t f0, uint64_t r0, u32x4 *lds) const
    {
        constexpr int kMF = Tl::kMF, kMR = Tl::kMR;
        constexpr int kRowPieces = 16 * kMF / T::kPiece, kAtOnce = 64 / kRowPieces;
        const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
        const uint64_t lo = clamp_row(a.starts[0], a.rows);
        const uint64_t hi = clamp_row(a.starts[a.n_groups], a.rows);
        float add[kMF][4];
#pragma unroll
        for (int m = 0; m < kMF; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) add[m][i] = 0.0f;
        if (bias) {
#pragma unroll
            for (int m = 0; m < kMF; ++m) {
                const uint32_t f = f0 + 16 * m + 4 * q;
                if (f < a.d_out) T::load4(bias + f, add[m]);
            }
        }
        const int piece = lane % kRowPieces;
        const uint32_t f = f0 + piece * T::kPiece;
#pragma unroll
        for (int n = 0; n < kMR; ++n) {
            wave_lds_sync();
#pragma unroll
            for (int m = 0; m < kMF; ++m) {
                f32x4 v;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = t.acc[m][n][i] + add[m][i];
                const int four = 4 * m + q, c = four * 4 / T::kPiece;
                typename T::elem *at = reinterpret_cast<typename T::elem *>(
                    lds + l16 * kRowPieces + (c ^ (l16 % kRowPieces))) + four * 4 % T::kPiece;
                store4(at, v);
            }
            wave_lds_sync();
#pragma unroll
            for (int i = 0; i < 16; i += kAtOnce) {
                const int r = i + lane / kRowPieces;
                const uint64_t row = r0 + 16 * n + r;
                const u32x4 v = lds[r * kRowPieces + (piece ^ (r % kRowPieces))];
                if (row >= lo && row < hi && f < a.d_out)
                    *reinterpret_cast<u32x4 *>(y + row * y_stride + f) = v;
            }
        }
    }
    static __device__ __forceinline__ void store4(float *p, f32x4 v) { *reinterpret_cast<f32x4 *>(p) = v; }
    static __device__ __forceinline__ void store4(uint16_t *p, f32x4 v)
    {
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
};

// Ending of zo_head_logprobs: per wave tile and row (m, s, t) over the tile's features.
struct EndHead {
    static constexpr bool kSlices = false;
    uint32_t features;
    uint64_t base, rows;        // places of this launch
    const int64_t *targets;     // of all rows, or nullptr
    const uint32_t *list;       // row of each place, or nullptr: place = row
    const uint32_t *count;
    float *m, *s, *t;           // [wave tile][place]
    float *tl;                  // logit of each place's target

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
        constexpr int kMF = Tl::kMF, kMR = Tl::kMR;
        const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
        const uint32_t part = f0 / (16 * kMF);
        if (f0 >= features) return;
        const uint64_t have = places(base, rows, count);
#pragma unroll
        for (int n = 0; n < kMR; ++n) {
            const uint64_t at = r0 + 16 * n + l16;
            SoftStats st = SoftStats::empty();
            int64_t tgt = -1;
            if (targets && at < have) tgt = targets[list ? list[base + at] : base + at];
            const auto feature = [&](int m4, int i) { return f0 + 16 * m4 + 4 * q + i; };
            if (f0 + 16 * kMF > features) {
#pragma unroll
                for (int m4 = 0; m4 < kMF; ++m4)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (feature(m4, i) >= features) tile.acc[m4][n][i] = -INFINITY;
            }
            float top = -INFINITY;
#pragma unroll
            for (int m4 = 0; m4 < kMF; ++m4)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, tile.acc[m4][n][i]);
            st.raise(top);
#pragma unroll
            for (int m4 = 0; m4 < kMF; ++m4)
#pragma unroll
                for (int i = 0; i < 4; ++i) st.add(tile.acc[m4][n][i]);
            // few waves hold a row's target
            const uint32_t in = (uint32_t)(tgt - f0);
            const bool here = at < have && tgt >= (int64_t)f0 && tgt < (int64_t)features && in < 16 * kMF;
            if (__any(here)) {
#pragma unroll
                for (int m4 = 0; m4 < kMF; ++m4)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (here && feature(m4, i) - f0 == in) tl[at] = tile.acc[m4][n][i];
            }
            st.wave_merge(32, 16);
            if (q == 0 && at < have) {
                m[(uint64_t)part * rows + at] = st.m;
                s[(uint64_t)part * rows + at] = st.s;
                t[(uint64_t)part * rows + at] = st.t;
            }
        }
    }
};

// Tile t of nf x nr: consecutive tiles run through eight row tiles, then the next features, so
// that tiles in flight together share rows and weights in L2.
__device__ __forceinline__ void tile_at(uint32_t t, uint32_t nf, uint32_t nr, uint32_t &f, uint32_t &r)
{
    constexpr uint32_t kDeep = 8;
    const uint32_t group = t / (kDeep * nf), in = t - group * kDeep * nf;
    const uint32_t deep = nr - group * kDeep < kDeep ? nr - group * kDeep : kDeep;
    f = in / deep;
    r = group * kDeep + in % deep;
}
// Which of n tiles workgroup b takes: each XCD (workgroup b runs on XCD b % 8) one contiguous
// range.  n or more: none.
__device__ __forceinline__ uint32_t tile_of_xcd(uint32_t b, uint32_t n)
{
    const uint64_t x = b & 7u;
    const uint64_t t = n * x / 8 + (b >> 3);
    return t < n * (x + 1) / 8 ? (uint32_t)t : n;
}

// Many rows: 256 features x 256 rows by eight waves of 128 x 64, in which the two waves of a
// SIMD take turns: four of the waves multiply while the other four read their next operands
// from LDS, one barrier apart.  A step of 128 bytes of k has two such turns, one for each half
// of a wave's features:
//   turn 0  reads F0, the first half of its features, and its rows R   multiplies (F0, R)
//   turn 1  reads F1, the second half                                  multiplies (F1, R)
// A part of the stage is free for the step after next as soon as both groups have read it, so
// its loads go out one turn later and have one and a half steps to arrive; each turn waits for
// the loads that the next turn reads: all but the eight issued since.  Loads past the end of k
// read zeros, so that the counts hold to the end.  Four turns of a quarter each, with operands
// read one turn ahead, were no faster and took 96 registers for operands instead of 64.
// What bounds it: MFMA issue, 77% of the cycles at 1.8 GHz, a clock that the load lowers (LDS
// reads and writes take about as many cycles as the products): 1475 TFLOP/s of bf16 at
// 4096 x 50272 x 7168.
//
// Tiles run one per CU, so their number is cut into whole rounds of kSlots and a rest.  When the
// rest fills at most half a round, each of its tiles is cut along k into as many slices as
// fit into the round; their sums, 256 KiB each, are added in order by k_slices.
constexpr int kBigF = 256, kBigR = 256;

struct Cut {
    uint32_t nf, nr;           // tiles of features and of rows
    uint32_t whole, rest;      // tiles done whole, and the sliced ones (or all whole: rest = 0)
    uint32_t slices;
    __device__ __forceinline__ Cut(const ProductArgs &p, uint64_t rows, uint32_t steps)
    {
        nf = (p.features + kBigF - 1) / kBigF;
        nr = (uint32_t)((rows + kBigR - 1) / kBigR);
        const uint32_t n = nf * nr;
        const uint32_t over = n % kBigSlots;
        slices = big_slices(over, steps);
        rest = p.slices && slices > 1 ? over : 0;
        whole = n - rest;
    }
};

template <class T, class End>
__global__ __launch_bounds__(512, 2) void k_big(ProductArgs p, const typename T::elem *x,
                                                const typename T::elem *w, const uint32_t *list,
                                                const uint32_t *count, End end)
{
    constexpr int kPieces = 8;
    constexpr uint32_t kStep = kPieces * T::kPiece;
    constexpr int kPart = 128 * kPieces;                    // a quarter of a stage, in pieces
    enum { F0, F1, R0, R1 };
    extern __shared__ u32x4 stage[];                        // [2][F0, F1, R0, R1][128][kPieces]
    const uint64_t rows = places(p.base, p.rows, count);
    const uint32_t steps = (p.k + kStep - 1) / kStep;
    const Cut cut(p, rows, steps);
    uint32_t tile, first = 0, last = steps;
    if constexpr (End::kSlices) {
        const uint32_t slice = blockIdx.x % cut.slices;
        if (blockIdx.x / cut.slices >= cut.rest) return;
        tile = cut.whole + blockIdx.x / cut.slices;
        first = (uint32_t)((uint64_t)steps * slice / cut.slices);
        last = (uint32_t)((uint64_t)steps * (slice + 1) / cut.slices);
    } else {
        tile = tile_of_xcd(blockIdx.x, cut.whole);
        if (tile >= cut.whole) return;
    }
    uint32_t tf, tr;
    tile_at(tile, cut.nf, cut.nr, tf, tr);
    const uint32_t f0 = tf * kBigF;
    const uint64_t r0 = (uint64_t)tr * kBigR;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    const int wf = wave & 1, wr = wave >> 1;
    // Staged row i holds its piece c at place c ^ (i / 2 % 8): sixteen rows read at one c then
    // cover all banks once.  This wave stages rows 8 wave .. + 7 and 64 more of each quarter.
    const uint32_t piece = (uint32_t)((lane & 7) ^ ((wave * 4 + (lane >> 4)) & 7)) * T::kPiece;
    // Sources in 16-byte units from the tile's first weight and from x: registers are short
    // here, and 32 bits of units reach 64 GiB.
    const u32x4 *const from_w = reinterpret_cast<const u32x4 *>(w + (uint64_t)f0 * p.k);
    const u32x4 *const from_x = reinterpret_cast<const u32x4 *>(x);
    uint32_t src[4][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = j * 64 + wave * 8 + (lane >> 3);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t f = (i >> 6) * 128 + h * 64 + (i & 63);
            src[F0 + h][j] = (uint32_t)(((uint64_t)(f0 + f < p.features ? f : p.features - 1 - f0) * p.k + piece) / T::kPiece);
            const uint64_t at = r0 + (i >> 5) * 64 + h * 32 + (i & 31);
            const uint64_t r = at < rows ? at : rows - 1;
            src[R0 + h][j] = (uint32_t)(((list ? list[p.base + r] : p.base + r) * p.x_stride + piece) / T::kPiece);
        }
    }
    const auto issue = [&](int part, uint32_t step) {
        const bool in = step < last && (uint64_t)step * kStep + piece < p.k;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const u32x4 *g = (part < R0 ? from_w : from_x) + (uint64_t)step * kPieces + src[part][j];
            if (!in) g = &kZeros;
            u32x4 *l = stage + ((step & 1) * 4 + part) * kPart + (j * 64 + wave * 8) * kPieces;
            __builtin_amdgcn_global_load_lds((gptr_t)g, (lptr_t)l, 16, 0, 0);
        }
    };
    Tile<8, 4> t;
    t.clear();
    u32x4 ff[2][4], fr[2][4];                   // [c][fragment]
    const auto read_f = [&](int h, uint32_t step) {
        const u32x4 *s = stage + ((step & 1) * 4 + F0 + h) * kPart + (wf * 64 + l16) * kPieces;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int m = 0; m < 4; ++m) ff[c][m] = s[m * 16 * kPieces + ((4 * c + q) ^ (l16 >> 1))];
    };
    const auto read_r = [&](uint32_t step) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4 *s = stage + ((step & 1) * 4 + R0 + h) * kPart + (wr * 32 + l16) * kPieces;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int n = 0; n < 2; ++n) fr[c][2 * h + n] = s[n * 16 * kPieces + ((4 * c + q) ^ (l16 >> 1))];
        }
    };
    const auto multiply = [&](int hf) {
        wait_for<8, true>();
        turn_barrier();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    t.acc[4 * hf + m][n] = T::mma(ff[c][m], fr[c][n], t.acc[4 * hf + m][n]);
        __builtin_amdgcn_s_setprio(0);
        turn_barrier();
    };
    uint32_t begun = 0;
    issue(F0, first);
    issue(R0, first);
    issue(R1, first);
    issue(F1, first);
    begun = end.begin(r0 + wr * 64);
    issue(F0, first + 1);
    issue(R0, first + 1);
    issue(R1, first + 1);
    wait_for<8, false>();                       // F0, R0 and R1 of the first step
    turn_barrier();
    if (wave >= 4) turn_barrier();              // one turn behind from here on
    for (uint32_t s = first; s < last; ++s) {
        read_f(0, s);
        read_r(s);
        issue(F1, s + 1);
        multiply(0);
        read_f(1, s);
        issue(F0, s + 2);
        issue(R0, s + 2);
        issue(R1, s + 2);
        multiply(1);
    }
    if (wave < 4) turn_barrier();
    wait_for<0, true>();
    turn_barrier();                             // the stage is free: no load is under way
    end.finish(t, begun, f0 + wf * 128, r0 + wr * 64, stage + wave * 512);
}

// The ending of a slice: its sums, to be added by k_slices.
struct EndSlice {
    static constexpr bool kSlices = true;
    float *slices;
    __device__ __forceinline__ uint32_t begin(uint64_t) const { return 0; }
    template <class Tl>
    __device__ __forceinline__ void finish(Tl &t, uint32_t, uint32_t, uint64_t, u32x4 *) const
    {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        f32x4 *to = reinterpret_cast<f32x4 *>(slices) + ((uint64_t)blockIdx.x * 8 + wave) * 32 * 64 + lane;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int m = 0; m < 8; ++m) to[(n * 8 + m) * 64] = t.acc[m][n];
    }
};

// Sums the slices of the last tiles and ends them: a workgroup takes 16 rows of one wave's tile
// of k_big; its four waves share the slices, and the first adds up and ends.
template <class T, class End>
__global__ __launch_bounds__(256) void k_slices(ProductArgs p, const uint32_t *count, End end)
{
    __shared__ u32x4 lds[3 * 8 * 64];
    const uint64_t rows = places(p.base, p.rows, count);
    const Cut cut(p, rows, (p.k + 8 * T::kPiece - 1) / (8 * T::kPiece));
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t i = blockIdx.x / 32, of = blockIdx.x / 4 % 8, n = blockIdx.x % 4;
    if (i >= cut.rest || cut.slices < 2) return;
    uint32_t tf, tr;
    tile_at(cut.whole + i, cut.nf, cut.nr, tf, tr);
    const uint32_t f0 = tf * kBigF + (of & 1) * 128;
    const uint64_t r0 = (uint64_t)tr * kBigR + (of >> 1) * 64 + n * 16;
    if (r0 >= rows) return;
    const f32x4 *from = reinterpret_cast<const f32x4 *>(p.slices) +
                        ((uint64_t)i * cut.slices * 8 + of) * 32 * 64 + (n * 8) * 64 + lane;
    Tile<8, 1> t;
    t.clear();
#pragma unroll 2
    for (uint32_t s = wave; s < cut.slices; s += 4)
#pragma unroll
        for (int m = 0; m < 8; ++m) t.acc[m][0] += from[(uint64_t)s * 8 * 32 * 64 + m * 64];
    f32x4 *sums = reinterpret_cast<f32x4 *>(lds);
    if (wave)
#pragma unroll
        for (int m = 0; m < 8; ++m) sums[((wave - 1) * 8 + m) * 64 + lane] = t.acc[m][0];
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int v = 0; v < 3; ++v)
#pragma unroll
        for (int m = 0; m < 8; ++m) t.acc[m][0] += sums[(v * 8 + m) * 64 + lane];
    end.finish(t, end.begin(r0), f0, r0, lds);
}

// Middling sizes, where tiles of 256 x 256 would leave CUs without one: 64 features x 64 rows
// by four waves.  Such a tile multiplies for a tenth of a microsecond a step, far less than a
// load takes, so four stages are under way at once; a step waits for its own alone.
constexpr int kMidStages = 4;
template <class T, class End>
__global__ __launch_bounds__(256) void k_mid(ProductArgs p, const typename T::elem *x,
                                             const typename T::elem *w, const uint32_t *list,
                                             const uint32_t *count, End end)
{
    constexpr int kSize = 64, kPieces = 8;
    constexpr uint32_t kStep = kPieces * T::kPiece;
    __shared__ u32x4 stage[kMidStages * 2 * kSize * kPieces];   // [stage][features, rows][kSize][kPieces]
    const uint64_t rows = places(p.base, p.rows, count);
    const uint32_t nf = (p.features + kSize - 1) / kSize, nr = (uint32_t)((rows + kSize - 1) / kSize);
    const uint32_t tile = tile_of_xcd(blockIdx.x, nf * nr);
    if (tile >= nf * nr) return;
    uint32_t tf, tr;
    tile_at(tile, nf, nr, tf, tr);
    const uint32_t f0 = tf * kSize;
    const uint64_t r0 = (uint64_t)tr * kSize;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    const int wf = wave & 1, wr = wave >> 1;
    // pieces placed as in k_big; this wave stages rows 8 wave .. + 7 of every 32 of both sides
    const uint32_t piece = (uint32_t)((lane & 7) ^ ((wave * 4 + (lane >> 4)) & 7)) * T::kPiece;
    const typename T::elem *src[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = j * 32 + wave * 8 + (lane >> 3);
        const uint32_t f = f0 + i < p.features ? f0 + i : p.features - 1;
        src[0][j] = w + (uint64_t)f * p.k + piece;
        const uint64_t r = r0 + i < rows ? r0 + i : rows - 1;
        src[1][j] = x + (list ? list[p.base + r] : p.base + r) * p.x_stride + piece;
    }
    const uint32_t steps = (p.k + kStep - 1) / kStep;
    const auto issue = [&](uint32_t step) {
        const bool in = (uint64_t)step * kStep + piece < p.k;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const void *g = src[h][j] + (uint64_t)step * kStep;
                if (!in) g = &kZeros;
                u32x4 *l = stage + ((step % kMidStages * 2 + h) * kSize + j * 32 + wave * 8) * kPieces;
                __builtin_amdgcn_global_load_lds((gptr_t)g, (lptr_t)l, 16, 0, 0);
            }
    };
    Tile<2, 2> t;
    t.clear();
#pragma unroll
    for (uint32_t s = 0; s < kMidStages - 1; ++s) issue(s);
    const auto g = end.begin(r0 + wr * 32);
    for (uint32_t s = 0; s < steps; ++s) {
        wait_for<4 * (kMidStages - 2), true>();     // this step's loads
        turn_barrier();                             // everyone's; and the last step's readers are done
        issue(s + kMidStages - 1);
        const u32x4 *sw = stage + (s % kMidStages * 2 * kSize + wf * 32 + l16) * kPieces;
        const u32x4 *sx = stage + ((s % kMidStages * 2 + 1) * kSize + wr * 32 + l16) * kPieces;
        u32x4 ff[2][2], fr[2][2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int at = (4 * c + q) ^ (l16 >> 1);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                ff[c][m] = sw[m * 16 * kPieces + at];
                fr[c][m] = sx[m * 16 * kPieces + at];
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < 2; ++n) t.acc[m][n] = T::mma(ff[c][m], fr[c][n], t.acc[m][n]);
    }
    wait_for<0, true>();
    turn_barrier();                                 // the stage is free: no load is under way
    end.finish(t, g, f0 + wf * 32, r0 + wr * 32, stage + wave * 512);
}

// Few rows.  What bounds the product is reading w once: a workgroup takes 16 kMF features and
// all rows, four waves take every fourth step of k, and their sums meet in LDS.  kMR more waves
// form the adapters' products meanwhile, add everything up and end 16 rows each.  32 features:
// with 16, x is read from L2 as often again (32 rows, 5120 to 5120, bf16: 14.8 us; 12.0 with
// 32); 64 where that takes fewer rounds (few_features; 32 rows, 5120 to 50272: 115 us, 106 with
// 64).  Three stages: two leave too little under way, four one workgroup per CU (8 rows, 5120
// to 50272, through the caches: 94 and 97 us; 88 with three; 81 past them, 6.4 TB/s).
constexpr int kFewWaves = 4, kFewStages = 3;
template <int kMR, int kMF>
constexpr uint32_t few_lds() { return kFewWaves * kFewStages * (kMF + kMR) * 16 * 128; }

template <class T, int kMR, int kMF, bool kOnce, class End>
__global__ __launch_bounds__((kFewWaves + kMR) * 64) void k_few(ProductArgs p,
                                                                const typename T::elem *x,
                                                                const typename T::elem *w, End end)
{
    typedef Feed<T, kMF + kMR, kFewStages, kOnce ? kMF : 0> F;
    extern __shared__ u32x4 stage[];            // [wave][stage][features, rows], then [wave] of sums
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t f0 = blockIdx.x * (16 * kMF);
    f32x4 *sums = reinterpret_cast<f32x4 *>(stage);
    if (wave >= kFewWaves) {
        const int n = wave - kFewWaves;
        Tile<kMF, 1> own;
        own.clear();
        end.add_rows(own, 0, f0, 16 * n);
        __syncthreads();                        // the stages are free
        __syncthreads();                        // the sums are there
#pragma unroll
        for (int m = 0; m < kMF; ++m)
#pragma unroll
            for (int v = 0; v < kFewWaves; ++v) own.acc[m][0] += sums[((v * kMF + m) * kMR + n) * 64 + lane];
        end.store(own, f0, 16 * n);
        return;
    }
    const F feed(stage + wave * kFewStages * F::kStage, p.k, [&](int i) {
        if (i < 16 * kMF) {
            const uint32_t f = f0 + i < p.features ? f0 + i : p.features - 1;
            return w + (uint64_t)f * p.k;
        }
        const uint64_t r = (uint64_t)(i - 16 * kMF) < p.rows ? i - 16 * kMF : p.rows - 1;
        return x + r * p.x_stride;
    });
    Tile<kMF, kMR> t;
    t.clear();
    const uint32_t steps = feed.steps();
    // Each workgroup begins elsewhere in k: rows a power of two apart lie on the same memory
    // channels, and all workgroups would walk over them together (8 rows, bf16 8192 to 28672: 98
    // us begun together, 74 apart; 4096 to 18000 39 and 27; 5120 to 50272 84 either way).
    const uint32_t turn = (blockIdx.x * 0x9E3779B1u >> 8) % steps;
    const auto turned = [&](uint32_t s) { return s >= steps ? s : s + turn < steps ? s + turn : s + turn - steps; };
#pragma unroll
    for (int i = 0; i < kFewStages - 1; ++i) feed.issue(turned(wave + i * kFewWaves), i);
    uint32_t at = 0, to = kFewStages - 1;
    for (uint32_t s = wave; s < steps; s += kFewWaves) {
        wait_for<F::kLoads * (kFewStages - 2), true>();
        asm volatile("" ::: "memory");
        u32x4 fw[2][kMF], fx[2][kMR];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int m = 0; m < kMF; ++m) fw[c][m] = feed.fragment(at, m, c);
#pragma unroll
            for (int n = 0; n < kMR; ++n) fx[c][n] = feed.fragment(at, kMF + n, c);
        }
        feed.issue(turned(s + (kFewStages - 1) * kFewWaves), to);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int m = 0; m < kMF; ++m)
#pragma unroll
                for (int n = 0; n < kMR; ++n) t.acc[m][n] = T::mma(fw[c][m], fx[c][n], t.acc[m][n]);
        at = at + 1 == kFewStages ? 0 : at + 1;
        to = to + 1 == kFewStages ? 0 : to + 1;
    }
    wait_for<0, true>();
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kMF; ++m)
#pragma unroll
        for (int n = 0; n < kMR; ++n) sums[((wave * kMF + m) * kMR + n) * 64 + lane] = t.acc[m][n];
    __syncthreads();
}

// ---- joining the head's partial statistics ----------------------------------------------

// The places of the rows that count, in order, and zeros for the others' outputs; one
// workgroup, eight rows of a thread in flight at once.
__global__ __launch_bounds__(1024) void k_counted(const int64_t *targets, uint64_t rows,
                                                  uint32_t *list, uint32_t *count, float *logp,
                                                  float *entropy)
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
}

// Joins the parts of each place: kOf places per workgroup of 1024 threads.  Eight read whole
// sectors; one, when there are few rows, has its parts in one or two rounds of loads.
template <int kOf>
__global__ __launch_bounds__(1024) void k_head_join(const float *m, const float *s, const float *t,
                                                    const float *tl, uint32_t parts, uint64_t base,
                                                    uint64_t rows, const uint32_t *list,
                                                    const uint32_t *count, const int64_t *targets,
                                                    uint32_t features, float *logp, float *entropy)
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
    if (logp)
        logp[row] = ignore ? 0.0f
                    : tgt >= 0 && tgt < (int64_t)features ? (tl[at] - st.m) - logs
                                                          : __builtin_nanf("");
    if (entropy) entropy[row] = ignore ? 0.0f : logs - st.t / st.s;
}

// ---- launches ---------------------------------------------------------------------------

template <class T, class End>
hipError_t big(const ProductArgs &p, const typename T::elem *x, const typename T::elem *w,
               const uint32_t *list, const uint32_t *count, const End &end, hipStream_t stream)
{
    const uint64_t n = (((uint64_t)p.features + kBigF - 1) / kBigF) * ((p.rows + kBigR - 1) / kBigR);
    if (n > kLaunchThreads / 512) return hipErrorInvalidValue;
    // without a count the tiles are known: no workgroups for slices that there are not
    const uint32_t over = (uint32_t)(n % kBigSlots);
    const uint32_t steps = (p.k + 8 * T::kPiece - 1) / (8 * T::kPiece);
    const bool sliced = p.slices && steps >= 2 * kBigSliceSteps && (count || big_slices(over, steps) > 1);
    hipError_t e = hipSuccess;
    if (count || !sliced || n > over) {
        k_big<T, End><<<(uint32_t)((n + 7) / 8 * 8), 512, 2 * 512 * 128, stream>>>(p, x, w, list, count, end);
        e = hipGetLastError();
    }
    if (e != hipSuccess || !sliced) return e;
    k_big<T, EndSlice><<<kBigSlots, 512, 2 * 512 * 128, stream>>>(p, x, w, list, count, EndSlice{p.slices});
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const uint32_t most = count ? kBigSlots / 2 : over;
    k_slices<T, End><<<most * 32, 256, 0, stream>>>(p, count, end);
    return hipGetLastError();
}

template <class T, class End>
hipError_t mid(const ProductArgs &p, const typename T::elem *x, const typename T::elem *w,
               const uint32_t *list, const uint32_t *count, const End &end, hipStream_t stream)
{
    const uint64_t n = ((uint64_t)p.features + 63) / 64 * ((p.rows + 63) / 64);
    if (n > kLaunchThreads / 256) return hipErrorInvalidValue;
    k_mid<T, End><<<(uint32_t)((n + 7) / 8 * 8), 256, 0, stream>>>(p, x, w, list, count, end);
    return hipGetLastError();
}

template <class T, class End>
hipError_t few(const ProductArgs &p, const typename T::elem *x, const typename T::elem *w,
               const End &end, hipStream_t stream)
{
    const auto launch = [&](auto of, auto wide, auto once) {
        constexpr int kMR = decltype(of)::value, kMF = decltype(wide)::value;
        k_few<T, kMR, kMF, decltype(once)::value, End>
            <<<(p.features + 16 * kMF - 1) / (16 * kMF), (kFewWaves + kMR) * 64, few_lds<kMR, kMF>(),
               stream>>>(p, x, w, end);
    };
    const auto sized = [&](auto once) {
        const std::integral_constant<int, 1> one;
        const std::integral_constant<int, 2> two;
        const std::integral_constant<int, 3> three;
        const std::integral_constant<int, 4> four;
        if (p.rows <= 16)
            launch(one, two, once);
        else if (p.rows <= 32)
            few_features(p.rows, p.features) == 32 ? launch(two, two, once) : launch(two, four, once);
        else
            p.rows <= 48 ? launch(three, two, once) : launch(four, two, once);
    };
    // weights of bf16 5120 -> 50272 (515 MB): 8 rows 95 -> 84 us, 32 rows 119 -> 115;
    // 5120 -> 20480 (210 MB) in the cache: 34 -> 38 and 39 -> 52, out of it 43 -> 38 and 54 -> 52
    if ((uint64_t)p.features * p.k * sizeof(*w) > kLastCache)
        sized(std::true_type());
    else
        sized(std::false_type());
    return hipGetLastError();
}

template <class T, class End>
hipError_t by_shape(Shape shape, const ProductArgs &p, const typename T::elem *x, const typename T::elem *w,
                    const uint32_t *list, const uint32_t *count, const End &end, hipStream_t stream)
{
    switch (shape) {
    case Shape::few: return few<T>(p, x, w, end, stream);
    case Shape::mid: return mid<T>(p, x, w, list, count, end, stream);
    case Shape::big: break;
    }
    return big<T>(p, x, w, list, count, end, stream);
}

template <class T>
hipError_t project(const AdapterArgs &a, const void *x, uint64_t x_stride, const void *w,
                   const void *bias, const void *adapters, float *u, float *slices, void *y,
                   uint64_t y_stride, hipStream_t stream)
{
    typedef typename T::elem E;
    const E *px = static_cast<const E *>(x), *pa = static_cast<const E *>(adapters);
    int32_t *group = reinterpret_cast<int32_t *>(u + a.rows * a.rank);
    // 32 rows per workgroup where the groups are long enough to fill them and still every CU
    // gets one
    const auto shrink = [&](auto kXF, auto kAF) {
        constexpr int kX = decltype(kXF)::value, kA = decltype(kAF)::value;
        k_shrink<T, kX, kA><<<(uint32_t)(a.rows / (16 * kX) + a.n_groups), shrink_waves<kX>() * 64,
                              shrink_lds<kX, kA>(), stream>>>(a, px, x_stride, pa, u, group);
    };
    typedef std::integral_constant<int, 1> One;
    typedef std::integral_constant<int, 2> Two;
    const bool long_groups = a.rows / 32 >= kBigSlots && a.rows / a.n_groups >= 32;
    if (a.rank <= 16)
        long_groups ? shrink(Two{}, One{}) : shrink(One{}, One{});
    else
        long_groups ? shrink(Two{}, Two{}) : shrink(One{}, Two{});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
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
        k_counted<<<1, 1024, 0, stream>>>(h.targets, h.rows, list, count, h.logp, h.entropy);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const E *px = static_cast<const E *>(x), *pw = static_cast<const E *>(w);
    for (uint64_t base = 0; base < h.rows; base += kHeadPlaces) {
        const uint64_t rows = h.rows - base < kHeadPlaces ? h.rows - base : kHeadPlaces;
        const ProductArgs p = {base, rows, h.x_stride, h.k, h.features, sp.slices};
        const EndHead end = {h.features, base, rows, h.targets, list, count, sp.m, sp.s, sp.t, sp.tl};
        hipError_t e = by_shape<T>(sp.shape, p, px, pw, list, count, end, stream);
        if (e != hipSuccess) return e;
        const auto join = [&](auto of) {
            constexpr int kOf = decltype(of)::value;
            k_head_join<kOf><<<(uint32_t)((rows + kOf - 1) / kOf), 1024, 0, stream>>>(
                sp.m, sp.s, sp.t, sp.tl, sp.parts, base, rows, list, count, h.targets, h.features, h.logp,
                h.entropy);
        };
        if (rows <= 256)
            join(std::integral_constant<int, 1>{});
        else
            join(std::integral_constant<int, 8>{});
        e = hipGetLastError();
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

hipError_t launch_head_logprobs(const HeadArgs &h, bool bf16, const void *x, const void *w,
                                hipStream_t stream)
{
    return bf16 ? head<Bf16>(h, x, w, stream) : head<Fp32>(h, x, w, stream);
}

}  // namespace zo
