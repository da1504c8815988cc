// k_q4.hip -- weights in 4 bits with group scales: w[f][k] = s (q[f][k] - z), q in 0..15, s and z of
// feature f and of k's group (z = 8 where none are given).
//   zo_q4_quantize, zo_q4_pack, zo_q4_unpack   to and from the codes' blocks;
//   zo_q4_project   y = x w^T + bias + scale (x A_g^T) B_g^T, as zo_adapter_project.
//
// Blocks.  16 features x 128 values of k lie in 1024 bytes, the order in which a wave uses them:
// lane 16 q + l of a wave loads the 16 bytes of feature l and of 32 values of k, and each 4 bytes c of these
// are its operand of one product of 32 values, k = 32 c + 8 q + 0 .. 7.  The eight codes of 4
// bytes lie so that (bytes >> 4 i) & 0x000F000F holds codes 2 i and 2 i + 1.
#include "zo_product.hpp"

namespace zo {
namespace {

constexpr uint32_t kBlockF = 16, kBlockK = 128;

// Where code j (of eight) lies in its 4 bytes.
__device__ __forceinline__ constexpr int code_shift(int j) { return (j & 1) * 16 + (j >> 1) * 4; }

// ---- codes ------------------------------------------------------------------------------

template <class T>
__device__ __forceinline__ void load8(const typename T::elem *p, float *v)
{
    T::load4(p, v);
    T::load4(p + 4, v + 4);
}
__device__ __forceinline__ void store8(float *p, const float *v)
{
    *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4 *>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(uint16_t *p, const float *v)
{
    *reinterpret_cast<u32x4 *>(p) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                          pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}
__device__ __forceinline__ float rounded(float v, const float *) { return v; }
__device__ __forceinline__ float rounded(float v, const uint16_t *) { return bf16lo_to_f32(pack_bf16x2(v, 0.0f)); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = (uint16_t)pack_bf16x2(v, 0.0f); }

// A block of codes per wave.
struct BlockAt {
    uint32_t f, k;          // this lane's feature and first value of k
    uint64_t block;
    bool there;             // the block is
    __device__ __forceinline__ BlockAt(uint32_t d_out, uint32_t d_in)
    {
        const uint32_t nk = (d_in + kBlockK - 1) / kBlockK;
        const int lane = threadIdx.x & 63;
        block = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
        const uint64_t fb = block / nk;
        there = fb * kBlockF < d_out;
        f = (uint32_t)fb * kBlockF + (lane & 15);
        k = (uint32_t)(block - fb * nk) * kBlockK + (lane >> 4) * 8;
    }
};

// s = max |w| / 7 over a group, rounded to the type; q - 8 is the whole number nearest to w / s,
// ties to even, found exactly: the remainder w - q s of a quotient that is off by at most one
// is a number of fp32.  A group of zeros has the scale 0 and the codes 8; one that holds an
// infinity or a NaN has the scale NaN.
template <class T, int kGroup>
__global__ __launch_bounds__(256) void k_quantize(const typename T::elem *w, uint64_t stride, uint32_t d_out,
                                                  uint32_t d_in, u32x4 *codes, typename T::elem *scales)
{
    constexpr int kC = kGroup / 32;                 // products of 32 values in a group
    const BlockAt b(d_out, d_in);
    if (!b.there) return;
    const int lane = threadIdx.x & 63;
    float v[4][8];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const bool in = b.f < d_out && b.k + 32 * c < d_in;
        if (in) load8<T>(w + (uint64_t)b.f * stride + b.k + 32 * c, v[c]);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = in ? v[c][j] : 0.0f;
    }
    u32x4 out;
#pragma unroll
    for (int c0 = 0; c0 < 4; c0 += kC) {
        float top = 0.0f, sum = 0.0f;
#pragma unroll
        for (int c = c0; c < c0 + kC; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                top = fmaxf(top, fabsf(v[c][j]));
                sum += v[c][j] * 0.0f;              // NaN where something is not finite
            }
        for (int o = 16; o < 64; o <<= 1) {
            top = fmaxf(top, __shfl_xor(top, o));
            sum += __shfl_xor(sum, o);
        }
        const float s = rounded(sum == 0.0f ? top / 7.0f : __builtin_nanf(""), w);
        // away from the ends of the exponent's range, where 1 / s would be lost
        const float up = s < 0x1p-64f ? 0x1p64f : s > 0x1p64f ? 0x1p-64f : 1.0f;
        const float t = s * up, inv = s > 0.0f ? 1.0f / t : 0.0f;
#pragma unroll
        for (int c = c0; c < c0 + kC; ++c) {
            uint32_t word = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = v[c][j] * up;
                float q = rintf(x * inv);
                const float r = 2.0f * fmaf(-q, t, x);          // exact
                const bool odd = ((int)q & 1) != 0;
                if (r > t || (r == t && odd)) q += 1.0f;
                else if (r < -t || (r == -t && odd)) q -= 1.0f;
                q = s > 0.0f ? fminf(fmaxf(q, -8.0f), 7.0f) : 0.0f;
                word |= (uint32_t)((int)q + 8) << code_shift(j);
            }
            out[c] = word;
        }
        const uint32_t k0 = b.k - (lane >> 4) * 8 + 32 * c0;
        if (lane < 16 && b.f < d_out && k0 < d_in) store1(scales + (uint64_t)(k0 / kGroup) * d_out + b.f, s);
    }
    codes[b.block * 64 + lane] = out;
}

// One value, 0 .. 15, a byte.
__global__ __launch_bounds__(256) void k_pack(const uint8_t *values, uint32_t d_out, uint32_t d_in, u32x4 *codes)
{
    const BlockAt b(d_out, d_in);
    if (!b.there) return;
    u32x4 out = {0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (b.f >= d_out || b.k + 32 * c >= d_in) continue;
        const uint2 v = *reinterpret_cast<const uint2 *>(values + (uint64_t)b.f * d_in + b.k + 32 * c);
#pragma unroll
        for (int j = 0; j < 8; ++j) out[c] |= ((j < 4 ? v.x : v.y) >> 8 * (j & 3) & 15u) << code_shift(j);
    }
    codes[b.block * 64 + (threadIdx.x & 63)] = out;
}

template <class T>
__global__ __launch_bounds__(256) void k_unpack(const u32x4 *codes, const typename T::elem *scales,
                                                const typename T::elem *zeros, uint32_t d_out, uint32_t d_in,
                                                uint32_t group, typename T::elem *w)
{
    const BlockAt b(d_out, d_in);
    if (!b.there || b.f >= d_out) return;
    const u32x4 word = codes[b.block * 64 + (threadIdx.x & 63)];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint32_t k = b.k + 32 * c;
        if (k >= d_in) continue;
        const uint64_t at = (uint64_t)(k / group) * d_out + b.f;
        const float s = T::widen(scales[at]), z = zeros ? T::widen(zeros[at]) : 8.0f;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = ((float)(word[c] >> code_shift(j) & 15u) - z) * s;
        store8(w + (uint64_t)b.f * d_in + k, v);
    }
}

// ---- few rows ---------------------------------------------------------------------------

// Codes as operands, exactly: bf16 kOffset + q (seven bits behind the leading one hold 128 + q),
// fp32 q.
struct CodesBf16 {
    typedef Bf16 T;
    static constexpr float kOffset = 128.0f;
    static constexpr int kParts = 1;                // pieces of the eight values
    static __device__ __forceinline__ u32x4 part(uint32_t w, int)
    {
        u32x4 f;
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = (w >> (4 * i) & 0x000F000Fu) | 0x43004300u;
        return f;
    }
    static __device__ __forceinline__ u32x4 ones() { return u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}; }
};
struct CodesFp32 {
    typedef Fp32 T;
    static constexpr float kOffset = 0.0f;
    static constexpr int kParts = 2;
    static __device__ __forceinline__ u32x4 part(uint32_t w, int h)
    {
        u32x4 f;
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __float_as_uint((float)(w >> code_shift(4 * h + i) & 15u));
        return f;
    }
    static __device__ __forceinline__ u32x4 ones()
    {
        const uint32_t o = __float_as_uint(1.0f);
        return u32x4{o, o, o, o};
    }
};

struct Q4Args {
    uint64_t rows, x_stride;
    uint32_t d_in, d_out, blocks;                   // blocks along k
};

// Few rows.  What bounds the product is reading the codes once: a workgroup takes 16 kMF features
// and all rows, four waves take every fourth block of k, and their sums meet in LDS; kMR more waves
// form the adapters' products meanwhile, add everything up and end 16 rows each (as k_few).
// Codes go straight to registers, a block a load; x through LDS.  A group's sum of products with codes is formed apart
// and enters the row's sum as s (sum x (o + q) - (o + z) sum x), the sums of x by products with
// ones, so that the weights are not rounded: every product is exact, all sums are fp32.
constexpr int kQ4Waves = 4;
template <class T, int kMR>
constexpr int q4_stages() { return T::kBf16 ? (kMR <= 2 ? 3 : 2) : (kMR == 1 ? 3 : 2); }
template <class T>
constexpr int q4_steps() { return kBlockK / (8 * T::kPiece); }
template <class T, int kMR>
constexpr uint32_t q4_lds() { return kQ4Waves * q4_stages<T, kMR>() * q4_steps<T>() * kMR * 16 * 128; }

template <class C, int kMR, int kMF, int kSplit, bool kZeros, class End>
__global__ __launch_bounds__((kQ4Waves + kMR) * 64) void k_q4_few(Q4Args p, const typename C::T::elem *x,
                                                                  const u32x4 *codes,
                                                                  const typename C::T::elem *scales,
                                                                  const typename C::T::elem *zeros, End end)
{
    typedef typename C::T T;
    constexpr int kStages = q4_stages<T, kMR>(), kSteps = q4_steps<T>(), kC = 4 / kSplit;
    typedef Feed<T, kMR, kStages * kSteps> F;
    static_assert(F::kStep * kSteps == kBlockK, "whole steps of x in a block");
    static_assert(kMF * kMR * 1024 * kQ4Waves <= (int)q4_lds<T, kMR>(), "the sums fit");
    extern __shared__ u32x4 stage[];                // [wave][stage][step][rows], then [wave] of sums
    const int lane = threadIdx.x & 63, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t f0 = blockIdx.x * (16 * kMF);
    f32x4 *sums = reinterpret_cast<f32x4 *>(stage);
    if (wave >= kQ4Waves) {
        const int n = wave - kQ4Waves;
        Tile<kMF, 1> own;
        own.clear();
        end.add_rows(own, 0, f0, 16 * n);
        __syncthreads();                            // the stages are free
        __syncthreads();                            // the sums are there
#pragma unroll
        for (int m = 0; m < kMF; ++m)
#pragma unroll
            for (int v = 0; v < kQ4Waves; ++v) own.acc[m][0] += sums[((v * kMF + m) * kMR + n) * 64 + lane];
        end.store(own, f0, 16 * n);
        return;
    }
    const F feed(stage + wave * kStages * kSteps * F::kStage, p.d_in, [&](int i) {
        const uint64_t r = (uint64_t)i < p.rows ? i : p.rows - 1;
        return x + r * p.x_stride;
    });
    Tile<kMF, kMR> t;
    t.clear();
    u32x4 word[kStages][kMF];
    f32x4 s[kStages][kMF][kSplit], z[kStages][kMF][kSplit];
    // features and groups past the last read the last: nothing of theirs is kept
    const uint32_t groups = (p.d_in + kC * 32 - 1) / (kC * 32);
    const u32x4 *from[kMF];
    uint32_t of[kMF];
#pragma unroll
    for (int m = 0; m < kMF; ++m) {
        const uint32_t f = f0 + 16 * m < p.d_out ? f0 + 16 * m : f0;
        from[m] = codes + (uint64_t)(f / 16) * p.blocks * 64 + lane;
        of[m] = f + 4 * q < p.d_out ? f + 4 * q : f;
    }
    const auto issue = [&](uint32_t b, int slot) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) feed.issue(b * kSteps + i, slot * kSteps + i);
        const uint32_t at = b < p.blocks ? b : p.blocks - 1;
#pragma unroll
        for (int m = 0; m < kMF; ++m) {
            word[slot][m] = from[m][(uint64_t)at * 64];
#pragma unroll
            for (int g = 0; g < kSplit; ++g) {
                const uint32_t group = at * kSplit + g < groups ? at * kSplit + g : groups - 1;
                float v[4];
                T::load4(scales + (uint64_t)group * p.d_out + of[m], v);
                s[slot][m][g] = f32x4{v[0], v[1], v[2], v[3]};
                if constexpr (kZeros) {
                    T::load4(zeros + (uint64_t)group * p.d_out + of[m], v);
                    z[slot][m][g] = f32x4{v[0], v[1], v[2], v[3]};
                }
            }
        }
        asm volatile("" ::: "memory");              // a wait counts whole blocks' loads
    };
    constexpr int kLoads = F::kLoads * kSteps + kMF * (1 + kSplit * (kZeros ? 2 : 1));
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(wave + i * kQ4Waves, i);
    for (uint32_t b0 = wave; b0 < p.blocks; b0 += kQ4Waves * kStages) {
#pragma unroll
        for (int u = 0; u < kStages; ++u) {
            const uint32_t b = b0 + u * kQ4Waves;
            wait_for<kLoads * (kStages - 2), true>();
            asm volatile("" ::: "memory");
            issue(b + (kStages - 1) * kQ4Waves, (u + kStages - 1) % kStages);
#pragma unroll
            for (int g = 0; g < kSplit; ++g) {
                f32x4 part[kMF][kMR], sum[kMR];
#pragma unroll
                for (int n = 0; n < kMR; ++n) {
                    sum[n] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int m = 0; m < kMF; ++m) part[m][n] = f32x4{0, 0, 0, 0};
                }
#pragma unroll
                for (int c = g * kC; c < (g + 1) * kC; ++c)
#pragma unroll
                    for (int h = 0; h < C::kParts; ++h) {
                        // values 32 c + 8 q + 4 h .. of the block: bf16 fragment c % 2 of step
                        // c / 2; fp32 pieces 2 q + h of step c
                        u32x4 fx[kMR];
#pragma unroll
                        for (int n = 0; n < kMR; ++n) {
                            if constexpr (T::kBf16) {
                                fx[n] = feed.fragment(u * kSteps + c / 2, n, c % 2);
                            } else {
                                const int l16 = lane & 15;
                                fx[n] = feed.lds[(u * kSteps + c) * F::kStage + (n * 16 + l16) * F::kPieces +
                                                 ((2 * q + h) ^ (l16 >> 1))];
                            }
                            sum[n] = T::mma(C::ones(), fx[n], sum[n]);
                        }
#pragma unroll
                        for (int m = 0; m < kMF; ++m) {
                            const u32x4 fw = C::part(word[u][m][c], h);
#pragma unroll
                            for (int n = 0; n < kMR; ++n) part[m][n] = T::mma(fw, fx[n], part[m][n]);
                        }
                    }
#pragma unroll
                for (int m = 0; m < kMF; ++m)
#pragma unroll
                    for (int n = 0; n < kMR; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float zero = C::kOffset + (kZeros ? z[u][m][g][i] : 8.0f);
                            t.acc[m][n][i] = fmaf(s[u][m][g][i], fmaf(-zero, sum[n][i], part[m][n][i]), t.acc[m][n][i]);
                        }
            }
        }
    }
    wait_for<0, true>();
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kMF; ++m)
#pragma unroll
        for (int n = 0; n < kMR; ++n) sums[((wave * kMF + m) * kMR + n) * 64 + lane] = t.acc[m][n];
    __syncthreads();
}

// ---- launches ---------------------------------------------------------------------------

uint32_t block_grid(uint32_t d_out, uint32_t d_in)
{
    const uint64_t blocks = ((uint64_t)d_out + kBlockF - 1) / kBlockF * (((uint64_t)d_in + kBlockK - 1) / kBlockK);
    return (uint32_t)((blocks + 3) / 4);
}

template <class C, int kMR, int kMF>
hipError_t few_q4(const AdapterArgs &a, const Q4Weights &w, const void *x, uint64_t x_stride, const void *bias,
                  const void *adapters, float *u, void *y, uint64_t y_stride, hipStream_t stream)
{
    typedef typename C::T T;
    typedef typename T::elem E;
    const EndProject<T> end = {a, u, reinterpret_cast<int32_t *>(u + a.rows * a.rank), static_cast<const E *>(adapters),
                               static_cast<const E *>(bias), static_cast<E *>(y), y_stride};
    const Q4Args p = {a.rows, x_stride, a.d_in, a.d_out, (a.d_in + kBlockK - 1) / kBlockK};
    const auto launch = [&](auto split, auto zeros) {
        k_q4_few<C, kMR, kMF, decltype(split)::value, decltype(zeros)::value, EndProject<T>>
            <<<(a.d_out + 16 * kMF - 1) / (16 * kMF), (kQ4Waves + kMR) * 64, q4_lds<T, kMR>(), stream>>>(
                p, static_cast<const E *>(x), static_cast<const u32x4 *>(w.codes), static_cast<const E *>(w.scales),
                static_cast<const E *>(w.zeros), end);
    };
    const auto sized = [&](auto zeros) {
        if (w.group == 128) launch(std::integral_constant<int, 1>(), zeros);
        else if (w.group == 64) launch(std::integral_constant<int, 2>(), zeros);
        else launch(std::integral_constant<int, 4>(), zeros);
    };
    w.zeros ? sized(std::true_type()) : sized(std::false_type());
    return hipGetLastError();
}

template <class C, int kMR, int kMF>
hipError_t prepare_few()
{
    typedef typename C::T T;
    hipError_t e = hipSuccess;
    const auto raise = [&](auto split, auto zeros) {
        if (e == hipSuccess)
            e = hipFuncSetAttribute(reinterpret_cast<const void *>(
                                        &k_q4_few<C, kMR, kMF, decltype(split)::value, decltype(zeros)::value, EndProject<T>>),
                                    hipFuncAttributeMaxDynamicSharedMemorySize, q4_lds<T, kMR>());
    };
    const auto both = [&](auto split) {
        raise(split, std::true_type());
        raise(split, std::false_type());
    };
    both(std::integral_constant<int, 1>());
    both(std::integral_constant<int, 2>());
    both(std::integral_constant<int, 4>());
    return e;
}

}  // namespace

hipError_t prepare_q4()
{
    const hipError_t all[] = {prepare_few<CodesBf16, 1, 2>(), prepare_few<CodesBf16, 2, 2>(), prepare_few<CodesBf16, 3, 2>(),
                              prepare_few<CodesBf16, 4, 2>(), prepare_few<CodesFp32, 1, 2>(), prepare_few<CodesFp32, 2, 2>()};
    for (const hipError_t e : all)
        if (e != hipSuccess) return e;
    return hipSuccess;
}

hipError_t launch_q4_quantize(const void *w, uint64_t stride, bool bf16, uint32_t d_out, uint32_t d_in, uint32_t group,
                              void *codes, void *scales, hipStream_t stream)
{
    const uint32_t n = block_grid(d_out, d_in);
    const auto typed = [&](auto t) {
        typedef decltype(t) T;
        typedef typename T::elem E;
        const auto launch = [&](auto size) {
            k_quantize<T, decltype(size)::value><<<n, 256, 0, stream>>>(
                static_cast<const E *>(w), stride, d_out, d_in, static_cast<u32x4 *>(codes), static_cast<E *>(scales));
        };
        if (group == 128) launch(std::integral_constant<int, 128>());
        else if (group == 64) launch(std::integral_constant<int, 64>());
        else launch(std::integral_constant<int, 32>());
    };
    bf16 ? typed(Bf16()) : typed(Fp32());
    return hipGetLastError();
}

hipError_t launch_q4_pack(const uint8_t *values, uint32_t d_out, uint32_t d_in, void *codes, hipStream_t stream)
{
    k_pack<<<block_grid(d_out, d_in), 256, 0, stream>>>(values, d_out, d_in, static_cast<u32x4 *>(codes));
    return hipGetLastError();
}

hipError_t launch_q4_unpack(const Q4Weights &q, bool bf16, uint32_t d_out, uint32_t d_in, void *w, hipStream_t stream)
{
    const auto typed = [&](auto t) {
        typedef decltype(t) T;
        typedef typename T::elem E;
        k_unpack<T><<<block_grid(d_out, d_in), 256, 0, stream>>>(
            static_cast<const u32x4 *>(q.codes), static_cast<const E *>(q.scales), static_cast<const E *>(q.zeros), d_out,
            d_in, q.group, static_cast<E *>(w));
    };
    bf16 ? typed(Bf16()) : typed(Fp32());
    return hipGetLastError();
}

hipError_t launch_q4_project(const AdapterArgs &a, bool bf16, const void *x, uint64_t x_stride, const Q4Weights &w,
                             const void *bias, const void *adapters, float *u, float *slices, void *unpacked, void *y,
                             uint64_t y_stride, hipStream_t stream)
{
    if (!q4_few(a.rows, bf16)) {
        const hipError_t e = launch_q4_unpack(w, bf16, a.d_out, a.d_in, unpacked, stream);
        if (e != hipSuccess) return e;
        return launch_adapter_project(a, bf16, x, x_stride, unpacked, bias, adapters, u, slices, y, y_stride, stream);
    }
    const hipError_t e = launch_adapter_shrink(a, bf16, x, x_stride, adapters, u, stream);
    if (e != hipSuccess) return e;
    const auto few = [&](auto codes, auto rows) {
        return few_q4<decltype(codes), decltype(rows)::value, 2>(a, w, x, x_stride, bias, adapters, u, y, y_stride, stream);
    };
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    if (!bf16) return a.rows <= 16 ? few(CodesFp32(), one) : few(CodesFp32(), two);
    if (a.rows <= 16) return few(CodesBf16(), one);
    if (a.rows <= 32) return few(CodesBf16(), two);
    return a.rows <= 48 ? few(CodesBf16(), std::integral_constant<int, 3>()) : few(CodesBf16(), std::integral_constant<int, 4>());
}

}  // namespace zo
