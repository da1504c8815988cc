// zo_lm.hpp -- device helpers of the language-model operators (k_token, k_project): softmax
// statistics in one pass, against e and against 2, and clamped row indices.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "zo_device.hpp"
#include "zo_launch.hpp"

namespace zo {

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float fast_exp(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

// Running softmax statistics: m the largest value so far, s = sum e^{x - m}, t = sum
// e^{x - m} (x - m).  Values of -inf add nothing (m stays -inf while there are only those);
// a NaN, or +inf, makes s NaN.
struct SoftStats {
    float m, s, t;

    static __device__ __forceinline__ SoftStats empty() { return {-INFINITY, 0.0f, 0.0f}; }

    // Make the maximum at least `top`.
    __device__ __forceinline__ void raise(float top)
    {
        if (top > m) {
            const float d = m - top;
            const float r = fast_exp(d);               // 0 from m = -inf, where s = t = 0
            t = r > 0.0f ? (t + s * d) * r : t * 0.0f;  // t * 0 keeps a NaN
            s *= r;
            m = top;
        }
    }
    // Add x <= m (or NaN).  The bound on d keeps 0 * -inf out of t: e is 0 far above it.
    __device__ __forceinline__ void add(float x)
    {
        const float d = x - (m == -INFINITY ? 0.0f : m);
        const float e = fast_exp(d);
        s += e;
        t = fmaf(e, fmaxf(d, -1e4f), t);
    }
    __device__ __forceinline__ void merge(const SoftStats &o)
    {
        raise(o.m);
        const float d = o.m - m;                        // <= 0; NaN if both are infinite
        const float r = o.m == m ? 1.0f : fast_exp(d);
        s += o.s * r;
        t += o.m == m ? o.t : (r > 0.0f ? (o.t + o.s * d) * r : 0.0f);
    }
    __device__ __forceinline__ void wave_merge(int from = kWave / 2, int to = 1)
    {
        for (int o = from; o >= to; o >>= 1) {
            SoftStats b;
            b.m = __shfl_xor(m, o);
            b.s = __shfl_xor(s, o);
            b.t = __shfl_xor(t, o);
            merge(b);
        }
    }
};

// The same statistics against powers of two, one operation a value shorter: with m2 = m log2 e,
// rounded, s = sum 2^y and t = sum 2^y y over y = x log2 e - m2, one multiply-add each.  m
// starts at -kReach: lower values, masks among them, add nothing.  Up to |m| = kReach the
// rounding of m2 moves y by 1/16 at most; it is the same for all y and natural() takes it out.
struct BinaryStats {
    static constexpr float kReach = 1048576.0f;
    float m, m2, s, t;

    static __device__ __forceinline__ BinaryStats empty() { return {-kReach, -kReach * kLog2e, 0.0f, 0.0f}; }
    __device__ __forceinline__ void raise(float top)
    {
        if (top > m) {
            const float next = top * kLog2e, d = m2 - next;
            const float r = __builtin_amdgcn_exp2f(d);
            t = r > 0.0f ? fmaf(s, d, t) * r : t * 0.0f;   // t * 0 keeps a NaN
            s *= r;
            m = top;
            m2 = next;
        }
    }
    __device__ __forceinline__ void add(float x)
    {
        const float y = fmaf(x, kLog2e, -m2);
        const float e = __builtin_amdgcn_exp2f(y);
        s += e;
        t = fmaf(e, fmaxf(y, -1e4f), t);       // y = -inf: e is 0, add 0
    }
    // y = (x - m) log2 e + c.
    __device__ __forceinline__ SoftStats natural() const
    {
        const float c = fmaf(m, kLog2e, -m2), f = __builtin_amdgcn_exp2f(-c);
        return {m, s * f, fmaf(-c, s, t) * f * 0.69314718055994530942f};
    }
    // Whether joined statistics are within reach: the maximum not above it, nor so far below
    // that the sum has lost it.  NaN and +inf are NaN either way.
    static __device__ __forceinline__ bool holds(const SoftStats &all)
    {
        return !(all.s < 0.5f) && !(all.m > kReach && all.m < INFINITY);
    }
};

// A row index from device memory, forced into [0, rows].
__device__ __forceinline__ uint64_t clamp_row(int64_t r, uint64_t rows)
{
    return r < 0 ? 0 : ((uint64_t)r > rows ? rows : (uint64_t)r);
}

}  // namespace zo
