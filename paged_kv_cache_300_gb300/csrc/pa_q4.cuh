// Format of the 4-bit paged pool, shared by the kernels that write and read
// it.  The format itself is stated in include/pa.h ("The 4-bit pool").
#pragma once

#include "pa_common.cuh"

namespace pa {

// Bytes of one record (one kv head of one block) and where its parts start.
__host__ __device__ constexpr int q4_record_bytes(int d, int bs) { return bs * (d + 8); }
__host__ __device__ constexpr int q4_v_offset(int d, int bs) { return bs * d / 2; }
__host__ __device__ constexpr int q4_scale_offset(int d, int bs) { return bs * d; }

// Number of the 16-bit unit that holds dims 4x..4x+3 of token t's value.
template <int D>
__device__ __forceinline__ int q4_v_unit(int t, int x)
{
    const int p = t >> 1;
    const int u = (x >> 3) ^ ((D == 128 ? p : p >> 1) & (D / 32 - 1));
    return 2 * (p * (D / 4) + u * 8 + (x & 7)) + (t & 1);
}

// Step, low and 16 / step of a row with the given extrema.  Each operation
// is rounded on its own (no contraction), because the codes are defined by
// these fp32 steps.
struct Q4Scale {
    float step, low;
    float low16; // low / 16
    float inv16; // 16 / step; 0 when every code is 0
};
// fp32 -> the next bf16 away from zero (bits), still in an fp32 register.
__device__ __forceinline__ float bf16_away(float x)
{
    return __uint_as_float((__float_as_uint(x) + 0xffffu) & 0xffff0000u);
}
// 1 / s for a positive bf16 s between 2^-100 and 2^125, correctly rounded: one
// Newton step with fused operations (Markstein).  The residual e = 1 - s r of
// an approximation within 2^-22 is exact (s has 8 bits, r has 24), r + r e is
// off by e^2 <= 2^-44 of it, and 1 / s of an 8-bit s is at least 2^-33 of it
// away from any rounding border.
__device__ __forceinline__ float q4_reciprocal(float s)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return fmaf(r, fmaf(-s, r, 1.f), r);
}
__device__ __forceinline__ Q4Scale q4_scale(float lo, float hi, bool finite)
{
    Q4Scale r;
    r.low = lo < 0.f ? bf16_away(lo) : __uint_as_float(__float_as_uint(lo) & 0xffff0000u);
    r.low16 = __fmul_rn(r.low, 0.0625f);
    const float range = __fmul_rn(__fsub_rn(__fmul_rn(hi, 0.0625f), r.low16), 16.0f / 15.0f);
    r.step = range < 7.888609052210118e-31f /* 2^-100 */ ? 0.f : bf16_away(range);
    if (!finite || fabsf(r.low) == INFINITY) {
        r.step = r.low = __int_as_float(0x7fc00000);
        r.inv16 = 0.f;
        r.low16 = 0.f;
    } else {
        r.inv16 = r.step > 0.f ? 16.0f * q4_reciprocal(r.step) : 0.f;
    }
    return r;
}
__device__ __forceinline__ float q4_value(uint32_t n, float step, float low)
{
    return fmaf((float)n, step, low); // n * step is exact
}
// Two bf16 (step, low) as one 32-bit word; the values are bf16 already.
__device__ __forceinline__ uint32_t q4_pack_scale(const Q4Scale &s)
{
    return (__float_as_uint(s.step) >> 16) | (__float_as_uint(s.low) & 0xffff0000u);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// N values of a row in the type they came in: bf16 stays packed in pairs until
// a value is needed.
template <typename T, int N>
struct Q4Row;
template <int N>
struct Q4Row<float, N> {
    float v[N];
    __device__ __forceinline__ void load(const float *p)
    {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(p + i));
            v[i] = x.x;
            v[i + 1] = x.y;
            v[i + 2] = x.z;
            v[i + 3] = x.w;
        }
    }
    __device__ __forceinline__ float get(int i) const { return v[i]; }
    // extrema over 16 neighbouring lanes; NaN anywhere leaves finite false
    __device__ __forceinline__ void extrema(float &lo, float &hi, bool &finite) const
    {
        lo = hi = v[0];
        bool ok = fabsf(v[0]) < INFINITY;
#pragma unroll
        for (int i = 1; i < N; ++i) {
            lo = fminf(lo, v[i]);
            hi = fmaxf(hi, v[i]);
            ok = ok && fabsf(v[i]) < INFINITY;
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        const unsigned row = 0xffffu << (threadIdx.x & 16);
        finite = (__ballot_sync(0xffffffffu, ok) & row) == row;
    }
};
template <int N>
struct Q4Row<__nv_bfloat16, N> {
    uint32_t w[N / 2];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p)
    {
        if constexpr (N == 8) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p));
            w[0] = x.x;
            w[1] = x.y;
            w[2] = x.z;
            w[3] = x.w;
        } else {
            const uint2 x = __ldg(reinterpret_cast<const uint2 *>(p));
            w[0] = x.x;
            w[1] = x.y;
        }
    }
    __device__ __forceinline__ float get(int i) const { return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); }
    // pairs at a time; then (max x, max -x) travel as one pair.  max with
    // NaN is NaN here.
    __device__ __forceinline__ void extrema(float &lo, float &hi, bool &finite) const
    {
        auto bf = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162 *>(&u); };
        auto un = [](__nv_bfloat162 h) { return *reinterpret_cast<const uint32_t *>(&h); };
        uint32_t a = w[0], b = w[0] ^ 0x80008000u;
#pragma unroll
        for (int i = 1; i < N / 2; ++i) {
            a = un(__hmax2_nan(bf(a), bf(w[i])));
            b = un(__hmax2_nan(bf(b), bf(w[i] ^ 0x80008000u)));
        }
        uint32_t m = un(__hmax2_nan(bf(__byte_perm(a, b, 0x5410)), bf(__byte_perm(a, b, 0x7632))));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = un(__hmax2_nan(bf(m), bf(__shfl_xor_sync(0xffffffffu, m, o))));
        hi = bf16_lo(m);
        lo = -bf16_hi(m);
        finite = fabsf(hi) < INFINITY && fabsf(lo) < INFINITY; // false for NaN
    }
};

// Quantises a row held by 16 neighbouring lanes, EPL = D / 16 values each (two
// rows a warp): s is the row's scale, the result the lane's codes, 4 bits each.
template <typename T, int EPL>
__device__ __forceinline__ uint32_t q4_half_warp(const Q4Row<T, EPL> &x, Q4Scale &s)
{
    float lo, hi;
    bool finite;
    x.extrema(lo, hi, finite);
    s = q4_scale(lo, hi, finite);
    // n = round-half-even((x / 16 - b / 16) * (16 / s)), which lies in 0..15: the
    // sum with 2^23 rounds it into the low bits.  x / 16 is exact, so the first
    // step is one rounding as a fused operation too; the product is not fused.
    // The sums of the bits leave out 0x4b000000 (the bits of 2^23) at every
    // step; only the first two places keep something of it.
    uint32_t c = 0;
#pragma unroll
    for (int i = EPL - 1; i >= 0; --i)
        c = c * 16u + __float_as_uint(__fadd_rn(__fmul_rn(fmaf(x.get(i), 0.0625f, -s.low16), s.inv16), 8388608.f));
    c -= 0xfb000000u;
    return s.inv16 > 0.f ? (EPL == 8 ? c : c & 0xffffu) : 0u;
}

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x)
{
    return x;
}
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x)
{
    return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x)
{
    return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x)
{
    return __float2bfloat16_rn(x);
}

// Four consecutive elements, rounded once.
__device__ __forceinline__ void store4(float *p, float a, float b, float c, float d)
{
    *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float a, float b, float c, float d)
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(a, b), pack_bf16(c, d));
}

}  // namespace pa
