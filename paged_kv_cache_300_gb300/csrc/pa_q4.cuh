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

constexpr float kBf16Max = 3.3895313892515355e38f; // (2 - 2^-7) 2^127

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
    // A top code past the largest number would read back as an infinity.  Two bf16
    // steps less always do: 15 s is within 2^-7 of max - b, each step takes at least
    // that much off, and the top value is then off by 30 2^-7 s < s / 2.  The 33K-row
    // update with its read-back: 76.2 us without this, 76.7 with it.
    if (fmaf(15.f, r.step, r.low) > kBf16Max) {
        r.step = __uint_as_float(__float_as_uint(r.step) - 0x10000u);
        if (fmaf(15.f, r.step, r.low) > kBf16Max) r.step = __uint_as_float(__float_as_uint(r.step) - 0x10000u);
    }
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

// The kernels here are launched while the kernel before them may still run, and wait for
// it first (grid_dep_wait).  What it may have written is read by ordinary loads behind
// the wait: a read-only load (__ldg) is for memory that nothing writes while the kernel
// lives, and the compiler may move it, the wait notwithstanding.  Without read-only loads
// 1024 sequences take 234.3 us instead of 233.1, 96 long ones 179.3 instead of 178.6,
// 33K rows with their read-back 76.7 instead of 76.4, and the gather the same.
//
// 16 bytes of shared memory, or of global memory that is written by an earlier kernel.
template <bool SHARED, typename V>
__device__ __forceinline__ V load16(const V *p)
{
    static_assert(sizeof(V) == 16, "one 16-byte load");
    if constexpr (SHARED) {
        return *p;
    } else {
        uint4 v;
        asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(__cvta_generic_to_global(p)));
        return *reinterpret_cast<const V *>(&v);
    }
}

// A row is held by 8 neighbouring lanes, four rows a warp: lane l has the dims
// 64 c + 8 l .. + 7, c < NC = D / 64, in the type they came in (bf16 stays
// packed in pairs until a value is needed).
template <typename T, int NC>
struct Q4Row;
template <int NC>
struct Q4Row<float, NC> {
    float v[NC][8];
    template <bool SHARED = false>
    __device__ __forceinline__ void load(const float *p)
    {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 x = load16<SHARED>(reinterpret_cast<const float4 *>(p + 64 * c + i));
                v[c][i] = x.x;
                v[c][i + 1] = x.y;
                v[c][i + 2] = x.z;
                v[c][i + 3] = x.w;
            }
    }
    __device__ __forceinline__ float2 pair(int c, int i) const { return make_float2(v[c][2 * i], v[c][2 * i + 1]); }
    // extrema of the row; NaN where it holds one
    __device__ __forceinline__ void extrema(float &lo, float &hi) const
    {
        auto lower = [](float x, float y) {
            float r;
            asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
            return r;
        };
        auto upper = [](float x, float y) {
            float r;
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
            return r;
        };
        lo = hi = v[0][0];
#pragma unroll
        for (int i = 1; i < 8 * NC; ++i) {
            lo = lower(lo, v[i >> 3][i & 7]);
            hi = upper(hi, v[i >> 3][i & 7]);
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
            lo = lower(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = upper(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
    }
};
template <int NC>
struct Q4Row<__nv_bfloat16, NC> {
    uint32_t w[NC][4];
    template <bool SHARED = false>
    __device__ __forceinline__ void load(const __nv_bfloat16 *p)
    {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const uint4 x = load16<SHARED>(reinterpret_cast<const uint4 *>(p + 64 * c));
            w[c][0] = x.x;
            w[c][1] = x.y;
            w[c][2] = x.z;
            w[c][3] = x.w;
        }
    }
    __device__ __forceinline__ float2 pair(int c, int i) const
    {
        return make_float2(bf16_lo(w[c][i]), bf16_hi(w[c][i]));
    }
    // pairs at a time; then (max x, max -x) travel as one pair
    __device__ __forceinline__ void extrema(float &lo, float &hi) const
    {
        auto bf = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162 *>(&u); };
        auto un = [](__nv_bfloat162 h) { return *reinterpret_cast<const uint32_t *>(&h); };
        uint32_t a = w[0][0], b = w[0][0];
#pragma unroll
        for (int i = 1; i < 4 * NC; ++i) {
            a = un(__hmax2_nan(bf(a), bf(w[i >> 2][i & 3])));
            b = un(__hmin2_nan(bf(b), bf(w[i >> 2][i & 3])));
        }
        b ^= 0x80008000u;
        uint32_t m = un(__hmax2_nan(bf(__byte_perm(a, b, 0x5410)), bf(__byte_perm(a, b, 0x7632))));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = un(__hmax2_nan(bf(m), bf(__shfl_xor_sync(0xffffffffu, m, o))));
        hi = bf16_lo(m);
        lo = -bf16_hi(m);
    }
};

// Two fp32 numbers to a register pair, which one instruction works on.
__device__ __forceinline__ uint64_t f32x2(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}

// Quantises a row: s is its scale, c the lane's codes, 4 bits each.
template <typename T, int NC>
__device__ __forceinline__ void q4_quantise(const Q4Row<T, NC> &x, Q4Scale &s, uint32_t (&c)[NC])
{
    float lo, hi;
    x.extrema(lo, hi);
    s = q4_scale(lo, hi, fabsf(lo) < INFINITY && fabsf(hi) < INFINITY); // false for NaN
    // n = round-half-even((x / 16 - b / 16) * (16 / s)), which lies in 0..15: the
    // sum with 2^23 rounds it into the low bits.  x / 16 is exact, so the first
    // step is one rounding as a fused operation too.  The product is rounded
    // before the sum: a packed mul, or an fma with a constant -0, is fused with
    // the packed add behind it all the same, so it is an fma with a computed -0.
    // The sums of the bits leave out 0x4b000000 (the bits of 2^23) at every
    // step; only the first two places keep something of it.
    const uint64_t sixteenth = f32x2(0.0625f, 0.0625f), low = f32x2(-s.low16, -s.low16), inv = f32x2(s.inv16, s.inv16),
                   big = f32x2(8388608.f, 8388608.f);
    const float zero = __fmul_rn(s.inv16, -0.f);
    const uint64_t minus_zero = f32x2(zero, zero);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        uint32_t n = 0;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            const float2 v = x.pair(k, i);
            uint32_t n0, n1;
            asm("{\n\t.reg .b64 t;\n\t"
                "fma.rn.f32x2 t, %2, %3, %4;\n\t"
                "fma.rn.f32x2 t, t, %5, %7;\n\t"
                "add.rn.f32x2 t, t, %6;\n\t"
                "mov.b64 {%0, %1}, t;\n\t}"
                : "=r"(n0), "=r"(n1)
                : "l"(f32x2(v.x, v.y)), "l"(sixteenth), "l"(low), "l"(inv), "l"(big),
                  "l"(minus_zero));
            n = (n * 16u + n1) * 16u + n0;
        }
        c[k] = s.inv16 > 0.f ? n - 0xfb000000u : 0u;
    }
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
