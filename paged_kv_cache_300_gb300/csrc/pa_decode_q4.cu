// Decode attention over the 4-bit paged pool (include/pa.h, pa_decode_q4).
#include "pa_internal.h"
#include "pa_q4.cuh"

#include <math.h>

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// Quantises one row held as EPL values a lane (dims lane*EPL ..) by a whole
// warp; returns the lane's codes, 4 bits each.
template <int EPL>
__device__ __forceinline__ uint32_t quantise_row(const float (&x)[EPL], Q4Scale &s)
{
    float lo = INFINITY, hi = -INFINITY;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        finite = finite && fabsf(x[i]) < INFINITY;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
    }
    s = q4_scale(lo, hi, __all_sync(kFull, finite));
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) c |= q4_code(x[i], s) << (4 * i);
    return c;
}

// One warp per (sequence, query head), fp32 arithmetic throughout.
template <int D, typename T>
__global__ void __launch_bounds__(128) decode_q4_kernel(const DecodeQ4Args a)
{
    constexpr int EPL = D / 32;
    const int lane = threadIdx.x & 31;
    const long long gw = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (gw >= (long long)a.batch * a.num_heads) return;
    const int b = (int)(gw / a.num_heads), h = (int)(gw % a.num_heads);
    const int G = a.group, kvh = h / G, Hkv = a.num_kv_heads, bs = a.block_size;
    const int mbps = a.max_blocks_per_seq, L = a.cache_seqlens[b];
    T *out = static_cast<T *>(a.out) + ((size_t)b * a.num_heads + h) * D + lane * EPL;
    bool bad = L < 0 || (long long)L + 1 > (long long)mbps * bs;
    if (bad && lane == 0) flag_error(a.dev_err, PA_DEVERR_OVERFLOW);
    const int nblk = bad ? 0 : L / bs + 1;
    const int32_t *tab = a.block_table + (size_t)b * mbps;
    for (int j = 0; j < nblk && !bad; ++j)
        if (tab[j] < 0 || tab[j] >= a.num_blocks) {
            bad = true;
            if (lane == 0) flag_error(a.dev_err, PA_DEVERR_BAD_BLOCK);
        }
    if (bad) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) out[i] = from_f32<T>(0.f);
        return;
    }
    // the new token's row, quantised as it is stored
    float kn[EPL], vn[EPL], qv[EPL], acc[EPL];
    const size_t src = ((size_t)b * Hkv + kvh) * D + lane * EPL;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        kn[i] = to_f32<T>(static_cast<const T *>(a.k_new)[src + i]);
        vn[i] = to_f32<T>(static_cast<const T *>(a.v_new)[src + i]);
        qv[i] = to_f32<T>(static_cast<const T *>(a.q)[((size_t)b * a.num_heads + h) * D + lane * EPL + i]);
        acc[i] = 0.f;
    }
    Q4Scale ks, vs;
    uint32_t kc = quantise_row<EPL>(kn, ks), vc = quantise_row<EPL>(vn, vs);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        kn[i] = q4_value((kc >> (4 * i)) & 15u, ks.step, ks.low);
        vn[i] = q4_value((vc >> (4 * i)) & 15u, vs.step, vs.low);
    }
    const size_t rb = q4_record_bytes(D, bs);
    uint8_t *pool = static_cast<uint8_t *>(a.kv_cache);
    if (h % G == 0) { // one warp per kv head appends
        uint8_t *rec = pool + ((size_t)tab[nblk - 1] * Hkv + kvh) * rb;
        const int t = L % bs;
        uint32_t kw = kc, vw = vc;
        if (EPL == 2) {
            kw |= __shfl_down_sync(kFull, kc, 1) << 8;
            vw |= __shfl_down_sync(kFull, vc, 1) << 8;
        }
        if (EPL == 4 || (lane & 1) == 0) {
            const int unit = EPL == 4 ? lane : lane >> 1;
            reinterpret_cast<uint16_t *>(rec)[t * (D / 4) + unit] = (uint16_t)kw;
            reinterpret_cast<uint16_t *>(rec + q4_v_offset(D, bs))[q4_v_unit<D>(t, unit)] = (uint16_t)vw;
        }
        if (lane == 0)
            *reinterpret_cast<uint2 *>(rec + q4_scale_offset(D, bs) + t * 8) =
                make_uint2(q4_pack_scale(ks), q4_pack_scale(vs));
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (a.k_stored) static_cast<T *>(a.k_stored)[src + i] = from_f32<T>(kn[i]);
            if (a.v_stored) static_cast<T *>(a.v_stored)[src + i] = from_f32<T>(vn[i]);
        }
    }
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j <= L; ++j) {
        float kr[EPL], vr[EPL];
        if (j == L) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                kr[i] = kn[i];
                vr[i] = vn[i];
            }
        } else {
            const uint8_t *rec = pool + ((size_t)tab[j / bs] * Hkv + kvh) * rb;
            const int t = j % bs, unit = lane * EPL / 4;
            uint32_t kw = reinterpret_cast<const uint16_t *>(rec)[t * (D / 4) + unit];
            uint32_t vw = reinterpret_cast<const uint16_t *>(rec + q4_v_offset(D, bs))[q4_v_unit<D>(t, unit)];
            if (EPL == 2) {
                kw >>= 8 * (lane & 1);
                vw >>= 8 * (lane & 1);
            }
            const uint2 sc = *reinterpret_cast<const uint2 *>(rec + q4_scale_offset(D, bs) + t * 8);
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                kr[i] = q4_value((kw >> (4 * i)) & 15u, bf16_lo(sc.x), bf16_hi(sc.x));
                vr[i] = q4_value((vw >> (4 * i)) & 15u, bf16_lo(sc.y), bf16_hi(sc.y));
            }
        }
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) dot = fmaf(qv[i], kr[i], dot);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
        const float s = dot * a.scale;
        const float mn = fmaxf(m, s);
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float alpha = expf(m - mu), p = expf(s - mu);
        l = l * alpha + p;
#pragma unroll
        for (int i = 0; i < EPL; ++i) acc[i] = acc[i] * alpha + p * vr[i];
        m = mn;
    }
    const float inv = 1.f / l;
#pragma unroll
    for (int i = 0; i < EPL; ++i) out[i] = from_f32<T>(acc[i] * inv);
}

}  // namespace

size_t decode_q4_workspace(int, int, int, int, int) { return 0; }

int decode_q4_launch(const DecodeQ4Args &a, bool f32, cudaStream_t s)
{
    const long long warps = (long long)a.batch * a.num_heads;
    const unsigned grid = (unsigned)((warps + 3) / 4);
    if (a.head_dim == 64) {
        if (f32) decode_q4_kernel<64, float><<<grid, 128, 0, s>>>(a);
        else decode_q4_kernel<64, __nv_bfloat16><<<grid, 128, 0, s>>>(a);
    } else {
        if (f32) decode_q4_kernel<128, float><<<grid, 128, 0, s>>>(a);
        else decode_q4_kernel<128, __nv_bfloat16><<<grid, 128, 0, s>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_LAUNCH;
}

}  // namespace pa
