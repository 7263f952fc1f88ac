// The 4-bit pool's cache update (quantise and scatter) and its read-back
// (gather and dequantise).  Formulas and layout: include/pa.h, "The 4-bit
// pool".
#include "pa_internal.h"
#include "pa_q4.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// One warp per (chunk row, kv head): lane l holds dims l*EPL .. l*EPL+EPL-1
// of K and of V.
template <int D, typename T>
__global__ void __launch_bounds__(256) update_q4_kernel(const CacheQ4Args a)
{
    constexpr int EPL = D / 32;
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int hkv = a.num_kv_heads, bs = a.block_size;
    if (w >= (long long)a.total * hkv) return;
    const long long row = w / hkv;
    const int h = (int)(w % hkv);
    const int slot = a.slot_map[row];
    if (slot < 0) return;
    if (slot >= (long long)a.num_blocks * bs) {
        if (lane == 0) flag_error(a.dev_err, PA_DEVERR_BAD_BLOCK);
        return;
    }
    uint8_t *rec = static_cast<uint8_t *>(a.kv_cache) +
                   ((size_t)(slot / bs) * hkv + h) * q4_record_bytes(D, bs);
    const int t = slot % bs;
    const T *src[2] = {static_cast<const T *>(a.k), static_cast<const T *>(a.v)};
    for (int kv = 0; kv < 2; ++kv) {
        float x[EPL];
        float lo = INFINITY, hi = -INFINITY;
        bool finite = true;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            x[i] = to_f32<T>(src[kv][(row * hkv + h) * D + lane * EPL + i]);
            lo = fminf(lo, x[i]);
            hi = fmaxf(hi, x[i]);
            finite = finite && fabsf(x[i]) < INFINITY;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
        }
        finite = __all_sync(kFull, finite);
        const Q4Scale s = q4_scale(lo, hi, finite);
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) c |= q4_code(x[i], s) << (4 * i);
        if (EPL == 2) c |= __shfl_down_sync(kFull, c, 1) << 8; // 4 dims in even lanes
        if (EPL == 4 || (lane & 1) == 0) {
            const int unit = EPL == 4 ? lane : lane >> 1;
            uint16_t *dst = kv == 0 ? reinterpret_cast<uint16_t *>(rec) + t * (D / 4) + unit
                                    : reinterpret_cast<uint16_t *>(rec + q4_v_offset(D, bs)) +
                                          q4_v_unit<D>(t, unit);
            *dst = (uint16_t)c;
        }
        if (lane == 0)
            *reinterpret_cast<uint32_t *>(rec + q4_scale_offset(D, bs) + t * 8 + kv * 4) =
                q4_pack_scale(s);
    }
}

// Largest r in [0, n) with cu[r] <= x.
__device__ __forceinline__ int owner(const int32_t *cu, int n, long long x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid) <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The cumulative lengths start at 0, never decrease and end inside k_full
// (one block looks at all of them).
__device__ __forceinline__ void check_cu(const CacheQ4Args &a)
{
    bool bad = threadIdx.x == 0 && (__ldg(a.cu_k) != 0 || __ldg(a.cu_k + a.batch) > a.total);
    for (int b = threadIdx.x; b < a.batch; b += blockDim.x)
        bad = bad || __ldg(a.cu_k + b + 1) < __ldg(a.cu_k + b);
    if (bad) flag_error(a.dev_err, PA_DEVERR_BAD_CU);
}

// One warp per (packed row, kv head).
template <int D, typename T>
__global__ void __launch_bounds__(256) gather_q4_kernel(const CacheQ4Args a)
{
    constexpr int EPL = D / 32;
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int hkv = a.num_kv_heads, bs = a.block_size;
    if (blockIdx.x == 0) check_cu(a);
    if (w >= (long long)a.total * hkv) return;
    const int row = (int)(w / hkv), h = (int)(w % hkv);
    const int b = owner(a.cu_k, a.batch, row);
    const int k0 = __ldg(a.cu_k + b), k1 = __ldg(a.cu_k + b + 1);
    if (k0 < 0 || row < k0 || row >= k1) return; // behind the last row, or flagged by check_cu
    const int pos = row - k0, lb = pos / bs, t = pos % bs;
    int blk = -1;
    if (lb >= a.max_blocks_per_seq) {
        if (lane == 0) flag_error(a.dev_err, PA_DEVERR_OVERFLOW);
    } else {
        blk = __ldg(a.block_table + (size_t)b * a.max_blocks_per_seq + lb);
        if (blk < 0 || blk >= a.num_blocks) {
            if (lane == 0) flag_error(a.dev_err, PA_DEVERR_BAD_BLOCK);
            blk = -1;
        }
    }
    const uint8_t *rec = static_cast<const uint8_t *>(a.kv_cache) +
                         ((size_t)(blk < 0 ? 0 : blk) * hkv + h) * q4_record_bytes(D, bs);
    T *dst[2] = {static_cast<T *>(a.k_full), static_cast<T *>(a.v_full)};
    for (int kv = 0; kv < 2; ++kv) {
        T *o = dst[kv] + ((size_t)row * hkv + h) * D + lane * EPL;
        uint32_t c = 0;
        float step = 0.f, low = 0.f;
        if (blk >= 0) {
            const int unit = lane * EPL / 4;
            const uint16_t *p = kv == 0 ? reinterpret_cast<const uint16_t *>(rec) + t * (D / 4) + unit
                                        : reinterpret_cast<const uint16_t *>(rec + q4_v_offset(D, bs)) +
                                              q4_v_unit<D>(t, unit);
            c = *p;
            if (EPL == 2) c >>= 8 * (lane & 1);
            const uint32_t s = *reinterpret_cast<const uint32_t *>(rec + q4_scale_offset(D, bs) +
                                                                   t * 8 + kv * 4);
            step = bf16_lo(s);
            low = bf16_hi(s);
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) o[i] = from_f32<T>(q4_value((c >> (4 * i)) & 15u, step, low));
    }
}

template <int D, typename T>
int launch(const CacheQ4Args &a, bool gather, cudaStream_t s)
{
    const long long warps = (long long)a.total * a.num_kv_heads;
    const unsigned grid = (unsigned)((warps + 7) / 8);
    if (gather)
        gather_q4_kernel<D, T><<<grid, 256, 0, s>>>(a);
    else
        update_q4_kernel<D, T><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_LAUNCH;
}

}  // namespace

int cache_q4_launch(const CacheQ4Args &a, bool f32, bool gather, cudaStream_t s)
{
    if (a.head_dim == 64) return f32 ? launch<64, float>(a, gather, s) : launch<64, __nv_bfloat16>(a, gather, s);
    return f32 ? launch<128, float>(a, gather, s) : launch<128, __nv_bfloat16>(a, gather, s);
}

}  // namespace pa
