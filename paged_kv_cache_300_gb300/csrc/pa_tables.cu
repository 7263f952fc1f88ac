// pa_block_tables: a serving step's block tables, slot map and cumulative
// lengths from the requests' lengths (include/pa.h states the rules).
//
// Everything follows from four prefix sums over the requests: new tokens,
// blocks taken, blocks given back, lengths after the step.
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 1024;

// What one request adds to the four sums.
struct Need {
    long long tok, take, back, after;
};

__device__ __forceinline__ Need need_of(const TablesArgs &a, int b, int &err)
{
    const int L = a.cache_seqlens[b], n = a.new_lens[b], bs = a.block_size;
    Need r{0, 0, 0, 0};
    if (L < 0 || n < -1 || (long long)L + (n > 0 ? n : 0) > (long long)a.max_blocks_per_seq * bs) {
        err |= PA_DEVERR_OVERFLOW;
        return r;
    }
    const long long held = ((long long)L + bs - 1) / bs;
    if (n < 0) {
        r.back = held;
    } else {
        r.tok = n;
        r.after = (long long)L + n;
        r.take = (r.after + bs - 1) / bs - held;
    }
    return r;
}

// Inclusive sum of x over the block; *total is the block's sum.
__device__ __forceinline__ long long block_scan(long long x, long long *s_warp, long long *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += t;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        long long w = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(kFull, w, o);
            if (lane >= o) w += t;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    *total = s_warp[kThreads / 32 - 1];
    return x + (warp > 0 ? s_warp[warp - 1] : 0);
}

__global__ void __launch_bounds__(kThreads) tables_kernel(const TablesArgs a)
{
    extern __shared__ int s_off[]; // [B + 1] new tokens before a request, [B] blocks taken before it
    __shared__ long long s_warp[kThreads / 32];
    __shared__ int s_err;
    const int tid = threadIdx.x, B = a.batch, bs = a.block_size;
    int *s_cu = s_off, *s_take = s_off + B + 1;
    if (tid == 0) s_err = 0;
    __syncthreads();
    const int F = *a.num_free;
    int err = F < 0 || F > a.num_blocks ? PA_DEVERR_BAD_BLOCK : 0;
    long long tok = 0, take = 0, back = 0, after = 0;
    // ---- sums, and the offsets that need nothing else
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + tid;
        const Need r = b < B ? need_of(a, b, err) : Need{0, 0, 0, 0};
        long long t0, t1, t2, t3;
        const long long x0 = tok + block_scan(r.tok, s_warp, &t0);
        const long long x1 = take + block_scan(r.take, s_warp, &t1);
        block_scan(r.back, s_warp, &t2);
        block_scan(r.after, s_warp, &t3);
        if (b < B) {
            s_cu[b + 1] = (int)x0;
            s_take[b] = (int)(x1 - r.take);
        }
        tok += t0;
        take += t1;
        back += t2;
        after += t3;
    }
    if (tid == 0) s_cu[0] = 0;
    if (after > 0x7fffffffll || tok > 0x7fffffffll) err |= PA_DEVERR_BAD_CU;
    if (tok > a.total_slots || take > F + back) err |= PA_DEVERR_NO_SPACE;
    if (F + back > a.num_blocks) err |= PA_DEVERR_BAD_BLOCK;
    if (err) atomicOr(&s_err, err);
    __syncthreads();
    const bool refused = s_err != 0;
    if (refused) {
        if (tid == 0) {
            flag_error(a.dev_err, s_err);
            a.cu_q[0] = a.cu_k[0] = 0;
            *a.num_free_out = F;
        }
        for (int b = tid; b < B; b += kThreads) {
            a.cu_q[b + 1] = a.cu_k[b + 1] = 0;
            a.seqlens_k[b] = a.cache_seqlens[b];
        }
        for (int i = tid; i < a.total_slots; i += kThreads) a.slot_map[i] = -1;
        return;
    }
    // ---- ended requests push their blocks
    const int warp = tid >> 5, lane = tid & 31;
    int flags = 0;
    if (back > 0) {
        long long base = F;
        for (int b0 = 0; b0 < B; b0 += kThreads) {
            const int b = b0 + tid;
            int e = 0;
            const Need r = b < B ? need_of(a, b, e) : Need{0, 0, 0, 0};
            long long t;
            const long long x = base + block_scan(r.back, s_warp, &t) - r.back;
            for (int j = 0; j < r.back; ++j) {
                int p = a.block_table[(size_t)b * a.max_blocks_per_seq + j];
                if (p < 0 || p >= a.num_blocks) {
                    p = -1;
                    flags |= PA_DEVERR_BAD_BLOCK;
                }
                a.free_blocks[x + j] = p;
            }
            base += t;
        }
    }
    __syncthreads();
    // ---- slots and new table entries, token by token
    const long long top = F + back;
    for (int i = tid; i < a.total_slots; i += kThreads) {
        int slot = -1;
        if (i < tok) {
            int lo = 0, hi = B; // the request with s_cu[lo] <= i < s_cu[lo + 1]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_cu[mid] <= i)
                    lo = mid;
                else
                    hi = mid;
            }
            const int b = lo, L = a.cache_seqlens[b];
            const int pos = L + (i - s_cu[b]), lb = pos / bs;
            const int held = (int)(((long long)L + bs - 1) / bs);
            int32_t *entry = a.block_table + (size_t)b * a.max_blocks_per_seq + lb;
            int p = lb < held ? *entry : a.free_blocks[top - 1 - (s_take[b] + lb - held)];
            if (p < 0 || p >= a.num_blocks) {
                p = -1;
                flags |= PA_DEVERR_BAD_BLOCK;
            }
            if (lb >= held && pos % bs == 0) *entry = p;
            if (p >= 0) slot = p * bs + pos % bs;
        }
        a.slot_map[i] = slot;
    }
    if (flags) flag_error(a.dev_err, flags);
    __syncthreads(); // lengths may be rewritten in place from here on
    long long sum = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + tid;
        int e = 0;
        const Need r = b < B ? need_of(a, b, e) : Need{0, 0, 0, 0};
        long long t;
        const long long x = sum + block_scan(r.after, s_warp, &t);
        if (b < B) {
            a.cu_q[b + 1] = s_cu[b + 1];
            a.cu_k[b + 1] = (int)x;
            a.seqlens_k[b] = (int)r.after;
        }
        sum += t;
    }
    (void)warp;
    (void)lane;
    if (tid == 0) {
        a.cu_q[0] = a.cu_k[0] = 0;
        *a.num_free_out = (int)(top - take);
    }
}

}  // namespace

int tables_launch(const TablesArgs &a, cudaStream_t s)
{
    const int smem = (2 * a.batch + 1) * 4;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return PA_ERR_LAUNCH;
    tables_kernel<<<1, kThreads, smem, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_LAUNCH;
}

}  // namespace pa
