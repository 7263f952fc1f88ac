// pa_block_tables: a serving step's block tables, slot map and cumulative
// lengths from the requests' lengths (include/pa.h states the rules).
//
// Everything follows from four prefix sums over the requests: new tokens,
// blocks taken, blocks given back, lengths after the step.  The bytes are few
// (4 a slot, 20 a request); what a call costs is latency.  So one launch does
// it all: a cluster of CTAs in which each makes all the sums for itself (no
// traffic between CTAs), then takes its share of the requests and of the
// slots.  One cluster barrier orders the rest: given-back blocks are on the
// stack before a block is taken from it, and lengths and the stack's size,
// which may be written in place, have been read by everybody before they are.  A small step
// is one CTA (kClusterSlots).  Up to 4096 requests of a token each: 8.9 us, the
// host's time for a call; 4096 requests, 585 of them ending, with 512K new
// tokens: 20.2 us, of which the 2.4 MB would take 0.4: the rest is the chain of
// dependent steps (lengths, sums, barrier, search, stack, store).
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 1024;
// From this many slots on the step is a cluster's work, 8 CTAs (the portable
// size) or 16.  One CTA, 8 and 16 of them: 8192 slots of 1024 requests 14.6, 9.3
// and 9.1 us; 32K slots of 4096 requests 52.9, 13.0 and 9.9; 16K slots of as many
// requests -, 40.2 and 37.7.  Below 4096 slots all three take what the host needs.
constexpr int kClusterSlots = 4096, kLargeSlots = 16384;
constexpr int kRun = 8; // neighbouring slots of a thread

// What requests add to the four sums.
struct Need {
    long long tok, take, back, after;
    __device__ __forceinline__ void add(const Need &o)
    {
        tok += o.tok;
        take += o.take;
        back += o.back;
        after += o.after;
    }
};

// x / block_size for x >= 0: a shift for the usual sizes.
__device__ __forceinline__ int div_bs(const TablesArgs &a, int x)
{
    return a.shift >= 0 ? x >> a.shift : x / a.block_size;
}
__device__ __forceinline__ int ceil_bs(const TablesArgs &a, int x)
{
    const int q = div_bs(a, x);
    return q + (q * a.block_size != x);
}

__device__ __forceinline__ Need need_of(const TablesArgs &a, int L, int n, int &err)
{
    const int bs = a.block_size;
    Need r{0, 0, 0, 0};
    if (L < 0 || n < -1 || (long long)L + max(n, 0) > (long long)a.max_blocks_per_seq * bs) {
        err |= PA_DEVERR_OVERFLOW;
        return r;
    }
    const int held = ceil_bs(a, L);
    if (n < 0) {
        r.back = held;
    } else {
        r.tok = n;
        r.after = L + n; // at most max_blocks_per_seq * block_size < 2^31
        r.take = ceil_bs(a, L + n) - held;
    }
    return r;
}

__device__ __forceinline__ void cluster_sync(bool cluster)
{
    if (cluster) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kThreads) tables_kernel(const TablesArgs a)
{
    extern __shared__ int s_dyn[];
    __shared__ Need s_warp[kThreads / 32];
    __shared__ int s_err;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.batch, bs = a.block_size;
    const int ncta = gridDim.x, cta = blockIdx.x;
    const bool cluster = ncta > 1;
    int *s_cu = s_dyn;             // [B + 1] new tokens before a request
    int *s_take = s_dyn + B + 1;   // [B] blocks taken before it
    int *s_len = s_dyn + 2 * B + 1; // [B] its length
    if (tid == 0) {
        s_err = 0;
        s_cu[0] = 0;
    }
    grid_dep_trigger();
    grid_dep_wait();
    const int F = *a.num_free;
    for (int b = tid; b < B; b += kThreads) {
        s_len[b] = a.cache_seqlens[b];
        s_cu[b + 1] = a.new_lens[b]; // until the sum takes its place
    }
    __syncthreads();
    int err = F < 0 || F > a.num_blocks ? PA_DEVERR_BAD_BLOCK : 0;

    // ---- the sums: a thread's run of requests, then over the threads
    const int per = (B + kThreads - 1) / kThreads;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    Need mine{0, 0, 0, 0};
    for (int b = b0; b < b1; ++b) mine.add(need_of(a, s_len[b], s_cu[b + 1], err));
    Need incl = mine;
    auto warp_scan = [&](Need &x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Need t{__shfl_up_sync(kFull, x.tok, o), __shfl_up_sync(kFull, x.take, o),
                         __shfl_up_sync(kFull, x.back, o), __shfl_up_sync(kFull, x.after, o)};
            if (lane >= o) x.add(t);
        }
    };
    warp_scan(incl);
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        Need w = s_warp[lane];
        warp_scan(w);
        s_warp[lane] = w;
    }
    if (err) atomicOr(&s_err, err);
    __syncthreads();
    const Need all = s_warp[kThreads / 32 - 1];
    if (warp > 0) incl.add(s_warp[warp - 1]);
    err = s_err;
    if (all.after > 0x7fffffffll || all.tok > 0x7fffffffll) err |= PA_DEVERR_BAD_CU;
    if (all.tok > a.total_slots || all.take > F + all.back) err |= PA_DEVERR_NO_SPACE;
    if (F + all.back > a.num_blocks) err |= PA_DEVERR_BAD_BLOCK;
    if (err) { // the same in every CTA: nothing changes
        cluster_sync(cluster);
        if (cta == 0) {
            if (tid == 0) {
                flag_error(a.dev_err, err);
                a.cu_q[0] = a.cu_k[0] = 0;
                *a.num_free_out = F;
            }
            for (int b = tid; b < B; b += kThreads) {
                a.cu_q[b + 1] = a.cu_k[b + 1] = 0;
                a.seqlens_k[b] = s_len[b];
                if (a.decode_lens) a.decode_lens[b] = PA_LEFT_OUT;
            }
        }
        // (the last step of a slot map of nearly 2^31 entries passes 32 bits)
        for (long long i = cta * kThreads + tid; i < a.total_slots; i += ncta * kThreads) a.slot_map[i] = -1;
        return;
    }

    // ---- offsets; ended requests push their blocks
    int flags = 0;
    {
        Need at = incl; // sums before the thread's run
        at.tok -= mine.tok;
        at.take -= mine.take;
        at.back -= mine.back;
        at.after -= mine.after;
        for (int k = 0; k < per; ++k) { // the same count in every lane
            const int b = b0 + k;
            const bool in = b < b1;
            const Need r = in ? need_of(a, s_len[b], s_cu[b + 1], err) : Need{0, 0, 0, 0};
            // the warp's ended requests, one after the other, 32 blocks at a time
            unsigned ended = __ballot_sync(kFull, r.back > 0 && b % ncta == cta);
            while (ended) {
                const int who = __ffs(ended) - 1;
                ended &= ended - 1;
                const int n = __shfl_sync(kFull, (int)r.back, who), q = __shfl_sync(kFull, b, who);
                const int to = F + __shfl_sync(kFull, (int)at.back, who);
                const int32_t *row = a.block_table + (size_t)q * a.max_blocks_per_seq;
                // Read-only loads here: no one writes an ended request's row in this step, and
                // the lengths that lead to it have passed two barriers since the wait.  With
                // ordinary loads, which the stores hold up, the large step takes 21.0 us
                // instead of 20.2.
#pragma unroll 4
                for (int j = lane; j < n; j += 32) {
                    int p = __ldg(row + j);
                    if (p < 0 || p >= a.num_blocks) {
                        p = -1;
                        flags |= PA_DEVERR_BAD_BLOCK;
                    }
                    a.free_blocks[to + j] = p;
                }
            }
            if (in) {
                s_take[b] = (int)at.take;
                at.add(r);
                s_cu[b + 1] = (int)at.tok;
                if (b % ncta == cta) {
                    a.cu_q[b + 1] = (int)at.tok;
                    a.cu_k[b + 1] = (int)at.after;
                }
            }
        }
    }
    cluster_sync(cluster);

    // ---- slots and new table entries
    const int top = (int)(F + all.back), tok = (int)all.tok;
    // Neighbouring slots have one request and few blocks where requests bring
    // several tokens: a thread takes a run of them.  8 tokens a request, 32K
    // slots: runs 9.7 us, single slots 13.0; 1 token a request, 4096 slots: 11.7
    // and 8.9.
    const bool tall = (long long)tok >= 4ll * B;
    const int run = tall ? kRun : 1;
    for (long long i0 = ((long long)cta * kThreads + tid) * run; i0 < a.total_slots;
         i0 += (long long)ncta * kThreads * run) {
        int slot[kRun];
#pragma unroll
        for (int k = 0; k < kRun; ++k) slot[k] = -1;
        if (i0 < tok) {
            const int i = (int)i0, n = min(run, tok - i);
            int b = 0, hi = B; // the request with s_cu[b] <= i < s_cu[b + 1]
            while (hi - b > 1) {
                const int mid = (b + hi) >> 1;
                if (s_cu[mid] <= i)
                    b = mid;
                else
                    hi = mid;
            }
            // one piece after the other that lies in one block of one request
            for (int k = 0; k < n;) {
                const int L = s_len[b], pos = L + (i + k - s_cu[b]);
                const int lb = div_bs(a, pos), off = pos - lb * bs, held = ceil_bs(a, L);
                int32_t *entry = a.block_table + (size_t)b * a.max_blocks_per_seq + lb;
                int p = __ldcg(lb < held ? entry : a.free_blocks + (top - 1 - (s_take[b] + lb - held)));
                if (p < 0 || p >= a.num_blocks) {
                    p = -1;
                    flags |= PA_DEVERR_BAD_BLOCK;
                }
                if (off == 0 && lb >= held) *entry = p;
                const int m = min(min(n - k, bs - off), s_cu[b + 1] - (i + k));
                const int base = p * bs + off - k;
#pragma unroll
                for (int q = 0; q < kRun; ++q)
                    if (q >= k && q < k + m && p >= 0) slot[q] = base + q;
                k += m;
                if (k < n)
                    while (s_cu[b + 1] <= i + k) ++b; // past requests without new tokens
            }
        }
        int32_t *dst = a.slot_map + i0;
        if (!tall) {
            *dst = slot[0];
        } else if (i0 + kRun <= a.total_slots && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
            reinterpret_cast<int4 *>(dst)[0] = make_int4(slot[0], slot[1], slot[2], slot[3]);
            reinterpret_cast<int4 *>(dst)[1] = make_int4(slot[4], slot[5], slot[6], slot[7]);
        } else {
#pragma unroll
            for (int k = 0; k < kRun; ++k)
                if (i0 + k < a.total_slots) dst[k] = slot[k];
        }
    }
    if (flags) flag_error(a.dev_err, flags);
    // ---- what may be written in place: everybody has read it before the
    // last barrier (lengths and new_lens above it, the stack's size first)
    for (int b = cta * kThreads + tid; b < B; b += ncta * kThreads) {
        const int n = s_cu[b + 1] - s_cu[b];
        // an ended request's length is 0: its slice of cu_k is empty
        a.seqlens_k[b] = a.new_lens[b] < 0 ? 0 : s_len[b] + n;
        if (a.decode_lens) a.decode_lens[b] = n == 1 ? s_len[b] : PA_LEFT_OUT;
    }
    if (cta == 0 && tid == 0) {
        a.cu_q[0] = a.cu_k[0] = 0;
        *a.num_free_out = (int)(top - all.take);
    }
}

}  // namespace

int tables_launch(const TablesArgs &args, cudaStream_t s)
{
    const size_t smem = (size_t)(3 * args.batch + 1) * 4;
    TablesArgs a = args;
    a.shift = -1;
    for (int k = 0; k < 31; ++k)
        if (a.block_size == 1 << k) a.shift = k;
    static int raised[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PA_ERR_DEVICE;
    if (!__atomic_load_n(&raised[dev], __ATOMIC_ACQUIRE)) {
        cudaError_t e = cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (3 * kTablesMaxBatch + 1) * 4);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return launch_status(e);
        __atomic_store_n(&raised[dev], 1, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg = {};
    const int ctas = a.total_slots >= kLargeSlots ? 16 : a.total_slots >= kClusterSlots ? 8 : 1;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return launch_status(cudaLaunchKernelEx(&cfg, tables_kernel, a));
}

}  // namespace pa
