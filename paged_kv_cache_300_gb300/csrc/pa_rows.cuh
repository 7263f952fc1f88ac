// What the block-sparse kernels share: where a query row stands in its request,
// and access to a cluster's shared memory.
#pragma once

#include "pa_common.cuh"

namespace pa {

// All of these read with ordinary loads what the kernel before may have written: a launch with
// programmatic dependence begins while that one runs, when read-only loads may keep old lines.

// Largest r in [0, n] with value(r) <= t, -1 if there is none; value does not decrease.  The whole
// warp searches, 32 values a step (one step up to 32 of them, two up to 1024).
template <typename Value>
__device__ __forceinline__ int find_last(const Value &value, int n, long long t, int lane)
{
    int lo = 0, count = n + 1;
    while (true) {
        const int step = (count + 31) / 32, at = lane * step;
        const uint32_t m = __ballot_sync(0xffffffffu, at < count && value(lo + at) <= t);
        if (m == 0) return lo == 0 ? -1 : lo; // lo > 0 was a hit of the step before
        const int hit = 31 - __clz(m);
        lo += hit * step;
        count = min(step, count - hit * step);
        if (step == 1) return lo;
    }
}

// The first CTA's threads look over the cumulative lengths.
template <typename Args>
__device__ __forceinline__ void check_lengths(const Args &a)
{
    if (a.cu_q == nullptr || blockIdx.x != 0) return;
    bool bad = threadIdx.x == 0 && a.cu_q[0] != 0;
    for (int i = threadIdx.x; i < a.batch; i += blockDim.x) bad |= a.cu_q[i + 1] < a.cu_q[i];
    if (bad) flag_error(a.dev_err, PA_DEVERR_BAD_CU);
}

// Row t of the packed queries: its request and the last position it sees.
struct QueryRow {
    int req;
    int pos;   // < 0: sees nothing (the rows behind it may, but for the same error or left-out request)
    bool skip; // behind the last request: its outputs are left as they are
    int err;   // PA_DEVERR_* bits
};

// The same for the row with `back` queries of its request `req` behind it.
template <typename Args>
__device__ __forceinline__ QueryRow request_row(const Args &a, int req, int back)
{
    QueryRow q{req, -(1 << 30), false, 0};
    const int kl = a.seqlens_k[req];
    if (kl == PA_LEFT_OUT) return q;
    if (kl < 0 || (long long)kl > (long long)a.max_blocks_per_seq * a.block_size) {
        q.err = PA_DEVERR_OVERFLOW;
        return q;
    }
    q.pos = kl - 1 - back;
    return q;
}

template <typename Args>
__device__ __forceinline__ QueryRow query_row(const Args &a, int t, int lane)
{
    if (a.cu_q == nullptr) return request_row(a, t, 0);
    QueryRow q{t, -(1 << 30), false, 0};
    q.req = find_last([&](int r) { return (long long)a.cu_q[r]; }, a.batch, t, lane);
    if (q.req == a.batch) {
        q.skip = true;
        return q;
    }
    const int c1 = q.req >= 0 ? a.cu_q[q.req + 1] : 0;
    if (q.req < 0 || c1 <= t || a.cu_q[0] != 0) {
        q.err = PA_DEVERR_BAD_CU;
        return q;
    }
    return request_row(a, q.req, c1 - 1 - t);
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Address of `p` (this CTA's shared memory) in the CTA of rank `rank`.
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_store(uint32_t addr, uint32_t x)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ void cluster_store4(uint32_t addr, const float4 &x)
{
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w) : "memory");
}
__device__ __forceinline__ void cluster_min(uint32_t addr, uint32_t x)
{
    asm volatile("red.relaxed.cluster.shared::cluster.min.u32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ void cluster_max(uint32_t addr, uint32_t x)
{
    asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}

}  // namespace pa
