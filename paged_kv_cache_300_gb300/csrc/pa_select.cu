// pa_select_blocks: the blocks a query attends to, chosen by the bounds of their keys.
//
// For a query row (token, kv head) with G query heads and a block whose keys'
// channels lie in [lo_d, hi_d], no key of the block scores more than
//   s = max_g sum_d (max(q_gd, 0) hi_d + min(q_gd, 0) lo_d).
// The row keeps the `top_k` visible blocks of largest s, the first and the last
// ones always among them, in ascending order.
//
// Scores.  Bound by the bytes of the bounds (2 D elements a block and head, 1 / bs
// of the keys and values).  In bf16 the operands are exact and the sum is a
// product of [q+, q-] with [hi, lo]: mma.sync m16n8k16 with 16 blocks on M and the
// heads on N.  The order of the sum over d is free, so a lane's 16-byte load of a
// row is two k-steps' fragments as it stands: bounds go from memory to the tensor
// cores without shared memory, 8 KB a warp in flight.  A row is one CTA's; with
// few rows a cluster's, whose CTAs score a share each and store the scores in
// the first one's shared memory.
//
// Choice.  The answer is that of the exact scores, ties to the lowest block,
// whatever the order of the sums in fp32.  The k-th largest of the fp32 scores, t,
// is found by histograms; with every score off by at most E, blocks above t + 2 E
// are in and blocks below t - 2 E out for certain.  Where those between are more
// than the places left, their scores are made again in 64 bits, as differences
// from t, and chosen among by the same histograms.
//   E: an m16n8k16 step is taken to be off by at most 2^-22 of the magnitudes it adds
//   (|accumulator| + |products|); D / 16 steps a chain: E < 2^-22 (D / 16 + 2) S with S = sum |q||b|
//   <= L1(q) max|b|.  2^-17 L1(q) max|b| is 3 times that.  (fp32: D / 16 + 5 roundings
//   of 2^-24 a lane's share.)
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_rows.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBins = 2048, kBinBits = 11;
constexpr int kGroup = 8; // most query heads of a kv head

// Order-preserving map of floats to integers; a NaN is above everything, 0 is no float's.
__device__ __forceinline__ uint32_t key_of(float x)
{
    if (x != x) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x + 0.f); // -0 is 0
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k)
{
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min_nan2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) // the other one of a NaN
{
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float low_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

// What the CTAs of a row tell its first one.
struct Shared {
    uint32_t least, most; // of the keys
    uint32_t mag;         // largest |bound| of blocks whose score is finite (bits of a float >= 0)
    uint32_t bad;         // a needed table entry is no block
    uint32_t bin, above, listed, result;
    uint32_t list[32];
    uint32_t warp[kWarps];
    uint32_t count[kWarps][2];
    uint32_t hist[kBins];
};

// The need-th largest of the keys in [lo, hi] (need >= 1, at most as many as there are).
__device__ __forceinline__ uint32_t kth_largest(const uint32_t *key, int n, uint32_t need, uint32_t lo, uint32_t hi,
                                                Shared &sh)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int PER = kBins / kThreads;
    while (lo < hi) { // at most three times: 11 bits each
        const int bits = 32 - __clz(hi - lo), shift = max(bits - kBinBits, 0);
        for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
        if (tid == 0) sh.listed = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
            const uint32_t k = key[i];
            if (k >= lo && k <= hi) atomicAdd(&sh.hist[(k - lo) >> shift], 1u);
        }
        __syncthreads();
        // sums from the top bin down: thread t has bins PER * t ..
        uint32_t bin[PER], sum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += bin[i] = sh.hist[tid * PER + i];
        uint32_t incl = sum; // of this thread and the lanes above
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_down_sync(kFull, incl, o);
            if (lane + o < 32) incl += x;
        }
        if (lane == 0) sh.warp[warp] = incl;
        __syncthreads();
        uint32_t above = incl - sum;
        for (int w = warp + 1; w < kWarps; ++w) above += sh.warp[w];
        if (above < need && need <= above + sum) { // one thread
            for (int i = PER - 1; i >= 0; --i) {
                if (need <= above + bin[i]) {
                    sh.bin = tid * PER + i;
                    sh.above = above;
                    sh.result = bin[i];
                    break;
                }
                above += bin[i];
            }
        }
        __syncthreads();
        const uint32_t in = sh.result;
        need -= sh.above;
        lo += sh.bin << shift;
        if (shift == 0) return lo; // a bin is one key
        hi = min(hi, lo + ((1u << shift) - 1));
        if (in <= 32) { // few enough to look at one by one
            for (int i = tid; i < n; i += kThreads) {
                const uint32_t k = key[i];
                if (k >= lo && k <= hi) sh.list[atomicAdd(&sh.listed, 1u)] = k;
            }
            __syncthreads();
            if (warp == 0) {
                const uint32_t k = lane < in ? sh.list[lane] : 0;
                uint32_t more = 0, same = 0;
                for (uint32_t i = 0; i < in; ++i) {
                    const uint32_t x = __shfl_sync(kFull, k, i);
                    more += x > k;
                    same += x == k;
                }
                if (lane < in && more < need && need <= more + same) sh.result = k;
            }
            __syncthreads();
            return sh.result;
        }
        __syncthreads();
    }
    return lo;
}

// The row's score of one block in 64 bits; the warp's lanes share the channels.
template <typename T, int D>
__device__ __forceinline__ double exact_score(const T *q, const T *bounds, int G, int lane)
{
    double best = 0;
    for (int g = 0; g < G; ++g) {
        double s = 0;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const int d = i * 32 + lane;
            const float x = to_float(q[(size_t)g * D + d]);
            // one of the two factors is 0
            s += (double)x * (double)to_float(bounds[x > 0.f ? D + d : d]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
        best = g == 0 || s > best ? s : best;
    }
    return best;
}

// What one warp has of the row's keys.
struct Range {
    uint32_t least = 0xffffffffu, most = 0;
    float mag = 0.f;
    __device__ __forceinline__ void take(uint32_t k, float score, float m)
    {
        least = min(least, k);
        most = max(most, k);
        if (fabsf(score) < INFINITY) mag = fmaxf(mag, m);
    }
};

template <int D>
__device__ __forceinline__ void score_blocks(const SelectArgs &a, const __nv_bfloat16 *q, const int32_t *table, int h,
                                             int j0, int n, int first, int stride, int lane, uint32_t keys, Range &range,
                                             float &l1, bool &bad)
{
    constexpr int NC = D / 32; // 16-byte pieces of a row per lane
    const int g = lane >> 2, c = (lane & 3) * 8, G = a.group;
    uint4 qp[NC], qn[NC];
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (g < G) x = *reinterpret_cast<const uint4 *>(q + (size_t)g * D + i * 32 + c);
        qp[i] = make_uint4(max_nan2(x.x, 0), max_nan2(x.y, 0), max_nan2(x.z, 0), max_nan2(x.w, 0));
        qn[i] = make_uint4(min_nan2(x.x, 0), min_nan2(x.y, 0), min_nan2(x.z, 0), min_nan2(x.w, 0));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) mine += fabsf(low_bf16(w[j])) + fabsf(high_bf16(w[j]));
    }
    mine += __shfl_xor_sync(kFull, mine, 1);
    mine += __shfl_xor_sync(kFull, mine, 2);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) mine = fmaxf(mine, __shfl_xor_sync(kFull, mine, o));
    l1 = mine;

    const __nv_bfloat16 *bounds = static_cast<const __nv_bfloat16 *>(a.bounds) + (size_t)h * 2 * D + c;
    const size_t block = (size_t)a.num_kv_heads * 2 * D;
    const int tiles = (n + 15) / 16;
    const int col = 2 * (lane & 3);
    auto entry_of = [&](int tile) {
        const int j = tile * 16 + (lane & 15);
        return tile < tiles && j < n ? __ldg(table + j0 + j) : 0;
    };
    int entry = entry_of(first);
    for (int tile = first; tile < tiles; tile += stride) {
        const bool wrong = entry < 0 || entry >= a.num_blocks;
        bad |= wrong;
        const int at = wrong ? 0 : entry; // (a row behind the last reads block 0 and is left out)
        entry = entry_of(tile + stride);
        const __nv_bfloat16 *r0 = bounds + (size_t)__shfl_sync(kFull, at, g) * block;
        const __nv_bfloat16 *r1 = bounds + (size_t)__shfl_sync(kFull, at, g + 8) * block;
        uint4 lo[NC][2], hi[NC][2];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            lo[i][0] = __ldg(reinterpret_cast<const uint4 *>(r0 + i * 32));
            lo[i][1] = __ldg(reinterpret_cast<const uint4 *>(r1 + i * 32));
            hi[i][0] = __ldg(reinterpret_cast<const uint4 *>(r0 + D + i * 32));
            hi[i][1] = __ldg(reinterpret_cast<const uint4 *>(r1 + D + i * 32));
        }
        float sh[4] = {0.f, 0.f, 0.f, 0.f}, sl[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t m0 = 0, m1 = 0;
        const uint32_t abs2 = 0x7fff7fffu;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            mma_bf16_16816(sh, hi[i][0].x, hi[i][1].x, hi[i][0].y, hi[i][1].y, qp[i].x, qp[i].y);
            mma_bf16_16816(sl, lo[i][0].x, lo[i][1].x, lo[i][0].y, lo[i][1].y, qn[i].x, qn[i].y);
            mma_bf16_16816(sh, hi[i][0].z, hi[i][1].z, hi[i][0].w, hi[i][1].w, qp[i].z, qp[i].w);
            mma_bf16_16816(sl, lo[i][0].z, lo[i][1].z, lo[i][0].w, lo[i][1].w, qn[i].z, qn[i].w);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t &m = k ? m1 : m0;
                m = max2(m, max2(max2(hi[i][k].x & abs2, hi[i][k].y & abs2), max2(hi[i][k].z & abs2, hi[i][k].w & abs2)));
                m = max2(m, max2(max2(lo[i][k].x & abs2, lo[i][k].y & abs2), max2(lo[i][k].z & abs2, lo[i][k].w & abs2)));
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) { // rows g and g + 8
            float s = col < G ? sh[2 * k] + sl[2 * k] : -INFINITY;
            if (col + 1 < G) s = max_nan(s, sh[2 * k + 1] + sl[2 * k + 1]);
            const uint32_t mw = k ? m1 : m0;
            float m = fmaxf(low_bf16(mw), high_bf16(mw));
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                s = max_nan(s, __shfl_xor_sync(kFull, s, o));
                m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
            }
            const int j = tile * 16 + g + 8 * k;
            if (j < n) {
                const uint32_t key = key_of(s);
                range.take(key, s, m);
                if ((lane & 3) == 0) cluster_store(keys + 4 * j, key);
            }
        }
    }
}

// fp32: a warp scores kBatch blocks at a time, its lanes share the channels.
template <int D>
__device__ __forceinline__ void score_blocks(const SelectArgs &a, const float *q, const int32_t *table, int h, int j0,
                                             int n, int first, int stride, int lane, uint32_t keys, Range &range, float &l1,
                                             bool &bad)
{
    constexpr int E = D / 32, kBatch = 4;
    const int G = a.group;
    float x[kGroup][E];
    l1 = 0.f;
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
        float mine = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            x[g][i] = g < G ? q[(size_t)g * D + lane * E + i] : 0.f;
            mine += fabsf(x[g][i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(kFull, mine, o);
        l1 = fmaxf(l1, mine);
    }
    using Vec = typename std::conditional<E == 4, float4, float2>::type;
    const float *bounds = static_cast<const float *>(a.bounds) + (size_t)h * 2 * D + lane * E;
    const size_t block = (size_t)a.num_kv_heads * 2 * D;
    const int tiles = (n + kBatch - 1) / kBatch;
    for (int tile = first; tile < tiles; tile += stride) {
        float lo[kBatch][E], hi[kBatch][E];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int j = tile * kBatch + b;
            int e = j < n ? __ldg(table + j0 + j) : 0;
            if (e < 0 || e >= a.num_blocks) {
                bad = true;
                e = 0;
            }
            *reinterpret_cast<Vec *>(lo[b]) = __ldg(reinterpret_cast<const Vec *>(bounds + (size_t)e * block));
            *reinterpret_cast<Vec *>(hi[b]) = __ldg(reinterpret_cast<const Vec *>(bounds + (size_t)e * block + D));
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int j = tile * kBatch + b;
            float s[kGroup], m = 0.f;
#pragma unroll
            for (int g = 0; g < kGroup; ++g) s[g] = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                m = fmaxf(m, fmaxf(fabsf(lo[b][i]), fabsf(hi[b][i])));
#pragma unroll
                for (int g = 0; g < kGroup; ++g)
                    if (g < G) s[g] = fmaf(max_nan(x[g][i], 0.f), hi[b][i], fmaf(min_nan(x[g][i], 0.f), lo[b][i], s[g]));
            }
            float best = -INFINITY;
#pragma unroll
            for (int g = 0; g < kGroup; ++g) {
                if (g >= G) break;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s[g] += __shfl_xor_sync(kFull, s[g], o);
                best = max_nan(best, s[g]);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
            if (j < n) {
                const uint32_t key = key_of(best);
                range.take(key, best, m);
                if (lane == 0) cluster_store(keys + 4 * j, key);
            }
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2) select_kernel(const SelectArgs a, int ctas)
{
    extern __shared__ uint32_t key[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = ctas > 1 ? (int)cluster_rank() : 0;
    if (tid == 0) {
        sh.least = 0xffffffffu;
        sh.most = sh.mag = sh.bad = 0;
    }
    __syncwarp();
    grid_dep_trigger();
    if (ctas > 1)
        cluster_arrive();
    else
        __syncthreads();
    grid_dep_wait();

    const int row = blockIdx.x / ctas, t = row / a.num_kv_heads, h = row % a.num_kv_heads;
    const QueryRow at = query_row(a, t, lane);
    int32_t *out = a.selected + (size_t)row * a.top_k;
    const int seen = at.pos < 0 ? 0 : at.pos / a.block_size + 1;
    const int need = a.top_k - a.first - a.last;
    // nothing to choose (the same for all CTAs of the row)
    if (at.skip || seen <= a.top_k || need == 0) {
        if (rank == 0 && !at.skip) {
            if (at.err && tid == 0) flag_error(a.dev_err, at.err);
            for (int i = tid; i < a.top_k; i += kThreads)
                out[i] = seen > a.top_k ? (i < a.first ? i : seen - a.top_k + i) : i < seen ? i : -1;
        }
        if (ctas > 1) cluster_wait();
        return;
    }
    const int32_t *table = a.block_table + (size_t)at.req * a.max_blocks_per_seq;
    const T *q = static_cast<const T *>(a.q) + ((size_t)t * a.num_heads + (size_t)h * a.group) * D;
    const int j0 = a.first, n = seen - a.first - a.last;

    if (ctas > 1) cluster_wait(); // the first CTA's shared memory is there
    Range range;
    float l1 = 0.f;
    bool bad = false;
    score_blocks<D>(a, q, table, h, j0, n, rank * kWarps + warp, ctas * kWarps, lane, cluster_addr(key, 0), range, l1, bad);
    range.least = __reduce_min_sync(kFull, range.least);
    range.most = __reduce_max_sync(kFull, range.most);
    const uint32_t mag = __reduce_max_sync(kFull, __float_as_uint(range.mag));
    bad = __any_sync(kFull, bad);
    if (lane == 0 && range.most != 0) { // the warp has scored a block
        cluster_min(cluster_addr(&sh.least, 0), range.least);
        cluster_max(cluster_addr(&sh.most, 0), range.most);
        cluster_max(cluster_addr(&sh.mag, 0), mag);
        if (bad) cluster_max(cluster_addr(&sh.bad, 0), 1u);
    }
    __syncwarp();
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }
    if (sh.bad) {
        if (tid == 0) flag_error(a.dev_err, PA_DEVERR_BAD_BLOCK);
        for (int i = tid; i < a.top_k; i += kThreads) out[i] = -1;
        return;
    }

    // ---- the choice: keys above `high` are in, `quota` of those from `low` to `high`
    uint32_t low = kth_largest(key, n, need, sh.least, sh.most, sh), high = low;
    const float cut = value_of(low), width = l1 * __uint_as_float(sh.mag) * 0x1p-16f;
    const bool blurred = fabsf(cut) < INFINITY && width > 0.f && width < INFINITY;
    if (blurred) {
        low = key_of(cut - width);
        high = key_of(cut + width);
    }
    // each warp has a run of 32 keys' multiples, so that places follow from counts
    const int per = ((n + kThreads - 1) / kThreads) * 32, i0 = warp * per, i1 = min(n, i0 + per);
    int sure = 0, open = 0, sure_before = 0, open_before = 0;
    for (int pass = 0;; ++pass) {
        int mine_sure = 0, mine_open = 0;
        for (int i = i0 + lane; i - lane < i1; i += 32) {
            const uint32_t k = i < i1 ? key[i] : 0;
            mine_sure += __popc(__ballot_sync(kFull, i < i1 && k > high));
            mine_open += __popc(__ballot_sync(kFull, i < i1 && k >= low && k <= high));
        }
        if (lane == 0) {
            sh.count[warp][0] = mine_sure;
            sh.count[warp][1] = mine_open;
        }
        __syncthreads();
        sure = open = sure_before = open_before = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) {
                sure_before = sure;
                open_before = open;
            }
            sure += sh.count[w][0];
            open += sh.count[w][1];
        }
        if (pass > 0 || !blurred || sure + open == need) break;
        // more blocks than places within the error of the scores: again in 64 bits,
        // as the difference from the cut (a float holds it to 2^-40 of the scores)
        for (int i = i0 + lane; i - lane < i1; i += 32) {
            const uint32_t k = i < i1 ? key[i] : 0;
            uint32_t todo = __ballot_sync(kFull, i < i1 && k >= low && k <= high);
            uint32_t now = k > high ? 0xffffffffu : 0u;
            while (todo) {
                const int b = __ffs(todo) - 1;
                todo &= todo - 1;
                const int e = __ldg(table + j0 + (i - lane) + b);
                const T *bounds = static_cast<const T *>(a.bounds) + ((size_t)e * a.num_kv_heads + h) * 2 * D;
                const uint32_t k64 = key_of((float)(exact_score<T, D>(q, bounds, a.group, lane) - (double)cut));
                if (lane == b) now = k64;
            }
            if (i < i1) key[i] = now;
        }
        __syncthreads();
        low = high = kth_largest(key, n, need - sure, 1u, 0xfffffffeu, sh);
        __syncthreads();
    }
    const int quota = need - sure;
    int place = a.first + sure_before + min(open_before, quota), ties = open_before;
    for (int i = i0 + lane; i - lane < i1; i += 32) {
        const uint32_t k = i < i1 ? key[i] : 0;
        const uint32_t eq = __ballot_sync(kFull, i < i1 && k >= low && k <= high);
        const uint32_t below = (1u << lane) - 1;
        const bool in = i < i1 && (k > high || (((eq >> lane) & 1) && ties + __popc(eq & below) < quota));
        const uint32_t chosen = __ballot_sync(kFull, in);
        if (in) out[place + __popc(chosen & below)] = j0 + i;
        place += __popc(chosen);
        ties += __popc(eq);
    }
    for (int i = tid; i < a.first; i += kThreads) out[i] = i;
    for (int i = tid; i < a.last; i += kThreads) out[a.top_k - a.last + i] = seen - a.last + i;
}

template <typename T, int D>
int launch(const SelectArgs &a, cudaStream_t s)
{
    const size_t smem = (size_t)a.max_blocks_per_seq * 4;
    static int raised[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PA_ERR_DEVICE;
    if (!__atomic_load_n(&raised[dev], __ATOMIC_ACQUIRE)) {
        cudaError_t e = cudaFuncSetAttribute(select_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kSelectMaxBlocks * 4);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(select_kernel<T, D>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return launch_status(e);
        __atomic_store_n(&raised[dev], 1, __ATOMIC_RELEASE);
    }
    const long long rows = (long long)a.total_q * a.num_kv_heads;
    // few rows: as many CTAs a row as fit the GPU beside one another
    int ctas = 1;
    while (ctas < 16 && rows * ctas * 2 <= 2 * num_sms() && a.max_blocks_per_seq > 16 * kWarps * ctas) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * ctas));
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
    return launch_status(cudaLaunchKernelEx(&cfg, select_kernel<T, D>, a, ctas));
}

}  // namespace

int select_launch(const SelectArgs &a, int head_dim, bool f32, cudaStream_t s)
{
    if (f32) return head_dim == 64 ? launch<float, 64>(a, s) : launch<float, 128>(a, s);
    return head_dim == 64 ? launch<__nv_bfloat16, 64>(a, s) : launch<__nv_bfloat16, 128>(a, s);
}

}  // namespace pa
