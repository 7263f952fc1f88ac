// pa_sparse: attention of each query over the selected blocks of the paged cache.
//
// A query row (token, kv head: G query heads) has a list of logical blocks; its
// output is softmax(scale q K^T) V over the positions of those blocks that are not
// behind the query, a zero row where there is none.  Bound by the bytes of the
// keys and values, 4 D bytes a token and head in bf16, each read once.
//
// A row is a cluster of 1 to 16 CTAs of kWarps warps, all of which take list
// entries in turn and keep a softmax (m, l, accumulator) of their own: no split of
// a row needs memory or counters outside the cluster, so calls share nothing and
// can be captured as they are.  At the end a CTA joins its warps in shared memory
// and sends each of the cluster's CTAs its share of the channels, which joins what it is sent.
//
// bf16.  A warp has a ring of its own: 16 tokens of one head are one TMA box for K
// and one for V (128-byte swizzled), requested by the warp's first lane as soon as the
// slot has been read.  The heads are on N of mma.sync as in the decode kernel:
// S^T = K q^T, then O^T += V^T P^T with P moved by movmatrix, each weight as three bf16
// numbers, which hold all of its 24 bits (values whose sum cancels show what one or two leave out;
// the further products cost no loads).  Units are summed by fp32 additions.  V rows behind the query
// are zeroed in shared memory, so that what an unused slot holds (even NaN) meets a
// weight of 0 as a zero.
//
// fp32.  Lanes share the channels, four each; a warp has the rows of kTokens tokens in
// registers at a time, products by FMA, exp2f.  Rows of up to four heads have a kernel of
// their own, whose smaller state leaves room for twice the tokens and takes fewer shuffles
// (64 requests, 8 kv heads of 128, 64 blocks of 16, 537 MB: 4 heads each 86 us, 111 in the kernel for 8; 8 heads each 123).
//
// Measured (one GB300): 96 requests, 64 / 8 heads of 128, 128 blocks of 16 tokens each: 123 us for 805 MB, 6.5 TB/s (97% of a
// copy).  565 tokens of 5 chunks, 32 / 8 heads, 64 blocks each: 138 us for 2.4 GB out of L2 (160 MB of it from DRAM), 17 TB/s;
// tensor pipe 44%, issue slots 48% (129 us with two numbers a weight, summed in the products).  One token of 64 blocks: 5.4 us, of
// which the join of 8 CTAs is 1.9.  fp32, 13 requests, 12 / 3 heads of 64, 17 blocks of 32: 7.0 us.
#include <algorithm>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_rows.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kGroup = 8; // most query heads of a kv head
constexpr int kList = 64; // units that a warp looks up at a time
// How far a score may pass the reference of its row's weights (log2).  Weights are 2^-kSlack (exact) of the
// power: none passes 1, and sums reach no further than with the row's maximum as the reference.
constexpr float kSlack = 8.f, kUnslack = 1.f / 256.f;
// Tokens of a unit of the fp32 kernel: 4 KB of K.  (64 channels, 1200 rows of 64 blocks of 16: units of 16 tokens 103 us, of 8 137;
// with blocks of 8, where a unit is half a load, 4000 rows 264 and 235.)
constexpr int unit_f32(int d) { return 1024 / d; }

// One row's partial results in shared memory: [kGroup][D] accumulators, [kGroup]
// maxima (log2 domain), [kGroup] sums; a negative sum marks a row that failed.
template <int D>
struct alignas(16) Part {
    float acc[kGroup][D];
    float m[kGroup], l[kGroup];
};

// Join of partials for four channels of a head.
struct Joined {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    bool bad = false;
    __device__ __forceinline__ void add(const float4 &x, float xm, float xl)
    {
        bad |= xl < 0.f;
        const float mn = fmaxf(m, xm), mu = mn == -INFINITY ? 0.f : mn;
        const float wa = exp2_approx(m - mu), wb = exp2_approx(xm - mu);
        acc.x = acc.x * wa + x.x * wb;
        acc.y = acc.y * wa + x.y * wb;
        acc.z = acc.z * wa + x.z * wb;
        acc.w = acc.w * wa + x.w * wb;
        l = l * wa + xl * wb;
        m = mn;
    }
    __device__ __forceinline__ float4 value() const
    {
        if (bad || l == 0.f) return make_float4(0.f, 0.f, 0.f, 0.f);
        const float i = 1.f / l;
        return make_float4(acc.x * i, acc.y * i, acc.z * i, acc.w * i);
    }
};

__device__ __forceinline__ void put(__nv_bfloat16 *p, const float4 &x)
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
}
__device__ __forceinline__ void put(float *p, const float4 &x) { *reinterpret_cast<float4 *>(p) = x; }

// Threads of a row's W warps: all of the CTA's, or a group of them.
template <int W>
__device__ __forceinline__ void row_sync(int group)
{
    if constexpr (W == kWarps)
        __syncthreads();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * W) : "memory");
}

// What the CTAs of a cluster send one of them: their partials of its share of the channels.
template <int D>
struct alignas(16) Inbox {
    float4 acc[kGroup * D / 4 + 16]; // [CTA][share]
    float m[16][kGroup], l[16][kGroup];
};

// Joins the partials of the row's W warps, `step` bytes apart, and writes the row; in a cluster
// each CTA sends its partial, a share of the channels to each, and joins what it is sent (one barrier;
// reading the others' partials took another and two round trips).  `tid` counts the row's threads.
template <typename T, int D, int W>
__device__ __forceinline__ void finish_row(const void *parts, int step, Inbox<D> *inbox, T *out, int G, int ctas, int rank, int tid,
                                           int group)
{
    const int share = (G * D / 4 + ctas - 1) / ctas; // four channels each
    row_sync<W>(group);
    if (ctas > 1) cluster_wait(); // all CTAs have begun
    for (int f = tid; f < G * D / 4; f += W * 32) {
        const int g = f * 4 / D, d = f * 4 % D;
        Joined j;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const Part<D> *p = reinterpret_cast<const Part<D> *>(static_cast<const uint8_t *>(parts) + w * step);
            j.add(*reinterpret_cast<const float4 *>(&p->acc[g][d]), p->m[g], p->l[g]);
        }
        if (ctas == 1) {
            put(out + 4 * f, j.value());
            continue;
        }
        const int to = f / share;
        cluster_store4(cluster_addr(&inbox->acc[rank * share + f - to * share], to), j.acc);
        if (d / 4 < ctas) { // one of the head's threads for each CTA
            cluster_store(cluster_addr(&inbox->m[rank][g], d / 4), __float_as_uint(j.m));
            cluster_store(cluster_addr(&inbox->l[rank][g], d / 4), __float_as_uint(j.bad ? -1.f : j.l));
        }
    }
    if (ctas == 1) return;
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    for (int i = tid; i < share; i += kThreads) {
        const int f = rank * share + i;
        if (f >= G * D / 4) break;
        const int g = f * 4 / D;
        Joined j;
        for (int c = 0; c < ctas; ++c) j.add(inbox->acc[c * share + i], inbox->m[c][g], inbox->l[c][g]);
        put(out + 4 * f, j.value());
    }
}

// A row that sees nothing, or was refused: zeros.  The same for all CTAs of the row.
template <typename T, int W>
__device__ __forceinline__ void zero_row(T *out, int elements, int rank, int tid)
{
    if (rank != 0) return;
    for (int e = tid * 4; e < elements; e += W * 128) put(out + e, make_float4(0.f, 0.f, 0.f, 0.f));
}

// Units of UNIT tokens that a row's list makes up, `per_block` of them an entry.  The warp's
// next kList of them from `u0`, one in `stride`: those with a visible position, as (first row
// in the pool, first position); their count.
template <int UNIT>
__device__ __forceinline__ int look_up(const SparseArgs &a, const int32_t *list, const int32_t *table, int u0, int stride,
                                       int units, int per_block, int pos, int lane, int2 *items, bool &bad)
{
    int count = 0;
    const int last_block = pos / a.block_size;
    int2 found[kList / 32];
    bool use[kList / 32];
#pragma unroll
    for (int k = 0; k < kList / 32; ++k) {
        const long long u = u0 + (long long)(k * 32 + lane) * stride;
        const int e = u < units ? (int)u / per_block : 0, part = u < units ? (int)u - e * per_block : 0;
        const int lb = u < units ? list[e] : -1;
        found[k] = make_int2(part * UNIT, lb);
    }
#pragma unroll
    for (int k = 0; k < kList / 32; ++k) {
        const int lb = found[k].y, part = found[k].x;
        use[k] = lb >= 0 && lb <= last_block && (long long)lb * a.block_size + part <= pos;
        const int phys = use[k] ? table[lb] : 0;
        const bool wrong = use[k] && (phys < 0 || phys >= a.num_blocks);
        bad |= wrong;
        use[k] &= !wrong;
        found[k] = make_int2(phys * a.block_size + part, lb * a.block_size + part);
    }
#pragma unroll
    for (int k = 0; k < kList / 32; ++k) {
        const uint32_t m = __ballot_sync(kFull, use[k]);
        if (use[k]) items[count + __popc(m & ((1u << lane) - 1))] = found[k];
        count += __popc(m);
    }
    __syncwarp();
    return count;
}

// lo, hi as a bf16 pair; what that leaves stays in them (exact).
__device__ __forceinline__ uint32_t take_bf16(float &lo, float &hi)
{
    const uint32_t w = pack_bf16(lo, hi);
    lo -= __uint_as_float(w << 16);
    hi -= __uint_as_float(w & 0xffff0000u);
    return w;
}

template <int D>
struct Ring {
    static constexpr int KB = D / 64;               // 128-byte slabs of a row
    static constexpr int SLAB = kSparseUnit * 128;  // 16 rows x 64 dims
    static constexpr int HALF = KB * SLAB;          // K (or V) of a unit
    static constexpr int UNIT = 2 * HALF;
    static constexpr int STAGES = D == 128 ? 2 : 4; // 16 KB a warp, 64 KB a CTA, three CTAs an SM
    static constexpr int BYTES = kWarps * STAGES * UNIT;
    static_assert(sizeof(Part<D>) <= STAGES * UNIT, "a warp's partial takes the place of its ring");
};

// W warps a row: kWarps / W rows a CTA, or a cluster of `ctas` for one row (W = kWarps).
template <int D, int W>
__global__ void __launch_bounds__(kThreads, 3)
    sparse_bf16_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const SparseArgs a,
                       int ctas)
{
    using R = Ring<D>;
    constexpr int KS = D / 16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t bars[kWarps][R::STAGES];
    __shared__ int2 lists[kWarps][kList];
    __shared__ Inbox<D> inbox;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = ctas > 1 ? (int)cluster_rank() : 0;
    uint8_t *ring = smem + warp * R::STAGES * R::UNIT;
    uint64_t *bar = bars[warp];
    if (lane == 0) {
        for (int s = 0; s < R::STAGES; ++s) mbar_init(&bar[s], 1);
        fence_mbar_init();
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    __syncwarp();
    grid_dep_trigger();
    if (ctas > 1) cluster_arrive();
    grid_dep_wait();
    check_lengths(a);
    // what the kernel before has stored in the caches is read by copies
    asm volatile("fence.proxy.async.global;" ::: "memory");
    __syncwarp();

    const int group = warp / W, tr = tid % (32 * W);
    const int row = W == kWarps ? (int)(blockIdx.x / ctas) : (int)blockIdx.x * (kWarps / W) + group;
    const int t = row / a.num_kv_heads, h = row % a.num_kv_heads, G = a.group;
    if (W < kWarps && t >= a.total_q) return;
    const QueryRow at = query_row(a, t, lane);
    if (ctas > 1 && (at.skip || at.pos < 0)) cluster_wait(); // (the same for the whole cluster)
    if (at.skip) return;
    const size_t off = ((size_t)t * a.num_heads + (size_t)h * G) * D;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + off;
    if (at.pos < 0) {
        if (at.err && rank == 0 && tr == 0) flag_error(a.dev_err, at.err);
        zero_row<__nv_bfloat16, W>(out, G * D, rank, tr);
        return;
    }
    const int32_t *list = a.selected + (size_t)row * a.top_k;
    const int32_t *table = a.block_table + (size_t)at.req * a.max_blocks_per_seq;

    // q fragments: N = head, K = channel
    uint32_t qf[KS][2];
    {
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + off + (size_t)(lane >> 2) * D + 2 * (lane & 3);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            qf[ks][0] = (lane >> 2) < G ? *reinterpret_cast<const uint32_t *>(q + ks * 16) : 0u;
            qf[ks][1] = (lane >> 2) < G ? *reinterpret_cast<const uint32_t *>(q + ks * 16 + 8) : 0u;
        }
    }
    float acc[KS][4];
#pragma unroll
    for (int i = 0; i < KS; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    bool bad = false;

    const int trow = lane >> 2;
    const int mi = lane >> 3, mr = lane & 7;
    const int k_toff = (mi & 1) * 8 + mr, k_doff = (mi >> 1) * 8; // ldmatrix A = K
    const int v_toff = (mi >> 1) * 8 + mr, v_doff = (mi & 1) * 8; // ldmatrix.trans A = V^T
    const int upb = a.block_size / kSparseUnit, all = a.top_k * upb; // units a block, and of the list
    const int stride = ctas * W;
    int2 *items = lists[warp];
    int stage = 0;
    uint32_t phase = 0;

    bool stuck = false; // a wait gave up: the row fails
    for (int u0 = rank * W + warp % W; u0 < all && !stuck; u0 += kList * stride) {
        const int units = look_up<kSparseUnit>(a, list, table, u0, stride, all, upb, at.pos, lane, items, bad);
        const int2 item0 = items[lane], item1 = items[lane + 32]; // (from `units` on: leftovers)
        auto request = [&](int r0, int s) { // lane 0
            const uint32_t dst = smem_u32(ring + s * R::UNIT);
            mbar_arrive_expect_tx(&bar[s], R::UNIT);
            tma_load_3d(dst, &tm_k, &bar[s], 0, r0, h * R::KB);
            tma_load_3d(dst + R::HALF, &tm_v, &bar[s], 0, r0, h * R::KB);
        };
        if (lane == 0)
            for (int u = 0, s = stage; u < min(units, R::STAGES); ++u) {
                request(items[u].x, s);
                s = s + 1 == R::STAGES ? 0 : s + 1;
            }
        __syncwarp();
        for (int u = 0; u < units; ++u) {
            // the unit's first position, the next request's row
            const int pos0 = __shfl_sync(kFull, u < 32 ? item0.y : item1.y, u & 31);
            const int ahead = u + R::STAGES, r0 = __shfl_sync(kFull, ahead < 32 ? item0.x : item1.x, ahead & 31);
            if (!__all_sync(kFull, mbar_wait(&bar[stage], phase))) {
                stuck = true;
                break;
            }
            uint8_t *kst = ring + stage * R::UNIT, *vst = kst + R::HALF;
            const int live = min(at.pos - pos0 + 1, kSparseUnit); // tokens that the query sees, from 1
            if (live < kSparseUnit) {
                const int chunks = (kSparseUnit - live) * 8;
                for (int ci = lane; ci < chunks * R::KB; ci += 32) {
                    const int slab = ci / chunks, rem = ci % chunks;
                    *reinterpret_cast<uint4 *>(vst + slab * R::SLAB + (live + rem / 8) * 128 + (rem % 8) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            // ---- S^T[token, head] = K q^T, even and odd steps apart (two chains)
            const uint32_t kbase = smem_u32(kst), vbase = smem_u32(vst);
            float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int d = ks * 16 + k_doff;
                uint32_t r0, r1, r2, r3;
                ldsm_x4(kbase + (d >> 6) * R::SLAB + sw128_offset(k_toff, d & 63), r0, r1, r2, r3);
                mma_bf16_16816(ks & 1 ? s2 : s, r0, r1, r2, r3, qf[ks][0], qf[ks][1]);
            }
            // ---- scale (log2 domain), mask
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = (s[i] + s2[i]) * a.scale_log2;
            if (live < kSparseUnit) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (trow + ((i >> 1) << 3) >= live) s[i] = -INFINITY;
            }
            // ---- the reference of the weights follows the maximum when that has grown by
            // more than 2^kSlack: no maximum over the lanes and no rescaling for most units
            const bool grown = fmaxf(s[0], s[2]) > m0 + kSlack || fmaxf(s[1], s[3]) > m1 + kSlack;
            if (__any_sync(kFull, grown)) {
                float t0 = fmaxf(s[0], s[2]), t1 = fmaxf(s[1], s[3]);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    t0 = fmaxf(t0, __shfl_xor_sync(kFull, t0, o));
                    t1 = fmaxf(t1, __shfl_xor_sync(kFull, t1, o));
                }
                t0 = fmaxf(m0, t0), t1 = fmaxf(m1, t1);
                const float al0 = t0 == -INFINITY ? 1.f : exp2_approx(m0 - t0), al1 = t1 == -INFINITY ? 1.f : exp2_approx(m1 - t1);
                m0 = t0;
                m1 = t1;
                l0 *= al0;
                l1 *= al1;
#pragma unroll
                for (int dm = 0; dm < KS; ++dm) {
                    acc[dm][0] *= al0;
                    acc[dm][1] *= al1;
                    acc[dm][2] *= al0;
                    acc[dm][3] *= al1;
                }
            }
            const float mu0 = m0 == -INFINITY ? 0.f : m0, mu1 = m1 == -INFINITY ? 0.f : m1;
            s[0] = exp2_approx(s[0] - mu0) * kUnslack;
            s[1] = exp2_approx(s[1] - mu1) * kUnslack;
            s[2] = exp2_approx(s[2] - mu0) * kUnslack;
            s[3] = exp2_approx(s[3] - mu1) * kUnslack;
            l0 += s[0] + s[2];
            l1 += s[1] + s[3];
            // ---- O^T[channel, head] += V^T P^T, a weight as the sum of three bf16 numbers, the least
            // first.  The unit's products are added to the row's by an fp32 addition: a matrix product
            // cuts its sum off (a row of 2048 units summed in it was off by 2^-15.5 of its magnitudes).
            uint32_t w[3][2];
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    w[i][j] = movmatrix_trans(take_bf16(s[2 * j], s[2 * j + 1]));
#pragma unroll
            for (int dm = 0; dm < KS; ++dm) {
                const int d = dm * 16 + v_doff;
                uint32_t r0, r1, r2, r3;
                ldsm_x4_trans(vbase + (d >> 6) * R::SLAB + sw128_offset(v_toff, d & 63), r0, r1, r2, r3);
                float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 2; i >= 0; --i) mma_bf16_16816(o, r0, r1, r2, r3, w[i][0], w[i][1]);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[dm][i] += o[i];
            }
            __syncwarp(); // every lane has read the slot
            if (lane == 0 && ahead < units) request(r0, stage);
            if (++stage == R::STAGES) {
                stage = 0;
                phase ^= 1;
            }
        }
    }
    // ---- the warp's partial, where its ring was
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        l0 += __shfl_xor_sync(kFull, l0, o);
        l1 += __shfl_xor_sync(kFull, l1, o);
    }
    bad = __any_sync(kFull, bad);
    if (bad && lane == 0) flag_error(a.dev_err, PA_DEVERR_BAD_BLOCK);
    if (stuck && lane == 0) flag_error(a.dev_err, PA_DEVERR_TIMEOUT);
    bad |= stuck;
    Part<D> *part = reinterpret_cast<Part<D> *>(ring);
    const int g0 = 2 * (lane & 3);
#pragma unroll
    for (int dm = 0; dm < KS; ++dm)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            part->acc[g0 + (i & 1)][dm * 16 + trow + ((i >> 1) << 3)] = acc[dm][i];
    if (trow == 0) {
        part->m[g0] = m0;
        part->m[g0 + 1] = m1;
        part->l[g0] = bad ? -1.f : l0;
        part->l[g0 + 1] = bad ? -1.f : l1;
    }
    finish_row<__nv_bfloat16, D, W>(smem + group * W * R::STAGES * R::UNIT, R::STAGES * R::UNIT, &inbox, out, G, ctas, rank, tr,
                                    group);
}

// ------------------------------------------------------------------ fp32
// The sums of v[0..H-1] over L lanes, powers of two: lane l of them gets head
// l / (L / H)'s (the heads a lane holds are halved until one is left).
template <int H, int L>
__device__ __forceinline__ float sum_heads(float (&v)[H], int lane)
{
    int o = L / 2;
#pragma unroll
    for (int n = H / 2; n > 0; n /= 2, o /= 2) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = lane & o ? v[i] : v[i + n], keep = lane & o ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(kFull, give, o);
        }
    }
    float x = v[0];
#pragma unroll
    for (; o > 0; o /= 2) x += __shfl_xor_sync(kFull, x, o);
    return x;
}

// H: heads that a row has room for.  A lane has four channels, so the warp has one token of
// 128 channels or two of 64 side by side, each side with a softmax state of its own (lanes of two
// channels shuffle and broadcast twice as often: 64 requests, 8 heads on each of 8 kv heads of 64, 86 us and 67).
template <int D, int H>
__global__ void __launch_bounds__(kThreads, 4) sparse_f32_kernel(const SparseArgs a, int ctas)
{
    constexpr int kUnit = unit_f32(D), L = D / 4, kSides = 32 / L, kLanes = L / H; // lanes a token, and of them a head
    constexpr int kTokens = 4096 / (H * D), kBatch = kTokens / kSides; // at a time: of the warp, of a side
    __shared__ Part<D> parts[kWarps];
    __shared__ Inbox<D> inbox;
    __shared__ int2 lists[kWarps][kList];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, side = lane / L, sub = lane % L;
    const int rank = ctas > 1 ? (int)cluster_rank() : 0;
    grid_dep_trigger();
    if (ctas > 1) cluster_arrive();
    grid_dep_wait();
    check_lengths(a);
    __syncwarp();
    const int row = blockIdx.x / ctas, t = row / a.num_kv_heads, h = row % a.num_kv_heads, G = a.group;
    const QueryRow at = query_row(a, t, lane);
    if (ctas > 1 && (at.skip || at.pos < 0)) cluster_wait(); // (the same for the whole cluster)
    if (at.skip) return;
    const size_t off = ((size_t)t * a.num_heads + (size_t)h * G) * D;
    float *out = static_cast<float *>(a.out) + off;
    if (at.pos < 0) {
        if (at.err && rank == 0 && tid == 0) flag_error(a.dev_err, at.err);
        zero_row<float, kWarps>(out, G * D, rank, tid);
        return;
    }
    const int32_t *list = a.selected + (size_t)row * a.top_k;
    const int32_t *table = a.block_table + (size_t)at.req * a.max_blocks_per_seq;
    const float *q = static_cast<const float *>(a.q) + off + sub * 4;
    float x[H][4], acc[H][4];
#pragma unroll
    for (int g = 0; g < H; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[g][i] = g < G ? q[(size_t)g * D + i] : 0.f;
            acc[g][i] = 0.f;
        }
    // softmax state of head sub / kLanes of the side's tokens, in the log2 domain
    float m = -INFINITY, l = 0.f;
    bool bad = false;
    const float *kc = static_cast<const float *>(a.k_cache) + (size_t)h * D + sub * 4;
    const float *vc = static_cast<const float *>(a.v_cache) + (size_t)h * D + sub * 4;
    const size_t rowlen = (size_t)a.num_kv_heads * D;
    const int upb = (a.block_size + kUnit - 1) / kUnit, all = a.top_k * upb, stride = ctas * kWarps;
    int2 *items = lists[warp];
    for (int u0 = rank * kWarps + warp; u0 < all; u0 += kList * stride) {
        const int count = look_up<kUnit>(a, list, table, u0, stride, all, upb, at.pos, lane, items, bad);
        for (int it = 0; it < count; ++it) {
            const int2 item = items[it];
            // up to the query, the end of the unit and of the block
            const int live = min(min(at.pos - item.y + 1, kUnit), a.block_size - item.y % a.block_size);
            for (int t0 = 0; t0 < live; t0 += kTokens) {
                float k[kBatch][4], v[kBatch][4], s[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const size_t r = (size_t)(item.x + min(t0 + b * kSides + side, live - 1)) * rowlen;
                    *reinterpret_cast<float4 *>(k[b]) = *reinterpret_cast<const float4 *>(kc + r);
                    *reinterpret_cast<float4 *>(v[b]) = *reinterpret_cast<const float4 *>(vc + r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[b][i] = t0 + b * kSides + side < live ? v[b][i] : 0.f;
                }
                float most = -INFINITY;
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    float dot[H];
#pragma unroll
                    for (int g = 0; g < H; ++g) {
                        dot[g] = 0.f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) dot[g] = fmaf(x[g][i], k[b][i], dot[g]);
                    }
                    s[b] = sum_heads<H, L>(dot, lane) * a.scale_log2;
                    if (t0 + b * kSides + side >= live) s[b] = -INFINITY;
                    most = fmaxf(most, s[b]);
                }
                if (__any_sync(kFull, most > m + kSlack)) { // as in bf16
                    most = fmaxf(most, m);
                    const float al = most == -INFINITY ? 1.f : exp2f(m - most);
                    m = most;
                    l *= al;
#pragma unroll
                    for (int g = 0; g < H; ++g) {
                        const float w = __shfl_sync(kFull, al, side * L + kLanes * g);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[g][i] *= w;
                    }
                }
                const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    s[b] = exp2f(s[b] - mu) * kUnslack;
                    l += s[b];
                }
#pragma unroll
                for (int g = 0; g < H; ++g) {
                    if (g >= G) break;
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        const float p = __shfl_sync(kFull, s[b], side * L + kLanes * g);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[g][i] = fmaf(p, v[b][i], acc[g][i]);
                    }
                }
            }
        }
    }
    bad = __any_sync(kFull, bad);
    if (bad && lane == 0) flag_error(a.dev_err, PA_DEVERR_BAD_BLOCK);
    if (kSides == 2) {
        const float most = fmaxf(m, __shfl_xor_sync(kFull, m, 16)), al = most == -INFINITY ? 1.f : exp2f(m - most);
        m = most;
        l *= al;
        l += __shfl_xor_sync(kFull, l, 16);
#pragma unroll
        for (int g = 0; g < H; ++g) {
            const float w = __shfl_sync(kFull, al, side * L + kLanes * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[g][i] *= w;
                acc[g][i] += __shfl_xor_sync(kFull, acc[g][i], 16);
            }
        }
    }
    Part<D> &part = parts[warp];
    if (side == 0) {
#pragma unroll
        for (int g = 0; g < H; ++g)
            *reinterpret_cast<float4 *>(&part.acc[g][sub * 4]) = *reinterpret_cast<float4 *>(acc[g]);
        if (sub % kLanes == 0) {
            part.m[sub / kLanes] = m;
            part.l[sub / kLanes] = bad ? -1.f : l;
        }
    }
    finish_row<float, D, kWarps>(parts, sizeof(Part<D>), &inbox, out, G, ctas, rank, tid, 0);
}

// How a row is split.  Few rows: a cluster of CTAs each, up to four CTAs an SM in all, while each warp
// has two units.  Many (`pairs` an SM and more):
// two warps a row instead of four, which spend less on beginning and joining rows.  64 blocks of
// 16 tokens, four warps and two, us, rows of one chunk: head_dim 128, 896 rows 32.4 and 29.4, 1600 rows 58.0 and 56.0,
// 7000 rows 233 and 213; head_dim 64, 3000 rows 81.5 and 77.5, 7000 rows 181 and 160.  Rows with blocks of their own, out
// of DRAM: 896 rows 74.9 and 75.0, 7000 rows 528 and 529; head_dim 64, 3000 rows 151 and 154, 7000 rows 339 and 341.
struct Split {
    int ctas, warps;
};
Split split_of(const SparseArgs &a, int unit, int pairs)
{
    const long long rows = (long long)a.total_q * a.num_kv_heads, units = (long long)a.top_k * ((a.block_size + unit - 1) / unit);
    Split s{1, kWarps};
    const long long fit = std::min<long long>(4ll * num_sms() / rows, (units + 2 * kWarps - 1) / (2 * kWarps));
    s.ctas = fit <= 1 ? 1 : fit <= 8 ? (int)fit : fit >= 16 && rows * 16 <= 2 * num_sms() ? 16 : 8; // (9 to 15 are slower than 8)
    if (pairs > 0 && rows >= (long long)pairs * num_sms()) s.warps = 2;
    return s;
}

template <typename Kernel, typename... A>
int launch(Kernel kernel, int *raised, size_t smem, const Split &split, const SparseArgs &a, cudaStream_t s, const A &...args)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PA_ERR_DEVICE;
    if (!__atomic_load_n(&raised[dev], __ATOMIC_ACQUIRE)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return launch_status(e);
        __atomic_store_n(&raised[dev], 1, __ATOMIC_RELEASE);
    }
    const long long rows = (long long)a.total_q * a.num_kv_heads, per_cta = kWarps / split.warps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + per_cta - 1) / per_cta * split.ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split.ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split.ctas > 1 ? 2 : 1;
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, args..., a, split.ctas));
}

template <int D, int W>
int launch_bf16(const SparseArgs &a, const Split &split, const CUtensorMap &tm_k, const CUtensorMap &tm_v, cudaStream_t s)
{
    static int raised[64];
    return launch(sparse_bf16_kernel<D, W>, raised, Ring<D>::BYTES + 1024, split, a, s, tm_k, tm_v);
}

template <int D>
int launch_bf16(const SparseArgs &a, const CUtensorMap &tm_k, const CUtensorMap &tm_v, cudaStream_t s)
{
    const Split split = split_of(a, kSparseUnit, D == 128 ? 6 : 40);
    if (split.warps == 2) return launch_bf16<D, 2>(a, split, tm_k, tm_v, s);
    return launch_bf16<D, kWarps>(a, split, tm_k, tm_v, s);
}

template <int D, int H>
int launch_f32(const SparseArgs &a, const Split &split, cudaStream_t s)
{
    static int raised[64];
    return launch(sparse_f32_kernel<D, H>, raised, 0, split, a, s);
}

}  // namespace

int sparse_bf16_launch(const SparseArgs &a, int head_dim, const CUtensorMap &tm_k, const CUtensorMap &tm_v, cudaStream_t s)
{
    return head_dim == 64 ? launch_bf16<64>(a, tm_k, tm_v, s) : launch_bf16<128>(a, tm_k, tm_v, s);
}

int sparse_f32_launch(const SparseArgs &a, int head_dim, cudaStream_t s)
{
    const Split split = split_of(a, unit_f32(head_dim), 0);
    if (a.group <= 4) return head_dim == 64 ? launch_f32<64, 4>(a, split, s) : launch_f32<128, 4>(a, split, s);
    return head_dim == 64 ? launch_f32<64, kGroup>(a, split, s) : launch_f32<128, kGroup>(a, split, s);
}

}  // namespace pa
