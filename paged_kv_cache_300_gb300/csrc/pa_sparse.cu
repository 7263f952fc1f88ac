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
// can be captured as they are.  At the end a CTA joins its warps in shared memory,
// and the cluster's CTAs join a share of the channels each, read from one another.
//
// bf16.  A warp has a ring of its own: 16 tokens of one head are one TMA box for K
// and one for V (128-byte swizzled), requested by the warp's first lane as soon as the
// slot has been read.  The heads are on N of mma.sync as in the decode kernel:
// S^T = K q^T, then O^T += V^T P^T with P moved by movmatrix, each weight as two bf16
// numbers (one alone is off by 2^-9, which shows beside the output's own rounding; the
// second product costs no loads).  V rows behind the query
// are zeroed in shared memory, so that what an unused slot holds (even NaN) meets a
// weight of 0 as a zero.
//
// fp32.  Lanes share the channels; a warp has the rows of kBatch tokens in registers
// at a time, products by FMA, expf.
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_rows.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kGroup = 8; // most query heads of a kv head
constexpr int kList = 64; // list entries that a warp looks up at a time

// One row's partial results in shared memory: [kGroup][D] accumulators, [kGroup]
// maxima (log2 domain), [kGroup] sums; a negative sum marks a row that failed.
template <int D>
struct Part {
    float acc[kGroup][D];
    float m[kGroup], l[kGroup];
};

// Join of `count` partials for head g, channel d: the weights, the sum, the value.
struct Joined {
    float acc = 0.f, m = -INFINITY, l = 0.f;
    bool bad = false;
    __device__ __forceinline__ void add(float x, float xm, float xl)
    {
        bad |= xl < 0.f;
        const float mn = fmaxf(m, xm), mu = mn == -INFINITY ? 0.f : mn;
        const float wa = exp2_approx(m - mu), wb = exp2_approx(xm - mu);
        acc = acc * wa + x * wb;
        l = l * wa + xl * wb;
        m = mn;
    }
};

__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }

// Joins the CTA's kWarps partials, then the cluster's, and writes the row.
template <typename T, int D>
__device__ __forceinline__ void finish_row(Part<D> *parts, Part<D> *cta, T *out, int G, int ctas, int rank)
{
    const int tid = threadIdx.x;
    __syncthreads();
    for (int e = tid; e < G * D; e += kThreads) {
        const int g = e / D, d = e % D;
        Joined j;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) j.add(parts[w].acc[g][d], parts[w].m[g], parts[w].l[g]);
        if (ctas == 1) {
            put(out + e, j.bad || j.l == 0.f ? 0.f : j.acc / j.l);
        } else {
            cta->acc[g][d] = j.acc;
            if (d == 0) {
                cta->m[g] = j.m;
                cta->l[g] = j.bad ? -1.f : j.l;
            }
        }
    }
    if (ctas == 1) return;
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    for (int e = rank * kThreads + tid; e < G * D; e += ctas * kThreads) {
        const int g = e / D, d = e % D;
        Joined j;
        for (int c = 0; c < ctas; ++c)
            j.add(cluster_load(cluster_addr(&cta->acc[g][d], c)), cluster_load(cluster_addr(&cta->m[g], c)),
                  cluster_load(cluster_addr(&cta->l[g], c)));
        put(out + e, j.bad || j.l == 0.f ? 0.f : j.acc / j.l);
    }
    __syncwarp();
    cluster_arrive(); // the others' shared memory stays until all have read it
    cluster_wait();
}

// A row that sees nothing, or was refused: zeros.  The same for all CTAs of the row.
template <typename T>
__device__ __forceinline__ void zero_row(T *out, int elements, int rank)
{
    if (rank != 0) return;
    for (int e = threadIdx.x; e < elements; e += kThreads) put(out + e, 0.f);
}

// The warp's next kList list entries from `e0`, one in `stride`: those that are visible,
// as (first row in the pool, logical block), in list order; their count.
__device__ __forceinline__ int look_up(const SparseArgs &a, const int32_t *list, const int32_t *table, int e0, int stride,
                                       int last_block, int lane, int2 *items, bool &bad)
{
    int count = 0;
#pragma unroll
    for (int k = 0; k < kList / 32; ++k) {
        const long long e = e0 + (long long)(k * 32 + lane) * stride;
        int lb = -1, phys = 0;
        if (e < a.top_k) lb = __ldg(list + e);
        const bool use = lb >= 0 && lb <= last_block;
        if (use) phys = __ldg(table + lb);
        const bool wrong = use && (phys < 0 || phys >= a.num_blocks);
        bad |= wrong;
        const uint32_t m = __ballot_sync(kFull, use && !wrong);
        if (use && !wrong) items[count + __popc(m & ((1u << lane) - 1))] = make_int2(phys * a.block_size, lb);
        count += __popc(m);
    }
    __syncwarp();
    return count;
}

// What rounding lo, hi to the bf16 pair w has left, as a bf16 pair.
__device__ __forceinline__ uint32_t left_of(float lo, float hi, uint32_t w)
{
    return pack_bf16(lo - __uint_as_float(w << 16), hi - __uint_as_float(w & 0xffff0000u));
}

template <int D>
struct Ring {
    static constexpr int KB = D / 64;               // 128-byte slabs of a row
    static constexpr int SLAB = kSparseUnit * 128;  // 16 rows x 64 dims
    static constexpr int HALF = KB * SLAB;          // K (or V) of a unit
    static constexpr int UNIT = 2 * HALF;
    static constexpr int STAGES = D == 128 ? 3 : 6; // 24 KB a warp, 96 KB a CTA, two CTAs an SM
    static constexpr int BYTES = kWarps * STAGES * UNIT;
    static_assert(sizeof(Part<D>) <= STAGES * UNIT, "a warp's partial takes the place of its ring");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    sparse_bf16_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const SparseArgs a,
                       int ctas)
{
    using R = Ring<D>;
    constexpr int KS = D / 16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t bars[kWarps][R::STAGES];
    __shared__ int2 lists[kWarps][kList];
    __shared__ Part<D> cta_part;
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
    grid_dep_wait();

    const int row = blockIdx.x / ctas, t = row / a.num_kv_heads, h = row % a.num_kv_heads, G = a.group;
    const QueryRow at = query_row(a, t, lane);
    if (at.skip) return;
    const size_t off = ((size_t)t * a.num_heads + (size_t)h * G) * D;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + off;
    if (at.pos < 0) {
        if (at.err && rank == 0 && tid == 0) flag_error(a.dev_err, at.err);
        zero_row(out, G * D, rank);
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
    const int upb = a.block_size / kSparseUnit;                   // units a block
    const int stride = ctas * kWarps;
    int2 *items = lists[warp];
    int stage = 0;
    uint32_t phase = 0;

    bool stuck = false; // a wait gave up: the row fails
    for (int e0 = rank * kWarps + warp; e0 < a.top_k && !stuck; e0 += kList * stride) {
        const int units = look_up(a, list, table, e0, stride, at.pos / a.block_size, lane, items, bad) * upb;
        auto request = [&](int u, int s) { // lane 0
            const int r0 = items[u / upb].x + (u % upb) * kSparseUnit;
            const uint32_t dst = smem_u32(ring + s * R::UNIT);
            mbar_arrive_expect_tx(&bar[s], R::UNIT);
            tma_load_3d(dst, &tm_k, &bar[s], 0, r0, h * R::KB);
            tma_load_3d(dst + R::HALF, &tm_v, &bar[s], 0, r0, h * R::KB);
        };
        if (lane == 0)
            for (int u = 0, s = stage; u < min(units, R::STAGES); ++u) {
                request(u, s);
                s = s + 1 == R::STAGES ? 0 : s + 1;
            }
        __syncwarp();
        for (int u = 0; u < units; ++u) {
            if (!mbar_wait(&bar[stage], phase)) {
                if (lane == 0) flag_error(a.dev_err, PA_DEVERR_TIMEOUT);
                stuck = true;
                break;
            }
            const int pos0 = items[u / upb].y * a.block_size + (u % upb) * kSparseUnit; // of the unit's first token
            uint8_t *kst = ring + stage * R::UNIT, *vst = kst + R::HALF;
            const int live = min(at.pos - pos0 + 1, kSparseUnit); // tokens that the query sees
            if (live < kSparseUnit) {
                const int r0 = max(live, 0), chunks = (kSparseUnit - r0) * 8;
                for (int ci = lane; ci < chunks * R::KB; ci += 32) {
                    const int slab = ci / chunks, rem = ci % chunks;
                    *reinterpret_cast<uint4 *>(vst + slab * R::SLAB + (r0 + rem / 8) * 128 + (rem % 8) * 16) =
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
            // ---- mask, scale (log2 domain), online softmax
            float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool vis = trow + ((i >> 1) << 3) < live;
                s[i] = vis ? (s[i] + s2[i]) * a.scale_log2 : -INFINITY;
                if (i & 1)
                    t1 = fmaxf(t1, s[i]);
                else
                    t0 = fmaxf(t0, s[i]);
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                t0 = fmaxf(t0, __shfl_xor_sync(kFull, t0, o));
                t1 = fmaxf(t1, __shfl_xor_sync(kFull, t1, o));
            }
            const float mn0 = fmaxf(m0, t0), mn1 = fmaxf(m1, t1);
            const float mu0 = mn0 == -INFINITY ? 0.f : mn0, mu1 = mn1 == -INFINITY ? 0.f : mn1;
            const float al0 = exp2_approx(m0 - mu0), al1 = exp2_approx(m1 - mu1);
            m0 = mn0;
            m1 = mn1;
            s[0] = exp2_approx(s[0] - mu0);
            s[1] = exp2_approx(s[1] - mu1);
            s[2] = exp2_approx(s[2] - mu0);
            s[3] = exp2_approx(s[3] - mu1);
            l0 = l0 * al0 + (s[0] + s[2]);
            l1 = l1 * al1 + (s[1] + s[3]);
#pragma unroll
            for (int dm = 0; dm < KS; ++dm) {
                acc[dm][0] *= al0;
                acc[dm][1] *= al1;
                acc[dm][2] *= al0;
                acc[dm][3] *= al1;
            }
            // ---- O^T[channel, head] += V^T P^T, a weight as the sum of two bf16 numbers
            const uint32_t w0 = pack_bf16(s[0], s[1]), w1 = pack_bf16(s[2], s[3]);
            const uint32_t b0 = movmatrix_trans(w0), b1 = movmatrix_trans(w1);
            const uint32_t c0 = movmatrix_trans(left_of(s[0], s[1], w0)), c1 = movmatrix_trans(left_of(s[2], s[3], w1));
#pragma unroll
            for (int dm = 0; dm < KS; ++dm) {
                const int d = dm * 16 + v_doff;
                uint32_t r0, r1, r2, r3;
                ldsm_x4_trans(vbase + (d >> 6) * R::SLAB + sw128_offset(v_toff, d & 63), r0, r1, r2, r3);
                mma_bf16_16816(acc[dm], r0, r1, r2, r3, b0, b1);
                mma_bf16_16816(acc[dm], r0, r1, r2, r3, c0, c1);
            }
            __syncwarp(); // every lane has read the slot
            if (lane == 0 && u + R::STAGES < units) request(u + R::STAGES, stage);
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
    bad |= stuck;
    Part<D> *part = reinterpret_cast<Part<D> *>(smem) + warp;
    __syncthreads(); // partials lie closer than rings: all rings have been read
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
    finish_row<__nv_bfloat16, D>(reinterpret_cast<Part<D> *>(smem), &cta_part, out, G, ctas, rank);
}

// ------------------------------------------------------------------ fp32
// The sums of v[0..7] over the warp's lanes: lane l gets head l / 4's in one pass of
// 9 shuffles (halving the heads a lane holds at each of the first three).
__device__ __forceinline__ float sum_heads(float (&v)[kGroup], int lane)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float give = lane & 16 ? v[i] : v[i + 4], keep = lane & 16 ? v[i + 4] : v[i];
        v[i] = keep + __shfl_xor_sync(kFull, give, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float give = lane & 8 ? v[i] : v[i + 2], keep = lane & 8 ? v[i + 2] : v[i];
        v[i] = keep + __shfl_xor_sync(kFull, give, 8);
    }
    const float give = lane & 4 ? v[0] : v[1], keep = lane & 4 ? v[1] : v[0];
    float x = keep + __shfl_xor_sync(kFull, give, 4);
    x += __shfl_xor_sync(kFull, x, 2);
    x += __shfl_xor_sync(kFull, x, 1);
    return x;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 3) sparse_f32_kernel(const SparseArgs a, int ctas)
{
    constexpr int E = D / 32, kBatch = 4; // channels a lane, tokens at a time
    using Vec = typename std::conditional<E == 4, float4, float2>::type;
    __shared__ Part<D> parts[kWarps];
    __shared__ Part<D> cta_part;
    __shared__ int2 lists[kWarps][kList];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = ctas > 1 ? (int)cluster_rank() : 0;
    grid_dep_trigger();
    grid_dep_wait();
    const int row = blockIdx.x / ctas, t = row / a.num_kv_heads, h = row % a.num_kv_heads, G = a.group;
    const QueryRow at = query_row(a, t, lane);
    if (at.skip) return;
    const size_t off = ((size_t)t * a.num_heads + (size_t)h * G) * D;
    float *out = static_cast<float *>(a.out) + off;
    if (at.pos < 0) {
        if (at.err && rank == 0 && tid == 0) flag_error(a.dev_err, at.err);
        zero_row(out, G * D, rank);
        return;
    }
    const int32_t *list = a.selected + (size_t)row * a.top_k;
    const int32_t *table = a.block_table + (size_t)at.req * a.max_blocks_per_seq;
    const float *q = static_cast<const float *>(a.q) + off + lane * E;
    float x[kGroup][E], acc[kGroup][E];
#pragma unroll
    for (int g = 0; g < kGroup; ++g)
#pragma unroll
        for (int i = 0; i < E; ++i) {
            x[g][i] = g < G ? q[(size_t)g * D + i] : 0.f;
            acc[g][i] = 0.f;
        }
    // softmax state of head lane / 4, in the log2 domain
    float m = -INFINITY, l = 0.f;
    bool bad = false;
    const float *kc = static_cast<const float *>(a.k_cache) + (size_t)h * D + lane * E;
    const float *vc = static_cast<const float *>(a.v_cache) + (size_t)h * D + lane * E;
    const size_t rowlen = (size_t)a.num_kv_heads * D;
    const int stride = ctas * kWarps, bs = a.block_size;
    int2 *items = lists[warp];
    for (int e0 = rank * kWarps + warp; e0 < a.top_k; e0 += kList * stride) {
        const int count = look_up(a, list, table, e0, stride, at.pos / bs, lane, items, bad);
        for (int it = 0; it < count; ++it) {
            const int2 item = items[it];
            const int live = min(at.pos - item.y * bs + 1, bs); // >= 1
            for (int t0 = 0; t0 < live; t0 += kBatch) {
                float k[kBatch][E], v[kBatch][E], s[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const size_t r = (size_t)(item.x + min(t0 + b, live - 1)) * rowlen;
                    *reinterpret_cast<Vec *>(k[b]) = *reinterpret_cast<const Vec *>(kc + r);
                    *reinterpret_cast<Vec *>(v[b]) = *reinterpret_cast<const Vec *>(vc + r);
#pragma unroll
                    for (int i = 0; i < E; ++i) v[b][i] = t0 + b < live ? v[b][i] : 0.f;
                }
                float most = m;
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    float dot[kGroup];
#pragma unroll
                    for (int g = 0; g < kGroup; ++g) {
                        dot[g] = 0.f;
#pragma unroll
                        for (int i = 0; i < E; ++i) dot[g] = fmaf(x[g][i], k[b][i], dot[g]);
                    }
                    s[b] = sum_heads(dot, lane) * a.scale_log2;
                    if (t0 + b >= live) s[b] = -INFINITY;
                    most = fmaxf(most, s[b]);
                }
                const float mu = most == -INFINITY ? 0.f : most;
                const float al = exp2f(m - mu);
                m = most;
                l *= al;
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    s[b] = exp2f(s[b] - mu);
                    l += s[b];
                }
#pragma unroll
                for (int g = 0; g < kGroup; ++g) {
                    if (g >= G) break;
                    const float w = __shfl_sync(kFull, al, 4 * g);
#pragma unroll
                    for (int i = 0; i < E; ++i) acc[g][i] *= w;
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        const float p = __shfl_sync(kFull, s[b], 4 * g);
#pragma unroll
                        for (int i = 0; i < E; ++i) acc[g][i] = fmaf(p, v[b][i], acc[g][i]);
                    }
                }
            }
        }
    }
    bad = __any_sync(kFull, bad);
    if (bad && lane == 0) flag_error(a.dev_err, PA_DEVERR_BAD_BLOCK);
    Part<D> &part = parts[warp];
#pragma unroll
    for (int g = 0; g < kGroup; ++g)
        *reinterpret_cast<Vec *>(&part.acc[g][lane * E]) = *reinterpret_cast<Vec *>(acc[g]);
    if (lane % 4 == 0) {
        part.m[lane / 4] = m;
        part.l[lane / 4] = bad ? -1.f : l;
    }
    finish_row<float, D>(parts, &cta_part, out, G, ctas, rank);
}

// CTAs a row.  Enough of them for every SM to have a few, while each has work for
// its warps (a block and more).
int ctas_of(const SparseArgs &a)
{
    const long long rows = (long long)a.total_q * a.num_kv_heads;
    int ctas = 1;
    while (ctas < 16 && rows * ctas * 2 <= 4 * num_sms() && a.top_k > 2 * kWarps * ctas) ctas *= 2;
    return ctas;
}

template <typename Kernel, typename... A>
int launch(Kernel kernel, int *raised, size_t smem, const SparseArgs &a, cudaStream_t s, const A &...args)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PA_ERR_DEVICE;
    if (!__atomic_load_n(&raised[dev], __ATOMIC_ACQUIRE)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return launch_status(e);
        __atomic_store_n(&raised[dev], 1, __ATOMIC_RELEASE);
    }
    const int ctas = ctas_of(a);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.total_q * a.num_kv_heads * ctas));
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
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, args..., a, ctas));
}

}  // namespace

int sparse_bf16_launch(const SparseArgs &a, int head_dim, const CUtensorMap &tm_k, const CUtensorMap &tm_v, cudaStream_t s)
{
    static int raised64[64], raised128[64];
    if (head_dim == 64) return launch(sparse_bf16_kernel<64>, raised64, Ring<64>::BYTES + 1024, a, s, tm_k, tm_v);
    return launch(sparse_bf16_kernel<128>, raised128, Ring<128>::BYTES + 1024, a, s, tm_k, tm_v);
}

int sparse_f32_launch(const SparseArgs &a, int head_dim, cudaStream_t s)
{
    static int raised64[64], raised128[64];
    if (head_dim == 64) return launch(sparse_f32_kernel<64>, raised64, 0, a, s);
    return launch(sparse_f32_kernel<128>, raised128, 0, a, s);
}

}  // namespace pa
