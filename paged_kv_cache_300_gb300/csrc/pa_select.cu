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
// heads, of several tokens where there are fewer than 8, on N (or 8 tokens, head after head).  The order of the sum
// over d is free, so a lane's 16-byte load of a row is two k-steps' fragments as it
// stands: bounds go from memory to the tensor cores without shared memory, 8 KB a
// warp in flight.  A CTA takes a tile of neighbouring tokens (one, for decode) and a kv
// head, and reads the bounds once for all of the tile's tokens of a request.  With few
// rows a cluster takes a row; its CTAs score a share each and store the scores in the
// first one's shared memory.
//
// Choice.  The answer is that of the exact scores, ties to the lowest block,
// whatever the order of the sums in fp32.  The k-th largest of the fp32 scores, t,
// is found by histograms; with every score off by at most E, blocks above t + 2 E
// are in and blocks below t - 2 E out for certain.  Where those between are more
// than the places left, their scores are made again to some 60 bits, as differences
// from t, and chosen among by the same histograms.  A warp chooses for a token of a tile;
// the warps that scored it for a token alone: all of the CTA's, or with many rows 4, 2 or one.
//   E: an m16n8k16 step keeps of each of its 17 addends what is above 2^-25 of the largest and cuts its sum off to 24
//   bits (as measured with a product of 1 and others from 2^-20 to 2^-30 of it), so it is off by at most 2.5 2^-22 of the
//   magnitudes; a chain of 8 steps that begins with one large product is off by 2^-18 = 8 * 2 2^-22 of them.  D / 16 steps a
//   chain and the sum of two chains: E < 2^-22 (2.5 D / 16 + 1 / 2) S with S >=
//   sum |q||b| of every head and block.  S is the largest over the blocks of sum_d u_d max(|lo_d|, |hi_d|),
//   u the |q| of a head or, for tiles of tokens and in fp32, the largest |q| of all their heads (one column more).  (fp32: D / 16 + 5
//   roundings of 2^-24.)  L1(q) max|b| costs no product but is some 8 times as much, and then many rows
//   need exact scores (one request: 13.1 us instead of 6.4).
//
// Measured (one GB300): 96 requests of 4096 to 32768 tokens, 64 / 8 heads of 128, 128 of their blocks of 16: 86 us
// for 451 MB (83 with half the window of doubt and compared as floats); 7 TB/s while all CTAs score, less where some choose (4 us a row) and while the last rows end (20 us).
// 565 tokens of 5 chunks, 32 / 8 heads, 64 of up to 750 blocks: 45 us (6 more with the heads of a token on neighbouring
// columns), bound by the latency of two CTAs an SM (the products alone, 8 cycles each, are 8 us): some 24 us score, the rest
// chooses, 5 of it by exact scores.  One token of 313 blocks 6.5 us, 9.5 where a row is in doubt.
#include <algorithm>
#include <float.h>
#include <limits.h>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_rows.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kGroup = 8;   // most query heads of a kv head
constexpr int kTile = 16;   // most tokens of a CTA: a warp chooses for two
constexpr int kPad = 64;    // bytes behind a staged q row: neighbouring rows on other banks
// The largest |q| of all heads is kept divided by this: its sum with the bounds stays finite where each head's is.
constexpr float kShrink = 256.f;

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
__device__ __forceinline__ uint32_t abs2(uint32_t x) { return x & 0x7fff7fffu; }
// The larger magnitude; the other one of a NaN.
__device__ __forceinline__ uint32_t most2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return abs2(r);
}

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

// ------------------------------------------------------------------ the choice
// Shared memory of W warps that choose together.
template <int W>
struct Choice {
    static constexpr int BITS = W == 1 ? 8 : W == 2 ? 9 : W == 4 ? 10 : 11, BINS = 1 << BITS; // 8 bins a thread
    uint32_t bin, above, in, listed, result;
    uint32_t list[32];
    double exact[32];
    uint32_t warp[W][2];
    alignas(16) uint32_t hist[BINS];
};

// Of the calling thread's W neighbouring warps.  (With a numbered barrier for the CTA too, 96 requests
// take 2.6 us more.)
template <int W>
__device__ __forceinline__ void choice_sync()
{
    if (W == 1)
        __syncwarp();
    else if (W == kWarps)
        __syncthreads();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.x / (32 * W)), "n"(32 * W) : "memory");
}

// f(key, its index) for four neighbouring keys of a row in shared memory (16-byte aligned, n rounded
// up to 4 of them, 0 behind the last).
template <typename F>
__device__ __forceinline__ void each4(const uint32_t *key, int i, const F &f)
{
    const uint4 k = *reinterpret_cast<const uint4 *>(key + i);
    f(k.x, i);
    f(k.y, i + 1);
    f(k.z, i + 2);
    f(k.w, i + 3);
}

// Empties the histogram and the list.  `tid` counts the threads of the W warps, here and below.
template <int W>
__device__ __forceinline__ void clear(Choice<W> &sh, int tid)
{
    for (int i = 4 * tid; i < Choice<W>::BINS; i += 128 * W) *reinterpret_cast<uint4 *>(&sh.hist[i]) = make_uint4(0, 0, 0, 0);
    if (tid == 0) sh.listed = 0;
}

// The need-th largest of the keys in [lo, hi] (need >= 1, at most as many as there are; lo >= 1).
// `cleared`: the histogram and the list are empty already, for all threads to see.
template <int W>
__device__ __forceinline__ uint32_t kth_largest(const uint32_t *key, int n, uint32_t need, uint32_t lo, uint32_t hi,
                                                Choice<W> &sh, int tid, bool cleared)
{
    constexpr int T = 32 * W, PER = Choice<W>::BINS / T;
    const int lane = tid & 31, warp = tid >> 5;
    while (lo < hi) { // at most four times
        const int bits = 32 - __clz(hi - lo), shift = max(bits - Choice<W>::BITS, 0);
        if (!cleared) {
            clear(sh, tid);
            choice_sync<W>();
        }
        cleared = false;
#pragma unroll 2
        for (int i = 4 * tid; i < n; i += 4 * T)
            each4(key, i, [&](uint32_t k, int) {
                if (k >= lo && k <= hi) atomicAdd(&sh.hist[(k - lo) >> shift], 1u);
            });
        choice_sync<W>();
        // sums from the top bin down: thread t has bins PER * t ..
        uint32_t bin[PER], sum = 0;
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
            const uint4 b = *reinterpret_cast<const uint4 *>(&sh.hist[tid * PER + i]);
            bin[i] = b.x, bin[i + 1] = b.y, bin[i + 2] = b.z, bin[i + 3] = b.w;
            sum += b.x + b.y + b.z + b.w;
        }
        uint32_t incl = sum; // of this thread and the lanes above
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_down_sync(kFull, incl, o);
            if (lane + o < 32) incl += x;
        }
        uint32_t above = incl - sum;
        if (W > 1) {
            if (lane == 0) sh.warp[warp][0] = incl;
            choice_sync<W>();
#pragma unroll
            for (int w = 1; w < W; ++w) above += w > warp ? sh.warp[w][0] : 0;
        }
        if (above < need && need <= above + sum) { // one thread
#pragma unroll
            for (int i = PER - 1; i >= 0; --i) {
                if (above < need && need <= above + bin[i]) {
                    sh.bin = tid * PER + i;
                    sh.above = above;
                    sh.in = bin[i];
                }
                above += bin[i];
            }
        }
        choice_sync<W>();
        const uint32_t in = sh.in;
        need -= sh.above;
        lo += sh.bin << shift;
        if (shift == 0) return lo; // a bin is one key
        hi = lo + min(hi - lo, (1u << shift) - 1); // (lo + 2^shift may pass 2^32)
        if (in <= 32) { // few enough to look at one by one
#pragma unroll 2
            for (int i = 4 * tid; i < n; i += 4 * T)
                each4(key, i, [&](uint32_t k, int) {
                    if (k >= lo && k <= hi) sh.list[atomicAdd(&sh.listed, 1u)] = k;
                });
            choice_sync<W>();
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
            choice_sync<W>();
            return sh.result;
        }
        choice_sync<W>();
    }
    return lo;
}

// A sum of floats kept as three: what rounding leaves at each level goes to the next
// (the error-free sum of two numbers, Knuth), so the whole is off by some 2^-60 of the
// magnitudes.  64-bit arithmetic would do, but this GPU has little: 2 us a block here.
struct Sum3 {
    float a = 0.f, b = 0.f, c = 0.f;
    template <typename F>
    static __device__ __forceinline__ F two_sum(F x, F y, F &left)
    {
        const F s = x + y, t = s - x;
        left = (x - (s - t)) + (y - t);
        return s;
    }
    __device__ __forceinline__ void add(float x)
    {
        float e, f;
        a = two_sum(a, x, e);
        b = two_sum(b, e, f);
        c += f;
    }
};

// By how much the row's score of a block passes `cut`, which is near it: off by some 2^-60 of the magnitudes.  Four
// lanes share a head, and neighbouring `lanes` of them, a power of two, a block: `bounds` is theirs (null: none) and the
// result, in the first of them.
template <typename T, int D>
__device__ __forceinline__ double score_above(float cut, const T *q, const T *bounds, int G, int lanes, int lane)
{
    const int g = (lane & (lanes - 1)) >> 2;
    Sum3 sum;
    if (g < G && bounds != nullptr) {
        constexpr int N = D / 32;
        T x[N][8], lo[N][8], hi[N][8];
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < (int)sizeof(T) / 2; ++j) {
                const int d = i * 32 + (lane & 3) * 8;
                reinterpret_cast<uint4 *>(x[i])[j] = reinterpret_cast<const uint4 *>(q + (size_t)g * D + d)[j];
                reinterpret_cast<uint4 *>(lo[i])[j] = reinterpret_cast<const uint4 *>(bounds + d)[j];
                reinterpret_cast<uint4 *>(hi[i])[j] = reinterpret_cast<const uint4 *>(bounds + D + d)[j];
            }
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = to_float(x[i][j]), v = u > 0.f ? to_float(hi[i][j]) : to_float(lo[i][j]); // the other product is 0
                const float p = __fmul_rn(u, v); // (never taken into an addition: what it rounds off is added too)
                sum.add(p);
                if (sizeof(T) == 4) sum.add(fmaf(u, v, -p)); // (bf16 products are exact)
            }
    }
    double s = sum.a, rest = (double)sum.b + (double)sum.c;
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        double left;
        s = Sum3::two_sum(s, __shfl_xor_sync(kFull, s, o), left);
        rest += __shfl_xor_sync(kFull, rest, o) + left;
    }
    s = (s - (double)cut) + rest;
    // A head with an infinite q is -infinity where the row's fp32 score is finite; its sum above is NaN.
    if (!(s > -INFINITY)) s = -INFINITY;
    for (int k = 1; k < G; ++k) { // the largest
        const double x = __shfl_down_sync(kFull, s, 4 * k);
        if (g == 0 && x > s) s = x;
    }
    return s;
}

// What a row's choice is made from.
template <typename T>
struct Row {
    const T *q;           // of the row's G heads
    const T *bounds;      // of the kv head
    const int32_t *table; // of the scored blocks
    int n, first;         // scored blocks, the logical number of the first of them
    int need;             // to be chosen
    float width;          // 2 E
};

// Writes the `need` of the row's n scored blocks with the largest scores to out, ascending.
// `key` holds the scores; `heads` is a.group rounded up to a power of two.
template <typename T, int D, int W>
__device__ __forceinline__ void choose(uint32_t *key, const Row<T> &r, int32_t *out, const SelectArgs &a, int heads, Choice<W> &sh, int tid)
{
    const int lane = tid & 31, warp = tid >> 5, n = r.n, need = r.need;
    uint32_t least = 0xffffffffu, most = 0;
    clear(sh, tid);
#pragma unroll 2
    for (int i = 4 * tid; i < n; i += 128 * W) { // scores to keys
        uint32_t k[4];
        each4(key, i, [&](uint32_t x, int j) {
            k[j - i] = j < n ? key_of(__uint_as_float(x)) : 0u;
            if (j < n) least = min(least, k[j - i]);
            most = max(most, k[j - i]);
        });
        *reinterpret_cast<uint4 *>(key + i) = make_uint4(k[0], k[1], k[2], k[3]);
    }
    least = __reduce_min_sync(kFull, least);
    most = __reduce_max_sync(kFull, most);
    choice_sync<1>();
    if (W > 1) {
        if (lane == 0) {
            sh.warp[warp][0] = least;
            sh.warp[warp][1] = most;
        }
        choice_sync<W>();
#pragma unroll
        for (int w = 0; w < W; ++w) {
            least = min(least, sh.warp[w][0]);
            most = max(most, sh.warp[w][1]);
        }
        choice_sync<W>();
    }
    // keys above `high` are in, and `quota` of those from `low` to `high`
    uint32_t low = kth_largest<W>(key, n, need, least, most, sh, tid, true), high = low;
    const float cut = value_of(low);
    const bool blurred = fabsf(cut) < INFINITY && r.width > 0.f && r.width < INFINITY;
    if (blurred) {
        low = key_of(cut - r.width);
        high = key_of(fminf(cut + r.width, FLT_MAX)); // (infinities stay above)
    }
    // each warp has a run of a multiple of 128 keys, so that places follow from counts
    const int per = ((n + 128 * W - 1) / (128 * W)) * 128, i0 = warp * per, i1 = min(n, i0 + per);
    int sure = 0, open = 0, sure_before = 0, open_before = 0;
    for (int pass = 0;; ++pass) {
        int mine_sure = 0, mine_open = 0;
#pragma unroll 2
        for (int i = i0 + 4 * lane; i < i1; i += 128)
            each4(key, i, [&](uint32_t k, int) {
                mine_sure += k > high;
                mine_open += k >= low && k <= high;
            });
        mine_sure = __reduce_add_sync(kFull, mine_sure);
        mine_open = __reduce_add_sync(kFull, mine_open);
        if (W > 1) {
            if (lane == 0) {
                sh.warp[warp][0] = mine_sure;
                sh.warp[warp][1] = mine_open;
            }
            choice_sync<W>();
            sure = open = sure_before = open_before = 0;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                if (w == warp) {
                    sure_before = sure;
                    open_before = open;
                }
                sure += sh.warp[w][0];
                open += sh.warp[w][1];
            }
        } else {
            sure = mine_sure;
            open = mine_open;
        }
        if (pass == 2 || !blurred || sure + open == need) break;
        // more blocks than places within the error of the scores: again and exactly, as the difference
        // from the cut.  A few are compared as doubles; of many first what a float holds of the differences,
        // then, among those of the last float that is taken, what it has left (another 2^-24).
        if (open <= 32) {
            if (tid == 0) sh.listed = 0;
            choice_sync<W>();
            for (int i = i0 + lane; i < i1; i += 32)
                if (key[i] >= low && key[i] <= high) sh.list[atomicAdd(&sh.listed, 1u)] = i;
            choice_sync<W>();
            const int lanes = 4 * heads, blocks = 32 / lanes; // of a block, of a warp
            for (int c0 = warp * blocks; c0 < open; c0 += W * blocks) {
                const int c = c0 + lane / lanes;
                const T *bounds = c < open ? r.bounds + (size_t)r.table[sh.list[c]] * a.num_kv_heads * 2 * D : nullptr;
                const double x = score_above<T, D>(cut, r.q, bounds, a.group, lanes, lane);
                if (c < open && lane % lanes == 0) sh.exact[c] = x;
            }
            choice_sync<W>();
            if (tid < open) {
                int before = 0;
                for (int c = 0; c < open; ++c)
                    before += sh.exact[c] > sh.exact[tid] || (sh.exact[c] == sh.exact[tid] && sh.list[c] < sh.list[tid]);
                key[sh.list[tid]] = before < need - sure ? 0xffffffffu : 0u;
            }
            choice_sync<W>();
            low = high; // none is left there
            continue;
        }
        for (int i = i0 + lane; i - lane < i1; i += 32) {
            const uint32_t k = i < i1 ? key[i] : 0;
            uint32_t todo = __ballot_sync(kFull, i < i1 && k >= low && k <= high);
            uint32_t now = k > high ? 0xffffffffu : 0u;
            while (todo) {
                const int b = __ffs(todo) - 1;
                todo &= todo - 1;
                const T *bounds = r.bounds + (size_t)r.table[(i - lane) + b] * a.num_kv_heads * 2 * D;
                const double x = __shfl_sync(kFull, score_above<T, D>(cut, r.q, bounds, a.group, 32, lane), 0);
                if (lane == b) now = key_of(pass == 0 || !(fabs(x) < INFINITY) ? (float)x : (float)(x - (double)(float)x));
            }
            if (i < i1) key[i] = now;
        }
        choice_sync<W>();
        low = high = kth_largest<W>(key, n, need - sure, 1u, 0xfffffffeu, sh, tid, false);
        choice_sync<W>();
    }
    const int quota = need - sure;
    const uint32_t below = (1u << lane) - 1;
    int place = sure_before + min(open_before, quota), ties = open_before;
    for (int i = i0 + 4 * lane; i - 4 * lane < i1; i += 128) {
        bool in[4] = {false, false, false, false}, eq[4] = {false, false, false, false};
        if (i < i1)
            each4(key, i, [&](uint32_t k, int j) {
                in[j - i] = k > high;
                eq[j - i] = k >= low && k <= high;
            });
        if (open == quota) {
#pragma unroll
            for (int u = 0; u < 4; ++u) in[u] |= eq[u];
        } else { // the first `quota` of the open ones
            uint32_t m[4];
            int rank = ties;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                m[u] = __ballot_sync(kFull, eq[u]);
                rank += __popc(m[u] & below);
                ties += __popc(m[u]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                in[u] |= eq[u] && rank < quota;
                rank += eq[u];
            }
        }
        int to = place;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t m = __ballot_sync(kFull, in[u]);
            to += __popc(m & below);
            place += __popc(m);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (in[u]) out[to++] = r.first + i + u;
    }
}

// ------------------------------------------------------------------ the scores
// What a warp scores: blocks 0 .. n - 1 of a request's row of the table from `table` on, for
// the heads of `tokens` tokens, whose rows of q stand in shared memory ([token][heads' power
// of two], rows of D elements and kPad bytes, 0 where there is no head; behind them the
// largest |q| of all; what else is in the last 8 rows goes to columns that nobody reads).  Scores go to shared memory at `keys`, `stride` bytes a token.
struct Scoring {
    const int32_t *table;
    int head, n, tokens, heads_log2;
    uint32_t q, keys, stride;
};

__device__ __forceinline__ uint4 load_shared(uint32_t addr)
{
    uint4 x;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr));
    return x;
}

template <int D, bool ONE>
__device__ __forceinline__ void score_blocks(const SelectArgs &a, const Scoring &s, int first, int step, int lane, float &mag,
                                             int &bad, const __nv_bfloat16 *)
{
    constexpr int NC = D / 32; // 16-byte pieces of a row per lane
    constexpr int ROW = 2 * D + kPad;
    const int g = lane >> 2, c = lane & 3, n = s.n;
    const int per_log2 = 3 - s.heads_log2; // tokens of 8 columns
    const int groups = (s.tokens + (1 << per_log2) - 1) >> per_log2;
    const __nv_bfloat16 *bounds = static_cast<const __nv_bfloat16 *>(a.bounds) + (size_t)s.head * 2 * D + c * 8;
    const size_t block = (size_t)a.num_kv_heads * 2 * D;
    const int tiles = (n + 15) / 16;
    // the lane's entry of a tile's 16 blocks (a row behind the last reads block 0 and is left out)
    auto entry_of = [&](int tile) {
        const int j = tile * 16 + (lane & 15);
        const int e = tile < tiles && j < n ? s.table[j] : 0;
        const bool wrong = e < 0 || e >= a.num_blocks;
        if (wrong) bad = min(bad, j);
        return wrong ? 0 : e;
    };
    const __nv_bfloat16 *r0, *r1;
    uint4 lo[NC][2], hi[NC][2];
    auto load = [&](int i) {
        lo[i][0] = *reinterpret_cast<const uint4 *>(r0 + i * 32);
        lo[i][1] = *reinterpret_cast<const uint4 *>(r1 + i * 32);
        hi[i][0] = *reinterpret_cast<const uint4 *>(r0 + D + i * 32);
        hi[i][1] = *reinterpret_cast<const uint4 *>(r1 + D + i * 32);
    };
    int entry = entry_of(first);
    auto rows_of = [&](int tile) { // and looks up the one after it
        r0 = bounds + (size_t)__shfl_sync(kFull, entry, g) * block;
        r1 = bounds + (size_t)__shfl_sync(kFull, entry, g + 8) * block;
        entry = entry_of(tile + step);
    };
    if (ONE && first < tiles) {
        rows_of(first);
#pragma unroll
        for (int i = 0; i < NC; ++i) load(i);
    }
    for (int tile = first; tile < tiles; tile += step) {
        // One token has one pass of products, behind each of which the next tile's bounds take its place (96 requests:
        // 2.9 us less); with several the registers do not suffice for that.
        const bool more = ONE && tile + step < tiles;
        if (ONE) rows_of(tile + step);
        if (!ONE) {
            rows_of(tile);
#pragma unroll
            for (int i = 0; i < NC; ++i) load(i);
        }
        {   // S, of each head where there are 8 columns at most, else of the largest |q|
            float m[4] = {0.f, 0.f, 0.f, 0.f};
            const uint32_t q = s.q + (uint32_t)(ONE ? g : s.tokens << s.heads_log2) * ROW + c * 16;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const uint4 u = load_shared(q + i * 64);
                mma_bf16_16816(m, most2(hi[i][0].x, lo[i][0].x), most2(hi[i][1].x, lo[i][1].x),
                               most2(hi[i][0].y, lo[i][0].y), most2(hi[i][1].y, lo[i][1].y), abs2(u.x), abs2(u.y));
                mma_bf16_16816(m, most2(hi[i][0].z, lo[i][0].z), most2(hi[i][1].z, lo[i][1].z),
                               most2(hi[i][0].w, lo[i][0].w), most2(hi[i][1].w, lo[i][1].w), abs2(u.z), abs2(u.w));
            }
            // (infinities and NaN do not count: the scores are none either)
            const bool both = ONE && 2 * c + 1 < a.group;
            if (!ONE || 2 * c < a.group) {
                if (tile * 16 + g < n && m[0] < INFINITY) mag = fmaxf(mag, m[0]);
                if (tile * 16 + g + 8 < n && m[2] < INFINITY) mag = fmaxf(mag, m[2]);
            }
            if (both && tile * 16 + g < n && m[1] < INFINITY) mag = fmaxf(mag, m[1]);
            if (both && tile * 16 + g + 8 < n && m[3] < INFINITY) mag = fmaxf(mag, m[3]);
        }
        // GB groups of 8 columns at a time: 2 GB chains of products
        auto group = [&](int grp, auto count) {
            constexpr int GB = decltype(count)::value;
            float sh[GB][4], sl[GB][4];
#pragma unroll
            for (int b = 0; b < GB; ++b)
#pragma unroll
                for (int k = 0; k < 4; ++k) sh[b][k] = sl[b][k] = 0.f;
            const uint32_t q = s.q + (uint32_t)(grp * 8 + g) * ROW + c * 16;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
#pragma unroll
                for (int b = 0; b < GB; ++b) {
                    const uint4 x = load_shared(q + b * 8 * ROW + i * 64);
                    mma_bf16_16816(sh[b], hi[i][0].x, hi[i][1].x, hi[i][0].y, hi[i][1].y, max_nan2(x.x, 0), max_nan2(x.y, 0));
                    mma_bf16_16816(sl[b], lo[i][0].x, lo[i][1].x, lo[i][0].y, lo[i][1].y, min_nan2(x.x, 0), min_nan2(x.y, 0));
                    mma_bf16_16816(sh[b], hi[i][0].z, hi[i][1].z, hi[i][0].w, hi[i][1].w, max_nan2(x.z, 0), max_nan2(x.w, 0));
                    mma_bf16_16816(sl[b], lo[i][0].z, lo[i][1].z, lo[i][0].w, lo[i][1].w, min_nan2(x.z, 0), min_nan2(x.w, 0));
                }
                if (ONE && more) load(i);
            }
            // columns 2c and 2c + 1: heads of the same token unless a token has one column
            const int mask = (1 << s.heads_log2) - 1, h0 = (2 * c) & mask, h1 = (2 * c + 1) & mask;
#pragma unroll
            for (int b = 0; b < GB; ++b)
#pragma unroll
                for (int k = 0; k < 2; ++k) { // rows g and g + 8
                    const int j = tile * 16 + g + 8 * k;
                    float x = h0 < a.group ? sh[b][2 * k] + sl[b][2 * k] : -INFINITY;
                    const float y = h1 < a.group ? sh[b][2 * k + 1] + sl[b][2 * k + 1] : -INFINITY;
                    const int token = ((grp + b) << per_log2) + ((2 * c) >> s.heads_log2);
                    if (s.heads_log2 == 0) {
                        if (j < n && token < s.tokens) cluster_store(s.keys + token * s.stride + 4 * j, __float_as_uint(x));
                        if (j < n && token + 1 < s.tokens) cluster_store(s.keys + (token + 1) * s.stride + 4 * j, __float_as_uint(y));
                        continue;
                    }
                    x = max_nan(x, y);
                    if (s.heads_log2 > 1) x = max_nan(x, __shfl_xor_sync(kFull, x, 1));
                    if (s.heads_log2 > 2) x = max_nan(x, __shfl_xor_sync(kFull, x, 2));
                    if (j < n && token < s.tokens && h0 == 0) cluster_store(s.keys + token * s.stride + 4 * j, __float_as_uint(x));
                }
        };
        int grp = 0;
        if (!ONE)
            for (; grp + 1 < groups; grp += 2) group(grp, std::integral_constant<int, 2>());
        if (grp < groups) group(grp, std::integral_constant<int, 1>());
    }
}

// Tiles of eight tokens or more: a column is a token, and the heads take their turns, so that the largest
// of a token's is found without a word between lanes.  Rows of q [head][tokens rounded up to 8].
template <int D>
__device__ __forceinline__ void score_tokens(const SelectArgs &a, const Scoring &s, int first, int step, int lane, float &mag, int &bad)
{
    constexpr int NC = D / 32; // 16-byte pieces of a row per lane
    constexpr int ROW = 2 * D + kPad;
    const int g = lane >> 2, c = lane & 3, n = s.n, G = a.group;
    const __nv_bfloat16 *bounds = static_cast<const __nv_bfloat16 *>(a.bounds) + (size_t)s.head * 2 * D + c * 8;
    const size_t block = (size_t)a.num_kv_heads * 2 * D;
    const int tiles = (n + 15) / 16;
    const uint32_t of_head = (uint32_t)((s.tokens + 7) & ~7) * ROW; // bytes of a head's rows
    auto entry_of = [&](int tile) {
        const int j = tile * 16 + (lane & 15);
        const int e = tile < tiles && j < n ? s.table[j] : 0;
        const bool wrong = e < 0 || e >= a.num_blocks;
        if (wrong) bad = min(bad, j);
        return wrong ? 0 : e;
    };
    int entry = entry_of(first);
    for (int tile = first; tile < tiles; tile += step) {
        const __nv_bfloat16 *r0 = bounds + (size_t)__shfl_sync(kFull, entry, g) * block;
        const __nv_bfloat16 *r1 = bounds + (size_t)__shfl_sync(kFull, entry, g + 8) * block;
        uint4 lo[NC][2], hi[NC][2];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            lo[i][0] = *reinterpret_cast<const uint4 *>(r0 + i * 32);
            lo[i][1] = *reinterpret_cast<const uint4 *>(r1 + i * 32);
            hi[i][0] = *reinterpret_cast<const uint4 *>(r0 + D + i * 32);
            hi[i][1] = *reinterpret_cast<const uint4 *>(r1 + D + i * 32);
        }
        entry = entry_of(tile + step);
        const int j0 = tile * 16 + g;
        {   // S, of the largest |q|
            float m[4] = {0.f, 0.f, 0.f, 0.f};
            const uint32_t q = s.q + (uint32_t)G * of_head + c * 16;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const uint4 u = load_shared(q + i * 64);
                mma_bf16_16816(m, most2(hi[i][0].x, lo[i][0].x), most2(hi[i][1].x, lo[i][1].x), most2(hi[i][0].y, lo[i][0].y),
                               most2(hi[i][1].y, lo[i][1].y), u.x, u.y);
                mma_bf16_16816(m, most2(hi[i][0].z, lo[i][0].z), most2(hi[i][1].z, lo[i][1].z), most2(hi[i][0].w, lo[i][0].w),
                               most2(hi[i][1].w, lo[i][1].w), u.z, u.w);
            }
            // (infinities and NaN do not count: the scores are none either)
            if (j0 < n && m[0] < INFINITY) mag = fmaxf(mag, m[0]);
            if (j0 + 8 < n && m[2] < INFINITY) mag = fmaxf(mag, m[2]);
        }
        for (int t0 = 0; t0 < s.tokens; t0 += 8) {
            float best[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            // GB heads at a time: 2 GB chains of products
            auto heads = [&](uint32_t q, auto count) {
                constexpr int GB = decltype(count)::value;
                float sh[GB][4], sl[GB][4];
#pragma unroll
                for (int b = 0; b < GB; ++b)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sh[b][k] = sl[b][k] = 0.f;
#pragma unroll
                for (int i = 0; i < NC; ++i)
#pragma unroll
                    for (int b = 0; b < GB; ++b) {
                        const uint4 x = load_shared(q + b * of_head + i * 64);
                        mma_bf16_16816(sh[b], hi[i][0].x, hi[i][1].x, hi[i][0].y, hi[i][1].y, max_nan2(x.x, 0), max_nan2(x.y, 0));
                        mma_bf16_16816(sl[b], lo[i][0].x, lo[i][1].x, lo[i][0].y, lo[i][1].y, min_nan2(x.x, 0), min_nan2(x.y, 0));
                        mma_bf16_16816(sh[b], hi[i][0].z, hi[i][1].z, hi[i][0].w, hi[i][1].w, max_nan2(x.z, 0), max_nan2(x.w, 0));
                        mma_bf16_16816(sl[b], lo[i][0].z, lo[i][1].z, lo[i][0].w, lo[i][1].w, min_nan2(x.z, 0), min_nan2(x.w, 0));
                    }
#pragma unroll
                for (int b = 0; b < GB; ++b)
#pragma unroll
                    for (int k = 0; k < 4; ++k) best[k] = max_nan(best[k], sh[b][k] + sl[b][k]);
            };
            uint32_t q = s.q + (uint32_t)(t0 + g) * ROW + c * 16;
            int h = 0;
            for (; h + 1 < G; h += 2, q += 2 * of_head) heads(q, std::integral_constant<int, 2>());
            if (h < G) heads(q, std::integral_constant<int, 1>());
            // blocks g and g + 8 of columns 2c and 2c + 1
            const uint32_t to = s.keys + (t0 + 2 * c) * s.stride + 4 * j0;
            if (t0 + 2 * c < s.tokens) {
                if (j0 < n) cluster_store(to, __float_as_uint(best[0]));
                if (j0 + 8 < n) cluster_store(to + 32, __float_as_uint(best[2]));
            }
            if (t0 + 2 * c + 1 < s.tokens) {
                if (j0 < n) cluster_store(to + s.stride, __float_as_uint(best[1]));
                if (j0 + 8 < n) cluster_store(to + s.stride + 32, __float_as_uint(best[3]));
            }
        }
    }
}

// fp32: a warp scores kBatch blocks at a time, its lanes share the channels.
template <int D, int kBatch>
__device__ __forceinline__ void score_blocks_f32(const SelectArgs &a, const Scoring &s, int first, int step, int lane, float &mag,
                                             int &bad)
{
    constexpr int E = D / 32;
    constexpr int ROW = 4 * D + kPad;
    using Vec = typename std::conditional<E == 4, float4, float2>::type;
    const int n = s.n;
    const float *bounds = static_cast<const float *>(a.bounds) + (size_t)s.head * 2 * D + lane * E;
    const size_t block = (size_t)a.num_kv_heads * 2 * D;
    const int tiles = (n + kBatch - 1) / kBatch;
    auto row_of = [&](int r, float(&x)[E]) {
        const uint32_t at = s.q + (uint32_t)r * ROW + lane * E * 4;
        if constexpr (E == 4)
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(at));
        else
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x[0]), "=f"(x[1]) : "r"(at));
    };
    for (int tile = first; tile < tiles; tile += step) {
        float lo[kBatch][E], hi[kBatch][E];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int j = tile * kBatch + b;
            int e = j < n ? s.table[j] : 0;
            if (e < 0 || e >= a.num_blocks) {
                bad = min(bad, j);
                e = 0;
            }
            *reinterpret_cast<Vec *>(lo[b]) = *reinterpret_cast<const Vec *>(bounds + (size_t)e * block);
            *reinterpret_cast<Vec *>(hi[b]) = *reinterpret_cast<const Vec *>(bounds + (size_t)e * block + D);
        }
        float u[E];
        row_of(s.tokens << s.heads_log2, u);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) m = fmaf(u[i], fmaxf(fabsf(lo[b][i]), fabsf(hi[b][i])), m);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(kFull, m, o);
            if (tile * kBatch + b < n && m < INFINITY) mag = fmaxf(mag, m);
        }
        for (int t = 0; t < s.tokens; ++t) {
            float best = -INFINITY;
            for (int g = 0; g < a.group; ++g) {
                float x[E], p[kBatch];
                row_of((t << s.heads_log2) + g, x);
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    p[b] = 0.f;
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        p[b] = fmaf(max_nan(x[i], 0.f), hi[b][i], fmaf(min_nan(x[i], 0.f), lo[b][i], p[b]));
                }
                // the kBatch sums together: 32 / kBatch neighbouring lanes end up with one of them
                int mask = 16;
#pragma unroll
                for (int half = kBatch / 2; half >= 1; half /= 2, mask /= 2)
#pragma unroll
                    for (int i = 0; i < half; ++i) {
                        const float give = lane & mask ? p[i] : p[i + half], keep = lane & mask ? p[i + half] : p[i];
                        p[i] = keep + __shfl_xor_sync(kFull, give, mask);
                    }
                float z = p[0];
#pragma unroll
                for (; mask >= 1; mask /= 2) z += __shfl_xor_sync(kFull, z, mask);
                best = max_nan(best, z);
            }
            const int j = tile * kBatch + lane / (32 / kBatch); // these lanes' block
            if (j < n && lane % (32 / kBatch) == 0) cluster_store(s.keys + t * s.stride + 4 * j, __float_as_uint(best));
        }
    }
}

// Eight blocks at a time (8 KB in flight a warp at D = 128) for a token alone where every warp has two
// such, else four (and three CTAs an SM instead of two).
template <int D, bool ONE>
__device__ __forceinline__ void score_blocks(const SelectArgs &a, const Scoring &s, int first, int step, int lane, float &mag,
                                             int &bad, const float *)
{
    if (ONE && s.n >= 16 * step)
        score_blocks_f32<D, 8>(a, s, first, step, lane, mag, bad);
    else
        score_blocks_f32<D, 4>(a, s, first, step, lane, mag, bad);
}

// Tile `unit` of the packed queries: rows [first, first + count) of one request, `tile` of them but at
// its end; count 0: none.  Request r, with rows c0 to c1, has the tiles c0 / tile + r up to
// c1 / tile + r: one more than it may need, and found without the sums of those before.
struct TileRows {
    int first, count;
    QueryRow at; // the first of them
};
__device__ __forceinline__ TileRows tile_rows(const SelectArgs &a, int unit, int tile, int lane)
{
    TileRows t{0, 0, {0, -(1 << 30), false, 0}};
    const int c_first = a.cu_q[0];
    const int r = find_last([&](int i) { return (long long)a.cu_q[i] / tile + i; }, a.batch, unit, lane);
    if (c_first != 0) { // no row has a request: all are refused
        t.first = (int)min((long long)unit * tile, (long long)a.total_q);
        t.count = (int)min(tile, a.total_q - t.first);
        t.at.err = PA_DEVERR_BAD_CU;
        return t;
    }
    if (r < 0 || r >= a.batch) return t;
    const int c0 = a.cu_q[r], c1 = a.cu_q[r + 1], end = min(c1, a.total_q);
    t.at = request_row(a, r, 0);
    const long long first = c0 + (long long)(unit - (c0 / tile + r)) * tile;
    if (c0 < 0 || first < c0 || first >= end) return t;
    t.first = (int)first;
    t.count = min(tile, end - t.first);
    if (t.at.pos > -(1 << 30)) t.at.pos -= c1 - 1 - t.first;
    return t;
}

struct Shared {
    uint32_t mag; // S, the bits of a float >= 0
    int bad;      // the first scored block whose table entry is none
};

// TILE = 1: W warps a row, or (W = kWarps) a cluster of `ctas`.  Otherwise up to `tile` tokens of one
// request, scored by all warps, a warp choosing for each (W = 1).
template <typename T, int D, int TILE, int W>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 && TILE > 1 ? 3 : 2) select_kernel(const SelectArgs a, int ctas, int tile, int heads_log2)
{
    constexpr int SW = TILE == 1 ? W : kWarps; // warps that score together
    constexpr int ROW = (int)sizeof(T) * D + kPad;
    constexpr bool WIDE = sizeof(T) == 2 && TILE == kTile;
    extern __shared__ __align__(16) uint32_t smem[]; // of each SW warps: keys [tile][max_blocks_per_seq, a multiple of 4], then the rows of q
    __shared__ Shared shared[kWarps / SW];
    __shared__ Choice<W> choice[kWarps / W];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = warp / SW, st = tid % (32 * SW); // the warps that score together, the thread of them
    Shared &sh = shared[group];
    const bool cluster = ctas > 1;
    const int rank = cluster ? (int)cluster_rank() : 0;
    if (st == 0) {
        sh.mag = 0;
        sh.bad = INT_MAX;
    }
    __syncwarp();
    grid_dep_trigger();
    if (cluster) cluster_arrive();
    grid_dep_wait();
    check_lengths(a);
    __syncwarp();

    const int unit = (int)(blockIdx.x / ctas) * (kWarps / SW) + group;
    if (SW < kWarps && unit >= (long long)a.total_q * a.num_kv_heads) return;
    const int h = unit % a.num_kv_heads; // heads of a tile side by side
    int t = unit / a.num_kv_heads, count = 1;
    QueryRow at;
    if (TILE == 1) {
        at = query_row(a, t, lane);
    } else {
        const TileRows r = tile_rows(a, t, tile, lane);
        if (r.count == 0) {
            if (cluster) cluster_wait();
            return;
        }
        t = r.first;
        count = r.count;
        at = r.at;
    }
    const int cap = a.max_blocks_per_seq, row_keys = (cap + 3) & ~3, need = a.top_k - a.first - a.last;
    uint32_t *keys = smem + (SW < kWarps ? (size_t)group * (row_keys + 9 * ROW / 4) : 0);
    const int last_seen = at.pos + count - 1 < 0 ? 0 : (at.pos + count - 1) / a.block_size + 1; // by the last token
    const bool nothing = at.skip || last_seen <= a.top_k || need == 0; // to be scored
    if (nothing) {
        if (cluster) cluster_wait();
    } else {
        uint8_t *q_rows = reinterpret_cast<uint8_t *>(keys + (size_t)tile * row_keys);
        const T *q = static_cast<const T *>(a.q) + ((size_t)t * a.num_heads + (size_t)h * a.group) * D;
        Scoring s;
        s.table = a.block_table + (size_t)at.req * cap + a.first;
        s.head = h;
        s.n = last_seen - a.first - a.last;
        s.tokens = count;
        s.heads_log2 = heads_log2;
        s.q = smem_u32(q_rows);
        s.keys = cluster_addr(keys, 0);
        s.stride = row_keys * 4;
        // rows of q, 16 bytes a thread; then the largest |q| of each channel
        constexpr int PIECES = (int)sizeof(T) * D / 16;
        const int wide = (count + 7) & ~7, rows = WIDE ? a.group * wide : count << heads_log2;
        for (int i = st; i < rows * PIECES; i += 32 * SW) {
            const int r = i / PIECES, p = i % PIECES;
            const int g = WIDE ? r / wide : r & ((1 << heads_log2) - 1), tk = WIDE ? r - g * wide : r >> heads_log2;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (g < a.group && tk < count) x = reinterpret_cast<const uint4 *>(q + ((size_t)tk * a.num_heads + g) * D)[p];
            *reinterpret_cast<uint4 *>(q_rows + (size_t)r * ROW + p * 16) = x;
        }
        choice_sync<SW>();
        if (TILE > 1 || sizeof(T) == 4) {
            T *env = reinterpret_cast<T *>(q_rows + (size_t)rows * ROW);
            for (int d = st; d < D; d += 32 * SW) {
                float u = 0.f;
                for (int r = 0; r < rows; ++r) { // (a head with an infinity has no finite score)
                    const float x = fabsf(to_float(reinterpret_cast<const T *>(q_rows + (size_t)r * ROW)[d]));
                    if (x < INFINITY) u = fmaxf(u, x);
                }
                if constexpr (sizeof(T) == 2)
                    env[d] = __float2bfloat16_ru(u * (1.f / kShrink));
                else
                    env[d] = __fmul_ru(u, 1.f / kShrink);
            }
            choice_sync<SW>();
        }
        if (cluster) cluster_wait(); // the first CTA's shared memory is there
        float mag = 0.f;
        int bad = INT_MAX;
        if constexpr (WIDE)
            score_tokens<D>(a, s, rank * SW + warp % SW, ctas * SW, lane, mag, bad);
        else
            score_blocks<D, TILE == 1>(a, s, rank * SW + warp % SW, ctas * SW, lane, mag, bad, q);
        const uint32_t most = __reduce_max_sync(kFull, __float_as_uint(mag));
        bad = __reduce_min_sync(kFull, bad);
        if (lane == 0) {
            cluster_max(cluster_addr(&sh.mag, 0), most);
            if (bad != INT_MAX) cluster_min(cluster_addr(&sh.bad, 0), (uint32_t)bad);
        }
        __syncwarp();
        if (cluster) {
            cluster_arrive();
            cluster_wait();
        } else {
            choice_sync<SW>();
        }
    }
    if (rank != 0 || at.skip) return;
    const int bad_block = nothing ? INT_MAX : sh.bad;
    if (st == 0 && (at.err || bad_block != INT_MAX)) flag_error(a.dev_err, at.err ? at.err : PA_DEVERR_BAD_BLOCK);
    // the tokens' outputs, by W warps each
    for (int i = TILE == 1 ? 0 : warp; i < count; i += kWarps) {
        const int seen = at.pos + i < 0 ? 0 : (at.pos + i) / a.block_size + 1;
        int32_t *out = a.selected + ((size_t)(t + i) * a.num_kv_heads + h) * a.top_k;
        const int wt = tid % (32 * W);
        if (seen <= a.top_k) {
            for (int k = wt; k < a.top_k; k += 32 * W) out[k] = k < seen ? k : -1;
            continue;
        }
        const int n = seen - a.first - a.last;
        const bool failed = bad_block < n; // (not for entries that only later tokens need)
        for (int k = wt; k < a.first + a.last; k += 32 * W) {
            const int to = k < a.first ? k : k + need;
            out[to] = failed ? -1 : k < a.first ? k : seen - a.top_k + to;
        }
        if (failed)
            for (int k = wt; k < need; k += 32 * W) out[a.first + k] = -1;
        if (failed || need == 0) continue;
        Row<T> r;
        r.q = static_cast<const T *>(a.q) + ((size_t)(t + i) * a.num_heads + (size_t)h * a.group) * D;
        r.bounds = static_cast<const T *>(a.bounds) + (size_t)h * 2 * D;
        r.table = a.block_table + (size_t)at.req * cap + a.first;
        r.n = n;
        r.first = a.first;
        r.need = need;
        // 2 E, and the rounding of S
        r.width = (sizeof(T) == 2 ? (2.5f * (D / 16) + 0.5f) * 0x1.02p-21f : (D / 16 + 6) * 0x1.02p-23f) * __uint_as_float(sh.mag) *
                  (TILE > 1 || sizeof(T) == 4 ? kShrink : 1.f);
        choose<T, D, W>(keys + (size_t)i * row_keys, r, out + a.first, a, 1 << heads_log2, choice[warp / W], wt);
    }
}

template <typename T, int D, int TILE, int W>
int launch(const SelectArgs &a, int ctas, int tile, int heads_log2, size_t smem, cudaStream_t s)
{
    static int raised[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PA_ERR_DEVICE;
    if (!__atomic_load_n(&raised[dev], __ATOMIC_ACQUIRE)) {
        cudaError_t e = cudaFuncSetAttribute(select_kernel<T, D, TILE, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kSelectMaxBlocks * 4 + 16 + (kGroup + 1) * ((int)sizeof(T) * D + kPad));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(select_kernel<T, D, TILE, W>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return launch_status(e);
        __atomic_store_n(&raised[dev], 1, __ATOMIC_RELEASE);
    }
    // tiles do not pass the end of a request: one more for each
    const long long tiles = TILE == 1 ? a.total_q : a.total_q / tile + (long long)a.batch;
    const int per_cta = TILE == 1 ? kWarps / W : 1;
    const long long grid = (tiles * a.num_kv_heads + per_cta - 1) / per_cta * ctas;
    if (grid * per_cta >= 1ll << 31) return PA_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
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
    return launch_status(cudaLaunchKernelEx(&cfg, select_kernel<T, D, TILE, W>, a, ctas, tile, heads_log2));
}

template <typename T, int D>
int launch_tile(const SelectArgs &a, cudaStream_t s)
{
    const long long rows = (long long)a.total_q * a.num_kv_heads;
    const int heads_log2 = a.group > 4 ? 3 : a.group > 2 ? 2 : a.group > 1 ? 1 : 0;
    const size_t row = sizeof(T) * D + kPad;
    auto smem_of = [&](int tile) { return (size_t)tile * ((a.max_blocks_per_seq + 3) & ~3) * 4 + ((size_t)(((tile << heads_log2) + 7) & ~7) + 1) * row; };
    // Chunks: tiles of as many tokens as requests have on average, and shared memory holds twice an SM.
    int tile = 1;
    if (a.cu_q != nullptr)
        while (tile < kTile && smem_of(2 * tile) <= 100 * 1024 && a.total_q >= 2ll * tile * a.batch) tile *= 2;
    auto units_of = [&](int t) { return t == 1 ? rows : (a.total_q / t + (long long)a.batch) * a.num_kv_heads; };
    const long long fill = 2ll * num_sms();
    // .. 16 only where there are several for every place: they read the bounds half as often, but take longer
    // (8 kv heads, 565 tokens of 5 requests: 48.7 us, with 8 45.2; 4096 of 2: 248 and 288).
    if (tile == kTile && units_of(tile) < 2 * fill) tile /= 2;
    // Few rows or tiles: a cluster of CTAs each, as many as are resident at a time (two an SM)
    // while each warp has a tile of 16 blocks.
    const long long fit = std::min<long long>(fill / units_of(tile), (a.max_blocks_per_seq + 16 * kWarps - 1) / (16 * kWarps));
    const int ctas = fit <= 1 ? 1 : fit <= 8 ? (int)fit : fit >= 16 ? 16 : 8; // (9 to 15 are slower than 8)
    if constexpr (sizeof(T) == 2)
        if (tile > 1 && tile < 8) return launch<T, D, 4, 1>(a, ctas, tile, heads_log2, smem_of(tile), s);
    if (tile > 1) return launch<T, D, kTile, 1>(a, ctas, tile, heads_log2, smem_of(tile), s);
    // Many rows: fewer warps each, which wait less for one another, while there are enough to fill two thirds of the
    // places and none has more than 14 tiles of 16 blocks (fp32: 8).  8 warps, 4, 2, 1, us, 8 kv heads of 128 in bf16: 1000
    // requests of up to 94 blocks 166, 100, 65, 52; 200 of up to 562 64, 57, 60, 72; 96 of up to 2034 86, 94, 122, 372;
    // 200 in fp32 118, 123, 142, 206.
    int warps = kWarps;
    while (ctas == 1 && warps > 1 && a.max_blocks_per_seq <= (sizeof(T) == 2 ? 14 : 8) * 16 * (warps / 2) && 3 * rows * (warps / 2) >= 2 * fill * kWarps &&
           smem_of(1) * (kWarps / (warps / 2)) <= 100 * 1024)
        warps /= 2;
    const size_t smem = smem_of(1) * (kWarps / warps);
    if (warps == 1) return launch<T, D, 1, 1>(a, 1, 1, heads_log2, smem, s);
    if (warps == 2) return launch<T, D, 1, 2>(a, 1, 1, heads_log2, smem, s);
    if (warps == 4) return launch<T, D, 1, 4>(a, 1, 1, heads_log2, smem, s);
    return launch<T, D, 1, kWarps>(a, ctas, 1, heads_log2, smem, s);
}

}  // namespace

int select_launch(const SelectArgs &a, int head_dim, bool f32, cudaStream_t s)
{
    if (f32) return head_dim == 64 ? launch_tile<float, 64>(a, s) : launch_tile<float, 128>(a, s);
    return head_dim == 64 ? launch_tile<__nv_bfloat16, 64>(a, s) : launch_tile<__nv_bfloat16, 128>(a, s);
}

}  // namespace pa
