// pa_rotary and pa_cache_append_rotary: queries and keys turned by their
// positions, and a step's keys and values put into the paged cache on the way.
//
// Pair i of a row's rotary_dim / 2 pairs (x, y) is turned by the angle of its
// axis' position, whose cosine c and sine s are a row of a table:
//   x' = x c - y s,  y' = y c + x s      (fp32, rounded once to the type)
// Dims behind rotary_dim pass through.  Bound by memory: a row is read and
// written once, with a few operations an element.
//
// Layout.  A lane holds two 16-byte-element groups ("chunks" of 8 elements) of a
// row: the 8 pairs 8c .. 8c + 7.  Split halves: chunks c and c + R / 16;
// neighbouring pairs: chunks 2c and 2c + 1.  Either way the lane's cosines and
// sines are the same 8 columns, both elements of a pair are its own (no
// shuffles), and head_dim / 16 lanes cover the row with 16-byte accesses.
//
// The append keeps the bounds of each block's keys (least and largest value of
// each channel) when asked.  Tokens of one block follow one another, so a run of
// them is one warp's work for one head: the lanes' groups take its tokens in
// turn, keep the extrema of the rounded keys in registers and join them by
// shuffles; a run that begins inside a block widens the bounds that are there.
// No atomics: the result does not depend on any order.
//
// Measured (one GB300, bf16, 32 + 8 heads of 128): 32761 tokens on three axes 99.5 us for 686 MB, 6.9 TB/s, a plain copy's
// rate (part of the outputs stays in L2: 619 MB of DRAM traffic); the append of 33116 tokens with bounds
// 130 us for 840 MB, 6.4 TB/s; a decode step of 64 tokens 3.5 us, one token 1.9.
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
// Heads of a thread group: their loads are in flight together, 32 bytes each and lane (fp32: 64).
template <typename T>
constexpr int kHeadsOf = 8 / (int)sizeof(T);
constexpr int kMaxAxes = 4;

enum Mode { kRotary, kAppend, kAppendBounds };

// Two chunks of 8 elements.
template <typename T>
struct Chunks {
    uint4 v[2][sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Chunks<T> load_chunks(const T *row, int c0, int c1)
{
    Chunks<T> x;
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j) {
        x.v[0][j] = reinterpret_cast<const uint4 *>(row + c0 * 8)[j];
        x.v[1][j] = reinterpret_cast<const uint4 *>(row + c1 * 8)[j];
    }
    return x;
}

template <typename T>
__device__ __forceinline__ void store_chunks(T *row, int c0, int c1, const Chunks<T> &x)
{
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j) {
        reinterpret_cast<uint4 *>(row + c0 * 8)[j] = x.v[0][j];
        reinterpret_cast<uint4 *>(row + c1 * 8)[j] = x.v[1][j];
    }
}

__device__ __forceinline__ void unpack(const uint4 (&v)[1], float (&x)[8])
{
    const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4 (&v)[2], float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x[4 * i] = __uint_as_float(v[i].x);
        x[4 * i + 1] = __uint_as_float(v[i].y);
        x[4 * i + 2] = __uint_as_float(v[i].z);
        x[4 * i + 3] = __uint_as_float(v[i].w);
    }
}
__device__ __forceinline__ void pack(uint4 (&v)[1], const float (&x)[8])
{
    v[0] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void pack(uint4 (&v)[2], const float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 2; ++i)
        v[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                          __float_as_uint(x[4 * i + 3]));
}

// Cosines and sines of a lane's 8 pairs.
struct Angles {
    float c[8], s[8];
};

// x and y of a pair in either style: with split halves chunk 0 holds the x and
// chunk 1 the y of the 8 pairs, otherwise the 16 elements are the pairs in order.
template <typename T, bool PAIRS>
__device__ __forceinline__ void turn(Chunks<T> &x, const Angles &a)
{
    float e[2][8];
    unpack(x.v[0], e[0]);
    unpack(x.v[1], e[1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float &p = PAIRS ? e[i / 4][2 * (i % 4)] : e[0][i];
        float &r = PAIRS ? e[i / 4][2 * (i % 4) + 1] : e[1][i];
        const float t = fmaf(p, a.c[i], -(r * a.s[i]));
        r = fmaf(r, a.c[i], p * a.s[i]);
        p = t;
    }
    pack(x.v[0], e[0]);
    pack(x.v[1], e[1]);
}

// Bounds: least and largest of the elements; a NaN stays one.
__device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b, __nv_bfloat16)
{
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t largest(uint32_t a, uint32_t b, __nv_bfloat16)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b, float)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
    return __float_as_uint(r);
}
__device__ __forceinline__ uint32_t largest(uint32_t a, uint32_t b, float)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
    return __float_as_uint(r);
}

template <typename T>
struct Bounds {
    uint32_t lo[4 * sizeof(T)], hi[4 * sizeof(T)]; // the words of two chunks

    __device__ __forceinline__ void clear()
    {
        const uint32_t inf = sizeof(T) == 2 ? 0x7f807f80u : 0x7f800000u;
        const uint32_t sign = sizeof(T) == 2 ? 0x80008000u : 0x80000000u;
#pragma unroll
        for (int i = 0; i < 4 * (int)sizeof(T); ++i) {
            lo[i] = inf;
            hi[i] = inf | sign;
        }
    }
    __device__ __forceinline__ void add(const Chunks<T> &l, const Chunks<T> &h)
    {
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int j = 0; j < (int)sizeof(T) / 2; ++j) {
                const uint4 a = l.v[p][j], b = h.v[p][j];
                uint32_t *lw = lo + (p * (int)sizeof(T) / 2 + j) * 4, *hw = hi + (p * (int)sizeof(T) / 2 + j) * 4;
                lw[0] = least(lw[0], a.x, T());
                lw[1] = least(lw[1], a.y, T());
                lw[2] = least(lw[2], a.z, T());
                lw[3] = least(lw[3], a.w, T());
                hw[0] = largest(hw[0], b.x, T());
                hw[1] = largest(hw[1], b.y, T());
                hw[2] = largest(hw[2], b.z, T());
                hw[3] = largest(hw[3], b.w, T());
            }
    }
    __device__ __forceinline__ void join(int lanes) // with the lane `lanes` away
    {
#pragma unroll
        for (int i = 0; i < 4 * (int)sizeof(T); ++i) {
            lo[i] = least(lo[i], __shfl_xor_sync(kFull, lo[i], lanes), T());
            hi[i] = largest(hi[i], __shfl_xor_sync(kFull, hi[i], lanes), T());
        }
    }
    __device__ __forceinline__ void store(T *row_lo, T *row_hi, int c0, int c1) const
    {
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int j = 0; j < (int)sizeof(T) / 2; ++j) {
                const uint32_t *lw = lo + (p * (int)sizeof(T) / 2 + j) * 4, *hw = hi + (p * (int)sizeof(T) / 2 + j) * 4;
                const int c = (p ? c1 : c0) * 8;
                reinterpret_cast<uint4 *>(row_lo + c)[j] = make_uint4(lw[0], lw[1], lw[2], lw[3]);
                reinterpret_cast<uint4 *>(row_hi + c)[j] = make_uint4(hw[0], hw[1], hw[2], hw[3]);
            }
    }
};

// What a lane does, whatever the token: its chunks, whether it turns them, the
// axes of its 8 pairs (two bits each).
struct Lane {
    int c, c0, c1;
    bool turns;
    uint32_t axes;
};

template <int D, bool PAIRS>
__device__ __forceinline__ Lane lane_of(const RotaryArgs &a, int lane)
{
    Lane l;
    const int rc = a.rotary_dim / 16;
    l.c = lane % (D / 16);
    l.turns = l.c < rc;
    const bool halves = !PAIRS && l.turns;
    l.c0 = halves ? l.c : 2 * l.c;
    l.c1 = halves ? rc + l.c : 2 * l.c + 1;
    l.axes = (uint32_t)(a.pair_axis[l.c / 4] >> (16 * (l.c % 4))) & 0xffffu;
    return l;
}

// Positions of a token on all axes; false when one is outside the table.
__device__ __forceinline__ bool load_positions(const RotaryArgs &a, int axes, int t, int (&pos)[kMaxAxes])
{
    bool ok = true;
#pragma unroll
    for (int i = 0; i < kMaxAxes; ++i) {
        pos[i] = 0;
        if (i < axes) {
            pos[i] = a.positions[(size_t)i * a.tokens + t];
            ok &= pos[i] >= 0 && pos[i] < a.max_position;
        }
    }
    return ok;
}

__device__ __forceinline__ void load_angles(const RotaryArgs &a, const Lane &l, const int (&pos)[kMaxAxes], Angles &w)
{
    const int half = a.rotary_dim / 2;
    const uint32_t first = l.axes & 3u;
    if (l.axes == first * 0x5555u) { // one axis: the columns of one row, 16 bytes at a time
        const int p = first == 0 ? pos[0] : first == 1 ? pos[1] : first == 2 ? pos[2] : pos[3];
        const float *row = a.cos_sin + (size_t)p * a.rotary_dim + 8 * l.c;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 c = reinterpret_cast<const float4 *>(row)[j];
            const float4 s = reinterpret_cast<const float4 *>(row + half)[j];
            w.c[4 * j] = c.x, w.c[4 * j + 1] = c.y, w.c[4 * j + 2] = c.z, w.c[4 * j + 3] = c.w;
            w.s[4 * j] = s.x, w.s[4 * j + 1] = s.y, w.s[4 * j + 2] = s.z, w.s[4 * j + 3] = s.w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t ax = (l.axes >> (2 * i)) & 3u;
        const int p = ax == 0 ? pos[0] : ax == 1 ? pos[1] : ax == 2 ? pos[2] : pos[3];
        const float *at = a.cos_sin + (size_t)p * a.rotary_dim + 8 * l.c + i;
        w.c[i] = *at;
        w.s[i] = at[half];
    }
}

// kHeadsOf heads of one token: turned (TURN) or copied.  `zero` writes zeros.
template <typename T, int D, bool PAIRS, bool TURN>
__device__ __forceinline__ void move_heads(const T *src, T *dst, int heads, const Lane &l, const Angles &w, bool zero)
{
    constexpr int N = kHeadsOf<T>;
    Chunks<T> x[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < heads) x[i] = load_chunks(src + i * D, l.c0, l.c1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (i >= heads) break;
        if (TURN && l.turns) turn<T, PAIRS>(x[i], w);
        if (zero) x[i] = Chunks<T>{};
        store_chunks(dst + i * D, l.c0, l.c1, x[i]);
    }
}

// Thread groups of D / 16 lanes take (token, kHeadsOf heads): first the queries',
// then (kRotary, kAppend) the keys'.  kAppendBounds: `run_ctas` CTAs, spread among the
// others (their chains of dependent loads need company), take the runs of tokens of one block
// that begin in TILE tokens, a warp one head of them.
template <typename T, int D, bool PAIRS, Mode MODE, int TILE>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) rotary_kernel(const RotaryArgs a, int axes, unsigned run_ctas)
{
    constexpr int LPR = D / 16, kHeads = kHeadsOf<T>;
    grid_dep_trigger();
    grid_dep_wait();
    const Lane l = lane_of<D, PAIRS>(a, threadIdx.x);
    const int hq = a.num_heads, hkv = a.num_kv_heads;
    const T *k = static_cast<const T *>(a.k), *v = static_cast<const T *>(a.v);
    T *kc = static_cast<T *>(a.k_out), *vc = static_cast<T *>(a.v_out);
    Angles w{};
    int pos[kMaxAxes];

    const unsigned every = MODE == kAppendBounds ? gridDim.x / run_ctas : 1, turns = blockIdx.x / every;
    const bool runs = MODE == kAppendBounds && turns * every == blockIdx.x && turns < run_ctas;
    if (!runs) {
        const int gq = (hq + kHeads - 1) / kHeads, gk = MODE == kAppendBounds ? 0 : (hkv + kHeads - 1) / kHeads;
        const unsigned cta = MODE == kAppendBounds ? blockIdx.x - min(turns + 1, run_ctas) : blockIdx.x;
        const long long item = (long long)cta * (kThreads / LPR) + threadIdx.x / LPR;
        const long long nq = (long long)a.tokens * gq;
        const bool is_q = item < nq;
        const long long it = is_q ? item : item - nq;
        const int per = is_q ? gq : gk;
        if (per == 0 || it >= (long long)a.tokens * per) return;
        const int t = (int)(it / per), h = (int)(it % per) * kHeads;
        int slot = 0;
        if (MODE != kRotary) {
            slot = a.slot_map[t];
            if (slot < 0) return; // padding: nothing of the row is read or written
        }
        const bool here = MODE == kRotary || slot / a.block_size < a.num_blocks;
        const bool ok = load_positions(a, axes, t, pos);
        if (l.c == 0 && h == 0 && !(here && ok))
            flag_error(a.dev_err, (here ? 0 : PA_DEVERR_BAD_BLOCK) | (ok ? 0 : PA_DEVERR_OVERFLOW));
        if (ok && l.turns) load_angles(a, l, pos, w);
        if (is_q) {
            const T *src = static_cast<const T *>(a.q) + t * a.q_stride + h * D;
            T *dst = static_cast<T *>(a.q_out) + t * a.q_out_stride + h * D;
            move_heads<T, D, PAIRS, true>(src, dst, min(hq - h, kHeads), l, w, !(here && ok));
        } else if (MODE == kRotary) {
            move_heads<T, D, PAIRS, true>(k + t * a.k_stride + h * D, kc + t * a.k_out_stride + h * D,
                                          min(hkv - h, kHeads), l, w, !ok);
        } else if (here && ok) {
            const long long at = ((long long)slot * hkv + h) * D;
            move_heads<T, D, PAIRS, true>(k + t * a.k_stride + h * D, kc + at, min(hkv - h, kHeads), l, w, false);
            move_heads<T, D, PAIRS, false>(v + t * a.v_stride + h * D, vc + at, min(hkv - h, kHeads), l, w, false);
        }
        return;
    }

    if constexpr (MODE == kAppendBounds) {
        constexpr int NG = 32 / LPR; // tokens of a warp at once
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = lane / LPR;
        const int bs = a.block_size;
        // a warp has one head of the runs that begin in TILE tokens
        const long long unit = (long long)turns * (kThreads / 32) + warp;
        const int h = (int)(unit % hkv);
        if (unit / hkv * TILE >= a.tokens) return;
        const int t0 = (int)(unit / hkv) * TILE;
        // a run begins where the block differs from the row's before
        int mine = -1, before = -1;
        if (lane < TILE && t0 + lane < a.tokens) {
            mine = a.slot_map[t0 + lane];
            before = t0 + lane > 0 ? a.slot_map[t0 + lane - 1] : -1;
        }
        const bool lead = mine >= 0 && (before < 0 || before / bs != mine / bs);
        for (uint32_t leads = __ballot_sync(kFull, lead); leads; leads &= leads - 1) {
            const int t1 = t0 + __ffs(leads) - 1;
            const int slot1 = __shfl_sync(kFull, mine, t1 - t0);
            const int block = slot1 / bs;
            const bool here = block < a.num_blocks;
            T *blo = static_cast<T *>(a.bounds) + ((size_t)block * hkv + h) * 2 * D, *bhi = blo + D;
            Bounds<T> b;
            b.clear();
            if (here && slot1 % bs != 0 && group == 0) // the block has keys already
                b.add(load_chunks(blo, l.c0, l.c1), load_chunks(bhi, l.c0, l.c1));
            bool any = false;
            for (int base = t1;; base += 32) { // 32 tokens of the run at a time
                int s = -1;
                bool ok = false;
                if (base + lane < a.tokens) {
                    s = a.slot_map[base + lane];
                    ok = load_positions(a, axes, base + lane, pos);
                }
                const uint32_t others = ~__ballot_sync(kFull, s >= 0 && s / bs == block);
                const int len = others ? __ffs(others) - 1 : 32;
                if (h == 0 && lane < len && !(here && ok))
                    flag_error(a.dev_err, (here ? 0 : PA_DEVERR_BAD_BLOCK) | (ok ? 0 : PA_DEVERR_OVERFLOW));
                for (int r0 = 0; r0 < len; r0 += NG) {
                    const int r = r0 + group, from = min(r, 31);
                    const int sl = __shfl_sync(kFull, s, from);
                    const bool good = __shfl_sync(kFull, (int)ok, from) && r < len && here;
                    int p[kMaxAxes];
#pragma unroll
                    for (int i = 0; i < kMaxAxes; ++i) p[i] = i < axes ? __shfl_sync(kFull, pos[i], from) : 0;
                    if (!good) continue;
                    const long long t = base + r, at = ((long long)sl * hkv + h) * D;
                    Chunks<T> x = load_chunks(k + t * a.k_stride + h * D, l.c0, l.c1);
                    const Chunks<T> y = load_chunks(v + t * a.v_stride + h * D, l.c0, l.c1);
                    if (l.turns) {
                        load_angles(a, l, p, w);
                        turn<T, PAIRS>(x, w);
                    }
                    store_chunks(kc + at, l.c0, l.c1, x);
                    store_chunks(vc + at, l.c0, l.c1, y);
                    b.add(x, x);
                    any = true;
                }
                if (len < 32) break;
            }
            if (__any_sync(kFull, any)) {
#pragma unroll
                for (int o = LPR; o < 32; o <<= 1) b.join(o);
                if (group == 0) b.store(blo, bhi, l.c0, l.c1);
            }
        }
    }
}

template <typename T, int D, bool PAIRS, Mode MODE, int TILE>
int launch(const RotaryArgs &a, int axes, long long run_ctas, long long ctas, cudaStream_t s)
{
    if (ctas >= 1ll << 31) return PA_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, rotary_kernel<T, D, PAIRS, MODE, TILE>, a, axes, (unsigned)run_ctas));
}

template <typename T, int D, bool PAIRS>
int launch_mode(const RotaryArgs &a, int axes, bool append, cudaStream_t s)
{
    constexpr int kHeads = kHeadsOf<T>;
    const long long per_cta = kThreads / (D / 16);
    const long long gq = (a.num_heads + kHeads - 1) / kHeads, gk = (a.num_kv_heads + kHeads - 1) / kHeads;
    const long long nq = a.tokens * gq, nk = a.tokens * gk;
    if (!append || a.bounds == nullptr) {
        const long long ctas = (nq + nk + per_cta - 1) / per_cta;
        return append ? launch<T, D, PAIRS, kAppend, 1>(a, axes, 0, ctas, s)
                      : launch<T, D, PAIRS, kRotary, 1>(a, axes, 0, ctas, s);
    }
    const long long qc = (nq + per_cta - 1) / per_cta;
    // Few tokens are mostly runs of their own: a warp for each and head.  Of many, most are
    // inside a run that begins before them, and a warp looks at several.  Looking at 1, 4 and 16, us
    // (tokens x kv heads, D = 128): 1024 x 8 of 1024 requests 11.7, 13.7, 35.2; 2051 x 16 of 316 19.0, 13.6, 17.1; 4096 x 8 of
    // as many 44.9, 42.0, 54.3; 5685 x 8 of 8 34.2, 30.1, 28.1; 33116 x 8 of 32 199, 145, 131.
    const long long warps = (long long)a.tokens * a.num_kv_heads, wave = 24ll * num_sms();
    auto go = [&](auto tile) {
        constexpr int TILE = decltype(tile)::value;
        const long long units = (a.tokens + TILE - 1) / TILE * (long long)a.num_kv_heads;
        const long long runs = (units + kThreads / 32 - 1) / (kThreads / 32);
        return launch<T, D, PAIRS, kAppendBounds, TILE>(a, axes, runs, runs + qc, s);
    };
    if (warps <= 3 * wave) return go(std::integral_constant<int, 1>());
    return warps <= 12 * wave ? go(std::integral_constant<int, 4>()) : go(std::integral_constant<int, 16>());
}

}  // namespace

int rotary_launch(const RotaryArgs &a, int axes, int head_dim, bool f32, bool interleaved, bool append, cudaStream_t s)
{
    if (f32) {
        if (head_dim == 64) return interleaved ? launch_mode<float, 64, true>(a, axes, append, s) : launch_mode<float, 64, false>(a, axes, append, s);
        return interleaved ? launch_mode<float, 128, true>(a, axes, append, s) : launch_mode<float, 128, false>(a, axes, append, s);
    }
    using B = __nv_bfloat16;
    if (head_dim == 64) return interleaved ? launch_mode<B, 64, true>(a, axes, append, s) : launch_mode<B, 64, false>(a, axes, append, s);
    return interleaved ? launch_mode<B, 128, true>(a, axes, append, s) : launch_mode<B, 128, false>(a, axes, append, s);
}

}  // namespace pa
