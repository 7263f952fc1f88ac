// Decode attention over the 4-bit paged pool (include/pa.h, pa_decode_q4).
//
// Mathematics.  With codes n, steps s and lows b (K and V each) a query's
// score of token j is  x_j = scale (s_j (q . n_j) + b_j sum(q))  and its output
// (sum_j (p_j s_j) n_j + sum_j p_j b_j) / sum_j p_j,  p_j = 2^(x_j log2 e - m).
// So both products run on the raw codes, and step and low enter once per
// (token, head) instead of once per element.
//
// Codes as matrix operands.  A nibble n at bits 0-3 of a half is the f16
// subnormal n 2^-24, at bits 4-7 it is n 2^-20, both exact, and mma.sync takes
// subnormals (its sums keep some 17 bits of their products: see operand()).  So
//  w & 0x000f000f  and  w & 0x00f000f0  of a
// word (and of w >> 8) are four operand registers: 5 instructions turn 8 codes
// into operands, with no conversion, subtraction or scaling.  The powers of two
// leave through q (its elements that meet the 2^-20 codes carry 2^-4) and
// through the output rows.
//  * S^T[token, head] = K q^T: A = 16 tokens x 16 dims, the lane's words of
//    rows lane/4 and lane/4 + 8; which dims share a k-step is free as long as
//    q's fragments follow, so rows are read 16 bytes at a time.
//  * O^T[dim, head] += V^T (p s)^T: A's registers hold token pairs, which is
//    how the pool stores V (a 32-bit word = 4 dims of tokens 2p, 2p + 1).
//  * Codes are not negative, and the tensor cores cut their sums instead of
//    rounding them: a plain sum of (p s) n drifts by 2^-25 a tile, which for
//    10,000 tokens is more than a bf16 step of an output that cancels against
//    sum p b.  So odd tokens run as -(p s) (15 - n) + (p s) 15: complementing
//    a code costs nothing (the mask above takes an xor in the same
//    instruction), the products come in both signs and the cuts cancel.
//  * q is scaled by a power of two per head into f16's range (a bf16 number
//    keeps all its bits); fp32 operands run as a sum of two f16 numbers.
//  * p s is rounded to f16 (half a step 2^-11; the sums of p and of p b are not
//    rounded), and what the rounding leaves is not dropped where that is cheap.
//    With fp32 operands, and where the heads stand in the columns more than once,
//    the rest goes along as a second f16 number, in the second case in a copy whose
//    columns would be zero for that tile, so it costs no product: 2^-22 of a weight.
//    bf16 groups of 5 to 8 heads fill the columns; a second pass of products took
//    96 long sequences from 176.5 to 206 us.  There the rest is applied to the
//    middle code: sum w n is off by sum (w' - w) (n - 7.5) instead of
//    sum (w' - w) n.  Distance to 64 bits, beside 1.663e-3 (64 sequences, two
//    copies), 1.657e-3 (1024, four) and 1.657e-3 (96, none) of the result's own
//    rounding: with w' alone 1.756, 1.733 and 1.755e-3 (42.0, 228.7 and 176.5 us),
//    now 1.663, 1.657 and 1.671e-3 (42.3, 233.6 and 178.5 us).
//  * The reference m of p s follows the maximum of x + log2(s), so that p s, not p, is
//    at most 2^14; it moves only when p s would pass that, and then
//    leaves it at 2^9.  So a weight keeps f16's 11 bits down to 2^-23 of the
//    largest one, and is off by 2^-34 of that at most below.
//
// Work.  HBM-bound on (D + 8) / 2D bytes an element.  One stage is 32 or 64
// tokens of one kv head: up to four records, each one bulk copy.  An SM has one
// CTA of 16 warps, TW of them sharing the tokens of each of HS kv heads; each
// resolves its part of the block table and fills its own ring of two stages.
// The flat list of (head group, sequence, block) is cut into equal ranges, one
// per CTA (every CTA derives them from cache_seqlens); a sequence cut by a
// range's border leaves partials (acc, m, l) that its last CTA joins in
// logical order.  The warps of a head join in shared memory first.
//
// What bounds it (bf16; algorithmic bytes over time, a copy runs at 6.8 TB/s):
//   96 sequences of 4K-16K, 64/8 heads x 128    1068 MB  179 us  6.0 TB/s  HBM; SMs end 5-8% apart
//   256 of 512-4096, 32/8 x 128                   648 MB  116 us  5.6 TB/s  the same
//   1024 of 257-768, 32/32 x 64                  1237 MB  234 us  5.3 TB/s  a sequence's ends, per head
//   64 of 512-4096, 32/8 x 128                    164 MB   42 us  3.9 TB/s  start 5-7 us, join 4-5 us
//   one of 5000, 32/8 x 128                       5.5 MB   14 us            latency: start, walk, join
// fp32 runs twice the products, operands of two halves and spilled registers:
//   96 sequences of 4K-16K, 64/8 heads x 128    1070 MB  319 us  3.4 TB/s
//   1024 of 257-768, 32/32 x 64                  1262 MB  349 us  3.6 TB/s
//   64 of 512-4096, 32/8 x 128                    166 MB   62 us  2.7 TB/s
#include "pa_internal.h"
#include "pa_q4.cuh"

#include <cuda_fp16.h>
#include <math.h>

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
// One CTA of 16 warps an SM: a warp takes up to 128 registers and 7 to 11 KB of
// ring.  With two CTAs of 8 warps, three slots a warp and twice the partials, 96
// long sequences took 183 us (175), 64 shorter ones 44.2 (42.0).
constexpr int kMaxWarps = 16;
// Slots of a warp's ring: 74 to 176 KB in flight an SM, which is more than HBM's
// latency needs.  More slots leave less L1 and were slower.
constexpr int kSlots = 2;
// Weights are p s in units of 2^14 (kUnit): for the largest steps, 2^125, the largest p
// is then 2^-102 and more, and those below 2^-24 of it, where f16 ends too, may flush to
// zero.  (In units of 1 it was 2^-13 of it.)
constexpr float kUnit = 6.103515625e-5f;
// Largest weight before the reference moves (2^14), and the log2 of the largest one
// after it has moved.
constexpr float kWeightMax = 16384.f, kWeightNew = 9.f;
// Steps below 2^-76, and below 2^-24 of the row's low value (of what is summed with
// p in its place, which is b + 15 s at most), count as that much there: p stays
// below 2^104, p b below 2^52, and their sums inside fp32.  (Rows of one value have a
// step of 0.)  Such a step's codes say less than fp32 holds of b.
constexpr float kStepFloor = 1.3234889800848443e-23f * kUnit, kLowPart = 5.9604644775390625e-8f * kUnit;

// A batch of at most this many sequences has its lengths in shared memory.
constexpr int kMaxLens = 512;

enum { kLast = 1, kAppend = 2, kBad = 4, kWhole = 8 };

// What the loader notes about one stage; the second half is written for a
// segment's last stage only.
struct alignas(16) Meta {
    int b, hg, len, cnt;       // sequence, head group, cache_seqlens[b], tokens | flags << 8
    int blocks, nblk, sb, blk; // blocks of the segment and of the sequence, blocks before the sequence; its new token's block
};

// A warp's loader, in shared memory, where it costs the sums no registers.
// The walk covers the warp's share of every segment: of a sequence's blocks
// [j0, je) in the CTA's range, the stages ct, ct + tw, ...  Table entries come
// in windows of kWindow of the warp's blocks, the next one (of this segment or of
// the next) fetched while the present one is used.
constexpr int kWindow = 64;
struct alignas(16) LoadState {
    uint64_t base; // the pool's record of the warp's head in block 0
    int e, elim;   // window cursor; stages before elim are SB whole blocks inside the segment
    int j0, je, ok, nblk;
    int b, hg, len, rem; // rem: units of the CTA's range from j0 on
    int sb, li0, lend, wsel; // blocks before b; stage at the window's start; last stage; window in use
    int len1, len2, pad[2];  // lengths of the next sequence and of the one after it
    int window[2 * kWindow];
};

struct DecodeQ4Geom {
    int hs, tw;          // kv heads of a CTA, warps that share one head
    int head_groups;
    int slot_floats;     // floats of one partial
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// D += A(16x16, row) * B(16x8, col), f16 inputs, fp32 accumulators.  Not
// volatile: independent products may be issued in any order.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (w & m) ^ x in one instruction.
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t m, uint32_t x)
{
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(d) : "r"(w), "r"(m), "r"(x));
    return d;
}

// Codes as they come out of a mask are f16 subnormals.  The tensor cores align
// a subnormal's product by the smallest exponent, so it keeps some 17 bits of
// the 24: plenty beside bf16 operands, too few for fp32 ones, whose codes are
// made normal numbers first (times 2^14, exact): the largest error against 64
// bits, over four shapes, goes from 1.6e-5 to 9e-7, and 64 fp32 sequences from 59.6 to
// 62.4 us, 1024 short ones from 315 to 349.
template <bool F32>
__device__ __forceinline__ uint32_t operand(uint32_t codes)
{
    if constexpr (F32) {
        const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&codes), __float2half2_rn(16384.f));
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    return codes;
}

__device__ __forceinline__ float log2_approx(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Wait for a barrier's phase without giving the thread up: an unsuccessful
// try_wait suspends it for microseconds on this GPU, many times the waits met
// here (a copy's rest, a neighbour's shuffles).  The limit is about a second.  A
// warp that gives up leaves: all its copies were under way before the wait began,
// so each has had the limit too.
__device__ __forceinline__ bool spin_wait(uint64_t *bar, uint32_t parity)
{
    for (uint32_t i = 0; i < (1u << 25); ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
    }
    return false;
}

// Barrier of the warps that share a head: one arrival a warp, and a wait with
// a limit like every other one here.  False when it gave up.
__device__ __forceinline__ bool group_sync(uint64_t *bar, int warps, uint32_t &phase)
{
    __syncwarp();
    if (warps == 1) return true;
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
    const bool ok = spin_wait(bar, phase);
    phase ^= 1;
    return __all_sync(kFull, ok);
}

template <int N>
__device__ __forceinline__ void lds(uint32_t (&w)[N], const uint8_t *p)
{
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x;
        w[1] = v.y;
    }
}

// N consecutive elements of q, N a multiple of 8, loaded 16 bytes at a time.
template <typename T, int N>
struct QWords;
template <int N>
struct QWords<__nv_bfloat16, N> {
    uint4 w[N / 8];
    template <bool SHARED>
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool ok)
    {
#pragma unroll
        for (int i = 0; i < N / 8; ++i)
            w[i] = ok ? load16<SHARED>(reinterpret_cast<const uint4 *>(p) + i) : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ float get(int i) const
    {
        const uint4 &v = w[i >> 3];
        const uint32_t x = (i >> 1 & 3) == 0 ? v.x : (i >> 1 & 3) == 1 ? v.y : (i >> 1 & 3) == 2 ? v.z : v.w;
        return i & 1 ? bf16_hi(x) : bf16_lo(x);
    }
};
template <int N>
struct QWords<float, N> {
    float4 w[N / 4];
    template <bool SHARED>
    __device__ __forceinline__ void load(const float *p, bool ok)
    {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            w[i] = ok ? load16<SHARED>(reinterpret_cast<const float4 *>(p) + i) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ float get(int i) const
    {
        const float4 &v = w[i >> 2];
        return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
    }
};

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

// The work's split.  Blocks stand in the order (head group, sequence, logical
// block), every sequence with cs positions of its own before them: what its
// start and end cost a CTA, in blocks (see kSeqTokens).  The positions are cut
// into P equal ranges.
struct Split {
    uint32_t q, r; // positions of a range, and the rest, spread over the ranges
    int P;
    float inv_p, inv; // 1 / P, ranges a position
    __device__ __forceinline__ Split(uint32_t total, int P_) : P(P_)
    {
        q = total / (uint32_t)P_;
        r = total - q * (uint32_t)P_;
        inv_p = __fdividef(1.f, (float)P_);
        inv = __fdividef((float)P_, (float)total);
    }
    // c r < P^2 < 2^20 here: half above a whole number, the quotient is never
    // nearer to the next one than the float's error
    __device__ __forceinline__ uint32_t start(int c) const
    {
        return c * q + (uint32_t)(((float)(c * r) + 0.5f) * inv_p);
    }
    __device__ __forceinline__ int range_of(uint32_t pos) const
    {
        int c = min(P - 1, (int)((float)pos * inv));
        while (start(c) > pos) --c;
        while (c + 1 < P && start(c + 1) <= pos) ++c;
        return c;
    }
};

// Blocks of a sequence with L cached tokens and its new one (1 where the
// length is refused).
__device__ __forceinline__ int seq_blocks(int L, long long cap, int bs, bool *ok)
{
    // positions of a stage's end stay below 2^31 too
    *ok = L >= 0 && L < 0x7fffff80 && (long long)L + 1 <= cap;
    return *ok ? L / bs + 1 : 1;
}

// A CTA's range holds at least this many tokens of its heads: below that,
// more CTAs cost more in partials than they save.  With 128, 256 and 512 a
// sequence of 300 tokens takes 11.9, 11.2 and 11.0 us, one of 2500 13.5, 12.8
// and 14.2, eight of 300 to 900 19.8, 19.3 and 20.9.
constexpr int kMinTokens = 256;
// What the start and end of a sequence cost a warp, in tokens of its head: with
// 0, 200 and 400, 64 sequences of 512 to 4096 take 51.4, 42.4 and 42.4 us, 256 of
// them 122.2, 116.1 and 122.5, 96 of 4K to 16K 175.0, 169.3 and 174.7.
constexpr int kSeqTokens = 200;
// Parts of a sequence that its last CTA joins, about (see make_plan).  With 4, 8
// and 16, 16 sequences of 512 to 4096 take 26.6, 25.8 and 27.1 us, eight of 20K to
// 40K 54.7, 53.2 and 53.7.
constexpr int kMaxParts = 8;

// A slot of a ring: a stage's records and behind them, where 16 warps' slots leave
// the room, the head's rows of q (with a segment's first stage) and its new rows
// (with the stage that takes them).  They come with the stage's copies and spare a
// warp two trips to L2 at every sequence, on which 16 warps with sequences of equal
// length wait at the same time: 1024 sequences of 257 to 768 tokens, 32 heads of
// either kind, 235 -> 228 us.
template <int D, int R, typename T>
struct Slot {
    static constexpr bool with_q = D == 64, with_new = D == 64 || R == 2;
    static constexpr int tokens = 16 * (R < 2 ? 2 : R), row = D * (int)sizeof(T);
    static constexpr int q = tokens * (D + 8); // where q starts
    static constexpr int k_new = q + (with_q ? 8 / R * row : 0);
    static constexpr int v_new = k_new + (with_new ? row : 0);
    static constexpr int bytes = v_new + (with_new ? row : 0);
};

// Quantise the new token's rows of the warp's head, K in lanes 0-7 and V in 8-15,
// and write them into the pool and into the stage at `st`, whose last token it is
// (cnt tokens; `mt` is its note).
template <int D, int BS, int R, typename T>
__device__ __noinline__ void append(const DecodeQ4Args &a, const Meta &mt, int hs, int ch, int cnt, uint8_t *st)
{
    constexpr int NC = D / 64;
    using S = Slot<D, R, T>;
    const int lane = threadIdx.x & 31, l = lane & 7;
    const bool value = lane & 8;
    const int kvh = mt.hg * hs + ch, blk = mt.blk, t = (cnt - 1) % BS;
    uint8_t *rec = st + (cnt - 1) / BS * q4_record_bytes(D, BS);
    const size_t src = ((size_t)mt.b * a.num_kv_heads + kvh) * D + l * 8;
    Q4Row<T, NC> x;
    if constexpr (S::with_new)
        x.template load<true>(reinterpret_cast<const T *>(st + (value ? S::v_new : S::k_new)) + l * 8);
    else
        x.template load<false>(static_cast<const T *>(value ? a.v_new : a.k_new) + src);
    Q4Scale s;
    uint32_t c[NC];
    q4_quantise(x, s, c);
    if (lane < 16) {
        if (T *kept = static_cast<T *>(value ? a.v_stored : a.k_stored)) {
#pragma unroll
            for (int i = 0; i < 2 * NC; ++i) {
                const uint32_t n = c[i >> 1] >> (i & 1) * 16;
                store4(kept + src + (i >> 1) * 64 + (i & 1) * 4, q4_value(n & 15u, s.step, s.low),
                       q4_value(n >> 4 & 15u, s.step, s.low), q4_value(n >> 8 & 15u, s.step, s.low),
                       q4_value(n >> 12 & 15u, s.step, s.low));
            }
        }
        uint8_t *dst = static_cast<uint8_t *>(a.kv_cache) +
                       ((size_t)blk * a.num_kv_heads + kvh) * q4_record_bytes(D, BS);
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            uint8_t *p = side ? dst : rec;
#pragma unroll
            for (int u = 0; u < NC; ++u) {
                if (value) {
                    uint16_t *unit = reinterpret_cast<uint16_t *>(p + q4_v_offset(D, BS)) +
                                     q4_v_unit<D>(t, u * 16 + 2 * l);
                    unit[0] = (uint16_t)c[u];
                    unit[2] = (uint16_t)(c[u] >> 16);
                } else {
                    *reinterpret_cast<uint32_t *>(p + t * (D / 2) + u * 32 + l * 4) = c[u];
                }
            }
            if (l == 0)
                *reinterpret_cast<uint32_t *>(p + q4_scale_offset(D, BS) + t * 8 + (value ? 4 : 0)) = q4_pack_scale(s);
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// Join the parts of a sequence in logical order and store its output rows.
// A part is `group` rows of D sums and, behind them, (m, l) of each row; a
// refused part has l = -inf.  D / 4 lanes stand for a row's columns, four dims
// each, and for as many parts' (m, l): they find the weights 2^(m - max m) by
// shuffles while the first KU parts' columns are on their way.  A warp takes NE
// such rows (or pairs of rows) at a time.  Not inlined: it runs once a sequence
// and its registers would weigh on the loop.
template <int D, typename T, int NE>
__device__ __noinline__ void fold(const float *first, size_t step, int nseg, int group, int warp, int warps, T *out)
{
    constexpr int HL = D / 4, RW = 32 / HL; // lanes of a row, rows of a warp
    constexpr int KU = NE == 1 ? 8 : 5;
    const int lane = threadIdx.x & 31, sub = lane % HL;
#pragma unroll 1
    for (int r0 = warp * NE * RW; r0 < group; r0 += warps * NE * RW) {
        int g[NE];
        float M[NE], l[NE];
        float4 o[NE];
        bool refused[NE];
#pragma unroll
        for (int n = 0; n < NE; ++n) {
            g[n] = min(r0 + n * RW + lane / HL, group - 1);
            M[n] = -INFINITY;
            l[n] = 0.f;
            o[n] = make_float4(0.f, 0.f, 0.f, 0.f);
            refused[n] = false;
        }
#pragma unroll 1
        for (int k0 = 0; k0 < nseg; k0 += HL) {
            const int parts = min(HL, nseg - k0);
            const float *base = first + (size_t)k0 * step;
            float2 z[NE];
            float f[NE];
#pragma unroll
            for (int n = 0; n < NE; ++n)
                z[n] = sub < parts ? __ldcg(reinterpret_cast<const float2 *>(base + sub * step + group * D + 2 * g[n]))
                                   : make_float2(-INFINITY, 0.f);
#pragma unroll 1
            for (int k = 0; k < parts; k += KU) {
                float4 x[NE][KU];
#pragma unroll
                for (int n = 0; n < NE; ++n)
#pragma unroll
                    for (int u = 0; u < KU; ++u)
                        x[n][u] = k + u < parts ? __ldcg(reinterpret_cast<const float4 *>(
                                                      base + (size_t)(k + u) * step + g[n] * D + 4 * sub))
                                                : make_float4(0.f, 0.f, 0.f, 0.f);
                if (k == 0) { // the chunk's weights
#pragma unroll
                    for (int n = 0; n < NE; ++n) {
                        float top = fmaxf(M[n], z[n].x);
#pragma unroll
                        for (int q = HL / 2; q > 0; q >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, q));
                        const float fo = top == -INFINITY ? 1.f : exp2_approx(M[n] - top);
                        f[n] = top == -INFINITY ? 1.f : exp2_approx(z[n].x - top);
                        const unsigned bad = __ballot_sync(kFull, z[n].y == -INFINITY);
                        refused[n] = refused[n] || (HL == 32 ? bad : bad >> (lane & 16) & 0xffffu);
                        float s = z[n].y * f[n];
#pragma unroll
                        for (int q = HL / 2; q > 0; q >>= 1) s += __shfl_xor_sync(kFull, s, q);
                        M[n] = top;
                        l[n] = fmaf(l[n], fo, s);
                        o[n].x *= fo;
                        o[n].y *= fo;
                        o[n].z *= fo;
                        o[n].w *= fo;
                    }
                }
#pragma unroll
                for (int n = 0; n < NE; ++n)
#pragma unroll
                    for (int u = 0; u < KU; ++u) {
                        if (k + u >= parts) break;
                        const float w = __shfl_sync(kFull, f[n], k + u, HL);
                        o[n].x = fmaf(x[n][u].x, w, o[n].x);
                        o[n].y = fmaf(x[n][u].y, w, o[n].y);
                        o[n].z = fmaf(x[n][u].z, w, o[n].z);
                        o[n].w = fmaf(x[n][u].w, w, o[n].w);
                    }
            }
        }
#pragma unroll
        for (int n = 0; n < NE; ++n) {
            if (r0 + n * RW + lane / HL >= group) break;
            const float inv = 1.f / l[n];
            T *y = out + (size_t)g[n] * D + 4 * sub;
            if (refused[n])
                store4(y, 0.f, 0.f, 0.f, 0.f);
            else
                store4(y, o[n].x * inv, o[n].y * inv, o[n].z * inv, o[n].w * inv);
        }
    }
}

__device__ __forceinline__ void copy4_async(void *dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_wait()
{
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
}

// The loader's slower steps: everything but a stage of whole blocks inside a
// segment.  Not inlined, so that its registers do not weigh on the sums.
template <int D, int BS, int R, typename T>
struct Loader {
    using S = Slot<D, R, T>;
    static constexpr int REC = q4_record_bytes(D, BS);
    static constexpr int SB = S::tokens / BS; // blocks of a stage

    // fetch the entries of the warp's blocks o0.. of a segment into window w
    static __device__ __forceinline__ void fetch(const DecodeQ4Args &a, LoadState &ld, int w, int b, bool ok, int j0,
                                                 int je, int o0, int tw, int ct)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int k = lane; k < kWindow; k += 32) {
            const int o = o0 + k;
            const int blk = j0 + ((o / SB) * tw + ct) * SB + o % SB;
            if (ok && blk < je)
                copy4_async(&ld.window[w * kWindow + k], a.block_table + (size_t)b * a.max_blocks_per_seq + blk);
            else
                ld.window[w * kWindow + k] = -1;
        }
    }
    // q and the new rows of a sequence: in L2 by the time they are read
    static __device__ __forceinline__ void warm(const DecodeQ4Args &a, int b, int kvh, bool ends)
    {
        const int lane = threadIdx.x & 31;
        const size_t row = (size_t)b * a.num_kv_heads + kvh;
        for (int o = lane * 128; !S::with_q && o < a.group * S::row; o += 32 * 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(a.q) +
                                                          row * a.group * S::row + o));
        if (!S::with_new && ends && lane < 2)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(
                static_cast<const char *>(lane ? a.v_new : a.k_new) + row * S::row));
    }
    // start of the segment (b, hg) from block j0 on, with `rem` units left;
    // len2 has been fetched
    static __device__ __forceinline__ void enter(const DecodeQ4Args &a, LoadState &ld, int b, int hg, int len, int j0,
                                                 int rem, int sb, int tw, int ct, int kvh)
    {
        const int lane = threadIdx.x & 31, B = a.batch;
        bool ok;
        const int nblk = seq_blocks(len, (long long)a.max_blocks_per_seq * BS, BS, &ok);
        const int je = min(nblk, j0 + rem), stages = (je - j0 + SB - 1) / SB;
        const int len1 = ld.len2;
        __syncwarp();
        if (lane == 0) {
            ld.j0 = j0;
            ld.je = je;
            ld.ok = ok;
            ld.nblk = nblk;
            ld.b = b;
            ld.hg = hg;
            ld.len = len;
            ld.rem = rem;
            ld.sb = sb;
            ld.li0 = 0;
            ld.lend = max(0, (stages - ct + tw - 1) / tw - 1);
            ld.len1 = len1;
            ld.base = reinterpret_cast<uint64_t>(a.kv_cache) + (size_t)kvh * REC;
            const int b2 = b + 2;
            copy4_async(&ld.len2, a.cache_seqlens + (b2 < B ? b2 : B > 1 ? b2 - B : 0));
        }
        __syncwarp();
    }
    // the window after the one in use, which starts at stage li0
    static __device__ __forceinline__ void fetch_next(const DecodeQ4Args &a, LoadState &ld, int tw, int ct, int hs,
                                                      int ch)
    {
        const int o0 = ld.li0 * SB + kWindow, j0 = ld.j0, je = ld.je, b = ld.b, rem = ld.rem - (je - j0);
        if (((o0 / SB) * tw + ct) * SB < je - j0) {
            fetch(a, ld, ld.wsel ^ 1, b, ld.ok, j0, je, o0, tw, ct);
        } else if (rem > 0) {
            const bool wrap = b + 1 == a.batch;
            bool ok;
            const int n = seq_blocks(ld.len1, (long long)a.max_blocks_per_seq * BS, BS, &ok);
            const int e = min(n, rem);
            fetch(a, ld, ld.wsel ^ 1, wrap ? 0 : b + 1, ok, 0, e, 0, tw, ct);
            warm(a, wrap ? 0 : b + 1, (wrap ? ld.hg + 1 : ld.hg) * hs + ch, e == n);
        }
    }
    // any stage into the slot (stage buffer dst, barrier, note)
    static __device__ __noinline__ void issue(const DecodeQ4Args &a, LoadState &ld, uint32_t dst, uint64_t *bar,
                                              Meta *meta, int tw, int ct, int hs, int ch)
    {
        const int lane = threadIdx.x & 31;
        copy_async_wait(); // windows and lengths
        const int rem0 = ld.rem;
        if (rem0 <= 0) return;
        const int j0 = ld.j0, je = ld.je, nblk = ld.nblk, len = ld.len, b = ld.b, hg = ld.hg, sb = ld.sb;
        const bool ok = ld.ok != 0;
        const int e = ld.e, li = ld.li0 + (e - ld.wsel * kWindow) / SB, lend = ld.lend;
        const int blk0 = j0 + (li * tw + ct) * SB;
        const int blocks = max(0, min(SB, je - blk0));
        const int p = ld.window[e + (lane & (SB - 1))];
        const bool here = lane < blocks;
        const bool valid = here && ok && p >= 0 && p < a.num_blocks;
        if (here && ok && !valid) flag_error(a.dev_err, PA_DEVERR_BAD_BLOCK);
        const int loads = __popc(__ballot_sync(kFull, valid));
        const bool last = li == lend;
        const int pos0 = blk0 * BS, kvh = hg * hs + ch;
        const bool takes = ok && loads == blocks && blocks > 0 && len < pos0 + blocks * BS; // the new token
        const int tail = __shfl_sync(kFull, p, (blocks - 1) & 31);
        if (lane == 0) {
            const int cnt = blocks > 0 && ok ? min(blocks * BS, len - pos0 + 1) : 0;
            int flags = last ? kLast : 0;
            if (loads < blocks || !ok) flags |= kBad;
            if (takes) flags |= kAppend;
            if (j0 == 0 && je == nblk) flags |= kWhole;
            int4 *mt = reinterpret_cast<int4 *>(meta);
            mt[0] = make_int4(b, hg, len, cnt | flags << 8);
            mt[1] = make_int4(je - j0, nblk, sb, tail);
            uint32_t bytes = loads * REC;
            if (S::with_q && li == 0) bytes += a.group * S::row;
            if (S::with_new && takes) bytes += 2 * S::row;
            if (bytes > 0)
                mbar_arrive_expect_tx(bar, bytes);
            else
                mbar_arrive(bar);
        }
        __syncwarp();
        const size_t row = (size_t)b * a.num_kv_heads + kvh;
        if (S::with_q && lane == 31 && li == 0)
            bulk_load(dst + S::q, static_cast<const char *>(a.q) + row * a.group * S::row, a.group * S::row, bar);
        if (S::with_new && lane >= 29 && lane < 31 && takes)
            bulk_load(dst + (lane == 29 ? S::k_new : S::v_new),
                      static_cast<const char *>(lane == 29 ? a.k_new : a.v_new) + row * S::row, S::row, bar);
        if (valid)
            bulk_load(dst + lane * REC,
                      static_cast<const uint8_t *>(a.kv_cache) + ((size_t)p * a.num_kv_heads + kvh) * REC, REC, bar);
        bool switched = false;
        if (last) {
            const int rem = rem0 - (je - j0);
            if (rem <= 0) {
                if (lane == 0) ld.rem = ld.e = ld.elim = 0;
                __syncwarp();
                return;
            }
            const bool wrap = b + 1 == a.batch;
            const int hg1 = wrap ? hg + 1 : hg;
            enter(a, ld, wrap ? 0 : b + 1, hg1, ld.len1, 0, rem, wrap ? 0 : sb + nblk, tw, ct, hg1 * hs + ch);
            switched = true;
        } else if (((li + 1) * SB & (kWindow - 1)) == 0) {
            if (lane == 0) ld.li0 = li + 1;
            switched = true;
        }
        const int w = ld.wsel ^ (switched ? 1 : 0);
        __syncwarp();
        const int first = w * kWindow, at = switched ? first : e + SB; // the cursor
        const int li1 = switched ? ld.li0 : li + 1, li0 = ld.li0;
        if (lane == 0) ld.wsel = w;
        __syncwarp();
        // whole blocks inside the segment, in this window; the first stage of
        // a segment and the last one of a segment or a window come here
        const int upto = min(ld.lend, li0 + kWindow / SB - 1); // stages before this one
        bool fine = true;
#pragma unroll
        for (int k = lane; k < kWindow; k += 32) {
            const int v = ld.window[first + k];
            fine = fine && (k >= (upto - li0) * SB || (v >= 0 && v < a.num_blocks));
        }
        fine = __all_sync(kFull, fine);
        if (lane == 0) {
            ld.e = at;
            ld.elim = fine && li1 > 0 ? first + (upto - li0) * SB : 0;
        }
        __syncwarp();
        if (switched) fetch_next(a, ld, tw, ct, hs, ch);
    }
};

// Columns of the products.  A product has 8 columns; a group of at most 8 / R
// query heads stands in them R times, and copy `rep` of a score belongs to
// tile `rep` of R: every lane then turns the scores of its own tile into
// weights (1 / R of the work), the weights of a tile are left in its own copy
// (bf16: what their rounding left in the neighbouring one; the others are masked to
// zero), and the copies' sums are added at the end.
// R = 1 has two tiles a stage as well, and every lane works on both.
template <int D, int BS, int R, typename T>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
    decode_q4_kernel(const DecodeQ4Args a, const DecodeQ4Geom gm)
{
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int REC = q4_record_bytes(D, BS);
    constexpr int NTILE = R < 2 ? 2 : R;            // 16-token tiles of a stage
    constexpr int ST = 16 * NTILE;                  // tokens of a stage
    constexpr int SB = ST / BS;                     // blocks of a stage
    using S = Slot<D, R, T>;
    constexpr int KW = D / 32;                      // words of a lane's row part
    constexpr int MT = D / 16;                      // 16-dim tiles of the output
    constexpr int DL = D / 8;                       // output dims of a lane
    constexpr int CW = 8 / R;                       // columns of one copy
    constexpr int XT = NTILE / R;                   // tiles whose scores a lane works on
    constexpr int kCodeShift = F32 ? 10 : 24;       // operands are codes times 2^-shift
    constexpr float kCodeScale = F32 ? 1024.f : 16777216.f;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_warp[kMaxWarps];
    __shared__ int s_total;
    __shared__ int s_first[4];  // first sequence, blocks before it, its length, the next one's
    __shared__ uint32_t s_u[2]; // first and one-past-last block of the range
    __shared__ int s_lens[kMaxLens];
    __shared__ float s_m[kMaxWarps][8], s_l[kMaxWarps][8], s_b[kMaxWarps][8];
    __shared__ int s_last[kMaxWarps];
    __shared__ uint64_t s_group[kMaxWarps];
    __shared__ LoadState s_load[kMaxWarps];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int nst = kSlots;
    const int hs = gm.hs, tw = gm.tw, ncw = hs * tw;
    const int NT = ncw * 32;
    const int B = a.batch, mbps = a.max_blocks_per_seq;
    const long long cap = (long long)mbps * BS;
    // rings of the consumers, barriers, metadata, join buffers
    uint8_t *ring = smem;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + (size_t)ncw * nst * S::bytes);
    Meta *meta = reinterpret_cast<Meta *>(full + ((ncw * nst + 1) & ~1));
    float *join = reinterpret_cast<float *>(meta + ncw * nst);

    if (tid < ncw * nst) {
        mbar_init(&full[tid], 1);
        if (tid < hs) mbar_init(&s_group[tid], tw);
        fence_mbar_init();
    }
    grid_dep_trigger();
    for (int b = tid * 32; b < B; b += NT * 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.cache_seqlens + b));
    // nothing above read or wrote memory that a predecessor may write
    grid_dep_wait();

    // ---- block-wide scan of the sequences' block counts
    const int per = (B + NT - 1) / NT;
    const int b_lo = min(B, tid * per), b_hi = min(B, b_lo + per);
    int local = 0;
    const bool cached = B <= kMaxLens;
    auto len_of = [&](int b) { return cached ? s_lens[b] : a.cache_seqlens[b]; };
    for (int b = b_lo; b < b_hi; ++b) {
        bool ok;
        const int len = a.cache_seqlens[b];
        if (cached) s_lens[b] = len;
        local += seq_blocks(len, cap, BS, &ok);
        if (!ok && len != PA_LEFT_OUT && blockIdx.x == 0) flag_error(a.dev_err, PA_DEVERR_OVERFLOW);
    }
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int v = lane < ncw ? s_warp[lane] : 0;
        int inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += t;
        }
        if (lane < ncw) s_warp[lane] = inc - v;
        if (lane == ncw - 1) s_total = inc;
    }
    __syncthreads();
    const uint32_t ublk = s_total, U = ublk * gm.head_groups;
    // ranges: one a CTA, as many as the work fills (a sequence of a head group
    // at least), and the same number for every head group
    int P = min((int)gridDim.x, max((int)(U / (uint32_t)(kMinTokens / BS)), B * gm.head_groups));
    if (gm.head_groups > 1 && P > gm.head_groups) P = P / gm.head_groups * gm.head_groups;
    if ((int)blockIdx.x >= P) return;
    const uint32_t cs = min((uint32_t)(kSeqTokens * tw / BS), U / (uint32_t)P / 4);
    const uint32_t cblk = ublk + cs * B; // positions of a head group
    const Split split(cblk * gm.head_groups, P);
    {
        // first block at or after the range's first position, and after its last
        const uint32_t sbt = s_warp[warp] + incl - local; // blocks before b_lo
        const uint32_t sct = sbt + cs * b_lo, span = local + cs * (b_hi - b_lo);
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
            const uint32_t cc = split.start(blockIdx.x + e);
            if ((int)blockIdx.x + e == P) {
                if (tid == 0) s_u[e] = U;
                continue;
            }
            const uint32_t h = gm.head_groups == 1 ? 0 : cc / cblk, r = cc - h * cblk;
            if (r < sct || r >= sct + span) continue;
            uint32_t sb = sbt, sc = sct;
            for (int b = b_lo; b < b_hi; ++b) {
                bool ok;
                const int len = len_of(b);
                const int n = seq_blocks(len, cap, BS, &ok);
                if (r < sc + cs + n) {
                    const uint32_t j = r < sc + cs ? 0 : r - sc - cs;
                    s_u[e] = h * ublk + sb + j;
                    if (e == 0) {
                        s_first[0] = b;
                        s_first[1] = sb;
                        s_first[2] = len;
                        s_first[3] = len_of(b + 1 < B ? b + 1 : 0);
                    }
                    break;
                }
                sb += n;
                sc += cs + n;
            }
        }
    }
    __syncthreads();
    const uint32_t u0 = s_u[0], u1 = s_u[1];
    if (u0 >= u1) return;
    const int G = a.group, Hkv = a.num_kv_heads, Hq = a.num_heads;

    const int ct = warp / hs, ch = warp % hs; // token share, head within the group
    const uint32_t block_bytes = (uint32_t)Hkv * REC;

    // ================= loader =================
    // Every warp fills its own ring: it issues a stage's copies as soon as it
    // has used the slot up, so no other warp and no second barrier is waited
    // for.
    using L = Loader<D, BS, R, T>;
    LoadState &ld = s_load[warp];
    auto issue = [&](int at) {
        const uint32_t dst = smem_u32(ring + at * S::bytes);
        const int e = ld.e;
        if (e < ld.elim) { // SB whole blocks inside a segment
            if (elect_one()) {
                const uint8_t *base = reinterpret_cast<const uint8_t *>(ld.base);
                meta[at].cnt = ST;
                mbar_arrive_expect_tx(&full[at], SB * REC);
#pragma unroll
                for (int k = 0; k < SB; ++k)
                    bulk_load(dst + k * REC, base + (size_t)ld.window[e + k] * block_bytes, REC, &full[at]);
                ld.e = e + SB;
            }
            __syncwarp();
        } else {
            L::issue(a, ld, dst, &full[at], &meta[at], tw, ct, hs, ch);
        }
    };
    {
        const int b = s_first[0], hg = gm.head_groups == 1 ? 0 : (int)(u0 / ublk);
        const int j0 = (int)(u0 - hg * ublk) - s_first[1];
        if (lane == 0) {
            ld.len2 = s_first[3];
            ld.e = ld.elim = ld.wsel = 0;
        }
        __syncwarp();
        L::enter(a, ld, b, hg, s_first[2], j0, (int)(u1 - u0), s_first[1], tw, ct, hg * hs + ch);
        L::fetch(a, ld, 0, b, ld.ok, j0, ld.je, 0, tw, ct);
        L::warm(a, b, hg * hs + ch, ld.je == ld.nblk);
        L::fetch_next(a, ld, tw, ct, hs, ch);
#pragma unroll 1
        for (int i = 0; i < nst; ++i) issue(warp * nst + i);
    }

    // ================= sums =================
    const int r = lane >> 2, c = lane & 3; // C fragment: rows r, r + 8; columns 2c, 2c + 1
    const int rep = R == 1 ? 0 : c / (4 / R);  // copy of the lane's C columns: its tile
    const int col = 2 * c % CW;                // head of the lane's first column
    const int brep = r / CW;                   // copy of the lane's B column r
    const int gthreads = tw * 32, gtid = ct * 32 + lane; // threads that share the head
    const uint32_t k_off = r * (D / 2) + c * (D / 8);
    const uint32_t v_off = q4_v_offset(D, BS) +
                           (D == 128 ? c * 128 + (((r >> 1) ^ c) << 5) + ((r & 1) << 4)
                                     : c * 64 + (((r >> 2) ^ (c >> 1)) << 5) + ((r & 3) << 3));
    // place of tile t's parts: whole records for 16-token blocks, halves of a
    // record for 32-token ones
    auto tile_at = [](int t, int row_bytes) { return BS == 16 ? t * REC : (t >> 1) * REC + (t & 1) * 16 * row_bytes; };
    const uint32_t s_off = q4_scale_offset(D, BS) + r * 8;
    T *outp = static_cast<T *>(a.out);
    // rows r and r + 8 are tokens of r's parity
    constexpr bool SECOND = F32 || R > 1; // the weights as two f16 numbers
    const float base = (SECOND ? (r & 1) ? 15.f : 0.f : 7.5f) / kUnit;
    const float centre = ((r & 1) ? 7.5f : -7.5f) / kUnit;
    const uint32_t odd_sign = (r & 1) ? 0x80008000u : 0u;

    uint32_t qh[KW][2][2], ql[F32 ? KW : 1][2][2];
    float acc[MT][4];
    float c0 = 0.f, c1 = 0.f, qs0 = 0.f, qs1 = 0.f, h0 = 0.f, h1 = 0.f; // score factors of the two columns
    float m0, m1, l0, l1, lo0, lo1;
    int stage = 0;
    uint32_t phase = 0, gphase = 0;
    auto sync = [&] {
        const bool ok = group_sync(&s_group[ch], tw, gphase);
        if (!ok && lane == 0) flag_error(a.dev_err, PA_DEVERR_TIMEOUT);
        return ok;
    };
    int left = (int)(u1 - u0); // units whose segments have not ended here

    while (left > 0) { // segments
        bool bad = false, fresh; // fresh: no reference yet
        int at = warp * nst + stage;
        { // q of column r's head, the dims of this lane's words; its loads run beside the first stage's copies
            m0 = m1 = 0.f;
            fresh = true;
            l0 = l1 = lo0 = lo1 = 0.f;
            const int g = r % CW;
            QWords<T, KW * 8> qw;
            if constexpr (S::with_q) {
                if (!spin_wait(&full[at], phase)) {
                    if (lane == 0) flag_error(a.dev_err, PA_DEVERR_TIMEOUT);
                    return;
                }
                qw.template load<true>(reinterpret_cast<const T *>(ring + at * S::bytes + S::q) + g * D + c * (KW * 8), g < G);
            } else {
                qw.template load<false>(static_cast<const T *>(a.q) +
                                            ((size_t)meta[at].b * Hq + (size_t)(meta[at].hg * hs + ch) * G + g) * D +
                                            c * (KW * 8),
                                        g < G);
            }
            float amax = 0.f, sum = 0.f;
#pragma unroll
            for (int i = 0; i < KW * 8; ++i) {
                const float x = qw.get(i);
                amax = fmaxf(amax, fabsf(x));
                sum += x;
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
                sum += __shfl_xor_sync(kFull, sum, o);
            }
            // 2^e brings the largest element to [2^14, 2^15)
            int e = amax > 0.f ? 14 - ((int)(__float_as_uint(amax) >> 23) - 127) : 0;
            e = max(-100, min(100, e));
            const float up = __uint_as_float((uint32_t)(127 + e) << 23);
            const float down = __uint_as_float((uint32_t)(127 + kCodeShift - e) << 23) * a.scale_log2;
#pragma unroll
            for (int i = 0; i < KW; ++i)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const float x0 = qw.get(8 * i + 2 * s) * up, x1 = qw.get(8 * i + 2 * s + 4) * up;
                    const float y0 = qw.get(8 * i + 2 * s + 1) * up * 0.0625f, y1 = qw.get(8 * i + 2 * s + 5) * up * 0.0625f;
                    qh[i][s][0] = pack_f16(x0, x1);
                    qh[i][s][1] = pack_f16(y0, y1);
                    if constexpr (F32) {
                        const __half2 hx = *reinterpret_cast<__half2 *>(&qh[i][s][0]);
                        const __half2 hy = *reinterpret_cast<__half2 *>(&qh[i][s][1]);
                        ql[i][s][0] = pack_f16(x0 - __low2float(hx), x1 - __high2float(hx));
                        ql[i][s][1] = pack_f16(y0 - __low2float(hy), y1 - __high2float(hy));
                    }
                }
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
            // 7.5 sum q in the products' units (fp32 only)
            const float half = sum * up * (7.5f / kCodeScale);
            if constexpr (F32) {
                h0 = __shfl_sync(kFull, half, 4 * col);
                h1 = __shfl_sync(kFull, half, 4 * col + 4);
            }
            sum *= a.scale_log2;
            c0 = __shfl_sync(kFull, down, 4 * col);
            c1 = __shfl_sync(kFull, down, 4 * col + 4);
            qs0 = __shfl_sync(kFull, sum, 4 * col);
            qs1 = __shfl_sync(kFull, sum, 4 * col + 4);
        }
        Meta mt;
        int flags;
#pragma unroll 1
        do { // stages
        const int cf = meta[at].cnt; // written by this warp when it issued the stage
        flags = cf >> 8;
        if (!spin_wait(&full[at], phase)) {
            if (lane == 0) flag_error(a.dev_err, PA_DEVERR_TIMEOUT);
            return;
        }
        uint8_t *st = ring + at * S::bytes;
        int cnt = ST;
        if (cf != ST) { // not SB whole blocks inside a segment
            bad |= (flags & kBad) != 0;
            cnt = (flags & kBad) ? 0 : cf & 255;
            if (flags & kAppend)
                append<D, BS, R, T>(a, meta[at], hs, ch, cnt, st);
        }
        if (cnt > 0) {
            // ---- products of the tiles, one chain each
            float dot[NTILE][4] = {};
#pragma unroll
            for (int tile = 0; tile < NTILE; ++tile) {
                uint32_t ka[KW], kb[KW];
                const uint8_t *tk = st + tile_at(tile, D / 2) + k_off;
                lds<KW>(ka, tk);
                lds<KW>(kb, tk + 4 * D);
#pragma unroll
                for (int i = 0; i < KW; ++i)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint32_t wa = s ? ka[i] >> 8 : ka[i], wb = s ? kb[i] >> 8 : kb[i];
                        const uint32_t a0 = operand<F32>(wa & 0x000f000fu), a1 = operand<F32>(wb & 0x000f000fu);
                        const uint32_t a2 = operand<F32>(wa & 0x00f000f0u), a3 = operand<F32>(wb & 0x00f000f0u);
                        if constexpr (F32) {
                            // small part first, one sum of 16 at a time: the
                            // tensor cores cut each sum at the size of its
                            // largest term
                            float part[4] = {0.f, 0.f, 0.f, 0.f};
                            mma_f16(part, a0, a1, a2, a3, ql[i][s][0], ql[i][s][1]);
                            mma_f16(part, a0, a1, a2, a3, qh[i][s][0], qh[i][s][1]);
#pragma unroll
                            for (int k = 0; k < 4; ++k) dot[tile][k] += part[k];
                        } else {
                            mma_f16(dot[tile], a0, a1, a2, a3, qh[i][s][0], qh[i][s][1]);
                        }
                    }
            }
            if constexpr (R == 2) {
#pragma unroll
                for (int k = 0; k < 4; ++k) dot[0][k] = rep ? dot[1][k] : dot[0][k];
            } else if constexpr (R == 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float u = (rep & 1) ? dot[1][k] : dot[0][k], v = (rep & 1) ? dot[3][k] : dot[2][k];
                    dot[0][k] = (rep & 2) ? v : u;
                }
            }
            // ---- scores of the lane's tokens r, r + 8 of its tiles
            float x[XT][4], vst[XT][2], vlo[XT][2];
#pragma unroll
            for (int t = 0; t < XT; ++t) {
                const int tile = R == 1 ? t : rep;
                const uint8_t *ts = st + (BS == 16 ? tile * REC : (tile >> 1) * REC + (tile & 1) * 128) + s_off;
                uint32_t sc[2][2];
                lds<2>(sc[0], ts);
                lds<2>(sc[1], ts + 64);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float ks = bf16_lo(sc[k][0]), kl = bf16_hi(sc[k][0]);
                    vst[t][k] = bf16_lo(sc[k][1]) * kUnit;
                    vlo[t][k] = fmaf(vst[t][k], base, bf16_hi(sc[k][1]));
                    if constexpr (F32) {
                        // around the middle code, where the two terms do not cancel
                        const float mid = fmaf(ks, 7.5f, kl);
                        x[t][2 * k] = fmaf(ks * c0, dot[t][2 * k] - h0, fmaf(mid, qs0, -m0));
                        x[t][2 * k + 1] = fmaf(ks * c1, dot[t][2 * k + 1] - h1, fmaf(mid, qs1, -m1));
                    } else {
                        x[t][2 * k] = fmaf(ks * c0, dot[t][2 * k], fmaf(kl, qs0, -m0));
                        x[t][2 * k + 1] = fmaf(ks * c1, dot[t][2 * k + 1], fmaf(kl, qs1, -m1));
                    }
                }
            }
            if (cnt < ST) { // tokens behind the sequence's: whatever the pool holds there
#pragma unroll
                for (int t = 0; t < XT; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if ((R == 1 ? t : rep) * 16 + k * 8 + r >= cnt) {
                            x[t][2 * k] = x[t][2 * k + 1] = -INFINITY;
                            vst[t][k] = vlo[t][k] = 0.f;
                        }
            }
            // ---- the reference moves where a weight p s would leave its range
            // (or p b or p, where the step is very small)
            auto size = [&](int t, int k) {
                return fmaxf(fmaxf(vst[t][k], kStepFloor), fabsf(vlo[t][k]) * kLowPart);
            };
            float top = 0.f;
#pragma unroll
            for (int t = 0; t < XT; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    top = fmaxf(top, exp2_approx(fmaxf(x[t][2 * k], x[t][2 * k + 1])) * size(t, k));
            if (__any_sync(kFull, top > kWeightMax) || fresh) {
                float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                for (int t = 0; t < XT; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float lv = log2_approx(size(t, k));
                        t0 = fmaxf(t0, x[t][2 * k] + lv);
                        t1 = fmaxf(t1, x[t][2 * k + 1] + lv);
                    }
#pragma unroll
                for (int o = R == 4 ? 1 : R == 2 ? 2 : 4; o < 32; o <<= 1) {
                    t0 = fmaxf(t0, __shfl_xor_sync(kFull, t0, o));
                    t1 = fmaxf(t1, __shfl_xor_sync(kFull, t1, o));
                }
                // by how much; a column without a number keeps its reference
                const float s0 = t0 == -INFINITY ? 0.f : fresh ? t0 - kWeightNew : fmaxf(0.f, t0 - kWeightNew);
                const float s1 = t1 == -INFINITY ? 0.f : fresh ? t1 - kWeightNew : fmaxf(0.f, t1 - kWeightNew);
                const float f0 = fresh ? 0.f : exp2_approx(-s0), f1 = fresh ? 0.f : exp2_approx(-s1);
                fresh = false;
                m0 += s0;
                m1 += s1;
                l0 *= f0;
                l1 *= f1;
                lo0 *= f0;
                lo1 *= f1;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    acc[i][0] *= f0;
                    acc[i][1] *= f1;
                    acc[i][2] *= f0;
                    acc[i][3] *= f1;
                }
#pragma unroll
                for (int t = 0; t < XT; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        x[t][2 * k] -= s0;
                        x[t][2 * k + 1] -= s1;
                    }
            }
            // ---- weights, their sums, and the values' B operand
            uint32_t wh[XT][2], wl[SECOND ? XT : 1][2];
#pragma unroll
            for (int t = 0; t < XT; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float p0 = exp2_approx(x[t][2 * k]), p1 = exp2_approx(x[t][2 * k + 1]);
                    l0 += p0;
                    l1 += p1;
                    lo0 = fmaf(p0, vlo[t][k], lo0);
                    lo1 = fmaf(p1, vlo[t][k], lo1);
                    const float w0 = p0 * vst[t][k], w1 = p1 * vst[t][k];
                    const uint32_t pk = pack_f16(w0, w1);
                    const __half2 h = *reinterpret_cast<const __half2 *>(&pk);
                    wh[t][k] = movmatrix_trans(pk ^ odd_sign);
                    if constexpr (SECOND) {
                        wl[t][k] = movmatrix_trans(pack_f16(w0 - __low2float(h), w1 - __high2float(h)) ^ odd_sign);
                        // to the columns of the neighbouring copy
                        if constexpr (!F32) wl[t][k] = __shfl_xor_sync(kFull, wl[t][k], 4 * CW);
                    } else { // an even token's 7.5 w - 7.5 w', an odd one's 7.5 w + 7.5 w'
                        lo0 = fmaf(__low2float(h), centre, lo0);
                        lo1 = fmaf(__high2float(h), centre, lo1);
                    }
                }
            // ---- O^T += V^T (p s)^T
#pragma unroll
            for (int pair = 0; pair < NTILE / 2; ++pair) {
                uint32_t va[2][2][KW], bh[2][2], bl[2][2];
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    const int tile = 2 * pair + tt;
                    const uint8_t *tv = st + tile_at(tile, D / 2) + v_off;
                    lds<KW>(va[tt][0], tv);
                    lds<KW>(va[tt][1], tv + 4 * D);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const bool own = R == 1 || brep == tile;
                        bh[tt][k] = own ? wh[R == 1 ? tt : 0][k] : 0u;
                        if constexpr (F32)
                            bl[tt][k] = own ? wl[R == 1 ? tt : 0][k] : 0u;
                        else if constexpr (SECOND)
                            bh[tt][k] = brep == (tile ^ 1) ? wl[0][k] : bh[tt][k];
                    }
                }
#pragma unroll
                for (int i = 0; i < KW; ++i)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        float(&o)[4] = acc[2 * i + s];
                        uint32_t va4[2][4];
#pragma unroll
                        for (int tt = 0; tt < 2; ++tt) {
                            // the high halves are the odd tokens: 15 - n
                            const uint32_t wa = s ? va[tt][0][i] >> 8 : va[tt][0][i];
                            const uint32_t wb = s ? va[tt][1][i] >> 8 : va[tt][1][i];
                            va4[tt][0] = operand<F32>(and_xor(wa, 0x000f000fu, 0x000f0000u));
                            va4[tt][1] = operand<F32>(and_xor(wa, 0x00f000f0u, 0x00f00000u));
                            va4[tt][2] = operand<F32>(and_xor(wb, 0x000f000fu, 0x000f0000u));
                            va4[tt][3] = operand<F32>(and_xor(wb, 0x00f000f0u, 0x00f00000u));
                        }
                        if constexpr (F32) { // small part first, each sum added with rounding
                            float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int tt = 0; tt < 2; ++tt)
                                mma_f16(part, va4[tt][0], va4[tt][1], va4[tt][2], va4[tt][3], bl[tt][0], bl[tt][1]);
#pragma unroll
                            for (int tt = 0; tt < 2; ++tt)
                                mma_f16(part, va4[tt][0], va4[tt][1], va4[tt][2], va4[tt][3], bh[tt][0], bh[tt][1]);
#pragma unroll
                            for (int k = 0; k < 4; ++k) o[k] += part[k];
                        } else {
#pragma unroll
                            for (int tt = 0; tt < 2; ++tt)
                                mma_f16(o, va4[tt][0], va4[tt][1], va4[tt][2], va4[tt][3], bh[tt][0], bh[tt][1]);
                        }
                    }
            }
        }
        if (flags & kLast) mt = meta[at];
        __syncwarp(); // the slot is used up
        issue(at);
        ++at;
        if (++stage == nst) {
            stage = 0;
            at = warp * nst;
            phase ^= 1;
        }
        } while (!(flags & kLast));

        // ================= end of this CTA's share of the sequence =================
        const int kvh = mt.hg * hs + ch;
        left -= mt.blocks;
#pragma unroll
        for (int o = R == 4 ? 1 : R == 2 ? 2 : 4; o < 32; o <<= 1) {
            l0 += __shfl_xor_sync(kFull, l0, o);
            l1 += __shfl_xor_sync(kFull, l1, o);
            lo0 += __shfl_xor_sync(kFull, lo0, o);
            lo1 += __shfl_xor_sync(kFull, lo1, o);
        }
        if (fresh) m0 = m1 = -INFINITY; // no token of the share was summed
        // Codes of odd dims were 16 times those of even ones.  With copies, a
        // lane keeps one of its two columns (R = 4: and half of its dims) and
        // hands the rest to the lane that keeps those.
        constexpr int NV = 2 * DL / R;      // values of a lane
        constexpr int NH = R == 1 ? 2 : 1;  // heads of a lane
        float val[NV];
        const bool second = R > 1 && (R == 2 ? rep : rep & 1);
        const int head0 = R == 1 ? col : R == 2 ? col + rep : (rep & 1);
        const int dim0 = r * DL + (R == 4 ? (rep >> 1) * (DL / 2) : 0);
#pragma unroll
        for (int k = 0; k < DL; ++k) {
            const float sc = (k & 1) ? kCodeScale / kUnit / 16.f : kCodeScale / kUnit;
            const float v0 = acc[k >> 1][2 * (k & 1)] * sc, v1 = acc[k >> 1][2 * (k & 1) + 1] * sc;
            if constexpr (R == 1) {
                val[k] = v0;
                val[DL + k] = v1;
            } else {
                const float give = second ? v0 : v1, keep = second ? v1 : v0;
                const float sum = keep + __shfl_xor_sync(kFull, give, R == 2 ? 2 : 1);
                if constexpr (R == 2) {
                    val[k] = sum;
                } else {
                    acc[k >> 1][2 * (k & 1)] = sum;
                }
            }
        }
        if constexpr (R == 4) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const float lo_half = acc[k >> 1][2 * (k & 1)], hi_half = acc[(k + NV) >> 1][2 * (k & 1)];
                const float give = (rep & 2) ? lo_half : hi_half, keep = (rep & 2) ? hi_half : lo_half;
                val[k] = keep + __shfl_xor_sync(kFull, give, 2);
            }
        }
        float mh[NH], lh[NH], bh[NH];
        mh[0] = second ? m1 : m0;
        lh[0] = second ? l1 : l0;
        bh[0] = second ? lo1 : lo0;
        if constexpr (NH == 2) {
            mh[1] = m1;
            lh[1] = l1;
            bh[1] = lo1;
        }
        const size_t orow = ((size_t)mt.b * Hq + (size_t)kvh * G) * D;
        const long long segrow = (long long)mt.hg * B + mt.b;
        float *slot = a.part + ((size_t)(blockIdx.x + segrow) * hs + ch) * gm.slot_floats;
        const bool whole = (flags & kWhole) != 0;
        if (tw == 1) {
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                const int g = head0 + n;
                if (g >= G) continue;
                const float inv = 1.f / lh[n];
#pragma unroll
                for (int k = 0; k < NV / NH; k += 4) {
                    const float *v = val + n * (NV / NH) + k;
                    const float y0 = v[0] + bh[n], y1 = v[1] + bh[n], y2 = v[2] + bh[n], y3 = v[3] + bh[n];
                    if (whole) {
                        T *o = outp + orow + (size_t)g * D + dim0 + k;
                        if (bad)
                            store4(o, 0.f, 0.f, 0.f, 0.f);
                        else
                            store4(o, y0 * inv, y1 * inv, y2 * inv, y3 * inv);
                    } else {
                        *reinterpret_cast<float4 *>(slot + g * D + dim0 + k) = make_float4(y0, y1, y2, y3);
                    }
                }
                if (!whole && r == 0 && (R < 4 || rep < 2))
                    *reinterpret_cast<float2 *>(slot + G * D + 2 * g) = make_float2(mh[n], bad ? -INFINITY : lh[n]);
            }
        } else {
            // join the warps that share the head in shared memory
            if (r == 0 && (R < 4 || rep < 2)) {
#pragma unroll
                for (int n = 0; n < NH; ++n) {
                    s_m[warp][head0 + n] = mh[n];
                    s_l[warp][head0 + n] = bad ? -INFINITY : lh[n];
                    s_b[warp][head0 + n] = bh[n];
                }
            }
            float *mine = join + (size_t)warp * G * D;
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                if (head0 + n >= G) continue;
#pragma unroll
                for (int k = 0; k < NV / NH; k += 4) {
                    const float *v = val + n * (NV / NH) + k;
                    *reinterpret_cast<float4 *>(mine + (head0 + n) * D + dim0 + k) = make_float4(v[0], v[1], v[2], v[3]);
                }
            }
            if (!sync()) return;
            for (int e = gtid; e < G * (D / 4); e += gthreads) {
                const int g = e / (D / 4), d = e % (D / 4) * 4;
                float M = -INFINITY;
#pragma unroll 4
                for (int t = 0; t < tw; ++t) M = fmaxf(M, s_m[t * hs + ch][g]);
                float l = 0.f, low = 0.f;
                bool refused = false; // a block or the length was
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int t = 0; t < tw; ++t) {
                    const int w = t * hs + ch;
                    const float f = M == -INFINITY ? 1.f : exp2_approx(s_m[w][g] - M);
                    refused |= s_l[w][g] == -INFINITY;
                    l = fmaf(s_l[w][g], f, l);
                    low = fmaf(s_b[w][g], f, low);
                    const float4 x = *reinterpret_cast<const float4 *>(join + (size_t)w * G * D + g * D + d);
                    o.x = fmaf(x.x, f, o.x);
                    o.y = fmaf(x.y, f, o.y);
                    o.z = fmaf(x.z, f, o.z);
                    o.w = fmaf(x.w, f, o.w);
                }
                o.x += low;
                o.y += low;
                o.z += low;
                o.w += low;
                if (whole) {
                    const float inv = 1.f / l;
                    if (refused)
                        store4(outp + orow + (size_t)g * D + d, 0.f, 0.f, 0.f, 0.f);
                    else
                        store4(outp + orow + (size_t)g * D + d, o.x * inv, o.y * inv, o.z * inv, o.w * inv);
                } else {
                    *reinterpret_cast<float4 *>(slot + g * D + d) = o;
                    if (d == 0)
                        *reinterpret_cast<float2 *>(slot + G * D + 2 * g) = make_float2(M, refused ? -INFINITY : l);
                }
            }
        }
        if (!whole) {
            // The partial is ordered before the ticket by the barrier, and
            // the ticket is an acquire-release at GPU scope.
            const uint32_t pos = mt.hg * cblk + mt.sb + cs * (mt.b + 1); // of the sequence's first block
            const int cfirst = split.range_of(pos), nseg = split.range_of(pos + mt.nblk - 1) - cfirst + 1;
            if (!sync()) return;
            int32_t *ticket = a.tickets + (size_t)mt.b * Hkv + kvh;
            int last = 0;
            if (gtid == 0) {
                int old;
                asm volatile("atom.add.acq_rel.gpu.s32 %0, [%1], 1;" : "=r"(old) : "l"(ticket) : "memory");
                last = old == nseg - 1;
                if (last) *ticket = 0;
                s_last[ch] = last;
            }
            if (!sync()) return;
            last = tw == 1 ? __shfl_sync(kFull, last, 0) : s_last[ch];
            if (last) {
                const float *first = a.part + ((size_t)(cfirst + segrow) * hs + ch) * gm.slot_floats;
                const size_t step = (size_t)hs * gm.slot_floats;
                if (CW * D / 128 > 1 && G * D > tw * 128) // more rows than warps
                    fold<D, T, 2>(first, step, nseg, G, ct, tw, outp + orow);
                else
                    fold<D, T, 1>(first, step, nseg, G, ct, tw, outp + orow);
            }
        }
        if (!sync()) return; // the join buffers are free again
    }
}

constexpr int kMaxDev = 64;
constexpr size_t kSmemPerCta = 210 * 1024; // of 227, beside the static arrays

template <int D, int R, typename T>
size_t smem_bytes(int ncw, int tw, int group)
{
    return (size_t)ncw * kSlots * (Slot<D, R, T>::bytes + 8 + sizeof(Meta)) + 8 +
           (tw > 1 ? (size_t)ncw * group * D * 4 : 0);
}

struct Plan {
    DecodeQ4Geom gm;
    int ctas;
    size_t smem;
};

template <int D, int BS, int R, typename T>
int make_plan(int batch, int num_kv_heads, int group, Plan *p)
{
    const int sms = num_sms();
    if (sms <= 0) return PA_ERR_DEVICE;
    p->ctas = sms;
    // Heads of a CTA: the most that leave a sequence cut into at most
    // kMaxParts parts by the CTAs' ranges.  With fewer rows than that, the
    // warps of a CTA share a head's tokens and join in shared memory.
    int hs = 1;
    for (int h = 2; h <= kMaxWarps && h <= num_kv_heads; ++h)
        if (num_kv_heads % h == 0 && (long long)kMaxParts * batch * num_kv_heads >= (long long)p->ctas * h) hs = h;
    const int tw = kMaxWarps / hs, ncw = hs * tw;
    static_assert(kMaxWarps * (kSlots * (Slot<D, R, T>::bytes + 8 + sizeof(Meta)) + 8 / R * D * 4) + 8 <=
                  kSmemPerCta, "a full CTA's rings and join buffers fit");
    p->smem = smem_bytes<D, R, T>(ncw, tw, group);
    static int raised[kMaxDev];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return PA_ERR_DEVICE;
    if (!__atomic_load_n(&raised[dev], __ATOMIC_ACQUIRE)) {
        const cudaError_t e = cudaFuncSetAttribute(
            decode_q4_kernel<D, BS, R, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemPerCta);
        if (e != cudaSuccess) return launch_status(e);
        __atomic_store_n(&raised[dev], 1, __ATOMIC_RELEASE);
    }
    p->gm.hs = hs;
    p->gm.tw = tw;
    p->gm.head_groups = num_kv_heads / hs;
    p->gm.slot_floats = group * D + 16;
    return PA_OK;
}

size_t plan_workspace(const Plan &p, int batch)
{
    return kTicketRegionBytes + ((size_t)p.ctas + (size_t)p.gm.head_groups * batch) * p.gm.hs * p.gm.slot_floats * 4;
}

template <int D, int BS, int R, typename T>
int plan_and_launch(const DecodeQ4Args *a, int batch, int num_kv_heads, int group, size_t have, size_t *need,
                    cudaStream_t s)
{
    Plan p;
    const int rc = make_plan<D, BS, R, T>(batch, num_kv_heads, group, &p);
    if (rc != PA_OK) return rc;
    *need = plan_workspace(p, batch);
    if (a == nullptr) return PA_OK;
    if (have < *need) return PA_ERR_WORKSPACE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.ctas);
    cfg.blockDim = dim3(p.gm.hs * p.gm.tw * 32);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, decode_q4_kernel<D, BS, R, T>, *a, p.gm));
}

// Copies of the head group in the products' columns: as many as fit, up to
// the tiles of a stage.  1024 sequences with D 64 and one head a kv head: 234 us
// with four copies, 288 with two.  256 sequences with D 128 and four heads a kv head:
// 116 us with two, 121.5 with none.
// Four copies (64-token stages) are for head_dim 64 only: at 128 their rings
// would not fit 16 warps.
template <int D, int BS, typename T>
int by_copies(const DecodeQ4Args *a, int batch, int num_kv_heads, int group, size_t have, size_t *need, cudaStream_t s)
{
    if constexpr (D == 64) {
        if (group <= 2) return plan_and_launch<D, BS, 4, T>(a, batch, num_kv_heads, group, have, need, s);
    }
    if (group <= 4) return plan_and_launch<D, BS, 2, T>(a, batch, num_kv_heads, group, have, need, s);
    return plan_and_launch<D, BS, 1, T>(a, batch, num_kv_heads, group, have, need, s);
}

int dispatch(const DecodeQ4Args *a, int batch, int num_kv_heads, int group, int d, int bs, bool f32, size_t have,
             size_t *need, cudaStream_t s)
{
#define PA_Q4(D_, BS_)                                                                                        \
    if (d == D_ && bs == BS_)                                                                                 \
        return f32 ? by_copies<D_, BS_, float>(a, batch, num_kv_heads, group, have, need, s)                  \
                   : by_copies<D_, BS_, __nv_bfloat16>(a, batch, num_kv_heads, group, have, need, s);
    PA_Q4(64, 16)
    PA_Q4(64, 32)
    PA_Q4(128, 16)
    PA_Q4(128, 32)
#undef PA_Q4
    return PA_ERR_UNSUPPORTED;
}

}  // namespace

size_t decode_q4_workspace(int batch, int num_heads, int num_kv_heads, int head_dim, int block_size, bool f32)
{
    size_t need = 0;
    const int rc = dispatch(nullptr, batch, num_kv_heads, num_heads / num_kv_heads, head_dim, block_size, f32, 0,
                            &need, nullptr);
    return rc == PA_OK ? need : 0;
}

int decode_q4_launch(const DecodeQ4Args &a, bool f32, size_t workspace_bytes, cudaStream_t s)
{
    size_t need = 0;
    return dispatch(&a, a.batch, a.num_kv_heads, a.group, a.head_dim, a.block_size, f32, workspace_bytes, &need, s);
}

}  // namespace pa
