// The 4-bit pool's cache update (quantise and scatter) and its read-back
// (gather and dequantise).  Formulas and layout: include/pa.h, "The 4-bit
// pool".
#include "pa_internal.h"
#include "pa_q4.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;

// ------------------------------------------------------------------ update
// A CTA looks at kRows chunk rows.  A warp takes one of them, or two where they
// are neighbours in one token pair of a block, and `heads` of its kv heads:
// eight lanes a row, K and V of the first token, then of the second.  Two
// tokens of a pair share the words of V, so a pair's V is written as whole
// words, each token's lanes writing half of them; a lone token writes its halves
// of the words.
//
// What bounds it: moving the bytes (a bf16 chunk's, and a quarter of them again)
// on one side, instructions on the other.  33K rows of 8 bf16 heads x 128 dims
// (174 MB): 34 us, 5.1 TB/s; of fp32 (306 MB): 51 us, 6.0 TB/s.  With 16 lanes a
// row, a pair's rows one after the other, bf16 took 44 us and 289 instructions for four
// rows of 128; now 178, because a row's scale is computed once for 16 elements a lane
// and arithmetic goes in pairs.
constexpr int kRows = 16;
// Heads whose rows are held or on their way.  The same chunk with the read-back
// behind it: 82 us with 1 (no loads beside the sums), 76 with 2, 75 with 3.
constexpr int kAhead = 2;
// Warps that an update is spread over, at least, before a warp takes several
// heads: about half of what the SMs hold.  A decode step's few rows then run a
// head a warp, and a large chunk reads its slots once for all heads.
constexpr int kMinWarps = 4096;
template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 5)
    update_q4_kernel(const CacheQ4Args a, const int heads, const int bs_shift)
{
    constexpr int NC = D / 64;
    const int lane = threadIdx.x & 31, l = lane & 7;
    const bool value = lane & 16, second = lane & 8;
    grid_dep_trigger();
    grid_dep_wait();
    // Rows that lead: all but the odd token of a pair whose even one stands
    // before it in the chunk, and padding.
    const int row0 = blockIdx.x * kRows, mine = row0 + (lane & (kRows - 1));
    const int slot_l = mine < a.total ? a.slot_map[mine] : -1;
    const int before = mine > 0 && mine < a.total ? a.slot_map[mine - 1] : -1;
    const int after = mine + 1 < a.total ? a.slot_map[mine + 1] : -1;
    const bool inside = slot_l < a.num_blocks << bs_shift;
    if (!inside && lane < kRows && threadIdx.x < 32 && blockIdx.y == 0) flag_error(a.dev_err, PA_DEVERR_BAD_BLOCK);
    const bool leads = lane < kRows && slot_l >= 0 && inside && !((slot_l & 1) && before == slot_l - 1);
    const bool paired = !(slot_l & 1) && after == slot_l + 1;
    const unsigned todo = __ballot_sync(kFull, leads), pairs = __ballot_sync(kFull, paired);
    const int rank = __popc(todo & ((1u << lane) - 1u));
    const int hkv = a.num_kv_heads, bs = 1 << bs_shift;
    const int h0 = blockIdx.y * heads, n = min(hkv, h0 + heads) - h0;
    const int rec_bytes = q4_record_bytes(D, bs);
    for (int k = threadIdx.x >> 5; k < __popc(todo); k += kThreads / 32) {
        // the warp's k-th leading row
        const int i = __ffs(__ballot_sync(kFull, leads && rank == k)) - 1;
        const int slot = __shfl_sync(kFull, slot_l, i), t = slot & (bs - 1);
        const bool two = pairs >> i & 1, mute = second && !two;
        uint8_t *rec = static_cast<uint8_t *>(a.kv_cache) + ((size_t)(slot >> bs_shift) * hkv + h0) * rec_bytes;
        const T *src = static_cast<const T *>(value ? a.v : a.k) +
                       ((size_t)(row0 + i + (second && two)) * hkv + h0) * D + l * 8;
        // of a pair's V, the first token's lanes write the words of chunk 0 (D = 64:
        // of their first unit), the second token's those of chunk 1
        uint8_t *dst = rec;
        if (!value)
            dst += (t + (second && two)) * (D / 2) + l * 4;
        else if (two)
            dst += q4_v_offset(D, bs) + 2 * q4_v_unit<D>(t, 2 * l + (second ? (NC == 2 ? 16 : 1) : 0));
        else
            dst += q4_v_offset(D, bs) + 2 * q4_v_unit<D>(t, 2 * l);
        // of a lone token's V: from the units of chunk 0 to those of chunk 1
        const int chunk = q4_v_unit<D>(t, NC == 2 ? 16 + 2 * l : 2 * l) - q4_v_unit<D>(t, 2 * l);
        uint32_t *scale = reinterpret_cast<uint32_t *>(rec + q4_scale_offset(D, bs) + (t + second) * 8 + (value ? 4 : 0));
        Q4Row<T, NC> rows[kAhead];
#pragma unroll
        for (int p = 0; p < kAhead; ++p, src += D)
            if (p < n) rows[p].load(src);
        int left = n;
        for (;;) {
#pragma unroll
            for (int p = 0; p < kAhead; ++p) {
                if (left-- <= 0) break;
                Q4Scale s;
                uint32_t c[NC];
                q4_quantise(rows[p], s, c);
                if (left >= kAhead) rows[p].load(src);
                src += D;
                if (two) {
                    const uint32_t got = __shfl_xor_sync(kFull, NC == 2 && !second ? c[NC - 1] : c[0], 8);
                    if (!value) {
#pragma unroll
                        for (int u = 0; u < NC; ++u) *reinterpret_cast<uint32_t *>(dst + 32 * u) = c[u];
                    } else { // the first token in the low halves
                        const uint32_t even = second ? got : c[0], odd = second ? c[NC - 1] : got;
                        const uint32_t w0 = __byte_perm(even, odd, 0x5410), w1 = __byte_perm(even, odd, 0x7632);
                        if constexpr (NC == 2)
                            *reinterpret_cast<uint2 *>(dst) = make_uint2(w0, w1);
                        else
                            *reinterpret_cast<uint32_t *>(dst) = second ? w1 : w0;
                    }
                } else if (!mute) {
                    if (!value) {
#pragma unroll
                        for (int u = 0; u < NC; ++u) *reinterpret_cast<uint32_t *>(dst + 32 * u) = c[u];
                    } else {
                        uint16_t *unit = reinterpret_cast<uint16_t *>(dst);
#pragma unroll
                        for (int u = 0; u < NC; ++u) {
                            unit[u * chunk] = (uint16_t)c[u];
                            unit[u * chunk + 2] = (uint16_t)(c[u] >> 16);
                        }
                    }
                }
                if (l == 0 && !mute) *scale = q4_pack_scale(s);
                dst += rec_bytes;
                scale += rec_bytes / 4;
            }
            if (left <= 0) break;
        }
    }
}

// ------------------------------------------------------------------ gather
// What bounds it: writing the rows.  145K rows of 8 bf16 heads x 128 dims (750
// MB): 116 us, 6.5 TB/s, 95% of a copy's rate; fp32 208 us, the same rate.  fp32, 24K rows of 6 heads x 64
// dims (84 MB): 18 us, 4.6 TB/s; with 8 values a thread, whose two stores leave
// every other 16 bytes to the next instruction, it was 24.5 us.
//
// Largest r in [0, n) with off(r) <= x, off(r) = cu[r] / bs + r (never
// decreasing), by the whole warp: 32 probes a step.
__device__ __forceinline__ int tile_owner(const int32_t *cu, int n, int x, int bs_shift)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n; // the answer is in [lo, lo + len)
    while (len > 1) {
        const int step = (len + 31) / 32, r = lo + lane * step;
        const bool below = lane * step < len && (cu[r] >> bs_shift) + r <= x;
        const int last = 31 - __clz((int)(__ballot_sync(kFull, below) | 1u));
        const int end = lo + len;
        lo += last * step;
        len = min(step, end - lo);
    }
    return lo;
}

// The cumulative lengths start at 0, never decrease and end inside k_full
// (one block looks at all of them).
__device__ __forceinline__ void check_cu(const CacheQ4Args &a)
{
    bool bad = threadIdx.x == 0 && (a.cu_k[0] != 0 || a.cu_k[a.batch] > a.total);
    for (int b = threadIdx.x; b < a.batch; b += blockDim.x)
        bad = bad || a.cu_k[b + 1] < a.cu_k[b];
    if (bad) flag_error(a.dev_err, PA_DEVERR_BAD_CU);
}

// N codes of 4 bits as values, rounded once; 2^23 + n is made of bits.
template <int N>
__device__ __forceinline__ void unpack(float (&v)[N], uint32_t c, float step, float low)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = fmaf(__uint_as_float(((c >> (4 * i)) & 15u) | 0x4b000000u) - 8388608.f, step, low);
}
// 16 bytes of values; they are read again, if at all, by another kernel.
__device__ __forceinline__ void store16(float *p, const float (&v)[4])
{
    __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
}
__device__ __forceinline__ void store16(__nv_bfloat16 *p, const float (&v)[8])
{
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                                    pack_bf16(v[6], v[7])));
}

// A CTA takes one block of one request: tile i belongs to the last request r
// with cu[r] / bs + r <= i (every request has at least as many tiles as
// blocks).  A thread turns N dims of a token pair of one head, K and V, into
// four stores of 16 bytes; neighbours in dims, then heads, are neighbours in the
// packed rows, so a warp stores whole sectors.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads) gather_q4_kernel(const CacheQ4Args a, const int bs_shift)
{
    constexpr int N = 16 / sizeof(T), I = D / N;
    grid_dep_trigger();
    grid_dep_wait();
    if (blockIdx.x == 0) check_cu(a);
    const int bs = 1 << bs_shift, hkv = a.num_kv_heads;
    const int b = tile_owner(a.cu_k, a.batch, blockIdx.x, bs_shift);
    const int k0 = a.cu_k[b], k1 = min(a.cu_k[b + 1], a.total);
    const int lb = (int)blockIdx.x - (k0 >> bs_shift) - b;
    if (k0 < 0 || lb < 0 || (long long)lb << bs_shift >= k1 - k0) return; // no tile, or flagged by check_cu
    const int pos0 = lb << bs_shift, rows = min(bs, k1 - k0 - pos0);
    int blk = -1;
    if (lb >= a.max_blocks_per_seq) {
        if (threadIdx.x == 0) flag_error(a.dev_err, PA_DEVERR_OVERFLOW);
    } else {
        blk = a.block_table[(size_t)b * a.max_blocks_per_seq + lb];
        if (blk < 0 || blk >= a.num_blocks) {
            if (threadIdx.x == 0) flag_error(a.dev_err, PA_DEVERR_BAD_BLOCK);
            blk = -1;
        }
    }
    const int rec_bytes = q4_record_bytes(D, bs);
    const uint8_t *base = static_cast<const uint8_t *>(a.kv_cache) + (size_t)(blk < 0 ? 0 : blk) * hkv * rec_bytes;
    const size_t row_elts = (size_t)hkv * D;
    const size_t out0 = (size_t)(k0 + pos0) * row_elts;
    T *ko = static_cast<T *>(a.k_full) + out0, *vo = static_cast<T *>(a.v_full) + out0;
    const int items = ((rows + 1) >> 1) * hkv * I;
#pragma unroll 2
    for (int e = threadIdx.x; e < items; e += kThreads) {
        const int i = e % I, hp = e / I, h = hp % hkv, p = hp / hkv;
        uint32_t kc[2] = {0u, 0u}, vc[2] = {0u, 0u};
        uint4 sc = make_uint4(0u, 0u, 0u, 0u);
        if (blk >= 0) {
            const uint8_t *rec = base + (size_t)h * rec_bytes;
            const uint8_t *kr = rec + p * D + i * (N / 2);
            const uint8_t *vr = rec + q4_v_offset(D, bs) + 2 * q4_v_unit<D>(2 * p, i * (N / 4));
            if constexpr (N == 8) {
                kc[0] = *reinterpret_cast<const uint32_t *>(kr);
                kc[1] = *reinterpret_cast<const uint32_t *>(kr + D / 2);
                const uint2 w = *reinterpret_cast<const uint2 *>(vr);
                vc[0] = __byte_perm(w.x, w.y, 0x5410);
                vc[1] = __byte_perm(w.x, w.y, 0x7632);
            } else {
                kc[0] = *reinterpret_cast<const uint16_t *>(kr);
                kc[1] = *reinterpret_cast<const uint16_t *>(kr + D / 2);
                const uint32_t w = *reinterpret_cast<const uint32_t *>(vr);
                vc[0] = w & 0xffffu;
                vc[1] = w >> 16;
            }
            sc = *reinterpret_cast<const uint4 *>(rec + q4_scale_offset(D, bs) + p * 16);
        }
        const size_t o = (size_t)(2 * p) * row_elts + h * D + i * N;
        float v[N];
        unpack<N>(v, kc[0], bf16_lo(sc.x), bf16_hi(sc.x));
        store16(ko + o, v);
        unpack<N>(v, vc[0], bf16_lo(sc.y), bf16_hi(sc.y));
        store16(vo + o, v);
        if (2 * p + 1 < rows) {
            unpack<N>(v, kc[1], bf16_lo(sc.z), bf16_hi(sc.z));
            store16(ko + o + row_elts, v);
            unpack<N>(v, vc[1], bf16_lo(sc.w), bf16_hi(sc.w));
            store16(vo + o + row_elts, v);
        }
    }
}

// Launches that may start while the kernel before them ends; they wait for it
// before they read anything.
template <typename... A>
int launch_after(void (*kernel)(A...), dim3 grid, cudaStream_t s, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, args...));
}

template <int D, typename T>
int launch(const CacheQ4Args &a, bool gather, cudaStream_t s)
{
    const int shift = a.block_size == 32 ? 5 : 4;
    if (gather) return launch_after(gather_q4_kernel<D, T>, dim3((a.total >> shift) + a.batch), s, a, shift);
    // heads of a warp: few rows are spread over more warps
    const int hkv = a.num_kv_heads;
    int heads = (int)min((long long)hkv, max(1ll, (long long)a.total * hkv / kMinWarps));
    if (hkv / heads > 65535) heads = (hkv + 65534) / 65535;
    const unsigned gx = ((unsigned)a.total + kRows - 1) / kRows;
    return launch_after(update_q4_kernel<D, T>, dim3(gx, (hkv + heads - 1) / heads), s, a, heads, shift);
}

}  // namespace

int cache_q4_launch(const CacheQ4Args &a, bool f32, bool gather, cudaStream_t s)
{
    if (a.head_dim == 64) return f32 ? launch<64, float>(a, gather, s) : launch<64, __nv_bfloat16>(a, gather, s);
    return f32 ? launch<128, float>(a, gather, s) : launch<128, __nv_bfloat16>(a, gather, s);
}

}  // namespace pa
