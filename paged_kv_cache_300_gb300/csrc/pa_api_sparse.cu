// C ABI of the rotary calls and of block-sparse attention: argument checks and
// dispatch.  As in pa_api.cu nothing here allocates device memory or synchronises,
// and a refused call has launched nothing.
#include "pa_internal.h"

#include <math.h>

using namespace pa;

namespace {

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A token's rows `stride` elements apart: whole 16-byte pieces; outputs do not overlap.
bool stride_ok(long long stride, int heads, int head_dim, int size, bool output)
{
    if (stride < 0 || stride > (1ll << 40) || stride * size % 16 != 0) return false;
    return !output || stride >= (long long)heads * head_dim;
}

// What the two rotary calls share: sizes, the table, the axes.
int check_rotary(RotaryArgs *a, int head_dim, int num_axes, const uint8_t *pair_axis, pa_dtype dtype)
{
    if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_DTYPE;
    if (a->tokens < 0 || a->num_heads < 0 || a->num_kv_heads < 0 || head_dim <= 0 || a->rotary_dim < 0 ||
        a->rotary_dim > head_dim)
        return PA_ERR_SHAPE;
    if ((head_dim != 64 && head_dim != 128) || a->rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (a->rotary_dim == 0) return PA_OK;
    if (a->max_position <= 0 || num_axes <= 0) return PA_ERR_SHAPE;
    if (num_axes > 4) return PA_ERR_UNSUPPORTED;
    if (num_axes > 1 && pair_axis == nullptr) return PA_ERR_NULL;
    for (int i = 0; pair_axis != nullptr && i < a->rotary_dim / 2; ++i) {
        if (pair_axis[i] >= num_axes) return PA_ERR_SHAPE;
        a->pair_axis[i / 32] |= (unsigned long long)pair_axis[i] << (2 * (i % 32));
    }
    if (a->tokens == 0) return PA_OK;
    if (!a->positions || !a->cos_sin) return PA_ERR_NULL;
    if (!aligned(a->positions, 4) || !aligned(a->cos_sin, 16)) return PA_ERR_SHAPE;
    return PA_OK;
}

// What the two calls of block-sparse attention share.
int check_rows(const void *cu, int batch, int total_q, int num_heads, int num_kv_heads, int head_dim, int num_blocks,
               int block_size, int max_blocks_per_seq, int top_k, pa_dtype dtype)
{
    if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_DTYPE;
    if (batch < 0 || total_q < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks <= 0 ||
        block_size <= 0 || max_blocks_per_seq <= 0 || top_k <= 0 || num_heads % num_kv_heads != 0)
        return PA_ERR_SHAPE;
    if (cu == nullptr && total_q != batch) return PA_ERR_SHAPE;
    if ((head_dim != 64 && head_dim != 128) || num_heads / num_kv_heads > 8) return PA_ERR_UNSUPPORTED;
    // rows of the pool and positions are 32-bit numbers, and so is the grid, of 16 CTAs a row at most
    if ((long long)num_blocks * block_size >= 1ll << 31 || (long long)max_blocks_per_seq * block_size >= 1ll << 31)
        return PA_ERR_UNSUPPORTED;
    if ((long long)total_q * num_kv_heads >= 1ll << 27 || top_k > 1 << 20) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

}  // namespace

extern "C" {

int pa_rotary(const void *q, const void *k, const int32_t *positions, const float *cos_sin,
              void *q_out, void *k_out, int tokens, int num_heads, int num_kv_heads, int head_dim,
              int rotary_dim, int max_position, int num_axes, const uint8_t *pair_axis,
              int interleaved, long long q_stride, long long k_stride, long long q_out_stride,
              long long k_out_stride, pa_dtype dtype, int32_t *dev_err, void *stream)
{
    RotaryArgs a{};
    a.q = q;
    a.k = k;
    a.q_out = q_out;
    a.k_out = k_out;
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.dev_err = dev_err;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.q_out_stride = q_out_stride;
    a.k_out_stride = k_out_stride;
    a.tokens = tokens;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.rotary_dim = rotary_dim;
    a.max_position = max_position;
    const int rc = check_rotary(&a, head_dim, num_axes, pair_axis, dtype);
    if (rc != PA_OK) return rc;
    if (rotary_dim == 0) return PA_ERR_SHAPE;
    const int size = dtype == PA_F32 ? 4 : 2;
    if (!stride_ok(q_stride, num_heads, head_dim, size, false) || !stride_ok(q_out_stride, num_heads, head_dim, size, true) ||
        !stride_ok(k_stride, num_kv_heads, head_dim, size, false) ||
        !stride_ok(k_out_stride, num_kv_heads, head_dim, size, true))
        return PA_ERR_SHAPE;
    if (tokens == 0 || num_heads + num_kv_heads == 0) return PA_OK;
    if ((num_heads > 0 && (!q || !q_out)) || (num_kv_heads > 0 && (!k || !k_out))) return PA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16)) return PA_ERR_SHAPE;
    return rotary_launch(a, num_axes, head_dim, dtype == PA_F32, interleaved != 0, false, static_cast<cudaStream_t>(stream));
}

int pa_cache_append_rotary(const void *q, const void *k, const void *v, const int32_t *slot_map,
                           void *k_cache, void *v_cache, void *bounds, const int32_t *positions,
                           const float *cos_sin, void *q_out, int tokens, int num_heads,
                           int num_kv_heads, int head_dim, int rotary_dim, int max_position,
                           int num_axes, const uint8_t *pair_axis, int interleaved,
                           long long q_stride, long long k_stride, long long v_stride,
                           long long q_out_stride, int num_blocks, int block_size, pa_dtype dtype,
                           int32_t *dev_err, void *stream)
{
    RotaryArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.k_out = k_cache;
    a.v_out = v_cache;
    a.bounds = bounds;
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.slot_map = slot_map;
    a.dev_err = dev_err;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out_stride = q_out_stride;
    a.tokens = tokens;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.rotary_dim = rotary_dim;
    a.max_position = max_position;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    const int rc = check_rotary(&a, head_dim, num_axes, pair_axis, dtype);
    if (rc != PA_OK) return rc;
    if (num_kv_heads == 0 || num_blocks <= 0 || block_size <= 0) return PA_ERR_SHAPE;
    if ((long long)num_blocks * block_size >= 1ll << 31) return PA_ERR_UNSUPPORTED;
    const int size = dtype == PA_F32 ? 4 : 2;
    if (!stride_ok(q_stride, num_heads, head_dim, size, false) || !stride_ok(q_out_stride, num_heads, head_dim, size, true) ||
        !stride_ok(k_stride, num_kv_heads, head_dim, size, false) || !stride_ok(v_stride, num_kv_heads, head_dim, size, false))
        return PA_ERR_SHAPE;
    if (tokens == 0) return PA_OK;
    if (!k || !v || !slot_map || !k_cache || !v_cache || (num_heads > 0 && (!q || !q_out))) return PA_ERR_NULL;
    for (const void *p : {q, k, v, (const void *)q_out, (const void *)k_cache, (const void *)v_cache, (const void *)bounds})
        if (!aligned(p, 16)) return PA_ERR_SHAPE;
    if (!aligned(slot_map, 4)) return PA_ERR_SHAPE;
    return rotary_launch(a, rotary_dim == 0 ? 0 : num_axes, head_dim, dtype == PA_F32, interleaved != 0, true,
                         static_cast<cudaStream_t>(stream));
}

int pa_select_blocks(const void *q, const void *bounds, const int32_t *block_table,
                     const int32_t *seqlens_k, const int32_t *cu_seq_lens_q, int32_t *selected,
                     int batch, int total_q, int num_heads, int num_kv_heads, int head_dim,
                     int num_blocks, int block_size, int max_blocks_per_seq, int top_k,
                     int first_blocks, int last_blocks, pa_dtype dtype, int32_t *dev_err,
                     void *stream)
{
    const int rc = check_rows(cu_seq_lens_q, batch, total_q, num_heads, num_kv_heads, head_dim, num_blocks, block_size,
                              max_blocks_per_seq, top_k, dtype);
    if (rc != PA_OK) return rc;
    if (first_blocks < 0 || last_blocks < 0 || (long long)first_blocks + last_blocks > top_k) return PA_ERR_SHAPE;
    if (max_blocks_per_seq > kSelectMaxBlocks) return PA_ERR_UNSUPPORTED;
    if (batch == 0 || total_q == 0) return PA_OK;
    if (!q || !bounds || !block_table || !seqlens_k || !selected) return PA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(block_table, 4) || !aligned(seqlens_k, 4) ||
        !aligned(cu_seq_lens_q, 4) || !aligned(selected, 4))
        return PA_ERR_SHAPE;
    SelectArgs a{};
    a.q = q;
    a.bounds = bounds;
    a.block_table = block_table;
    a.seqlens_k = seqlens_k;
    a.cu_q = cu_seq_lens_q;
    a.selected = selected;
    a.dev_err = dev_err;
    a.batch = batch;
    a.total_q = total_q;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.group = num_heads / num_kv_heads;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.top_k = top_k;
    a.first = first_blocks;
    a.last = last_blocks;
    return select_launch(a, head_dim, dtype == PA_F32, static_cast<cudaStream_t>(stream));
}

int pa_sparse(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_table,
              const int32_t *seqlens_k, const int32_t *cu_seq_lens_q, const int32_t *selected,
              void *out, int batch, int total_q, int num_heads, int num_kv_heads, int head_dim,
              int num_blocks, int block_size, int max_blocks_per_seq, int top_k, pa_dtype dtype,
              float softmax_scale, int32_t *dev_err, void *stream)
{
    const int rc = check_rows(cu_seq_lens_q, batch, total_q, num_heads, num_kv_heads, head_dim, num_blocks, block_size,
                              max_blocks_per_seq, top_k, dtype);
    if (rc != PA_OK) return rc;
    if (dtype == PA_BF16 && block_size % kSparseUnit != 0) return PA_ERR_UNSUPPORTED;
    if ((long long)top_k * block_size >= 1ll << 30) return PA_ERR_UNSUPPORTED; // tokens of a list in 32 bits
    if (batch == 0 || total_q == 0) return PA_OK;
    if (!q || !k_cache || !v_cache || !block_table || !seqlens_k || !selected || !out) return PA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(block_table, 4) ||
        !aligned(seqlens_k, 4) || !aligned(cu_seq_lens_q, 4) || !aligned(selected, 4))
        return PA_ERR_SHAPE;
    SparseArgs a{};
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_table = block_table;
    a.seqlens_k = seqlens_k;
    a.cu_q = cu_seq_lens_q;
    a.selected = selected;
    a.out = out;
    a.dev_err = dev_err;
    a.batch = batch;
    a.total_q = total_q;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.group = num_heads / num_kv_heads;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.top_k = top_k;
    const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)head_dim);
    a.scale_log2 = scale * 1.4426950408889634f;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == PA_F32) return sparse_f32_launch(a, head_dim, s);
    CUtensorMap tm_k, tm_v;
    const uint64_t rows = (uint64_t)num_blocks * block_size;
    int e = cached_unit_map(&tm_k, k_cache, rows, num_kv_heads, head_dim, kSparseUnit, 1);
    if (e == PA_OK) e = cached_unit_map(&tm_v, v_cache, rows, num_kv_heads, head_dim, kSparseUnit, 1);
    if (e != PA_OK) return e;
    return sparse_bf16_launch(a, head_dim, tm_k, tm_v, s);
}

}  // extern "C"
