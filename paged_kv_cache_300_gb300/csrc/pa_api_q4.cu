// C ABI of the 4-bit pool and of the GPU-built block tables: argument checks
// and dispatch.  As in pa_api.cu nothing here allocates device memory or
// synchronises, and a refused call has launched nothing.
#include "pa_internal.h"
#include "pa_q4.cuh"

#include <math.h>

using namespace pa;

namespace {

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_pool(int num_kv_heads, int head_dim, int num_blocks, int block_size)
{
    if (num_kv_heads <= 0 || head_dim <= 0 || num_blocks <= 0 || block_size <= 0) return PA_ERR_SHAPE;
    if ((head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32))
        return PA_ERR_UNSUPPORTED;
    if ((long long)num_blocks * block_size >= (1ll << 31)) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

}  // namespace

extern "C" {

size_t pa_q4_block_bytes(int num_kv_heads, int head_dim, int block_size)
{
    if (check_pool(num_kv_heads, head_dim, 1, block_size) != PA_OK) return 0;
    return (size_t)num_kv_heads * q4_record_bytes(head_dim, block_size);
}

int pa_cache_update_q4(const void *k_chunk, const void *v_chunk, const int32_t *slot_map,
                       void *kv_cache, int total_q, int num_kv_heads, int head_dim,
                       int num_blocks, int block_size, pa_dtype dtype, int32_t *dev_err,
                       void *stream)
{
    if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_DTYPE;
    const int rc = check_pool(num_kv_heads, head_dim, num_blocks, block_size);
    if (rc != PA_OK) return rc;
    if (total_q < 0) return PA_ERR_SHAPE;
    // rows are counted in 32 bits, sixteen at a time
    if ((long long)total_q * num_kv_heads >= (1ll << 31) - 64) return PA_ERR_UNSUPPORTED;
    if (total_q == 0) return PA_OK;
    if (!k_chunk || !v_chunk || !slot_map || !kv_cache) return PA_ERR_NULL;
    if (!aligned(k_chunk, 16) || !aligned(v_chunk, 16) || !aligned(kv_cache, 16) || !aligned(slot_map, 4))
        return PA_ERR_SHAPE;
    CacheQ4Args a{};
    a.k = k_chunk;
    a.v = v_chunk;
    a.slot_map = slot_map;
    a.kv_cache = kv_cache;
    a.dev_err = dev_err;
    a.total = total_q;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    return cache_q4_launch(a, dtype == PA_F32, false, static_cast<cudaStream_t>(stream));
}

int pa_cache_gather_q4(const void *kv_cache, const int32_t *block_table,
                       const int32_t *cu_seq_lens_k, void *k_full, void *v_full, int batch,
                       int total_k, int num_kv_heads, int head_dim, int num_blocks,
                       int block_size, int max_blocks_per_seq, pa_dtype dtype, int32_t *dev_err,
                       void *stream)
{
    if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_DTYPE;
    const int rc = check_pool(num_kv_heads, head_dim, num_blocks, block_size);
    if (rc != PA_OK) return rc;
    if (batch < 0 || total_k < 0 || max_blocks_per_seq <= 0) return PA_ERR_SHAPE;
    if ((long long)total_k * num_kv_heads >= (1ll << 31) - 64) return PA_ERR_UNSUPPORTED;
    // the grid has a CTA for every block of total_k rows and one more for every request
    if ((long long)total_k / block_size + batch >= 1ll << 31) return PA_ERR_UNSUPPORTED;
    if (batch == 0 || total_k == 0) return PA_OK;
    if (!kv_cache || !block_table || !cu_seq_lens_k || !k_full || !v_full) return PA_ERR_NULL;
    if (!aligned(kv_cache, 16) || !aligned(k_full, 16) || !aligned(v_full, 16) || !aligned(block_table, 4) ||
        !aligned(cu_seq_lens_k, 4))
        return PA_ERR_SHAPE;
    CacheQ4Args a{};
    a.kv_cache = const_cast<void *>(kv_cache);
    a.block_table = block_table;
    a.cu_k = cu_seq_lens_k;
    a.k_full = k_full;
    a.v_full = v_full;
    a.dev_err = dev_err;
    a.total = total_k;
    a.batch = batch;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.max_blocks_per_seq = max_blocks_per_seq;
    return cache_q4_launch(a, dtype == PA_F32, true, static_cast<cudaStream_t>(stream));
}

size_t pa_decode_q4_workspace_size(int batch, int num_heads, int num_kv_heads, int head_dim,
                                   int block_size, pa_dtype dtype)
{
    if ((dtype != PA_F32 && dtype != PA_BF16) || batch <= 0 || num_heads <= 0) return 0;
    if (check_pool(num_kv_heads, head_dim, 1, block_size) != PA_OK || num_heads % num_kv_heads != 0)
        return 0;
    return decode_q4_workspace(batch, num_heads, num_kv_heads, head_dim, block_size, dtype == PA_F32);
}

int pa_decode_q4(const void *q, void *kv_cache, const int32_t *block_table,
                 const int32_t *cache_seqlens, const void *k_new, const void *v_new, void *out,
                 void *k_stored, void *v_stored, int batch, int num_heads, int num_kv_heads,
                 int head_dim, int num_blocks, int block_size, int max_blocks_per_seq,
                 pa_dtype dtype, float softmax_scale, void *workspace, size_t workspace_bytes,
                 int32_t *dev_err, void *stream)
{
    if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_DTYPE;
    if (batch < 0 || num_heads <= 0 || max_blocks_per_seq <= 0) return PA_ERR_SHAPE;
    const int rc = check_pool(num_kv_heads, head_dim, num_blocks, block_size);
    if (rc != PA_OK) return rc;
    if (num_heads % num_kv_heads != 0) return PA_ERR_SHAPE;
    if (num_heads / num_kv_heads > 8 || (long long)batch * num_kv_heads * 4 > (long long)kTicketRegionBytes)
        return PA_ERR_UNSUPPORTED;
    // positions of the work's split are 32-bit numbers
    if ((long long)batch * max_blocks_per_seq >= (1ll << 31) / num_kv_heads) return PA_ERR_UNSUPPORTED;
    if (batch == 0) return PA_OK;
    if (!q || !kv_cache || !block_table || !cache_seqlens || !k_new || !v_new || !out) return PA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) ||
        !aligned(out, 16) || !aligned(k_stored, 16) || !aligned(v_stored, 16) || !aligned(block_table, 4) ||
        !aligned(cache_seqlens, 4))
        return PA_ERR_SHAPE;
    if (!workspace || !aligned(workspace, 16)) return PA_ERR_WORKSPACE;
    DecodeQ4Args a{};
    a.q = q;
    a.kv_cache = kv_cache;
    a.block_table = block_table;
    a.cache_seqlens = cache_seqlens;
    a.k_new = k_new;
    a.v_new = v_new;
    a.out = out;
    a.k_stored = k_stored;
    a.v_stored = v_stored;
    a.tickets = static_cast<int32_t *>(workspace);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kTicketRegionBytes);
    a.dev_err = dev_err;
    a.batch = batch;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.group = num_heads / num_kv_heads;
    a.scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)head_dim);
    a.scale_log2 = a.scale * 1.4426950408889634f;
    return decode_q4_launch(a, dtype == PA_F32, workspace_bytes, static_cast<cudaStream_t>(stream));
}

int pa_block_tables(const int32_t *cache_seqlens, const int32_t *new_lens, int32_t *block_table,
                    int32_t *free_blocks, const int32_t *num_free, int32_t *slot_map,
                    int32_t *cu_seq_lens_q, int32_t *cu_seq_lens_k, int32_t *seqlens_k,
                    int32_t *num_free_out, int batch, int total_slots, int num_blocks,
                    int block_size, int max_blocks_per_seq, int32_t *dev_err, void *stream)
{
    return pa_block_tables_decode(cache_seqlens, new_lens, block_table, free_blocks, num_free, slot_map,
                                  cu_seq_lens_q, cu_seq_lens_k, seqlens_k, num_free_out, nullptr, batch,
                                  total_slots, num_blocks, block_size, max_blocks_per_seq, dev_err, stream);
}

int pa_block_tables_decode(const int32_t *cache_seqlens, const int32_t *new_lens,
                           int32_t *block_table, int32_t *free_blocks, const int32_t *num_free,
                           int32_t *slot_map, int32_t *cu_seq_lens_q, int32_t *cu_seq_lens_k,
                           int32_t *seqlens_k, int32_t *num_free_out, int32_t *decode_lens,
                           int batch, int total_slots, int num_blocks, int block_size,
                           int max_blocks_per_seq, int32_t *dev_err, void *stream)
{
    if (batch < 0 || total_slots < 0 || num_blocks <= 0 || block_size <= 0 || max_blocks_per_seq <= 0)
        return PA_ERR_SHAPE;
    if (batch > kTablesMaxBatch || (long long)num_blocks * block_size >= (1ll << 31) ||
        (long long)max_blocks_per_seq * block_size >= (1ll << 31))
        return PA_ERR_UNSUPPORTED;
    if (!cu_seq_lens_q || !cu_seq_lens_k || !num_free || !num_free_out || !free_blocks) return PA_ERR_NULL;
    if (batch > 0 && (!cache_seqlens || !new_lens || !block_table || !seqlens_k)) return PA_ERR_NULL;
    if (total_slots > 0 && !slot_map) return PA_ERR_NULL;
    for (const void *p : {(const void *)cache_seqlens, (const void *)new_lens, (const void *)block_table,
                          (const void *)free_blocks, (const void *)num_free, (const void *)slot_map,
                          (const void *)cu_seq_lens_q, (const void *)cu_seq_lens_k, (const void *)seqlens_k,
                          (const void *)num_free_out, (const void *)decode_lens})
        if (!aligned(p, 4)) return PA_ERR_SHAPE;
    TablesArgs a{};
    a.cache_seqlens = cache_seqlens;
    a.new_lens = new_lens;
    a.block_table = block_table;
    a.free_blocks = free_blocks;
    a.num_free = num_free;
    a.slot_map = slot_map;
    a.cu_q = cu_seq_lens_q;
    a.cu_k = cu_seq_lens_k;
    a.seqlens_k = seqlens_k;
    a.num_free_out = num_free_out;
    a.decode_lens = decode_lens;
    a.dev_err = dev_err;
    a.batch = batch;
    a.total_slots = total_slots;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.max_blocks_per_seq = max_blocks_per_seq;
    return tables_launch(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
