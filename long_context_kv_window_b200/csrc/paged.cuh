// paged.cuh -- the paged cache as the kernels see it, and the checks its entry points share.
#pragma once

#include "common.cuh"

namespace kvc {

// Device view of a kvc_paged_cache.
struct Paged {
  uint16_t* k;
  uint16_t* v;
  float* weights;
  int32_t* pos;
  const int32_t* table;
  int32_t* seq_lens;
  int32_t* next_pos;
  int64_t page_stride, table_stride;
  int num_pages, page, log_page, max_pages, batch, Hkv, d;

  // Entries a sequence has room for in the block table.
  __host__ __device__ int64_t room() const { return (int64_t)max_pages * page; }
  // The page of entry s of sequence b, or -1 if the table names none in the pool.
  __device__ __forceinline__ int page_of(int b, int64_t s) const {
    const int p = table[(int64_t)b * table_stride + (s >> log_page)];
    return p >= 0 && p < num_pages ? p : -1;
  }
  // Elements from k (or v) to the row of slot s in page p, KV head g.
  __device__ __forceinline__ int64_t row(int p, int g, int64_t s) const {
    return (int64_t)p * page_stride + ((int64_t)g * page + (s & (page - 1))) * d;
  }
  // Index of the same entry's weight and position.
  __device__ __forceinline__ int64_t entry(int p, int g, int64_t s) const {
    return ((int64_t)p * Hkv + g) * page + (s & (page - 1));
  }
};

inline kvc_status check_paged(const kvc_paged_cache* c, Paged* out) {
  KVC_CHECK_ARG(c != nullptr, "the paged cache must be non-NULL");
  if (c->head_dim != 64 && c->head_dim != 128) return fail(KVC_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  const int page = c->page_size;
  if (page < 16 || page > 256 || (page & (page - 1)) != 0)
    return fail(KVC_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
  KVC_CHECK_ARG(c->batch >= 1 && c->batch <= 1024, "batch must be in 1..1024");
  KVC_CHECK_ARG(c->num_kv_heads >= 1 && c->num_kv_heads <= 65535, "num_kv_heads must be in 1..65535");
  KVC_CHECK_ARG(c->num_pages >= 1 && c->max_pages >= 1, "num_pages and max_pages must be positive");
  KVC_CHECK_ARG((int64_t)c->max_pages * page <= (int64_t(1) << 30), "max_pages * page_size must be at most 2^30");
  KVC_CHECK_ARG(c->table_stride >= c->max_pages, "table_stride must be >= max_pages");
  KVC_CHECK_ARG(c->page_stride >= (int64_t)c->num_kv_heads * page * c->head_dim && c->page_stride % 8 == 0,
                "page_stride must cover a page and be a multiple of 8 elements");
  out->k = c->k;
  out->v = c->v;
  out->weights = c->weights;
  out->pos = c->pos;
  out->table = c->block_table;
  out->seq_lens = c->seq_lens;
  out->next_pos = c->next_pos;
  out->page_stride = c->page_stride;
  out->table_stride = c->table_stride;
  out->num_pages = c->num_pages;
  out->page = page;
  out->log_page = __builtin_ctz((unsigned)page);
  out->max_pages = c->max_pages;
  out->batch = c->batch;
  out->Hkv = c->num_kv_heads;
  out->d = c->head_dim;
  return KVC_OK;
}

// The pointers, which only the launching calls need (a workspace size needs the shapes alone).
inline kvc_status check_paged_pointers(const Paged& c) {
  KVC_CHECK_ARG(c.k && c.v && c.table && c.seq_lens, "k, v, block_table and seq_lens must be non-NULL");
  KVC_CHECK_ARG(aligned(c.k, 16) && aligned(c.v, 16), "k and v must be 16-byte aligned");
  KVC_CHECK_ARG((c.pos == nullptr) == (c.next_pos == nullptr), "pos and next_pos go together");
  return KVC_OK;
}

}  // namespace kvc
