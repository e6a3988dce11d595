// wq_kv_api.hip -- C entry points of the 4-bit key/value cache: validation,
// launch shapes, dispatch.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "wq_checks.hpp"
#include "wq_kv.hpp"

using namespace wq;

namespace {

// The shape of a cache: every page of every kv head.
wq_status check_cache(int num_pages, int page_size, int kv_heads, int head_dim, int group) {
  if (num_pages <= 0 || page_size <= 0 || kv_heads <= 0 || head_dim <= 0 || group <= 0) return WQ_EINVAL;
  if (head_dim % group != 0) return WQ_EINVAL;
  if (!kv_head_dim_ok(head_dim) || !kv_group_ok(head_dim, group)) return WQ_EUNSUPPORTED;
  if (!power_of_two(page_size) || page_size < 16 || page_size > 1024 || kv_heads > 1024) return WQ_EUNSUPPORTED;
  // record numbers are 32-bit
  if ((int64_t)num_pages * kv_heads * (page_size / 16) >= ((int64_t)1 << 31)) return WQ_EUNSUPPORTED;
  return WQ_OK;
}

// The sequences of a call; WQ_OK with s.rows == 0 means nothing to do.
wq_status make_seqs(KvSeqs& s, const int32_t* block_table, const int32_t* kv_lens, const int32_t* cu_q, int rows,
                    int batch, int max_pages, int num_pages, int page_size, int kv_heads) {
  if (rows < 0 || batch < 0 || max_pages < 0) return WQ_EINVAL;
  if (rows > 0 && batch == 0) return WQ_EINVAL;
  if (!cu_q && batch > 0 && rows % batch != 0) return WQ_EINVAL;
  if (rows > (1 << 24) || batch > (1 << 20)) return WQ_EUNSUPPORTED;
  if ((int64_t)max_pages * page_size > ((int64_t)1 << 30)) return WQ_EUNSUPPORTED;  // positions are 32-bit
  if (rows > 0 && (!kv_lens || (!block_table && max_pages > 0))) return WQ_EINVAL;
  s.table = block_table;
  s.lens = kv_lens;
  s.cu_q = cu_q;
  s.rows = rows;
  s.batch = batch;
  s.max_pages = max_pages;
  s.num_pages = num_pages;
  s.rpp_shift = __builtin_ctz((unsigned)page_size) - 4;
  s.kv_heads = kv_heads;
  return WQ_OK;
}

wq_status kv_rows(bool write, void* cache, const void* k, const void* v, int64_t ld_k, int64_t ld_v, wq_dtype dt,
                  const int32_t* block_table, const int32_t* kv_lens, const int32_t* cu_q, int rows, int batch,
                  int max_pages, int num_pages, int page_size, int kv_heads, int head_dim, int group, void* stream) {
  wq_status st = check_cache(num_pages, page_size, kv_heads, head_dim, group);
  if (st != WQ_OK) return st;
  if (dt != WQ_F16 && dt != WQ_BF16) return WQ_EINVAL;
  KvSeqs s;
  st = make_seqs(s, block_table, kv_lens, cu_q, rows, batch, max_pages, num_pages, page_size, kv_heads);
  if (st != WQ_OK) return st;
  if (rows == 0) return WQ_OK;
  if (!cache) return WQ_EINVAL;
  if ((uintptr_t)cache & 127) return WQ_EUNSUPPORTED;
  if ((st = check_rows(k, ld_k, rows, kv_heads * head_dim)) != WQ_OK) return st;
  if ((st = check_rows(v, ld_v, rows, kv_heads * head_dim)) != WQ_OK) return st;
  if (!write && rows_meet(k, ld_k, kv_heads * head_dim, v, ld_v, kv_heads * head_dim, rows)) return WQ_EINVAL;
  // grid: four records of one head, keys or values, to a workgroup
  if (((int64_t)rows / 16 + 2 * (int64_t)batch) * kv_heads * 2 >= ((int64_t)1 << 31)) return WQ_EUNSUPPORTED;
  return launch_kv_rows(write, s, (uint8_t*)cache, (uint16_t*)const_cast<void*>(k),
                        (uint16_t*)const_cast<void*>(v), ld_k, ld_v, (int)dt, head_dim, group, (hipStream_t)stream);
}

bool plan_of(KvPlan& p, int rows, int batch, int ragged, int q_heads, int kv_heads, int head_dim, int group,
             int64_t max_kv) {
  if (rows <= 0 || batch <= 0 || q_heads <= 0 || kv_heads <= 0 || max_kv < 0) return false;
  if (rows > (1 << 24) || batch > (1 << 20) || q_heads > 4096 || kv_heads > 1024 || max_kv > ((int64_t)1 << 30))
    return false;
  if (q_heads % kv_heads != 0 || !kv_head_dim_ok(head_dim) || group <= 0 || !kv_group_ok(head_dim, group) ||
      (!ragged && rows % batch != 0))
    return false;
  p = kv_plan(rows, batch, ragged != 0, q_heads / kv_heads, kv_heads, head_dim, group, max_kv);
  return true;
}

}  // namespace

extern "C" {

size_t wq_kv_cache_bytes(int num_pages, int page_size, int kv_heads, int head_dim, int group) {
  if (check_cache(num_pages, page_size, kv_heads, head_dim, group) != WQ_OK) return 0;
  return (size_t)num_pages * kv_heads * (page_size / 16) * kv_record_bytes(head_dim, head_dim / group);
}

wq_status wq_kv_write(const void* k, const void* v, int64_t ld_k, int64_t ld_v, wq_dtype dt, void* cache,
                      const int32_t* block_table, const int32_t* kv_lens, const int32_t* cu_q, int rows, int batch,
                      int max_pages, int num_pages, int page_size, int kv_heads, int head_dim, int group,
                      void* stream) {
  return kv_rows(true, cache, k, v, ld_k, ld_v, dt, block_table, kv_lens, cu_q, rows, batch, max_pages, num_pages,
                 page_size, kv_heads, head_dim, group, stream);
}

wq_status wq_kv_read(const void* cache, void* k, void* v, int64_t ld_k, int64_t ld_v, wq_dtype dt,
                     const int32_t* block_table, const int32_t* kv_lens, const int32_t* cu_q, int rows, int batch,
                     int max_pages, int num_pages, int page_size, int kv_heads, int head_dim, int group,
                     void* stream) {
  return kv_rows(false, const_cast<void*>(cache), k, v, ld_k, ld_v, dt, block_table, kv_lens, cu_q, rows, batch,
                 max_pages, num_pages, page_size, kv_heads, head_dim, group, stream);
}

size_t wq_kv_workspace_bytes(int rows, int batch, int ragged, int q_heads, int kv_heads, int head_dim,
                             int group, int max_kv_len) {
  KvPlan p;
  if (!plan_of(p, rows, batch, ragged, q_heads, kv_heads, head_dim, group, max_kv_len)) return 0;
  return kv_part_bytes(p, rows, q_heads, head_dim) + kv_ml_bytes(p, rows, q_heads);
}

wq_status wq_kv_attention(const void* q, int64_t ld_q, wq_dtype dt, const void* cache, const int32_t* block_table,
                          const int32_t* kv_lens, const int32_t* cu_q, void* out, int64_t ld_out, int rows, int batch,
                          int max_pages, int num_pages, int page_size, int q_heads, int kv_heads, int head_dim,
                          int group, float scale, int causal, int window, int max_kv_len, void* ws, size_t ws_bytes,
                          void* stream) {
  wq_status st = check_cache(num_pages, page_size, kv_heads, head_dim, group);
  if (st != WQ_OK) return st;
  if (dt != WQ_F16 && dt != WQ_BF16) return WQ_EINVAL;
  if (q_heads <= 0 || q_heads % kv_heads != 0) return WQ_EINVAL;
  if (q_heads > 4096) return WQ_EUNSUPPORTED;
  if (!(scale > 0.0f) || !isfinite(scale) || (causal != 0 && causal != 1) || window < 0 || max_kv_len < 0)
    return WQ_EINVAL;
  KvAttnArgs a;
  st = make_seqs(a.seqs, block_table, kv_lens, cu_q, rows, batch, max_pages, num_pages, page_size, kv_heads);
  if (st != WQ_OK) return st;
  if (rows == 0) return WQ_OK;
  if (!cache) return WQ_EINVAL;
  if ((uintptr_t)cache & 127) return WQ_EUNSUPPORTED;
  if ((st = check_rows(q, ld_q, rows, q_heads * head_dim)) != WQ_OK) return st;
  if ((st = check_rows(out, ld_out, rows, q_heads * head_dim)) != WQ_OK) return st;
  KvPlan p;
  if (!plan_of(p, rows, batch, cu_q != nullptr, q_heads, kv_heads, head_dim, group, max_kv_len))
    return WQ_EUNSUPPORTED;
  // one grid dimension: workgroups of up to 512 threads, fewer than 2^32 threads
  if ((int64_t)p.slots * p.splits * kv_heads >= ((int64_t)1 << 23) || (int64_t)rows * q_heads > ((int64_t)1 << 30))
    return WQ_EUNSUPPORTED;
  // in place, or apart: other rows of q would be overwritten before they are read
  if (!(q == out && (rows == 1 || ld_q == ld_out)) && rows_meet(q, ld_q, q_heads * head_dim, out, ld_out, q_heads * head_dim, rows))
    return WQ_EINVAL;
  const size_t part = kv_part_bytes(p, rows, q_heads, head_dim), need = part + kv_ml_bytes(p, rows, q_heads);
  if (need && (!ws || ws_bytes < need)) return WQ_ENOSPACE;
  if (need && ((uintptr_t)ws & 15)) return WQ_EUNSUPPORTED;
  a.q = (const uint16_t*)q;
  a.ldq = ld_q;
  a.out = (uint16_t*)out;
  a.ldo = ld_out;
  a.cache = (const uint8_t*)cache;
  a.q_heads = q_heads;
  a.heads_per_kv = q_heads / kv_heads;
  a.scale_log2 = scale * 1.44269504088896340736f;
  a.causal = causal;
  a.window = window < (1 << 30) ? window : 1 << 30;  // positions are below that
  a.splits = p.splits;
  a.part = need ? (float*)ws : nullptr;
  a.part_ml = need ? (float*)((uint8_t*)ws + part) : nullptr;
  a.slots = p.slots;
  a.tiles = p.tiles;
  a.stream = (hipStream_t)stream;
  switch (head_dim) {
    case 64: return launch_kv_attention_64(a, (int)dt, group, p);
    case 96: return launch_kv_attention_96(a, (int)dt, group, p);
    case 128: return launch_kv_attention_128(a, (int)dt, group, p);
    case 192: return launch_kv_attention_192(a, (int)dt, group, p);
    case 256: return launch_kv_attention_256(a, (int)dt, group, p);
  }
  return WQ_EUNSUPPORTED;
}

}  // extern "C"
