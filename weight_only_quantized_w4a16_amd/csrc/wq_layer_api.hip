// wq_layer_api.hip -- C entry points of the norm, rotary positions, adapters and
// page tables: validation, dispatch.
#include <hip/hip_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "wq_checks.hpp"
#include "wq_layer.hpp"

using namespace wq;

namespace {

bool dtype_ok(wq_dtype dt) { return dt == WQ_F16 || dt == WQ_BF16; }

// The sequences of a call that reads no page table; WQ_OK with rows == 0 means nothing to do.
wq_status make_seqs(KvSeqs& s, const int32_t* kv_lens, const int32_t* cu_q, int rows, int batch) {
  if (rows < 0 || batch < 0) return WQ_EINVAL;
  if (rows > 0 && batch == 0) return WQ_EINVAL;
  if (!cu_q && batch > 0 && rows % batch != 0) return WQ_EINVAL;
  if (rows > (1 << 24) || batch > (1 << 20)) return WQ_EUNSUPPORTED;
  s = KvSeqs{};
  s.lens = kv_lens;
  s.cu_q = cu_q;
  s.rows = rows;
  s.batch = batch;
  return WQ_OK;
}

struct Rows {
  const void* p;
  int64_t ld;
  int width;
};
// An output meets an input only as that very matrix (in place).
bool clash(const Rows& out, const Rows& in, int rows, bool in_place) {
  if (!out.p || !in.p) return false;
  if (in_place && out.p == in.p && out.width == in.width && (rows == 1 || out.ld == in.ld)) return false;
  return rows_meet(out.p, out.ld, out.width, in.p, in.ld, in.width, rows);
}
// Whether a row matrix meets a plain range of n bytes.
bool range_meets(const Rows& m, int rows, const void* p, int64_t n) {
  if (!m.p || !p || n <= 0) return false;
  typedef __int128 Z;
  const Z d = (Z)(uintptr_t)p - (Z)(uintptr_t)m.p, w = (Z)m.width * 2, ld = rows > 1 ? (Z)m.ld * 2 : w;
  if (d + n <= 0 || d >= (rows - 1) * ld + w) return false;
  const Z i = d < w ? 0 : (d - w) / ld + 1;  // the first row that ends behind the range's beginning
  return i < rows && i * ld < d + n;
}

}  // namespace

extern "C" {

wq_status wq_rms_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual, const void* weight,
                      float eps, wq_dtype dt, void* y, int64_t ld_y, void* sum, int64_t ld_sum, int rows, int heads,
                      int dim, void* stream) {
  if (!dtype_ok(dt) || rows < 0 || heads <= 0 || dim <= 0) return WQ_EINVAL;
  if (!(eps >= FLT_MIN) || !isfinite(eps)) return WQ_EINVAL;
  if (sum && !residual) return WQ_EINVAL;
  if (dim % 8 != 0 || dim > 65536 || heads > 4096 || rows > (1 << 24) || (int64_t)rows * heads > (1 << 28) ||
      (int64_t)rows * heads * dim > ((int64_t)1 << 33))
    return WQ_EUNSUPPORTED;
  if (rows == 0) return WQ_OK;
  const int width = heads * dim;
  wq_status st;
  if ((st = check_rows(x, ld_x, rows, width)) != WQ_OK) return st;
  if ((st = check_rows(y, ld_y, rows, width)) != WQ_OK) return st;
  if (residual && (st = check_rows(residual, ld_residual, rows, width)) != WQ_OK) return st;
  if (sum && (st = check_rows(sum, ld_sum, rows, width)) != WQ_OK) return st;
  if (!weight) return WQ_EINVAL;
  const Rows X{x, ld_x, width}, R{residual, ld_residual, width}, Y{y, ld_y, width}, S{sum, ld_sum, width};
  for (const Rows& out : {Y, S}) {
    if (clash(out, X, rows, true) || clash(out, R, rows, true)) return WQ_EINVAL;
    if (range_meets(out, rows, weight, (int64_t)dim * 2)) return WQ_EINVAL;
  }
  if (clash(Y, S, rows, false)) return WQ_EINVAL;
  if ((uintptr_t)weight & 15) return WQ_EUNSUPPORTED;
  NormArgs a;
  a.x = (const uint16_t*)x;
  a.residual = (const uint16_t*)residual;
  a.weight = (const uint16_t*)weight;
  a.y = (uint16_t*)y;
  a.sum = (uint16_t*)sum;
  a.ld_x = ld_x;
  a.ld_r = ld_residual;
  a.ld_y = ld_y;
  a.ld_s = ld_sum;
  a.eps = eps;
  a.rows = rows;
  a.heads = heads;
  a.dim = dim;
  return launch_rms_norm(a, (int)dt, (hipStream_t)stream);
}

wq_status wq_rotary(const void* q, int64_t ld_q, const void* k, int64_t ld_k, wq_dtype dt, const uint64_t* turns,
                    const int32_t* axis, float factor, const int32_t* positions, int64_t ld_positions,
                    const int32_t* kv_lens, const int32_t* cu_q, void* q_out, int64_t ld_q_out, void* k_out,
                    int64_t ld_k_out, int rows, int batch, int q_heads, int kv_heads, int head_dim, int rotary_dim,
                    int adjacent, int axes, void* stream) {
  if (!dtype_ok(dt) || rows < 0 || q_heads <= 0 || kv_heads < 0 || head_dim <= 0 || rotary_dim <= 0 || axes <= 0)
    return WQ_EINVAL;
  if (rotary_dim > head_dim || rotary_dim % 2 != 0 || (adjacent != 0 && adjacent != 1) || !isfinite(factor))
    return WQ_EINVAL;
  if ((k != nullptr) != (kv_heads > 0) || (k_out != nullptr) != (kv_heads > 0)) return WQ_EINVAL;
  if (head_dim % 8 != 0 || head_dim > 512 || rotary_dim % (adjacent ? 8 : 16) != 0 || axes > 16 || q_heads > 4096 ||
      kv_heads > 4096 || rows > (1 << 24))
    return WQ_EUNSUPPORTED;
  RotaryArgs a;
  if (positions) {
    if (ld_positions < 0 || (axes > 1 && ld_positions > 0 && ld_positions < rows)) return WQ_EINVAL;
    a.seqs = KvSeqs{};
    a.seqs.rows = rows;
  } else {
    const wq_status st = make_seqs(a.seqs, kv_lens, cu_q, rows, batch);
    if (st != WQ_OK) return st;
    if (rows > 0 && !kv_lens) return WQ_EINVAL;
  }
  if (rows == 0) return WQ_OK;
  const int wq_ = q_heads * head_dim, wk = kv_heads * head_dim;
  wq_status st;
  if ((st = check_rows(q, ld_q, rows, wq_)) != WQ_OK) return st;
  if ((st = check_rows(q_out, ld_q_out, rows, wq_)) != WQ_OK) return st;
  if (kv_heads) {
    if ((st = check_rows(k, ld_k, rows, wk)) != WQ_OK) return st;
    if ((st = check_rows(k_out, ld_k_out, rows, wk)) != WQ_OK) return st;
  }
  if (!turns) return WQ_EINVAL;
  const Rows Q{q, ld_q, wq_}, K{k, ld_k, wk}, QO{q_out, ld_q_out, wq_}, KO{k_out, ld_k_out, wk};
  if (clash(QO, Q, rows, true) || clash(KO, K, rows, true) || clash(QO, K, rows, false) ||
      clash(KO, Q, rows, false) || clash(QO, KO, rows, false))
    return WQ_EINVAL;
  if ((uintptr_t)turns & 7) return WQ_EUNSUPPORTED;
  // (every row's threads read these)
  const int64_t pairs = rotary_dim / 2, per = (int64_t)batch * 4, step = axes > 1 ? ld_positions : 0;
  const struct {
    const void* p;
    int64_t n;
  } small[] = {{turns, pairs * 8}, {axis, pairs * 4}, {positions ? nullptr : kv_lens, per},
               {positions ? nullptr : cu_q, per + 4}};
  for (const auto& m : small) {
    if ((uintptr_t)m.p & 3) return WQ_EUNSUPPORTED;
    if (range_meets(QO, rows, m.p, m.n) || range_meets(KO, rows, m.p, m.n)) return WQ_EINVAL;
  }
  if ((uintptr_t)positions & 3) return WQ_EUNSUPPORTED;
  for (int ax = 0; positions && ax < (step ? axes : 1); ++ax) {
    const int32_t* p = positions + ax * step;
    if (range_meets(QO, rows, p, (int64_t)rows * 4) || range_meets(KO, rows, p, (int64_t)rows * 4)) return WQ_EINVAL;
  }
  a.x[0] = (const uint16_t*)q;
  a.x[1] = (const uint16_t*)k;
  a.y[0] = (uint16_t*)q_out;
  a.y[1] = (uint16_t*)k_out;
  a.ld_x[0] = ld_q;
  a.ld_x[1] = ld_k;
  a.ld_y[0] = ld_q_out;
  a.ld_y[1] = ld_k_out;
  a.turns = turns;
  a.axis = axis;
  a.positions = positions;
  a.ld_pos = axes > 1 ? ld_positions : 0;
  a.factor = factor;
  a.heads[0] = q_heads;
  a.heads[1] = kv_heads;
  a.head_dim = head_dim;
  a.half = rotary_dim / 2;
  a.axes = axes;
  return launch_rotary(a, (int)dt, adjacent, (hipStream_t)stream);
}

size_t wq_lora_workspace_bytes(int rows, int batch, int K, int rank, int slices) {
  if (rows <= 0 || batch <= 0 || K <= 0 || rank <= 0 || slices <= 0) return 0;
  if (rows > (1 << 24) || batch > (1 << 20) || K % 128 != 0 || K > (1 << 20) || rank % 8 != 0 || rank > 128 ||
      slices > kLoraMaxSlices)
    return 0;
  return lora_workspace_bytes(rows, batch, K, rank, slices);
}

wq_status wq_lora(const void* x, wq_dtype dt, const void* a, const void* b, const float* scales, const int32_t* ranks,
                  const int32_t* adapters, const int32_t* cu_q, const void* y, void* out, int rows, int batch,
                  int num_adapters, int N, int K, int rank, int slices, const int32_t* slice_ends_host, void* ws,
                  size_t ws_bytes, void* stream) {
  if (!dtype_ok(dt) || num_adapters <= 0 || N <= 0 || K <= 0 || rank <= 0 || slices <= 0 || !slice_ends_host)
    return WQ_EINVAL;
  if (slices > kLoraMaxSlices || K % 128 != 0 || K > (1 << 20) || N % 16 != 0 || N > (1 << 20) || rank % 8 != 0 ||
      rank > 128 || num_adapters > (1 << 24))
    return WQ_EUNSUPPORTED;
  LoraArgs r;
  int at = 0;
  for (int s = 0; s < slices; ++s) {
    if (slice_ends_host[s] <= at) return WQ_EINVAL;
    if (slice_ends_host[s] % 16 != 0) return WQ_EUNSUPPORTED;
    at = r.ends[s] = slice_ends_host[s];
  }
  if (at != N) return WQ_EINVAL;
  for (int s = slices; s < kLoraMaxSlices; ++s) r.ends[s] = N;
  wq_status st = make_seqs(r.seqs, nullptr, cu_q, rows, batch);
  if (st != WQ_OK) return st;
  if (rows == 0) return WQ_OK;
  if ((int64_t)rows * N > (int64_t)1 << 38) return WQ_EUNSUPPORTED;  // (more than a GPU holds, and than one grid)
  if (!x || !a || !b || !scales || !adapters || !y || !out) return WQ_EINVAL;
  if (((uintptr_t)x | (uintptr_t)a | (uintptr_t)b | (uintptr_t)y | (uintptr_t)out) & 15) return WQ_EUNSUPPORTED;
  const size_t ny = (size_t)rows * N * 2;
  const size_t na = (size_t)num_adapters * slices * rank * K * 2, nb = (size_t)num_adapters * N * rank * 2;
  if ((y != out && bytes_meet(y, ny, out, ny)) || bytes_meet(x, (size_t)rows * K * 2, out, ny) ||
      bytes_meet(a, na, out, ny) || bytes_meet(b, nb, out, ny))
    return WQ_EINVAL;
  const size_t need = lora_workspace_bytes(rows, batch, K, rank, slices);
  if (need && (!ws || ws_bytes < need)) return WQ_ENOSPACE;
  if (need && ((uintptr_t)ws & 15)) return WQ_EUNSUPPORTED;
  if (bytes_meet(ws, need, out, ny) || bytes_meet(ws, need, x, (size_t)rows * K * 2) || bytes_meet(ws, need, y, ny) ||
      bytes_meet(ws, need, a, na) || bytes_meet(ws, need, b, nb))
    return WQ_EINVAL;
  // (every workgroup reads these, and the second product again)
  const size_t each = (size_t)num_adapters * 4, per = (size_t)batch * 4;
  const struct {
    const void* p;
    size_t n;
  } small[] = {{scales, each}, {ranks, each}, {adapters, per}, {cu_q, per + 4}};
  for (const auto& m : small) {
    if ((uintptr_t)m.p & 3) return WQ_EUNSUPPORTED;
    if (bytes_meet(m.p, m.n, out, ny) || bytes_meet(m.p, m.n, ws, need)) return WQ_EINVAL;
  }
  r.x = (const uint16_t*)x;
  r.a = (const uint16_t*)a;
  r.b = (const uint16_t*)b;
  r.scales = scales;
  r.ranks = ranks;
  r.adapters = adapters;
  r.y = (const uint16_t*)y;
  r.out = (uint16_t*)out;
  r.part = (float*)ws;
  r.num = num_adapters;
  r.N = N;
  r.K = K;
  r.rank = rank;
  r.slices = slices;
  return launch_lora(r, (int)dt, (hipStream_t)stream);
}

size_t wq_kv_resize_workspace_bytes(int batch, int max_pages, int num_pages, int rows) {
  if (batch < 0 || batch > (1 << 16) || max_pages < 0 || num_pages <= 0 || num_pages > kMaxPages || rows < 0 ||
      rows > (1 << 24))
    return 0;
  return pages_workspace_bytes(batch, max_pages, num_pages, rows);
}

wq_status wq_kv_resize(int32_t* block_table, int32_t* kv_lens, const int32_t* want_lens, int32_t* free_pages,
                       int32_t* counts, int32_t* cu_q, int32_t* positions, int64_t* slots, int rows, int batch,
                       int max_pages, int num_pages, int page_size, void* ws, size_t ws_bytes, void* stream) {
  if (rows < 0 || batch < 0 || max_pages < 0 || num_pages <= 0 || page_size <= 0) return WQ_EINVAL;
  if (!power_of_two(page_size) || page_size < 16 || page_size > 1024) return WQ_EUNSUPPORTED;
  if (rows > (1 << 24) || batch > (1 << 16) || (int64_t)max_pages * page_size > ((int64_t)1 << 30) ||
      num_pages > kMaxPages)
    return WQ_EUNSUPPORTED;
  if (!free_pages || !counts || (batch > 0 && (!kv_lens || !want_lens || (max_pages > 0 && !block_table))))
    return WQ_EINVAL;
  const size_t need = pages_workspace_bytes(batch, max_pages, num_pages, rows);
  if (need && (!ws || ws_bytes < need)) return WQ_ENOSPACE;
  if (need && ((uintptr_t)ws & 15)) return WQ_EUNSUPPORTED;
  const size_t nb = (size_t)batch * 4;
  const struct {
    const void* p;
    size_t n;
    int align;
  } all[] = {{block_table, nb * max_pages, 4}, {kv_lens, nb, 4}, {want_lens, nb, 4},
             {free_pages, (size_t)num_pages * 4, 4}, {counts, 8, 4}, {cu_q, nb + 4, 4},
             {positions, (size_t)rows * 4, 4}, {slots, (size_t)rows * 8, 8}, {ws, need, 16}};
  for (size_t i = 0; i < sizeof all / sizeof *all; ++i) {
    if ((uintptr_t)all[i].p & (all[i].align - 1)) return WQ_EUNSUPPORTED;
    for (size_t j = 0; j < i; ++j)
      if (bytes_meet(all[i].p, all[i].n, all[j].p, all[j].n)) return WQ_EINVAL;
  }
  PagesArgs a;
  a.table = block_table;
  a.lens = kv_lens;
  a.want = want_lens;
  a.free_pages = free_pages;
  a.counts = counts;
  a.cu_q = cu_q;
  a.positions = positions;
  a.slots = slots;
  a.offsets = (int32_t*)ws;
  a.rows = rows;
  a.batch = batch;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.page_shift = __builtin_ctz((unsigned)page_size);
  return launch_resize(a, (hipStream_t)stream);
}

}  // extern "C"
