// wq_layer.hpp -- launch arguments of the norm, rotary, adapter and page-table
// kernels (validated by the entry points in wq_layer_api.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wq_kv.hpp"

namespace wq {

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;  // or null
  const uint16_t* weight;
  uint16_t* y;
  uint16_t* sum;             // or null
  int64_t ld_x, ld_r, ld_y, ld_s;
  float eps;
  int rows, heads, dim;
};
wq_status launch_rms_norm(const NormArgs& a, int dt, hipStream_t s);

struct RotaryArgs {
  const uint16_t* x[2];  // q, k
  uint16_t* y[2];
  int64_t ld_x[2], ld_y[2];
  const uint64_t* turns;
  const int32_t* axis;       // or null
  const int32_t* positions;  // or null: positions of the sequences
  int64_t ld_pos;
  KvSeqs seqs;               // lens, cu_q, rows, batch
  float factor;
  int heads[2], head_dim, half, axes;
};
wq_status launch_rotary(const RotaryArgs& a, int dt, int adjacent, hipStream_t s);

constexpr int kLoraMaxSlices = 4;
struct LoraArgs {
  const uint16_t* x;
  const uint16_t* a;
  const uint16_t* b;
  const float* scales;
  const int32_t* ranks;  // or null
  const int32_t* adapters;
  const uint16_t* y;
  uint16_t* out;
  float* part;           // workspace: parts of x A^T, [parts][rows][slices * rank]; launch_lora sets the next two
  uint16_t* v;
  float* down;
  KvSeqs seqs;           // cu_q, rows, batch
  int num, N, K, rank, slices;
  int ends[kLoraMaxSlices];
};
size_t lora_workspace_bytes(int rows, int batch, int K, int rank, int slices);
wq_status launch_lora(const LoraArgs& a, int dt, hipStream_t s);

struct PagesArgs {
  int32_t* table;
  int32_t* lens;
  const int32_t* want;
  int32_t* free_pages;
  int32_t* counts;
  int32_t* cu_q;       // outputs: may be null
  int32_t* positions;
  int64_t* slots;
  int32_t* offsets;    // workspace: back [batch + 1], taken [batch + 1], new rows [batch + 1]
  int rows, batch, max_pages, num_pages, page_shift;
};
// Pages of a table: a thread's next one is up to 2^18 further, in 32 bits (and a cache of
// 2^30 pages, 1152 bytes each at least, would be 1.2 TB).
constexpr int kMaxPages = 1 << 30;
size_t pages_workspace_bytes(int batch, int max_pages, int num_pages, int rows);
wq_status launch_resize(const PagesArgs& a, hipStream_t s);

}  // namespace wq
