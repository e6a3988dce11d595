// wq_lora.hip -- low-rank adapters of many sequences beside a shared projection.
//
// out = y + scale (x A^T) B^T, each row with its sequence's adapter.
#include "wq_layer.hpp"

namespace wq {
namespace {

// Adapter of row `row` (-1: none), or -2 outside every sequence.
__device__ inline int row_adapter(const LoraArgs& a, int row, int lane) {
  int b;
  if (a.seqs.cu_q) {
    b = kv_find_seq(a.seqs, row, 1, 1, 0, lane);
    if (b < 0 || row >= kv_row_offset(a.seqs, b + 1)) return -2;
  } else {
    b = (uint32_t)row / (uint32_t)(a.seqs.rows / a.seqs.batch);
  }
  const int id = a.adapters[b];
  return id < 0 || id >= a.num ? -1 : id;
}
__device__ inline int adapter_rank(const LoraArgs& a, int id) {
  const int r = a.ranks ? a.ranks[id] : a.rank;
  return r < 0 ? 0 : r > a.rank ? a.rank : r;
}

// One wave to an element of x A^T.
template <int DT>
__global__ __launch_bounds__(64) void lora_shrink_kernel(const LoraArgs a) {
  const int lane = threadIdx.x, row = blockIdx.x, j = blockIdx.y;
  const int id = row_adapter(a, row, lane);
  if (id < 0 || j % a.rank >= adapter_rank(a, id)) return;
  const uint16_t* x = a.x + (int64_t)row * a.K;
  const uint16_t* w = a.a + ((int64_t)id * a.slices * a.rank + j) * a.K;
  float v = 0.f;
  for (int k = lane * 8; k < a.K; k += 512) {
    const u32x4 p = *(const u32x4*)(x + k), q = *(const u32x4*)(w + k);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v = __builtin_fmaf(act_lo<DT>(p[i]), act_lo<DT>(q[i]), v);
      v = __builtin_fmaf(act_hi<DT>(p[i]), act_hi<DT>(q[i]), v);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  if (lane == 0) a.part[(int64_t)row * a.slices * a.rank + j] = v;
}

// One thread to an element of out.
template <int DT>
__global__ __launch_bounds__(256) void lora_expand_kernel(const LoraArgs a) {
  const int row = blockIdx.x, n = blockIdx.y * 256 + threadIdx.x;
  const int id = row_adapter(a, row, threadIdx.x & 63);
  if (id < -1 || n >= a.N || (id < 0 && a.y == a.out)) return;
  const int64_t at = (int64_t)row * a.N + n;
  float v = act_to_f32<DT>(a.y[at]);
  if (id >= 0) {
    int s = 0;
    while (n >= a.ends[s]) ++s;
    const float* p = a.part + ((int64_t)row * a.slices + s) * a.rank;
    const uint16_t* b = a.b + ((int64_t)id * a.N + n) * a.rank;
    float d = 0.f;
    const int rank = adapter_rank(a, id);
    for (int j = 0; j < rank; ++j) d = __builtin_fmaf(p[j], act_to_f32<DT>(b[j]), d);
    v = __builtin_fmaf(d, a.scales[id], v);
  }
  a.out[at] = (uint16_t)pack2<DT>(v, 0.f);
}

template <int DT>
wq_status launch(const LoraArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((lora_shrink_kernel<DT>), dim3(a.seqs.rows, a.slices * a.rank), dim3(64), 0, s, a);
  hipLaunchKernelGGL((lora_expand_kernel<DT>), dim3(a.seqs.rows, (a.N + 255) / 256), dim3(256), 0, s, a);
  return launch_status();
}

}  // namespace

size_t lora_workspace_bytes(int rows, int, int, int rank, int slices) {
  return (size_t)rows * rank * slices * 4;
}

wq_status launch_lora(const LoraArgs& a, int dt, hipStream_t s) {
  return dt == F16 ? launch<F16>(a, s) : launch<BF16>(a, s);
}

}  // namespace wq
