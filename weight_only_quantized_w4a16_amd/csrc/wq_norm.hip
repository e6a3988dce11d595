// wq_norm.hip -- root-mean-square norm of rows, with the residual's addition.
//
// h = x + r and y = w h / sqrt(mean h^2 + eps) in fp32; y and the stored h are
// each rounded once, y from the unrounded h.  One pass over memory: a row's
// chunks of 8 channels (one 16-byte load) stay in the registers of the threads
// that share it between the sum of squares and the multiplication, so inputs
// are read once, and either output may be written over either input (a row is
// read whole before its barrier, or by its own wave, and written behind it).
//
// What bounds it: memory (4099 x 8192 with residual, 269 MB, in 51.5 us, 5.2 TB/s,
// above a 4 GiB copy's 4.75; without, 134 MB in 26.2, 5.1; 64032 heads of 128, 33 MB, in
// 7.3 us), for single rows a launch (1 x 4096: 2.7 us, 2.4 without residual).  Rows of
// 520 to 1024 channels leave half or more of their 256 threads without a chunk: 4096 x
// 1024 takes 5.9 us for 17 MB (2.8 TB/s), 7.8 with the residual (4.3).
#include "wq_layer.hpp"

namespace wq {
namespace {

// TPR threads share a row (a power of two; up to 64 of them lie in one wave, a
// workgroup of 256 then takes 256 / TPR rows), CH chunks each.
template <int DT, int TPR, int CH, bool RES>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rms_norm_kernel(const NormArgs a) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR, RPW = THREADS / TPR;
  const int t = threadIdx.x % TPR;
  const uint32_t item = blockIdx.x * RPW + threadIdx.x / TPR;
  const uint32_t items = (uint32_t)a.rows * a.heads;
  const bool live = item < items;
  const uint32_t row = live ? item / (uint32_t)a.heads : 0, head = live ? item % (uint32_t)a.heads : 0;
  const int chunks = live ? a.dim >> 3 : 0;
  const int64_t at = (int64_t)head * a.dim;
  const uint16_t* x = a.x + row * a.ld_x + at;
  float h[CH][8];
  u32x4 w[CH];
  float ss = 0.f;
  {
    u32x4 xv[CH], rv[CH];
    const uint16_t* r = RES ? a.residual + row * a.ld_r + at : nullptr;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * TPR;
      xv[i] = rv[i] = w[i] = u32x4{0u, 0u, 0u, 0u};
      if (c < chunks) {
        xv[i] = *(const u32x4*)(x + 8 * c);
        if constexpr (RES) rv[i] = *(const u32x4*)(r + 8 * c);
        w[i] = *(const u32x4*)(a.weight + 8 * c);
      }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float lo = act_lo<DT>(xv[i][q]), hi = act_hi<DT>(xv[i][q]);
        if constexpr (RES) {
          lo += act_lo<DT>(rv[i][q]);
          hi += act_hi<DT>(rv[i][q]);
        }
        h[i][2 * q] = lo;
        h[i][2 * q + 1] = hi;
        ss = __builtin_fmaf(lo, lo, ss);
        ss = __builtin_fmaf(hi, hi, ss);
      }
  }
#pragma unroll
  for (int d = 1; d < (TPR < 64 ? TPR : 64); d <<= 1) ss += __shfl_xor(ss, d, 64);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    __shared__ float part[THREADS / 64];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = ss;
    __syncthreads();
    const int first = (threadIdx.x / TPR) * W;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) ss += part[first + i];
  }
  const float inv = rsqrtf(ss / (float)a.dim + a.eps);
  uint16_t* y = a.y + row * a.ld_y + at;
  uint16_t* s = RES && a.sum ? a.sum + row * a.ld_s + at : nullptr;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * TPR;
    if (c >= chunks) continue;
    u32x4 o;
    if (RES && s) {
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = pack2<DT>(h[i][2 * q], h[i][2 * q + 1]);
      *(u32x4*)(s + 8 * c) = o;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      o[q] = pack2<DT>(h[i][2 * q] * inv * act_lo<DT>(w[i][q]), h[i][2 * q + 1] * inv * act_hi<DT>(w[i][q]));
    *(u32x4*)(y + 8 * c) = o;
  }
}

template <int DT, int TPR, int CH>
wq_status launch(const NormArgs& a, hipStream_t s) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR, RPW = THREADS / TPR;
  const dim3 grid((uint32_t)(((int64_t)a.rows * a.heads + RPW - 1) / RPW)), block(THREADS);
  if (a.residual)
    hipLaunchKernelGGL((rms_norm_kernel<DT, TPR, CH, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((rms_norm_kernel<DT, TPR, CH, false>), grid, block, 0, s, a);
  return launch_status();
}

template <int DT>
wq_status pick(const NormArgs& a, hipStream_t s) {
  const int chunks = a.dim / 8;
  if (chunks <= 8) return launch<DT, 8, 1>(a, s);
  if (chunks <= 16) return launch<DT, 16, 1>(a, s);
  if (chunks <= 32) return launch<DT, 32, 1>(a, s);
  if (chunks <= 64) return launch<DT, 64, 1>(a, s);
  if (chunks <= 256) return launch<DT, 256, 1>(a, s);
  // few rows: a chunk to a thread (256 threads : 1024, us: 1 x 8192 3.8 : 2.9, 256 x 8192
  // 5.6 : 4.6, 512 x 4096 5.0 : 4.8, 1000 x 5120 8.9 : 8.9, 4096 x 4096 26.6 : 28.6)
  if (chunks <= 1024 && (int64_t)a.rows * a.heads <= 512) return launch<DT, 1024, 1>(a, s);
  if (chunks <= 512) return launch<DT, 256, 2>(a, s);
  if (chunks <= 1024) return launch<DT, 256, 4>(a, s);
  if (chunks <= 2048) return launch<DT, 1024, 2>(a, s);
  if (chunks <= 4096) return launch<DT, 1024, 4>(a, s);
  return launch<DT, 1024, 8>(a, s);
}

}  // namespace

wq_status launch_rms_norm(const NormArgs& a, int dt, hipStream_t s) {
  return dt == F16 ? pick<F16>(a, s) : pick<BF16>(a, s);
}

}  // namespace wq
