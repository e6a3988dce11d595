// wq_rotary.hip -- rotary positions of one or several axes on queries and keys.
//
// Pair i of a head turns by p f_i, p the row's position on the pair's axis.  The
// frequency comes as a fraction of a turn in units of 2^-64, u = 2^64 f / 2 pi:
// p u mod 2^64 is the angle's fraction of a turn, by one integer product that
// wraps where the angle does, so a position of a million costs no accuracy (a
// 32-bit product p f would be off by 2^-24 p f).  The two bits next to the top
// pick the quadrant, what is left is at most an eighth of a turn either way,
// where the Taylor series of sine (to x^9) and cosine (to x^10) are off by less
// than 2e-9.
//
// A row's sines and cosines serve all its heads: the threads of a row compute
// them once into LDS, one pair each, and then take 8 pairs of one head at a
// time (two 16-byte loads that lie rotary_dim / 2 apart, or 8 adjacent
// channels).  Every thread reads what it writes before it does, so outputs may
// be written over inputs.
//
// What bounds it: memory for prompts (7001 rows of 32 + 8 heads of 128, three axes,
// 143 MB: 30.2 us from memory, 4.7 TB/s, 25.5 with part of it in the last cache; a copy
// runs at 4.75), for single tokens a launch and the chain offsets -> length -> rows (64
// rows of 64 + 8 heads: 3.7 us).
#include "wq_layer.hpp"

namespace wq {
namespace {

constexpr int kMaxHalf = 256;

// cosine and sine of u / 2^32 of a turn
__device__ inline f2 turn(uint32_t u) {
  const uint32_t quadrant = (u + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(u - (quadrant << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float z = x * x;
  float s = 2.7557319e-6f;  // 1 / 9!
  s = __builtin_fmaf(s, z, -1.9841270e-4f);
  s = __builtin_fmaf(s, z, 8.3333333e-3f);
  s = __builtin_fmaf(s, z, -0.16666667f);
  s = __builtin_fmaf(s * z, x, x);
  float c = -2.7557319e-7f;  // 1 / 10!
  c = __builtin_fmaf(c, z, 2.4801587e-5f);
  c = __builtin_fmaf(c, z, -1.3888889e-3f);
  c = __builtin_fmaf(c, z, 4.1666667e-2f);
  c = __builtin_fmaf(c, z, -0.5f);
  c = __builtin_fmaf(c, z, 1.f);
  const float a = quadrant & 1 ? s : c, b = quadrant & 1 ? c : s;
  return f2{(quadrant + 1) & 2 ? -a : a, quadrant & 2 ? -b : b};
}

// Position of row `row` as the last rows of its sequence; false outside every sequence.
__device__ inline bool row_position(const KvSeqs& s, int row, int lane, int& pos) {
  int b;
  if (s.cu_q) {
    b = kv_find_seq(s, row, 1, 1, 0, lane);
    if (b < 0) return false;
  } else {
    b = (uint32_t)row / (uint32_t)(s.rows / s.batch);
  }
  const KvSeq q = kv_seq(s, b);
  pos = q.pos0 + (row - q.row0);
  return row >= q.row0 && row - q.row0 < q.n;
}

// W waves to a row, 4 / W rows to a workgroup.
template <int DT, bool ADJ, int W>
__global__ __launch_bounds__(256) void rotary_kernel(const RotaryArgs a) {
  constexpr int THREADS = 64 * W;
  __shared__ f2 cs_all[4 / W][kMaxHalf];
  const int t = threadIdx.x % THREADS;
  const int row = blockIdx.x * (4 / W) + threadIdx.x / THREADS;
  f2* cs = cs_all[threadIdx.x / THREADS];
  bool live = row < a.seqs.rows;
  int pos = 0;
  if (live && !a.positions) live = row_position(a.seqs, row, threadIdx.x & 63, pos);
  if (live) {
    for (int i = t; i < a.half; i += THREADS) {
      int p = pos;
      if (a.positions) {
        int ax = a.axis ? a.axis[i] : 0;
        ax = ax < 0 ? 0 : ax >= a.axes ? a.axes - 1 : ax;
        p = a.positions[ax * a.ld_pos + row];
      }
      const uint64_t u = (uint64_t)(int64_t)p * a.turns[i];
      cs[i] = turn((uint32_t)(u >> 32)) * a.factor;
    }
  }
  __syncthreads();
  if (!live) return;
  const int per = a.half >> (ADJ ? 2 : 3);                // items of turning pairs in a head
  const int rest = (a.head_dim - 2 * a.half) >> 3;        // 16-byte chunks that are copied
  const int items = per + rest, total = (a.heads[0] + a.heads[1]) * items;
  for (int it = t; it < total; it += THREADS) {
    int head = it / items;
    const int c = it % items;
    const int which = head >= a.heads[0];
    if (which) head -= a.heads[0];
    const uint16_t* x = a.x[which] + row * a.ld_x[which] + head * a.head_dim;
    uint16_t* y = a.y[which] + row * a.ld_y[which] + head * a.head_dim;
    if (c >= per) {
      const int at = 2 * a.half + 8 * (c - per);
      if (x != y) *(u32x4*)(y + at) = *(const u32x4*)(x + at);
    } else if constexpr (ADJ) {
      const u32x4 v = *(const u32x4*)(x + 8 * c);
      u32x4 o;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f2 r = cs[4 * c + q];
        const float p0 = act_lo<DT>(v[q]), p1 = act_hi<DT>(v[q]);
        o[q] = pack2<DT>(p0 * r[0] - p1 * r[1], p0 * r[1] + p1 * r[0]);
      }
      *(u32x4*)(y + 8 * c) = o;
    } else {
      const u32x4 v = *(const u32x4*)(x + 8 * c), w = *(const u32x4*)(x + a.half + 8 * c);
      u32x4 o, n;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f2 r = cs[8 * c + 2 * q], s = cs[8 * c + 2 * q + 1];
        const float p0 = act_lo<DT>(v[q]), p1 = act_hi<DT>(v[q]), m0 = act_lo<DT>(w[q]), m1 = act_hi<DT>(w[q]);
        o[q] = pack2<DT>(p0 * r[0] - m0 * r[1], p1 * s[0] - m1 * s[1]);
        n[q] = pack2<DT>(p0 * r[1] + m0 * r[0], p1 * s[1] + m1 * s[0]);
      }
      *(u32x4*)(y + 8 * c) = o;
      *(u32x4*)(y + a.half + 8 * c) = n;
    }
  }
}

template <int DT, bool ADJ>
wq_status launch(const RotaryArgs& a, hipStream_t s) {
  // Four waves to a row where it has work for them (32 + 8 heads of 128, one wave : four,
  // us: 64 rows 4.5 : 3.2, 1024 rows 7.3 : 6.0, 8192 rows 36.7 : 33.0) or rows are few;
  // else one (8 + 1 heads of 64: 1024 rows 3.1 : 3.4, 8192 rows 7.1 : 11.6; 64 rows 2.9
  // : 2.7).
  const int chunks = (a.half >> (ADJ ? 2 : 3)) + ((a.head_dim - 2 * a.half) >> 3);
  if (((a.heads[0] + a.heads[1]) * chunks >= 256 || a.seqs.rows <= 256) && a.seqs.rows < (1 << 24))  // (grid limit)
    hipLaunchKernelGGL((rotary_kernel<DT, ADJ, 4>), dim3(a.seqs.rows), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((rotary_kernel<DT, ADJ, 1>), dim3((a.seqs.rows + 3) / 4), dim3(256), 0, s, a);
  return launch_status();
}

}  // namespace

wq_status launch_rotary(const RotaryArgs& a, int dt, int adjacent, hipStream_t s) {
  if (dt == F16) return adjacent ? launch<F16, true>(a, s) : launch<F16, false>(a, s);
  return adjacent ? launch<BF16, true>(a, s) : launch<BF16, false>(a, s);
}

}  // namespace wq
