// wq_lora.hip -- low-rank adapters of many sequences beside a shared projection.
//
// out = y + scale (x A^T) B^T, each row with its sequence's adapter, in two
// products on the matrix cores: v = x A^T in fp32 parts of the K axis, then
// v B^T added to y.  Rows are taken in tiles of 16 or 64 whatever sequences they
// belong to; a tile works through the distinct adapters among its rows, each
// read once for all of that adapter's rows, the columns of other rows left out
// of loads and stores.  Where rows are few (decode steps: a tile may hold 16
// adapters) the distinct adapters of a tile are spread over workgroups.
//
// In the first product the rows of A are the MFMA's first operand, so a lane
// ends with four consecutive entries of one row's v; the waves of a workgroup
// split K and add up through LDS.  In the second the rows of B are, two tiles of
// 16 columns dealt out so that a lane ends with eight consecutive columns of one
// row: y is read and out written 16 bytes at a time.  v is fp32 and enters that
// product as a sum of two 16-bit numbers (with one, its rounding alone would show
// as much as the output's own); for fp16 each row's v is first scaled by a power
// of two into the upper range of the type, exactly, and back behind the product.
#include "wq_layer.hpp"

namespace wq {
namespace {

// Shape of a call, a function of the sizes the host knows.
struct LoraPlan {
  int rt;      // tiles of 16 rows per workgroup
  int groups;  // workgroups that share a tile's distinct adapters
  int ct;      // tiles of 16 rows of A per workgroup (first product)
  int splits;  // parts of K
  int blocks;  // blocks of 32 columns per wave (second product)
};
LoraPlan lora_plan(int rows, int batch, int K, int columns) {
  LoraPlan p;
  p.rt = rows > 256 ? 4 : 1;
  p.groups = p.rt > 1 ? 1 : batch < 16 ? batch : 16;
  p.ct = p.rt > 1 ? 4 : 1;
  const int64_t tiles = ((int64_t)rows + 16 * p.rt - 1) / (16 * p.rt);
  const int64_t wgs = tiles * p.groups * ((columns + 16 * p.ct - 1) / (16 * p.ct));
  // a wave keeps 256 of K at least
  int64_t s = 1024 / wgs;
  if (s > K / 1024) s = K / 1024;
  p.splits = s < 1 ? 1 : s > 16 ? 16 : (int)s;
  p.blocks = p.rt > 1 ? 8 : 2;
  return p;
}

__device__ inline u32x4 load16(rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0);
}
__device__ inline void store16(rsrc_t r, u32x4 v, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, voff, soff, 0);
}

// Adapter of row row0 + lane (lane < TM): -1 for none, -2 outside every sequence.
// The wave finds the first row's sequence and counts, for every row, the offsets
// of the next 64 sequences that do not lie behind it.
template <int TM>
__device__ inline int tile_adapters(const LoraArgs& a, int row0, int lane) {
  const KvSeqs& s = a.seqs;
  int seq = -1;
  if (!s.cu_q) {
    if (lane < TM && row0 + lane < s.rows) seq = (uint32_t)(row0 + lane) / (uint32_t)(s.rows / s.batch);
  } else {
    int first = kv_find_seq(s, row0, 1, 1, 0, lane);
    first = __builtin_amdgcn_readfirstlane(first < 0 ? 0 : first);
    const int off = first + lane <= s.batch ? kv_row_offset(s, first + lane) : 0x7FFFFFFF;
    bool beyond = false;
    for (int i = 0; i < TM; ++i) {
      const int n = __popcll(__ballot(off <= row0 + i));
      beyond |= n == 64;
      if (lane == i) seq = first + n - 1;  // (first - 1 where nothing is: before the first offset)
      if (n == 0 && lane == i) seq = -1;
    }
    if (beyond) {  // more than 63 sequences without rows among them
      for (int i = 0; i < TM; ++i) {
        int b = kv_find_seq(s, row0 + i, 1, 1, 0, lane);
        if (b >= 0 && row0 + i >= kv_row_offset(s, s.batch)) b = -1;
        if (lane == i) seq = b;
      }
    }
    if (seq >= s.batch || row0 + lane >= s.rows) seq = -1;
  }
  if (seq < 0) return -2;
  const int id = a.adapters[seq];
  return id < 0 || id >= a.num ? -1 : id;
}
__device__ inline int adapter_rank(const LoraArgs& a, int id) {
  const int r = a.ranks ? a.ranks[id] : a.rank;
  return __builtin_amdgcn_readfirstlane(r < 0 ? 0 : r > a.rank ? a.rank : r);
}

// f(adapter) for the distinct values (from `least` on) among the first TM lanes'
// ids: every `of`-th of them, from the `at`-th on.
template <int TM, typename F>
__device__ inline void each_adapter(int ids, int lane, int least, int at, int of, F&& f) {
  uint64_t left = __ballot(lane < TM && ids >= least);
  for (int g = 0; left; ++g) {
    const int cur = __builtin_amdgcn_readlane(ids, __builtin_ctzll(left));
    left &= ~__ballot(ids == cur);
    if (g % of == at) f(cur);
  }
}

// v = x A^T, RT x CT tiles to a workgroup, its four waves (and the parts) split K.
template <int DT, int RT, int CT>
__global__ __launch_bounds__(256) void lora_shrink_kernel(const LoraArgs a, int splits) {
  constexpr int G = RT == 1 ? 4 : 1;  // steps of 32 along K that are loaded together
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, h = lane >> 4;
  const int row0 = blockIdx.x * 16 * RT, C = a.slices * a.rank;
  const int split = blockIdx.y % splits, col0 = blockIdx.y / splits * 16 * CT;
  const int ids = tile_adapters<16 * RT>(a, row0, lane);
  int mine[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) mine[r] = __shfl(ids, 16 * r + c, 64);
  const int left = a.seqs.rows - row0, tile_rows = left < 16 * RT ? left : 16 * RT;
  const rsrc_t xr = make_rsrc(a.x + (int64_t)row0 * a.K, (uint32_t)tile_rows * a.K * 2);
  // this wave's steps of 32 G
  const int units = a.K / 128, part = split * 4 + wave, parts = splits * 4;
  const int k0 = (int)((int64_t)units * part / parts) * 128, k1 = (int)((int64_t)units * (part + 1) / parts) * 128;
  __shared__ f4 red[4][RT * CT][64];

  each_adapter<16 * RT>(ids, lane, 0, blockIdx.z, gridDim.z, [&](int cur) {
    const int rank = adapter_rank(a, cur);
    uint32_t xo[RT], ao[CT];
    bool any = false;
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      const int j = col0 + 16 * t + c;
      const bool ok = j < C && j % a.rank < rank;
      any |= ok;
      ao[t] = ok ? ((uint32_t)j * a.K + 8 * h) * 2 : kOutOfRange;
    }
    if (!__any(any)) return;  // (the same in every wave)
#pragma unroll
    for (int r = 0; r < RT; ++r) xo[r] = mine[r] == cur ? ((uint32_t)(16 * r + c) * a.K + 8 * h) * 2 : kOutOfRange;
    const rsrc_t ar = make_rsrc(a.a + (int64_t)cur * C * a.K, (uint32_t)C * a.K * 2);
    f4 acc[RT][CT] = {};
    u32x4 xf[2][G][RT], af[2][G][CT];
    auto load = [&](int b, int k) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int t = 0; t < CT; ++t) af[b][g][t] = load16(ar, ao[t], (k + 32 * g) * 2);
#pragma unroll
        for (int r = 0; r < RT; ++r) xf[b][g][r] = load16(xr, xo[r], (k + 32 * g) * 2);
      }
    };
    auto multiply = [&](int b) {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int t = 0; t < CT; ++t) acc[r][t] = mfma16<DT>(af[b][g][t], xf[b][g][r], acc[r][t]);
    };
    if (k0 < k1) {
      load(0, k0);
      for (int k = k0; k < k1; k += 64 * G) {
        if (k + 32 * G < k1) load(1, k + 32 * G);
        multiply(0);
        if (k + 32 * G >= k1) break;
        if (k + 64 * G < k1) load(0, k + 64 * G);
        multiply(1);
      }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < CT; ++t) red[wave][r * CT + t][lane] = acc[r][t];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        const int i = r * CT + t;
        if (i % 4 != wave) continue;
        const f4 v = (red[0][i][lane] + red[1][i][lane]) + (red[2][i][lane] + red[3][i][lane]);
        const int j = col0 + 16 * t + 4 * h;
        if (mine[r] == cur && j < C)
          *(f4*)(a.part + ((int64_t)split * a.seqs.rows + row0 + 16 * r + c) * C + j) = v;
      }
    __syncthreads();
  });
}

// 16-bit words of 8 entries, those from `n` on cleared
__device__ inline u32x4 keep_first(u32x4 w, int n) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (n <= 2 * q) w[q] = 0;
    else if (n == 2 * q + 1) w[q] &= 0xFFFFu;
  }
  return w;
}

// out = y + scale v B^T; KC: blocks of 32 of the rank.
template <int DT, int RT, int KC>
__global__ __launch_bounds__(256) void lora_expand_kernel(const LoraArgs a, int splits, int blocks) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, h = lane >> 4;
  const int row0 = blockIdx.x * 16 * RT, C = a.slices * a.rank;
  const int ids = tile_adapters<16 * RT>(a, row0, lane);
  int mine[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) mine[r] = __shfl(ids, 16 * r + c, 64);
  const int left = a.seqs.rows - row0, tile_rows = left < 16 * RT ? left : 16 * RT;
  const rsrc_t yr = make_rsrc(a.y + (int64_t)row0 * a.N, (uint32_t)tile_rows * a.N * 2);
  const rsrc_t outr = make_rsrc(a.out + (int64_t)row0 * a.N, (uint32_t)tile_rows * a.N * 2);
  // this wave's blocks of 32 columns: no block spans two slices
  const int first = (blockIdx.y * 4 + wave) * blocks;
  int s0 = 0, b0 = first;
  while (s0 < a.slices) {
    const int w = a.ends[s0] - (s0 ? a.ends[s0 - 1] : 0), n = (w + 31) >> 5;
    if (b0 < n) break;
    b0 -= n;
    ++s0;
  }
  if (s0 == a.slices) return;

  each_adapter<16 * RT>(ids, lane, a.y == a.out ? 0 : -1, blockIdx.z, gridDim.z, [&](int cur) {
    const int rank = cur < 0 ? 0 : adapter_rank(a, cur);
    const float scale = cur < 0 ? 0.f : a.scales[cur];
    const rsrc_t br = make_rsrc(a.b + (int64_t)(cur < 0 ? 0 : cur) * a.N * a.rank, (uint32_t)a.N * a.rank * 2);
    uint32_t yo[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) yo[r] = ((uint32_t)(16 * r + c) * a.N + 8 * h) * 2;
    const uint32_t bo = ((uint32_t)(8 * (c >> 2) + (c & 3)) * a.rank + 8 * h) * 2;
    u32x4 hi[RT][KC], lo[RT][KC];
    float back[RT];
    u32x4 yv[RT], bv[2][KC];
    int s = s0, base = (s0 ? a.ends[s0 - 1] : 0) + 32 * b0, have = -1;
    auto load = [&] {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < KC; ++k)
          bv[i][k] = load16(br, base + 8 * (c >> 2) + (c & 3) + 4 * i < a.ends[s] && 32 * k + 8 * h < rank
                                    ? bo + (uint32_t)(4 * i * a.rank + 32 * k) * 2 : kOutOfRange,
                            (uint32_t)base * a.rank * 2);
#pragma unroll
      for (int r = 0; r < RT; ++r)
        yv[r] = load16(yr, mine[r] == cur && base + 8 * h < a.ends[s] ? yo[r] : kOutOfRange, (uint32_t)base * 2);
    };
    load();
    for (int n = 0; n < blocks; ++n) {
      if (have != s) {
        have = s;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          f4 v[KC][2] = {};
          for (int p = 0; p < splits; ++p) {
            const rsrc_t pr = make_rsrc(a.part + ((int64_t)p * a.seqs.rows + row0) * C, (uint32_t)tile_rows * C * 4);
#pragma unroll
            for (int k = 0; k < KC; ++k)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t at = (uint32_t)((16 * r + c) * C + s * a.rank + 32 * k + 8 * h + 4 * i) * 4;
                v[k][i] += __builtin_bit_cast(f4, load16(pr, mine[r] == cur && 32 * k + 8 * h + 4 * i < rank ? at : kOutOfRange, 0));
              }
          }
          float m = 0.f;
#pragma unroll
          for (int k = 0; k < KC; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              // (past the rank nothing was written)
              const float x = 32 * k + 8 * h + e < rank ? v[k][e / 4][e % 4] : 0.f;
              v[k][e / 4][e % 4] = x;
              m = fmaxf(m, fabsf(x));
            }
          back[r] = scale;
          float up = 1.f;
          if constexpr (DT == F16) {
            m = fmaxf(m, __shfl_xor(m, 16, 64));
            m = fmaxf(m, __shfl_xor(m, 32, 64));
            // exponent of the largest to 2^13: 2^(13 - e), 2^(e - 13), both normal numbers
            int e = (int)(__float_as_uint(m) >> 23) - 127;
            e = e < -100 ? -100 : e > 120 ? 13 : e;  // (tiny; an infinity or NaN is left as it is)
            up = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
            back[r] = scale * __uint_as_float((uint32_t)(127 - 13 + e) << 23);
          }
#pragma unroll
          for (int k = 0; k < KC; ++k)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float x0 = v[k][q / 2][2 * (q % 2)] * up, x1 = v[k][q / 2][2 * (q % 2) + 1] * up;
              const uint32_t w = pack2<DT>(x0, x1);
              const float h0 = act_lo<DT>(w), h1 = act_hi<DT>(w);
              hi[r][k][q] = w;
              // (an infinity is whole in its first part)
              lo[r][k][q] = pack2<DT>(__builtin_isinf(h0) ? 0.f : x0 - h0, __builtin_isinf(h1) ? 0.f : x1 - h1);
            }
        }
      }
      u32x4 yc[RT], bc[2][KC];
#pragma unroll
      for (int r = 0; r < RT; ++r) yc[r] = yv[r];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < KC; ++k) bc[i][k] = a.ranks ? keep_first(bv[i][k], rank - 32 * k - 8 * h) : bv[i][k];
      const int at = base, end = a.ends[s];
      base += 32;
      if (base >= end) base = end, ++s;
      const bool more = n + 1 < blocks && s < a.slices;
      if (more) load();
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        f4 d[2] = {};
#pragma unroll
        for (int k = 0; k < KC; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) d[i] = mfma16<DT>(bc[i][k], lo[r][k], d[i]);
#pragma unroll
        for (int k = 0; k < KC; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) d[i] = mfma16<DT>(bc[i][k], hi[r][k], d[i]);
        u32x4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          o[q] = pack2<DT>(__builtin_fmaf(d[q / 2][2 * (q % 2)], back[r], act_lo<DT>(yc[r][q])),
                           __builtin_fmaf(d[q / 2][2 * (q % 2) + 1], back[r], act_hi<DT>(yc[r][q])));
        if (rank == 0) o = yc[r];  // (no adapter: a copy)
        store16(outr, o, mine[r] == cur && at + 8 * h < end ? yo[r] : kOutOfRange, (uint32_t)at * 2);
      }
      if (!more) break;
    }
  });
}

template <int DT, int RT, int CT>
void shrink(const LoraArgs& a, const LoraPlan& p, hipStream_t s) {
  const int tiles = (a.seqs.rows + 16 * RT - 1) / (16 * RT), cols = (a.slices * a.rank + 16 * CT - 1) / (16 * CT);
  hipLaunchKernelGGL((lora_shrink_kernel<DT, RT, CT>), dim3(tiles, cols * p.splits, p.groups), dim3(256), 0, s, a, p.splits);
}
template <int DT, int RT, int KC>
void expand(const LoraArgs& a, const LoraPlan& p, hipStream_t s) {
  const int tiles = (a.seqs.rows + 16 * RT - 1) / (16 * RT);
  int n = 0;
  for (int i = 0; i < a.slices; ++i) n += (a.ends[i] - (i ? a.ends[i - 1] : 0) + 31) / 32;
  hipLaunchKernelGGL((lora_expand_kernel<DT, RT, KC>), dim3(tiles, (n + 4 * p.blocks - 1) / (4 * p.blocks), p.groups), dim3(256),
                     0, s, a, p.splits, p.blocks);
}

template <int DT>
wq_status launch(const LoraArgs& a, hipStream_t s) {
  const LoraPlan p = lora_plan(a.seqs.rows, a.seqs.batch, a.K, a.slices * a.rank);
  const int kc = (a.rank + 31) / 32;
  if (p.rt == 1) {
    shrink<DT, 1, 1>(a, p, s);
    if (kc == 1) expand<DT, 1, 1>(a, p, s);
    else if (kc == 2) expand<DT, 1, 2>(a, p, s);
    else expand<DT, 1, 4>(a, p, s);
  } else {
    shrink<DT, 4, 4>(a, p, s);
    if (kc == 1) expand<DT, 4, 1>(a, p, s);
    else if (kc == 2) expand<DT, 4, 2>(a, p, s);
    else expand<DT, 2, 4>(a, p, s);
  }
  return launch_status();
}

}  // namespace

size_t lora_workspace_bytes(int rows, int batch, int K, int rank, int slices) {
  return (size_t)lora_plan(rows, batch, K, rank * slices).splits * rows * rank * slices * 4;
}

wq_status launch_lora(const LoraArgs& a, int dt, hipStream_t s) {
  return dt == F16 ? launch<F16>(a, s) : launch<BF16>(a, s);
}

}  // namespace wq
