// wq_kv_rows.hip -- rows into the 4-bit key/value cache and back.
//
// A group of G channels of one token and head becomes lo = min x (exact: it is
// one of the values), s = RN((max x - min x) / 15) in the model's 16-bit type,
// and codes c = floor((x - lo) / s + 1/2) held to 0..15; the cached value is
// lo + s c.  The codes are those of the real quotient of the 32-bit difference:
// an estimate t * rcp(s) is corrected with the remainder t - c s, which fp32
// holds exactly (c s has 15 bits, and the remainder is below s), so a value
// half way between two codes always takes the upper one.  Differences and
// remainders are formed at half size, where the range of the type cannot
// overflow them.  A group holding an infinity or NaN gets lo = NaN, s = 0.
//
// Both kernels stream: one wave per record (16 tokens of one head), keys or
// values, 16 bytes of a row per lane (8 tokens x 8 chunks of 8 channels per
// load).  A lane's 8 codes of one token are one word of the key layout; for
// the values, 8 lanes transpose their 8 x 8 codes with three exchanges.
#include "wq_kv.hpp"

namespace wq {
namespace {

struct KvRowsArgs {
  KvSeqs s;
  uint8_t* cache;
  uint16_t* x[2];      // keys, values
  int64_t ld[2];       // elements between rows
  int blocks_per_seq;  // cu_q null: records a sequence's rows can touch
  int64_t items;       // slots * kv_heads * 2
};

// The record an item works on: tokens t0 .. t1 - 1 of the record belong to the
// call, token t of it is row row0 + t.  rec is -1 where the rows have no place
// (no page, or a position below 0).  False if there is nothing to do.
struct KvItem {
  int rec, t0, t1, head, kv;
  int64_t row0;
};
__device__ inline bool kv_item(const KvRowsArgs& a, int64_t item, int lane, KvItem& o) {
  o.kv = (int)(item & 1);
  const int64_t rest = item >> 1;
  o.head = (int)(rest % a.s.kv_heads);
  const int64_t slot = rest / a.s.kv_heads;
  int b;
  int64_t first;
  if (a.s.cu_q) {
    // rows behind the start of a record add one slot more than whole records
    b = kv_find_seq(a.s, slot, 1, 16, 2, lane);
    if (b < 0) return false;
    first = kv_row_offset(a.s, b) / 16 + (int64_t)b * 2;
  } else {
    b = (int)(slot / a.blocks_per_seq);
    first = (int64_t)b * a.blocks_per_seq;
  }
  const KvSeq q = kv_seq(a.s, b);
  const int pos0 = q.len - q.n;  // position of the first row, below 0 if the length is too small
  const int blk = (pos0 >> 4) + (int)(slot - first);
  o.t0 = pos0 - blk * 16;
  if (o.t0 < 0) o.t0 = 0;
  o.t1 = q.len - blk * 16;
  if (o.t1 > 16) o.t1 = 16;
  if (o.t0 >= o.t1) return false;
  o.rec = kv_record(a.s, b, blk, o.head);
  o.row0 = (int64_t)q.row0 + (int64_t)blk * 16 - pos0;
  return true;
}

// 8 x 8 transposition of 4-bit entries over the 8 lanes that differ in lane
// bits 3..5: lane t's nibble j goes to lane j's nibble t.
__device__ inline uint32_t transpose_nibbles(uint32_t w, int t) {
  auto step = [&](int b, uint32_t keep) {
    const uint32_t p = __shfl_xor(w, b * 8, 64);
    w = (t & b) ? (w & ~keep) | ((p & ~keep) >> (4 * b)) : (w & keep) | ((p & keep) << (4 * b));
  };
  step(4, 0x0000FFFFu);
  step(2, 0x00FF00FFu);
  step(1, 0x0F0F0F0Fu);
  return w;
}

// nibble mask of tokens t0 .. t1 - 1 within the 8 tokens from 8 half on
__device__ inline uint32_t token_mask(int half, int t0, int t1) {
  const int a = t0 - 8 * half < 0 ? 0 : t0 - 8 * half, b = t1 - 8 * half > 8 ? 8 : t1 - 8 * half;
  if (a >= b) return 0u;
  const uint32_t upto = b == 8 ? 0xFFFFFFFFu : (1u << (4 * b)) - 1u;
  return upto & ~((1u << (4 * a)) - 1u);
}

template <int D>
__device__ inline int value_word(int c, int t) {  // first word (half 0) of channel 8 c + t
  const int d = 8 * c + t, dt = d >> 4, i = d & 15;
  return ((dt >> 1) * 16 + i) * 4 + (dt & 1) * 2;
}

template <int DT, int D, int G>
__global__ __launch_bounds__(256) void kv_write_kernel(const KvRowsArgs a) {
  constexpr int NG = D / G, NC = D / 8, NS = (NC + 7) / 8, W = D / 32, GC = G / 8;
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= a.items) return;
  KvItem it;
  if (!kv_item(a, item, lane, it) || it.rec < 0) return;
  const int t = lane >> 3, ch = lane & 7;
  const uint16_t* x = a.x[it.kv];
  const int64_t ld = a.ld[it.kv];
  u32x4 raw[2][NS];
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int set = 0; set < NS; ++set) {
      const int tok = 8 * half + t, c = 8 * set + ch;
      raw[half][set] = u32x4{0u, 0u, 0u, 0u};
      if (tok >= it.t0 && tok < it.t1 && c < NC)
        raw[half][set] = *(const u32x4*)(x + (it.row0 + tok) * ld + (int64_t)it.head * D + 8 * c);
    }
  uint8_t* rec = a.cache + (size_t)it.rec * kv_record_bytes(D, NG);
  uint32_t words[2][NS];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int tok = 8 * half + t;
    const bool live = tok >= it.t0 && tok < it.t1;
    float v[NS][8], mn[NS], mx[NS];
    uint32_t ex[NS];  // largest magnitude pattern: shows infinities and NaN
#pragma unroll
    for (int set = 0; set < NS; ++set) {
      typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
      u16x2 m = {0, 0};
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t w = raw[half][set][p];
        v[set][2 * p] = act_lo<DT>(w);
        v[set][2 * p + 1] = act_hi<DT>(w);
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu));
      }
      ex[set] = m[0] > m[1] ? m[0] : m[1];
      mn[set] = mx[set] = v[set][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) {
        mn[set] = fminf(mn[set], v[set][e]);
        mx[set] = fmaxf(mx[set], v[set][e]);
      }
#pragma unroll
      for (int b = 1; b < 8 && b < GC; b <<= 1) {
        mn[set] = fminf(mn[set], __shfl_xor(mn[set], b, 64));
        mx[set] = fmaxf(mx[set], __shfl_xor(mx[set], b, 64));
        const uint32_t o = __shfl_xor(ex[set], b, 64);
        ex[set] = ex[set] > o ? ex[set] : o;
      }
    }
    if constexpr (GC == 16) {  // a group is two sets of 8 chunks
#pragma unroll
      for (int set = 0; set < NS; set += 2) {
        mn[set] = mn[set + 1] = fminf(mn[set], mn[set + 1]);
        mx[set] = mx[set + 1] = fmaxf(mx[set], mx[set + 1]);
        ex[set] = ex[set + 1] = ex[set] > ex[set + 1] ? ex[set] : ex[set + 1];
      }
    }
#pragma unroll
    for (int set = 0; set < NS; ++set) {
      const int c = 8 * set + ch;
      const bool finite = ex[set] < (DT == F16 ? 0x7C00u : 0x7F80u);
      const uint32_t lo16 = finite ? pack2<DT>(mn[set], 0.0f) & 0xFFFFu : (DT == F16 ? 0x7E00u : 0x7FC0u);
      const uint32_t s16 = finite ? pack2<DT>((0.5f * mx[set] - 0.5f * mn[set]) / 7.5f, 0.0f) & 0xFFFFu : 0u;
      const float s = act_lo<DT>(s16);
      // steps below the range of the reciprocal are lifted with the difference
      const float k = s < 0x1p-100f ? 0x1p63f : 0.5f;
      const float sk = s * k, base = -mn[set] * k;
      const float inv = s > 0.0f ? __builtin_amdgcn_rcpf(sk) : 0.0f;
      const float hh = s > 0.0f ? 0.5f * sk : INFINITY;
      float q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = __builtin_fmaf(v[set][e], k, base);  // the 32-bit difference, scaled by a power of two
        const float c0 = floorf(__builtin_fmaf(d, inv, 0.5f));
        const float r = __builtin_fmaf(-c0, sk, d);
        const float c1 = r >= hh ? c0 + 1.0f : r < -hh ? c0 - 1.0f : c0;
        q[e] = fminf(fmaxf(c1, 0.0f), 15.0f);
      }
      // four codes are exact in the 24 bits of a float
      const float lo4 = __builtin_fmaf(__builtin_fmaf(__builtin_fmaf(q[3], 16.0f, q[2]), 16.0f, q[1]), 16.0f, q[0]);
      const float hi4 = __builtin_fmaf(__builtin_fmaf(__builtin_fmaf(q[7], 16.0f, q[6]), 16.0f, q[5]), 16.0f, q[4]);
      words[half][set] = (uint32_t)lo4 | ((uint32_t)hi4 << 16);
      const bool first = (ch & (GC - 1)) == 0 && (GC != 16 || set % 2 == 0);  // one lane per group writes (s, lo)
      if (live && first && c < NC) {
        uint32_t* meta = (uint32_t*)(rec + 16 * D + it.kv * 64 * NG);
        meta[(8 * c / G) * 16 + tok] = s16 | (lo16 << 16);
      }
      if (it.kv == 0 && live && c < NC)
        ((uint32_t*)rec)[tok * NC + (c & 3) * W + (c >> 2)] = words[half][set];
    }
  }
  if (it.kv == 0) return;
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const uint32_t m0 = token_mask(0, it.t0, it.t1), m1 = token_mask(1, it.t0, it.t1);
  const bool whole = (m0 & m1) == 0xFFFFFFFFu;
#pragma unroll
  for (int set = 0; set < NS; ++set) {
    const int c = 8 * set + ch;
    const uint32_t w0 = transpose_nibbles(words[0][set], t), w1 = transpose_nibbles(words[1][set], t);
    if (c >= NC) continue;
    u32x2* dst = (u32x2*)(rec + 8 * D + 4 * value_word<D>(c, t));
    u32x2 w = {w0, w1};
    if (!whole) {  // the record's other tokens keep their codes
      const u32x2 old = *dst;
      w = u32x2{(old[0] & ~m0) | (w0 & m0), (old[1] & ~m1) | (w1 & m1)};
    }
    *dst = w;
  }
}

template <int DT, int D, int G>
__global__ __launch_bounds__(256) void kv_read_kernel(const KvRowsArgs a) {
  constexpr int NG = D / G, NC = D / 8, NS = (NC + 7) / 8, W = D / 32;
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= a.items) return;
  KvItem it;
  if (!kv_item(a, item, lane, it)) return;
  const int t = lane >> 3, ch = lane & 7;
  // rows without a place read as zero (record 0 is read in their stead)
  const bool none = it.rec < 0;
  const uint8_t* rec = a.cache + (size_t)(none ? 0 : it.rec) * kv_record_bytes(D, NG);
  const uint32_t* meta = (const uint32_t*)(rec + 16 * D + it.kv * 64 * NG);
  uint16_t* x = a.x[it.kv];
  const int64_t ld = a.ld[it.kv];
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  uint32_t words[2][NS], m[2][NS];
#pragma unroll
  for (int set = 0; set < NS; ++set) {
    const int c = 8 * set + ch < NC ? 8 * set + ch : NC - 1;
    if (it.kv) {
      const u32x2 w = *(const u32x2*)(rec + 8 * D + 4 * value_word<D>(c, t));
      words[0][set] = w[0];
      words[1][set] = w[1];
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int tok = 8 * half + t;
      if (!it.kv) words[half][set] = ((const uint32_t*)rec)[tok * NC + (c & 3) * W + (c >> 2)];
      m[half][set] = meta[(8 * c / G) * 16 + tok];
    }
  }
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int set = 0; set < NS; ++set) {
      const int tok = 8 * half + t, c = 8 * set + ch;
      const uint32_t w = it.kv ? transpose_nibbles(words[half][set], t) : words[half][set];
      const float s = act_lo<DT>(m[half][set]), lo = act_hi<DT>(m[half][set]);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = none ? 0.0f : __builtin_fmaf(s, (float)((w >> (4 * e)) & 15u), lo);
      if (tok >= it.t0 && tok < it.t1 && c < NC)
        *(u32x4*)(x + (it.row0 + tok) * ld + (int64_t)it.head * D + 8 * c) =
            u32x4{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])};
    }
}

template <int DT>
wq_status launch(bool write, const KvRowsArgs& a, int D, int G, hipStream_t s) {
  const dim3 grid((unsigned)((a.items + 3) / 4)), block(256);
  bool done = false;
  auto go = [&](auto dc, auto gc) {
    constexpr int DD = decltype(dc)::value, GG = decltype(gc)::value;
    if constexpr (DD % GG == 0) {
      if (DD != D || GG != G) return;
      if (write) hipLaunchKernelGGL((kv_write_kernel<DT, DD, GG>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((kv_read_kernel<DT, DD, GG>), grid, block, 0, s, a);
      done = true;
    }
  };
  auto dims = [&](auto gc) {
    go(std::integral_constant<int, 64>{}, gc);
    go(std::integral_constant<int, 96>{}, gc);
    go(std::integral_constant<int, 128>{}, gc);
    go(std::integral_constant<int, 192>{}, gc);
    go(std::integral_constant<int, 256>{}, gc);
  };
  dims(std::integral_constant<int, 32>{});
  dims(std::integral_constant<int, 64>{});
  dims(std::integral_constant<int, 128>{});
  return done ? launch_status() : WQ_EINVAL;
}

}  // namespace

wq_status launch_kv_rows(bool write, const KvSeqs& s, uint8_t* cache, uint16_t* k, uint16_t* v, int64_t ld_k,
                         int64_t ld_v, int dt, int D, int G, hipStream_t stream) {
  KvRowsArgs a;
  a.s = s;
  a.cache = cache;
  a.x[0] = k;
  a.x[1] = v;
  a.ld[0] = ld_k;
  a.ld[1] = ld_v;
  // n rows from any position touch at most (n + 14) / 16 + 1 records
  const int64_t per = (int64_t)s.rows / s.batch;
  a.blocks_per_seq = (int)((per + 14) / 16 + 1);
  const int64_t slots = s.cu_q ? (int64_t)s.rows / 16 + 2 * (int64_t)s.batch : (int64_t)a.blocks_per_seq * s.batch;
  a.items = slots * s.kv_heads * 2;
  return dt == F16 ? launch<F16>(write, a, D, G, stream) : launch<BF16>(write, a, D, G, stream);
}

}  // namespace wq
