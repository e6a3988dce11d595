// wq_kv_rows.hip -- rows into the 4-bit key/value cache and back.
//
// A group of G channels of one token and head becomes lo = min x (exact: it is
// one of the values), s = RN((max x - min x) / 15) in the model's 16-bit type,
// and codes c = floor((x - lo) / s + 1/2) held to 0..15; the cached value is
// lo + s c.  The codes are those of the real quotient of the 32-bit difference
// t: the nearest integer to t (1 - 2^-18) / s is c or, just above a half, c - 1,
// and the remainder t - c s, which fp32 holds exactly (c s has 15 bits, and the
// remainder is below s), tells which; a value half way between two codes takes
// the upper one.  Differences and remainders are formed at half size, where the
// range of the type cannot overflow them.  Minima and maxima propagate NaN, so a
// group holding an infinity or NaN shows in them: it gets lo = NaN, s = 0.
//
// Both kernels stream: one wave per record (16 tokens of one head), keys or
// values, 16 bytes of a row per lane (8 tokens x 8 chunks of 8 channels per
// load).  A lane's 8 codes of one token are one word of the key layout; for
// the values, 8 lanes transpose their 8 x 8 codes with three exchanges.
//
// What bounds them: reading back, the memory -- 60001 rows of 8 heads, D = 128,
// 311 MB, in 62-64 us (4.9 TB/s, the rate of a copy).  Writing, latency and
// vector instructions (about ten per channel): 11479 prompt rows of 8 heads,
// 60 MB, in 17.1 us (3.5 TB/s); 64 single rows in 5.3 us, a launch and four
// dependent accesses (length, page, the record's other codes, store).
#include "wq_kv.hpp"

namespace wq {
namespace {

struct KvRowsArgs {
  KvSeqs s;
  uint8_t* cache;
  uint16_t* x[2];      // keys, values
  int64_t ld[2];       // elements between rows
  int blocks_per_seq;  // cu_q null: records a sequence's rows can touch
  int slots;           // grid: (slots / 4, kv heads, keys and values)
};

// The record an item works on: tokens t0 .. t1 - 1 of the record belong to the
// call, token t of it is row row0 + t.  False if there is nothing to do.
struct KvItem {
  int t0, t1, head, kv;
  int64_t row0;
  int b, blk;
};
__device__ inline bool kv_item(const KvRowsArgs& a, int lane, KvItem& o) {
  const int slot = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (slot >= a.slots) return false;
  o.head = blockIdx.y;
  o.kv = blockIdx.z;
  int b, first;
  if (a.s.cu_q) {
    // rows behind the start of a record add one slot more than whole records
    b = kv_find_seq(a.s, slot, 1, 16, 2, lane);
    if (b < 0) return false;
    b = __builtin_amdgcn_readfirstlane(b);
    first = kv_row_offset(a.s, b) / 16 + b * 2;
  } else {
    b = (unsigned)slot / (unsigned)a.blocks_per_seq;
    first = b * a.blocks_per_seq;
  }
  const KvSeq q = kv_seq(a.s, b);
  const int blk = (q.pos0 >> 4) + (slot - first);
  o.t0 = q.pos0 - blk * 16;
  if (o.t0 < 0) o.t0 = 0;
  o.t1 = q.pos0 + q.n - blk * 16;
  if (o.t1 > 16) o.t1 = 16;
  if (o.t0 >= o.t1) return false;
  o.b = b;
  o.blk = blk;
  o.row0 = (int64_t)q.row0 + (int64_t)blk * 16 - q.pos0;
  return true;
}

// 8 x 8 transposition of 4-bit entries over the 8 lanes that differ in lane
// bits 3..5: lane t's nibble j goes to lane j's nibble t.
__device__ inline uint32_t transpose_nibbles(uint32_t w, int t) {
  auto step = [&](int b, uint32_t keep) {
    const uint32_t p = b == 1 ? (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x128, 0xf, 0xf, true)  // row_ror:8
                              : __shfl_xor(w, b * 8, 64);
    w = (t & b) ? (w & ~keep) | ((p & ~keep) >> (4 * b)) : (w & keep) | ((p & keep) << (4 * b));
  };
  step(4, 0x0000FFFFu);
  step(2, 0x00FF00FFu);
  step(1, 0x0F0F0F0Fu);
  return w;
}

// minimum / maximum over the aligned 2, 4 or 8 lanes around a lane, by DPP:
// quads swap neighbours, then pairs, then the two quads of 8 lanes mirror
template <bool MAX>
__device__ inline float pick(float a, float b) {
  return MAX ? __builtin_elementwise_maximum(a, b) : __builtin_elementwise_minimum(a, b);
}
template <bool MAX, int N>
__device__ inline float reduce_lanes(float v) {
  auto dpp = [](float x, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  v = pick<MAX>(v, dpp(v, std::integral_constant<int, 0xB1>{}));
  v = pick<MAX>(v, dpp(v, std::integral_constant<int, 0x4E>{}));
  if constexpr (N > 4) v = pick<MAX>(v, dpp(v, std::integral_constant<int, 0x141>{}));
  return v;
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
  KvItem it;
  if (!kv_item(a, lane, it)) return;
  const int t = lane >> 3, ch = lane & 7;
  const uint16_t* x = a.x[it.kv];
  const int64_t ld = a.ld[it.kv];
  u32x4 raw[2][NS];
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int set = 0; set < NS; ++set) {
      // lanes without a row or a chunk of their own load a neighbour's
      const int tok = min(max(8 * half + t, it.t0), it.t1 - 1), c = min(8 * set + ch, NC - 1);
      raw[half][set] = *(const u32x4*)(x + (it.row0 + tok) * ld + (int64_t)it.head * D + 8 * c);
    }
  // (the page number is looked up while the rows are on their way)
  const int r = kv_record(a.s, it.b, it.blk, it.head);
  if (r < 0) return;
  uint8_t* rec = a.cache + (size_t)r * kv_record_bytes(D, NG);
  uint32_t words[2][NS];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int tok = 8 * half + t;
    const bool live = tok >= it.t0 && tok < it.t1;
    float v[NS][8], mn[NS], mx[NS];
#pragma unroll
    for (int set = 0; set < NS; ++set) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t w = raw[half][set][p];
        v[set][2 * p] = act_lo<DT>(w);
        v[set][2 * p + 1] = act_hi<DT>(w);
      }
      mn[set] = mx[set] = v[set][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) {
        mn[set] = pick<false>(mn[set], v[set][e]);
        mx[set] = pick<true>(mx[set], v[set][e]);
      }
      mn[set] = reduce_lanes<false, GC>(mn[set]);
      mx[set] = reduce_lanes<true, GC>(mx[set]);
    }
    if constexpr (GC == 16) {  // a group is two sets of 8 chunks
#pragma unroll
      for (int set = 0; set < NS; set += 2) {
        mn[set] = mn[set + 1] = pick<false>(mn[set], mn[set + 1]);
        mx[set] = mx[set + 1] = pick<true>(mx[set], mx[set + 1]);
      }
    }
#pragma unroll
    for (int set = 0; set < NS; ++set) {
      const int c = 8 * set + ch;
      const float range = 0.5f * mx[set] - 0.5f * mn[set];  // finite exactly if every channel is
      const bool finite = range < INFINITY;
      const uint32_t lo16 = finite ? pack2<DT>(mn[set], 0.0f) & 0xFFFFu : (DT == F16 ? 0x7E00u : 0x7FC0u);
      // RN(range / 7.5): a product and its remainder give it for every mantissa
      // (the division's own sequence only where subnormals come in)
      float step = range * (1.0f / 7.5f);
      step = __builtin_fmaf(__builtin_fmaf(-step, 7.5f, range), 1.0f / 7.5f, step);
      if (__any(range < 0x1p-90f)) step = range / 7.5f;
      const uint32_t s16 = finite ? pack2<DT>(step, 0.0f) & 0xFFFFu : 0u;
      const float s = act_lo<DT>(s16);
      // steps below the range of the reciprocal are lifted with the difference
      const float k = s < 0x1p-100f ? 0x1p63f : 0.5f;
      const float sk = s * k, base = -mn[set] * k;
      const float inv = s > 0.0f ? __builtin_amdgcn_rcpf(sk) * (1.0f - 0x1p-18f) : 0.0f;
      const float hh = s > 0.0f ? 0.5f * sk : INFINITY;
      float q[8], left = -1.0f;  // nearest integers, largest remainder
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = __builtin_fmaf(v[set][e], k, base);  // the 32-bit difference, scaled by a power of two
        q[e] = __builtin_fmaf(d, inv, 0x1p23f) - 0x1p23f;
        left = fmaxf(left, __builtin_fmaf(-q[e], sk, d));
      }
      // Rarely: values on or just above a half take the upper code, and a step
      // that is a subnormal may be so much too small that a code passes 15.
      if (__any(left >= hh || s < (DT == F16 ? 0x1p-14f : 0x1p-126f))) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float r = __builtin_fmaf(-q[e], sk, __builtin_fmaf(v[set][e], k, base));
          q[e] = fminf(q[e] + (r >= hh ? 1.0f : 0.0f), 15.0f);
        }
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
  KvItem it;
  if (!kv_item(a, lane, it)) return;
  const int t = lane >> 3, ch = lane & 7;
  // rows without a place read as zero (record 0 is read in their stead)
  const int r = kv_record(a.s, it.b, it.blk, it.head);
  const uint8_t* rec = a.cache + (size_t)(r < 0 ? 0 : r) * kv_record_bytes(D, NG);
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
      m[half][set] = r < 0 ? 0u : meta[(8 * c / G) * 16 + tok];
    }
  }
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int set = 0; set < NS; ++set) {
      const int tok = 8 * half + t, c = 8 * set + ch;
      const uint32_t w = it.kv ? transpose_nibbles(words[half][set], t) : words[half][set];
      const float s = act_lo<DT>(m[half][set]), lo = act_hi<DT>(m[half][set]);
      // codes as bytes: even channels, odd channels (opaque, so that the byte
      // conversions apply to them and not to fields of w)
      uint32_t even = w & 0x0F0F0F0Fu, odd = w >> 4 & 0x0F0F0F0Fu;
      asm("" : "+v"(even), "+v"(odd));
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        v[e] = __builtin_fmaf(s, (float)(uint8_t)(even >> (4 * e)), lo);
        v[e + 1] = __builtin_fmaf(s, (float)(uint8_t)(odd >> (4 * e)), lo);
      }
      if (tok >= it.t0 && tok < it.t1 && c < NC)
        *(u32x4*)(x + (it.row0 + tok) * ld + (int64_t)it.head * D + 8 * c) =
            u32x4{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])};
    }
}

template <int DT>
wq_status launch(bool write, const KvRowsArgs& a, int D, int G, hipStream_t s) {
  const dim3 grid((a.slots + 3) / 4, a.s.kv_heads, 2), block(256);
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
  a.slots = s.cu_q ? s.rows / 16 + 2 * s.batch : a.blocks_per_seq * s.batch;
  return dt == F16 ? launch<F16>(write, a, D, G, stream) : launch<BF16>(write, a, D, G, stream);
}

}  // namespace wq
