// wq_kv_attention.hip -- attention over the 4-bit key/value cache.
//
// For a row (query position p, head h) and the keys j it sees,
//     a_j = scale * sum_d q_d (lo_j + s_j c_jd)      (s, lo per group of channels)
//     o_d = sum_j e^(a_j - m) (lo_j + s_j c_jd) / sum_j e^(a_j - m).
// No value is dequantised: the codes themselves are the MFMA operands.  A code
// in the low bits of an fp16 is the subnormal c 2^-24, which the matrix cores
// multiply exactly, so eight codes become operands with four ANDs and three
// shifts.  The steps follow in fp32: on the scores, sum q (lo + s c) =
// lo (sum q) + s (sum q c) per group; on the outputs s_j goes into the
// probability and sum_j p_j lo_j is one more running sum.
//
// Layout of the work: rows are (token, head) pairs that share a kv head, 16 to
// an MFMA tile, so the heads of a group share every code that is read.  A wave
// takes NQ such tiles through blocks of 64 keys with an online softmax.  The
// score tiles are computed transposed (keys x rows): a lane then holds 16 keys
// of one row, exactly the inner dimension the second product wants from it,
// and the cache holds the value codes transposed; nothing is exchanged between
// lanes in the loop but the row maximum, and nothing goes through LDS.
// Key 64 b + 16 h + 4 j + i of a block sits in lane group h, tile j, element i.
//
// Numbers: q is scaled by a power of two per row so that its largest channel
// lies in [2^13, 2^14) and converted to fp16 (exact for fp16 and bf16 inputs
// but for channels 2^-27 below the largest).  p s is rounded to fp16 once; its
// reference is held so that the largest lies near 2^14, so products 2^-28
// smaller are still normal numbers.  Scores, maxima and sums are fp32.
//
// Two forms.  Few rows per sequence (decode): the four waves of a workgroup
// take the blocks of 64 keys in turn and merge through LDS.  Many rows: each
// wave has its own rows and all read the same codes through the L1.  Where the
// rows do not fill the GPU the keys are split over workgroups as well, and a
// second kernel joins the parts in a fixed order.
#include "wq_kv.hpp"

#ifndef WQ_HEAD_DIM
#error "compiled once per head size: WQ_HEAD_DIM"
#endif

namespace wq {
namespace {

constexpr float kNone = -1e30f;    // reference of a row that has seen no key
constexpr float kSlack = 8.0f;     // log2 a score may exceed its row's reference by
constexpr int kStepMin = -60;      // smallest exponent the value steps are referred to

// Steps and offsets travel with the codes where they fit the registers (one or
// two groups); with more groups they are read where they are used.
constexpr int kMetaHeld = 2;

template <int D, int NG>
struct KvBlock {  // one lane's share of a block of 64 keys
  static constexpr int HELD = NG <= kMetaHeld ? NG : 0;
  uint32_t k[4][D / 32];
  u32x4 v[D / 32];
  u32x4 km[HELD ? HELD : 1][4], vm[HELD ? HELD : 1][4];
  const u32x4* meta;  // of this lane's 16 keys
  int rec;            // their record, -1: none
};

// W consecutive words, W = 2, 3, 4, 6 or 8
template <int W>
__device__ inline void load_words(uint32_t (&dst)[W], const uint32_t* src) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  typedef uint32_t u32x3 __attribute__((ext_vector_type(3), aligned(4)));
  if constexpr (W == 3) {
    const u32x3 v = *(const u32x3*)src;
#pragma unroll
    for (int i = 0; i < 3; ++i) dst[i] = v[i];
  } else if constexpr (W % 4 == 0) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const u32x4 v = *(const u32x4*)(src + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[i + e] = v[e];
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      const u32x2 v = *(const u32x2*)(src + i);
      dst[i] = v[0];
      dst[i + 1] = v[1];
    }
  }
}

// eight codes of a word as fp16 c 2^-24, in the order 0 4 1 5 2 6 3 7
__device__ inline u32x4 code_frag(uint32_t w) {
  constexpr uint32_t m = 0x000F000Fu;
  return u32x4{w & m, (w >> 4) & m, (w >> 8) & m, (w >> 12) & m};
}

template <int DT, int D, int NG, int NQ, bool ROWS>
__global__ __launch_bounds__(256) void kv_attention_kernel(const KvAttnArgs a) {
  constexpr int W = D / 32, DTL = D / 16, G = D / NG, REC = kv_record_bytes(D, NG);
  constexpr int BM = ROWS ? 64 * NQ : 16 * NQ;  // rows of a workgroup
  constexpr int LDO = D + 4, HELD = KvBlock<D, NG>::HELD;
  // the merge of the waves: references and sums, then outputs
  __shared__ __attribute__((aligned(16))) float lds[ROWS ? 4 : 4 * BM * (2 + LDO)];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, h = lane >> 4;

  // workgroup -> kv head (fastest: the tiles of one head meet in one XCD's L2
  // when the head count is a multiple of 8), part, row tile (last tiles first:
  // under a causal mask they are the longest)
  unsigned idx = blockIdx.x;
  const int kvh = idx % a.seqs.kv_heads;
  idx /= a.seqs.kv_heads;
  const int split = idx % a.splits;
  const int slot = a.slots - 1 - (int)(idx / a.splits);
  int b, tile;
  if (a.seqs.cu_q) {
    b = kv_find_seq(a.seqs, slot, a.heads_per_kv, BM, 1, lane);
    if (b < 0) return;
    tile = slot - (int)((int64_t)kv_row_offset(a.seqs, b) * a.heads_per_kv / BM) - b;
  } else {
    b = slot / a.tiles;
    tile = slot - b * a.tiles;
  }
  const KvSeq sq = kv_seq(a.seqs, b);
  const int R = a.heads_per_kv, nrows = sq.n * R, pos0 = sq.len - sq.n;
  const int r0 = tile * BM;  // below 2^31: rows * q_heads <= 2^30
  if (tile < 0 || r0 >= nrows) return;  // the same for every wave of the workgroup
  const int w0 = ROWS ? r0 + wave * 16 * NQ : r0;

  // rows of this lane, their limits and operands
  float cq[NQ], qs[NQ][NG];
  u32x4 qf[NQ][W];
  int hi[NQ], lo[NQ];
  int hi_min = 0x7FFFFFFF, hi_max = 0, lo_min = 0x7FFFFFFF, lo_max = 0;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int r = w0 + 16 * n + c;
    const bool live = r < nrows;
    const int tok = live ? r / R : 0, head = kvh * R + (live ? r - tok * R : 0);
    const int pos = pos0 + tok;
    hi[n] = a.causal ? (pos + 1 < sq.len ? pos + 1 : sq.len) : sq.len;
    if (pos < 0) hi[n] = 0;
    lo[n] = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
    if (live) {
      hi_min = min(hi_min, hi[n]);
      hi_max = max(hi_max, hi[n]);
      lo_min = min(lo_min, lo[n]);
      lo_max = max(lo_max, lo[n]);
    } else {
      hi[n] = 0;
    }
    const uint16_t* qp = a.q + (int64_t)(sq.row0 + tok) * a.ldq + (int64_t)head * D;
    u32x4 raw[W];
    float big = 0.0f;
#pragma unroll
    for (int kb = 0; kb < W; ++kb) {
      raw[kb] = u32x4{0u, 0u, 0u, 0u};
      if (live) raw[kb] = *(const u32x4*)(qp + 32 * kb + 8 * h);
#pragma unroll
      for (int p = 0; p < 4; ++p)
        big = fmaxf(big, fmaxf(fabsf(act_lo<DT>(raw[kb][p])), fabsf(act_hi<DT>(raw[kb][p]))));
    }
    big = fmaxf(big, __shfl_xor(big, 16, 64));
    big = fmaxf(big, __shfl_xor(big, 32, 64));
    int ex = (int)((__float_as_uint(big) >> 23) & 255) - 127;  // floor(log2 big)
    if (ex == 128) ex = 13;                                     // an infinity: the row is NaN anyway
    if (ex < -100) ex = -100;
    const float f = __uint_as_float((uint32_t)(127 + 13 - ex) << 23);
    // scale log2(e) 2^24 / f, kept off 0 and infinity (a masked score is -inf)
    cq[n] = a.scale_log2 * 0x1p11f * __uint_as_float((uint32_t)(127 + ex) << 23);
    cq[n] = fminf(fmaxf(cq[n], 1e-37f), 1e37f);
#pragma unroll
    for (int g = 0; g < NG; ++g) qs[n][g] = 0.0f;
#pragma unroll
    for (int kb = 0; kb < W; ++kb) {
      float v[8];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        v[2 * p] = act_lo<DT>(raw[kb][p]) * f;
        v[2 * p + 1] = act_hi<DT>(raw[kb][p]) * f;
      }
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t w = pack2<F16>(v[p], v[p + 4]);  // the order of code_frag
        qf[n][kb][p] = w;
        qs[n][kb * 32 / G] += f16_to_f32((uint16_t)w) + f16_to_f32((uint16_t)(w >> 16));
      }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      qs[n][g] += __shfl_xor(qs[n][g], 16, 64);
      qs[n][g] += __shfl_xor(qs[n][g], 32, 64);
      qs[n][g] *= 0x1p-24f;
    }
  }
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    hi_min = min(hi_min, __shfl_xor(hi_min, o, 64));
    hi_max = max(hi_max, __shfl_xor(hi_max, o, 64));
    lo_min = min(lo_min, __shfl_xor(lo_min, o, 64));
    lo_max = max(lo_max, __shfl_xor(lo_max, o, 64));
  }
  hi_min = __builtin_amdgcn_readfirstlane(hi_min);
  hi_max = __builtin_amdgcn_readfirstlane(hi_max);
  lo_min = __builtin_amdgcn_readfirstlane(lo_min);
  lo_max = __builtin_amdgcn_readfirstlane(lo_max);

  // blocks of 64 keys this wave takes: begin, begin + stride, ... below end
  int begin = 0, end = 0;
  if (hi_max > lo_min) {
    const int first = lo_min >> 6, last = (hi_max + 63) >> 6;
    // parts of whole rounds over the workgroup's waves; a wave's rows alone
    // decide its range, so the parts of the row form may differ between waves
    const int round = ROWS ? 1 : 4;
    const int rounds = (last - first + round - 1) / round;
    const int per = (rounds + a.splits - 1) / a.splits * round;
    begin = first + split * per;
    end = begin + per < last ? begin + per : last;
    if (!ROWS) begin += wave;
  }
  constexpr int stride = ROWS ? 1 : 4;
  const int nblk = begin < end ? (end - begin + stride - 1) / stride : 0;

  f4 acc[NQ][DTL];
  float ref[NQ], m[NQ], sum[NQ], lsum[NQ][NG];
  int step_exp = kStepMin;  // the steps of the values seen are below 2^(step_exp + 6)
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = kNone;
    ref[n] = kNone + kStepMin;
    sum[n] = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g) lsum[n][g] = 0.0f;
#pragma unroll
    for (int t = 0; t < DTL; ++t) acc[n][t] = f4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // Records of 16 blocks at a time: lane 4 t + r has record r of the wave's
  // t-th block from `at` on.
  auto records = [&](int at) {
    const int blk = begin + (at + (lane >> 2)) * stride;
    return blk < end ? kv_record(a.seqs, b, blk * 4 + (lane & 3), kvh) : -1;
  };
  auto load = [&](KvBlock<D, NG>& f, int recs, int t) __attribute__((always_inline)) {
    const int rk = __shfl(recs, 4 * t + (c >> 2), 64), rv = __shfl(recs, 4 * t + h, 64);
    // a block that is not there is read as record 0 and masked
    const uint8_t* pk = a.cache + (size_t)(uint32_t)(rk < 0 ? 0 : rk) * REC;
    const uint8_t* pv = a.cache + (size_t)(uint32_t)(rv < 0 ? 0 : rv) * REC;
    f.rec = rv;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      load_words<W>(f.k[j], (const uint32_t*)pk + (4 * j + (c & 3)) * (4 * W) + h * W);
    }
#pragma unroll
    for (int p = 0; p < W; ++p) f.v[p] = ((const u32x4*)(pv + 8 * D))[p * 16 + c];
    f.meta = (const u32x4*)(pv + 16 * D);
#pragma unroll
    for (int g = 0; g < HELD; ++g)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f.km[g][j] = f.meta[4 * g + j];
        f.vm[g][j] = f.meta[4 * NG + 4 * g + j];
      }
  };

  auto compute = [&](KvBlock<D, NG>& f, int blk) __attribute__((always_inline)) {
    const int key0 = blk * 64;
    const bool edge = key0 + 64 > hi_min || key0 < lo_max || __any(f.rec < 0);
    const int kl = key0 + 16 * h;  // this lane's first key
    auto key_meta = [&](int g, int j) __attribute__((always_inline)) {
      if constexpr (HELD) return f.km[g][j];
      else return f.meta[4 * g + j];
    };
    auto value_meta = [&](int g, int j) __attribute__((always_inline)) {
      u32x4 v;
      if constexpr (HELD) v = f.vm[g][j];
      else v = f.meta[4 * NG + 4 * g + j];
      if (edge) {  // keys that are not there count as zero whatever the memory holds
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (f.rec < 0 || kl + 4 * j + i >= sq.len) v[i] = 0u;
      }
      return v;
    };
    // scores: keys x rows
    f4 u[NQ][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        f4 d[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) d[n] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kb = g * (G / 32); kb < (g + 1) * (G / 32); ++kb) {
          const u32x4 kf = code_frag(f.k[j][kb]);
#pragma unroll
          for (int n = 0; n < NQ; ++n) d[n] = mfma16<F16>(kf, qf[n][kb], d[n]);
        }
        const u32x4 km = key_meta(g, j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float s = act_lo<DT>(km[i]), l = act_hi<DT>(km[i]);
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            const float base = g == 0 ? l * qs[n][g] : __builtin_fmaf(l, qs[n][g], u[n][j][i]);
            u[n][j][i] = __builtin_fmaf(s, d[n][i], base);
          }
        }
      }
    }
    // largest value step of this lane's keys
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 sm = {0, 0};
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4 vm = value_meta(g, j);
#pragma unroll
        for (int i = 0; i < 4; ++i) sm = __builtin_elementwise_max(sm, __builtin_bit_cast(u16x2, vm[i]));
      }
    if constexpr (!HELD) asm volatile("" ::: "memory");  // read again below rather than kept
    const float smax = act_lo<DT>((uint32_t)sm[0]);
    bool over = smax > ldexpf(1.0f, step_exp + 6);
    float top[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      if (edge) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = kl + 4 * j + i;
            if (f.rec < 0 || key >= hi[n] || key < lo[n]) u[n][j][i] = -INFINITY;
          }
      }
      float t = fmaxf(fmaxf(u[n][0][0], u[n][0][1]), fmaxf(u[n][0][2], u[n][0][3]));
#pragma unroll
      for (int j = 1; j < 4; ++j)
        t = fmaxf(t, fmaxf(fmaxf(u[n][j][0], u[n][j][1]), fmaxf(u[n][j][2], u[n][j][3])));
      top[n] = t * cq[n];
      over |= top[n] > m[n] + kSlack;
    }
    if (__any(over)) {
      // new references: sums so far are brought to them
      float sx = fmaxf(smax, __shfl_xor(smax, 16, 64));
      sx = fmaxf(sx, __shfl_xor(sx, 32, 64));
      int e = (int)((__float_as_uint(sx) >> 23) & 255) - 127 - 2;  // sx 2^-e in [4, 8)
      if (e > 123) e = 123;
      e = __builtin_amdgcn_readfirstlane(e);
      if (e > step_exp) step_exp = e;
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float t = fmaxf(top[n], __shfl_xor(top[n], 16, 64));
        t = fmaxf(t, __shfl_xor(t, 32, 64));
        if (t > m[n]) m[n] = t;
        const float nref = m[n] + (float)step_exp;
        const float al = __builtin_amdgcn_exp2f(ref[n] - nref);
        ref[n] = nref;
        sum[n] *= al;
#pragma unroll
        for (int g = 0; g < NG; ++g) lsum[n][g] *= al;
#pragma unroll
        for (int x = 0; x < DTL; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][x][i] *= al;
      }
    }
    // probabilities, times the value step of each group, as operands: element
    // 2 i of half hf is key 4 (2 hf) + i, element 2 i + 1 key 4 (2 hf + 1) + i
    u32x4 pf[NQ][NG][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      f4 p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[j][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(u[n][j][i], cq[n], -ref[n]));
          sum[n] += p[j][i];
        }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        f4 ps[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4 vm = value_meta(g, j);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float l = act_hi<DT>(vm[i]), s = act_lo<DT>(vm[i]);
            if (edge) {  // a hidden key may hold anything
              const int key = kl + 4 * j + i;
              if (key >= hi[n] || key < lo[n]) l = s = 0.0f;
            }
            lsum[n][g] = __builtin_fmaf(p[j][i], l, lsum[n][g]);
            ps[j][i] = p[j][i] * s;
          }
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int i = 0; i < 4; ++i) pf[n][g][hf][i] = pack2<F16>(ps[2 * hf][i], ps[2 * hf + 1][i]);
      }
    }
    // outputs, transposed: channels x rows
#pragma unroll
    for (int p = 0; p < W; ++p)
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int t = 2 * p + o, g = 16 * t / G;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const u32x4 vf = code_frag(f.v[p][2 * o + hf]);
#pragma unroll
          for (int n = 0; n < NQ; ++n) acc[n][t] = mfma16<F16>(vf, pf[n][g][hf], acc[n][t]);
        }
      }
  };

  if (nblk > 0) {
    KvBlock<D, NG> f0, f1;
    int recs = records(0), next = nblk > 16 ? records(16) : -1;
    load(f0, recs, 0);
    for (int t = 0; t < nblk; t += 2) {
      // blocks past the last one load record 0 and are not computed
      load(f1, recs, (t + 1) & 15);
      compute(f0, begin + t * stride);
      if (t + 1 >= nblk) break;
      if (((t + 2) & 15) == 0) {
        recs = next;
        next = records(t + 18);
      }
      load(f0, recs, (t + 2) & 15);
      compute(f1, begin + (t + 1) * stride);
    }
  }

  // whole sums of each row, and the offsets' part of the outputs
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    sum[n] += __shfl_xor(sum[n], 16, 64);
    sum[n] += __shfl_xor(sum[n], 32, 64);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      lsum[n][g] += __shfl_xor(lsum[n][g], 16, 64);
      lsum[n][g] += __shfl_xor(lsum[n][g], 32, 64);
    }
#pragma unroll
    for (int t = 0; t < DTL; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][t][i] = __builtin_fmaf(acc[n][t][i], 0x1p24f, lsum[n][16 * t / G]);
  }

  // Store 4 channels of row r (of the sequence's packed rows): the output, or
  // this part's sums for the joining kernel.
  auto place = [&](int r, int64_t& row, int& head) {
    const int tok = r / R;
    row = sq.row0 + tok;
    head = kvh * R + (r - tok * R);
  };
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  auto store = [&](int64_t row, int head, int d, f4 v, float total) {
    if (a.splits > 1) {
      *(f4*)(a.part + (((int64_t)split * a.seqs.rows + row) * a.q_heads + head) * D + d) = v;
    } else {
      // a row that sees no key is zero
      const float inv = total != 0.0f ? 1.0f / total : 0.0f;
      if (total == 0.0f) v = f4{0.0f, 0.0f, 0.0f, 0.0f};
      *(u32x2*)(a.out + row * a.ldo + (int64_t)head * D + d) =
          u32x2{pack2<DT>(v[0] * inv, v[1] * inv), pack2<DT>(v[2] * inv, v[3] * inv)};
    }
  };
  auto store_ml = [&](int64_t row, int head, float r, float s) {
    float* p = a.part_ml + (((int64_t)split * a.seqs.rows + row) * a.q_heads + head) * 2;
    p[0] = r;
    p[1] = s;
  };

  if constexpr (ROWS) {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int r = w0 + 16 * n + c;
      if (r >= nrows) continue;
      int64_t row;
      int head;
      place(r, row, head);
#pragma unroll
      for (int t = 0; t < DTL; ++t) store(row, head, 16 * t + 4 * h, acc[n][t], sum[n]);
      if (a.splits > 1 && h == 0) store_ml(row, head, ref[n], sum[n]);
    }
  } else {
    // merge the four waves: [wave][row] references and sums, then sums scaled
    // to the largest reference
    float* ml = lds;                      // [4][BM][2]
    float* od = lds + 4 * BM * 2;         // [4][BM][LDO]
    if (h == 0) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        ml[(wave * BM + 16 * n + c) * 2] = ref[n];
        ml[(wave * BM + 16 * n + c) * 2 + 1] = sum[n];
      }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int x = 16 * n + c;
      float top = ml[x * 2];
#pragma unroll
      for (int w = 1; w < 4; ++w) top = fmaxf(top, ml[(w * BM + x) * 2]);
      const float al = __builtin_amdgcn_exp2f(ref[n] - top);
#pragma unroll
      for (int t = 0; t < DTL; ++t) {
        f4 v = acc[n][t];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= al;
        *(f4*)(od + (wave * BM + x) * LDO + 16 * t + 4 * h) = v;
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < BM * (D / 4); i += 256) {
      const int x = i / (D / 4), d = 4 * (i % (D / 4));
      if (r0 + x >= nrows) continue;
      float top = ml[x * 2];
#pragma unroll
      for (int w = 1; w < 4; ++w) top = fmaxf(top, ml[(w * BM + x) * 2]);
      float total = 0.0f;
      f4 v = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        total += ml[(w * BM + x) * 2 + 1] * __builtin_amdgcn_exp2f(ml[(w * BM + x) * 2] - top);
        v += *(const f4*)(od + (w * BM + x) * LDO + d);
      }
      int64_t row;
      int head;
      place(r0 + x, row, head);
      store(row, head, d, v, total);
      if (a.splits > 1 && d == 0) store_ml(row, head, top, total);
    }
  }
}

// Joins the parts of the keys: one wave per (row, head), channels over lanes,
// parts in order.
template <int DT, int D>
__global__ __launch_bounds__(256) void kv_join_kernel(const KvAttnArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t all = (int64_t)a.seqs.rows * a.q_heads;
  if (item >= all) return;
  const int64_t row = item / a.q_heads;
  const int head = (int)(item - row * a.q_heads);
  // rows before the first or behind the last sequence belong to nobody
  if (a.seqs.cu_q && (row < kv_row_offset(a.seqs, 0) || row >= kv_row_offset(a.seqs, a.seqs.batch))) return;
  float top = kNone * 2.0f;
  for (int s = 0; s < a.splits; ++s) top = fmaxf(top, a.part_ml[((int64_t)s * all + item) * 2]);
  float total = 0.0f;
  constexpr int V = (D + 63) / 64;
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = 0.0f;
  for (int s = 0; s < a.splits; ++s) {
    const float w = a.part_ml[((int64_t)s * all + item) * 2 + 1];
    if (w == 0.0f) continue;  // a part without keys (NaN goes on)
    const float al = __builtin_amdgcn_exp2f(a.part_ml[((int64_t)s * all + item) * 2] - top);
    total += w * al;
    const float* p = a.part + ((int64_t)s * all + item) * D;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 64 * i < D) v[i] = __builtin_fmaf(p[lane + 64 * i], al, v[i]);
  }
  const float inv = total != 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (lane + 64 * i < D) {
      const float o = v[i] * inv;
      a.out[row * a.ldo + (int64_t)head * D + lane + 64 * i] = DT == F16 ? f32_to_f16(o) : f32_to_bf16(o);
    }
}

template <int DT, int NG, int NQ, bool ROWS>
wq_status run(const KvAttnArgs& a) {
  constexpr int D = WQ_HEAD_DIM;
  const int64_t grid = (int64_t)a.slots * a.splits * a.seqs.kv_heads;
  hipLaunchKernelGGL((kv_attention_kernel<DT, D, NG, NQ, ROWS>), dim3((unsigned)grid), dim3(256), 0, a.stream, a);
  wq_status st = launch_status();
  if (st != WQ_OK || a.splits == 1) return st;
  const int64_t items = (int64_t)a.seqs.rows * a.q_heads;
  hipLaunchKernelGGL((kv_join_kernel<DT, D>), dim3((unsigned)((items + 3) / 4)), dim3(256), 0, a.stream, a);
  return launch_status();
}

template <int DT>
wq_status pick(const KvAttnArgs& a, int G, const KvPlan& p) {
  wq_status st = WQ_EINVAL;
  auto go = [&](auto gc) {
    constexpr int GG = decltype(gc)::value;
    if constexpr (WQ_HEAD_DIM % GG == 0) {
      if (GG != G) return;
      constexpr int NG = WQ_HEAD_DIM / GG;
      if (p.rows_form) st = run<DT, NG, kv_rows_form_tiles(WQ_HEAD_DIM), true>(a);
      else if (p.nq == 1) st = run<DT, NG, 1, false>(a);
      else if constexpr (kv_wide_keys_form(WQ_HEAD_DIM)) st = run<DT, NG, 2, false>(a);
    }
  };
  go(std::integral_constant<int, 32>{});
  go(std::integral_constant<int, 64>{});
  go(std::integral_constant<int, 128>{});
  return st;
}

}  // namespace

wq_status WQ_CAT(launch_kv_attention_, WQ_HEAD_DIM)(const KvAttnArgs& a, int dt, int G, const KvPlan& p) {
  return dt == F16 ? pick<F16>(a, G, p) : pick<BF16>(a, G, p);
}

}  // namespace wq
