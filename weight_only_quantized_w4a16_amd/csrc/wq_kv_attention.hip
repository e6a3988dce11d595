// wq_kv_attention.hip -- attention over the 4-bit key/value cache.
//
// For a row (query position p, head h) and the keys j it sees,
//     a_j = scale * sum_d q_d (lo_j + s_j c_jd)      (s, lo per group of channels)
//     o_d = sum_j e^(a_j - m) (lo_j + s_j c_jd) / sum_j e^(a_j - m).
// No value is dequantised: the codes themselves are the MFMA operands.  A code
// in the low bits of an fp16 is the subnormal c 2^-24 (four bits further up,
// c 2^-20), which the matrix cores multiply exactly, so eight codes become
// operands with four ANDs and one shift; the other operand carries the 2^-4 of
// every second pair.  Steps and offsets follow per group: the scores are
// s ((lo / s) sum q + sum q c), the first term being the accumulator's start;
// on the outputs s_j goes into the probability.
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
// but for channels 2^-23 below the largest).  P = p s is rounded to fp16 once.
// What it is relative to is the row's own: set so that the largest p s of the keys
// it has seen lies at 2^6 (up to 2^7 with several groups), and set anew once one
// may pass 2^15.5.  Every second key's P carries a 2^-4 (its codes the 2^4), so
// products down to 2^-16 of the row's largest are normal numbers, and half a step
// of the smallest is 2^-27 of it.  Keys a row does not see, and keys that count for
// nothing however large their values, have no part in that.  (The room upwards is
// what keeps the sums from being scaled again and again: a prompt with 2^10 to 2^14
// took 366 us, 346 with 2^6 to 2^15.5.)  The offsets are added as
// sum P lo / s beside sum P c, from the same rounded P, so that a rounding of P
// shows times v / s rather than times c: lo / s, as the sum of two fp16, is one
// more operand tile of the second product (rows 0 and 1 of it).  fp16 outputs,
// one row over 1037 keys: 0.39e-3 of the norm when the offsets were summed apart,
// 0.25e-3 now; the rounding of the output alone is 0.20e-3.  A group without a step
// (all channels alike) takes |lo| for one.  Scores, maxima and sums are fp32.
//
// What bounds it (D = 128, one group, MI355X).  Decode: the bytes of the cache --
// 48 rows of 8 heads over 2000 to 8000 keys, 260 MB, in 54-57 us, 4.6-4.8 TB/s
// where a copy of 4 GiB reaches 4.9; about half of the vector instructions' time
// fits beside it.  Many rows: vector instructions.  By the counters a wave issues
// 618 for a block of 64 keys and 32 rows, its prologue, masked blocks and new
// references shared out among them: 68 are MFMAs of 16 cycles, 160 unpack 32 words
// of codes, which two row tiles share, and about nine go to each of a lane's 32
// scores, one of them the exponential at a quarter of the rate.  4096-row prompts
// run in 346 us (795 TFLOP/s, vector units 81 % busy, matrix units 34 %).
// Measured and not kept: three and four row tiles per wave (their sums spill or
// leave one wave per SIMD: 444 and 549 us), a wave of 48 rows with D = 64 (187 us
// against 137 on 1792 rows of 7 sequences), runs of blocks with and without hidden
// keys in loops of their own (copies of the sums, spills: 2066 us), wave
// priorities (-3 to +7 % by shape), the offsets' start of the scores from the
// matrix cores (351 us).
//
// Registers: every form fits the 256 of two waves per SIMD but two row tiles of
// D = 128 in groups of 64 (11 to 13 words spilled) and D = 256 in groups of 32 (36
// to 39; in groups of 64 one, rows split).  Those lie furthest from
// the memory's and the matrix cores' rates: a 4096-row prompt of 32 heads of 128 in
// groups of 128 / 64 / 32 takes 189 / 236 / 404 us, one of 16 heads of 256 takes
// 215 / 270 / 480, and 32 rows of 16 heads of 256 over 4000 keys 49 / 52 / 138.
//
// Two forms.  Few rows per sequence (decode): the waves of a workgroup
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
constexpr float kTop = 6.0f;       // log2 of a row's largest p s when its reference is set, at least
constexpr float kOver = 15.5f;     // log2 that p s may reach before it is set anew (fp16 ends at 16)
constexpr float kStepMin = 0x1p-60f;    // references count smaller value steps as this
constexpr float kStepZero = 0x1p-100f;  // smaller value steps (bf16 only) count as none

template <int D, int NG>
struct KvBlock {  // one lane's share of a block of 64 keys
  uint32_t k[4][D / 32];
  u32x4 v[D / 32];
  uint32_t km[NG], vm[NG];  // step and offset of key c of this lane group's 16
};

// value of lane I of each row of 16 lanes (DPP row broadcast: an operand
// modifier of the instruction that uses it)
template <int I>
__device__ inline uint32_t row_bcast_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x150 + I, 0xf, 0xf, true);
}
template <int I>
__device__ inline float row_bcast(float v) {
  return __uint_as_float(row_bcast_u<I>(__float_as_uint(v)));
}

// Largest of three, NaN if one of them is: one instruction.  (The maximum that
// drops NaN quiets every operand with one of its own first, 32 more for a block
// of 64 keys and 32 rows; written as inline assembly it would be outside the
// compiler's view of what the matrix cores still read.)
__device__ inline float max3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

// Factor 2^x of a sum of probabilities, in two halves: between keys whose value
// steps are far apart x may lie below the exponents of fp32 and the product still
// be one of its numbers.
__device__ inline float scale_sum(float sum, float x) {
  const float half = __builtin_amdgcn_exp2f(0.5f * x);
  return sum * half * half;
}

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

// eight codes of a word as fp16, in the order 0 4 | 1 5 | 2 6 | 3 7: c 2^-24 in
// the first and third pair, c 2^-20 in the second and fourth
__device__ inline u32x4 code_frag(uint32_t w) {
  const uint32_t v = w >> 8;
  return u32x4{w & 0x000F000Fu, w & 0x00F000F0u, v & 0x000F000Fu, v & 0x00F000F0u};
}

// NW: waves of a workgroup.
template <int DT, int D, int NG, int NQ, bool ROWS, int NW>
__global__ __launch_bounds__(64 * NW, NQ == 1 && !ROWS && NW == 4 ? kv_key_waves(D, D / NG) : 2)
void kv_attention_kernel(const KvAttnArgs a) {
  constexpr int W = D / 32, DTL = D / 16, G = D / NG, REC = kv_record_bytes(D, NG);
  constexpr int BM = ROWS ? 16 * NW * NQ : 16 * NQ;  // rows of a workgroup
  constexpr int LDO = D + 4;
  // the merge of the waves: references and sums, then outputs
  __shared__ __attribute__((aligned(16))) float lds[ROWS ? 4 : NW * BM * (2 + LDO)];
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
  const int R = a.heads_per_kv, nrows = sq.n * R, pos0 = sq.pos0;
  const int r0 = tile * BM;  // below 2^31: rows * q_heads <= 2^30
  if (tile < 0 || r0 >= nrows) return;  // the same for every wave of the workgroup
  const int w0 = ROWS ? r0 + wave * 16 * NQ : r0;

  // rows of this lane, their limits and operands; with more than
  // four the operands stay in LDS (every lane its own, so no wave waits for another)
  constexpr bool QLDS = NQ * W > 4;
  __shared__ u32x4 qstage[QLDS ? (ROWS ? NW : 1) * NQ * W * 64 : 1];
  u32x4* qlds = qstage + (QLDS && ROWS ? wave * NQ * W * 64 : 0);
  float cq[NQ], qs[NQ][NG];
  u32x4 qf[QLDS ? 1 : NQ][W];
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
    // an infinite channel makes every score infinite or NaN and the row NaN; as
    // infinities, scores that are all -inf would pass for keys that are not there
    const bool infinite = ex == 128;
    if (infinite) ex = 13;
    if (ex < -100) ex = -100;
    const float f = infinite ? __builtin_nanf("") : __uint_as_float((uint32_t)(127 + 13 - ex) << 23);
    // scale log2(e) 2^24 / f, kept off 0 and infinity (a masked score is -inf)
    cq[n] = a.scale_log2 * 0x1p11f * __uint_as_float((uint32_t)(127 + ex) << 23);
    cq[n] = fminf(fmaxf(cq[n], 1e-37f), 1e37f);
#pragma unroll
    for (int g = 0; g < NG; ++g) qs[n][g] = 0.0f;
#pragma unroll
    for (int kb = 0; kb < W; ++kb) {
      float v[8];
      u32x4 row;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        v[2 * p] = act_lo<DT>(raw[kb][p]) * f;
        v[2 * p + 1] = act_hi<DT>(raw[kb][p]) * f;
      }
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float f = p & 1 ? 0x1p-4f : 1.0f;  // the order and scale of code_frag
        const uint32_t w = pack2<F16>(v[p] * f, v[p + 4] * f);
        row[p] = w;
        qs[n][kb * 32 / G] += (f16_to_f32((uint16_t)w) + f16_to_f32((uint16_t)(w >> 16))) * (p & 1 ? 0x1p4f : 1.0f);
      }
      if constexpr (QLDS) qlds[(n * W + kb) * 64 + lane] = row;
      else qf[n][kb] = row;
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
    const int round = ROWS ? 1 : NW;
    const int rounds = (last - first + round - 1) / round;
    const int per = (rounds + a.splits - 1) / a.splits * round;
    begin = first + split * per;
    end = begin + per < last ? begin + per : last;
    if (!ROWS) begin += wave;
  }
  constexpr int stride = ROWS ? 1 : NW;
  const int nblk = begin < end ? (end - begin + stride - 1) / stride : 0;

  f4 acc[NQ][DTL], off[NQ][NG];
  // log2 of what a row's probabilities are relative to: kTop below the largest
  // p s of the keys it has seen, within kOver - kTop
  float ref[NQ], sum[NQ];
  // Every block is only asked whether its steps stay below step_limit and its
  // scores below limit (what p s <= 2^kOver leaves them at such a step).
  float step_limit = 0.0f, limit[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    ref[n] = limit[n] = kNone;
    sum[n] = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g) off[n][g] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int t = 0; t < DTL; ++t) acc[n][t] = f4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // Records of 16 blocks at a time: lane 4 t + r has record r of the wave's
  // t-th block from `at` on.
  auto records = [&](int at) {
    const int blk = begin + (at + (lane >> 2)) * stride;
    return blk < end ? kv_record(a.seqs, b, blk * 4 + (lane & 3), kvh) : -1;
  };
  // blocks and records that are not there are read as record 0 and masked
  auto record_at = [&](int rec) { return a.cache + (size_t)(uint32_t)(rec < 0 ? 0 : rec) * REC; };
  auto load_keys = [&](KvBlock<D, NG>& f, int recs, int t) __attribute__((always_inline)) {
    const uint8_t* pk = record_at(__shfl(recs, 4 * t + (c >> 2), 64));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      load_words<W>(f.k[j], (const uint32_t*)pk + (4 * j + (c & 3)) * (4 * W) + h * W);
    const uint8_t* pm = record_at(__shfl(recs, 4 * t + h, 64)) + 16 * D;
#pragma unroll
    for (int g = 0; g < NG; ++g) f.km[g] = ((const uint32_t*)pm)[16 * g + c];
  };
  auto load_values = [&](KvBlock<D, NG>& f, int recs, int t) __attribute__((always_inline)) {
    const uint8_t* pv = record_at(__shfl(recs, 4 * t + h, 64));
#pragma unroll
    for (int p = 0; p < W; ++p) f.v[p] = ((const u32x4*)(pv + 8 * D))[p * 16 + c];
#pragma unroll
    for (int g = 0; g < NG; ++g) f.vm[g] = ((const uint32_t*)(pv + 16 * D))[16 * (NG + g) + c];
  };

  // which half of (hi, lo) pairs of two keys this lane's row of the offset
  // operand takes: row 0 the first, row 1 the second (the other rows are not used)
  const uint32_t offset_sel = c & 1 ? 0x07060302u : 0x05040100u;

  // one block: rec is the record of this lane's 16 keys (-1: none); `scored` is
  // called when its keys are not needed any more
  auto compute = [&](KvBlock<D, NG>& f, int blk, int rec, auto scored) __attribute__((always_inline)) {
    const int kl = blk * 64 + 16 * h;  // this lane's first key
    // whether some key is hidden from some row (the same for the whole wave)
    const bool edge = blk * 64 + 64 > hi_min || blk * 64 < lo_max || __any(rec < 0);
    // step and offset / step of this lane's key
    float ks[NG], kr[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      ks[g] = act_lo<DT>(f.km[g]);
      kr[g] = act_hi<DT>(f.km[g]);
      // a group without a step (its codes are 0) takes 1 for one; the subnormals of
      // bf16 count as its smallest normal number, whose reciprocal is one too
      const bool flat = ks[g] == 0.0f;
      ks[g] = flat ? 1.0f : fmaxf(ks[g], 0x1p-126f);
      kr[g] *= __builtin_amdgcn_rcpf(ks[g]);
    }
    // scores: keys x rows
    f4 u[NQ][4];
    if constexpr (QLDS) asm volatile("" ::: "memory");  // the row operands are read again, not kept
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f4 d[NQ][4];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        // a copy for every tile: the broadcasts then stay operand modifiers (not
        // where more would spill: D = 128 in two groups, 502 us against 475)
        float r = kr[g];
        if (NQ > 1 && (NG == 1 || D == 64)) asm volatile("" : "+v"(r));
        sfor<16>([&](auto ic) __attribute__((always_inline)) {
          constexpr int i = decltype(ic)::value;
          d[n][i / 4][i % 4] = row_bcast<i>(r) * qs[n][g];
        });
      }
#pragma unroll
      for (int kb = g * (G / 32); kb < (g + 1) * (G / 32); ++kb) {
        u32x4 q[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          if constexpr (QLDS) q[n] = qlds[(n * W + kb) * 64 + lane];
          else q[n] = qf[n][kb];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4 kf = code_frag(f.k[j][kb]);
#pragma unroll
          for (int n = 0; n < NQ; ++n) d[n][j] = mfma16<F16>(kf, q[n], d[n][j]);
        }
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float s = ks[g];
        if (NQ > 1 && (NG == 1 || D == 64)) asm volatile("" : "+v"(s));
        sfor<16>([&](auto ic) __attribute__((always_inline)) {
          constexpr int i = decltype(ic)::value;
          const float x = row_bcast<i>(s) * d[n][i / 4][i % 4];
          u[n][i / 4][i % 4] = g == 0 ? x : u[n][i / 4][i % 4] + x;
        });
      }
    }
    scored();
    // step and offset / step of this lane's value
    float vs[NG], smax = kStepMin;
    uint32_t vr[NG];
    bool nan_value = false;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      // values of keys that are not there, or that no row of the wave sees (pages
      // before a window may never have been written), count as zero whatever the
      // memory holds
      const uint32_t m = rec < 0 || (uint32_t)(kl + c - lo_min) >= (uint32_t)(hi_max - lo_min) ? 0u : f.vm[g];
      const float l = act_hi<DT>(m);
      float st = act_lo<DT>(m);
      if (st < kStepZero) st = fabsf(l);  // NaN for a group of NaN
      if (st < kStepZero) st = 0.0f;
      // lo / s of the tokens with a factor 2^-4 in their probability as it is,
      // of the others times 2^-4
      float r = st > 0.0f ? l * __builtin_amdgcn_rcpf(st) : 0.0f;
      r *= c & 1 ? 1.0f : 0x1p-4f;
      const float r1 = f16_to_f32(f32_to_f16(r));
      vr[g] = pack2<F16>(r1, r - r1);
      nan_value |= st != st;
      smax = st > smax ? st : smax;  // (drops NaN)
      vs[g] = c & 1 ? st * 0x1p-4f : st;
    }
    bool over = smax > step_limit;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      if (edge) {
        // the key's limits relative to this lane's first key; opaque, or the
        // comparisons are made for every block and only used for these
        int a0 = rec < 0 ? 16 : lo[n] - kl, a1 = hi[n] - kl;
        asm volatile("" : "+v"(a0), "+v"(a1));
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (4 * j + i >= a1 || 4 * j + i < a0) u[n][j][i] = -INFINITY;
      }
      float t = max3(u[n][0][0], u[n][0][1], u[n][0][2]);
#pragma unroll
      for (int i = 3; i < 15; i += 2) t = max3(t, u[n][i / 4][i % 4], u[n][(i + 1) / 4][(i + 1) % 4]);
      t = max3(t, u[n][3][3], t);
      over |= t * cq[n] > limit[n];
    }
    if (__any(over)) {
      // The bound on the steps follows this block's, down too: a block of larger
      // ones costs itself and the next block this pass (half again as much room as
      // this block needs: a prompt in 348 us; the next power of two: 352).  New references where
      // a key the row sees calls for one (a hidden key's score is -inf): sums so far
      // are brought to them.
      int sx = __float_as_int(smax);  // positive: ordered as integers
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) sx = max(sx, __shfl_xor(sx, o, 64));
      step_limit = __int_as_float(__builtin_amdgcn_readfirstlane(sx)) * 1.5f;
      const float step_top = __builtin_amdgcn_logf(step_limit), step = __builtin_amdgcn_logf(smax);  // log2
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float t = -INFINITY;
        sfor<16>([&](auto ic) __attribute__((always_inline)) {
          constexpr int i = decltype(ic)::value;
          t = fmaxf(t, __builtin_fmaf(u[n][i / 4][i % 4], cq[n], row_bcast<i>(step)));
        });
        t = fmaxf(t, __shfl_xor(t, 16, 64));
        t = fmaxf(t, __shfl_xor(t, 32, 64));
        // With several groups, a whole number of octaves from the largest score: the
        // key that counts most then has P = s 2^e, which fp16 holds exactly in every
        // group (with one group its P is 2^kTop).
        float to = t - kTop;
        if constexpr (NG > 1) {
          float m = u[n][0][0];
#pragma unroll
          for (int i = 1; i < 16; ++i) m = fmaxf(m, u[n][i / 4][i % 4]);
          m = fmaxf(m, __shfl_xor(m, 16, 64));
          m = fmaxf(m, __shfl_xor(m, 32, 64)) * cq[n];
          to = m + __builtin_floorf(to - m);
        }
        const float nref = fmaxf(ref[n], to);
        const float al = __builtin_amdgcn_exp2f(ref[n] - nref);
        sum[n] = scale_sum(sum[n], ref[n] - nref);
        ref[n] = nref;
        // (less what large scores may be rounded by: 2 ulp of the reference)
        limit[n] = nref + (kOver - step_top) - 0x1p-22f * fabsf(nref);
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) off[n][g][i] *= al;
#pragma unroll
        for (int x = 0; x < DTL; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][x][i] *= al;
      }
    }
    // probabilities (in the scores' registers)
    const bool hidden_nan = edge && __any(nan_value);
    uint32_t hide[NQ];  // bit 4 j + i: the key is hidden, where that matters below
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      hide[n] = 0;
      if (hidden_nan) {
        float none = -INFINITY;
        asm volatile("" : "+v"(none));
#pragma unroll
        for (int i = 0; i < 16; ++i) hide[n] |= u[n][i / 4][i % 4] == none ? 1u << i : 0u;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[n][j][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(u[n][j][i], cq[n], -ref[n]));
          sum[n] += u[n][j][i];
        }
    }
    // Group by group: times the value step as operands -- element 2 i of half
    // hf is key 4 (2 hf) + i, element 2 i + 1 key 4 (2 hf + 1) + i -- and the
    // outputs, transposed: channels x rows.
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      u32x4 pf[NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        f4 ps[4];
        sfor<16>([&](auto ic) __attribute__((always_inline)) {
          constexpr int i = decltype(ic)::value;
          ps[i / 4][i % 4] = row_bcast<i>(vs[g]) * u[n][i / 4][i % 4];
        });
        if (hidden_nan) {  // 0 NaN of a hidden key is 0
#pragma unroll
          for (int i = 0; i < 16; ++i) ps[i / 4][i % 4] = hide[n] >> i & 1 ? 0.0f : ps[i / 4][i % 4];
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int i = 0; i < 4; ++i) pf[n][hf][i] = pack2<F16>(ps[2 * hf][i], ps[2 * hf + 1][i]);
      }
      sfor<2>([&](auto hc) __attribute__((always_inline)) {
        constexpr int hf = decltype(hc)::value;
        u32x4 rf;
        sfor<4>([&](auto ic) __attribute__((always_inline)) {
          constexpr int i = decltype(ic)::value;
          const uint32_t a0 = row_bcast_u<8 * hf + i>(vr[g]), a1 = row_bcast_u<8 * hf + 4 + i>(vr[g]);
          rf[i] = __builtin_amdgcn_perm(a1, a0, offset_sel);
        });
#pragma unroll
        for (int n = 0; n < NQ; ++n) off[n][g] = mfma16<F16>(rf, pf[n][hf], off[n][g]);
      });
#pragma unroll
      for (int t = g * (G / 16); t < (g + 1) * (G / 16); ++t)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const u32x4 vf = code_frag(f.v[t / 2][2 * (t % 2) + hf]);
#pragma unroll
          for (int n = 0; n < NQ; ++n) acc[n][t] = mfma16<F16>(vf, pf[n][hf], acc[n][t]);
        }
    }
  };

  if (nblk > 0) {
    // The loads of the next block's keys follow this block's scores, those of
    // its values this block's outputs: each into the registers just read, so a
    // block is held once and its loads have most of a block's work to arrive in.
    // (With one tile, loading a whole block ahead takes 42 registers more and
    // gains nothing: 8 waves on a CU, 20.5 us over 4000 keys against 19.9.)
    auto rec_at = [&](int recs, int t) { return __shfl(recs, 4 * t + h, 64); };
    KvBlock<D, NG> f;
    int recs = records(0), rec = rec_at(recs, 0);
    load_keys(f, recs, 0);
    load_values(f, recs, 0);
    for (int t = 0; t < nblk; ++t) {
      // the next block (past the last one: record 0, loaded and not used)
      const int next = (t + 1) & 15;
      if (next == 0) recs = records(t + 1);
      compute(f, begin + t * stride, rec, [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        load_keys(f, recs, next);
      });
      __builtin_amdgcn_sched_barrier(0);
      load_values(f, recs, next);
      rec = rec_at(recs, next);
    }
  }

  // whole sums of each row, and the offsets' part of the outputs
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    sum[n] += __shfl_xor(sum[n], 16, 64);
    sum[n] += __shfl_xor(sum[n], 32, 64);
    float lsum[NG];  // rows 0 and 1 of the offset tile are with lane group 0
#pragma unroll
    for (int g = 0; g < NG; ++g) lsum[g] = __shfl(off[n][g][0] + off[n][g][1], c, 64) * 0x1p4f;
#pragma unroll
    for (int t = 0; t < DTL; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][t][i] = __builtin_fmaf(acc[n][t][i], 0x1p24f, lsum[16 * t / G]);
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
    // merge the waves: [wave][row] references and sums, then sums scaled
    // to the largest reference
    float* ml = lds;                // [NW][BM][2]
    float* od = lds + NW * BM * 2;  // [NW][BM][LDO]
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
      for (int w = 1; w < NW; ++w) top = fmaxf(top, ml[(w * BM + x) * 2]);
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
    for (int i = threadIdx.x; i < BM * (D / 4); i += 64 * NW) {
      const int x = i / (D / 4), d = 4 * (i % (D / 4));
      if (r0 + x >= nrows) continue;
      float top = ml[x * 2];
#pragma unroll
      for (int w = 1; w < NW; ++w) top = fmaxf(top, ml[(w * BM + x) * 2]);
      float total = 0.0f;
      f4 v = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        total += scale_sum(ml[(w * BM + x) * 2 + 1], ml[(w * BM + x) * 2] - top);
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

// Joins the parts of the keys: one workgroup per (row, head), as many parts at
// a time as it has rows of D / 4 threads, the parts of a thread and then the
// threads of a channel in order: a fixed order, so the same call gives the same
// bits.  Latency bound: 64 parts of 64 rows, D = 128, in 4.2 us (50 us with one
// wave that took the parts one after the other).
template <int DT, int D>
__global__ __launch_bounds__(256) void kv_join_kernel(const KvAttnArgs a) {
  constexpr int VL = D / 4;
  __shared__ float weight[kKvMaxSplits];
  __shared__ f4 red[256];
  const int64_t item = blockIdx.x, all = (int64_t)a.seqs.rows * a.q_heads;
  const int64_t row = item / a.q_heads;
  const int head = (int)(item - row * a.q_heads);
  // rows before the first or behind the last sequence belong to nobody
  if (a.seqs.cu_q && (row < kv_row_offset(a.seqs, 0) || row >= kv_row_offset(a.seqs, a.seqs.batch))) return;
  // every wave: weight of each part against the largest reference
  const int lane = threadIdx.x & 63;
  float r[2] = {kNone * 2.0f, kNone * 2.0f}, w[2] = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int s = lane + 64 * k;
    if (s < a.splits) {
      const float* ml = a.part_ml + ((int64_t)s * all + item) * 2;
      r[k] = ml[0];
      w[k] = ml[1];
    }
  }
  float top = fmaxf(r[0], r[1]);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  float total = 0.0f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float al = __builtin_amdgcn_exp2f(r[k] - top);
    // a part that saw no key holds nothing (NaN goes on)
    if (threadIdx.x < 64) weight[lane + 64 * k] = w[k] == 0.0f ? 0.0f : al;
    total += scale_sum(w[k], r[k] - top);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) total += __shfl_xor(total, o, 64);
  __syncthreads();
  const int par = blockDim.x / VL, x = threadIdx.x % VL, y = threadIdx.x / VL;
  f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (y < par) {
    const float* p = a.part + item * D + 4 * x;
#pragma unroll 4
    for (int s = y; s < a.splits; s += par) {
      const float al = weight[s];
      const f4 t = *(const f4*)(p + (int64_t)s * all * D);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = al == 0.0f ? v[i] : __builtin_fmaf(t[i], al, v[i]);
    }
  }
  red[threadIdx.x] = v;
  __syncthreads();
  if (y != 0) return;
  for (int k = 1; k < par; ++k) v += red[k * VL + x];
  const float inv = total != 0.0f ? 1.0f / total : 0.0f;
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  *(u32x2*)(a.out + row * a.ldo + (int64_t)head * D + 4 * x) =
      u32x2{pack2<DT>(v[0] * inv, v[1] * inv), pack2<DT>(v[2] * inv, v[3] * inv)};
}

// The same for few parts (at most 8) and any number of rows: D / 4 threads for
// a (row, head), which take its parts in order.
template <int DT, int D>
__global__ __launch_bounds__(256) void kv_join_few_kernel(const KvAttnArgs a) {
  constexpr int VL = D / 4, PER = 256 / VL;  // items of a workgroup
  const int x = threadIdx.x % VL, y = threadIdx.x / VL;
  const int64_t item = (int64_t)blockIdx.x * PER + y, all = (int64_t)a.seqs.rows * a.q_heads;
  if (y >= PER || item >= all) return;
  const int64_t row = item / a.q_heads;
  const int head = (int)(item - row * a.q_heads);
  if (a.seqs.cu_q && (row < kv_row_offset(a.seqs, 0) || row >= kv_row_offset(a.seqs, a.seqs.batch))) return;
  float r[8], w[8];
  float top = kNone * 2.0f, total = 0.0f;
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    r[s] = kNone * 2.0f;
    w[s] = 0.0f;
    if (s < a.splits) {
      const float* ml = a.part_ml + ((int64_t)s * all + item) * 2;
      r[s] = ml[0];
      w[s] = ml[1];
    }
    top = fmaxf(top, r[s]);
  }
  f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* p = a.part + item * D + 4 * x;
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    if (s >= a.splits || w[s] == 0.0f) continue;  // a part that saw no key (NaN goes on)
    const float al = __builtin_amdgcn_exp2f(r[s] - top);
    const f4 t = *(const f4*)(p + (int64_t)s * all * D);
    total += scale_sum(w[s], r[s] - top);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf(t[i], al, v[i]);
  }
  const float inv = total != 0.0f ? 1.0f / total : 0.0f;
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  *(u32x2*)(a.out + row * a.ldo + (int64_t)head * D + 4 * x) =
      u32x2{pack2<DT>(v[0] * inv, v[1] * inv), pack2<DT>(v[2] * inv, v[3] * inv)};
}

template <int DT, int NG, int NQ, bool ROWS, int NW = 4>
wq_status run(const KvAttnArgs& a) {
  constexpr int D = WQ_HEAD_DIM;
  const int64_t grid = (int64_t)a.slots * a.splits * a.seqs.kv_heads;
  hipLaunchKernelGGL((kv_attention_kernel<DT, D, NG, NQ, ROWS, NW>), dim3((unsigned)grid), dim3(64 * NW), 0, a.stream, a);
  wq_status st = launch_status();
  if (st != WQ_OK || a.splits == 1) return st;
  const int64_t items = (int64_t)a.seqs.rows * a.q_heads;
  // (32 rows of 8 parts: the whole call 14.3 us with the second kernel, 12.9 with
  // the first; 32000 rows of 2: 38.5 against 51.3)
  if (a.splits <= 8 && items >= 2048) {
    constexpr int PER = 256 / (D / 4);
    hipLaunchKernelGGL((kv_join_few_kernel<DT, D>), dim3((unsigned)((items + PER - 1) / PER)), dim3(256), 0, a.stream,
                       a);
  } else {
    hipLaunchKernelGGL((kv_join_kernel<DT, D>), dim3((unsigned)items), dim3(256), 0, a.stream, a);
  }
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
      constexpr int NQ = kv_two_tiles(WQ_HEAD_DIM, GG) ? 2 : 1;
      if (p.rows_form) st = run<DT, NG, NQ, true>(a);
      else if (p.nw == 8) st = run<DT, NG, 1, false, 8>(a);
      else if (p.nq == 1) st = run<DT, NG, 1, false>(a);
      else st = run<DT, NG, NQ, false>(a);
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
