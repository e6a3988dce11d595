// wq_kv.hpp -- layout of the 4-bit paged key/value cache and the device
// helpers its kernels share.
//
// A page holds `page_size` tokens of one layer for every kv head, as records
// of 16 tokens and one head (page_size is a power of two, at least 16):
//   cache[page][kv_head][page_size / 16] records of 16 D + 128 NG bytes,
//   D = head_dim, G = group, NG = D / G, W = D / 32:
//   * key codes, 8 D bytes: [token 16][word D / 8].  Word h W + kb of a token
//     holds channels 32 kb + 8 h .. + 7, channel e in bits 4 e .. 4 e + 3, so
//     the W consecutive words of lane (token, h) are its 16x16x32 MFMA
//     operands for the 32-channel blocks kb, and every block lies in one
//     quantisation group (G is a multiple of 32);
//   * value codes, 8 D bytes, transposed: word ((dt / 2) 16 + i) 4 + (dt % 2) 2
//     + half holds channel 16 dt + i of tokens 8 half .. 8 half + 7, token j in
//     bits 4 j .. 4 j + 3: a lane's 16 bytes are the MFMA operands of two
//     16-channel tiles whose inner dimension runs over the tokens, with no
//     transposition where the cache is read;
//   * key steps and offsets, uint32 [NG][token 16], s in the low and lo in the
//     high 16 bits (the model's 16-bit type), then the same for the values.
// A record is contiguous and a multiple of 128 bytes.  The price of the
// transposed values is paid by the write of part of a record, which reads the
// words it shares with the record's other tokens and writes them back.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wq_common.hpp"
#include "wq_decode.hpp"

namespace wq {

// Bytes of one record (16 tokens of one kv head).
__host__ __device__ constexpr int kv_record_bytes(int head_dim, int groups) { return 16 * head_dim + 128 * groups; }
constexpr bool kv_head_dim_ok(int d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }
constexpr bool kv_group_ok(int d, int g) { return (g == 32 || g == 64 || g == 128) && d % g == 0; }

// The sequences of a call, as every cache kernel sees them.  Nothing in device
// memory is trusted: row offsets, lengths and page numbers are held to the
// sizes the host knows, so a wrong entry gives a wrong result and never an
// access outside the buffers.
struct KvSeqs {
  const int32_t* table;  // [batch][max_pages]
  const int32_t* lens;   // [batch] tokens in the cache, the call's rows included
  const int32_t* cu_q;   // [batch + 1] row offsets, or null: rows / batch rows each
  int rows, batch, max_pages, num_pages;
  int rpp_shift;         // log2(records per page)
  int kv_heads;
};

__device__ inline int kv_row_offset(const KvSeqs& s, int b) {
  const int v = s.cu_q ? s.cu_q[b] : (int)((int64_t)s.rows / s.batch * b);
  return v < 0 ? 0 : v > s.rows ? s.rows : v;
}

// First row, number of rows, position of the first row (below 0 or past the
// table if the length says so) and length within the table of sequence b.
struct KvSeq {
  int row0, n, pos0, len;
};
__device__ inline KvSeq kv_seq(const KvSeqs& s, int b) {
  KvSeq q;
  q.row0 = kv_row_offset(s, b);
  q.n = kv_row_offset(s, b + 1) - q.row0;
  if (q.n < 0) q.n = 0;
  // (positions of the table are below 2^30 and rows at most 2^24: a length
  // beyond the first bound has all its rows past the table, and stays in 31 bits)
  int len = s.lens[b];
  if (len < 0) len = 0;
  if (len > (1 << 30) + (1 << 25)) len = (1 << 30) + (1 << 25);
  q.pos0 = len - q.n;
  const int cap = s.max_pages << (s.rpp_shift + 4);
  q.len = len < cap ? len : cap;
  return q;
}

// Work items ("slots") of ragged batches are numbered without a pass over the
// lengths: sequence b owns the slots from (row0 * mul) / per + b * extra on,
// which leaves it at least ceil(n * mul / per) (extra = 1) of them.  The wave
// finds the sequence of its slot by a 64-ary search; -1 if there is none.
__device__ inline int kv_find_seq(const KvSeqs& s, int64_t slot, int mul, int per, int extra, int lane) {
  int lo = 0, n = s.batch;
  for (;;) {
    const int step = (n + 63) >> 6;
    const int i = lane * step;
    bool p = false;
    if (i < n) p = (int64_t)kv_row_offset(s, lo + i) * mul / per + (int64_t)(lo + i) * extra <= slot;
    const int cnt = __popcll(__ballot(p));
    if (cnt == 0) return -1;
    const int at = (cnt - 1) * step;
    if (step == 1) return lo + at;
    lo += at;
    n = n - at < step ? n - at : step;
  }
}

// Record number of 16-token block r of sequence b for head `head`, or -1 when
// the block lies past the table or its page number is not a page.
__device__ inline int kv_record(const KvSeqs& s, int b, int r, int head) {
  const int page_i = r >> s.rpp_shift;
  if (r < 0 || page_i >= s.max_pages) return -1;
  const int page = s.table[(int64_t)b * s.max_pages + page_i];
  if (page < 0 || page >= s.num_pages) return -1;
  return (((page * s.kv_heads + head) << s.rpp_shift) + (r & ((1 << s.rpp_shift) - 1)));  // < 2^31: checked by the host
}

template <int DT>
__device__ inline float act_to_f32(uint32_t bits16) {
  return DT == F16 ? f16_to_f32((uint16_t)bits16) : __uint_as_float(bits16 << 16);
}
// low / high 16 bits of a word as fp32
template <int DT>
__device__ inline float act_lo(uint32_t w) {
  return DT == F16 ? f16_to_f32((uint16_t)w) : __uint_as_float(w << 16);
}
template <int DT>
__device__ inline float act_hi(uint32_t w) {
  return DT == F16 ? f16_to_f32((uint16_t)(w >> 16)) : __uint_as_float(w & 0xFFFF0000u);
}

// Host-side launchers (validated arguments).
struct KvAttnArgs {
  const uint16_t* q;
  int64_t ldq;           // elements between rows
  uint16_t* out;
  int64_t ldo;
  const uint8_t* cache;
  KvSeqs seqs;
  int q_heads, heads_per_kv;
  float scale_log2;      // scale * log2(e)
  int causal, window;
  int splits;            // parts the keys are split into
  float* part;           // splits > 1: [splits][rows * q_heads][D] sums, then (reference, weight) pairs
  float* part_ml;
  int slots, tiles;      // grid: row-tile slots; tiles per sequence (cu_q null)
  hipStream_t stream;
};

constexpr int kKvMaxSplits = 128;
// Launch shape of an attention call: a function of the sizes the host knows.
struct KvPlan {
  int rows_form;  // each wave its own rows (else the waves take the keys in turn)
  int nq;         // tiles of 16 rows per wave
  int nw;         // waves of a workgroup
  int splits;     // parts of the keys
  int slots, tiles;
};
// Whether a wave may take two row tiles (they share every code it unpacks):
// the sums of a tile take 16 registers per lane for every 64 channels, the
// offsets 4 for every group.  256 registers hold that for every pair but 128
// channels in groups of 64, which spills 11 to 13.
constexpr bool kv_two_tiles(int head_dim, int group) { return head_dim <= 128 && head_dim / group <= 2; }
// Waves per SIMD the registers of the one-tile key form leave room for.
constexpr int kv_key_waves(int head_dim, int group) {
  return head_dim == 64 || (head_dim == 128 && group == 128) ? 3 : 2;
}

inline KvPlan kv_plan(int rows, int batch, bool ragged, int heads_per_kv, int kv_heads, int head_dim,
                      int group, int64_t max_kv) {
  KvPlan p;
  // Packed rows (token, head) of a sequence, on average: the host does not know
  // the offsets of a ragged batch.  A long chunk beside many single tokens then
  // runs in a form that suits only one of them: 500 rows and 50 single ones of 32
  // heads (8 of the cache) over 4000 keys take 159 us, 63 and 36 as two calls.
  const int64_t per = ((int64_t)rows * heads_per_kv + batch - 1) / batch;
  p.rows_form = per > 32;
  p.nq = per > 16 && kv_two_tiles(head_dim, group) ? 2 : 1;
  const int bm = (p.rows_form ? 64 : 16) * p.nq;
  p.tiles = (int)((per + bm - 1) / bm);
  p.slots = ragged ? (int)((int64_t)rows * heads_per_kv / bm + batch) : p.tiles * batch;
  // Parts.  Row form: about two workgroups to a CU (its limit by registers).
  // Key form: 256 workgroups of four waves already take the memory's rate, so
  // the parts only even out what each CU gets: the part count of least
  // ceil(workgroups / 256) / parts, with 4 % for every workgroup of a CU.
  // (131071 keys of 8 heads: 34.9 us with 256 workgroups, 35.7 with 512, 39.1 with
  // 768; 192 workgroups over up to 16000 keys: 84 us whole, 60 in 4 parts; 256
  // over up to 4000: 26.7 us whole, 28.8 in 2.)  A part has at least one round
  // of blocks of 64 keys in the key form (a row over 1037 keys, 32 heads: 10.0 us
  // in 5 parts, 11.7 in 2), four blocks in the row form.
  const int64_t wgs = (int64_t)p.slots * kv_heads;
  const int64_t rounds = p.rows_form ? max_kv / 256 : (max_kv + 255) / 256;
  int64_t s = p.rows_form ? (wgs >= 512 ? 1 : 512 / wgs) : 1;
  if (!p.rows_form) {
    double best = 1e30;
    for (int64_t t = 1; t <= kKvMaxSplits && t <= rounds && (t == 1 || t * wgs <= 1024); ++t) {
      const double cost = (double)((t * wgs + 255) / 256) / (double)t * (1.0 + 0.04 * (double)(t * wgs) / 256.0);
      if (cost < best) {
        best = cost;
        s = t;
      }
    }
  }
  if (s > rounds) s = rounds;
  if (s > kKvMaxSplits) s = kKvMaxSplits;
  p.splits = s < 1 ? 1 : (int)s;
  p.nw = 4;
  // Short contexts of few rows take one workgroup of eight waves instead of
  // parts and their join.  On the GPU, 32 heads of 128 / 64 heads of 64, in us
  // against parts: 7.8 : 9.7 / 6.4 : 8.8 over 512 keys, 10.0 : 9.8 / 7.9 : 8.9
  // over 1037, 10.1 : 9.8 / 8.1 : 8.8 over 1280, 11.1 : 9.8 / 8.9 : 8.9 over 1536,
  // 12.8 : 9.9 / 10.1 : 8.9 over 2048.  A call that is not captured (one launch,
  // no workspace) is bound by the host: 10.1 against 14.1 up to 1280, 12.6 against
  // 14.0 over 2048.
  if (!p.rows_form && p.nq == 1 && p.splits > 1 && max_kv <= 1280) {
    p.nw = 8;
    p.splits = 1;
  }
  return p;
}
// Workspace: sums of every part, then (reference, weight) pairs.
inline size_t kv_part_bytes(const KvPlan& p, int rows, int q_heads, int head_dim) {
  return p.splits > 1 ? (size_t)p.splits * rows * q_heads * head_dim * 4 : 0;
}
inline size_t kv_ml_bytes(const KvPlan& p, int rows, int q_heads) {
  return p.splits > 1 ? (size_t)p.splits * rows * q_heads * 8 : 0;
}

wq_status launch_kv_rows(bool write, const KvSeqs& s, uint8_t* cache, uint16_t* k, uint16_t* v, int64_t ld_k,
                         int64_t ld_v, int dt, int D, int G, hipStream_t stream);
#define WQ_DECLARE_HEAD_DIM(d) wq_status launch_kv_attention_##d(const KvAttnArgs& a, int dt, int G, const KvPlan& p);
WQ_DECLARE_HEAD_DIM(64)
WQ_DECLARE_HEAD_DIM(96)
WQ_DECLARE_HEAD_DIM(128)
WQ_DECLARE_HEAD_DIM(192)
WQ_DECLARE_HEAD_DIM(256)
#undef WQ_DECLARE_HEAD_DIM

}  // namespace wq
