// wq_lora.hip -- low-rank adapters of many sequences beside a shared projection.
//
// out = y + scale (x A^T) B^T, each row with its sequence's adapter, in two
// products on the matrix cores: v = x A^T in fp32 parts of the K axis, then
// v B^T added to y.  Rows are taken in tiles of 64 whatever sequences they belong
// to; a tile works through the distinct adapters among its rows, each read once
// for all of that adapter's rows in the tile, other rows left out of loads and
// stores.  Where rows are few the tile's work items -- an adapter and up to four
// (first product) or 16 (second) of its rows -- are spread over workgroups.
//
// v is fp32 and enters the second product as a sum of two 16-bit numbers: with
// one, its rounding alone would show as much as the output's own.  For fp16 each
// row's v is first scaled by a power of two into the upper range of the type,
// exactly, and back behind the product.
//
// What bounds them (MI355X, graph-replayed, banks and rows from memory).  Few rows:
// launches and the chain offsets -> adapter -> rank -> data; one row of rank 16
// beside 4096 -> 4096 takes 6.3 us for 0.3 MB, 64 tokens of 40 adapters of ranks 8
// to 32 beside 8192 -> 10240 20.8 us for 52 MB (first product 10.8 us at 3.3
// TB/s, second 9.2).  Many: 6400 prompt rows of rank 64 beside 4096 -> 12288 take
// 101 us: 30 us for x A^T (LDS and the latency of its stages), 6 to put its parts
// together, 63 us for the 315 MB of y and out (5.0 TB/s, y partly from the caches; a copy: 4.75).
#include "wq_layer.hpp"

namespace wq {
namespace {

// Shape of a call, a function of the sizes the host knows.
struct LoraPlan {
  int few;     // the first product row by row
  int groups;  // workgroups that share a tile's work items, second product
  int first;   // and first product
  int splits;  // parts of K
  int blocks;  // blocks of 128 columns per workgroup (second product)
};
// Items of up to four rows that a tile of 64 rows has, with sequences of one length and an
// adapter to each: what a workgroup of their own is launched for (more are taken in turn;
// with as many workgroups as sequences 64 rows of one sequence took 47 us, now 9.5).
int few_items(int rows, int batch) {
  const int tile = rows < 64 ? rows : 64;
  const int64_t seqs = ((int64_t)batch * tile + rows - 1) / rows;
  return seqs < tile ? (int)seqs + (tile - (int)seqs) / 4 : tile;
}
// (Where `part` lies and how long it is follows from the first four alone.)
LoraPlan lora_plan(int rows, int batch, int K, int columns, int N = 0, int kinds = 1) {
  LoraPlan p;
  // Row by row up to 128 rows, and up to 1024 where there are not many to a sequence, else
  // in tiles of 64 (us, ranks 16 and 64; 4096 -> 6144): 128 single rows of 200 adapters 27 56
  // : 37 72, of one adapter 11 17 : 13 15; 256 rows of 200 adapters 41 82 : 57 110, of
  // sequences of 16 rows 14 20 : 16 20, of one sequence 13 19 : 14 17; 300 rows, five to a
  // sequence 20 40 : 26 39; 1000 single rows of 100 adapters 101 258 : 161 344, of 8 adapters
  // 39 88 : 40 67, five to a sequence 48 125 : 51 100; 4000 rows 360 974 : 544 1071 and 151 383
  // : 106 189.  Rank and number of adapters are not in the rule, and where they decide it
  // is up to a third off: 1000 single rows of 8 adapters of rank 64 run in the 88 of these,
  // 128 single rows of one adapter of that rank in the 17.
  p.few = rows <= 128 || (rows <= 1024 && (int64_t)rows * rows <= (int64_t)3000 * batch);
  if (p.few) {
    p.first = p.groups = few_items(rows, batch);
  } else {
    // as many workgroups as a tile has sequences on average, or as there are adapters (and
    // none); the first product one more, which most tiles of prompts send home, so that a
    // tile of two takes no longer than the others.  The average suits neither part of a
    // mixed batch: the tile of single tokens beside a prompt works through its adapters in
    // turn (63 tokens of 40 adapters and 1000 rows of one more, ranks 16 and 64: 110 and
    // 148 us; as two calls 19 + 19 and 31 + 24)
    const int64_t seqs = (int64_t)batch * 64 / rows, most = kinds < 64 ? kinds : 64;
    p.groups = (int)(seqs < 1 ? 1 : seqs > most ? most : seqs);
    p.first = p.groups + (batch > 1 && p.groups < most);
  }
  const int64_t tiles = ((int64_t)rows + 63) / 64, width = p.few ? 16 : 64;
  const int64_t wgs = tiles * (p.few ? p.groups : 1) * ((columns + width - 1) / width);
  if (p.few) {
    // about 1024 workgroups, of which those without an item leave at once, and 1024 of K
    // to each (64 tokens of 40 adapters: 10.9 us, 12.9 with 2048, 19.3 with 4096)
    int64_t s = 1024 / wgs;
    if (s > K / 1024) s = K / 1024;
    p.splits = s < 1 ? 1 : s > 16 ? 16 : (int)s;
  } else {
    // rounds of two workgroups per CU, and 1.5 % of one for every part that is written
    // and read back (6400 rows of 192 columns: 129 us in one part, 117 in five)
    double best = 1e30;
    for (int s = 1; s == 1 || (s <= 16 && s * 512 <= K); ++s) {
      const double cost = (double)((wgs * s + 511) / 512) / s + 0.015 * s;
      if (cost < best) {
        best = cost;
        p.splits = s;
      }
    }
  }
  // 1280 to 2560 workgroups (64 tokens of 40 adapters: 20.2 us, 21.6 with 640, 25.9 with
  // 3840), each with a power of two of column blocks: a tile's workgroups are then mostly a
  // multiple of the eight XCDs, whose caches so keep the same columns' B (the prompts'
  // second product 63.4 us with 24 workgroups a tile; 70.6 with 15, 68 with 18 or 21, 67.3
  // with 33)
  const int64_t blocks = (int64_t)((N + 127) / 128) * tiles * p.groups / 1280;
  p.blocks = blocks < 2 ? 1 : blocks < 4 ? 2 : blocks < 8 ? 4 : 8;
  return p;
}

// One launch, for calls whose time is launches; every workgroup then reads the slice's A
// for itself.  Captured, two launches : one, us, beside 4096 -> 4096 (or 3 x 4096): one
// row of rank 16 7.3 : 6.3 (7.4 : 6.4), of rank 32 7.4 : 8.3, of 11008 -> 4096 8.6 : 8.5;
// 16 rows of one adapter of rank 16 8.1 : 7.9, of many (11.5 : 11.6) to (14.4 : 11.8), of
// rank 8 from 11008 9.4 : 11.3; 64 rows of one 10.1 : 11.6.  Not captured, the launch
// and the workspace it saves are 3.5 us of host time, and that is why some shapes that
// lose up to 1.9 us captured are in: rank 32 up to K = 2048 (one row 7.4 : 8.2, four of
// four adapters 7.8 : 8.5, 16 of 16 8.6 : 10.3), four rows of one adapter from 8192 (8.7 :
// 9.1) and 11008 (9.4 : 10.6), 16 rows of rank 8 from 8192 (8.8 : 10.6).  Up to rank 16 and
// K = 2048 one launch gains everywhere (7.4 : 6.2 to 8.6 : 7.4).  Out of it: rank 32 from
// 4096 (one row 7.6 : 8.3, 16 rows of 16 9.5 : 12.3) and 11008 (8.8 : 12.5), 16 rows of rank
// 16 from 8192 (9.0 : 10.7).
bool lora_fused(int rows, int K, int rank) {
  if (rank > 32) return false;
  return rows <= 4 && rank <= 16 ? rank * K <= 180224 : rows <= 16 && rank * K <= 65536;
}

__device__ inline u32x4 load16(rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0);
}
// (The offset is added up here: behind a 128-bit store with a scalar offset the compiler
// may rewrite the first data register in the very next instruction, and that value then
// reached memory now and then; without one it keeps the distance.)
__device__ inline void store16(rsrc_t r, u32x4 v, uint32_t off) { __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, 0); }

// Adapter of row row0 + lane (lane < TM): -1 for none, -2 outside every sequence.
// The wave finds the first row's sequence and walks the offsets of those behind it
// that begin in the tile.
template <int TM>
__device__ inline int tile_adapters(const LoraArgs& a, int row0, int lane) {
  const KvSeqs& s = a.seqs;
  int seq = -1;
  if (!s.cu_q) {
    if (lane < TM && row0 + lane < s.rows) seq = (uint32_t)(row0 + lane) / (uint32_t)(s.rows / s.batch);
  } else if (s.batch < 64) {  // all offsets at once, and the adapters with them
    const int off = lane <= s.batch ? kv_row_offset(s, lane) : 0x7FFFFFFF;
    const int each = lane < s.batch ? a.adapters[lane] : -1;
    const int row = row0 + lane;
    seq = __popcll(__ballot(off <= row0)) - 1;
    uint64_t inside = __ballot(off > row0 && off < row0 + TM);
    while (inside) {
      const int i = __builtin_ctzll(inside);
      inside &= inside - 1;
      if (row >= __builtin_amdgcn_readlane(off, i)) seq = i;
    }
    const int id = __shfl(each, seq & 63, 64);
    if (lane >= TM || row >= s.rows || seq < 0 || seq >= s.batch) return -2;
    return id < 0 || id >= a.num ? -1 : id;
  } else {
    int first = kv_find_seq(s, row0, 1, 1, 0, lane);
    first = __builtin_amdgcn_readfirstlane(first < 0 ? 0 : first);
    const int row = row0 + lane, off = first + lane <= s.batch ? kv_row_offset(s, first + lane) : 0x7FFFFFFF;
    uint64_t inside = __ballot(off < row0 + TM);
    if (inside >> 63) {  // more than 63 sequences begin in the tile, most of them without rows
      for (int i = 0; i < TM; ++i) {
        int b = kv_find_seq(s, row0 + i, 1, 1, 0, lane);
        if (b >= 0 && row0 + i >= kv_row_offset(s, s.batch)) b = -1;
        if (lane == i) seq = b;
      }
    } else {
      seq = -1;
      while (inside) {
        const int i = __builtin_ctzll(inside);
        inside &= inside - 1;
        if (row >= __builtin_amdgcn_readlane(off, i)) seq = first + i;
      }
    }
    if (seq >= s.batch || row0 + lane >= s.rows) seq = -1;
  }
  if (seq < 0) return -2;
  const int id = a.adapters[seq];
  return id < 0 || id >= a.num ? -1 : id;
}
__device__ inline int adapter_rank(const LoraArgs& a, int id) {
  int r = a.rank;
  asm("" : "+s"(r));  // (keeps the compiler from choosing between two addresses by a flat load)
  if (a.ranks) r = a.ranks[id];
  return __builtin_amdgcn_readfirstlane(r < 0 ? 0 : r > a.rank ? a.rank : r);
}

// f(adapter, first) for the distinct values (from `least` on) among the 64 lanes' ids and
// every PER of the rows that have one (0: all of them together): every `of`-th of these
// items, from the `at`-th on.
template <int PER, typename F>
__device__ inline void each_adapter(int ids, int least, int at, int of, F&& f) {
  uint64_t left = __ballot(ids >= least);
  for (int skip = at; left;) {
    const int cur = __builtin_amdgcn_readlane(ids, __builtin_ctzll(left));
    const uint64_t same = __ballot(ids == cur);
    left &= ~same;
    const int items = PER ? (__popcll(same) + PER - 1) / (PER ? PER : 1) : 1;
    for (; skip < items; skip += of) f(cur, skip * PER);
    skip -= items;
  }
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));
// 16 products of 4 x 4 numbers along 4 of K each: lane 4 b + i gives row i of the
// first and column i of the second operand of product b, four entries of K, and gets
// column i of its result: result i of lane i is what its own operands give.
template <int DT>
__device__ inline f4 mfma4(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, f4 c) {
  const u32x2 a = {a0, a1}, b = {b0, b1};
  if constexpr (DT == F16)
    return __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(h4, a), __builtin_bit_cast(h4, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s4, a), __builtin_bit_cast(s4, b), c, 0, 0, 0);
}
// sum over the 16 lanes of a row
__device__ inline float sum_row(float v) {
  auto ror = [&](auto n) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + decltype(n)::value, 0xf, 0xf, true));
  };
  ror(std::integral_constant<int, 8>{});
  ror(std::integral_constant<int, 4>{});
  ror(std::integral_constant<int, 2>{});
  ror(std::integral_constant<int, 1>{});
  return v;
}

// v = x A^T for few rows: 16 rows of A for the rows of x that share the adapter, up to
// four of them to a workgroup.  The work is to read A: consecutive lanes take consecutive
// 16 bytes (a load is 256 bytes of four rows), every lane multiplies its entries of A and
// x, and the lanes are added up at the end.  (As operands of the 16-row product a load
// would be 64 bytes of sixteen rows at a stride of 16 lanes: 18.2 us instead of 10.8 for
// 64 tokens of 40 adapters.)  The four waves (and the parts) split K.
template <int DT>
__global__ __launch_bounds__(256, 3) void lora_shrink_rows_kernel(const LoraArgs a, int splits) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row0 = blockIdx.x * 64, C = a.slices * a.rank;
  const int split = blockIdx.y % splits, col0 = blockIdx.y / splits * 16;
  const int ids = tile_adapters<64>(a, row0, lane);
  const int left = a.seqs.rows - row0, tile_rows = __builtin_amdgcn_readfirstlane(left < 64 ? left : 64);
  const rsrc_t xr = make_rsrc(a.x + (int64_t)row0 * a.K, (uint32_t)tile_rows * a.K * 2);
  const int units = a.K / 128, part = split * 4 + wave, parts = splits * 4;
  const int k0 = (int)((int64_t)units * part / parts) * 128, k1 = (int)((int64_t)units * (part + 1) / parts) * 128;
  __shared__ float red[4][4][16];  // [wave][row of x][row of A]

  each_adapter<4>(ids, 0, blockIdx.z, gridDim.z, [&](int cur, int before) {
    const int rank = adapter_rank(a, cur);
    // rows of A past the rank are not read (rank is a multiple of 8: eight of the 16 rows
    // lie in one slice)
    const int n0 = rank - col0 % a.rank, n1 = rank - (col0 + 8) % a.rank;
    if (n0 <= 0 && (n1 <= 0 || col0 + 8 >= C)) return;
    uint32_t ao[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int j = 4 * r + (lane >> 4);
      const bool ok = col0 + j < C && (j & 7) < (r < 2 ? n0 : n1);
      ao[r] = ok ? ((uint32_t)(col0 + j) * a.K + 8 * (lane & 15)) * 2 : kOutOfRange;
    }
    const rsrc_t ar = make_rsrc(a.a + (int64_t)cur * C * a.K, (uint32_t)C * a.K * 2);
    uint64_t mask = __ballot(ids == cur);
    for (int i = 0; i < before; ++i) mask &= mask - 1;
    auto product = [&](auto tg) {
      constexpr int TG = decltype(tg)::value, D = TG == 1 ? 4 : 2;
      uint32_t xo[TG];
      int row[TG];
#pragma unroll
      for (int t = 0; t < TG; ++t) {
        row[t] = mask ? __builtin_ctzll(mask) : -1;
        mask &= mask - 1;
        xo[t] = row[t] >= 0 ? ((uint32_t)row[t] * a.K + 8 * (lane & 15)) * 2 : kOutOfRange;
      }
      f4 acc[4][TG] = {};
      // a ring of D units of 128 along K: all but one in flight while that one is
      // multiplied (past the end of the range the loads read nothing)
      u32x4 af[D][4], xf[D][TG];
      auto load = [&](int b, int k) {
#pragma unroll
        for (int r = 0; r < 4; ++r) af[b][r] = load16(ar, ao[r] | (k < k1 ? 0u : kOutOfRange), k * 2);
#pragma unroll
        for (int t = 0; t < TG; ++t) xf[b][t] = load16(xr, xo[t] | (k < k1 ? 0u : kOutOfRange), k * 2);
      };
      auto multiply = [&](int b) {
#pragma unroll
        for (int q = 0; q < 4; q += 2)
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int t = 0; t < TG; ++t)
              acc[r][t] = mfma4<DT>(af[b][r][q], af[b][r][q + 1], xf[b][t][q], xf[b][t][q + 1], acc[r][t]);
      };
      int k = k0;
      if (k < k1) {
#pragma unroll
        for (int u = 0; u < D - 1; ++u) load(u, k + 128 * u);
      }
      for (; k + 128 * (D - 1) < k1; k += 128 * D)
#pragma unroll
        for (int u = 0; u < D; ++u) {
          load((u + D - 1) % D, k + 128 * (u + D - 1));
          multiply(u);
        }
#pragma unroll
      for (int u = 0; u < D - 1; ++u)
        if (k + 128 * u < k1) multiply(u);
      __syncthreads();  // (the last product's sums are read)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int t = 0; t < TG; ++t) {
          const f4 v = acc[r][t];
          const float own = lane & 2 ? (lane & 1 ? v[3] : v[2]) : (lane & 1 ? v[1] : v[0]);
          const float s = sum_row(own);
          if ((lane & 15) == 0) red[wave][t][4 * r + (lane >> 4)] = s;
        }
      __syncthreads();
      if (threadIdx.x < 16 * TG) {
        const int t = threadIdx.x >> 4, j = threadIdx.x & 15;
        float v = (red[0][t][j] + red[1][t][j]) + (red[2][t][j] + red[3][t][j]);
        if ((j & 7) >= (j < 8 ? n0 : n1)) v = 0.f;  // (0 x is not 0 for every x)
        int to = row[0];
#pragma unroll
        for (int o = 1; o < TG; ++o) to = t == o ? row[o] : to;
        if (to >= 0 && col0 + j < C) a.part[((int64_t)split * a.seqs.rows + row0 + to) * C + col0 + j] = v;
      }
    };
    if (mask & (mask - 1)) product(std::integral_constant<int, 4>{});
    else product(std::integral_constant<int, 1>{});
  });
}

// A buffer resource as the four words make_rsrc puts into it.
__device__ inline u32x4 words_of(const void* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  return u32x4{(uint32_t)b, (uint32_t)(b >> 32) & 0xFFFFu, bytes, 0x00020000u};
}
// 16 bytes per lane into LDS (lane l writes lds[l]; lds is wave-uniform).  By
// hand, because of what the compiler does behind its own form of it: it waits for
// all such loads in flight before any LDS read that it cannot tell from them.
// The waits are barrier_behind's.
__device__ inline void load_lds(u32x4 r, const void* lds, uint32_t voff, uint32_t soff) {
  const uint32_t to = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)lds;
  uint32_t kept;  // m0 is the compiler's
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds\n\ts_mov_b32 m0, %0"
               : "=&s"(kept) : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(voff), "s"(r), "s"(soff) : "memory");
}

// Barrier of a workgroup that waits until at most n vector memory operations of
// this wave are outstanding and all its LDS reads are done (s_waitcnt, gfx9
// encoding).  __syncthreads would wait for every LDS-destination load in flight.
template <int N>
__device__ inline void barrier_behind() {
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// v = x A^T for many rows: 64 rows of x and 64 of A, 64 of K at a time, in a ring of
// three stages in LDS that LDS-destination loads fill, two of them in flight (two stages
// 32 us, three 31, four 34 for 6400 rows of 192 columns: three leave room for three
// workgroups on a CU).  A load takes 128 consecutive bytes of eight rows by consecutive
// lanes (operands loaded straight into registers, 64 bytes of sixteen rows at a stride of
// 16 lanes, took 55 us); 16-byte chunk j of a row lies at j ^ (row % 8), so that the
// operands are read without bank conflicts.  A wave multiplies all the rows by 16 of A.
template <int DT>
__global__ __launch_bounds__(256) void lora_shrink_kernel(const LoraArgs a, int splits) {
  constexpr int S = 3, LOADS = 4;  // stages; loads of a wave for one, two of x and two of A
  __shared__ u32x4 stage[S][8 * 128];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, h = lane >> 4;
  const int row0 = blockIdx.x * 64, C = a.slices * a.rank;
  const int split = blockIdx.y % splits, col0 = blockIdx.y / splits * 64;
  const int ids = tile_adapters<64>(a, row0, lane);
  const int left = a.seqs.rows - row0, tile_rows = __builtin_amdgcn_readfirstlane(left < 64 ? left : 64);
  const u32x4 xr = words_of(a.x + (int64_t)row0 * a.K, (uint32_t)tile_rows * a.K * 2);
  const int units = a.K / 64;
  const int u0 = (int)((int64_t)units * split / splits), u1 = (int)((int64_t)units * (split + 1) / splits);

  each_adapter<0>(ids, 0, blockIdx.z, gridDim.z, [&](int cur, int) {
    const int rank = adapter_rank(a, cur);
    const u32x4 ar = words_of(a.a + (int64_t)cur * C * a.K, (uint32_t)C * a.K * 2);
    // rows of others and past the rank are not loaded: what lies in their places only
    // reaches results that are not kept
    const int lr = lane >> 3;
    const uint32_t lk = (uint32_t)((lane & 7) ^ lr) * 16;
    uint32_t off[LOADS];
    bool any = false;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int q = wave + 4 * i;
      if (i < 2) {
        const int row = 8 * q + lr;
        off[i] = __shfl(ids, row, 64) == cur ? (uint32_t)row * a.K * 2 + lk : kOutOfRange;
      } else {
        const int j = col0 + 8 * (q - 8) + lr;
        const bool ok = j < C && j % a.rank < rank;
        any |= ok;
        off[i] = ok ? (uint32_t)j * a.K * 2 + lk : kOutOfRange;
      }
    }
    if (!__syncthreads_or(any)) return;  // (also: the last adapter's stages are read)
    auto issue = [&](int u) {
      const u32x4* to = stage[(u - u0) % S];
#pragma unroll
      for (int i = 0; i < LOADS; ++i) load_lds(i < 2 ? xr : ar, to + (wave + 4 * i) * 64, off[i], (uint32_t)u * 128);
    };
    f4 acc[4] = {};
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
      if (u0 + i < u1) issue(u0 + i);
    for (int u = u0; u < u1; ++u) {
      // stage u is there for all, and stage u - 1 has been read by all
      if (u + 1 < u1) barrier_behind<LOADS>();
      else barrier_behind<0>();
      if (u + S - 1 < u1) issue(u + S - 1);
      const u32x4* from = stage[(u - u0) % S];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int at = (4 * k + h) ^ (c & 7);
        const u32x4 af = from[(64 + 16 * wave + c) * 8 + at];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] = mfma16<DT>(af, from[(16 * r + c) * 8 + at], acc[r]);
      }
    }
    const int j = col0 + 16 * wave + 4 * h, past = rank - j % a.rank;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      f4 v = acc[r];
#pragma unroll
      for (int q = 0; q < 4; ++q)  // (0 x is not 0 for every x)
        if (q >= past) v[q] = 0.f;
      if (__shfl(ids, 16 * r + c, 64) == cur && j < C)
        *(f4*)(a.part + ((int64_t)split * a.seqs.rows + row0 + 16 * r + c) * C + j) = v;
    }
  });
}

// 8 entries of v times a power of two as the sum of two 16-bit numbers.
template <int DT>
__device__ inline void two_parts(f4 v0, f4 v1, float up, u32x4& hi, u32x4& lo) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const f4 v = q < 2 ? v0 : v1;
    const float x0 = v[2 * (q % 2)] * up, x1 = v[2 * (q % 2) + 1] * up;
    const uint32_t w = pack2<DT>(x0, x1);
    const float h0 = act_lo<DT>(w), h1 = act_hi<DT>(w);
    hi[q] = w;
    // (an infinity is whole in its first part)
    lo[q] = pack2<DT>(__builtin_isinf(h0) ? 0.f : x0 - h0, __builtin_isinf(h1) ? 0.f : x1 - h1);
  }
}
// The largest finite one: beside an infinity the others must stay within fp16 too, or
// they would be infinities of either sign.
__device__ inline float largest(f4 a, f4 b) {
  float m = 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float x = fabsf(a[q]), y = fabsf(b[q]);
    m = fmaxf(m, fmaxf(x < __builtin_inff() ? x : 0.f, y < __builtin_inff() ? y : 0.f));
  }
  return m;
}
// fp16: the power of two that takes a row's largest to 2^13 .. 2^14, and the one back,
// both normal numbers (m is below 2^53: 2^20 products of numbers below 2^16)
__device__ inline void powers(float m, float& up, float& down) {
  int e = (int)(__float_as_uint(m) >> 23) - 127;
  e = e < -100 ? -100 : e;  // (tiny)
  up = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
  down = __uint_as_float((uint32_t)(127 - 13 + e) << 23);
}

// A row's v as it enters the second product (lane (c, h): entries 32 k + 8 h .. + 7 of
// lane c's row), the parts of K added up; returns the power of two that undoes its own.
template <int DT, int KC>
__device__ inline float split_v(const LoraArgs& a, int splits, int row, bool own, int slice, int rank, int h, u32x4* hi,
                                u32x4* lo) {
  const int C = a.slices * a.rank;
  f4 v[KC][2] = {};
  if (own) {
    const float* part = a.part + (int64_t)row * C + slice * a.rank + 8 * h;
    const int64_t next = (int64_t)a.seqs.rows * C;
    constexpr int P = 4 / KC;  // parts that are loaded together
    for (int p = 0; p < splits; p += P, part += P * next) {
      f4 w[P][KC][2] = {};
#pragma unroll
      for (int o = 0; o < P; ++o)
#pragma unroll
        for (int k = 0; k < KC; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (p + o < splits && 32 * k + 8 * h + 4 * i < rank) w[o][k][i] = *(const f4*)(part + o * next + 32 * k + 4 * i);
#pragma unroll
      for (int o = 0; o < P; ++o)
#pragma unroll
        for (int k = 0; k < KC; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) v[k][i] += w[o][k][i];
    }
  }
  float up = 1.f, down = 1.f;
  if constexpr (DT == F16) {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < KC; ++k) m = fmaxf(m, largest(v[k][0], v[k][1]));
    m = fmaxf(m, __shfl_xor(m, 16, 64));
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    powers(m, up, down);
  }
#pragma unroll
  for (int k = 0; k < KC; ++k) two_parts<DT>(v[k][0], v[k][1], up, hi[k], lo[k]);
  return down;
}

// The same once for all workgroups that will use it, where they are many: 16 rows of one
// slice, 16 lanes to a row.  The parts go to [row][slice][first, second][rank], the
// powers behind them.
template <int DT>
__global__ __launch_bounds__(256) void lora_split_kernel(const LoraArgs a, int splits) {
  const int row0 = blockIdx.x * 16, slice = blockIdx.y, C = a.slices * a.rank, i = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int id = __shfl(tile_adapters<16>(a, row0, threadIdx.x & 63), r, 64);
  if (id < 0) return;  // (the same in the 16 lanes)
  const int64_t next = (int64_t)a.seqs.rows * C;
  const int rank = a.ranks ? a.ranks[id] : a.rank, row = row0 + r;
  f4 v[2] = {};
  const float* part = a.part + (int64_t)row * C + slice * a.rank + 8 * i;
  for (int p = 0; p < splits; p += 4, part += 4 * next) {
    f4 w[4][2] = {};
#pragma unroll
    for (int o = 0; o < 4; ++o)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (p + o < splits && 8 * i + 4 * e < rank && 8 * i < a.rank) w[o][e] = *(const f4*)(part + o * next + 4 * e);
#pragma unroll
    for (int o = 0; o < 4; ++o)
#pragma unroll
      for (int e = 0; e < 2; ++e) v[e] += w[o][e];
  }
  float up = 1.f, down = 1.f;
  if constexpr (DT == F16) {
    float m = largest(v[0], v[1]);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
    powers(m, up, down);
  }
  u32x4 hi, lo;
  two_parts<DT>(v[0], v[1], up, hi, lo);
  if (8 * i < a.rank) {
    u32x4* to = (u32x4*)a.v + ((int64_t)row * a.slices + slice) * (a.rank >> 2) + i;
    to[0] = hi;
    to[a.rank >> 3] = lo;
  }
  if (i == 0) a.down[(int64_t)row * a.slices + slice] = down;
}

// out = y + scale v B^T; KC: blocks of 32 of the rank.  A workgroup takes 64 rows and
// `blocks` blocks of 128 columns of one slice.  B goes through LDS: consecutive threads
// load consecutive 16 bytes of it (chunk s of a block, which belongs to column s / R8, R8 to
// a column, lies at s ^ (s / 8 R8 % 16), % 8 with odd R8: that spreads the operands over
// the banks), and column 8 j + t is column j of tile t, so that
// the results of the eight tiles are eight consecutive columns of four rows in a lane:
// y is read and out written 256 consecutive bytes at a time.  (With 64 bytes of sixteen
// rows a load, B straight from memory: 91 us instead of 75 for the prompts.)  Many rows:
// a wave to 16 of them, all eight tiles.  Few: the waves share up to 16 rows of an
// adapter and take two tiles each.
template <int DT, bool FEW, int KC>
__global__ __launch_bounds__(256, KC == 4 ? 2 : 3) void lora_expand_kernel(const LoraArgs a, int splits, int blocks, uint32_t chunks) {
  constexpr int NT = FEW ? 2 : 8, NL = 2 * KC;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, h = lane >> 4;
  const int row0 = (int)(blockIdx.x / chunks) * 64, R8 = a.rank >> 3, magic = (65535 + R8) / R8;  // x / R8 = x magic >> 16, x < 2048
  const int spread = R8 & 1 ? 7 : 15;
  int slice = 0, first = 0, end = a.ends[0], chunk = (int)(blockIdx.x % chunks);
  for (;;) {
    const int n = (end - first + 128 * blocks - 1) / (128 * blocks);
    if (chunk < n) break;
    chunk -= n;
    first = end;
    end = a.ends[++slice];
  }
  const int base0 = first + chunk * blocks * 128, stop = base0 + blocks * 128 < end ? base0 + blocks * 128 : end;
  const int ids = tile_adapters<64>(a, row0, lane);
  const int left = a.seqs.rows - row0, tile_rows = __builtin_amdgcn_readfirstlane(left < 64 ? left : 64);
  const rsrc_t yr = make_rsrc(a.y + (int64_t)row0 * a.N, (uint32_t)tile_rows * a.N * 2);
  const rsrc_t outr = make_rsrc(a.out + (int64_t)row0 * a.N, (uint32_t)tile_rows * a.N * 2);
  __shared__ u32x4 stage[2][512 * KC];
  int buf = 0;

  each_adapter<FEW ? 16 : 0>(ids, a.y == a.out ? 0 : -1, blockIdx.z, gridDim.z, [&](int cur, int before) {
    const int rank = cur < 0 ? 0 : adapter_rank(a, cur);
    const float scale = cur < 0 ? 0.f : a.scales[cur];
    const rsrc_t br = make_rsrc(a.b + (int64_t)(cur < 0 ? 0 : cur) * a.N * a.rank, (uint32_t)a.N * a.rank * 2);
    uint32_t bo[NL];
    int bn[NL];  // column of the chunk this thread loads
#pragma unroll
    for (int l = 0; l < NL; ++l) {
      const int at = l * 256 + threadIdx.x, s = at ^ (((at >> 3) * magic >> 16) & spread), n = s * magic >> 16;
      const bool ok = at < 128 * R8 && 8 * (s - n * R8) < rank;
      bo[l] = (uint32_t)s * 16;
      bn[l] = ok ? n : 1 << 24;
    }
    u32x4 keep[KC];  // B past the rank is not used, whatever it holds
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      const int n = rank - 32 * k - 8 * h;
#pragma unroll
      for (int q = 0; q < 4; ++q) keep[k][q] = n <= 2 * q ? 0u : n == 2 * q + 1 ? 0xFFFFu : 0xFFFFFFFFu;
    }
    const uint64_t mask = __ballot(ids == cur);
    int list = 0;
    if constexpr (FEW) {  // the adapter's rows in a row
      const int at = __popcll(mask & ((1ull << lane) - 1));
      list = __builtin_amdgcn_ds_permute(4 * ((mask >> lane) & 1 ? at : 63 - (lane - at)), lane);
    }
    // the row of lane c, and those of the results (4 h + q)
    int row;
    if constexpr (FEW) {
      row = __shfl(list, (before + c) & 63, 64);
      if (before + c >= __popcll(mask)) row = -1;
    } else {
      row = 16 * wave + c;
      if (__shfl(ids, row, 64) != cur) row = -1;
    }
    uint32_t yo[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = __shfl(row, 4 * h + q, 64);
      yo[q] = r >= 0 ? ((uint32_t)r * a.N + 8 * c + (FEW ? 2 * wave : 0)) * 2 : kOutOfRange;
    }
    u32x4 bv[NL], yv[4];
    auto load = [&](int base) {
#pragma unroll
      for (int l = 0; l < NL; ++l)
        bv[l] = load16(br, base + bn[l] < end ? bo[l] : kOutOfRange, (uint32_t)base * a.rank * 2);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t o = base + 8 * c < end ? yo[q] : kOutOfRange;
        if constexpr (FEW) yv[q][0] = __builtin_amdgcn_raw_buffer_load_b32(yr, o, (uint32_t)base * 2, 0);
        else yv[q] = __builtin_amdgcn_raw_buffer_load_b128(yr, o, (uint32_t)base * 2, kNontemporal);  // (read once)
      }
    };
    load(base0);
    u32x4 hi[KC], lo[KC];
    float down = 1.f;
    if constexpr (FEW) {
      down = split_v<DT, KC>(a, splits, row0 + row, row >= 0, slice, rank, h, hi, lo);
    } else {
      const int64_t at = (int64_t)(row0 + (row < 0 ? 0 : row)) * a.slices + slice;
      if (DT == F16 && row >= 0) down = a.down[at];
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        hi[k] = lo[k] = u32x4{0u, 0u, 0u, 0u};
        if (row >= 0 && 32 * k + 8 * h < rank) {
          const u32x4* from = (const u32x4*)a.v + at * (a.rank >> 2) + 4 * k + h;
          hi[k] = from[0];
          lo[k] = from[a.rank >> 3];
        }
      }
    }
    down *= scale;
    float back[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) back[q] = __shfl(down, 4 * h + q, 64);
    for (int base = base0; base < stop; base += 128, buf ^= 1) {
      u32x4 yc[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) yc[q] = yv[q];
#pragma unroll
      for (int l = 0; l < NL; ++l) stage[buf][l * 256 + threadIdx.x] = bv[l];
      if (base + 128 < stop) load(base + 128);
      __syncthreads();  // (the block before the last one has been read by all)
      f4 d[NT] = {};
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < KC; ++k) {
          const u32x4 bt = stage[buf][((8 * c + t + (FEW ? 2 * wave : 0)) * R8 + 4 * k + h) ^ (c & spread)] & keep[k];
          d[t] = mfma16<DT>(lo[k], bt, d[t]);
          d[t] = mfma16<DT>(hi[k], bt, d[t]);
        }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        u32x4 o = yc[q];
        if (rank > 0) {  // (no adapter: a copy)
#pragma unroll
          for (int w = 0; w < NT / 2; ++w)
            o[w] = pack2<DT>(__builtin_fmaf(d[2 * w][q], back[q], act_lo<DT>(yc[q][w])),
                             __builtin_fmaf(d[2 * w + 1][q], back[q], act_hi<DT>(yc[q][w])));
        }
        const uint32_t to = (base + 8 * c < end ? yo[q] : kOutOfRange) + (uint32_t)base * 2;
        if constexpr (FEW) __builtin_amdgcn_raw_buffer_store_b32(o[0], outr, to, 0, 0);
        else store16(outr, o, to);
      }
    }
  });
}

// Both products in one launch, for calls whose time is launches.  A workgroup takes up to
// four rows of one adapter and `blocks` pairs of 128 columns of one slice: its eight waves
// form the slice's v themselves (row by row, as lora_shrink_rows_kernel does; every
// workgroup of the slice reads A again, from the caches), add it up in LDS, and multiply B
// by it, four waves to a block of columns (as lora_expand_kernel's few rows do).
template <int DT>
__global__ __launch_bounds__(512) void lora_fused_kernel(const LoraArgs a, int blocks) {
  constexpr int KC = 1, NL = 2;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, h = lane >> 4;
  const int half = wave >> 2, part = wave & 3, t256 = threadIdx.x & 255;
  const int row0 = blockIdx.x * 64, C = a.slices * a.rank, R8 = a.rank >> 3, magic = (65535 + R8) / R8;
  const int spread = R8 & 1 ? 7 : 15;
  int slice = 0, first = 0, end = a.ends[0], chunk = blockIdx.y;
  for (;;) {
    const int n = (end - first + 256 * blocks - 1) / (256 * blocks);
    if (chunk < n) break;
    chunk -= n;
    first = end;
    end = a.ends[++slice];
  }
  const int base0 = first + chunk * blocks * 256, stop = base0 + blocks * 256 < end ? base0 + blocks * 256 : end;
  const int ids = tile_adapters<64>(a, row0, lane);
  const int left = a.seqs.rows - row0, tile_rows = __builtin_amdgcn_readfirstlane(left < 64 ? left : 64);
  const rsrc_t xr = make_rsrc(a.x + (int64_t)row0 * a.K, (uint32_t)tile_rows * a.K * 2);
  const rsrc_t yr = make_rsrc(a.y + (int64_t)row0 * a.N, (uint32_t)tile_rows * a.N * 2);
  const rsrc_t outr = make_rsrc(a.out + (int64_t)row0 * a.N, (uint32_t)tile_rows * a.N * 2);
  const int units = a.K / 128;
  const int k0 = units * wave / 8 * 128, k1 = units * (wave + 1) / 8 * 128;
  __shared__ u32x4 stage[2][2][512 * KC];
  __shared__ f4 red[8][4][32 * KC / 4];  // [wave][row of x][row of A]
  int buf = 0;

  each_adapter<4>(ids, a.y == a.out ? 0 : -1, blockIdx.z, gridDim.z, [&](int cur, int before) {
    const int rank = cur < 0 ? 0 : adapter_rank(a, cur);
    const float scale = cur < 0 ? 0.f : a.scales[cur];
    const rsrc_t ar = make_rsrc(a.a + (int64_t)(cur < 0 ? 0 : cur) * C * a.K, (uint32_t)C * a.K * 2);
    const rsrc_t br = make_rsrc(a.b + (int64_t)(cur < 0 ? 0 : cur) * a.N * a.rank, (uint32_t)a.N * a.rank * 2);
    uint64_t mask = __ballot(ids == cur);
    for (int i = 0; i < before; ++i) mask &= mask - 1;
    int row[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      row[t] = mask ? __builtin_ctzll(mask) : -1;
      mask &= mask - 1;
    }
    // B and y of the first columns, needed last
    uint32_t bo[NL], yo[4];
    int bn[NL];  // column of the chunk this thread loads
#pragma unroll
    for (int l = 0; l < NL; ++l) {
      const int at = l * 256 + t256, s = at ^ (((at >> 3) * magic >> 16) & spread), n = s * magic >> 16;
      const bool ok = at < 128 * R8 && 8 * (s - n * R8) < rank;
      bo[l] = (uint32_t)s * 16;
      bn[l] = ok ? n : 1 << 24;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)  // (the results' rows 4 h + q are rows of x for h = 0)
      yo[q] = h == 0 && row[q] >= 0 ? ((uint32_t)row[q] * a.N + 8 * c + 2 * part) * 2 : kOutOfRange;
    u32x4 bv[NL];
    uint32_t yv[4];
    auto load = [&](int base) {
#pragma unroll
      for (int l = 0; l < NL; ++l)
        bv[l] = load16(br, base + bn[l] < end ? bo[l] : kOutOfRange, (uint32_t)base * a.rank * 2);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        yv[q] = __builtin_amdgcn_raw_buffer_load_b32(yr, base + 8 * c < end ? yo[q] : kOutOfRange, (uint32_t)base * 2, 0);
    };
    load(base0 + 128 * half);
    // v of this slice, 16 rows of A at a time
    auto product = [&](auto tg) {
      constexpr int TG = decltype(tg)::value, D = TG == 1 ? 4 : 2;
      uint32_t xo[TG];
#pragma unroll
      for (int t = 0; t < TG; ++t) xo[t] = row[t] >= 0 ? ((uint32_t)row[t] * a.K + 8 * c) * 2 : kOutOfRange;
      for (int b = 0; 16 * b < rank; ++b) {
        uint32_t ao[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * b + 4 * r + h;
          ao[r] = j < rank ? ((uint32_t)(slice * a.rank + j) * a.K + 8 * c) * 2 : kOutOfRange;
        }
        f4 acc[4][TG] = {};
        u32x4 af[D][4], xf[D][TG];
        auto fetch = [&](int u, int k) {
          const uint32_t out = k < k1 ? 0u : kOutOfRange;
#pragma unroll
          for (int r = 0; r < 4; ++r) af[u][r] = load16(ar, ao[r] | out, k * 2);
#pragma unroll
          for (int t = 0; t < TG; ++t) xf[u][t] = load16(xr, xo[t] | out, k * 2);
        };
#pragma unroll
        for (int u = 0; u < D - 1; ++u) fetch(u, k0 + 128 * u);
        for (int k = k0; k < k1; k += 128 * D)  // (what lies past the range comes as zeros)
#pragma unroll
          for (int u = 0; u < D; ++u) {
            fetch((u + D - 1) % D, k + 128 * (u + D - 1));
#pragma unroll
            for (int q = 0; q < 4; q += 2)
#pragma unroll
              for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int t = 0; t < TG; ++t)
                  acc[r][t] = mfma4<DT>(af[u][r][q], af[u][r][q + 1], xf[u][t][q], xf[u][t][q + 1], acc[r][t]);
          }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int t = 0; t < TG; ++t) {
            const f4 v = acc[r][t];
            const float own = lane & 2 ? (lane & 1 ? v[3] : v[2]) : (lane & 1 ? v[1] : v[0]);
            float s = sum_row(own);
            if (16 * b + 4 * r + h >= rank) s = 0.f;  // (0 x is not 0 for every x)
            if (c == 0) ((float*)red[wave][t])[16 * b + 4 * r + h] = s;
          }
      }
    };
    if (row[1] >= 0) product(std::integral_constant<int, 4>{});
    else product(std::integral_constant<int, 1>{});
    __syncthreads();
    u32x4 hi[KC], lo[KC], keep[KC];
    f4 v[KC][2] = {};
    const bool own = c == 0 || (c < 4 && row[1] >= 0);  // (with one row the others' sums are not there)
#pragma unroll
    for (int k = 0; k < KC; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (own && 32 * k + 8 * h + 4 * i < rank)
#pragma unroll
          for (int w = 0; w < 8; ++w) v[k][i] += red[w][c & 3][8 * k + 2 * h + i];
    float up = 1.f, down = 1.f;
    if constexpr (DT == F16) {
      float m = 0.f;
#pragma unroll
      for (int k = 0; k < KC; ++k) m = fmaxf(m, largest(v[k][0], v[k][1]));
      m = fmaxf(m, __shfl_xor(m, 16, 64));
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      powers(m, up, down);
    }
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      two_parts<DT>(v[k][0], v[k][1], up, hi[k], lo[k]);
      const int n = rank - 32 * k - 8 * h;
#pragma unroll
      for (int q = 0; q < 4; ++q) keep[k][q] = n <= 2 * q ? 0u : n == 2 * q + 1 ? 0xFFFFu : 0xFFFFFFFFu;
    }
    down *= scale;
    float back[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) back[q] = __shfl(down, q, 64);
    for (int at = base0; at < stop; at += 256, buf ^= 1) {  // (both halves go round as often)
      const int base = at + 128 * half;
      uint32_t yc[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) yc[q] = yv[q];
#pragma unroll
      for (int l = 0; l < NL; ++l) stage[buf][half][l * 256 + t256] = bv[l];
      if (at + 256 < stop) load(base + 256);
      __syncthreads();  // (the block before the last one has been read by all, and red by all)
      f4 d[2] = {};
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int k = 0; k < KC; ++k) {
          const u32x4 bt = stage[buf][half][((8 * c + t + 2 * part) * R8 + 4 * k + h) ^ (c & spread)] & keep[k];
          d[t] = mfma16<DT>(lo[k], bt, d[t]);
          d[t] = mfma16<DT>(hi[k], bt, d[t]);
        }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t o = pack2<DT>(__builtin_fmaf(d[0][q], back[q], act_lo<DT>(yc[q])),
                               __builtin_fmaf(d[1][q], back[q], act_hi<DT>(yc[q])));
        if (rank == 0) o = yc[q];  // (no adapter: a copy)
        __builtin_amdgcn_raw_buffer_store_b32(o, outr, (base + 8 * c < end ? yo[q] : kOutOfRange) + (uint32_t)base * 2, 0, 0);
      }
    }
  });
}

template <int DT, bool FEW, int KC>
void expand(const LoraArgs& a, const LoraPlan& p, int tiles, hipStream_t s) {
  int chunks = 0;
  for (int i = 0; i < a.slices; ++i)
    chunks += (a.ends[i] - (i ? a.ends[i - 1] : 0) + 128 * p.blocks - 1) / (128 * p.blocks);
  // (a tile's workgroups lie next to each other, so that whole rows of y are read and
  // written at a time: 70.6 us for the prompts, 75 with a column's next to each other)
  hipLaunchKernelGGL((lora_expand_kernel<DT, FEW, KC>), dim3((uint32_t)tiles * chunks, 1, p.groups), dim3(256), 0, s, a,
                     p.splits, p.blocks, (uint32_t)chunks);
}

template <int DT>
wq_status launch(const LoraArgs& a, hipStream_t s) {
  const int columns = a.slices * a.rank;
  if (lora_fused(a.seqs.rows, a.K, a.rank)) {
    const int groups = few_items(a.seqs.rows, a.seqs.batch);
    int blocks = (a.N + 255) / 256 * groups / 128;  // (128 workgroups: 16 rows of 16 adapters 11.8 us, 256 18.7)
    blocks = blocks < 1 ? 1 : blocks > 16 ? 16 : blocks;
    int chunks = 0;
    for (int i = 0; i < a.slices; ++i) chunks += (a.ends[i] - (i ? a.ends[i - 1] : 0) + 256 * blocks - 1) / (256 * blocks);
    const dim3 grid((a.seqs.rows + 63) / 64, chunks, groups), block(512);
    hipLaunchKernelGGL((lora_fused_kernel<DT>), grid, block, 0, s, a, blocks);
    return launch_status();
  }
  const LoraPlan p = lora_plan(a.seqs.rows, a.seqs.batch, a.K, columns, a.N, a.num + (a.y != a.out));
  const int tiles = (a.seqs.rows + 63) / 64, kc = (a.rank + 31) / 32;
  const int width = p.few ? 16 : 64;
  const dim3 grid(tiles, (columns + width - 1) / width * p.splits, p.first), block(256);
  if (p.few) hipLaunchKernelGGL((lora_shrink_rows_kernel<DT>), grid, block, 0, s, a, p.splits);
  else hipLaunchKernelGGL((lora_shrink_kernel<DT>), grid, block, 0, s, a, p.splits);
  if (!p.few) hipLaunchKernelGGL((lora_split_kernel<DT>), dim3((a.seqs.rows + 15) / 16, a.slices), block, 0, s, a, p.splits);
  if (p.few) {
    if (kc == 1) expand<DT, true, 1>(a, p, tiles, s);
    else if (kc == 2) expand<DT, true, 2>(a, p, tiles, s);
    else expand<DT, true, 4>(a, p, tiles, s);
  } else {
    if (kc == 1) expand<DT, false, 1>(a, p, tiles, s);
    else if (kc == 2) expand<DT, false, 2>(a, p, tiles, s);
    else expand<DT, false, 4>(a, p, tiles, s);
  }
  return launch_status();
}

}  // namespace

// Parts of v; for many rows then its two 16-bit parts and the powers of two.
static size_t part_bytes(const LoraPlan& p, int rows, int columns) { return (size_t)p.splits * rows * columns * 4; }
size_t lora_workspace_bytes(int rows, int batch, int K, int rank, int slices) {
  if (lora_fused(rows, K, rank)) return 0;
  const LoraPlan p = lora_plan(rows, batch, K, rank * slices);
  return part_bytes(p, rows, rank * slices) + (p.few ? 0 : (size_t)rows * slices * (4 * rank + 4));
}

wq_status launch_lora(const LoraArgs& args, int dt, hipStream_t s) {
  LoraArgs a = args;
  const int rows = a.seqs.rows, columns = a.slices * a.rank;
  a.v = (uint16_t*)a.part + part_bytes(lora_plan(rows, a.seqs.batch, a.K, columns), rows, columns) / 2;
  a.down = (float*)(a.v + (size_t)rows * columns * 2);
  return dt == F16 ? launch<F16>(a, s) : launch<BF16>(a, s);
}

}  // namespace wq
