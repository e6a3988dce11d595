// wq_kv_pages.hip -- sequences of the paged cache grow and shrink on the GPU.
//
// A sequence of n tokens holds ceil(n / P) pages.  Three sums over the sequences
// -- pages that go back, pages that are taken, new rows -- number every page and
// row of a call in the order (sequence, entry).  The f-th page taken is the f-th
// given back; what is left over on either side comes from or goes to the stack's
// place top - 1 - f, top counting the pages given back.  One thread moves the
// f-th page of both kinds (it alone reads that table entry, or that place of the
// stack, and it alone writes the other), so nothing waits on anything but the
// sums, and a sequence that grows and shrinks again leaves the stack as it was.
//
// Behind the sums everything follows from them and the wanted lengths, so the
// lengths are written at once: a sequence's taken entries are its last ones, the
// entries given back those behind its last.
//
// A step of few sequences and rows is one workgroup, its sums in LDS: the time is
// a launch and the chain lengths -> sums -> pages -> rows.  Prompts take two
// launches, one thread to a page and to four rows; every workgroup of the first
// forms the sums for itself.  Batches whose sums LDS does not hold take three, the
// sums in one of their own.
#include "wq_layer.hpp"

namespace wq {
namespace {

constexpr int kThreads = 1024;

struct Sums {
  int64_t back, taken, rows;
  __device__ Sums operator+(const Sums& o) const { return {back + o.back, taken + o.taken, rows + o.rows}; }
};
__device__ inline Sums up(const Sums& v, int d) {
  return {__shfl_up(v.back, d, 64), __shfl_up(v.taken, d, 64), __shfl_up(v.rows, d, 64)};
}

struct Lens {
  int old, want;  // tokens
  bool bad;       // the wanted length has no place
};
__device__ inline Lens lens_of(const PagesArgs& a, int b) {
  const int cap = a.max_pages << a.page_shift;
  Lens l;
  l.old = a.lens[b];
  l.old = l.old < 0 ? 0 : l.old > cap ? cap : l.old;
  l.want = a.want[b];
  l.bad = l.want < 0 || l.want > cap;
  return l;
}
__device__ inline int pages_of(const PagesArgs& a, int n) { return (n + (1 << a.page_shift) - 1) >> a.page_shift; }

// last i with off[i] <= f (off ascending, off[0] = 0, f below off[n])
__device__ inline int owner(const int32_t* off, int n, int f) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= f) lo = mid; else hi = mid;
  }
  return lo;
}

// The sums before this thread's sequences and in all, over a workgroup of kThreads.
__device__ inline void sum_before(Sums own, Sums& before, Sums& total) {
  __shared__ Sums part[kThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Sums run = own;
  if (__any((own.back | own.taken | own.rows) != 0))
    for (int d = 1; d < 64; d <<= 1) {
      const Sums p = up(run, d);
      if (lane >= d) run = run + p;
    }
  if (lane == 63) part[wave] = run;
  __syncthreads();
  before = {run.back - own.back, run.taken - own.taken, run.rows - own.rows};
  total = {0, 0, 0};
  for (int w = 0; w < kThreads / 64; ++w) {
    if (w == wave) before = before + total;
    total = total + part[w];
  }
}
__device__ inline Sums change(const PagesArgs& a, const Lens& l) {
  const int d = pages_of(a, l.want) - pages_of(a, l.old);
  return {d < 0 ? -d : 0, d > 0 ? d : 0, l.want > l.old ? l.want - l.old : 0};
}

// Offsets of the sequences' pages given back and taken and of their new rows.
struct Offsets {
  int32_t *back, *taken, *rows;  // [batch + 1] each
};
__device__ inline Offsets offsets_in(int32_t* p, int batch) { return {p, p + (batch + 1), p + 2 * (batch + 1)}; }

// What the sums say; all zeros and the stack as it is where nothing may change.
struct Verdict {
  Sums total;
  int64_t top;
  int status;
};
__device__ inline void set_counts(const PagesArgs& a, int status, int free) {
  if (status == 0) a.counts[0] = free;
  a.counts[1] = status;
}

// The sums and the verdict, for a workgroup of kThreads; with WRITE also lengths, counts
// and the offsets the caller gets.  (Every thread has read what it needs of lengths and
// counts before any writes.)
template <bool WRITE>
__device__ inline Verdict settle(const PagesArgs& a, const Offsets& o) {
  const int t = threadIdx.x, B = a.batch;
  const int per = (B + kThreads - 1) / kThreads, b0 = t * per < B ? t * per : B, b1 = b0 + per < B ? b0 + per : B;
  Sums own = {0, 0, 0};
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const Lens l = lens_of(a, b);
    bad |= l.bad;
    own = own + change(a, l);
  }
  int count = a.counts[0];
  count = count < 0 ? 0 : count > a.num_pages ? a.num_pages : count;
  Sums at, total;
  sum_before(own, at, total);
  bad = __syncthreads_or(bad);
  Verdict v = {total, count + total.back, 0};
  // (the offsets are 32-bit; within them the pages taken are no more than the rows)
  if (bad || v.top > a.num_pages || total.rows > 0x7FFFFFFF) v.status = -1;
  else if (total.taken > v.top) v.status = (int)(total.taken - v.top);
  if (v.status) {
    v.total = at = {0, 0, 0};
    v.top = count;
  }
  for (int b = b0; b < b1; ++b) {
    o.back[b] = (int)at.back;
    o.taken[b] = (int)at.taken;
    o.rows[b] = (int)at.rows;
    if (WRITE && a.cu_q) a.cu_q[b] = (int)at.rows;
    if (v.status) continue;
    const Lens l = lens_of(a, b);
    at = at + change(a, l);
    if (WRITE) a.lens[b] = l.want;
  }
  if (t == 0) {
    o.back[B] = (int)v.total.back;
    o.taken[B] = (int)v.total.taken;
    o.rows[B] = (int)v.total.rows;
    if (WRITE) {
      if (a.cu_q) a.cu_q[B] = (int)v.total.rows;
      set_counts(a, v.status, (int)(v.top - v.total.taken));
    }
  }
  return v;
}

// The f-th page given back and the f-th taken.
__device__ inline void move_page(const PagesArgs& a, const Offsets& o, int nback, int ntake, int64_t top, int f) {
  int page;
  if (f < nback) {
    const int b = owner(o.back, a.batch, f);
    int32_t* from = a.table + (int64_t)b * a.max_pages + pages_of(a, a.want[b]) + (f - o.back[b]);
    page = *from;
    *from = -1;
  } else {
    page = a.free_pages[top - 1 - f];
  }
  if (f < ntake) {
    const int b = owner(o.taken, a.batch, f);
    a.table[(int64_t)b * a.max_pages + pages_of(a, a.want[b]) - (o.taken[b + 1] - f)] = page;
  } else {
    a.free_pages[top - 1 - f] = page;
  }
}

// Position and slot of new row r of sequence b (-1: none).
__device__ inline void map_row(const PagesArgs& a, const Offsets& o, int b, int r, int& pos, int64_t& slot) {
  pos = -1;
  slot = -1;
  if (b < 0) return;
  pos = a.want[b] - (o.rows[b + 1] - r);
  const int page = a.table[(int64_t)b * a.max_pages + (pos >> a.page_shift)];
  slot = ((int64_t)page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

// One workgroup does all of it (batch up to kThreads).
__global__ __launch_bounds__(kThreads) void resize_kernel(const PagesArgs a) {
  __shared__ int32_t sums[3 * (kThreads + 1)];
  const Offsets o = offsets_in(sums, a.batch);
  const Verdict v = settle<true>(a, o);
  __syncthreads();
  const int nback = (int)v.total.back, ntake = (int)v.total.taken, new_rows = (int)v.total.rows;
  for (int f = threadIdx.x; f < (nback > ntake ? nback : ntake); f += kThreads) move_page(a, o, nback, ntake, v.top, f);
  __syncthreads();
  for (int r = threadIdx.x; r < a.rows; r += kThreads) {
    int pos;
    int64_t slot;
    map_row(a, o, r < new_rows ? owner(o.rows, a.batch, r) : -1, r, pos, slot);
    if (a.positions) a.positions[r] = pos;
    if (a.slots) a.slots[r] = slot;
  }
}

// Two launches (batch up to kThreads): pages, then rows.  The first changes nothing that
// its sums come from: lengths and counts are the second's.
__global__ __launch_bounds__(kThreads) void resize_pages_kernel(const PagesArgs a) {
  __shared__ int32_t sums[3 * (kThreads + 1)];
  const Offsets o = offsets_in(sums, a.batch);
  const Verdict v = settle<false>(a, o);
  __syncthreads();
  const int nback = (int)v.total.back, ntake = (int)v.total.taken;
  for (int f = blockIdx.x * kThreads + threadIdx.x; f < (nback > ntake ? nback : ntake); f += gridDim.x * kThreads)
    move_page(a, o, nback, ntake, v.top, f);
  if (blockIdx.x) return;
  if (threadIdx.x <= a.batch) a.offsets[threadIdx.x] = o.rows[threadIdx.x];
  if (threadIdx.x == 0) {
    a.offsets[a.batch] = o.rows[a.batch];
    a.offsets[a.batch + 1] = v.status;
    a.offsets[a.batch + 2] = (int)(v.top - v.total.taken);
  }
}

// Position and slot of four rows from r0 on.
__device__ inline void map_rows(const PagesArgs& a, const Offsets& o, int r0) {
  if (r0 >= a.rows) return;
  const int new_rows = o.rows[a.batch];
  int b = r0 < new_rows ? owner(o.rows, a.batch, r0) : -1;
  int pos[4];
  int64_t slot[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + i;
    if (r >= new_rows) b = -1;
    else
      while (o.rows[b + 1] <= r) ++b;  // (the last offset lies behind every new row)
    map_row(a, o, b, r, pos[i], slot[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (r0 + i < a.rows) {
      if (a.positions) a.positions[r0 + i] = pos[i];
      if (a.slots) a.slots[r0 + i] = slot[i];
    }
}

__global__ __launch_bounds__(256) void resize_rows_kernel(const PagesArgs a) {
  __shared__ int32_t rows[kThreads + 1];
  const int B = a.batch, status = a.offsets[B + 1];
  for (int i = threadIdx.x; i <= B; i += 256) {
    rows[i] = a.offsets[i];
    if (blockIdx.x == 0) {
      if (a.cu_q) a.cu_q[i] = rows[i];
      if (i < B && status == 0) a.lens[i] = a.want[i];
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) set_counts(a, status, a.offsets[B + 2]);
  __syncthreads();
  map_rows(a, {nullptr, nullptr, rows}, (blockIdx.x * 256 + threadIdx.x) * 4);
}

// Three launches, for any batch.
__global__ __launch_bounds__(kThreads) void resize_sums_kernel(const PagesArgs a) {
  const Verdict v = settle<true>(a, offsets_in(a.offsets, a.batch));
  if (threadIdx.x == 0) a.offsets[3 * (a.batch + 1)] = (int)v.top;
}
__global__ __launch_bounds__(256) void resize_move_kernel(const PagesArgs a) {
  const Offsets o = offsets_in(a.offsets, a.batch);
  const int nback = o.back[a.batch], ntake = o.taken[a.batch], top = a.offsets[3 * (a.batch + 1)];
  for (int f = blockIdx.x * 256 + threadIdx.x; f < (nback > ntake ? nback : ntake); f += gridDim.x * 256)
    move_page(a, o, nback, ntake, top, f);
}
__global__ __launch_bounds__(256) void resize_map_kernel(const PagesArgs a) {
  map_rows(a, offsets_in(a.offsets, a.batch), (blockIdx.x * 256 + threadIdx.x) * 4);
}

// One workgroup up to this many sequences and new rows.  Two changes of 64 sequences, us in
// one : two launches: 357 rows 12.3 : 14.6, 2850 14.0 : 15.1, 4795 15.4
// : 15.4, 11003 19.9 : 15.5; of 300 sequences and 375000 rows each 1630 : 26 (33 in three).
// The pages are not in the rule.  One workgroup moves 1024 of them at a time, so a call of
// few rows that begins or ends many long sequences at once takes longer in it, us a call
// in one : two: 64 sequences of 1000 tokens 8.4 : 9.1, 16 of 5000 8.5 : 9.0, 300 of 5000 87
// : 11, 1024 of 4096 262 : 16.  (1500 of 2000 tokens, in three: 12.)
constexpr int kOneBatch = kThreads, kOneRows = 4096;

}  // namespace

size_t pages_workspace_bytes(int batch, int, int, int rows) {
  return batch <= kOneBatch && rows <= kOneRows ? 0 : (size_t)(batch + 1) * 12 + 4;
}

wq_status launch_resize(const PagesArgs& a, hipStream_t s) {
  if (a.batch <= kOneBatch && a.rows <= kOneRows) {
    hipLaunchKernelGGL(resize_kernel, dim3(1), dim3(kThreads), 0, s, a);
    return launch_status();
  }
  const int64_t most = (int64_t)a.batch * a.max_pages < a.num_pages ? (int64_t)a.batch * a.max_pages : a.num_pages;
  const int map = (a.rows + 1023) / 1024;
  if (a.batch <= kOneBatch) {
    const int64_t wgs = (most + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(resize_pages_kernel, dim3((int)(wgs < 1 ? 1 : wgs < 64 ? wgs : 64)), dim3(kThreads), 0, s, a);
    hipLaunchKernelGGL(resize_rows_kernel, dim3(a.positions || a.slots ? map : 1), dim3(256), 0, s, a);
    return launch_status();
  }
  hipLaunchKernelGGL(resize_sums_kernel, dim3(1), dim3(kThreads), 0, s, a);
  const int64_t wgs = (most + 255) / 256;
  if (wgs) hipLaunchKernelGGL(resize_move_kernel, dim3((int)(wgs < 1024 ? wgs : 1024)), dim3(256), 0, s, a);
  if (a.rows && (a.positions || a.slots)) hipLaunchKernelGGL(resize_map_kernel, dim3(map), dim3(256), 0, s, a);
  return launch_status();
}

}  // namespace wq
