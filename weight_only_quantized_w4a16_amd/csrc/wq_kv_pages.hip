// wq_kv_pages.hip -- sequences of the paged cache grow and shrink on the GPU.
//
// A sequence of n tokens holds ceil(n / P) pages.  Three sums over the sequences
// -- pages that go back, pages that are taken, new rows -- number every page of a
// call in the order (sequence, entry); the f-th page taken is the f-th given
// back, what is left over on either side comes from or goes to the stack's place
// top - 1 - f, top counting the pages given back.  One thread then moves the f-th
// page of both kinds (it alone reads that table entry, or that place of the
// stack, and it alone writes the other), so nothing waits on anything but the
// sums, and a sequence that grows and shrinks again leaves the stack as it was.
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

// One workgroup does all of it.
__global__ __launch_bounds__(kThreads) void resize_kernel(const PagesArgs a) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, B = a.batch;
  int32_t *back_off = a.offsets, *take_off = back_off + (B + 1), *row_off = take_off + (B + 1);
  __shared__ Sums part[kThreads / 64];
  __shared__ int bad_any;
  if (t == 0) bad_any = 0;
  const int per = (B + kThreads - 1) / kThreads, b0 = t * per < B ? t * per : B, b1 = b0 + per < B ? b0 + per : B;
  Sums own = {0, 0, 0};
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const Lens l = lens_of(a, b);
    bad |= l.bad;
    const int d = pages_of(a, l.want) - pages_of(a, l.old);
    own = own + Sums{d < 0 ? -d : 0, d > 0 ? d : 0, l.want > l.old ? l.want - l.old : 0};
  }
  Sums run = own;
  for (int d = 1; d < 64; d <<= 1) {
    const Sums p = up(run, d);
    if (lane >= d) run = run + p;
  }
  if (lane == 63) part[wave] = run;
  __syncthreads();
  if (bad) bad_any = 1;
  Sums before = {0, 0, 0}, total = {0, 0, 0};
  for (int w = 0; w < kThreads / 64; ++w) {
    if (w < wave) before = before + part[w];
    total = total + part[w];
  }
  Sums at = before + run;
  at = {at.back - own.back, at.taken - own.taken, at.rows - own.rows};
  int count = a.counts[0];
  count = count < 0 ? 0 : count > a.num_pages ? a.num_pages : count;
  __syncthreads();
  const int64_t top = count + total.back;
  int status = 0;
  if (bad_any || top > a.num_pages || total.rows > (1 << 24)) status = -1;
  else if (total.taken > top) status = (int)(total.taken - top);
  __syncthreads();  // every thread has read counts[0] and the lengths' verdict
  if (t == 0) a.counts[1] = status;
  if (status != 0) {
    if (a.cu_q)
      for (int b = t; b <= B; b += kThreads) a.cu_q[b] = 0;
    for (int r = t; r < a.rows; r += kThreads) {
      if (a.positions) a.positions[r] = -1;
      if (a.slots) a.slots[r] = -1;
    }
    return;
  }
  for (int b = b0; b < b1; ++b) {
    back_off[b] = (int)at.back;
    take_off[b] = (int)at.taken;
    row_off[b] = (int)at.rows;
    if (a.cu_q) a.cu_q[b] = (int)at.rows;
    const Lens l = lens_of(a, b);
    const int d = pages_of(a, l.want) - pages_of(a, l.old);
    at = at + Sums{d < 0 ? -d : 0, d > 0 ? d : 0, l.want > l.old ? l.want - l.old : 0};
  }
  if (t == 0) {
    back_off[B] = (int)total.back;
    take_off[B] = (int)total.taken;
    row_off[B] = (int)total.rows;
    if (a.cu_q) a.cu_q[B] = (int)total.rows;
    a.counts[0] = (int)(top - total.taken);
  }
  __syncthreads();
  const int nback = (int)total.back, ntake = (int)total.taken;
  for (int f = t; f < (nback > ntake ? nback : ntake); f += kThreads) {
    int page;
    if (f < nback) {
      const int b = owner(back_off, B, f);
      const Lens l = lens_of(a, b);
      int32_t* from = a.table + (int64_t)b * a.max_pages + pages_of(a, l.want) + (f - back_off[b]);
      page = *from;
      *from = -1;
    } else {
      page = a.free_pages[top - 1 - f];
    }
    if (f < ntake) {
      const int b = owner(take_off, B, f);
      const Lens l = lens_of(a, b);
      a.table[(int64_t)b * a.max_pages + pages_of(a, l.old) + (f - take_off[b])] = page;
    } else {
      a.free_pages[top - 1 - f] = page;
    }
  }
  __syncthreads();
  const int new_rows = (int)total.rows;
  for (int r = t; r < a.rows; r += kThreads) {
    int pos = -1;
    int64_t slot = -1;
    if (r < new_rows) {
      const int b = owner(row_off, B, r);
      pos = lens_of(a, b).old + (r - row_off[b]);
      const int page = a.table[(int64_t)b * a.max_pages + (pos >> a.page_shift)];
      slot = ((int64_t)page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
    }
    if (a.positions) a.positions[r] = pos;
    if (a.slots) a.slots[r] = slot;
  }
  __syncthreads();
  for (int b = t; b < B; b += kThreads) a.lens[b] = a.want[b];
}

}  // namespace

size_t pages_workspace_bytes(int batch, int, int, int) { return (size_t)(batch + 1) * 12; }

wq_status launch_resize(const PagesArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(resize_kernel, dim3(1), dim3(kThreads), 0, s, a);
  return launch_status();
}

}  // namespace wq
