// The paged memory's book-keeping and its data movement: pages reserved for
// new rows (copy on write where a page is shared), rows written, pages
// copied, slots forked, the oldest rows freed, the live pages compacted.
//
// A slot's live rows are rows start .. start + rows - 1 of the concatenation
// of its pages table[slot][0], table[slot][1], ... (page_rows rows each);
// refs[p] counts the table entries that name page p, 0: free.  Every call
// works on device state alone (no host copy of a length), so a serving step
// can be captured into a graph and replayed, and every result is a function
// of the state before the call: free pages are given out by ascending id in
// the order of the call's entries, whatever order the threads run in.
//
// Bad entries (a slot, page or length out of range, the same slot twice) are
// refused, touch nothing and raise the pages bit of the status word.  A page id
// is looked at where a call reads it, ahead of the entry's first change.
#include <algorithm>
#include <climits>
#include <cstdint>

#include "pages.h"
#include "pdl.cuh"
#include "txl_internal.h"

namespace txl {
namespace {

constexpr int kBlock = 1024;    // threads of the single-CTA kernels
constexpr int kPerThread = 16;  // refs a thread looks at per tile
constexpr int kList = 4096;     // pages placed at a time

__device__ __forceinline__ void report_pages(unsigned int* status) { atomicOr(status, kStatusPagesBit); }

__device__ __forceinline__ int ceil_div(long long a, int b) { return static_cast<int>((a + b - 1) / b); }

// Inclusive sums of x and of y over the CTA, saturating at `cap` (min(a + b,
// cap) is associative for non-negative terms; cap < 2^30, so no sum overflows),
// and the CTA's sums.  Every warp adds up the warps' sums itself: one barrier,
// and two buffers used in turn, so that a sum is read before it is replaced.
struct Scan {
  int2 at, all;
};
__device__ __forceinline__ Scan block_scan(int2 v, int cap, int2 (*sums)[32], int& turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](int2 a) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, a.x, d), y = __shfl_up_sync(0xffffffffu, a.y, d);
      if (lane >= d) a = make_int2(min(a.x + x, cap), min(a.y + y, cap));
    }
    return a;
  };
  v = scan(v);
  turn ^= 1;
  if (lane == 31) sums[turn][warp] = v;
  __syncthreads();
  const int2 w = scan(sums[turn][lane]);
  const int before = warp > 0 ? warp - 1 : 0;
  const int2 b = make_int2(__shfl_sync(0xffffffffu, w.x, before), __shfl_sync(0xffffffffu, w.y, before));
  Scan r;
  r.at = warp > 0 ? make_int2(min(v.x + b.x, cap), min(v.y + b.y, cap)) : v;
  r.all = make_int2(__shfl_sync(0xffffffffu, w.x, 31), __shfl_sync(0xffffffffu, w.y, 31));
  return r;
}
static_assert(kBlock == 1024, "block_scan sums 32 warps");

// A slot's state as the calls read it; ok: the slot and its lengths are in
// range.
struct Slot {
  int s, start, rows;
  bool ok;
};

__device__ __forceinline__ Slot read_slot(const PageBook& b, int s) {
  Slot r{s, 0, 0, s >= 0 && s < b.n_slots};
  if (r.ok) {
    r.start = b.start[s];
    r.rows = b.rows[s];
    r.ok = r.start >= 0 && r.start < b.page_rows && r.rows >= 0 &&
           static_cast<long long>(r.start) + r.rows <= static_cast<long long>(b.max_pages) * b.page_rows;
  }
  return r;
}

__device__ __forceinline__ int* table_row(const PageBook& b, int s) {
  return b.table + static_cast<size_t>(s) * b.max_pages;
}

// The 16 refs of this thread in the tile at `base`, as a mask of the pages
// in use (past the end: in use).
__device__ __forceinline__ uint32_t used_mask(const PageBook& b, int base) {
  const int p0 = base + threadIdx.x * kPerThread;
  uint32_t m = 0;
  if (p0 + kPerThread <= b.n_pages && (reinterpret_cast<uintptr_t>(b.refs) & 15) == 0) {
#pragma unroll
    for (int q = 0; q < kPerThread / 4; ++q) {
      const int4 v = *reinterpret_cast<const int4*>(b.refs + p0 + 4 * q);
      m |= ((v.x != 0) | (v.y != 0) << 1 | (v.z != 0) << 2 | (v.w != 0) << 3) << (4 * q);
    }
  } else {
#pragma unroll
    for (int q = 0; q < kPerThread; ++q) m |= (p0 + q >= b.n_pages || b.refs[p0 + q] != 0 ? 1u : 0u) << q;
  }
  return m;
}

// ---------------------------------------------------------------------------
// reserve
// ---------------------------------------------------------------------------
// One CTA: the entries' needs are summed in order, then the free pages are
// found by scanning refs in ascending order, 16384 pages a step, only as far
// as the needs go.  A free page's rank names its entry (binary search in the
// sums) and its place in the entry's table row.
//
// Nothing here is large: the kernel is the chain of its loads (an entry's slot,
// its lengths, its last page, that page's count, each a trip to L2) and its
// barriers.  With SMALL, up to 1024 entries, a thread keeps its entry's answer
// in registers and leaves what the pages' owners need of it in shared memory,
// and the first 16384 pages are read once, beside the entries' first loads, and
// counted in the same scan as the needs.  (With reserve, append and free, 22
// segments of 512 rows: 18 us, of which 7 are append's 46 MB; half as long again
// with the entries read anew in each phase and 64-bit divisions in append.  64
// single tokens: 9 us, about 3 a launch.)
struct Ask {  // what an entry asks for
  int slot, rows, count, have, need, last;  // need: pages (0 where it asks for none or is refused)
  bool ok, shared, idle;              // shared: its last page, which is copied; idle: a valid entry without rows
};

template <bool SMALL>
__global__ void __launch_bounds__(kBlock) reserve_kernel(PageBook b, const int* __restrict__ slots,
                                                         const int* __restrict__ cu, int n, int* granted,
                                                         int* copy_src, int* copy_dst, unsigned int* status) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  extern __shared__ int smem[];
  int* first = smem;             // [n_slots] the entry that names the slot first
  int* upto = smem + b.n_slots;  // [n] pages needed by entries 0 .. i
  int* slot_of = upto + n;       // SMALL: [n] the entry's slot
  int* place = slot_of + n;      // SMALL: [n] 2 * (its first new place in its table row) + (that place's page is copied)
  __shared__ int2 sums[2][32];
  __shared__ int s_lim;
  __shared__ int list[kList];  // pages of a window of ranks
  const int tid = threadIdx.x;
  const int cap = b.n_pages + 1;
  constexpr int kTile = kBlock * kPerThread;
  int turn = 0;

  const uint32_t used0 = used_mask(b, 0);
  for (int i = tid; i < n; i += kBlock)
    if (const int s = slots[i]; s >= 0 && s < b.n_slots) first[s] = INT_MAX;
  if (tid == 0) s_lim = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kBlock)
    if (const int s = slots[i]; s >= 0 && s < b.n_slots) atomicMin(&first[s], i);

  auto ask = [&](int i) {
    const Slot sl = read_slot(b, slots[i]);
    const int row0 = cu[i];
    Ask a{sl.s, sl.rows, cu[i + 1] - row0, 0, 0, -1, false, false, false};
    if (!sl.ok || row0 < 0) return a;  // (append has no such row, and would leave what is granted unwritten)
    a.idle = a.count == 0;
    const long long end = static_cast<long long>(sl.start) + sl.rows;
    a.have = ceil_div(end, b.page_rows);
    if (a.count <= 0) return a;
    const long long want = (end + a.count + b.page_rows - 1) / b.page_rows;
    a.ok = want <= b.max_pages;
    if (a.ok && end % b.page_rows != 0) {
      a.last = table_row(b, sl.s)[a.have - 1];
      a.ok = a.last >= 0 && a.last < b.n_pages;
      a.shared = a.ok && b.refs[a.last] > 1;
    }
    if (a.ok) a.need = static_cast<int>(want) - a.have + (a.shared ? 1 : 0);
    return a;
  };
  auto mine = [&](int i) {  // behind the barrier: of a slot named twice the first entry counts
    Ask a = ask(i);
    if (a.ok && first[a.slot] != i) a.ok = a.shared = false, a.need = 0;
    return a;
  };

  Ask own{};
  if (SMALL && tid < n) own = ask(tid);
  __syncthreads();
  if (SMALL && own.ok && first[own.slot] != tid) own.ok = own.shared = false, own.need = 0;

  // Sums of the needs, and of the first tile's free pages.
  const int free0 = kPerThread - __popc(used0);
  int carry = 0;
  Scan scan{};
  for (int base = 0; base < n || base == 0; base += kBlock) {
    const int i = base + tid;
    const int need = i < n ? min((SMALL ? own : mine(i)).need, cap) : 0;
    scan = block_scan(make_int2(need, free0), cap, sums, turn);
    if (i < n) upto[i] = min(carry + scan.at.x, cap);
    carry = min(carry + scan.all.x, cap);
  }
  const int total = carry;
  if (SMALL && tid < n) {
    slot_of[tid] = own.slot;
    place[tid] = 2 * (own.have - (own.shared ? 1 : 0)) + (own.shared ? 1 : 0);
  }
  __syncthreads();

  // Free pages there are, counted as far as `total`; lim: pages given out.
  int lim = total, found = scan.all.y;
  const int rank_first = scan.at.y - free0;
  for (int base = kTile; base < b.n_pages && found < total; base += kTile) {
    const Scan x = block_scan(make_int2(kPerThread - __popc(used_mask(b, base)), 0), cap, sums, turn);
    found = min(found + x.all.x, cap);
  }
  const int found_first = scan.all.y;
  if (found < total) {
    for (int i = tid; i < n; i += kBlock)
      if (upto[i] <= found) atomicMax(&s_lim, upto[i]);
    __syncthreads();
    lim = s_lim;
  }

  // The entries' answers, from the state before any change; the pages of
  // the copies follow below.
  for (int i = tid; i < n; i += kBlock) {
    const Ask a = SMALL ? own : mine(i);
    const bool given = a.ok && (a.need == 0 || upto[i] <= lim);
    if (SMALL) own.ok = given;  // from here on
    granted[i] = given ? a.count : 0;
    copy_src[i] = given && a.shared ? a.last : -1;
    copy_dst[i] = -1;
    if (!given && !a.idle) report_pages(status);
  }
  __syncthreads();

  // Free pages 0 .. lim-1 to their places.  A page's ref changes only after
  // its tile has been read.
  int rank0 = 0;
  for (int base = 0; base < b.n_pages && rank0 < lim; base += kTile) {
    const int tile_rank = rank0;
    uint32_t used = used0;
    int rank = rank_first;
    if (base == 0) {
      rank0 = found_first;
    } else {
      used = used_mask(b, base);
      const int free = kPerThread - __popc(used);
      const Scan x = block_scan(make_int2(free, 0), cap, sums, turn);
      rank = rank0 + x.at.x - free;
      rank0 += x.all.x;
    }
    // By rank in shared memory first: free pages stand together, so that one
    // thread has up to 16 of them to place.
    uint32_t m = ~used & 0xffffu;
    const int end = min(rank0, lim);
    for (int w0 = tile_rank; w0 < end; w0 += kList) {
      const int w1 = min(w0 + kList, end);
      for (; m != 0 && rank < w1; m &= m - 1, ++rank) list[rank - w0] = base + tid * kPerThread + __ffs(m) - 1;
      __syncthreads();
      for (int x = w0 + tid; x < w1; x += kBlock) {
        int lo = 0, hi = n - 1;  // the first entry with upto > x
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (upto[mid] > x)
            hi = mid;
          else
            lo = mid + 1;
        }
        const int j = x - (lo > 0 ? upto[lo - 1] : 0), page = list[x - w0];
        int s, at, copied;
        if (SMALL) {
          s = slot_of[lo];
          at = place[lo] >> 1;
          copied = place[lo] & 1;
        } else {
          s = slots[lo];
          copied = copy_src[lo] >= 0 ? 1 : 0;
          at = ceil_div(static_cast<long long>(b.start[s]) + b.rows[s], b.page_rows) - copied;
        }
        b.refs[page] = 1;
        table_row(b, s)[at + j] = page;
        if (j < copied) copy_dst[lo] = page;
      }
      __syncthreads();
    }
  }
  __syncthreads();
  if (SMALL) {
    if (tid < n && own.ok) {
      b.rows[own.slot] = own.rows + own.count;
      if (own.shared) atomicSub(&b.refs[own.last], 1);
    }
    return;
  }
  for (int i = tid; i < n; i += kBlock) {
    const int rows = granted[i], from = copy_src[i];
    if (rows > 0) b.rows[slots[i]] += rows;
    if (from >= 0) atomicSub(&b.refs[from], 1);
  }
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
// Division by a number that the host knows: q = (mulhi(x, m) + x) >> s, exact
// for x < 2^31 (m = floor(2^32 (2^s - d) / d) + 1, s = ceil(log2 d)).
struct Divisor {
  uint32_t d, m, s;
  explicit Divisor(uint32_t y) : d(y), s(0) {
    while (s < 31 && (1u << s) < y) ++s;
    m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - y)) / y + 1);
  }
  __device__ __forceinline__ uint32_t over(uint32_t x) const { return (__umulhi(x, m) + x) >> s; }
};

// CTA (x, i) writes rows of entry i: first the rows of the copied page that
// lie before the new ones, then the new rows, each as H pieces of D values,
// `tile` rows (about 1024 vectors) at a time.  What it waits for is the chain
// of its loads, so those that do not need one another go out together: an
// entry's numbers, then its slot's lengths, then a tile's pages beside its new
// rows.
template <typename V>
__global__ void __launch_bounds__(256) append_kernel(PageBook b, V* __restrict__ kp, V* __restrict__ vp, int H, int DV,
                                                     const int* __restrict__ slots, const int* __restrict__ cu,
                                                     const int* __restrict__ granted,
                                                     const int* __restrict__ copy_src,
                                                     const int* __restrict__ copy_dst, const V* __restrict__ kn,
                                                     const V* __restrict__ vn, int T, int tile, Divisor by_row,
                                                     Divisor by_head, int log_page, unsigned int* status) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int i = blockIdx.y;
  const int count = granted[i], t0 = cu[i], t1 = cu[i + 1], s = slots[i];
  int from = -1, to = -1;
  if (copy_src != nullptr) from = copy_src[i], to = copy_dst[i];
  const Slot sl = read_slot(b, s);
  if (count <= 0) return;
  if (!sl.ok || count > sl.rows || t0 < 0 || count != t1 - t0 || static_cast<long long>(t0) + count > T) {
    if (threadIdx.x == 0) report_pages(status);
    return;
  }
  const int P = b.page_rows;
  const int x0 = sl.start + sl.rows - count;  // first new row
  const bool copies = from >= 0 && to >= 0;
  if (copies && (from >= b.n_pages || to >= b.n_pages)) {
    if (threadIdx.x == 0) report_pages(status);
    return;
  }
  const int old = copies ? x0 & (P - 1) : 0;
  const int* row = table_row(b, sl.s);
  // Every page of the new rows ahead of the first write: each warp looks for
  // itself, at what all of them see.
  bool pages_ok = true;
  for (int j = (x0 >> log_page) + (threadIdx.x & 31); j <= (x0 + count - 1) >> log_page; j += 32)
    pages_ok &= static_cast<unsigned>(row[j]) < static_cast<unsigned>(b.n_pages);
  if (!__all_sync(0xffffffffu, pages_ok)) {
    if (threadIdx.x == 0) report_pages(status);
    return;
  }
  const uint32_t per = by_row.d;  // vectors of a row
  const size_t page = static_cast<size_t>(H) * P * DV;
  constexpr int U = 4;
  for (int y0 = static_cast<int>(blockIdx.x) * tile; y0 < old + count; y0 += static_cast<int>(gridDim.x) * tile) {
    const uint32_t total = static_cast<uint32_t>(min(tile, old + count - y0)) * per;
    for (uint32_t e0 = threadIdx.x; e0 < total; e0 += 256 * U) {
      V kx[U], vx[U];
      size_t dst[U];
      bool on[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t e = e0 + u * 256;
        on[u] = e < total;
        if (!on[u]) continue;
        const uint32_t line = by_row.over(e), rem = e - line * per;
        const uint32_t h = by_head.over(rem), c = rem - h * by_head.d;
        const int y = y0 + static_cast<int>(line);
        if (y < old) {
          const size_t at = (static_cast<size_t>(h) * P + y) * DV + c;
          dst[u] = to * page + at;
          kx[u] = kp[from * page + at];
          vx[u] = vp[from * page + at];
        } else {
          const int x = x0 + y - old;
          const int id = row[x >> log_page];
          const size_t src = static_cast<size_t>(t0 + y - old) * per + rem;
          kx[u] = __ldg(kn + src);
          vx[u] = __ldg(vn + src);
          dst[u] = id * page + (static_cast<size_t>(h) * P + (x & (P - 1))) * DV + c;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (on[u]) {
          kp[dst[u]] = kx[u];
          vp[dst[u]] = vx[u];
        }
    }
  }
}

// ---------------------------------------------------------------------------
// copy
// ---------------------------------------------------------------------------
// Whole pages src[i] -> dst[i] of both pools, in chunks of 256 x 4 vectors
// spread over the CTAs; each CTA looks 256 of its chunks ahead at a time, so
// that the entries without a copy (-1) cost one load per 256.
template <typename V>
__global__ void __launch_bounds__(256) copy_kernel(V* kp, V* vp, int n_pages, long long page_vecs,
                                                   const int* __restrict__ src, const int* __restrict__ dst, int n,
                                                   unsigned int* status) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  constexpr int U = 4;
  __shared__ int list[256];
  __shared__ int counts[8];
  const long long per = (page_vecs + 256 * U - 1) / (256 * U);  // chunks of a page of one pool
  const long long total = 2 * per * n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (long long k0 = 0; blockIdx.x + k0 * gridDim.x < total; k0 += 256) {
    const long long q = blockIdx.x + (k0 + threadIdx.x) * gridDim.x;
    bool on = false;
    if (q < total) {
      const int i = static_cast<int>(q / (2 * per));
      const int a = src[i], z = dst[i];
      on = a >= 0 && z >= 0;
      if (on && (a >= n_pages || z >= n_pages)) {
        report_pages(status);
        on = false;
      }
    }
    const uint32_t votes = __ballot_sync(0xffffffffu, on);
    if (lane == 0) counts[warp] = __popc(votes);
    __syncthreads();
    int at = 0, m = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      at += w < warp ? counts[w] : 0;
      m += counts[w];
    }
    if (on) list[at + __popc(votes & ((1u << lane) - 1))] = threadIdx.x;
    __syncthreads();
    for (int y = 0; y < m; ++y) {
      const long long c = blockIdx.x + (k0 + list[y]) * gridDim.x;
      const int i = static_cast<int>(c / (2 * per));
      const long long part = c % (2 * per);
      V* pool = part < per ? kp : vp;
      const V* from = pool + src[i] * static_cast<size_t>(page_vecs);
      V* to = pool + dst[i] * static_cast<size_t>(page_vecs);
      const long long e0 = (part < per ? part : part - per) * (256 * U) + threadIdx.x;
      V x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (e0 + u * 256 < page_vecs) x[u] = from[e0 + u * 256];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (e0 + u * 256 < page_vecs) to[e0 + u * 256] = x[u];
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// fork, free
// ---------------------------------------------------------------------------
// CTA i: dst[i] becomes a second owner of src[i]'s pages.  dst must be empty
// and named once, src not named as a dst: then no CTA writes what another
// reads, and the counts' atomic sums do not depend on their order.
__global__ void __launch_bounds__(128) fork_kernel(PageBook b, const int* __restrict__ src,
                                                   const int* __restrict__ dst, int n, int* ok_out,
                                                   unsigned int* status) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int i = blockIdx.x;
  const int d = dst[i];
  const Slot a = read_slot(b, src[i]);
  bool ok = a.ok && d >= 0 && d < b.n_slots && d != a.s;
  for (int j = threadIdx.x; ok && j < n; j += blockDim.x) ok = dst[j] != a.s && (j >= i || dst[j] != d);
  if (ok) ok = b.rows[d] == 0;
  ok = __syncthreads_and(ok);
  int pages = 0;
  if (ok) {
    pages = ceil_div(static_cast<long long>(a.start) + a.rows, b.page_rows);
    const int* row = table_row(b, a.s);
    for (int j = threadIdx.x; ok && j < pages; j += blockDim.x) ok = row[j] >= 0 && row[j] < b.n_pages;
  }
  ok = __syncthreads_and(ok);
  if (threadIdx.x == 0) {
    ok_out[i] = ok ? 1 : 0;
    if (!ok) report_pages(status);
  }
  if (!ok || a.rows == 0) return;
  const int* row = table_row(b, a.s);
  int* out = table_row(b, d);
  for (int j = threadIdx.x; j < pages; j += blockDim.x) {
    const int p = row[j];
    out[j] = p;
    atomicAdd(&b.refs[p], 1);
  }
  if (threadIdx.x == 0) {
    b.start[d] = a.start;
    b.rows[d] = a.rows;
  }
}

// CTA i: slot slots[i] keeps its newest keep[i] rows; pages that hold none of
// them leave the table row, which moves up and is filled with -1.
__global__ void __launch_bounds__(128) free_kernel(PageBook b, const int* __restrict__ slots,
                                                   const int* __restrict__ keep, int n, unsigned int* status) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int i = blockIdx.x;
  const int s = slots[i], want = keep == nullptr ? 0 : keep[i];
  // The entry that names the slot first changes it, which no other does; what a
  // later one reads here, at whatever time, it does not use.
  const Slot a = read_slot(b, s);
  bool first = true;
  for (int j = threadIdx.x; j < i; j += blockDim.x) first &= slots[j] != s;
  // (Every thread has read the state behind this barrier.)
  if (!__syncthreads_and(first) || !__syncthreads_and(a.ok)) {
    if (threadIdx.x == 0) report_pages(status);
    return;
  }
  const int kept = min(a.rows, max(want, 0));
  const int begin = a.start + (a.rows - kept);  // in range: start + rows <= max_pages * page_rows
  const int pages = ceil_div(static_cast<long long>(a.start) + a.rows, b.page_rows);
  const int dead = kept > 0 ? begin / b.page_rows : pages;
  int* row = table_row(b, a.s);
  if (dead > 0) {  // the row is read: every page of it ahead of the first change
    bool good = true;
    for (int j = threadIdx.x; j < pages; j += blockDim.x) good &= row[j] >= 0 && row[j] < b.n_pages;
    if (!__syncthreads_and(good)) {
      if (threadIdx.x == 0) report_pages(status);
      return;
    }
  }
  if (threadIdx.x == 0) {
    b.start[a.s] = kept > 0 ? begin % b.page_rows : 0;
    b.rows[a.s] = kept;
  }
  if (dead == 0) return;
  for (int j = threadIdx.x; j < dead; j += blockDim.x) atomicSub(&b.refs[row[j]], 1);
  // The row moves up `dead` places, a block of entries at a time: a block's
  // entries are read before any is written, and lie above every entry written
  // before it.
  for (int j0 = 0; j0 < pages; j0 += blockDim.x) {
    const int j = j0 + threadIdx.x;
    const int p = j + dead < pages ? row[j + dead] : -1;
    __syncthreads();
    if (j < pages) row[j] = p;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
// One CTA: the live pages are counted (N), then the k-th live page at or
// past N and the k-th free page before N are paired by rank.
__global__ void __launch_bounds__(kBlock) compact_kernel(PageBook b, int* __restrict__ new_id,
                                                         int* __restrict__ copy_src, int* __restrict__ copy_dst,
                                                         int* __restrict__ count) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ int2 sums[2][32];
  const int cap = b.n_pages + 1;
  constexpr int kTile = kBlock * kPerThread;
  __shared__ uint32_t masks[kBlock];
  int live = 0, turn = 0;
  const uint32_t used0 = used_mask(b, 0);
  for (int base = 0; base < b.n_pages; base += kTile) {
    const int past = max(0, min(kPerThread, base + static_cast<int>(threadIdx.x + 1) * kPerThread - b.n_pages));
    const uint32_t used = base == 0 ? used0 : used_mask(b, base);
    live += block_scan(make_int2(__popc(used) - past, 0), cap, sums, turn).all.x;
  }
  int holes = 0, moved = 0;
  for (int base = 0; base < b.n_pages; base += kTile) {
    const int p0 = base + threadIdx.x * kPerThread;
    const uint32_t used = base == 0 ? used0 : used_mask(b, base);
    // Bits of this thread's pages: in the pool, before N.
    auto upto = [&](int end) { return 0xffffu >> (kPerThread - max(0, min(kPerThread, end - p0))); };
    const uint32_t hole = ~used & upto(live), move = used & ~upto(live) & upto(b.n_pages);
    masks[threadIdx.x] = used;
    __syncthreads();
#pragma unroll 4
    for (int q = 0; q < kPerThread; ++q) {  // a warp's pages side by side
      const int e = q * kBlock + threadIdx.x, p = base + e;
      if (p >= b.n_pages) break;
      const bool u = masks[e / kPerThread] >> (e % kPerThread) & 1;
      if (!u || p < live) new_id[p] = u ? p : -1;
    }
    const Scan x = block_scan(make_int2(__popc(hole), __popc(move)), cap, sums, turn);
    int h = holes + x.at.x - __popc(hole);
    int m = moved + x.at.y - __popc(move);
    holes += x.all.x;
    moved += x.all.y;
    for (uint32_t x = hole; x != 0; x &= x - 1) copy_dst[h++] = p0 + __ffs(x) - 1;
    for (uint32_t x = move; x != 0; x &= x - 1) copy_src[m++] = p0 + __ffs(x) - 1;
  }
  __syncthreads();
  // As many holes before N as live pages past it: N pages are live.
  // No page is both, so a thread's four moves are loaded together.
  constexpr int U = 4;
  for (int k0 = threadIdx.x; k0 < b.n_pages; k0 += U * kBlock) {
    int a[U], z[U], refs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * kBlock;
      a[u] = k < moved ? copy_src[k] : -1;
      z[u] = k < moved ? copy_dst[k] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) refs[u] = a[u] >= 0 ? b.refs[a[u]] : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * kBlock;
      if (a[u] >= 0) {
        new_id[a[u]] = z[u];
        b.refs[z[u]] = refs[u];
        b.refs[a[u]] = 0;
      } else if (k < b.n_pages) {
        copy_src[k] = copy_dst[k] = -1;
      }
    }
  }
  if (threadIdx.x == 0) *count = moved;
}

// Table entries to their pages' new ids.
__global__ void __launch_bounds__(256) rename_kernel(PageBook b, const int* __restrict__ new_id,
                                                     unsigned int* status) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const long long total = static_cast<long long>(b.n_slots) * b.max_pages;
  for (long long e = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; e < total;
       e += static_cast<long long>(gridDim.x) * 256) {
    const int p = b.table[e];
    if (p < 0) continue;
    if (p < b.n_pages)
      b.table[e] = new_id[p];
    else
      report_pages(status);
  }
}

unsigned grid_for(long long work, long long most) {
  return static_cast<unsigned>(work < 1 ? 1 : (work < most ? work : most));
}

// Calls f with a vector type that divides `bits` (addresses and sizes or'ed).
template <typename F>
cudaError_t by_vector(uintptr_t bits, F f) {
  if (bits % 16 == 0) return f(uint4());
  if (bits % 4 == 0) return f(uint32_t());
  return f(uint16_t());
}

}  // namespace

cudaError_t launch_pages_reserve(const PageBook& b, const int* slots, const int* cu, int n, int* granted,
                                 int* copy_src, int* copy_dst, unsigned int* status, cudaStream_t stream) {
  const bool small = n <= kBlock;
  auto kern = small ? reserve_kernel<true> : reserve_kernel<false>;
  const size_t smem = (static_cast<size_t>(b.n_slots) + (small ? 3 : 1) * static_cast<size_t>(n)) * sizeof(int);
  if (smem > 24 * 1024) {  // beside 17 KB that every launch has
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               2 * kMaxSlots * static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(kern, dim3(1), dim3(kBlock), smem, stream, b, slots, cu, n, granted, copy_src,
                          copy_dst, status);
}

cudaError_t launch_pages_append(const PageBook& b, void* kp, void* vp, int H, int D, int elem, const int* slots,
                                const int* cu, int n, const int* granted, const int* copy_src, const int* copy_dst,
                                const void* kn, const void* vn, int T, unsigned int* status, cudaStream_t stream) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(kp) | reinterpret_cast<uintptr_t>(vp) |
                         reinterpret_cast<uintptr_t>(kn) | reinterpret_cast<uintptr_t>(vn) |
                         static_cast<uintptr_t>(D * elem);
  return by_vector(bits, [&](auto v) {
    using V = decltype(v);
    const int dv = D * elem / static_cast<int>(sizeof(V));
    // CTAs of an entry: by its mean share of the new rows and half a page of
    // copied ones, within about 8 CTAs per SM over all entries.
    const long long rows = T / n + 1 + (copy_src != nullptr ? b.page_rows / 2 : 0);
    const long long most = (152 * 8 + n - 1) / n;
    const dim3 grid(grid_for((rows * H * dv + 1023) / 1024, most), static_cast<unsigned>(n));
    return launch_dependent(append_kernel<V>, grid, dim3(256), 0, stream, b, static_cast<V*>(kp),
                            static_cast<V*>(vp), H, dv, slots, cu, granted, copy_src, copy_dst,
                            static_cast<const V*>(kn), static_cast<const V*>(vn), T,
                            std::max(1, 1024 / (H * dv)), Divisor(H * dv), Divisor(dv),
                            __builtin_ctz(b.page_rows), status);
  });
}

cudaError_t launch_pages_copy(void* kp, void* vp, int n_pages, long long page_bytes, const int* src, const int* dst,
                              int n, unsigned int* status, cudaStream_t stream) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(kp) | reinterpret_cast<uintptr_t>(vp) |
                         static_cast<uintptr_t>(page_bytes);
  return by_vector(bits, [&](auto v) {
    using V = decltype(v);
    const long long vecs = page_bytes / static_cast<long long>(sizeof(V));
    const long long chunks = 2 * ((vecs + 1023) / 1024) * n;
    return launch_dependent(copy_kernel<V>, dim3(grid_for(chunks, 152 * 8)), dim3(256), 0, stream,
                            static_cast<V*>(kp), static_cast<V*>(vp), n_pages, vecs, src, dst, n, status);
  });
}

cudaError_t launch_pages_fork(const PageBook& b, const int* src, const int* dst, int n, int* ok,
                              unsigned int* status, cudaStream_t stream) {
  return launch_dependent(fork_kernel, dim3(n), dim3(128), 0, stream, b, src, dst, n, ok, status);
}

cudaError_t launch_pages_free(const PageBook& b, const int* slots, const int* keep, int n, unsigned int* status,
                              cudaStream_t stream) {
  return launch_dependent(free_kernel, dim3(n), dim3(128), 0, stream, b, slots, keep, n, status);
}

cudaError_t launch_pages_compact(const PageBook& b, int* new_id, int* copy_src, int* copy_dst, int* count,
                                 unsigned int* status, cudaStream_t stream) {
  cudaError_t e =
      launch_dependent(compact_kernel, dim3(1), dim3(kBlock), 0, stream, b, new_id, copy_src, copy_dst, count);
  if (e != cudaSuccess) return e;
  const long long entries = static_cast<long long>(b.n_slots) * b.max_pages;
  return launch_dependent(rename_kernel, dim3(grid_for((entries + 255) / 256, 152 * 8)), dim3(256), 0, stream, b,
                          static_cast<const int*>(new_id), status);
}

}  // namespace txl
