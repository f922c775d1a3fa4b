// Pages that requests share: a block table, the uses of every page, and a pool for each layer.
//
// fork     out rows are copies of in rows; uses go up for one and down for the other (atomic additions, whose
//          order does not matter).  Bound: latency, an entry and an addition; 64 rows of 127 entries 2.0 us.
// reserve  a CTA looks at the entries that new rows touch, counts what they need, finds that many free
//          pages (the lowest, by ordered scans over the uses) and hands them out in order; the shared pages' rows
//          are copied in every layer.  Bound: the latency of lengths, table, uses and free pages one after another, then HBM
//          for the copies.  64 beams in fours, 8 layers of 8 heads: 9 us, 5 of them the plan; without copies 6.2.
//          Pages in use in front of the free ones cost 0.9 us per 4096 (32 us in a pool of 131072 whose last are free: every CTA
//          reads them, from L2; 16384 at a time took 30, and 2.5 longer where the pool is small).
// trim     entries behind a request's rows lose their pages: 1.9 us.
// accept   a warp per request, head and layer moves the rows of the accepted nodes to the tree's front, K by
//          one half and V by the other.  A row's place is never above where it comes from, so with all loads of eight
//          rows before their stores, in ascending order, nothing is overwritten before it is read.  Bound: latency, path,
//          entry, row and store one after another: 4.2 us for 32 requests of 8 heads and 8 layers.
#include <algorithm>

#include "../../include/kvsel.h"
#include "step.cuh"

namespace kvsel {
namespace {

constexpr int kThreads = 1024;

// rows of request b's shortest and longest head
__device__ __forceinline__ bool rows_of(const PagesArgs& a, const int32_t* lens, int b, int& lo, int& hi) {
  if (!a.per_head) {
    lo = hi = lens[b];
  } else {
    lo = hi = lens[b * a.H];
    for (int h = 1; h < a.H; ++h) {
      const int n = lens[b * a.H + h];
      lo = min(lo, n);
      hi = max(hi, n);
    }
  }
  return lo >= 0 && hi <= static_cast<long long>(a.max_blocks) << a.shift;
}

__global__ void __launch_bounds__(256) pages_fork_kernel(const PagesArgs a) {
  const int b = blockIdx.x % a.B, per = a.per_head ? a.H : 1;
  bool bad = false;
  if (static_cast<int>(blockIdx.x) < a.B) {
    int s = __ldg(a.src + b);
    if (s < -1 || s >= a.B) {
      bad = true;
      s = -1;
    }
    int32_t* to = a.table + static_cast<long long>(b) * a.max_blocks;
    const int32_t* of = a.table_in + static_cast<long long>(s) * a.max_blocks;
    for (int i = threadIdx.x; i < a.max_blocks; i += blockDim.x) {
      int page = s < 0 ? -1 : __ldg(of + i);
      if (page < -1 || page >= a.num_blocks) {
        bad = true;
        page = -1;
      }
      to[i] = page;
      if (page >= 0) atomicAdd(a.ref + page, 1);
    }
    for (int h = threadIdx.x; h < per; h += blockDim.x) a.lens_out[b * per + h] = s < 0 ? 0 : __ldg(a.lens_in + s * per + h);
  } else {
    const int32_t* of = a.table_in + static_cast<long long>(b) * a.max_blocks;
    for (int i = threadIdx.x; i < a.max_blocks; i += blockDim.x) {
      const int page = __ldg(of + i);
      if (page >= 0 && page < a.num_blocks) atomicSub(a.ref + page, 1);
    }
  }
  if (bad) atomicOr(a.status, DEV_BAD_INDEX);
}

__global__ void __launch_bounds__(256) pages_trim_kernel(const PagesArgs a) {
  const int b = blockIdx.x;
  int lo, hi;
  if (!rows_of(a, a.lens, b, lo, hi)) {
    if (threadIdx.x == 0) atomicOr(a.status, DEV_BAD_INDEX);
    return;
  }
  int32_t* row = a.table + static_cast<long long>(b) * a.max_blocks;
  const int keep = (hi + a.block_size - 1) >> a.shift;
  for (int i = keep + threadIdx.x; i < a.max_blocks; i += blockDim.x) {
    const int page = row[i];
    if (page == -1) continue;
    row[i] = -1;
    if (page >= 0 && page < a.num_blocks)
      atomicSub(a.ref + page, 1);
    else
      atomicOr(a.status, DEV_BAD_INDEX);
  }
}

// inclusive block-wide scan
__device__ __forceinline__ int block_scan(int v, int* s_w, int& total) {
  const int lane = lane_id(), warp = warp_id();
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) s_w[warp] = v;
  __syncthreads();
  int y = s_w[lane];                                 // every warp scans the 32 sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  total = __shfl_sync(0xffffffffu, y, 31);
  if (warp > 0) v += __shfl_sync(0xffffffffu, y, warp - 1);
  __syncthreads();
  return v;
}

// The first entry that the new rows of a request touch (rows [lo, end) are written to), and whether entry i is one.  A request
// that is not served touches none (end = 0) whatever its lengths are: a negative one would lead to words before the table,
// one near 2^31 to numbers that pass 32 bits.  (Where the entry is looked up does not wait for whether it is served.)
__host__ __device__ constexpr int first_entry(int lo, int shift) { return (lo > 0 ? lo : 0) >> shift; }
__host__ __device__ constexpr bool touched(int i, int end, int shift) { return static_cast<long long>(i) << shift < end; }
static_assert(first_entry(17, 4) == 1 && touched(1, 18, 4) && touched(2, 33, 4) && !touched(2, 32, 4) && touched(0, 1, 3));
static_assert(first_entry(-1, 3) == 0 && first_entry(-0x7FFFFFFF - 1, 6) == 0 && !touched(0, 0, 3) && !touched(1, 0, 6));
static_assert(!touched(first_entry(0x7FFFFFFF, 3), 0, 3) && !touched(first_entry(0x7FFFFFFF, 6) + (1 << 17) + 1, 0, 6));

struct Reserve {
  int lo, end, page0, m;          // first and last row that are written, the first's entry; new rows
  bool ok;
};
__device__ __forceinline__ Reserve reserve_of(const PagesArgs& a, int b) {
  Reserve r;
  int hi;
  const int raw = a.new_lens ? __ldg(a.new_lens + b) : a.m;
  r.m = min(max(raw, 0), a.m);
  r.ok = rows_of(a, a.lens, b, r.lo, hi) && raw == r.m &&
         static_cast<long long>(hi) + r.m <= static_cast<long long>(a.max_blocks) << a.shift;
  r.page0 = first_entry(r.lo, a.shift);
  r.end = r.ok ? hi + r.m : 0;
  // heads so far apart that their entries do not fit the plan
  if (r.ok && r.m > 0 && ((r.end - 1) >> a.shift) - r.page0 >= a.per) {
    r.ok = false;
    r.end = 0;
  }
  if (!r.ok || r.m == 0) r.end = 0;
  return r;
}

// kKeep: a shared page that its last writer takes over, without a page from the pool
enum Need : int { kNothing, kKeep, kPage, kCopy };
__device__ __forceinline__ bool wants(int need) { return need >= kPage; }

// What a reservation of up to kItems touched entries keeps in shared memory (larger ones: `need`, `pages`, `copies` and the
// list of shared entries are in the workspace).
constexpr int kItems = 1024;
struct PlanShared {
  int w[32];
  int end[KVSEL_MAX_ATTN_BATCH + 1];                 // pages wanted up to request b, at b + 1
  unsigned bad[KVSEL_MAX_ATTN_BATCH / 32], keeps[KVSEL_MAX_ATTN_BATCH / 32];
  int have;                                          // free pages found, as many as are wanted at most
  int copies;
  __device__ __forceinline__ static bool has(const unsigned* bits, int b) { return bits[b >> 5] >> (b & 31) & 1u; }
  // a request that takes a page over needs those before it to leave it: all that is asked for up to it
  __device__ __forceinline__ bool served(int b) const {
    return !has(bad, b) && ((end[b + 1] == end[b] && !has(keeps, b)) || end[b + 1] <= have);
  }
};

// The plan of a reservation, by one CTA: needs, pages and copies {from, to, rows} of all entries, in their order.  It
// writes nothing but these.  Returns the number of copies.
// SMALL: up to kItems entries: two numbers of them in one scan, and each shared page looked for among those before it.
// Otherwise shared pages are counted in a table of at least twice as many places (open addressing, linear steps): 2^20 of
// them, ranked against one another, would take a CTA half a minute.
template <bool SMALL>
__device__ __forceinline__ int plan_pages(const PagesArgs& a, PlanShared& s, int* need, int* pages, int4* copies, int* list) {
  constexpr int kMany = 1 << 15;                     // (kItems is less)
  const int tid = threadIdx.x, items = a.B * a.per;
  // the first uses are on their way before anything else is looked at
  int uses[4];
  auto fetch = [&](int p0) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int p = p0 + tid * 4 + u;
      uses[u] = p < a.num_blocks ? a.ref[p] : 1;
    }
  };
  fetch(0);
  if (tid == 0) s.end[0] = s.copies = 0;
  if (tid < KVSEL_MAX_ATTN_BATCH / 32) s.bad[tid] = s.keeps[tid] = 0;
  __syncthreads();
  // a thread has `each` entries in a row, as a rule one or none
  const int each = (items + kThreads - 1) / kThreads;
  const int i0 = min(items, tid * each), i1 = min(items, i0 + each);
  Reserve r{};
  int of = -1;                                       // whose r is
  auto range = [&](int b) -> const Reserve& {
    if (b != of) r = reserve_of(a, b);
    of = b;
    return r;
  };
  int mine = 0, shared = 0;
  for (int it = i0; it < i1; ++it) {
    const int b = it / a.per, u = it - b * a.per;
    range(b);
    int n = kNothing;
    const int i = r.page0 + u;
    if (!r.ok && u == 0) atomicOr(&s.bad[b >> 5], 1u << (b & 31));
    if (touched(i, r.end, a.shift)) {
      const int page = a.table[static_cast<long long>(b) * a.max_blocks + i];
      if (page == -1) {
        n = kPage;
      } else if (page < 0 || page >= a.num_blocks) {
        atomicOr(&s.bad[b >> 5], 1u << (b & 31));
      } else if (a.ref[page] > 1) {
        n = kCopy;                                   // to be seen
        ++shared;
      }
    }
    need[it] = n;
  }
  int sharers;
  int at = block_scan(shared, s.w, sharers) - shared;
  if (sharers) {
    // Of the requests that write to a shared page the last keeps it where no other uses it: as many of them before it
    // as the page has other uses (requests that are not served for what their entries hold do not count).  `list`, in
    // order of entries: their pages, or the places that count them (-1: of a request that is not served).
    auto page_at = [&](int it) {
      const int b = it / a.per;
      return s.has(s.bad, b) ? -1 : a.table[static_cast<long long>(b) * a.max_blocks + range(b).page0 + it % a.per];
    };
    auto keep = [&](int it) {
      need[it] = kKeep;
      atomicOr(&s.keeps[it / a.per >> 5], 1u << (it / a.per & 31));
    };
    if constexpr (SMALL) {
      for (int it = i0, k = at; it < i1; ++it)
        if (need[it] == kCopy) list[k++] = page_at(it);
      __syncthreads();
      for (int it = i0; it < i1; ++it) {
        if (need[it] != kCopy) continue;
        const int page = list[at];
        int before = 0;
#pragma unroll 8
        for (int c = 0; c < at; ++c) before += list[c] == page;
        ++at;
        if (page >= 0 && before >= a.ref[page] - 1) keep(it);
      }
    } else {
      int log = 6;
      while (1 << log < 2 * sharers) ++log;
      const int slots = 1 << log;
      // of a place: the page, the last entry that writes to it, and the number of those
      int32_t *key = a.seats, *last = a.seats + slots, *writers = a.seats + 2 * slots;
      for (int i = tid; i < 3 * slots; i += kThreads) a.seats[i] = i < 2 * slots ? -1 : 0;
      __syncthreads();
      for (int it = i0, k = at; it < i1; ++it) {
        if (need[it] != kCopy) continue;
        const int page = page_at(it);
        int y = -1;
        if (page >= 0) {
          y = static_cast<int>(static_cast<unsigned>(page) * 2654435769u >> (32 - log));   // (2^32 by the golden ratio)
          while (true) {                             // (half of the places stay empty)
            const int other = atomicCAS(key + y, -1, page);
            if (other == -1 || other == page) break;
            y = (y + 1) & (slots - 1);
          }
          atomicMax(last + y, it);
          atomicAdd(writers + y, 1);
        }
        list[k++] = y;
      }
      __syncthreads();
      for (int it = i0; it < i1; ++it) {
        if (need[it] != kCopy) continue;
        const int y = list[at++];
        if (y >= 0 && __ldcg(last + y) == it && __ldcg(writers + y) >= a.ref[__ldcg(key + y)]) keep(it);
      }
    }
  }
  __syncthreads();
  for (int it = i0; it < i1; ++it) {
    const int b = it / a.per;
    if (s.has(s.bad, b)) need[it] = kNothing;
    mine += wants(need[it]) + (SMALL && need[it] == kCopy ? kMany : 0);
  }
  // pages wanted before this thread's entries, and copies among them
  int total, before, c;
  if (SMALL) {
    const int sum = block_scan(mine, s.w, total) - mine;
    before = sum & (kMany - 1);
    c = sum / kMany;
    total &= kMany - 1;
  } else {
    before = block_scan(mine, s.w, total) - mine;
    int copied = 0;
    for (int it = i0; it < i1; ++it) copied += need[it] == kCopy;
    int all;
    c = block_scan(copied, s.w, all) - copied;
  }
  for (int it = i0, upto = before; it < i1; ++it) {
    upto += wants(need[it]);
    if ((it + 1) % a.per == 0) s.end[(it + 1) / a.per] = upto;
  }
  // the lowest free pages, as many as are wanted
  int have = 0;
  for (int p0 = 0; p0 < a.num_blocks && have < total; p0 += kThreads * 4) {
    int free = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) free |= (uses[u] == 0) << u;
    fetch(p0 + kThreads * 4);
    int got;
    int k = have + block_scan(__popc(free), s.w, got) - __popc(free);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (free >> u & 1) {
        if (k < total) pages[k] = p0 + tid * 4 + u;
        ++k;
      }
    have += got;
  }
  if (tid == 0) s.have = have;
  __syncthreads();
  // requests in order while the pages last (the copies of those that are not served come behind all others)
  for (int it = i0, k = before; it < i1; ++it) {
    const int b = it / a.per, u = it - b * a.per, n = need[it];
    if (n == kCopy) {
      if (s.end[b + 1] <= have) {
        range(b);
        const int i = r.page0 + u;
        copies[c] = make_int4(a.table[static_cast<long long>(b) * a.max_blocks + i], pages[k],
                              min(a.block_size, r.end - r.m - (i << a.shift)), 0);
        atomicMax(&s.copies, c + 1);
      }
      ++c;
    }
    k += wants(n);
  }
  __syncthreads();
  return s.copies;
}

// The plan's table entries, uses and what was granted, by one CTA.
__device__ __forceinline__ void apply_pages(const PagesArgs& a, const PlanShared& s, const int* need, const int* pages) {
  const int tid = threadIdx.x, items = a.B * a.per, each = (items + kThreads - 1) / kThreads;
  const int i0 = min(items, tid * each), i1 = min(items, i0 + each);
  if (tid < KVSEL_MAX_ATTN_BATCH / 32 && s.bad[tid]) atomicOr(a.status, DEV_BAD_INDEX);
  int k = 0;                                         // the entry's place among the pages, if it wants one
  for (int it = i0; it < i1; ++it) {
    const int b = it / a.per, u = it - b * a.per;
    const bool served = s.served(b);
    const Reserve r = reserve_of(a, b);
    if (u == 0) a.granted[b] = served ? r.m : 0;
    if (u == 0 || it == i0) {
      k = s.end[b];
      for (int v = 0; v < u; ++v) k += wants(need[b * a.per + v]);
    }
    if (!wants(need[it])) continue;
    ++k;
    if (!served) continue;
    const int page = pages[k - 1];
    int32_t* entry = a.table + static_cast<long long>(b) * a.max_blocks + r.page0 + u;
    if (need[it] == kCopy) atomicSub(a.ref + *entry, 1);
    *entry = page;
    a.ref[page] = 1;
  }
}

// Rows of all heads of a page lie together: one side (K, V) of a copy in a layer by a group of 256 threads, all loads of a
// batch before its first store.
constexpr int kAtOnce = 8;
__device__ __forceinline__ void copy_page(const PagesArgs& a, const int4& x, int layer, int side, int tid) {
  const long long page = static_cast<long long>(a.block_size) * a.H * (kHeadDim / 8);   // in 16-byte pieces
  const int pieces = x.z * a.H * (kHeadDim / 8);
  uint4* rows = reinterpret_cast<uint4*>((side ? a.v : a.k) + layer * a.stride_layer);
  for (int i0 = tid; i0 < pieces; i0 += 256 * kAtOnce) {
    uint4 y[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      if (i0 + u * 256 < pieces) y[u] = rows[x.x * page + i0 + u * 256];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      if (i0 + u * 256 < pieces) rows[x.y * page + i0 + u * 256] = y[u];
  }
}

// A reservation of up to kItems entries in one launch: every CTA makes the same plan for itself and copies its share of
// the pages; the last of them to have made it (`ticket`; none waits for another) writes the table and the uses, which
// all have read by then.  (Two launches: 1.9 us more on the GPU and 2.3 on the host.)
__global__ void __launch_bounds__(kThreads, 1) pages_reserve_kernel(const PagesArgs a) {
  __shared__ PlanShared s;
  __shared__ int s_need[kItems], s_pages[kItems], s_list[kItems];
  __shared__ int4 s_copies[kItems];
  __shared__ bool s_last;
  const int copies = plan_pages<true>(a, s, s_need, s_pages, s_copies, s_list);
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(a.ticket, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (s_last) {
    __threadfence();
    apply_pages(a, s, s_need, s_pages);
    if (threadIdx.x == 0) *a.ticket = 0;
  }
  const int groups = gridDim.x * (kThreads / 256), units = copies * a.layers * 2;
  for (int i = blockIdx.x + gridDim.x * (threadIdx.x >> 8); i < units; i += groups)
    copy_page(a, s_copies[(i >> 1) / a.layers], (i >> 1) % a.layers, i & 1, threadIdx.x & 255);
}

// Larger ones: a launch of one CTA for the plan, and one for the copies.
__global__ void __launch_bounds__(kThreads) pages_plan_kernel(const PagesArgs a) {
  __shared__ PlanShared s;
  const int copies = plan_pages<false>(a, s, a.need, a.pages, a.copies + 1, a.list);
  apply_pages(a, s, a.need, a.pages);
  if (threadIdx.x == 0) a.copies[0].x = copies;
}
__global__ void __launch_bounds__(256) pages_copy_kernel(const PagesArgs a) {
  const int n = a.copies[0].x;
  for (int c = blockIdx.x; c < n; c += gridDim.x)
    for (int layer = blockIdx.y; layer < a.layers; layer += gridDim.y)
      for (int side = 0; side < 2; ++side) copy_page(a, a.copies[1 + c], layer, side, threadIdx.x);
}

constexpr int kRows = 8;                             // of a path at a time
__global__ void __launch_bounds__(256) pages_accept_kernel(const PagesArgs a) {
  const int lane = lane_id(), item = blockIdx.x * 8 + warp_id();
  if (item >= a.B * a.H * a.layers) return;
  const int layer = item / (a.B * a.H), bh = item - layer * a.B * a.H, b = bh / a.H, h = bh - b * a.H;
  const int raw_m = a.new_lens ? __ldg(a.new_lens + b) : a.m, m = min(max(raw_m, 0), a.m);
  const int raw_n = a.lens[a.per_head ? bh : b], raw_c = __ldg(a.counts + b);
  const int n = static_cast<int>(min(static_cast<long long>(max(raw_n, 0)), static_cast<long long>(a.max_blocks) << a.shift));
  const int base = max(0, n - m), count = min(max(raw_c, 0), n - base);
  bool bad = raw_m != m || raw_n != n || raw_c != count || n < m;
  if (a.lens_out && layer == 0 && (a.per_head || h == 0) && lane == 0) a.lens_out[a.per_head ? bh : b] = base + count;
  const int32_t* row = a.table + static_cast<long long>(b) * a.max_blocks;
  const int32_t* path = a.path + static_cast<long long>(b) * a.m;
  uint4* cache = reinterpret_cast<uint4*>((lane >> 4 ? a.v : a.k) + layer * a.stride_layer) + (lane & 15);
  auto place = [&](int j) -> long long {
    const int page = row[j >> a.shift];
    if (page < 0 || page >= a.num_blocks) return -1;
    return ((static_cast<long long>(page) << a.shift) + (j & (a.block_size - 1))) * a.H + h;
  };
  for (int i0 = 0; i0 < count; i0 += kRows) {
    // lane i: entry i0 + i of the path
    long long of = -1, to = -1;
    const int i = i0 + lane;
    if (lane < kRows && i < count) {
      const int x = __ldg(path + i);
      if (x < i || x >= n - base || (i > 0 && x <= __ldg(path + i - 1))) {
        bad = true;
      } else if (x > i) {
        of = place(base + x);
        to = place(base + i);
        if (of < 0 || to < 0) {
          bad = true;
          of = to = -1;
        }
      }
    }
    uint4 y[kRows];
    long long dst[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const long long src = __shfl_sync(0xffffffffu, of, u);
      dst[u] = __shfl_sync(0xffffffffu, to, u);
      y[u] = make_uint4(0u, 0u, 0u, 0u);
      if (dst[u] >= 0) y[u] = cache[src * (kHeadDim / 8)];
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      if (dst[u] >= 0) cache[dst[u] * (kHeadDim / 8)] = y[u];
  }
  if (bad && layer == 0) atomicOr(a.status, DEV_BAD_INDEX);
}

// after the rows have moved, where lens_out is lens
__global__ void __launch_bounds__(256) pages_lens_kernel(const PagesArgs a) {
  const int i = blockIdx.x * 256 + threadIdx.x, b = a.per_head ? i / a.H : i;
  if (b >= a.B) return;
  const int m = min(max(a.new_lens ? __ldg(a.new_lens + b) : a.m, 0), a.m);
  const int n = static_cast<int>(min(static_cast<long long>(max(a.lens[i], 0)), static_cast<long long>(a.max_blocks) << a.shift));
  const int base = max(0, n - m);
  a.lens_out[i] = base + min(max(__ldg(a.counts + b), 0), n - base);
}

}  // namespace

cudaError_t launch_pages_fork(const PagesArgs& a, cudaStream_t st) {
  pages_fork_kernel<<<2 * a.B, 256, 0, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_pages_trim(const PagesArgs& a, cudaStream_t st) {
  pages_trim_kernel<<<a.B, 256, 0, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_pages_reserve(const PagesArgs& a, int sms, cudaStream_t st) {
  if (a.B * a.per <= kItems) {
    // a CTA per SM, or one for every four sides of copies that there may be
    const long long units = 2ll * a.B * a.layers;
    pages_reserve_kernel<<<static_cast<unsigned>(std::min<long long>(sms, (units + 3) / 4)), kThreads, 0, st>>>(a);
    note_launch();
    return cudaGetLastError();
  }
  pages_plan_kernel<<<1, kThreads, 0, st>>>(a);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.m == 0) return e;
  // requests share one page each as a rule
  const int layers = std::min(a.layers, 64), gx = std::max(1, std::min(a.B, 8 * sms / layers));
  pages_copy_kernel<<<dim3(gx, layers), 256, 0, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_pages_accept(const PagesArgs& args, cudaStream_t st) {
  PagesArgs a = args;
  const bool apart = args.lens_out != args.lens;     // otherwise after all rows have moved
  if (!apart) a.lens_out = nullptr;
  const long long items = static_cast<long long>(a.B) * a.H * a.layers;
  pages_accept_kernel<<<static_cast<unsigned>((items + 7) / 8), 256, 0, st>>>(a);
  note_launch();
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || apart) return e;
  const int n = a.per_head ? a.B * a.H : a.B;
  pages_lens_kernel<<<(n + 255) / 256, 256, 0, st>>>(args);
  note_launch();
  return cudaGetLastError();
}

}  // namespace kvsel
