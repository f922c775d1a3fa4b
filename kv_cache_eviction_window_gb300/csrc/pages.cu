// Pages that requests share: a block table, the uses of every page, and a pool for each layer.
//
// fork     out rows are copies of in rows; uses go up for one and down for the other (atomic additions, whose
//          order does not matter).  Bound: latency, an entry and an addition.
// reserve  one CTA looks at the entries that new rows touch, counts what they need, finds that many free
//          pages (the lowest, by ordered scans over the uses) and hands them out in order; a second launch copies
//          the shared pages' rows in every layer.  Bound: latency, then HBM for the copies.
// trim     entries behind a request's rows lose their pages.
// accept   a warp per request, head and layer moves the rows of the accepted nodes to the tree's front, K by
//          one half and V by the other.  A row's place is never above where it comes from, so with all loads of eight
//          rows before their stores, in ascending order, nothing is overwritten before it is read.
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
  r.page0 = r.lo >> a.shift;
  r.end = r.ok ? hi + r.m : 0;
  // heads so far apart that their entries do not fit the plan
  if (r.ok && r.m > 0 && ((r.end - 1) >> a.shift) - r.page0 >= a.per) {
    r.ok = false;
    r.end = 0;
  }
  if (!r.ok || r.m == 0) r.end = 0;
  return r;
}

enum Need : int { kNothing, kPage, kCopy };
constexpr int kShared = 4096;                        // entries with a shared page that are kept in shared memory

__global__ void __launch_bounds__(kThreads) pages_plan_kernel(const PagesArgs a) {
  __shared__ int s_w[32];
  __shared__ int s_copies;
  __shared__ int s_end[KVSEL_MAX_ATTN_BATCH + 1];    // pages wanted up to request b, at b + 1
  __shared__ unsigned s_bad[KVSEL_MAX_ATTN_BATCH / 32];
  __shared__ int s_shared[kShared];
  const int tid = threadIdx.x, items = a.B * a.per;
  if (tid == 0) s_copies = s_end[0] = 0;
  if (tid < KVSEL_MAX_ATTN_BATCH / 32) s_bad[tid] = 0;
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
    int need = kNothing;
    const int i = r.page0 + u;
    if (!r.ok && u == 0) atomicOr(&s_bad[b >> 5], 1u << (b & 31));
    if ((static_cast<long long>(i) << a.shift) < r.end) {
      const int page = a.table[static_cast<long long>(b) * a.max_blocks + i];
      if (page < 0) {
        need = kPage;
      } else if (page >= a.num_blocks) {
        atomicOr(&s_bad[b >> 5], 1u << (b & 31));
      } else if (a.ref[page] > 1) {
        need = kCopy;                                // to be seen
        ++shared;
      }
    }
    a.need[it] = need;
  }
  int sharers;
  int at = block_scan(shared, s_w, sharers) - shared;
  if (sharers) {
    // Of the requests that write to a shared page the last keeps it where no other uses it: as many of them before it
    // as the page has other uses.  The pages in order of entries: here, or where the free ones go later.
    int* list = sharers <= kShared ? s_shared : a.pages;
    int k = at;
    for (int it = i0; it < i1; ++it)
      if (a.need[it] == kCopy) list[k++] = a.table[static_cast<long long>(it / a.per) * a.max_blocks + range(it / a.per).page0 + it % a.per];
    __syncthreads();
    for (int it = i0; it < i1; ++it) {
      if (a.need[it] != kCopy) continue;
      const int page = list[at];
      int before = 0;
      for (int c = 0; c < at; ++c) before += list[c] == page;
      if (before >= a.ref[page] - 1) a.need[it] = kNothing;
      ++at;
    }
  }
  __syncthreads();
  for (int it = i0; it < i1; ++it) {
    const int b = it / a.per;
    if (s_bad[b >> 5] >> (b & 31) & 1u) a.need[it] = kNothing;
    mine += a.need[it] != kNothing;
  }
  if (tid < KVSEL_MAX_ATTN_BATCH / 32 && s_bad[tid]) atomicOr(a.status, DEV_BAD_INDEX);
  int total;
  int before = block_scan(mine, s_w, total) - mine;
  for (int it = i0, upto = before; it < i1; ++it) {
    upto += a.need[it] != kNothing;
    if ((it + 1) % a.per == 0) s_end[(it + 1) / a.per] = upto;
  }
  // the lowest free pages, as many as are wanted
  int have = 0;
  for (int p0 = 0; p0 < a.num_blocks && have < total; p0 += kThreads * 4) {
    const int p = p0 + tid * 4;
    int free = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (p + u < a.num_blocks && a.ref[p + u] == 0) free |= 1 << u;
    int got;
    int at = have + block_scan(__popc(free), s_w, got) - __popc(free);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (free >> u & 1) {
        if (at < total) a.pages[at] = p + u;
        ++at;
      }
    have += got;
  }
  __syncthreads();
  // requests in order while the pages last
  for (int it = i0; it < i1; ++it) {
    const int b = it / a.per, u = it - b * a.per;
    const bool served = s_end[b + 1] == s_end[b] || s_end[b + 1] <= have;
    const int need = a.need[it];
    if (u == 0) {
      const bool bad = s_bad[b >> 5] >> (b & 31) & 1u;
      a.granted[b] = served && !bad ? range(b).m : 0;
    }
    if (need != kNothing) {
      if (served) {
        range(b);
        const int i = r.page0 + u, page = a.pages[before];
        int32_t* entry = a.table + static_cast<long long>(b) * a.max_blocks + i;
        if (need == kCopy) {
          const int old = *entry, at = atomicAdd(&s_copies, 1);
          a.copies[1 + at] = make_int4(old, page, min(a.block_size, r.end - r.m - (i << a.shift)), 0);
          atomicSub(a.ref + old, 1);
        }
        *entry = page;
        a.ref[page] = 1;
      }
      ++before;
    }
  }
  __syncthreads();
  if (tid == 0) a.copies[0].x = s_copies;
}

constexpr int kAtOnce = 4;
// grid (copies, layer): rows of all heads of a page lie together
__global__ void __launch_bounds__(256) pages_copy_kernel(const PagesArgs a) {
  const int n = a.copies[0].x;
  const long long page = static_cast<long long>(a.block_size) * a.H * (kHeadDim / 8);   // in 16-byte pieces
  for (int c = blockIdx.x; c < n; c += gridDim.x) {
    const int4 x = a.copies[1 + c];
    const int pieces = x.z * a.H * (kHeadDim / 8);
    for (int layer = blockIdx.y; layer < a.layers; layer += gridDim.y) {
      uint4* k = reinterpret_cast<uint4*>(a.k + layer * a.stride_layer);
      uint4* v = reinterpret_cast<uint4*>(a.v + layer * a.stride_layer);
      // (all loads of a batch come before its first store)
      for (int i0 = threadIdx.x; i0 < pieces; i0 += 256 * kAtOnce) {
        uint4 y[kAtOnce], z[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
          if (i0 + u * 256 < pieces) {
            y[u] = k[x.x * page + i0 + u * 256];
            z[u] = v[x.x * page + i0 + u * 256];
          }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
          if (i0 + u * 256 < pieces) {
            k[x.y * page + i0 + u * 256] = y[u];
            v[x.y * page + i0 + u * 256] = z[u];
          }
      }
    }
  }
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
