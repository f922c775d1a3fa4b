// Eviction by accumulated attention weight, with room made for new rows.  A segment keeps
// `keep` = min(rows, budget - new rows) of its rows: first the protected ones (first and most
// recent positions), then those with the largest accumulated weight, ties by the lower slot.
// Evicted slots below `keep` are holes; the kept rows at or behind `keep` fill them, in
// order; the new rows follow at `keep`.  So a row moves only when it has to, nothing that is
// read is written by another slot, and the new rows are the segment's last.
//
// evict_few_kernel: up to four rows to evict (a decode step): one CTA per segment finds them by
// as many block-wide minima and moves the rows itself.  Bound: latency.
// evict_select_kernel: one CTA per segment ranks the slots: the keep-th largest key by a radix
// selection in three digits at most (it ends when a whole bin stays: then there are no ties to rank
// either; 4 to 5 us less for 200 to 16384 slots), then ordered scans for ties, holes and fills.  The keys stay in
// shared memory (up to 49,152 slots); a thread owns an odd number of consecutive slots, so that
// its walk through them meets no bank twice and equal neighbours cost one count.
// With no more segments than SMs and at most 64 rows to move, the same CTA moves them (200 slots, five
// rows, 8 us with the second launch, 6 without; 256 segments 20.5 and 24, two CTAs an SM no longer).
// evict_move_kernel: slot keep + i of a segment is handled by one half warp per side: its old
// row goes to its hole, then new row i takes the slot.  A warp takes two slots at a time (one: 37.2
// us for the call with 2048 rows of 32 segments of 16384, two 35.7, four 38.3; 31.6 now, 17 of them the selection).  Bound: the latency
// of a slot's chain of loads (its rank, its hole, their pages, its row), then HBM, 512 B per moved
// or new row read and written (and 8 B per slot before).
#include <algorithm>

#include "evict.cuh"

namespace kvsel {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32, kEach = 2;   // of the second launch; slots per warp at a time

// Rank of a weight as an unsigned number: larger weight, larger number; NaN below all.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  const uint32_t k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return min(k, 0xFFFFFFFEu);
}

struct Seg {
  int n, m, keep, seen, recent0;  // recent0: first protected recent position
};
__device__ __forceinline__ Seg seg_of(const EvictArgs& a, int seg) {
  Seg s;
  const int raw = a.lens[seg];
  s.n = min(max(raw, 0), a.capacity);
  const int mr = a.new_lens ? __ldg(a.new_lens + seg / a.H) : a.m;
  s.m = min(max(mr, 0), a.m);
  if (s.n != raw || s.m != mr) atomicOr(a.status, DEV_BAD_INDEX);
  s.keep = min(s.n, a.budget - s.m);
  s.seen = a.seen[seg];
  s.recent0 = s.seen + s.m - a.n_recent;
  return s;
}
__device__ __forceinline__ uint32_t slot_key(const EvictArgs& a, const Seg& s, long long base, int i) {
  const int p = a.pos[base + i];
  const float w = a.acc[base + i];                   // (both loads before the test)
  return p < a.n_sink || p >= s.recent0 ? 0xFFFFFFFFu : weight_key(w);
}

// inclusive block-wide scan
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* s_w,
                                                         unsigned long long& total) {
  const int lane = lane_id(), warp = warp_id();
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) s_w[warp] = v;
  __syncthreads();
  unsigned long long y = s_w[lane];                  // every warp scans the 32 sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  total = __shfl_sync(0xffffffffu, y, 31);
  if (warp > 0) v += __shfl_sync(0xffffffffu, y, warp - 1);
  __syncthreads();
  return v;
}

__device__ __forceinline__ long long slot_elem(const EvictArgs& a, int b, int h, int i) {
  if (!a.src.paged) return b * a.stride_req + h * a.stride_head + static_cast<long long>(i) * a.stride_tok;
  const int bs = a.src.block_size;
  const int pb = __ldg(a.src.block_table + static_cast<size_t>(b) * a.src.max_blocks + i / bs);
  if (pb < 0 || pb >= a.src.num_blocks) return -1;
  return ((static_cast<long long>(pb) * bs + (i % bs)) * a.H + h) * kHeadDim;
}

// Slots i of a segment, by one warp: each slot's old row to slot `to` (-1: it does not stay, or stays where
// it is), then new row `fresh` (-1: none) in its place.  All loads come before the first store.
template <int N>
__device__ __forceinline__ void move_slots(const EvictArgs& a, int b, int h, long long base, const int (&i)[N],
                                           const int (&to)[N], const int (&fresh)[N], int seen) {
  const int lane = lane_id(), side = lane >> 4, piece = lane & 15;
  uint4* cache = reinterpret_cast<uint4*>(side ? a.v : a.k) + piece;
  const uint4* rows = reinterpret_cast<const uint4*>(side ? a.v_new : a.k_new) + piece;
  long long from[N], dst[N];
  uint4 old[N], add[N];
  int p[N];
  float w[N];
  bool bad = false;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    add[u] = make_uint4(0u, 0u, 0u, 0u);
    if (fresh[u] >= 0)
      add[u] = __ldg(rows + (b * a.new_req + h * a.new_head + static_cast<long long>(fresh[u]) * a.new_tok) / 8);
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    from[u] = to[u] >= 0 || fresh[u] >= 0 ? slot_elem(a, b, h, i[u]) : 0;
    dst[u] = to[u] >= 0 ? slot_elem(a, b, h, to[u]) : 0;
    bad |= from[u] < 0 || dst[u] < 0;
    old[u] = make_uint4(0u, 0u, 0u, 0u);
    if (to[u] >= 0) {
      if (from[u] >= 0 && dst[u] >= 0) old[u] = cache[from[u] / 8];
      if (lane == 0) {
        p[u] = a.pos[base + i[u]];
        w[u] = a.acc[base + i[u]];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    if (to[u] >= 0) {
      if (from[u] >= 0 && dst[u] >= 0) cache[dst[u] / 8] = old[u];
      if (lane == 0) {
        a.pos[base + to[u]] = p[u];
        a.acc[base + to[u]] = w[u];
      }
    }
    if (fresh[u] >= 0) {
      if (from[u] >= 0) cache[from[u] / 8] = add[u];
      if (lane == 0) {
        a.pos[base + i[u]] = seen + fresh[u];
        a.acc[base + i[u]] = 0.f;
      }
    }
  }
  if (bad && lane == 0) atomicOr(a.status, DEV_BAD_INDEX);
}

// The rows behind the `keep` that stay of n, and m new ones, by warp `warp` of `warps`.
__device__ __forceinline__ void move_rows(const EvictArgs& a, int seg, int keep, int n, int m, int seen, const int* holes,
                                          const int* fills, int warp, int warps) {
  const int b = seg / a.H, h = seg - b * a.H, slots = max(n - keep, m);
  const long long base = static_cast<long long>(seg) * a.capacity;
  for (int u0 = warp * kEach; u0 < slots; u0 += warps * kEach) {
    int i[kEach], to[kEach], fresh[kEach];
#pragma unroll
    for (int v = 0; v < kEach; ++v) {
      i[v] = keep + u0 + v;
      to[v] = u0 + v < n - keep ? fills[u0 + v] : -1;
      fresh[v] = u0 + v < m ? u0 + v : -1;
    }
#pragma unroll
    for (int v = 0; v < kEach; ++v)
      if (to[v] >= 0) to[v] = holes[to[v]];
    move_slots<kEach>(a, b, h, base, i, to, fresh, seen);
  }
}

constexpr int kKeptSlots = 49152;                    // slots whose keys fit into shared memory

constexpr int kHere = 64;                            // rows that the selecting CTA may move itself

// KEPT: the keys are in shared memory, else formed again from pos and acc in every pass.
// HERE: the CTA moves the rows too (evict_here).
template <bool KEPT, bool HERE>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t s_key[];
  __shared__ int s_hist[2048];
  __shared__ unsigned long long s_w[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need, s_all;
  __shared__ int s_holes[HERE ? kHere : 1], s_fills[HERE ? kHere : 1];
  const int seg = blockIdx.x, tid = threadIdx.x;
  const Seg s = seg_of(a, seg);
  const long long base = static_cast<long long>(seg) * a.capacity;
  __syncthreads();   // every thread has read lens and seen
  if (tid == 0) {
    if (!HERE) a.head[seg] = make_int4(s.keep, s.n, s.m, s.seen);
    a.lens[seg] = s.keep + s.m;
    a.seen[seg] = s.seen + s.m;
  }
  if (s.keep == s.n) {
    if (HERE) move_rows(a, seg, s.keep, s.n, s.m, s.seen, s_holes, s_fills, warp_id(), kSelThreads / 32);
    return;
  }
  if (KEPT) {
#pragma unroll 8
    for (int i = tid; i < s.n; i += kSelThreads) s_key[i] = slot_key(a, s, base, i);
  }
  const int run = ((s.n + kSelThreads - 1) / kSelThreads) | 1;
  const int i0 = static_cast<int>(min(static_cast<long long>(s.n), static_cast<long long>(tid) * run));
  const int i1 = static_cast<int>(min(static_cast<long long>(s.n), static_cast<long long>(i0) + run));
  auto key = [&](int i) { return KEPT ? s_key[i] : slot_key(a, s, base, i); };

  // the keep-th largest key, by digits of 11, 11 and 10 bits from the top
  uint32_t prefix = 0, mask = 0;
  int need = s.keep;                                 // rank among the keys that share the prefix
  if (s.keep == 0) prefix = 0xFFFFFFFFu, mask = 0xFFFFFFFFu, need = 0;
  bool all = false;                                  // every key that shares the prefix stays
  for (int pass = 0; pass < 3 && s.keep > 0 && !all; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bins = pass == 2 ? 1024 : 2048;
    for (int i = tid; i < bins; i += kSelThreads) s_hist[i] = 0;
    __syncthreads();
    int bin = -1, cnt = 0;
#pragma unroll 4
    for (int i = i0; i < i1; ++i) {
      const uint32_t k = key(i);
      if ((k & mask) != prefix) continue;
      const int d = static_cast<int>((k >> shift) & (bins - 1));
      if (d != bin) {
        if (cnt) atomicAdd(&s_hist[bin], cnt);
        bin = d;
        cnt = 0;
      }
      ++cnt;
    }
    if (cnt) atomicAdd(&s_hist[bin], cnt);
    __syncthreads();
    // thread t owns bins 2t and 2t + 1 counted from the top
    const int per = bins / kSelThreads;
    int own = 0;
    for (int u = 0; u < per; ++u) own += s_hist[bins - 1 - (tid * per + u)];
    unsigned long long total;
    int before = static_cast<int>(block_scan(own, s_w, total)) - own;
    for (int u = 0; u < per; ++u) {
      const int d = bins - 1 - (tid * per + u), c = s_hist[d];
      if (before < need && need <= before + c) {
        s_prefix = prefix | (static_cast<uint32_t>(d) << shift);
        s_need = need - before;
        s_all = need - before == c;
      }
      before += c;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    all = s_all;
    mask |= static_cast<uint32_t>(bins - 1) << shift;
  }
  // keys above `prefix` stay, and of the slots whose key equals it all, or the first `need`
  __syncthreads();
  unsigned long long total;
  int ties0 = 0;
  if (!all) {
    int ties = 0;
#pragma unroll 4
    for (int i = i0; i < i1; ++i) ties += key(i) == prefix;
    ties0 = static_cast<int>(block_scan(ties, s_w, total)) - ties;
  }
  auto stays = [&](uint32_t k, int& t) {
    k &= mask;
    return k > prefix || (k == prefix && (all || t++ < need));
  };
  unsigned long long v = 0;                          // holes above, fills below
  int t = ties0;
#pragma unroll 4
  for (int i = i0; i < i1; ++i) {
    const bool kept = stays(key(i), t);
    if (!kept && i < s.keep) v += 1ull << 32;
    if (kept && i >= s.keep) v += 1;
  }
  const unsigned long long sc = block_scan(v, s_w, total) - v;
  int* holes = HERE ? s_holes : a.holes + static_cast<long long>(seg) * a.most;
  int* fills = HERE ? s_fills : a.fills + static_cast<long long>(seg) * a.most;
  int hole = static_cast<int>(sc >> 32), fill = static_cast<int>(sc & 0xFFFFFFFFu);
  t = ties0;
  for (int i = i0; i < i1; ++i) {
    const bool kept = stays(key(i), t);
    if (!kept && i < s.keep) holes[hole++] = i;
    if (i >= s.keep) fills[i - s.keep] = kept ? fill++ : -1;
  }
  if (HERE) {
    __syncthreads();
    move_rows(a, seg, s.keep, s.n, s.m, s.seen, s_holes, s_fills, warp_id(), kSelThreads / 32);
  }
}

// At most kFew rows to evict and to append.  A slot ranks by (key, then the later slot first): the
// first of that order leave.  A thread keeps the kFew lowest of its own slots, sorted.
constexpr int kFew = 4;
__global__ void __launch_bounds__(kSelThreads) evict_few_kernel(const EvictArgs a) {
  __shared__ unsigned long long s_min[kFew][32];
  const int seg = blockIdx.x, b = seg / a.H, h = seg - b * a.H;
  const Seg s = seg_of(a, seg);
  const long long base = static_cast<long long>(seg) * a.capacity;
  const int gone = s.n - s.keep;                     // rows that leave
  int out[kFew];
#pragma unroll
  for (int i = 0; i < kFew; ++i) out[i] = 0x7FFFFFFF;
  if (gone > 0) {
    unsigned long long low[kFew];
#pragma unroll
    for (int i = 0; i < kFew; ++i) low[i] = ~0ull;
#pragma unroll 4
    for (int i = threadIdx.x; i < s.n; i += kSelThreads) {
      unsigned long long k = (static_cast<unsigned long long>(slot_key(a, s, base, i)) << 32) | (0xFFFFFFFFu - i);
#pragma unroll
      for (int u = 0; u < kFew; ++u) {
        const unsigned long long x = min(low[u], k);
        k = max(low[u], k);
        low[u] = x;
      }
    }
    for (int r = 0; r < gone; ++r) {
      unsigned long long m = low[0];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = min(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (lane_id() == 0) s_min[r][warp_id()] = m;
      __syncthreads();
      m = s_min[r][lane_id()];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = min(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (low[0] == m) {                             // its owner goes on with its next one
#pragma unroll
        for (int u = 0; u + 1 < kFew; ++u) low[u] = low[u + 1];
        low[kFew - 1] = ~0ull;
      }
      // the slots that leave, in ascending order
      int x = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(m));
#pragma unroll
      for (int u = 0; u < kFew; ++u) {
        const int y = min(out[u], x);
        x = max(out[u], x);
        out[u] = y;
      }
    }
  }
  __syncthreads();   // every thread has read lens and seen
  if (threadIdx.x == 0) {
    a.lens[seg] = s.keep + s.m;
    a.seen[seg] = s.seen + s.m;
  }
  // warp u: slot keep + u; the f-th kept slot behind `keep` fills the f-th hole
  const int u = warp_id();
  if (u >= max(gone, s.m)) return;
  auto leaves = [&](int i) {
    bool y = false;
#pragma unroll
    for (int v = 0; v < kFew; ++v) y |= out[v] == i;
    return y;
  };
  int to = -1;
  if (u < gone && !leaves(s.keep + u)) {
    int f = 0;
    for (int v = 0; v < u; ++v) f += !leaves(s.keep + v);
#pragma unroll
    for (int v = 0; v < kFew; ++v)
      if (v == f) to = out[v];                       // holes are the lowest of the slots that leave
  }
  move_slots<1>(a, b, h, base, {s.keep + u}, {to}, {u < s.m ? u : -1}, s.seen);
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
  const int seg = blockIdx.y;
  const int4 hd = a.head[seg];
  const long long list = static_cast<long long>(seg) * a.most;
  move_rows(a, seg, hd.x, hd.y, hd.z, hd.w, a.holes + list, a.fills + list, blockIdx.x * kMoveWarps + warp_id(),
            gridDim.x * kMoveWarps);
}

}  // namespace

bool evict_in_one_launch(int most) { return most <= kFew; }

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  const int segs = a.B * a.H;
  if (evict_in_one_launch(a.most)) {
    evict_few_kernel<<<segs, kSelThreads, 0, st>>>(a);
    note_launch();
    return cudaGetLastError();
  }
  const bool kept = a.capacity <= kKeptSlots, here = a.most <= kHere && segs <= a.sms;
  const auto select = kept ? (here ? evict_select_kernel<true, true> : evict_select_kernel<true, false>)
                           : (here ? evict_select_kernel<false, true> : evict_select_kernel<false, false>);
  const size_t smem = kept ? static_cast<size_t>(a.capacity) * sizeof(uint32_t) : 0;
  cudaError_t e;
  if (kept && (e = ensure_smem(reinterpret_cast<const void*>(select), smem)) != cudaSuccess) return e;
  select<<<segs, kSelThreads, smem, st>>>(a);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess || here) return e;
  const int gx = std::min((a.most + kMoveWarps * kEach - 1) / (kMoveWarps * kEach), std::max(1, 16384 / segs));
  evict_move_kernel<<<dim3(gx, segs), kMoveThreads, 0, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace kvsel
