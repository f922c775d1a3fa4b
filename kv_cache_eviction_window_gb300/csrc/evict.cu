// Eviction by accumulated attention weight, with room made for new rows.  A segment keeps
// `keep` = min(rows, budget - new rows) of its rows: first the protected ones (first and most
// recent positions), then those with the largest accumulated weight, ties by the lower slot.
// Evicted slots below `keep` are holes; the kept rows at or behind `keep` fill them, in
// order; the new rows follow at `keep`.  So a row moves only when it has to, nothing that is
// read is written by another slot, and the new rows are the segment's last.
//
// evict_select_kernel: one CTA per segment ranks the slots (three-digit radix selection of
// the keep-th largest key, then an ordered scan for ties, holes and fills).
// evict_move_kernel: slot keep + i of a segment is handled by one half warp per side: its old
// row goes to its hole, then new row i takes the slot.  Bound by HBM: 8 B per slot read, 512 B
// per moved or new row read and written.
#include <algorithm>

#include "evict.cuh"

namespace kvsel {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveSlots = kMoveThreads / 32;        // slots per CTA of the second launch

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
  if (p < a.n_sink || p >= s.recent0) return 0xFFFFFFFFu;
  return weight_key(a.acc[base + i]);
}

// inclusive block-wide scan of three counters packed in 21-bit fields
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
  if (warp == 0) {
    unsigned long long y = s_w[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    s_w[lane] = y;
  }
  __syncthreads();
  if (warp > 0) v += s_w[warp - 1];
  total = s_w[31];
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ int s_hist[2048];
  __shared__ unsigned long long s_w[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int seg = blockIdx.x;
  const Seg s = seg_of(a, seg);
  const long long base = static_cast<long long>(seg) * a.capacity;
  __syncthreads();   // every thread has read lens and seen
  if (threadIdx.x == 0) {
    a.head[seg] = make_int4(s.keep, s.n, s.m, s.seen);
    a.lens[seg] = s.keep + s.m;
    a.seen[seg] = s.seen + s.m;
  }
  if (s.keep == s.n) return;

  // the keep-th largest key, by digits of 11, 11 and 10 bits from the top
  uint32_t prefix = 0, mask = 0;
  int need = s.keep;                                 // rank among the keys that share the prefix
  if (s.keep == 0) prefix = 0xFFFFFFFFu, mask = 0xFFFFFFFFu, need = 0;
  for (int pass = 0; pass < 3 && s.keep > 0; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bins = pass == 2 ? 1024 : 2048;
    for (int i = threadIdx.x; i < bins; i += kSelThreads) s_hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < s.n; i += kSelThreads) {
      const uint32_t k = slot_key(a, s, base, i);
      if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & (bins - 1)], 1);
    }
    __syncthreads();
    // thread t owns bins 2t and 2t + 1 counted from the top
    const int per = bins / kSelThreads;
    int own = 0;
    for (int u = 0; u < per; ++u) own += s_hist[bins - 1 - (threadIdx.x * per + u)];
    unsigned long long total;
    int before = static_cast<int>(block_scan(own, s_w, total)) - own;
    for (int u = 0; u < per; ++u) {
      const int bin = bins - 1 - (threadIdx.x * per + u), c = s_hist[bin];
      if (before < need && need <= before + c) {
        s_prefix = prefix | (static_cast<uint32_t>(bin) << shift);
        s_need = need - before;
      }
      before += c;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    mask |= static_cast<uint32_t>(bins - 1) << shift;
    __syncthreads();
  }
  // keys above `prefix` stay, and the first `need` slots whose key equals it
  int ties = 0, hole = 0, fill = 0;                  // before this block of slots
  for (int i0 = 0; i0 < s.n; i0 += kSelThreads) {
    const int i = i0 + threadIdx.x;
    const bool in = i < s.n;
    const uint32_t k = in ? slot_key(a, s, base, i) : 0u;
    const bool tie = in && k == prefix;
    unsigned long long total;
    const int tr = ties + static_cast<int>(block_scan(tie, s_w, total));   // ties up to and with i
    ties += static_cast<int>(total);
    const bool kept = in && (k > prefix || (tie && tr <= need));
    const bool is_hole = in && !kept && i < s.keep, is_fill = kept && i >= s.keep;
    const unsigned long long v = (static_cast<unsigned long long>(is_hole) << 32) | (is_fill ? 1u : 0u);
    const unsigned long long sc = block_scan(v, s_w, total);
    if (is_hole) a.holes[base + hole + static_cast<int>(sc >> 32) - 1] = i;
    if (in && i >= s.keep) a.fills[base + i - s.keep] = is_fill ? fill + static_cast<int>(sc & 0xFFFFFFFFu) - 1 : -1;
    hole += static_cast<int>(total >> 32);
    fill += static_cast<int>(total & 0xFFFFFFFFu);
  }
}

__device__ __forceinline__ long long slot_elem(const EvictArgs& a, int b, int h, int i) {
  if (!a.src.paged) return b * a.stride_req + h * a.stride_head + static_cast<long long>(i) * a.stride_tok;
  const int bs = a.src.block_size;
  const int pb = __ldg(a.src.block_table + static_cast<size_t>(b) * a.src.max_blocks + i / bs);
  if (pb < 0 || pb >= a.src.num_blocks) return -1;
  return ((static_cast<long long>(pb) * bs + (i % bs)) * a.H + h) * kHeadDim;
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
  const int seg = blockIdx.y, b = seg / a.H, h = seg - b * a.H;
  const int4 hd = a.head[seg];
  const int keep = hd.x, n = hd.y, m = hd.z, seen = hd.w;
  const long long base = static_cast<long long>(seg) * a.capacity;
  const int lane = lane_id(), side = lane >> 4, piece = lane & 15;
  uint16_t* cache = side ? a.v : a.k;
  const uint16_t* fresh = side ? a.v_new : a.k_new;
  const int slots = max(n - keep, m);
  for (int u = blockIdx.x * kMoveSlots + warp_id(); u < slots; u += gridDim.x * kMoveSlots) {
    const int i = keep + u;
    const long long e = slot_elem(a, b, h, i);
    const int rank = u < n - keep ? a.fills[base + u] : -1;
    int bad = e < 0;
    if (rank >= 0) {
      const int d = a.holes[base + rank];
      const long long ed = slot_elem(a, b, h, d);
      bad |= ed < 0;
      if (e >= 0 && ed >= 0)
        *(reinterpret_cast<uint4*>(cache + ed) + piece) = *(reinterpret_cast<const uint4*>(cache + e) + piece);
      if (lane == 0) {
        a.pos[base + d] = a.pos[base + i];
        a.acc[base + d] = a.acc[base + i];
      }
    }
    __syncwarp();
    if (u < m) {
      if (e >= 0)
        *(reinterpret_cast<uint4*>(cache + e) + piece) =
            __ldg(reinterpret_cast<const uint4*>(fresh + b * a.new_req + h * a.new_head +
                                                 static_cast<long long>(u) * a.new_tok) + piece);
      if (lane == 0) {
        a.pos[base + i] = seen + u;
        a.acc[base + i] = 0.f;
      }
    }
    if (bad && lane == 0) atomicOr(a.status, DEV_BAD_INDEX);
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  const int segs = a.B * a.H;
  evict_select_kernel<<<segs, kSelThreads, 0, st>>>(a);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int most = std::max(a.capacity - a.budget + a.m, a.m);
  if (most <= 0) return cudaSuccess;
  const int gx = std::min((most + kMoveSlots - 1) / kMoveSlots, 65535);
  evict_move_kernel<<<dim3(gx, segs), kMoveThreads, 0, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace kvsel
