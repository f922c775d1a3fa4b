// Kept rows left in their cache: of a segment with `count` kept positions idx (ascending), those below count
// stay where they are, and the j-th kept position at or behind count moves to the j-th hole below it.
// With k0 kept positions below count, the moves are idx[k0 + j] -> hole j, and a row p that is not kept is hole
// p minus the kept rows before it: a search for a block's first row, then a count over its rows.  Rows
// that move lie at or behind count, holes below it: nothing that is read is written.
// Bound: HBM, 512 B per moved row read and written, and 12 B per kept row.  Measured: 13107 of 32768 rows of 32 segments in
// pages of 16 49 us for 263 MB (38.7 at the copy rate); rows of 64 to 512 per CTA, two to eight rows per warp at a time and
// other numbers of CTAs per SM were no faster.  (A search for every hole: 92 us.)
#include <algorithm>

#include "step.cuh"

namespace kvsel {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRows = 4;                             // of a warp at a time: all loads before the first store

__device__ __forceinline__ long long row_of(const KeepArgs& a, int b, int h, int i) {
  if (!a.src.paged) return b * a.stride_req + h * a.stride_head + static_cast<long long>(i) * a.stride_tok;
  const int bs = a.src.block_size;
  const int pb = __ldg(a.src.block_table + static_cast<size_t>(b) * a.src.max_blocks + i / bs);
  if (pb < 0 || pb >= a.src.num_blocks) return -1;
  return ((static_cast<long long>(pb) * bs + (i % bs)) * a.rq.H + h) * kHeadDim;
}

// entries of idx[0, count) below x, by a warp: 32 probes at a time
__device__ __forceinline__ int below(const int32_t* idx, int count, int x) {
  int lo = 0, hi = count;                            // the answer is in [lo, hi]
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32, at = lo + (lane_id() + 1) * step - 1;   // the last of this lane's share
    const unsigned less = __ballot_sync(0xffffffffu, at < hi && __ldg(idx + at) < x);
    lo += __popc(less) * step;
    hi = min(hi, lo + step);
  }
  const int at = lo + lane_id();
  return lo + __popc(__ballot_sync(0xffffffffu, at < hi && __ldg(idx + at) < x));
}

// grid (segment, blocks of 256 of the first `count` rows), so that the heads of a page are read at about the same
// time: a thread per row finds out whether it is kept, a
// warp moves a row at a time
__global__ void __launch_bounds__(kThreads) keep_kernel(const KeepArgs a) {
  __shared__ int s_kept[kThreads], s_n[kWarps], s_at[2];
  __shared__ long long s_of[kThreads], s_to[kThreads];
  const int seg = blockIdx.x, b = seg / a.rq.H, h = seg - b * a.rq.H, tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  const int n = a.rq.n[b], count = __ldg(a.counts + seg);
  const long long off = __ldg(a.offsets + seg);
  const bool fits = count >= 0 && count <= n && off >= 0 && off <= a.n_kept - count;
  if (blockIdx.y == 0 && tid == 0) {
    a.lens[seg] = fits ? count : 0;
    if (a.seen) a.seen[seg] = n;
    if (!fits && a.status) atomicOr(a.status, DEV_BAD_INDEX);
  }
  if (!fits) return;
  const int32_t* idx = a.idx + off;
  int32_t* pos = a.pos + seg * a.capacity;
  float* acc = a.acc ? a.acc + seg * a.capacity : nullptr;
  const float* scores = a.scores ? a.scores + a.rq.soff[b] + static_cast<long long>(h) * n : nullptr;
  bool bad = false;
  for (int p0 = blockIdx.y * kThreads; p0 < count; p0 += gridDim.y * kThreads) {
    // kept rows before this block's, and below count
    if (warp < 2) {
      const int y = below(idx, count, warp ? count : p0);
      if (lane == 0) s_at[warp] = y;
    }
    s_kept[tid] = 0;
    __syncthreads();
    const int i0 = s_at[0], k0 = s_at[1];
    // this block's share of the check of the list
    const int ci = p0 + tid;
    if (ci < count) {
      const int x = __ldg(idx + ci);
      if (x < 0 || x >= n || (ci > 0 && x <= __ldg(idx + ci - 1))) bad = true;
    }
    if (i0 + tid < k0) {
      const int x = __ldg(idx + i0 + tid) - p0;
      if (x >= 0 && x < kThreads) s_kept[x] = 1;
    }
    __syncthreads();
    const int p = p0 + tid;
    const bool kept = s_kept[tid];
    const unsigned mask = __ballot_sync(0xffffffffu, kept);
    if (lane == 0) s_n[warp] = __popc(mask);
    __syncthreads();
    int before = i0 + __popc(mask & ((1u << lane) - 1u)), total = 0;   // kept rows before row p
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_n[w];
      total += s_n[w];
    }
    const int holes = min(kThreads, count - p0) - total;
    if (p < count) {
      int row = p;
      if (!kept) {
        // hole number p - before of the segment, and p - p0 - (before - i0) of this block
        const int j = k0 + p - before;
        row = j >= 0 && j < count ? __ldg(idx + j) : -1;
        long long of = -1, to = -1;
        if (row >= count && row < n) {
          of = row_of(a, b, h, row);
          to = row_of(a, b, h, p);
          if (of < 0 || to < 0) {
            bad = true;
            of = to = -1;
          }
        } else {
          bad = true;
          row = -1;
        }
        s_of[p - p0 - (before - i0)] = of;
        s_to[p - p0 - (before - i0)] = to;
      }
      pos[p] = row;
      if (acc) acc[p] = scores && row >= 0 ? __ldg(scores + row) : 0.f;
    }
    __syncthreads();
    const uint4* from = reinterpret_cast<const uint4*>(lane >> 4 ? a.v : a.k) + (lane & 15);
    uint4* into = reinterpret_cast<uint4*>(lane >> 4 ? a.v : a.k) + (lane & 15);
    for (int r0 = warp * kRows; r0 < holes; r0 += kWarps * kRows) {
      uint4 y[kRows];
      long long to[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        to[u] = -1;
        if (r0 + u < holes) {
          const long long of = s_of[r0 + u];
          to[u] = s_to[r0 + u];
          if (of >= 0) y[u] = from[of / 8];
        }
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u)
        if (to[u] >= 0) into[to[u] / 8] = y[u];
    }
    __syncthreads();
  }
  if (bad && a.status) atomicOr(a.status, DEV_BAD_INDEX);
}

}  // namespace

cudaError_t launch_keep(const KeepArgs& a, int max_count, cudaStream_t st) {
  const int blocks = (max_count + kThreads - 1) / kThreads;
  keep_kernel<<<dim3(a.rq.B * a.rq.H, std::max(1, std::min(blocks, 65535))), kThreads, 0, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace kvsel
