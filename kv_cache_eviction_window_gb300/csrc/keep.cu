// Kept rows left in their cache: of a segment with `count` kept positions idx (ascending), those below count
// stay where they are, and the j-th kept position at or behind count moves to the j-th hole below it.
// With k0 kept positions below count, the moves are idx[k0 + j] -> hole j; idx[i] - i holes lie before idx[i], so
// hole j is j + i for the first i with idx[i] - i > j (a binary search).  Rows that move lie at or behind
// count, holes below it: nothing that is read is written.
// Bound: HBM, 512 B per moved row read and written, and 12 B per kept row.
#include <algorithm>

#include "step.cuh"

namespace kvsel {
namespace {

constexpr int kThreads = 256;
constexpr int kHoles = 64;                           // of a CTA at a time
constexpr int kPer = kHoles * 32 / kThreads;         // 16-byte pieces of a thread

__device__ __forceinline__ long long row_of(const KeepArgs& a, int b, int h, int i) {
  if (!a.src.paged) return b * a.stride_req + h * a.stride_head + static_cast<long long>(i) * a.stride_tok;
  const int bs = a.src.block_size;
  const int pb = __ldg(a.src.block_table + static_cast<size_t>(b) * a.src.max_blocks + i / bs);
  if (pb < 0 || pb >= a.src.num_blocks) return -1;
  return ((static_cast<long long>(pb) * bs + (i % bs)) * a.rq.H + h) * kHeadDim;
}

__global__ void __launch_bounds__(kThreads) keep_kernel(const KeepArgs a) {
  __shared__ long long s_of[kHoles], s_to[kHoles];
  const int seg = blockIdx.y, b = seg / a.rq.H, h = seg - b * a.rq.H, tid = threadIdx.x;
  const int n = a.rq.n[b], count = __ldg(a.counts + seg);
  const long long off = __ldg(a.offsets + seg);
  const bool fits = count >= 0 && count <= n && off >= 0 && off <= a.n_kept - count;
  if (blockIdx.x == 0 && tid == 0) {
    a.lens[seg] = fits ? count : 0;
    if (a.seen) a.seen[seg] = n;
    if (!fits && a.status) atomicOr(a.status, DEV_BAD_INDEX);
  }
  if (!fits) return;
  const int32_t* idx = a.idx + off;
  // kept positions below count
  int k0 = 0;
  for (int lo = 0, hi = count;;) {
    if (lo >= hi) {
      k0 = lo;
      break;
    }
    const int mid = (lo + hi) >> 1;
    if (__ldg(idx + mid) < count)
      lo = mid + 1;
    else
      hi = mid;
  }
  int32_t* pos = a.pos + seg * a.capacity;
  float* acc = a.acc ? a.acc + seg * a.capacity : nullptr;
  const float* scores = a.scores ? a.scores + a.rq.soff[b] + static_cast<long long>(h) * n : nullptr;
  bool bad = false;
  for (int i = blockIdx.x * kThreads + tid; i < count; i += gridDim.x * kThreads) {
    const int x = __ldg(idx + i);
    if (x < 0 || x >= n || (i > 0 && x <= __ldg(idx + i - 1))) bad = true;
    if (i < k0 && x >= 0 && x < count) {
      pos[x] = x;
      if (acc) acc[x] = scores ? __ldg(scores + x) : 0.f;
    }
  }
  for (int j0 = blockIdx.x * kHoles; j0 < count - k0; j0 += gridDim.x * kHoles) {
    if (tid < kHoles) {
      long long of = -1, to = -1;
      const int j = j0 + tid;
      if (j < count - k0) {
        int lo = 0, hi = k0;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (__ldg(idx + mid) - mid > j)
            hi = mid;
          else
            lo = mid + 1;
        }
        const int hole = j + lo, fill = __ldg(idx + k0 + j);
        if (hole < count && fill >= count && fill < n) {
          of = row_of(a, b, h, fill);
          to = row_of(a, b, h, hole);
          if (of < 0 || to < 0) {
            bad = true;
            of = to = -1;
          }
          pos[hole] = fill;
          if (acc) acc[hole] = scores ? __ldg(scores + fill) : 0.f;
        } else {
          bad = true;
        }
      }
      s_of[tid] = of;
      s_to[tid] = to;
    }
    __syncthreads();
    uint4 y[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int pc = u * kThreads + tid, row = pc >> 5, side = (pc >> 4) & 1, piece = pc & 15;
      const long long e = s_of[row];
      y[u] = make_uint4(0u, 0u, 0u, 0u);
      if (e >= 0) y[u] = reinterpret_cast<const uint4*>((side ? a.v : a.k) + e)[piece];
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int pc = u * kThreads + tid, row = pc >> 5, side = (pc >> 4) & 1, piece = pc & 15;
      const long long e = s_to[row];
      if (e >= 0) reinterpret_cast<uint4*>((side ? a.v : a.k) + e)[piece] = y[u];
    }
    __syncthreads();
  }
  if (bad && a.status) atomicOr(a.status, DEV_BAD_INDEX);
}

}  // namespace

cudaError_t launch_keep(const KeepArgs& a, int max_count, cudaStream_t st) {
  const int segs = a.rq.B * a.rq.H, gx = std::max(1, std::min((max_count + kHoles - 1) / kHoles, std::max(1, 16384 / segs)));
  keep_kernel<<<dim3(gx, segs), kThreads, 0, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace kvsel
