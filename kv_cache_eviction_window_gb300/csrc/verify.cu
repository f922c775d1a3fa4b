// Trees of drafted tokens: their masks, and which of their nodes are accepted.
//
// tree_masks_kernel: a thread per node follows the parents.  Ancestors come in descending order, so a word
// of the mask is written when the walk has left it.  Bound: latency, a step of the walk from shared
// memory each.
//
// verify_kernel: a cluster of CTAs per request, each of which looks after a share of the vocabulary; all
// of them walk down the tree alike.  The rest of a node c after k rejections is r = max(p_c - A q_c, 0),
// A the masses before each of them (q is positive: taking it off twice or as a sum is the same), so only a
// sum over the vocabulary is needed where a sibling follows, and one for the last draw.  Probabilities
// count as integers in units of 2^-46 there: sums are exact and do not depend on their order, 2^18 of them
// fit 64 bits, and the draw is the comparison of integers.
// Bound: latency; a row of p and q is read for each rejection that a sibling follows and for the last draw.
#include <cooperative_groups.h>

#include "../../include/kvsel.h"
#include "step.cuh"

namespace cgx = cooperative_groups;

namespace kvsel {
namespace {

__global__ void __launch_bounds__(1024) tree_masks_kernel(const int32_t* __restrict__ parents,
                                                          const int32_t* __restrict__ new_lens,
                                                          const int32_t* __restrict__ first, int n_new, uint32_t* tree,
                                                          int32_t* pos) {
  __shared__ int s_par[KVSEL_MAX_TREE];
  const int b = blockIdx.x, t = threadIdx.x, words = (n_new + 31) / 32;
  const int m = new_lens ? min(max(__ldg(new_lens + b), 0), n_new) : n_new;
  const long long row = static_cast<long long>(b) * n_new;
  if (t < m) s_par[t] = parents[row + t];
  __syncthreads();
  if (t >= m) return;
  uint32_t* mask = tree + (row + t) * words;
  int at = t, w = words - 1, depth = 0;
  uint32_t bits = 0;
  while (true) {
    for (; w > at >> 5; --w) {
      mask[w] = bits;
      bits = 0;
    }
    bits |= 1u << (at & 31);
    const int p = s_par[at];
    if (p < 0 || p >= at) break;
    at = p;
    ++depth;
  }
  for (; w >= 0; --w) {
    mask[w] = bits;
    bits = 0;
  }
  if (pos) pos[row + t] = __ldg(first + b) + depth;
}

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kUnitBits = 46;                        // probabilities in units of 2^-46

template <class T>
__device__ __forceinline__ float value_of(T x);
template <>
__device__ __forceinline__ float value_of<float>(float x) { return x; }
template <>
__device__ __forceinline__ float value_of<uint16_t>(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// a probability in [0, 1] (NaN: 0), and in units of 2^-46, rounded
__device__ __forceinline__ float prob(float x) { return fminf(fmaxf(x, 0.f), 1.f); }
__device__ __forceinline__ unsigned long long units(float x) {
  return __float2ull_rn(prob(x) * 70368744177664.f);
}
// max(p - A q, 0) in units; A in units, below 2^56
__device__ __forceinline__ unsigned long long rest_units(float p, float q, unsigned long long A) {
  const unsigned long long P = units(p), Q = units(q);
  const unsigned long long AQ = __umul64hi(A << 8, Q << 10);
  return P > AQ ? P - AQ : 0;
}
// larger value, larger key; ties: the lower token; NaN below all
__device__ __forceinline__ unsigned long long arg_key(float x, int i) {
  uint32_t k = 0;
  if (x == x) {
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  }
  return (static_cast<unsigned long long>(k) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i));
}

// Vectors of 16 bytes of a row: elements [i0, i1) of it, by the threads of a group; f(i, x...) for each.
template <class T, class F>
__device__ __forceinline__ void each_of(const T* p, int i0, int i1, int at, int step, F f) {
  constexpr int N = 16 / sizeof(T);
  // the first element on a 16-byte boundary
  const int lead = static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(p + i0) & 15)) & 15) / sizeof(T));
  const int v0 = min(i1, i0 + lead), nv = (i1 - v0) / N, v1 = v0 + nv * N;
  if (at < v0 - i0) f(i0 + at, p[i0 + at]);
  if (at < i1 - v1) f(v1 + at, p[v1 + at]);
#pragma unroll 2
  for (int u = at; u < nv; u += step) {
    const uint4 raw = __ldg(reinterpret_cast<const uint4*>(p + v0) + u);
    T x[N];
    memcpy(x, &raw, 16);
#pragma unroll
    for (int c = 0; c < N; ++c) f(v0 + u * N + c, x[c]);
  }
}
template <class T, class F>
__device__ __forceinline__ void each_of(const T* p, const T* q, int i0, int i1, int at, int step, F f) {
  constexpr int N = 16 / sizeof(T);
  const int lead = static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(p + i0) & 15)) & 15) / sizeof(T));
  const int v0 = min(i1, i0 + lead), nv = (i1 - v0) / N, v1 = v0 + nv * N;
  const bool alike = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0;
  if (at < v0 - i0) f(i0 + at, p[i0 + at], q[i0 + at]);
  if (at < i1 - v1) f(v1 + at, p[v1 + at], q[v1 + at]);
  if (alike) {
#pragma unroll 2
    for (int u = at; u < nv; u += step) {
      const uint4 rp = __ldg(reinterpret_cast<const uint4*>(p + v0) + u), rq = __ldg(reinterpret_cast<const uint4*>(q + v0) + u);
      T x[N], y[N];
      memcpy(x, &rp, 16);
      memcpy(y, &rq, 16);
#pragma unroll
      for (int c = 0; c < N; ++c) f(v0 + u * N + c, x[c], y[c]);
    }
  } else {
    for (int i = v0 + at; i < v1; i += step) f(i, p[i], q[i]);
  }
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

enum Want : int { kMass, kDraw, kLargest, kDone };
struct Shared {
  int par[KVSEL_MAX_TREE], tok[KVSEL_MAX_TREE];
  float p[KVSEL_MAX_TREE], q[KVSEL_MAX_TREE], u[KVSEL_MAX_TREE];
  int out[KVSEL_MAX_TREE];                           // POINT: tokens rejected at the present node
  unsigned long long warp[kWarps];                   // sums of the warps' shares
  unsigned long long part[2][kWarps + 1];            // of this CTA, for the cluster: total, then by warp
  int cur, nout, want;
  unsigned long long A;
};

template <class T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a) {
  __shared__ Shared s;
  cgx::cluster_group cl = cgx::this_cluster();
  const int cs = static_cast<int>(cl.num_blocks()), rank = static_cast<int>(cl.block_rank());
  const int b = blockIdx.x / cs, tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  const T* target = static_cast<const T*>(a.target) + b * a.stride_req;
  const T* draft = a.draft ? static_cast<const T*>(a.draft) + b * a.stride_req : nullptr;
  const long long row = static_cast<long long>(b) * a.m;
  const int raw = a.new_lens ? __ldg(a.new_lens + b) : a.m, m = min(max(raw, 0), a.m);
  bool bad = raw != m;
  for (int t = tid; t < m; t += kThreads) {
    int p = t ? a.parents[row + t] : -1;
    const int x = a.tokens[row + t];
    if (t && (p < 0 || p >= t)) {
      bad = true;
      p = -1;
    }
    float pv = 0.f, qv = 1.f;
    if (t && (x < 0 || x >= a.vocab)) {
      bad = true;
    } else if (t && p >= 0 && a.mode != KVSEL_VERIFY_GREEDY) {
      pv = prob(value_of<T>(target[p * a.stride_node + x]));
      if (draft) qv = prob(value_of<T>(draft[p * a.stride_node + x]));
    }
    s.par[t] = p;
    s.tok[t] = x;
    s.p[t] = pv;
    s.q[t] = qv;
    s.u[t] = a.u ? a.u[row + t] : 0.f;
  }
  for (int t = tid + (rank ? a.m : 0); t < a.m; t += kThreads) a.path[row + t] = t ? -1 : (m ? 0 : -1);
  if (bad && rank == 0) atomicOr(a.status, DEV_BAD_INDEX);
  if (m == 0) {                                      // the whole cluster
    if (rank == 0 && tid == 0) {
      a.counts[b] = 0;
      a.next[b] = -1;
    }
    return;
  }
  __syncthreads();

  // this CTA's share of the vocabulary, and this warp's of that
  const int per_cta = (a.vocab + cs - 1) / cs, per_warp = ((per_cta + kWarps - 1) / kWarps + 31) & ~31;
  const int c0 = min(a.vocab, rank * per_cta), c1 = min(a.vocab, c0 + per_cta);
  const int w0 = min(c1, c0 + warp * per_warp), w1 = min(c1, w0 + per_warp);
  // Of warp 0, the same in every lane: the node, the last node that was looked at, accepted ones, and the
  // mass of the rest (units, and as a number), what A q_c has been taken off
  int cur = 0, last = 0, count = 1;
  unsigned long long A = 0, Z = 1ull << kUnitBits;
  int best = -1, nout = 0;
  int phase = 0;
  bool stale = a.mode == KVSEL_VERIFY_GREEDY;        // the largest value of the node is not known
  bool lean = false;                                 // Z is not known
  while (true) {
    if (warp == 0) {
      int want = kDone;
      while (true) {
        if (stale) {
          want = kLargest;
          break;
        }
        // the next child
        int child = -1;
        for (int t0 = (last + 1) & ~31; t0 < m && child < 0; t0 += 32) {
          const int t = t0 + lane;
          const unsigned hit = __ballot_sync(0xffffffffu, t > last && t < m && s.par[t] == cur);
          if (hit) child = t0 + __ffs(hit) - 1;
        }
        if (child < 0) {
          want = a.mode == KVSEL_VERIFY_GREEDY ? kDone : kDraw;
          break;
        }
        if (lean) {
          want = kMass;
          break;
        }
        last = child;
        const int x = s.tok[child];
        bool take;
        if (a.mode == KVSEL_VERIFY_GREEDY) {
          take = x == best;
        } else {
          const double unit = 1.0 / 70368744177664.0, z = static_cast<double>(Z) * unit;
          double r = s.p[child];
          if (a.mode == KVSEL_VERIFY_SAMPLED) {
            r = fmax(r - static_cast<double>(A) * unit * s.q[child], 0.0);
          } else {
            bool out = false;
            for (int i = lane; i < nout; i += 32) out |= s.out[i] == x;
            if (__any_sync(0xffffffffu, out)) r = 0.0;
          }
          take = static_cast<double>(s.u[child]) * s.q[child] * z < r && x >= 0 && x < a.vocab;
        }
        if (take) {
          cur = child;
          if (lane == 0 && rank == 0) a.path[row + count] = child;
          ++count;
          A = 0;
          Z = 1ull << kUnitBits;
          nout = 0;
          stale = a.mode == KVSEL_VERIFY_GREEDY;
        } else if (x < 0 || x >= a.vocab) {
          // takes nothing from the rest
        } else if (a.mode == KVSEL_VERIFY_SAMPLED) {
          A += Z;
          lean = true;
        } else if (a.mode == KVSEL_VERIFY_POINT) {
          bool out = false;
          for (int i = lane; i < nout; i += 32) out |= s.out[i] == x;
          if (!__any_sync(0xffffffffu, out)) {
            const unsigned long long gone = units(s.p[child]);
            Z = Z > gone ? Z - gone : 0;
            if (lane == 0) s.out[nout] = x;
            ++nout;
            __syncwarp();
          }
        }
      }
      if (lane == 0) {
        s.want = want;
        s.cur = cur;
        s.A = A;
        s.nout = nout;
      }
      lean = false;                                  // (the pass to come finds it)
    }
    __syncthreads();
    const int want = s.want;
    if (want == kDone) break;
    const T* p = target + s.cur * a.stride_node;
    const T* q = draft + s.cur * a.stride_node;
    const unsigned long long off = s.A;
    unsigned long long v = 0;
    if (want == kLargest) {
      each_of(p, w0, w1, lane, 32, [&](int i, T x) { v = max(v, arg_key(value_of<T>(x), i)); });
      v = warp_max(v);
    } else if (off) {
      each_of(p, q, w0, w1, lane, 32, [&](int, T x, T y) { v += rest_units(value_of<T>(x), value_of<T>(y), off); });
      v = warp_sum(v);
    } else {
      each_of(p, w0, w1, lane, 32, [&](int, T x) { v += units(value_of<T>(x)); });
      v = warp_sum(v);
      // POINT: what was rejected here has no weight any more
      for (int i = 0; i < s.nout; ++i)
        if (s.out[i] >= w0 && s.out[i] < w1) v -= units(value_of<T>(p[s.out[i]]));
    }
    unsigned long long* part = s.part[phase];
    if (lane == 0) part[1 + warp] = v;
    __syncthreads();
    if (warp == 0) {
      unsigned long long y = lane < kWarps ? part[1 + lane] : 0;
      y = want == kLargest ? warp_max(y) : warp_sum(y);
      if (lane == 0) part[0] = y;
    }
    cl.sync();
    unsigned long long mine = 0, all = 0, before = 0;
    for (int c = 0; c < cs; ++c) {
      const unsigned long long y = *cl.map_shared_rank(part, c);
      if (c == rank) mine = y;
      if (c < rank) before += y;
      all = want == kLargest ? max(all, y) : all + y;
    }
    phase ^= 1;
    if (want == kLargest) {
      best = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(all));
      stale = false;
      continue;
    }
    if (want == kMass) {
      Z = all;
      continue;
    }
    // the last draw: the smallest token whose sum passes u_0 of all
    if (all == 0 && (off || s.nout)) {               // nothing is left of the rest: from p_c itself
      __syncthreads();
      A = 0;
      nout = 0;
      continue;
    }
    if (all == 0) {
      best = -1;
      break;
    }
    const float u = fminf(fmaxf(s.u[0], 0.f), 0.99999994f);
    const unsigned long long goal = __umul64hi(all, __float2ull_rz(u * 18446744073709551616.f));
    if (before <= goal && goal < before + mine) {
      // in this CTA: the warp's share, then its elements 32 at a time
      if (warp == 0) {
        unsigned long long sum = before;
        int w = 0;
        while (w < kWarps - 1 && sum + part[1 + w] <= goal) sum += part[1 + w++];
        const int e0 = min(c1, c0 + w * per_warp), e1 = min(c1, e0 + per_warp);
        for (int i0 = e0; i0 < e1; i0 += 32) {
          const int i = i0 + lane;
          unsigned long long y = 0;
          if (i < e1) {
            y = off ? rest_units(value_of<T>(p[i]), value_of<T>(q[i]), off) : units(value_of<T>(p[i]));
            for (int k = 0; k < s.nout; ++k)
              if (s.out[k] == i) y = 0;
          }
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
          }
          const unsigned hit = __ballot_sync(0xffffffffu, sum + y > goal);
          if (hit) {
            if (lane == 0) a.next[b] = i0 + __ffs(hit) - 1;
            break;
          }
          sum += __shfl_sync(0xffffffffu, y, 31);
        }
      }
    }
    best = -2;                                       // written
    break;
  }
  if (rank == 0 && tid == 0) {
    a.counts[b] = count;
    if (best != -2) a.next[b] = best;
  }
  cl.sync();                                         // its shared memory has been read
}

}  // namespace

cudaError_t launch_tree_masks(const int32_t* parents, const int32_t* new_lens, const int32_t* first, int batch, int n_new,
                              uint32_t* tree, int32_t* pos, cudaStream_t st) {
  tree_masks_kernel<<<batch, (n_new + 31) / 32 * 32, 0, st>>>(parents, new_lens, first, n_new, tree, pos);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_verify(const VerifyArgs& a, int batch, bool bf16, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(batch * kCluster, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = bf16 ? cudaLaunchKernelEx(&cfg, verify_kernel<uint16_t>, a) : cudaLaunchKernelEx(&cfg, verify_kernel<float>, a);
  note_launch();
  return e;
}

}  // namespace kvsel
