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
// count as integers in units of 2^-45 there: sums are exact and do not depend on their order, 2^18 of them
// fit 64 bits, and the draw is the comparison of integers.
// Bound: latency, of loads and of instructions: code that runs once per launch is fetched from L2, so loops are kept
// small.  One request of one node, GREEDY, 131072 tokens, takes 4.6 us, each round over the vocabulary more 2.1: the row's
// loads 1, the numbers to all CTAs of the cluster (which a barrier there counts; a barrier of the cluster took 0.35 longer)
// and the walk.  A round is made for each rejection that a sibling follows, unless the sibling passes with the mass before,
// and one for the last draw; GREEDY makes one per accepted node.  Measured on one GB300: 32 chains of five drafted tokens
// over 50257 tokens, fp32, 10.0 us; 8 trees of 64 nodes over 131072, bf16, 13 to 28 us by what is rejected; 32 requests of
// 26 nodes, GREEDY, 14.6 us; 512 requests of one node, bf16, 87 us for 134 MB (the sums' instructions).  (512 threads per
// CTA: a tenth to a quarter less for hundreds of requests, 1 to 5 us more for small vocabularies.)
#include <cooperative_groups.h>

#include "../../include/kvsel.h"
#include "ptx.cuh"
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

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr long long kLandCycles = 1 << 17;           // after a wait that ran out: far longer than a remote store takes
constexpr unsigned long long kNapCycles = 1 << 16;   // shorter limits are not left to a wait of the hardware's own
constexpr int kUnitBits = 45;                        // probabilities in units of 2^-45
constexpr unsigned long long kOne = 1ull << kUnitBits;

template <class T>
__device__ __forceinline__ float value_of(T x);
template <>
__device__ __forceinline__ float value_of<float>(float x) { return x; }
template <>
__device__ __forceinline__ float value_of<uint16_t>(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// a probability in [0, 1] (NaN: 0)
__device__ __forceinline__ float prob(float x) { return __saturatef(x); }
// x in [0, 1] as hi 2^-22 + lo 2^-45, rounded to that: adding 2^23 leaves an integer in the last bits of a number.
// (A conversion to 64 bits takes a quarter of a cycle per SM: 25 us for 64 rows of 131072.)
struct Parts {
  int hi, lo;
};
__device__ __forceinline__ Parts parts(float x) {
  const float y = fmaf(x, 4194304.f, 8388608.f);
  const float r = fmaf(x, 4194304.f, 8388608.f - y);           // exact, in [-1/2, 1/2]
  return Parts{__float_as_int(y) - 0x4B000000, __float_as_int(fmaf(r, 8388608.f, 12582912.f)) - 0x4B400000};
}
__device__ __forceinline__ long long whole(long long hi, int lo) { return hi * 8388608 + lo; }
__device__ __forceinline__ unsigned long long units(float x) {
  const Parts a = parts(prob(x));
  return whole(a.hi, a.lo);
}
// max(p - A q, 0) in units.  A is the sum of up to 1023 masses of at most 17/16 (rows may sum to a sixteenth more than 1),
// 1087 in all: below 2^56 units, and Q is 2^45 at most.
__device__ __forceinline__ unsigned long long rest_units(float p, float q, unsigned long long A) {
  static_assert((KVSEL_MAX_TREE - 1) * 17ull / 16 + 1 < 1ull << (56 - kUnitBits), "A << 8 fits 64 bits");
  const unsigned long long P = units(p), Q = units(q);
  const unsigned long long AQ = A == kOne ? Q : __umul64hi(A << 8, Q << 11);
  return P > AQ ? P - AQ : 0;
}

// The 16-byte vectors in elements [i0, i1) of a row (or, with q, of two at the same places): nv from v0 on, which end at v1.
// Rows that do not share a boundary have none.
constexpr int kAhead = 4;
template <class T>
struct Span {
  static constexpr int N = 16 / sizeof(T), kChunk = 32 * kAhead * N;
  int i0, i1, v0, nv, v1;
  bool apart;
  // the last draw looks for a chunk first
  __device__ __forceinline__ bool wide() const { return nv > 32 * kAhead; }
  __device__ __forceinline__ Span(const T* p, const T* q, int from, int to) : i0(from), i1(to) {
    apart = q && ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15);
    const int lead = static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(p + i0) & 15)) & 15) / sizeof(T));
    v0 = apart ? i1 : min(i1, i0 + lead);
    nv = (i1 - v0) / N;
    v1 = v0 + nv * N;
  }
};
// f(x, y) for each element (y = 0 without q), by the lanes of a warp: kChunk elements at a time, a vector of each lane after
// another and all loaded before the first is used, with chunk() after them; then what lies before the vectors by the lower
// lanes and what lies behind by the upper ones, with edge() after one element of each.
// Loops are not unrolled where that only saves moves: code that runs once or twice costs more to fetch.
template <class T, class F, class G, class E>
__device__ __forceinline__ void each_of(const Span<T>& x, const T* p, const T* q, F f, G chunk, E edge) {
  constexpr int N = Span<T>::N;
  const int lane = lane_id();
  int i = x.apart || lane < 16 ? x.i0 + lane : x.v1 + lane - 16;
  const int end = x.apart || lane >= 16 ? x.i1 : x.v0;
  T ex = T(), ey = T();
  auto next = [&] {
    if (i >= end) return;
    ex = p[i];
    if (q) ey = q[i];
  };
  next();
  for (int c0 = 0; c0 < x.nv; c0 += 32 * kAhead) {
    const int u0 = c0 + lane;
    uint4 rp[kAhead], rq[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      rq[k] = make_uint4(0u, 0u, 0u, 0u);
      if (u0 + 32 * k < x.nv) {
        rp[k] = __ldg(reinterpret_cast<const uint4*>(p + x.v0) + u0 + 32 * k);
        if (q) rq[k] = __ldg(reinterpret_cast<const uint4*>(q + x.v0) + u0 + 32 * k);
      }
    }
#pragma unroll 1
    for (int u = u0; u < min(x.nv, u0 + 32 * kAhead); u += 32) {
      T a[N], b[N];
      memcpy(a, &rp[0], 16);
      memcpy(b, &rq[0], 16);
#pragma unroll
      for (int c = 0; c < N; ++c) f(a[c], b[c]);
#pragma unroll
      for (int k = 0; k + 1 < kAhead; ++k) {
        rp[k] = rp[k + 1];
        rq[k] = rq[k + 1];
      }
    }
    chunk();
  }
#pragma unroll 1
  while (i < end) {
    f(ex, ey);
    edge();
    i += 32;
    next();
  }
  __syncwarp();
}

// The largest value of elements [i0, i1) of a row and the lowest place that has it, by the lanes of a warp (each
// its own; at = -1: none but NaN): vectors first, then the place in the vector that has it.
__device__ __forceinline__ float vector_max(const uint4& v, float) {
  return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
}
__device__ __forceinline__ float vector_max(const uint4& v, uint16_t) {
  __nv_bfloat162 x[4];
  memcpy(x, &v, 16);
  const float2 y = __bfloat1622float2(__hmax2(__hmax2(x[0], x[1]), __hmax2(x[2], x[3])));
  return fmaxf(y.x, y.y);
}
template <class T>
__device__ __forceinline__ void largest_of(const T* p, int i0, int i1, float& top, int& at) {
  constexpr int N = 16 / sizeof(T), kLoads = 8;
  const int lane = lane_id();
  const int lead = static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(p + i0) & 15)) & 15) / sizeof(T));
  const int v0 = min(i1, i0 + lead), nv = (i1 - v0) / N, v1 = v0 + nv * N;
  top = -INFINITY;
  at = -1;
  auto look = [&](float y, int i) {
    if (y > top || (at < 0 && y == y)) {
      top = y;
      at = i;
    }
  };
  // what lies before and behind the vectors: at most one element per lane
  float edge[2] = {__int_as_float(0x7FC00000), __int_as_float(0x7FC00000)};
  if (lane < v0 - i0) edge[0] = value_of<T>(p[i0 + lane]);
  if (lane < i1 - v1) edge[1] = value_of<T>(p[v1 + lane]);
  for (int u0 = lane; u0 < nv; u0 += 32 * kLoads) {
    uint4 r[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
      if (u0 + 32 * k < nv) r[k] = __ldg(reinterpret_cast<const uint4*>(p + v0) + u0 + 32 * k);
    if (u0 == lane) look(edge[0], i0 + lane);
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
      if (u0 + 32 * k < nv) look(vector_max(r[k], T()), v0 + (u0 + 32 * k) * N);
  }
  if (lane >= nv) look(edge[0], i0 + lane);          // (no vector of this lane's)
  if (at >= v0) {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(p + at));
    T x[N];
    memcpy(x, &r, 16);
    int c = 0;
#pragma unroll
    for (int i = N - 1; i >= 0; --i)
      if (value_of<T>(x[i]) == top) c = i;
    at += c;
  }
  look(edge[1], v1 + lane);
}

// sums and maxima over a warp by its integer reductions: 27 bits at a time (a sum of 32 fits 32 bits), or a key's
// high word and then, of those that have it, the low word
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
  const uint32_t a = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v) & 0x7FFFFFFu);
  const uint32_t b = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> 27) & 0x7FFFFFFu);
  const uint32_t c = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> 54));
  return a + (static_cast<unsigned long long>(b) << 27) + (static_cast<unsigned long long>(c) << 54);
}
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return static_cast<unsigned long long>(hi) << 32 | lo;
}

// inclusive
__device__ __forceinline__ unsigned long long warp_scan(unsigned long long v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long z = __shfl_up_sync(0xffffffffu, v, o);
    if (lane_id() >= o) v += z;
  }
  return v;
}
// elements e .. of a row, as many as 16 bytes hold; zeros outside [i0, i1)
template <class T>
__device__ __forceinline__ void some_of(const T* p, int e, int i0, int i1, T (&x)[16 / sizeof(T)]) {
  constexpr int N = 16 / sizeof(T);
  if (e >= i0 && e + N <= i1 && !(reinterpret_cast<uintptr_t>(p + e) & 15)) {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(p + e));
    memcpy(x, &r, 16);
    return;
  }
#pragma unroll
  for (int c = 0; c < N; ++c) x[c] = e + c >= i0 && e + c < i1 ? p[e + c] : T();
}

// One number to a place of the cluster's CTA `rank`, counted by the barrier there.
__device__ __forceinline__ void send(unsigned long long* to, unsigned long long v, uint64_t* bar, int rank) {
  uint32_t at, there;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(to)), "r"(rank));
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem_u32(bar)), "r"(rank));
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u64 [%0], %1, [%2];" ::"r"(at), "l"(v), "r"(there) : "memory");
}
// Whether a phase of the barrier, and with it what others have sent, has come: at once (NOW), or after some time that the
// hardware waits itself.
template <bool NOW>
__device__ __forceinline__ bool came(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  if (NOW)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  return ok;
}

// which of a span's chunks token x is in: 0 before the vectors, then theirs, then what lies behind
template <class T>
__device__ __forceinline__ int chunk_of(const Span<T>& s, int x) {
  return x < s.v0 ? 0 : (min(x, s.v1) - s.v0 + (x < s.v1 ? 0 : Span<T>::kChunk - 1)) / Span<T>::kChunk + 1;
}

enum Want : int { kMass, kDraw, kLargest, kDone };
// of a node: its token is one, its first test (A = 0, Z = 1) passes, an earlier sibling has its token (POINT)
enum Flag : int { kValid = 1, kPasses = 2, kAgain = 4 };
constexpr int kChunks = KVSEL_MAX_VOCAB / kWarps / Span<float>::kChunk + 2;
struct Shared {
  int par[KVSEL_MAX_TREE], tok[KVSEL_MAX_TREE], flag[KVSEL_MAX_TREE];
  float p[KVSEL_MAX_TREE], q[KVSEL_MAX_TREE], u[KVSEL_MAX_TREE];
  int out[KVSEL_MAX_TREE], nout;                     // POINT: nodes whose tokens have no weight in the draw
  // what every warp of the cluster found in its share of the vocabulary, written by that warp to all CTAs
  unsigned long long part[2][kMaxCluster * kWarps];
  // the last draw: what every warp found before its vectors, in each chunk of them, and behind
  unsigned long long chunk[kWarps][kChunks];
  uint64_t came[2];                                  // bytes of `part` that have come
  int cur, want, lost;
  unsigned long long A;
};

template <class T, int MODE>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const VerifyArgs a) {
  __shared__ Shared s;
  cgx::cluster_group cl = cgx::this_cluster();
  const int cs = static_cast<int>(cl.num_blocks()), rank = static_cast<int>(cl.block_rank());
  const int b = blockIdx.x / cs, tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  const T* target = static_cast<const T*>(a.target) + b * a.stride_req;
  const T* draft = a.draft ? static_cast<const T*>(a.draft) + b * a.stride_req : nullptr;
  const long long row = static_cast<long long>(b) * a.m;
  constexpr bool greedy = MODE == KVSEL_VERIFY_GREEDY, point = MODE == KVSEL_VERIFY_POINT, sampled = MODE == KVSEL_VERIFY_SAMPLED;
  const int raw = a.new_lens ? __ldg(a.new_lens + b) : a.m, m = min(max(raw, 0), a.m);
  bool bad = raw != m;
  if (tid == 0) s.lost = 0;
  for (int t = tid; t < m; t += kThreads) {
    int p = t ? a.parents[row + t] : -1;
    const int x = a.tokens[row + t];
    const float u = a.u ? a.u[row + t] : 0.f;
    float pv = 0.f, qv = 1.f;
    int flag = 0;
    if (t && (p < 0 || p >= t)) {
      bad = true;
      p = -1;
    }
    if (t && (x < 0 || x >= a.vocab)) {
      bad = true;
    } else if (t && p >= 0) {
      flag = kValid;
      if (!greedy) {
        pv = prob(value_of<T>(target[p * a.stride_node + x]));
        if (sampled) qv = prob(value_of<T>(draft[p * a.stride_node + x]));
        if (static_cast<double>(u) * qv < static_cast<double>(pv)) flag |= kPasses;
      }
    }
    s.par[t] = p;
    s.tok[t] = x;
    s.flag[t] = flag;
    s.p[t] = pv;
    s.q[t] = qv;
    s.u[t] = u;
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
  if (point) {
    for (int t = tid; t < m; t += kThreads)
      for (int c = 1; c < t; ++c)
        if (s.par[c] == s.par[t] && s.tok[c] == s.tok[t]) {
          s.flag[t] |= kAgain;
          break;
        }
    __syncthreads();
  }
  if (cs > 1) {
    if (tid == 0) {
      mbar_init(&s.came[0], 1);
      mbar_init(&s.came[1], 1);
      fence_mbar_init();
    }
    cl.sync();                                       // every CTA of the cluster runs: its shared memory may be written
  }

  // this warp's share of the vocabulary
  const int per_warp = ((a.vocab + cs * kWarps - 1) / (cs * kWarps) + 7) & ~7;
  const int mine = rank * kWarps + warp;
  const int w0 = min(a.vocab, mine * per_warp), w1 = min(a.vocab, w0 + per_warp);
  // Of warp 0, the same in every lane: the node, the last child that was looked at, accepted nodes, and the
  // mass of the rest, which A q has been taken off
  int cur = 0, last = 0, count = 1;
  unsigned long long A = 0, Z = kOne;
  int best = -1;
  int pass = 0;
  int held = 0, my_par = -2, my_flag = 0, my_tok = 0;
  auto hold = [&](int t0) {
    held = t0;
    const int t = t0 + lane;
    my_par = t < m ? s.par[t] : -2;
    my_flag = t < m ? s.flag[t] : 0;
    my_tok = t < m ? s.tok[t] : 0;
  };
  if (warp == 0) hold(0);
  bool stale = greedy;                               // the largest value of the node is not known
  bool lean = false;                                 // Z is not known
  while (true) {
    if (warp == 0) {
      int want = kDone;
      const bool lost = s.lost;
      while (!lost) {
        if (stale) {
          want = kLargest;
          break;
        }
        // the next child: children come after their parents and are looked at in order, so the 32 nodes that the
        // lanes hold only move on
        unsigned hit = __ballot_sync(0xffffffffu, my_par == cur && held + lane > last);
        while (!hit && held + 32 < m) {
          hold(held + 32);
          hit = __ballot_sync(0xffffffffu, my_par == cur && held + lane > last);
        }
        const int child = hit ? held + __ffs(hit) - 1 : -1;
        if (child < 0) {
          want = greedy ? kDone : kDraw;
          int n = 0;
          if (point)          // all its children were rejected
            for (int t0 = 0; t0 < m; t0 += 32) {
              const int t = t0 + lane;
              const bool out = t < m && s.par[t] == cur && (s.flag[t] & (kValid | kAgain)) == kValid;
              const unsigned hit = __ballot_sync(0xffffffffu, out);
              if (out) s.out[n + __popc(hit & ((1u << lane) - 1u))] = t;
              n += __popc(hit);
            }
          if (lane == 0) s.nout = n;
          break;
        }
        const int flag = __shfl_sync(0xffffffffu, my_flag, child - held);
        if (!(flag & kValid)) {                      // takes nothing from the rest
          last = child;
          continue;
        }
        bool take;
        if (greedy) {
          take = __shfl_sync(0xffffffffu, my_tok, child - held) == best;
        } else if (A == 0 && Z == kOne) {
          take = flag & kPasses;
        } else {
          const double unit = 1.0 / 35184372088832.0;
          double r = s.p[child];
          if (sampled)
            r = fmax(r - static_cast<double>(A) * unit * s.q[child], 0.0);
          else if (flag & kAgain)
            r = 0.0;
          // the mass that is not known yet is at most the one before; the first, taken as 1, is what p sums to
          const double z = lean && A == kOne ? 1.0625 : static_cast<double>(Z) * unit;
          take = static_cast<double>(s.u[child]) * s.q[child] * z < r;
        }
        // (what passes with a larger mass is accepted, without a sum)
        if (lean && !take) {
          want = kMass;
          break;
        }
        last = child;
        lean = false;
        if (take) {
          cur = child;
          if (lane == 0 && rank == 0) a.path[row + count] = child;
          ++count;
          A = 0;
          Z = kOne;
          stale = greedy;
        } else if (sampled) {
          A += Z;
          lean = true;
        } else if (point && !(flag & kAgain)) {
          const unsigned long long gone = units(s.p[child]);
          Z = Z > gone ? Z - gone : 0;
        }
      }
      if (lane == 0) {
        s.want = want;
        s.cur = cur;
        s.A = A;
      }
      lean = false;                                  // (the pass to come finds it)
    }
    __syncthreads();
    const int want = s.want;
    if (want == kDone) break;
    const int node = s.cur;
    const T* p = target + node * a.stride_node;
    const T* q = draft + node * a.stride_node;
    const unsigned long long off = s.A;
    bool first = true, lost = false;                 // the draw is from the rest, not from p itself; a wait ran out
    unsigned long long v, all, before;
    while (true) {
      v = 0;
      unsigned long long sum = 0;
      int hi = 0, lo = 0, chunks = 0;
      const bool rest = sampled && off && first;
      const Span<T> span(p, rest ? q : nullptr, w0, w1);
      const bool wide = want == kDraw && span.wide();
      auto flush = [&] {
        v += static_cast<unsigned long long>(whole(hi, lo));
        hi = lo = 0;
      };
      auto chunk = [&] {
        flush();
        if (!wide) return;
        const unsigned long long y = warp_sum(v);
        if (lane == 0) s.chunk[warp][++chunks] = y;
        sum += y;
        v = 0;
      };
      if (greedy) {
        float top;
        int at;
        largest_of(p, w0, w1, top, at);
        // larger value, larger key; ties: the lower token; NaN below all
        if (at >= 0) {
          const uint32_t k = __float_as_uint(top == 0.f ? 0.f : top);
          v = static_cast<unsigned long long>((k & 0x80000000u) ? ~k : (k | 0x80000000u)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(at));
        }
        v = warp_max(v);
      } else if (rest && off != kOne) {
        each_of(span, p, q, [&](T x, T y) { v += rest_units(value_of<T>(x), value_of<T>(y), off); }, chunk, [] {});
      } else {
        // p itself, or after the first rejection p - q where that is positive
        each_of(span, p, rest ? q : nullptr, [&](T x, T y) {
          const float xp = prob(value_of<T>(x)), xq = prob(value_of<T>(y));
          const Parts P = parts(xp), Q = parts(xq);
          hi += xp > xq ? P.hi - Q.hi : 0;
          lo += xp > xq ? P.lo - Q.lo : 0;
        }, chunk, flush);
      }
      if (!greedy) {
        // POINT: what was rejected here has no weight any more
        unsigned long long gone = 0;
        if (wide) {
          const unsigned long long lead = warp_sum(span.apart || lane < 16 ? v : 0), tail = warp_sum(span.apart || lane < 16 ? 0 : v);
          if (lane == 0) {
            s.chunk[warp][0] = lead;
            s.chunk[warp][(span.nv + 32 * kAhead - 1) / (32 * kAhead) + 1] = tail;
          }
          __syncwarp();
        }
        if (point && first)
          for (int k = lane; k < s.nout; k += 32) {
            const int x = s.tok[s.out[k]];
            if (x < w0 || x >= w1) continue;
            const unsigned long long y = units(s.p[s.out[k]]);
            gone += y;
            if (wide) atomicAdd(&s.chunk[warp][chunk_of(span, x)], 0 - y);
          }
        v = sum + warp_sum(v - gone);
      }
      // All CTAs get all numbers.  A warp sends those of the next pass when this CTA has got all of this one, so those of
      // the pass after that, which go to the same places, find these read.
      const int side = pass & 1;
      if (cs == 1) {
        if (lane == 0) s.part[side][warp] = v;
        __syncthreads();
      } else {
        if (tid == 0) mbar_arrive_expect_tx(&s.came[side], cs * kWarps * 8);
        if (lane < cs) send(&s.part[side][mine], v, &s.came[side], lane);
        if (want == kDraw || warp == 0) {
          const uint32_t parity = pass >> 1 & 1;
          const bool brief = a.wait_cycles < kNapCycles;
          auto here = [&] { return brief ? came<true>(&s.came[side], parity) : came<false>(&s.came[side], parity); };
          bool have = here();
          const long long t0 = clock64();
          while (!have && !*static_cast<volatile int*>(&s.lost)) {
            if (static_cast<unsigned long long>(clock64() - t0) > a.wait_cycles) {
              s.lost = 1;
              atomicOr(a.status, DEV_TIMEOUT_PIPE);
            } else {
              have = here();
            }
          }
          lost = __any_sync(0xffffffffu, !have);
        }
      }
      const unsigned long long* part = s.part[side];
      ++pass;
      all = before = 0;
      if (want == kDraw || warp == 0) {
#pragma unroll
        for (int k = 0; k < kMaxCluster * kWarps / 32; ++k) {
          const int i = lane + 32 * k;
          if (i >= cs * kWarps) continue;
          const unsigned long long y = part[i];
          all = greedy ? max(all, y) : all + y;
          if (i < mine) before += y;
        }
        all = greedy ? warp_max(all) : warp_sum(all);
        if (!greedy && want == kDraw) before = warp_sum(before);
      }
      // (a warp that has not got all numbers makes no further pass: CTAs that have may be gone)
      if (want != kDraw || all || !first || lost) break;
      first = false;                                 // nothing is left of the rest
    }
    if (greedy) {
      best = all ? static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(all)) : 0;
      stale = false;
      continue;
    }
    if (want == kMass) {
      Z = all;
      continue;
    }
    // the last draw: the smallest token whose sum passes u_0 of all
    best = all ? -2 : -1;                            // -2: written here
    const float u = fminf(fmaxf(s.u[0], 0.f), 0.99999994f);
    const unsigned long long goal = __umul64hi(all, __float2ull_rz(u * 18446744073709551616.f));
    if (!lost && all && before <= goal && goal < before + v) {
      // In this warp's share: the chunk that passes the goal, in which each lane sums a run of tokens, and the run that
      // passes it is looked at again by all lanes.  (One warp that went over its whole share took 120 us of 150 for 512
      // requests of 131072 tokens.)
      constexpr int N = 16 / sizeof(T);
      const bool rest = sampled && off && first;
      const Span<T> span(p, rest ? q : nullptr, w0, w1);
      unsigned long long at = before;
      int f0 = w0, f1 = w1;
      if (span.wide()) {
        const int chunks = (span.nv + 32 * kAhead - 1) / (32 * kAhead) + 2;
        int here = 0;
#pragma unroll 1
        for (int c0 = 0; c0 < chunks; c0 += 32) {
          const unsigned long long y = c0 + lane < chunks ? s.chunk[warp][c0 + lane] : 0, sum = at + warp_scan(y);
          const unsigned hit = __ballot_sync(0xffffffffu, sum > goal);
          here = c0 + (hit ? __ffs(hit) - 1 : 0);
          at = __shfl_sync(0xffffffffu, hit ? sum - y : sum, hit ? here - c0 : 31);
          if (hit) break;
        }
        f0 = here == 0 ? w0 : here == chunks - 1 ? span.v1 : span.v0 + (here - 1) * Span<T>::kChunk;
        f1 = here == 0 ? span.v0 : here == chunks - 1 ? w1 : min(span.v1, span.v0 + here * Span<T>::kChunk);
      }
      const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(p + f0) & 15) / sizeof(T));
      const int per = ((f1 - f0 + lead + 31) / 32 + N - 1) / N * N, run = f0 - lead + lane * per;
      const int l0 = max(run, f0), l1 = min(run + per, f1);
      unsigned long long y = 0;
#pragma unroll 1
      for (int e = run; e < l1; e += N) {
        T x[N], z[N] = {};
        some_of(p, e, l0, l1, x);
        if (rest) some_of(q, e, l0, l1, z);
#pragma unroll
        for (int c = 0; c < N; ++c) y += rest_units(value_of<T>(x[c]), value_of<T>(z[c]), off);
      }
      for (int k = 0; point && first && k < s.nout; ++k) {
        const int t = s.out[k], x = s.tok[t];
        if (x >= l0 && x < l1) y -= units(s.p[t]);
      }
      at += warp_scan(y) - y;
      unsigned hit = __ballot_sync(0xffffffffu, at + y > goal);
      const int who = __ffs(hit) - 1, r0 = __shfl_sync(0xffffffffu, l0, who), r1 = __shfl_sync(0xffffffffu, l1, who);
      at = __shfl_sync(0xffffffffu, at, who);
#pragma unroll 1
      for (int i0 = r0; i0 < r1; i0 += 32) {
        const int i = i0 + lane;
        const float x = i < r1 ? value_of<T>(p[i]) : 0.f, z = rest && i < r1 ? value_of<T>(q[i]) : 0.f;
        unsigned long long w = rest_units(x, z, off);
        for (int k = 0; point && first && k < s.nout; ++k)
          if (s.tok[s.out[k]] == i) w = 0;
        const unsigned long long sum = at + warp_scan(w);
        hit = __ballot_sync(0xffffffffu, sum > goal);
        if (hit) {
          if (lane == 0) a.next[b] = i0 + __ffs(hit) - 1;
          break;
        }
        at = __shfl_sync(0xffffffffu, sum, 31);
      }
    }
    break;
  }
  // A wait ran out: what was sent from here lands, and no CTA ends before all that go on sending have given up, too.
  if (cs > 1 && __any_sync(0xffffffffu, *static_cast<volatile int*>(&s.lost))) {
    const long long t0 = clock64();
    while (clock64() - t0 < kLandCycles) {
    }
    cl.sync();
  }
  if (rank == 0 && tid == 0) {
    a.counts[b] = count;
    if (best != -2) a.next[b] = best;
  }
}

}  // namespace

cudaError_t launch_tree_masks(const int32_t* parents, const int32_t* new_lens, const int32_t* first, int batch, int n_new,
                              uint32_t* tree, int32_t* pos, cudaStream_t st) {
  tree_masks_kernel<<<batch, (n_new + 31) / 32 * 32, 0, st>>>(parents, new_lens, first, n_new, tree, pos);
  note_launch();
  return cudaGetLastError();
}

namespace {

template <class T>
auto kernel_of(int mode) {
  return mode == KVSEL_VERIFY_SAMPLED ? verify_kernel<T, KVSEL_VERIFY_SAMPLED>
         : mode == KVSEL_VERIFY_POINT ? verify_kernel<T, KVSEL_VERIFY_POINT>
                                      : verify_kernel<T, KVSEL_VERIFY_GREEDY>;
}

// CTAs of a request: no more than three per SM over all requests, with at least a thousand tokens each
int cluster_of(int batch, int vocab, int sms) {
  int c = 1;
  while (c < kMaxCluster && 2 * c * batch <= 3 * sms && 2 * c * 1024 <= vocab) c *= 2;
  return c;
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int batch, bool bf16, int sms, cudaStream_t st) {
  const auto kernel = bf16 ? kernel_of<uint16_t>(a.mode) : kernel_of<float>(a.mode);
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kernel), 1);   // (allows clusters of 16)
  if (e != cudaSuccess) return e;
  const int cluster = cluster_of(batch, a.vocab, sms);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(batch * cluster, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  note_launch();
  return e;
}

}  // namespace kvsel
