// Rotary positions.  Pair i of a row (columns (i, i + rot/2) or (2i, 2i + 1)) turns by pos * f_i:
//   y1 = x1 c - x2 s,  y2 = x2 c + x1 s,   c, s = scale * cos, scale * sin
// The angle is pos * f_i / 2 pi mod 1 in 64-bit fixed point: the product's high bits fall off at whole turns, so
// it is as exact at position 2^30 as at 1 (in fp32 an angle of 10^6 is off by 0.06).  Sine and cosine are the
// approximate ones, off by 2^-21 of the pair's length; the result's rounding to bf16 is 2^-9 of the value.
//
// A thread turns eight pairs (32 bytes of a row) by the same sines for all heads of a token that fall
// to it; cached keys have a position each.  Bound: HBM, a row read and written.  Measured: 8192 tokens of 32 + 8 heads
// 27.8 us for 168 MB (24.7 at the copy rate); 32 segments of 13107 cached keys 42 us for 216 MB (31.9), of which the
// launch, the first places and the last stores are some 5; half the columns turned take as long.
#include <algorithm>

#include "step.cuh"

namespace kvsel {
namespace {

constexpr int kThreads = 256;

// The eight pairs 8 * unit .. that a thread looks after: turns per position as hi 2^-32 + lo 2^-64, lo signed.  (Read
// by its own index from the kernel's parameters in the inner loop, eight units of a warp in turn, they cost as much
// as the rows.)
struct Turns {
  int hi[8], lo[8];
};
constexpr int kUnit = 9;                             // entries between units: the banks of eight units differ
__device__ __forceinline__ void load_turns(const RopeTable& t, int2* s_turns, int unit, Turns& w) {
  if (threadIdx.x < 64) {
    const unsigned long long y = t.turns[threadIdx.x];
    s_turns[threadIdx.x / 8 * kUnit + threadIdx.x % 8] = make_int2(static_cast<int>((y + 0x80000000ull) >> 32), static_cast<int>(y));
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int2 y = s_turns[unit * kUnit + i];
    w.hi[i] = y.x;
    w.lo[i] = y.y;
  }
}
// Their sines and cosines at position pos.  Bits 32 to 63 of pos * turns are the angle in units of 2^-32 turns; the
// upper 23 of them make a number in [1, 2) (the sign's bit flipped: half a turn more), and so the angle in [-pi, pi], off by
// at most 2^-23 turns (little beside a bf16 value's 2^-8).
// (A conversion from integer would go to the unit of the sine and cosine, which is the busier one.)
__device__ __forceinline__ void sincos8(const Turns& w, int pos, float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x = static_cast<uint32_t>(pos) * static_cast<uint32_t>(w.hi[i]) + static_cast<uint32_t>(__mulhi(pos, w.lo[i]));
    const float y = fmaf(__uint_as_float((x >> 9) ^ 0x3FC00000u), 6.2831853f, -9.4247780f);
    c[i] = __cosf(y);
    s[i] = __sinf(y);
  }
}
__device__ __forceinline__ void scale8(float scale, float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] *= scale;
    s[i] *= scale;
  }
}
__device__ __forceinline__ void unpack8(const uint4& a, float (&x)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The two 16-byte pieces of a row that unit u (0..7) looks after: pairs u * 8 .. of the turned columns (units
// below rot / 16), or columns behind them.
__device__ __forceinline__ void places(const RopeTable& t, int u, int& a, int& b) {
  const int half = t.rot >> 4;                       // units that turn; pieces of half the turned columns
  if (u < half && !t.interleaved) {
    a = u;
    b = u + half;
  } else {
    a = 2 * u;
    b = a + 1;
  }
}
__device__ __forceinline__ void turn(const RopeTable& t, const float (&c)[8], const float (&s)[8], uint4& a, uint4& b) {
  float x[8], y[8], p[8], q[8];
  unpack8(a, x);
  unpack8(b, y);
  if (!t.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = x[i] * c[i] - y[i] * s[i];
      q[i] = y[i] * c[i] + x[i] * s[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[2 * i] = x[2 * i] * c[i] - x[2 * i + 1] * s[i];
      p[2 * i + 1] = x[2 * i + 1] * c[i] + x[2 * i] * s[i];
      q[2 * i] = y[2 * i] * c[i + 4] - y[2 * i + 1] * s[i + 4];
      q[2 * i + 1] = y[2 * i + 1] * c[i + 4] + y[2 * i] * s[i + 4];
    }
  }
  a = pack8(p);
  b = pack8(q);
}

// Rows in flight per thread: all loads of a batch come before its first use.
constexpr int kBatch = 4;

// A group of eight lanes per (token, share of the heads): grid (tokens, shares of q's heads, then of k's), `each` heads
// per group.
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const __grid_constant__ RopeArgs a, const int each, const int q_shares) {
  __shared__ int2 s_turns[8 * kUnit];
  Turns w;
  const int u = threadIdx.x & 7;
  load_turns(a.t, s_turns, u, w);
  const unsigned tok = blockIdx.x * (kThreads / 8) + (threadIdx.x >> 3);
  const int b = tok / static_cast<unsigned>(a.n_tok), i = tok - b * static_cast<unsigned>(a.n_tok);
  if (b >= a.B) return;
  if (a.new_lens && i >= __ldg(a.new_lens + b)) return;
  const bool turns = u < (a.t.rot >> 4);
  const int pos = __ldg(a.pos + b * a.pos_req + i);
  int pa, pb;
  places(a.t, u, pa, pb);
  const bool is_k = static_cast<int>(blockIdx.y) >= q_shares;
  const int h0 = (blockIdx.y - (is_k ? q_shares : 0)) * each, h1 = min(h0 + each, is_k ? a.k_heads : a.heads);
  const long long in = is_k ? a.k_head : a.q_head, out = is_k ? a.ko_head : a.qo_head;
  const uint16_t* src = (is_k ? a.k + b * a.k_req + i * a.k_tok : a.q + b * a.q_req + i * a.q_tok) + h0 * in;
  uint16_t* dst = (is_k ? a.k_out + b * a.ko_req + i * a.ko_tok : a.q_out + b * a.qo_req + i * a.qo_tok) + h0 * out;
  if (!turns && src == dst) return;                  // (in place: the strides are the same)
  float c[8], s[8];
  for (int h = h0; h < h1; h += kBatch) {
    uint4 x[kBatch], y[kBatch];
#pragma unroll
    for (int r = 0; r < kBatch; ++r)
      if (h + r < h1) {
        x[r] = reinterpret_cast<const uint4*>(src)[pa];
        y[r] = reinterpret_cast<const uint4*>(src)[pb];
        src += in;
      }
    if (turns && h == h0) {
      sincos8(w, pos, c, s);
      scale8(a.t.scale, c, s);
    }
#pragma unroll
    for (int r = 0; r < kBatch; ++r)
      if (h + r < h1) {
        if (turns) turn(a.t, c, s, x[r], y[r]);
        reinterpret_cast<uint4*>(dst)[pa] = x[r];
        reinterpret_cast<uint4*>(dst)[pb] = y[r];
        dst += out;
      }
  }
}

// grid (segment, CTAs that share its blocks of kRows rows), so that the heads of a page are read at about the same time:
// eight lanes per row.  A thread works out a row's places for the eight that turn it, a block of rows ahead.
// SCALED: the turned values have a factor
constexpr int kEach = 4, kRows = kThreads / 8 * kEach;
struct Row {
  long long src, dst;                                // elements; src < 0: nothing to do
  int pos;
};
template <bool SCALED>
__global__ void __launch_bounds__(kThreads, 3) rope_cache_kernel(const __grid_constant__ RopeCacheArgs a) {
  __shared__ int2 s_turns[8 * kUnit];
  __shared__ Row s_row[2][kRows];
  const int seg = blockIdx.x, b = seg / a.H, h = seg - b * a.H, u = threadIdx.x & 7;
  const int raw = __ldg(a.lens + (a.per_head ? seg : b)), n = min(max(raw, 0), a.max_len);
  bool bad = raw != n;
  const int step = gridDim.y * kRows;
  auto place = [&](long long j0) {
    Row x{-1, 0, 0};
    const long long jl = j0 + threadIdx.x;
    if (threadIdx.x < kRows && jl < n) {
      const int j = static_cast<int>(jl);
      x.pos = a.pos ? __ldg(a.pos + seg * a.pos_stride + j) : j;
      if (a.src.paged) {
        const int page = __ldg(a.src.block_table + static_cast<size_t>(b) * a.src.max_blocks + (j >> a.page_shift));
        if (page < 0 || page >= a.src.num_blocks)
          bad = true;
        else
          x.src = (((static_cast<long long>(page) << a.page_shift) + (j & (a.src.block_size - 1))) * a.H + h) * kHeadDim;
      } else {
        x.src = b * a.stride_req + h * a.stride_head + j * a.stride_tok;
      }
      x.dst = a.out ? b * a.o_req + h * a.o_head + j * a.o_tok : x.src;
    }
    return x;
  };
  long long j0 = static_cast<long long>(blockIdx.y) * kRows;
  if (threadIdx.x < kRows) s_row[0][threadIdx.x] = place(j0);
  Turns w;
  load_turns(a.t, s_turns, u, w);                    // (a barrier)
  const bool turns = u < (a.t.rot >> 4);
  int pa, pb;
  places(a.t, u, pa, pb);
  uint16_t* to = a.out ? a.out : a.k;
  for (int side = 0; j0 < n; j0 += step, side ^= 1) {
    const Row* rows = s_row[side] + (threadIdx.x >> 3);
    uint4 x[kEach], y[kEach];
    const bool mine = turns || a.out;
#pragma unroll
    for (int r = 0; r < kEach; ++r) {
      const long long e = rows[r * (kThreads / 8)].src;
      if (e < 0 || !mine) continue;
      x[r] = reinterpret_cast<const uint4*>(a.k + e)[pa];
      y[r] = reinterpret_cast<const uint4*>(a.k + e)[pb];
    }
    const Row next = place(j0 + step);
#pragma unroll
    for (int r = 0; r < kEach; ++r) {
      const Row& at = rows[r * (kThreads / 8)];
      if (at.src < 0 || !mine) continue;
      if (turns) {
        float c[8], s[8];
        sincos8(w, at.pos, c, s);
        if (SCALED) scale8(a.t.scale, c, s);
        turn(a.t, c, s, x[r], y[r]);
      }
      reinterpret_cast<uint4*>(to + at.dst)[pa] = x[r];
      reinterpret_cast<uint4*>(to + at.dst)[pb] = y[r];
    }
    if (threadIdx.x < kRows) s_row[side ^ 1][threadIdx.x] = next;
    __syncthreads();
  }
  if (bad && a.status) atomicOr(a.status, DEV_BAD_INDEX);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int sms, cudaStream_t st) {
  const long long toks = static_cast<long long>(a.B) * a.n_tok;
  const unsigned gx = static_cast<unsigned>((toks + kThreads / 8 - 1) / (kThreads / 8));
  // heads per group: as many as leave every SM some blocks
  int each = 8;
  auto shares = [&](int heads) { return (heads + each - 1) / each; };
  while (each > 1 && static_cast<long long>(gx) * (shares(a.heads) + shares(a.k_heads)) < 8 * sms) each /= 2;
  rope_kernel<<<dim3(gx, shares(a.heads) + shares(a.k_heads)), kThreads, 0, st>>>(a, each, shares(a.heads));
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_rope_cache(const RopeCacheArgs& a, int sms, cudaStream_t st) {
  constexpr int kCtas = 3;
  const int segs = a.B * a.H, blocks = (a.max_len + kRows - 1) / kRows;
  const auto kernel = a.t.scale != 1.f ? rope_cache_kernel<true> : rope_cache_kernel<false>;
  // CTAs for every SM to hold kCtas, or as many blocks as there are
  kernel<<<dim3(segs, std::min({blocks, 65535, std::max(1, kCtas * sms / segs)})), kThreads, 0, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace kvsel
