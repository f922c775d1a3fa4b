// Rotary positions.  Pair i of a row (columns (i, i + rot/2) or (2i, 2i + 1)) turns by pos * f_i:
//   y1 = x1 c - x2 s,  y2 = x2 c + x1 s,   c, s = scale * cos, scale * sin
// The angle is pos * f_i / 2 pi mod 1 in 64-bit fixed point: the product's high bits fall off at whole turns, so
// it is as exact at position 2^30 as at 1 (in fp32 an angle of 10^6 is off by 0.06).  Sine and cosine are the
// approximate ones, off by 2^-21 of the pair's length; the result's rounding to bf16 is 2^-9 of the value.
//
// A thread turns eight pairs (32 bytes of a row) by the same sines for all heads of a token that fall
// to it.  Bound: HBM, a row read and written.
#include <algorithm>

#include "step.cuh"

namespace kvsel {
namespace {

constexpr int kThreads = 256;

// sines and cosines of the eight pairs 8 * unit .. of position pos
__device__ __forceinline__ void sincos8(const RopeTable& t, int unit, int pos, float (&c)[8], float (&s)[8]) {
  const float scale = t.scale, back = t.back ? -scale : scale;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(pos)) * t.turns[unit * 8 + i];
    // signed turns in units of 2^-32
    const float x = static_cast<float>(static_cast<int>(turn >> 32)) * 1.4629180792671596e-9f;   // 2 pi 2^-32
    c[i] = __cosf(x) * scale;
    s[i] = __sinf(x) * back;
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

// A group of eight lanes per (token, share of the heads): grid (tokens, share), `each` heads per group.
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a, const int each) {
  const long long tok = static_cast<long long>(blockIdx.x) * (kThreads / 8) + (threadIdx.x >> 3);
  const int u = threadIdx.x & 7, b = static_cast<int>(tok / a.n_tok), i = static_cast<int>(tok - static_cast<long long>(b) * a.n_tok);
  if (b >= a.B) return;
  if (a.new_lens && i >= __ldg(a.new_lens + b)) return;
  const bool turns = u < (a.t.rot >> 4);
  float c[8], s[8];
  if (turns) sincos8(a.t, u, __ldg(a.pos + b * a.pos_req + i), c, s);
  int pa, pb;
  places(a.t, u, pa, pb);
  const int h0 = blockIdx.y * each, h1 = min(h0 + each, a.heads + a.k_heads);
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const bool is_k = h >= a.heads;
    const int hh = is_k ? h - a.heads : h;
    const uint16_t* src = is_k ? a.k + b * a.k_req + hh * a.k_head + i * a.k_tok : a.q + b * a.q_req + hh * a.q_head + i * a.q_tok;
    uint16_t* dst = is_k ? a.k_out + b * a.ko_req + hh * a.ko_head + i * a.ko_tok
                         : a.q_out + b * a.qo_req + hh * a.qo_head + i * a.qo_tok;
    if (!turns && src == dst) continue;
    uint4 x = reinterpret_cast<const uint4*>(src)[pa], y = reinterpret_cast<const uint4*>(src)[pb];
    if (turns) turn(a.t, c, s, x, y);
    reinterpret_cast<uint4*>(dst)[pa] = x;
    reinterpret_cast<uint4*>(dst)[pb] = y;
  }
}

// grid (rows, segment): eight lanes per row
__global__ void __launch_bounds__(kThreads) rope_cache_kernel(const __grid_constant__ RopeCacheArgs a) {
  const int seg = blockIdx.y, b = seg / a.H, h = seg - b * a.H, u = threadIdx.x & 7;
  const int raw = __ldg(a.lens + (a.per_head ? seg : b)), n = min(max(raw, 0), a.max_len);
  bool bad = raw != n;
  const bool turns = u < (a.t.rot >> 4);
  int pa, pb;
  places(a.t, u, pa, pb);
  for (int j = blockIdx.x * (kThreads / 8) + (threadIdx.x >> 3); j < n; j += gridDim.x * (kThreads / 8)) {
    long long e;
    if (a.src.paged) {
      const int page = __ldg(a.src.block_table + static_cast<size_t>(b) * a.src.max_blocks + (j >> a.page_shift));
      if (page < 0 || page >= a.src.num_blocks) {
        bad = true;
        continue;
      }
      e = (((static_cast<long long>(page) << a.page_shift) + (j & (a.src.block_size - 1))) * a.H + h) * kHeadDim;
    } else {
      e = b * a.stride_req + h * a.stride_head + j * a.stride_tok;
    }
    uint16_t* src = a.k + e;
    uint16_t* dst = a.out ? a.out + b * a.o_req + h * a.o_head + j * a.o_tok : src;
    if (!turns && src == dst) continue;
    uint4 x = reinterpret_cast<const uint4*>(src)[pa], y = reinterpret_cast<const uint4*>(src)[pb];
    if (turns) {
      float c[8], s[8];
      sincos8(a.t, u, a.pos ? __ldg(a.pos + seg * a.pos_stride + j) : j, c, s);
      turn(a.t, c, s, x, y);
    }
    reinterpret_cast<uint4*>(dst)[pa] = x;
    reinterpret_cast<uint4*>(dst)[pb] = y;
  }
  if (bad && a.status) atomicOr(a.status, DEV_BAD_INDEX);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int sms, cudaStream_t st) {
  const long long toks = static_cast<long long>(a.B) * a.n_tok;
  const unsigned gx = static_cast<unsigned>((toks + kThreads / 8 - 1) / (kThreads / 8));
  // heads per group: as many as leave every SM some blocks
  const int heads = a.heads + a.k_heads;
  int each = 8;
  while (each > 1 && static_cast<long long>(gx) * ((heads + each - 1) / each) < 8 * sms) each /= 2;
  rope_kernel<<<dim3(gx, (heads + each - 1) / each), kThreads, 0, st>>>(a, each);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_rope_cache(const RopeCacheArgs& a, int sms, cudaStream_t st) {
  const int segs = a.B * a.H;
  const int rows = (a.max_len + kThreads / 8 - 1) / (kThreads / 8);
  rope_cache_kernel<<<dim3(std::min(rows, std::max(1, 64 * sms / segs)), segs), kThreads, 0, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace kvsel
