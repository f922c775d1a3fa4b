// Joins the pieces of items that several CTAs of attend_rows_kernel or attend_tile_kernel
// share.  Piece c of an item that starts in CTA x sits in slot 1 of CTA x (c = 0) or slot 0 of
// CTA x + c: unnormalised rows, their references (log2 units) and sums.  The factors of all
// pieces are formed first, so that the rows' loads do not wait for one another; pieces are
// added in a fixed order, so results repeat.
//
// Bound: latency (the pieces are in L2).  WPR warps work on a row: one where an item has few
// pieces, eight where it may have one per CTA.  (The same work by the CTA that finishes an
// item's last piece, without a second launch, took 38 us longer for 73 pieces of 7 rows.)
#include <algorithm>

#include "attend.cuh"

namespace kvsel {
namespace {

constexpr int kJoinWarps = 8;

template <int WPR>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(const AttnArgs a) {
  __shared__ float4 s_y[kJoinWarps][32];
  __shared__ float2 s_ml[kJoinWarps];
  const int4 rec = a.rec[blockIdx.x];
  if (rec.x < 0) return;
  const int seg = rec.x / a.rt, rt = rec.x - seg * a.rt;
  const int b = seg / a.H, h = seg - b * a.H;
  const int mr = a.new_lens ? __ldg(a.new_lens + b) : a.m;
  const int rows = min(a.tr, min(max(mr, 0), a.m) * a.G - rt * a.tr);
  const int warp = warp_id(), lane = lane_id(), part = warp % WPR, pieces = rec.y + 1;
  constexpr int kRowsPer = kJoinWarps / WPR;
  auto place = [&](int c, int r) { return (c == 0 ? 2ll * blockIdx.x + 1 : 2ll * (blockIdx.x + c)) * a.tr + r; };
  for (int r0 = blockIdx.y * kRowsPer; r0 < rows; r0 += gridDim.y * kRowsPer) {
    const int r = r0 + warp / WPR;
    float M = -INFINITY, L = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    // this warp's pieces are part, part + WPR, ...: 32 at a time, lane i the factor of the i-th
    for (int c0 = part; c0 < pieces && r < rows; c0 += 32 * WPR) {
      const int c = c0 + lane * WPR;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (c < pieces) ml = a.part_ml[place(c, r)];
      const int cnt = min(32, (pieces - c0 + WPR - 1) / WPR);
      float4 z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < cnt) z[i] = *reinterpret_cast<const float4*>(a.part_o + place(c0 + i * WPR, r) * kHeadDim + lane * 4);
      float m2 = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m2 = fmaxf(m2, __shfl_xor_sync(0xffffffffu, m2, o));
      m2 = fmaxf(m2, M);
      const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m2);
      float l = f * ml.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      const float old = M == -INFINITY ? 0.f : exp2f(M - m2);
      M = m2;
      L = L * old + l;
      y.x *= old;
      y.y *= old;
      y.z *= old;
      y.w *= old;
      for (int i0 = 0; i0 < cnt; i0 += 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i0 + i < cnt) {
            const float g = __shfl_sync(0xffffffffu, f, i0 + i);
            y.x += g * z[i].x;
            y.y += g * z[i].y;
            y.z += g * z[i].z;
            y.w += g * z[i].w;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i0 + 8 + i < cnt)
            z[i] = *reinterpret_cast<const float4*>(a.part_o + place(c0 + (i0 + 8 + i) * WPR, r) * kHeadDim + lane * 4);
      }
    }
    if (WPR > 1) {
      s_y[warp][lane] = y;
      if (lane == 0) s_ml[warp] = make_float2(M, L);
      __syncthreads();
      if (part == 0) {
        float m2 = M;
        for (int w = 1; w < WPR; ++w) m2 = fmaxf(m2, s_ml[warp + w].x);
        const float old = M == -INFINITY ? 0.f : exp2f(M - m2);
        L *= old;
        y = make_float4(y.x * old, y.y * old, y.z * old, y.w * old);
        for (int w = 1; w < WPR; ++w) {
          const float2 ml = s_ml[warp + w];
          const float g = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m2);
          const float4 z = s_y[warp + w][lane];
          L += g * ml.y;
          y.x += g * z.x;
          y.y += g * z.y;
          y.z += g * z.z;
          y.w += g * z.w;
        }
        M = m2;
      }
      __syncthreads();
    }
    if (r < rows && part == 0) {
      const int rr = rt * a.tr + r;
      const float inv = L > 0.f ? 1.f / L : 0.f;
      *reinterpret_cast<uint2*>(out_row(a, b, h, rr) + lane * 4) =
          make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
      if (lane == 0) write_lse(a, b, h, rr, M, L);
    }
  }
}

}  // namespace

cudaError_t launch_attend_join(const AttnArgs& a, int grid, cudaStream_t st) {
  const int rows = static_cast<int>(std::min<long long>(a.tr, static_cast<long long>(a.m) * a.G));
  // pieces per item: about grid / items
  if (static_cast<long long>(a.B) * a.H * a.rt * 8 < grid)
    attend_join_kernel<8><<<dim3(grid, std::min(rows, 64)), kJoinWarps * 32, 0, st>>>(a);
  else
    attend_join_kernel<1><<<dim3(grid, std::min((rows + 7) / 8, 16)), kJoinWarps * 32, 0, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace kvsel
