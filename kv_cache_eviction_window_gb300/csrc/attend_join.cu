// Joins the pieces of items that several CTAs of attend_rows_kernel or attend_tile_kernel
// share.  Piece c of an item that starts in CTA x sits in slot 1 of CTA x (c = 0) or slot 0 of
// CTA x + c: unnormalised rows, their references (log2 units) and sums.  The pieces of a row
// are added in cache order within a warp, the warps in order, so results repeat.
#include <algorithm>

#include "attend.cuh"

namespace kvsel {
namespace {

constexpr int kJoinWarps = 4;

struct Piece {
  float M, L;
  float4 y;
};
__device__ __forceinline__ void add_piece(Piece& p, float M, float L, const float4& z) {
  const float M2 = fmaxf(p.M, M);
  if (M2 == -INFINITY) return;
  const float f = exp2f(p.M - M2), g = exp2f(M - M2);
  p.M = M2;
  p.L = p.L * f + L * g;
  p.y.x = p.y.x * f + z.x * g;
  p.y.y = p.y.y * f + z.y * g;
  p.y.z = p.y.z * f + z.z * g;
  p.y.w = p.y.w * f + z.w * g;
}

// WPR warps per row.  One warp per row where an item has few pieces (many items); four where it
// may have one per CTA.
template <int WPR>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(const AttnArgs a) {
  __shared__ float4 s_y[kJoinWarps][32];
  __shared__ float2 s_ml[kJoinWarps];
  let_next_start();
  after_previous();
  const int4 rec = a.rec[blockIdx.x];
  if (rec.x < 0) return;
  const int seg = rec.x / a.rt, rt = rec.x - seg * a.rt;
  const int b = seg / a.H, h = seg - b * a.H;
  const int mr = a.new_lens ? __ldg(a.new_lens + b) : a.m;
  const int rows = min(a.tr, min(max(mr, 0), a.m) * a.G - rt * a.tr);
  const int warp = warp_id(), lane = lane_id();
  constexpr int kRowsPer = kJoinWarps / WPR;
  for (int r0 = blockIdx.y * kRowsPer; r0 < rows; r0 += gridDim.y * kRowsPer) {
    const int r = r0 + warp / WPR;
    Piece p{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (r < rows) {
#pragma unroll 4
      for (int c = warp % WPR; c <= rec.y; c += WPR) {
        const long long at = (c == 0 ? 2ll * blockIdx.x + 1 : 2ll * (blockIdx.x + c)) * a.tr + r;
        const float2 ml = a.part_ml[at];
        add_piece(p, ml.x, ml.y, *reinterpret_cast<const float4*>(a.part_o + at * kHeadDim + lane * 4));
      }
    }
    if (WPR > 1) {
      s_y[warp][lane] = p.y;
      if (lane == 0) s_ml[warp] = make_float2(p.M, p.L);
      __syncthreads();
      if (warp == 0)
        for (int w = 1; w < WPR; ++w) add_piece(p, s_ml[w].x, s_ml[w].y, s_y[w][lane]);
      __syncthreads();
    }
    if (r < rows && warp % WPR == 0) {
      const int rr = rt * a.tr + r;
      const float inv = p.L > 0.f ? 1.f / p.L : 0.f;
      *reinterpret_cast<uint2*>(out_row(a, b, h, rr) + lane * 4) =
          make_uint2(pack_bf16(p.y.x * inv, p.y.y * inv), pack_bf16(p.y.z * inv, p.y.w * inv));
      if (lane == 0) write_lse(a, b, h, rr, p.M, p.L);
    }
  }
}

}  // namespace

cudaError_t launch_attend_join(const AttnArgs& a, int grid, cudaStream_t st) {
  const int rows = static_cast<int>(std::min<long long>(a.tr, static_cast<long long>(a.m) * a.G));
  // pieces per item: about grid / items
  if (static_cast<long long>(a.B) * a.H * a.rt * 8 < grid)
    return launch_after(attend_join_kernel<4>, dim3(grid, std::min(rows, 64)), kJoinWarps * 32, 0, st, a);
  return launch_after(attend_join_kernel<1>, dim3(grid, std::min((rows + 3) / 4, 16)), kJoinWarps * 32, 0, st, a);
}

}  // namespace kvsel
