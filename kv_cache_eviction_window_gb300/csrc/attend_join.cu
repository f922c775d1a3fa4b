// Joins the pieces of items that several CTAs of attend_rows_kernel or attend_tile_kernel
// share.  Piece c of an item that starts in CTA x sits in slot 1 of CTA x (c = 0) or slot 0 of
// CTA x + c: unnormalised rows, their references (log2 units) and sums.  The loads of a row's
// pieces do not wait for one another; pieces are added in a fixed order, so results repeat.
//
// Bound: latency (the pieces are in L2).  Few items (by_item): a CTA per row, eight warps over its
// pieces, of which there may be one per CTA of the grid.  Many items, of two or three pieces: a
// warp per two rows (one row at a time took 2 to 3 us longer), five CTAs for each CTA before; those
// whose number starts no shared item end at once.
// (Joining in the CTA that finishes an item's last piece, without a second launch, took 38 us
// longer for 73 pieces of 7 rows.)
#include <algorithm>

#include "attend.cuh"

namespace kvsel {
namespace {

constexpr int kJoinWarps = 8;

struct Joined {
  float M, L;
  float4 y;
};
__device__ __forceinline__ Joined nothing() { return Joined{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)}; }
// N more pieces: references and sums ml (-inf, 0 where there is none) and rows z
template <int N>
__device__ __forceinline__ void add_pieces(Joined& p, const float2* ml, const float4* z) {
  float m2 = p.M;
#pragma unroll
  for (int i = 0; i < N; ++i) m2 = fmaxf(m2, ml[i].x);
  const float old = p.M == -INFINITY ? 0.f : exp2f(p.M - m2);
  p.M = m2;
  p.L *= old;
  p.y = make_float4(p.y.x * old, p.y.y * old, p.y.z * old, p.y.w * old);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float f = ml[i].x == -INFINITY ? 0.f : exp2f(ml[i].x - m2);
    p.L += f * ml[i].y;
    p.y.x += f * z[i].x;
    p.y.y += f * z[i].y;
    p.y.z += f * z[i].z;
    p.y.w += f * z[i].w;
  }
}
struct JoinItem {
  int b, h, rt, rows, leader, pieces;
};
__device__ __forceinline__ JoinItem join_item(const AttnArgs& a, int item, int leader, int follow) {
  JoinItem x;
  const int seg = a.by_rt(item);
  x.rt = item - seg * a.rt;
  x.b = a.by_H(seg);
  x.h = seg - x.b * a.H;
  const int mr = a.new_lens ? __ldg(a.new_lens + x.b) : a.m;
  x.rows = min(a.tr, min(max(mr, 0), a.m) * a.G - x.rt * a.tr);
  x.leader = leader;
  x.pieces = follow + 1;
  return x;
}
// pieces c, c + step, ... (N of them at most) of row r
template <int N>
__device__ __forceinline__ void fetch(const AttnArgs& a, const JoinItem& x, int r, int c, int step, float2* ml, float4* z) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int ci = c + i * step;
    ml[i] = make_float2(-INFINITY, 0.f);
    z[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < x.rows && ci < x.pieces) {
      const long long at = (ci == 0 ? 2ll * x.leader + 1 : 2ll * (x.leader + ci)) * a.tr + r;
      ml[i] = a.part_ml[at];
      z[i] = *reinterpret_cast<const float4*>(a.part_o + at * kHeadDim + lane_id() * 4);
    }
  }
}
__device__ __forceinline__ void finish(const AttnArgs& a, const JoinItem& x, int r, const Joined& p) {
  const int rr = x.rt * a.tr + r;
  const float inv = p.L > 0.f ? 1.f / p.L : 0.f;
  *reinterpret_cast<uint2*>(out_row(a, x.b, x.h, rr) + lane_id() * 4) =
      make_uint2(pack_bf16(p.y.x * inv, p.y.y * inv), pack_bf16(p.y.z * inv, p.y.w * inv));
  if (lane_id() == 0) write_lse(a, x.b, x.h, rr, p.M, p.L);
}

// grid (item, row)
__global__ void __launch_bounds__(kJoinWarps * 32) join_items_kernel(const AttnArgs a) {
  __shared__ float4 s_y[kJoinWarps][32];
  __shared__ float2 s_ml[kJoinWarps];
  const int warp = warp_id(), lane = lane_id(), r = blockIdx.y;
  // an item without rows has no record
  const int2 rec = a.rec[blockIdx.x];
  // (nor one whose kernel gave up on a wait: what lies there then is not followed)
  const JoinItem x = join_item(a, blockIdx.x, rec.x, rec.y);
  if (r >= x.rows || rec.x < 0 || rec.y < 0 || rec.x + rec.y >= a.grid || rec.x >= a.grid) return;
  Joined p = nothing();
  for (int c = warp; c < x.pieces; c += 8 * kJoinWarps) {
    float2 ml[8];
    float4 z[8];
    fetch<8>(a, x, r, c, kJoinWarps, ml, z);
    add_pieces<8>(p, ml, z);
  }
  s_y[warp][lane] = p.y;
  if (lane == 0) s_ml[warp] = make_float2(p.M, p.L);
  __syncthreads();
  if (warp) return;
  p = nothing();
  float2 ml[kJoinWarps];
  float4 z[kJoinWarps];
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    ml[w] = s_ml[w];
    z[w] = s_y[w][lane];
  }
  add_pieces<kJoinWarps>(p, ml, z);
  finish(a, x, r, p);
}

// grid (CTA of the kernel before, share of its rows): all CTAs resident at once, two rows per warp at a time
constexpr int kShares = 5;
__global__ void __launch_bounds__(kJoinWarps * 32, kShares) join_ctas_kernel(const AttnArgs a) {
  const int2 rec = a.rec[blockIdx.x];
  if (rec.x < 0) return;
  const JoinItem x = join_item(a, rec.x, blockIdx.x, rec.y);
  constexpr int kStep = kShares * kJoinWarps;
  for (int r = blockIdx.y * kJoinWarps + warp_id(); r < x.rows; r += 2 * kStep) {
    Joined p = nothing(), p2 = nothing();
    for (int c = 0; c < x.pieces; c += 2) {
      float2 ml[4];
      float4 z[4];
      fetch<2>(a, x, r, c, 1, ml, z);
      fetch<2>(a, x, r + kStep, c, 1, ml + 2, z + 2);
      add_pieces<2>(p, ml, z);
      add_pieces<2>(p2, ml + 2, z + 2);
    }
    finish(a, x, r, p);
    if (r + kStep < x.rows) finish(a, x, r + kStep, p2);
  }
}

}  // namespace

cudaError_t launch_attend_join(const AttnArgs& a, int grid, cudaStream_t st) {
  const int rows = static_cast<int>(std::min<long long>(a.tr, static_cast<long long>(a.m) * a.G));
  if (a.by_item)
    join_items_kernel<<<dim3(a.B * a.H * a.rt, rows), kJoinWarps * 32, 0, st>>>(a);
  else
    join_ctas_kernel<<<dim3(grid, kShares), kJoinWarps * 32, 0, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace kvsel
