// Joins the pieces of items that several CTAs of attend_rows_kernel or attend_tile_kernel
// share.  Piece c of an item that starts in CTA x sits in slot 1 of CTA x (c = 0) or slot 0 of
// CTA x + c: unnormalised rows, their references (log2 units) and sums.  The loads of a row's
// pieces do not wait for one another; pieces are added in a fixed order, so results repeat.
//
// Few rows of many pieces (by_item): a CTA per row, eight warps over its pieces, of which there may
// be one per CTA of the grid.  Bound: latency.  Otherwise eight rows per warp, and a thread for a
// row's reference, sum and place: a warp for each row spent 290 instructions on it, nearly all of
// them the same in every lane, and took 18 us for 38,000 rows; now 8.  Bound: the pieces' bytes, from
// L2.  (Joining in the CTA that finishes an item's last piece, without a second launch, took 38 us
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
// Whether an item's pieces lie in CTAs of the grid, whatever the record holds (the sum of its numbers could
// pass 32 bits).
__host__ __device__ constexpr bool pieces_fit(int leader, int follow, int grid) {
  return leader >= 0 && leader < grid && follow >= 0 && follow < grid - leader;
}
static_assert(pieces_fit(0, 0, 1) && pieces_fit(1, 2, 4) && !pieces_fit(1, 3, 4) && !pieces_fit(4, 0, 4));
static_assert(!pieces_fit(-1, 0, 4) && !pieces_fit(0, -1, 4) && !pieces_fit(3, 0x7FFFFFFF, 4));
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
  if (r >= x.rows || !pieces_fit(rec.x, rec.y, a.grid)) return;
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

// grid (CTA of the kernel before, share of its rows): eight rows per warp.  Lane l looks after row l & 7:
// its reference, sum and place; the rows themselves are read by the whole warp.
constexpr int kRows = 8;
__global__ void __launch_bounds__(kJoinWarps * 32, 3) join_ctas_kernel(const AttnArgs a) {
  const int2 rec = a.rec[blockIdx.x];
  if (rec.x < 0) return;
  const JoinItem x = join_item(a, rec.x, blockIdx.x, rec.y);
  const int lane = lane_id(), r0 = (blockIdx.y * (blockDim.x >> 5) + warp_id()) * kRows, r = r0 + (lane & 7);
  if (r0 >= x.rows) return;
  auto place = [&](int c) { return (c == 0 ? 2ll * x.leader + 1 : 2ll * (x.leader + c)) * a.tr; };
  auto stats = [&](int c) { return r < x.rows && c < x.pieces ? a.part_ml[place(c) + r] : make_float2(-INFINITY, 0.f); };
  float M = -INFINITY, L = 0.f;
  for (int c = 0; c < x.pieces; c += 4) {
    float2 ml[4];
    float m2 = M;
#pragma unroll
    for (int i = 0; i < 4; ++i) ml[i] = stats(c + i);
#pragma unroll
    for (int i = 0; i < 4; ++i) m2 = fmaxf(m2, ml[i].x);
    L *= M == -INFINITY ? 0.f : exp2f(M - m2);
    M = m2;
#pragma unroll
    for (int i = 0; i < 4; ++i) L += ml[i].x == -INFINITY ? 0.f : exp2f(ml[i].x - M) * ml[i].y;
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  const int rr = x.rt * a.tr + r;
  long long dst = 0;
  if (r < x.rows) {
    dst = out_row(a, x.b, x.h, rr) - a.out;
    if (lane < kRows) write_lse(a, x.b, x.h, rr, M, L);
  }
  float4 y[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = 0; c < x.pieces; ++c) {
    const float m = stats(c).x;
    const float w = m == -INFINITY ? 0.f : exp2f(m - M) * inv;
    const float4* src = reinterpret_cast<const float4*>(a.part_o + (place(c) + r0) * kHeadDim) + lane;
    float4 z[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) z[k] = r0 + k < x.rows ? src[k * (kHeadDim / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const float f = __shfl_sync(0xffffffffu, w, k);
      y[k].x += f * z[k].x;
      y[k].y += f * z[k].y;
      y[k].z += f * z[k].z;
      y[k].w += f * z[k].w;
    }
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const long long d = __shfl_sync(0xffffffffu, dst, k);
    if (r0 + k < x.rows)
      *reinterpret_cast<uint2*>(a.out + d + lane * 4) = make_uint2(pack_bf16(y[k].x, y[k].y), pack_bf16(y[k].z, y[k].w));
  }
}

// The same for the nodes of a tree, whose items have some tens to hundreds of rows in many pieces: grid (item, eight
// rows), a warp to every eighth piece, joined in shared memory.  Bound: latency, two or
// three pieces one after another.  (256 rows of 8 items, 19 pieces each: 16.6 us with eight rows per warp.)
__global__ void __launch_bounds__(kJoinWarps * 32) join_trees_kernel(const AttnArgs a) {
  __shared__ float4 s_y[kJoinWarps][kRows][32];
  __shared__ float2 s_ml[kJoinWarps][kRows];
  const int2 rec = a.rec[blockIdx.x];
  if (!pieces_fit(rec.x, rec.y, a.grid)) return;
  const JoinItem x = join_item(a, blockIdx.x, rec.x, rec.y);
  const int warp = warp_id(), lane = lane_id(), r0 = blockIdx.y * kRows, r = r0 + (lane & 7);
  if (r0 >= x.rows) return;
  float M = -INFINITY, L = 0.f;                      // of row r
  float4 y[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = warp; c < x.pieces; c += kJoinWarps) {
    const long long at = (c == 0 ? 2ll * x.leader + 1 : 2ll * (x.leader + c)) * a.tr;
    const float2 ml = r < x.rows ? a.part_ml[at + r] : make_float2(-INFINITY, 0.f);
    const float4* src = reinterpret_cast<const float4*>(a.part_o + (at + r0) * kHeadDim) + lane;
    float4 z[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) z[k] = r0 + k < x.rows ? src[k * (kHeadDim / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
    const float m2 = fmaxf(M, ml.x);
    const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m2), old = M == -INFINITY ? 0.f : exp2f(M - m2);
    M = m2;
    L = L * old + ml.y * f;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const float g = __shfl_sync(0xffffffffu, f, k), o = __shfl_sync(0xffffffffu, old, k);
      y[k].x = y[k].x * o + z[k].x * g;
      y[k].y = y[k].y * o + z[k].y * g;
      y[k].z = y[k].z * o + z[k].z * g;
      y[k].w = y[k].w * o + z[k].w * g;
    }
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) s_y[warp][k][lane] = y[k];
  if (lane < kRows) s_ml[warp][lane] = make_float2(M, L);
  __syncthreads();
  static_assert(kRows == kJoinWarps, "a warp per row");
  if (r0 + warp >= x.rows) return;
  Joined p = nothing();
  float2 ml[kJoinWarps];
  float4 z[kJoinWarps];
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    ml[w] = s_ml[w][warp];
    z[w] = s_y[w][warp][lane];
  }
  add_pieces<kJoinWarps>(p, ml, z);
  finish(a, x, r0 + warp, p);
}

}  // namespace

cudaError_t launch_attend_join(const AttnArgs& a, int grid, cudaStream_t st) {
  const int rows = static_cast<int>(std::min<long long>(a.tr, static_cast<long long>(a.m) * a.G));
  // (64 items of 128 rows, two or three pieces each: 9.6 us here and 6.6 with eight rows per warp)
  if (a.tree && a.by_item) {
    join_trees_kernel<<<dim3(a.B * a.H * a.rt, (rows + kRows - 1) / kRows), kJoinWarps * 32, 0, st>>>(a);
  } else if (a.by_item) {
    join_items_kernel<<<dim3(a.B * a.H * a.rt, rows), kJoinWarps * 32, 0, st>>>(a);
  } else {
    const int warps = (rows + kRows - 1) / kRows, per = std::min(warps, kJoinWarps);
    join_ctas_kernel<<<dim3(grid, (warps + per - 1) / per), per * 32, 0, st>>>(a);
  }
  note_launch();
  return cudaGetLastError();
}

}  // namespace kvsel
