// Attention of a few query rows (single tokens, drafted tokens) over a long cache:
//   out_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp2(s2 * <q_r, k_j> - ref_r),
// with the reference ref_r within kSlack of the running maximum (in log2 units), so that the
// accumulator is rescaled only when the maximum has grown by more than that; sums and
// accumulators in fp32.
//
// Bound: HBM.  A cached row costs 512 B and 512 flop per query row, so with at most 16 rows
// the tensor cores are idle most of the time and mma.sync m16n8k16, whose operands come
// straight from registers, is enough: a tcgen05 tile would have 128 rows to fill.  Every warp
// streams its own 16-row units of K and V through its own three-stage cp.async ring, without a
// block-wide barrier inside an item, and keeps its own reference, sum and accumulator; the
// four warps are merged once per item.  cp.async writes zeros for rows that no query row
// sees, so nothing that lies behind a segment's end can reach a product.
//
// Where few tiles fall to each CTA (attend_rows_cluster), an item belongs to a cluster, whose CTAs
// take a share of its tiles each and join them through distributed shared memory.  Otherwise
// items (16 query rows of one segment) are cut along the cache so that every CTA of the grid
// gets the same number of tiles whatever the lengths are (share_of); the pieces of an item
// that was cut are joined by attend_join.cu's kernels, in cache order.
//
// Measured, 8 KV heads, one token: 16 requests of 2048 to 65536 rows in pages of 16 342-345 us for
// 2.30 GB, the copy rate; eight requests, window of 4096 in pages of 64, 26 us for 134 MB
// (clusters of four; 30 us with plan and join); one request of 1111 rows 6.6 us (7.4).
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "attend.cuh"

namespace cgx = cooperative_groups;

namespace kvsel {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTR = 16;                              // query rows per item
constexpr int kUnit = 16;                            // cached rows per warp and step
constexpr int kTK = kUnit * kWarps;                  // cached rows per tile
constexpr int kStages = 3;
constexpr int kMaxCluster = 8;
// what the start of an item costs in the plan, in tiles (eight requests, window of 4096, without
// clusters: 32.1 us without it, 31.2 at one, 30.6 at two and four; a compacted cache of 4 heads 13.1,
// 12.3, 12.2)
constexpr int kStart = 2;
constexpr int kUnitBytes = kUnit * 256;              // one side (K or V) of a unit
constexpr int kStageBytes = 2 * kUnitBytes;
constexpr int kOPad = 132;                           // floats per accumulator row when merging
constexpr size_t kSmem = kWarps * kStages * kStageBytes;
static_assert(kWarps * kTR * kOPad * 4 <= kSmem, "the merge reuses the ring");

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(static_cast<unsigned long long>(__cvta_generic_to_global(src))), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t r[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t r[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// CLUSTER: an item's tiles are cut over the CTAs of a cluster instead, which join them.
template <bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 2) attend_rows_kernel(const AttnArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ float s_m[kWarps][kTR], s_l[kWarps][kTR];
  const int warp = warp_id(), lane = lane_id();
  const int quad = lane >> 2, ql = lane & 3;
  const int cs = CLUSTER ? static_cast<int>(cgx::this_cluster().num_blocks()) : 1;
  const int rank = CLUSTER ? static_cast<int>(cgx::this_cluster().block_rank()) : 0;
  Share<ItemRange> sh{};
  if (!CLUSTER) {
    rec_clear(a);
    sh = share_of<kThreads, false>(a.B * a.H * a.rt, [&](int i) { return item_range<kTK>(a, i); }, blockIdx.x, kStart);
    if (static_cast<int>(blockIdx.x) >= sh.grid) return;
  }
  const uint32_t ring = smem_u32(smem) + warp * (kStages * kStageBytes);
  float* s_o = reinterpret_cast<float*>(smem);

  long long base = sh.item_base;
  for (int item = CLUSTER ? static_cast<int>(blockIdx.x) / cs : sh.item; CLUSTER || base < sh.end; ++item) {
    const ItemRange x = !CLUSTER && item == sh.item ? sh.first : item_range<kTK>(a, item);
    int ta, tb;
    if (CLUSTER) {
      if (x.tiles == 0) return;                      // the whole cluster
      ta = static_cast<int>(static_cast<long long>(x.tiles) * rank / cs);
      tb = static_cast<int>(static_cast<long long>(x.tiles) * (rank + 1) / cs);
    } else if (!next_piece<false>(sh, item, x, base, ta, tb)) {
      continue;
    }
    const int cnt = tb - ta;

    // element offset of the cached row that this lane looks up for unit u (rows 0..15: lanes l
    // and l + 16), one unit ahead of the copies that use it; -1 where there is none
    auto lookup = [&](int u) -> long long {
      if (u >= cnt) return -1;
      int j0, j1;
      tile_rows<kTK>(x, ta + u, j0, j1);
      const int j = j0 + warp * kUnit + (lane & 15);
      if (unseen(a, x, j, j1)) return -1;
      const long long e = row_elem(a, x.b, x.h, x.row0, j);
      if (e < 0) atomicOr(a.wc.status, DEV_BAD_INDEX);
      return e;
    };
    auto issue = [&](int u, long long off) {
      if (u < cnt) {
        const uint32_t dst = ring + (u % kStages) * kStageBytes;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = i * 2 + (lane >> 4), c = lane & 15;
          const long long e = __shfl_sync(0xffffffffu, off, row);
          const long long s = e < 0 ? 0 : e + c * 8;
          const uint32_t d = dst + row * 256 + ((c ^ (row & 7)) << 4);
          cp_async16_zfill(d, a.k + s, e >= 0);
          cp_async16_zfill(d + kUnitBytes, a.v + s, e >= 0);
        }
      }
      cp_async_commit();
    };
    long long ahead = lookup(0);
#pragma unroll
    for (int u = 0; u < kStages - 1; ++u) {
      const long long off = ahead;
      ahead = lookup(u + 1);
      issue(u, off);
    }

    // query rows as mma A fragments: rows quad and quad + 8, two neighbouring columns each
    uint32_t qf[8][4];
    const int r0 = x.rt * kTR;
    int pos[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = r0 + quad + 8 * u;
      const int t = a.by_G(r), g = r - t * a.G;
      const bool live = quad + 8 * u < x.rows;
      pos[u] = live ? (a.causal ? x.n - x.m + t : x.n - 1) : -1;
      const uint16_t* src = a.q + x.b * a.q_req + static_cast<long long>(x.h * a.G + g) * a.q_head +
                            static_cast<long long>(t) * a.q_tok;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        qf[kk][u] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + kk * 16 + ql * 2)) : 0u;
        qf[kk][u + 2] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + kk * 16 + 8 + ql * 2)) : 0u;
      }
    }

    float o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float ref[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};

    for (int u = 0; u < cnt; ++u) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      {
        const long long off = ahead;
        ahead = lookup(u + kStages);
        issue(u + kStages - 1, off);
      }
      const uint32_t sk = ring + (u % kStages) * kStageBytes, sv = sk + kUnitBytes;
      float c[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[0][i] = c[1][i] = 0.f;
      {
        const int row = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          uint32_t b[4];
          ldmatrix4(sk + row * 256 + (((kk * 2 + ((lane >> 3) & 1)) ^ (row & 7)) << 4), b);
          mma16816(c[0], qf[kk], b[0], b[1]);
          mma16816(c[1], qf[kk], b[2], b[3]);
        }
      }
      int j0, j1;
      tile_rows<kTK>(x, ta + u, j0, j1);
      j0 += warp * kUnit;
      // every row of the block sees all 16 cached rows: no element masks
      const bool whole =
          j0 + kUnit <= j1 &&
          (!a.causal || (j0 + kUnit <= x.p0 + 1 && (a.window <= 0 || j0 > x.p1 - a.window || j0 + kUnit <= a.n_sink)));
      float p[2][4];
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float y = c[nt][i] * a.s2;
          if (!whole) {
            const int j = j0 + nt * 8 + ql * 2 + (i & 1);
            if (j >= j1 || !sees(a, pos[i >> 1], j)) y = -INFINITY;
          }
          p[nt][i] = y;
          top[i >> 1] = fmaxf(top[i >> 1], y);
        }
#pragma unroll
      for (int u2 = 0; u2 < 2; ++u2) {
        top[u2] = fmaxf(top[u2], __shfl_xor_sync(0xffffffffu, top[u2], 1));
        top[u2] = fmaxf(top[u2], __shfl_xor_sync(0xffffffffu, top[u2], 2));
      }
      if (a.logits) {
        // kept for the weights, which need the whole row's sum first (4 B per row and query row
        // instead of reading K again)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int u2 = 0; u2 < 2; ++u2) {
            const int r = quad + 8 * u2, j = j0 + nt * 8 + ql * 2;
            float* d = a.logits + (static_cast<long long>(x.seg) * a.m * a.G + r) * a.logit_stride + j;
            if (r < x.rows && j + 1 < j1)
              *reinterpret_cast<float2*>(d) = make_float2(p[nt][2 * u2], p[nt][2 * u2 + 1]);
            else if (r < x.rows && j < j1)
              *d = p[nt][2 * u2];
          }
      }
      if (__any_sync(0xffffffffu, top[0] > ref[0] + kSlack || top[1] > ref[1] + kSlack)) {
        float f[2];
#pragma unroll
        for (int u2 = 0; u2 < 2; ++u2) {
          const float r2 = top[u2] > ref[u2] + kSlack ? top[u2] : ref[u2];
          f[u2] = ref[u2] == -INFINITY ? 0.f : exp2f(ref[u2] - r2);
          ref[u2] = r2;
          sum[u2] *= f[u2];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          o[i][0] *= f[0];
          o[i][1] *= f[0];
          o[i][2] *= f[1];
          o[i][3] *= f[1];
        }
      }
      const float base0 = ref[0] == -INFINITY ? 0.f : ref[0], base1 = ref[1] == -INFINITY ? 0.f : ref[1];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        p[nt][0] = ex2_approx(p[nt][0] - base0);
        p[nt][1] = ex2_approx(p[nt][1] - base0);
        p[nt][2] = ex2_approx(p[nt][2] - base1);
        p[nt][3] = ex2_approx(p[nt][3] - base1);
        sum[0] += p[nt][0] + p[nt][1];
        sum[1] += p[nt][2] + p[nt][3];
      }
      // the weights enter the second product as a bf16 high part and remainder: the tensor
      // cores are idle here, and the result then carries the output's rounding alone
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y0 = p[i >> 1][(i & 1) * 2], y1 = p[i >> 1][(i & 1) * 2 + 1];
        const __nv_bfloat162 h2 = __floats2bfloat162_rn(y0, y1);
        const float2 hf = __bfloat1622float2(h2);
        hi[i] = *reinterpret_cast<const uint32_t*>(&h2);
        lo[i] = pack_bf16(y0 - hf.x, y1 - hf.y);
      }
      {
        const int row = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
        for (int nd = 0; nd < 8; ++nd) {
          uint32_t b[4];
          ldmatrix4_trans(sv + row * 256 + (((nd * 2 + (lane >> 4)) ^ (row & 7)) << 4), b);
          mma16816(o[nd * 2], hi, b[0], b[1]);
          mma16816(o[nd * 2 + 1], hi, b[2], b[3]);
          mma16816(o[nd * 2], lo, b[0], b[1]);
          mma16816(o[nd * 2 + 1], lo, b[2], b[3]);
        }
      }
      __syncwarp();   // the stage is refilled after every lane has read it
    }

    // merge the four warps: common reference, rescaled sums and accumulators
    cp_async_wait<0>();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], 1);
      sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], 2);
      if (ql == 0) {
        s_m[warp][quad + 8 * u] = ref[u];
        s_l[warp][quad + 8 * u] = sum[u];
      }
    }
    __syncthreads();   // the rings are free
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float* d = s_o + (warp * kTR + quad) * kOPad + i * 8 + ql * 2;
      if (quad < x.rows) *reinterpret_cast<float2*>(d) = make_float2(o[i][0], o[i][1]);
      if (quad + 8 < x.rows) *reinterpret_cast<float2*>(d + 8 * kOPad) = make_float2(o[i][2], o[i][3]);
    }
    __syncthreads();
    const bool first = ta == 0, last = tb == x.tiles;
    const int slot = 2 * blockIdx.x + (first ? 1 : 0);
    for (int r = warp; r < x.rows; r += kWarps) {
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = s_m[w][r] == -INFINITY ? 0.f : exp2f(s_m[w][r] - M);
        const float4 z = *reinterpret_cast<const float4*>(s_o + (w * kTR + r) * kOPad + lane * 4);
        L += f * s_l[w][r];
        y.x += f * z.x;
        y.y += f * z.y;
        y.z += f * z.z;
        y.w += f * z.w;
      }
      if (CLUSTER) {
        // stays here, in the place of the first warp's, for the CTA that joins the row
        *reinterpret_cast<float4*>(s_o + r * kOPad + lane * 4) = y;
        __syncwarp();
        if (lane == 0) {
          s_m[0][r] = M;
          s_l[0][r] = L;
        }
      } else if (first && last) {
        const float inv = L > 0.f ? 1.f / L : 0.f;
        *reinterpret_cast<uint2*>(out_row(a, x.b, x.h, r0 + r) + lane * 4) =
            make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
        if (lane == 0) write_lse(a, x.b, x.h, r0 + r, M, L);
      } else {
        *reinterpret_cast<float4*>(a.part_o + (static_cast<long long>(slot) * kTR + r) * kHeadDim + lane * 4) = y;
        if (lane == 0) a.part_ml[static_cast<long long>(slot) * kTR + r] = make_float2(M, L);
      }
    }
    if (CLUSTER) {
      cgx::cluster_group cl = cgx::this_cluster();
      cl.sync();
      for (int r = rank + cs * warp; r < x.rows; r += cs * kWarps) {
        float m[kMaxCluster], l[kMaxCluster], M = -INFINITY, L = 0.f;
        float4 z[kMaxCluster], y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          m[c] = -INFINITY;
          if (c < cs) {
            m[c] = *cl.map_shared_rank(&s_m[0][r], c);
            l[c] = *cl.map_shared_rank(&s_l[0][r], c);
            z[c] = *reinterpret_cast<const float4*>(cl.map_shared_rank(s_o + r * kOPad + lane * 4, c));
          }
          M = fmaxf(M, m[c]);
        }
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          if (m[c] == -INFINITY) continue;
          const float f = exp2f(m[c] - M);
          L += f * l[c];
          y.x += f * z[c].x;
          y.y += f * z[c].y;
          y.z += f * z[c].z;
          y.w += f * z[c].w;
        }
        const float inv = L > 0.f ? 1.f / L : 0.f;
        *reinterpret_cast<uint2*>(out_row(a, x.b, x.h, r0 + r) + lane * 4) =
            make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
        if (lane == 0) write_lse(a, x.b, x.h, r0 + r, M, L);
      }
      cl.sync();                                     // its shared memory has been read
      return;
    }
    if (first) rec_first(a, item, last ? 0 : last_cta(sh, base) - static_cast<int>(blockIdx.x));
    __syncthreads();   // s_m, s_l and the accumulators are read before the next item
  }
}

// Accumulated weights from the kept logits: acc_j += sum over query rows r of
// exp2(logit_rj - lse2_r).  A thread owns a cached row (EACH of them, 256 apart), so the order of
// additions is fixed.
// Bound: the logits, 4 B per cached row and query row, mostly from L2.
template <int EACH>
__global__ void __launch_bounds__(256) weights_kept_kernel(const AttnArgs a) {
  __shared__ float s_e[kTR];
  const int seg = blockIdx.y, R = a.m * a.G;
  const ItemRange x = item_range<kTK>(a, seg);       // one item per segment: R <= 16
  if (static_cast<long long>(blockIdx.x) * 256 * EACH >= x.n || x.rows == 0) return;
  if (static_cast<int>(threadIdx.x) < x.rows) s_e[threadIdx.x] = a.lse2[static_cast<long long>(seg) * R + threadIdx.x];
  __syncthreads();
  // rows outside the item's tiles have no logits: no query row sees them
  const int in_first = min(x.sink, x.ns * kTK);
  for (long long j0 = static_cast<long long>(blockIdx.x) * 256 * EACH + threadIdx.x; j0 < x.n; j0 += gridDim.x * 256ll * EACH) {
    float* acc = a.acc + seg * a.acc_stride + j0;
    const float* lg = a.logits + static_cast<long long>(seg) * R * a.logit_stride + j0;
    bool in[EACH];
    float old[EACH], w[EACH];
#pragma unroll
    for (int u = 0; u < EACH; ++u) {
      const long long j = j0 + u * 256;
      in[u] = j < in_first || (j >= x.lo && j < x.hi);
      old[u] = in[u] ? acc[u * 256] : 0.f;
      w[u] = 0.f;
    }
#pragma unroll 4
    for (int r = 0; r < x.rows; ++r) {
      const float e2 = s_e[r];
      if (e2 == -INFINITY) continue;
#pragma unroll
      for (int u = 0; u < EACH; ++u)
        if (in[u]) w[u] += ex2_approx(lg[r * a.logit_stride + u * 256] - e2);
    }
#pragma unroll
    for (int u = 0; u < EACH; ++u)
      if (in[u]) acc[u * 256] = old[u] + w[u];
  }
}

}  // namespace

int attend_rows_tile() { return kTR; }
int attend_rows_ctas_per_sm() { return 2; }

namespace {

cudaLaunchConfig_t cluster_config(int ctas, int cluster, cudaStream_t st, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = cluster;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Clusters of c CTAs that the current device holds at once (a cluster sits inside one GPC, so sizes that
// do not divide a GPC's CTAs leave some of them empty); asked once per device and size.
int clusters_at_once(int c) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][kMaxCluster + 1];   // plus one; 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < kDevices) {
    const int n = known[dev][c].load(std::memory_order_relaxed);
    if (n) return n - 1;
  }
  const void* kernel = reinterpret_cast<const void*>(attend_rows_kernel<true>);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = cluster_config(c, c, nullptr, attr);
  int n = 0;
  if (ensure_smem(kernel, kSmem) != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (dev < kDevices) known[dev][c].store(n + 1, std::memory_order_relaxed);
  return n;
}

}  // namespace

// CTAs of a cluster per item, or 0: a plan of the whole grid and a join.  `items`, of `tiles` tiles at
// most (with a window: most of them).
//
// The plan and the join cost some 3 us, and a tile takes a CTA 0.78 us as long as HBM keeps up, which
// it does for about 160 CTAs; so clusters win when the tiles of a CTA are less than 4 plus what
// HBM needs for all of them, items * tiles / 156.  Caches of one batch differ in length, and only a
// bound is known here: half of that is counted, and one tile less.  Measured, group 4, all caches as
// long as the bound, plan and cluster: 8 items of 64 rows 5.7 and 4.7 us, of 512 7.5 and 5.2, of 2048
// 8.1 and 7.7, of 4096 9.1 and 11.0; 40 items of 1111 rows 10.2 and 8.0; 128 items of 128 rows 9.3 and
// 5.9, of 2048 30.0 and 25.0; 64 items with a window of 4096 29.7 and 25.7.  More clusters than
// fit at once lose (512 items of 256 rows 17.9 and 35; 40 clusters of seven 12.4 and 16.7).
int attend_rows_cluster(long long items, long long tiles, bool window, int grid) {
  const int bound = static_cast<int>(3 + items * tiles / (window ? 156 : 312)), t = static_cast<int>(tiles);
  for (int c = static_cast<int>(std::min<long long>(kMaxCluster, grid / items)); c >= 1; --c) {
    const int serial = (t + c - 1) / c;
    if (serial > bound) return 0;
    // (as few CTAs as do it)
    if ((c == 1 || (t + c - 2) / (c - 1) > serial) && items <= clusters_at_once(c)) return c;
  }
  return 0;
}

cudaError_t launch_attend_rows(const AttnArgs& a, int grid, int cluster, cudaStream_t st) {
  const auto kernel = cluster ? attend_rows_kernel<true> : attend_rows_kernel<false>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kernel), kSmem);
  if (e != cudaSuccess) return e;
  if (cluster) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = cluster_config(a.B * a.H * a.rt * cluster, cluster, st, attr);
    e = cudaLaunchKernelEx(&cfg, kernel, a);
    note_launch();
    return e;
  }
  kernel<<<grid, kThreads, kSmem, st>>>(a);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_attend_join(a, grid, st);
}

// With more CTAs of 256 rows than the device holds at once, about, and few query rows, a thread takes four
// cached rows, so that as many loads are on their way.  The whole call, with one row each and with four (best
// of three, us; blocks: of 256 cached rows, over all segments):
//   query rows        4               5               7               8
//   1024 blocks  27.7 and 27.9   28.3 and 28.4   30.0 and 29.8   28.8 and 31.1
//   1280         34.2     34.0   35.3     35.1   36.7     36.7   36.2     38.7
//   1536         38.6     37.9   39.7     38.9   41.2     40.5   40.3     42.8
//   2048         48.8     47.2   50.3     48.7   52.6     50.5   51.7     53.3
//   4096         84.2     80.1   86.2     81.8   90.3     84.8   89.1     87.9
// (512 blocks lose 0.4 with four query rows, 2.7 with eight; 16 query rows lose everywhere, 3 to 9; two cached
// rows each mostly lie between the two.)
constexpr int kWave = 1200, kFewRows = 7;

template <int EACH>
void launch_weights_kept_of(const AttnArgs& a, cudaStream_t st) {
  const int segs = a.B * a.H, rows = 256 * EACH;
  weights_kept_kernel<EACH><<<dim3(std::min((a.max_len + rows - 1) / rows, std::max(1, 16384 / segs)), segs), 256, 0, st>>>(a);
}
cudaError_t launch_weights_kept(const AttnArgs& a, cudaStream_t st) {
  const bool many = static_cast<long long>((a.max_len + 255) / 256) * a.B * a.H > kWave;
  if (many && a.m * a.G <= kFewRows)
    launch_weights_kept_of<4>(a, st);
  else
    launch_weights_kept_of<1>(a, st);
  note_launch();
  return cudaGetLastError();
}

}  // namespace kvsel
