// Accumulated weights of the cached rows for many query rows, on tcgen05:
//   acc_j += sum over query rows r of exp2(s2 <k_j, q_r> - lse2_r)
// with lse2 from the attention itself.  S^T = K Q^T: a thread owns a cached row (a TMEM lane), so
// a row's weights add up in one register, in the order of the query rows, without shuffles.
//
// An item is 256 cached rows of a segment (two K tiles, loaded once); the query blocks that see
// any of them stream by, 128 rows each, double-buffered in TMEM (2 K tiles x 2 x 128 columns).
// All (item, query block) pairs are cut evenly over the grid; an item that several CTAs share
// leaves one 256-float partial per piece, and a last kernel adds them in order.
//
// Bound: the exponentials (one per cached row and query row) with their scaling and adding, then the
// tensor cores (half as many flops as the attention).  1024 tokens of 8 KV heads with 4 query heads
// each over 8192 rows: 72 us, 12 exponentials per clock and SM (17 in an item's middle), tensor pipe
// 43% active.  With few query rows: K, whose next two tiles are loaded while an item is worked on.
#include "attend.cuh"

namespace kvsel {
namespace {

constexpr int kKeys = 256;                           // cached rows per item
// what the start of an item costs, in blocks of query rows (512 tokens over 4096 rows: 80.6 us without it,
// 79.0 at three to six; 1024 over 8192: 194.6, 189.5; 64 over 1000 rows loses, 32.5 and 33.6)
constexpr int kStart = 6;
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kThreads = 320;
constexpr int kStages = 3;                           // query blocks on their way
constexpr int kItems = 2;                            // items whose K tiles are there or on their way
constexpr size_t kSmem = 1024 + (2 * kItems + kStages) * kTileBytes;

struct KeyItem {
  int seg, b, h, jb;              // first cached row
  int n, m, first;                // rows, new tokens, row of token 0
  int q0, tiles;                  // first query block, query blocks that see a row of the item
  int skip;                       // as ItemRange's
  long long row0;
};
// First row of block i of a segment whose first new token is row `first`.
__device__ __forceinline__ int key_block(const AttnArgs& a, int i, int first) {
  if (a.kb_sink < 0 || i < a.kb_sink) return i * kKeys;
  return max(a.kb_sink * kKeys, max(0, first - a.window + 1) & -kKeys) + (i - a.kb_sink) * kKeys;
}
__device__ __forceinline__ KeyItem key_item(const AttnArgs& a, int item, int tok) {
  KeyItem x;
  x.seg = a.by_kb(item);
  x.b = a.by_H(x.seg);
  x.h = x.seg - x.b * a.H;
  const SegLen s = seg_len(a, x.b, x.h);
  x.n = s.n;
  x.m = s.m;
  x.row0 = s.row0;
  x.first = s.n - s.m;
  x.jb = key_block(a, item - x.seg * a.kb, x.first);
  x.q0 = x.tiles = 0;
  x.skip = item;
  if (x.jb >= s.n || s.m == 0) {
    x.skip = x.seg * a.kb + a.kb - 1;
    return x;
  }
  int t0 = 0, t1 = s.m;           // tokens that see a row of the item
  if (a.causal) {
    t0 = max(0, x.jb - x.first);
    if (a.window > 0 && x.jb >= a.n_sink)
      t1 = static_cast<int>(min(static_cast<long long>(s.m),
                                static_cast<long long>(min(x.jb + kKeys, s.n)) - 1 + a.window - x.first));
  }
  if (t0 >= t1) return x;
  x.q0 = t0 / tok;
  x.tiles = (t1 + tok - 1) / tok - x.q0;
  return x;
}

__global__ void __launch_bounds__(kThreads, 1)
    weights_tile_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk, const AttnArgs a,
                        const int block, float* part) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align1024(smem_raw);
  uint8_t* sK = smem;
  uint8_t* sQ = smem + 2 * kItems * kTileBytes;
  __shared__ __align__(8) uint64_t kfull[kItems], kempty[kItems], qfull[kStages], qempty[kStages], lfull[2][2], lempty[2][2], done;
  __shared__ __align__(16) float s_e[kStages][128];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  const int warp = warp_id(), lane = lane_id();
  const int tok = block / a.G;
  // rows of a query stage behind the block's (the group does not divide 128) stay zero
  for (int i = threadIdx.x; i < kStages * kTileBytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (threadIdx.x == 0) {
    for (int u = 0; u < kItems; ++u) {
      mbar_init(&kfull[u], 2);
      mbar_init(&kempty[u], 1);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&qfull[s], 2);
      mbar_init(&qempty[s], 9);                      // its products are done, its sums are read
    }
    for (int w = 0; w < 2; ++w)
      for (int u = 0; u < 2; ++u) {
        mbar_init(&lfull[w][u], 1);
        mbar_init(&lempty[w][u], 4);
      }
    mbar_init(&done, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 0) a.rec[blockIdx.x] = make_int2(-1, 0);
  const auto sh =
      share_of<kThreads>(a.B * a.H * a.kb, [&](int i) { return key_item(a, i, tok); }, blockIdx.x,
                         kStart);
  if (static_cast<int>(blockIdx.x) >= sh.grid) return;   // the whole CTA
  if (warp == kMmaWarp) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = s_tmem;                     // K tile w, buffer u: column 256 w + 128 u

  if (warp == kLoadWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&tq);
      tma_prefetch_desc(&tk);
    }
    int use = 0, piece = 0;
    bool ok = true;
    long long base = sh.item_base;
    for (int item = sh.item; ok && base < sh.end; ++item) {
      const KeyItem x = item == sh.item ? sh.first : key_item(a, item, tok);
      int ta, tb;
      if (!next_piece(sh, item, x, base, ta, tb)) continue;
      const int kb = piece % kItems;
      ok = __all_sync(0xffffffffu, mbar_wait(&kempty[kb], ((piece / kItems) & 1) ^ 1, &s_abort, a.wc));
      if (!ok) break;
      for (int w = 0; w < 2; ++w)
        load_rows<128>(a, x.b, x.h, x.row0, &tk, x.jb + w * 128, x.n, sK + (2 * kb + w) * kTileBytes, &kfull[kb],
                       [&](int from, int to) {
          return a.window <= 0 || !a.causal || from < a.n_sink || to > x.first - a.window;
        });
      ++piece;
      for (int i = ta; i < tb; ++i) {
        const int s = use % kStages, t0 = (x.q0 + i) * tok;
        ok = __all_sync(0xffffffffu, mbar_wait(&qempty[s], ((use / kStages) & 1) ^ 1, &s_abort, a.wc));
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&qfull[s], 2 * block * 128);
          tma_load_4d(sQ + s * kTileBytes, &tq, &qfull[s], 0, x.h * a.G, t0, x.b);
          tma_load_4d(sQ + s * kTileBytes + kHalfBytes, &tq, &qfull[s], 64, x.h * a.G, t0, x.b);
        }
        // log-sums of the block's rows; rows that see nothing and rows behind the block weigh nothing
#pragma unroll
        for (int c = lane; c < 128; c += 32) {
          const int r = t0 * a.G + c;
          float e = INFINITY;
          if (c < block && r < x.m * a.G) {
            e = a.lse2[static_cast<long long>(x.seg) * a.m * a.G + r];
            if (e == -INFINITY) e = INFINITY;
          }
          s_e[s][c] = -e;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&qfull[s]);
        ++use;
      }
    }
    if (lane == 0) {
      for (int u = max(0, use - kStages); u < use; ++u) mbar_drain(&qfull[u % kStages], (u / kStages) & 1, a.wc.status);
      for (int u = max(0, piece - kItems); u < piece; ++u)
        mbar_drain(&kfull[u % kItems], (u / kItems) & 1, a.wc.status);
      if (ok) {
        ring_tail(qempty, kStages, use, &s_abort, a.wc);
        ring_tail(kempty, kItems, piece, &s_abort, a.wc);
      }
    }
  } else if (warp == kMmaWarp) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128);
    const StageLayout lay = stage_layout(a, 128);
    const uint64_t kd0 = sdesc_stage_k(smem_u32(sK), lay), qd0 = sdesc_kmajor_sw128(smem_u32(sQ));
    const uint32_t khalf = lay.half >> 4;
    int use = 0, piece = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase) {
      ok = __all_sync(0xffffffffu, ok && mbar_wait(bar, static_cast<uint32_t>(phase & 1), &s_abort, a.wc));
    };
    long long base = sh.item_base;
    for (int item = sh.item; ok && base < sh.end; ++item) {
      const KeyItem x = item == sh.item ? sh.first : key_item(a, item, tok);
      int ta, tb;
      if (!next_piece(sh, item, x, base, ta, tb)) continue;
      const int cnt = tb - ta;
      const int kb = piece % kItems;
      wait(&kfull[kb], piece / kItems);
      ++piece;
      for (int i = 0; i < cnt && ok; ++i, ++use) {
        const int s = use % kStages, u = use & 1;
        wait(&qfull[s], use / kStages);
        for (int w = 0; w < 2 && ok; ++w) {
          if (use >= 2) wait(&lempty[w][u], (use >> 1) - 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t qd = qd0 + s * (kTileBytes >> 4), kd = kd0 + (2 * kb + w) * (kTileBytes >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t in = ((k & 3) * 32) >> 4;
              umma_bf16(tbase + w * 256 + u * 128, kd + (k >> 2) * khalf + in, qd + (k >> 2) * (kHalfBytes >> 4) + in, idesc,
                        k ? 1u : 0u);
            }
            umma_commit(&lfull[w][u]);
            if (w == 1) umma_commit(&qempty[s]);
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      if (elect_one()) umma_commit(&kempty[kb]);
      __syncwarp();
    }
    if (elect_one()) umma_commit(&done);
    __syncwarp();
    if (lane == 0) mbar_drain(&done, 0, a.wc.status);
  } else {
    const int w = warp >> 2, key = threadIdx.x;      // cached row of the item
    const uint32_t tS = tbase + w * 256 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint64_t sc2 = pack2(a.s2, a.s2);
    int use = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase) {
      ok = __all_sync(0xffffffffu, ok && mbar_wait(bar, static_cast<uint32_t>(phase & 1), &s_abort, a.wc));
    };
    long long base = sh.item_base;
    for (int item = sh.item; ok && base < sh.end; ++item) {
      const KeyItem x = item == sh.item ? sh.first : key_item(a, item, tok);
      int ta, tb;
      if (!next_piece(sh, item, x, base, ta, tb)) continue;
      const int j = x.jb + key;
      // query rows [r0, r1) of the segment see the cached row (the rows behind the last token's are zeros
      // where no request has more tokens, and their log-sums infinity: they need no mask)
      const long long all = static_cast<long long>(x.m) * a.G;
      long long r0 = 0, r1 = j >= x.n ? 0 : x.m == a.m ? all + 128 : all;
      if (a.causal && j < x.n) {
        r0 = static_cast<long long>(max(0, j - x.first)) * a.G;
        if (a.window > 0 && j >= a.n_sink) r1 = min(r1, max(0ll, static_cast<long long>(j) + a.window - x.first) * a.G);
      }
      float sum = 0.f;
      for (int i = ta; i < tb; ++i, ++use) {
        const int s = use % kStages, u = use & 1;
        const long long rb = static_cast<long long>(x.q0 + i) * block;
        wait(&qfull[s], use / kStages);              // the log-sums
        wait(&lfull[w][u], use >> 1);
        if (!ok) break;
        tc_fence_after();
        const int lo = static_cast<int>(max(0ll, min(128ll, r0 - rb))), hi = static_cast<int>(max(0ll, min(128ll, r1 - rb)));
        // (rows behind the block have a sum of infinity and zeros for a query)
        const bool whole = __all_sync(0xffffffffu, lo == 0 && hi >= block);
        uint64_t acc0 = pack2(0.f, 0.f), acc1 = acc0;
        float masked = 0.f;
        __syncwarp();
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 64) {
          // (a warp skips the query rows that none of its cached rows is seen by)
          if (rb + c0 >= all || !__any_sync(0xffffffffu, lo < c0 + 64 && hi > c0)) continue;
          float y[64];
          tmem_ld32(tS + u * 128 + c0, y);
          tmem_ld32(tS + u * 128 + c0 + 32, y + 32);
          tmem_ld_wait();
          const float4* e4 = reinterpret_cast<const float4*>(&s_e[s][c0]);
          if (whole) {
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
              const float4 e = e4[c >> 2];
              float y0, y1, y2, y3;
              unpack2(ffma2(pack2(y[c], y[c + 1]), sc2, pack2(e.x, e.y)), y0, y1);
              unpack2(ffma2(pack2(y[c + 2], y[c + 3]), sc2, pack2(e.z, e.w)), y2, y3);
              acc0 = fadd2(acc0, pack2(ex2_approx(y0), ex2_approx(y1)));
              acc1 = fadd2(acc1, pack2(ex2_approx(y2), ex2_approx(y3)));
            }
          } else {
#pragma unroll
            for (int c = 0; c < 64; ++c) {
              const float p = ex2_approx(fmaf(y[c], a.s2, s_e[s][c0 + c]));
              if (c0 + c >= lo && c0 + c < hi) masked += p;
            }
          }
        }
        float y0, y1;
        unpack2(fadd2(acc0, acc1), y0, y1);
        sum += (y0 + y1) + masked;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&lempty[w][u]);
          mbar_arrive(&qempty[s]);
        }
        __syncwarp();
      }
      if (!ok) break;
      const bool first = ta == 0, last = tb == x.tiles;
      if (first && last) {
        if (j < x.n) a.acc[x.seg * a.acc_stride + j] += sum;
      } else {
        part[(2ll * blockIdx.x + (first ? 1 : 0)) * kKeys + key] = sum;
        if (first && threadIdx.x == 0)
          a.rec[blockIdx.x] = make_int2(item, last_cta(sh, base) - static_cast<int>(blockIdx.x));
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Items that several CTAs share: the partials in order (slots as in attend_join.cu).
__global__ void __launch_bounds__(kKeys) weights_join_kernel(const AttnArgs a, const float* part) {
  const int2 rec = a.rec[blockIdx.x];
  if (rec.x < 0) return;
  const int seg = a.by_kb(rec.x), b = a.by_H(seg);
  const SegLen s = seg_len(a, b, seg - b * a.H);
  const int j = key_block(a, rec.x - seg * a.kb, s.n - s.m) + threadIdx.x;
  if (j >= s.n) return;
  float sum = part[(2ll * blockIdx.x + 1) * kKeys + threadIdx.x];
  for (int c = 1; c <= rec.y; ++c) sum += part[2ll * (blockIdx.x + c) * kKeys + threadIdx.x];
  a.acc[seg * a.acc_stride + j] += sum;
}

}  // namespace

cudaError_t launch_weights_tile(const AttnArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, int block, float* part,
                                int grid, cudaStream_t st) {
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(weights_tile_kernel), kSmem);
  if (e != cudaSuccess) return e;
  weights_tile_kernel<<<grid, kThreads, kSmem, st>>>(tq, tk, a, block, part);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  weights_join_kernel<<<grid, kKeys, 0, st>>>(a, part);
  note_launch();
  return cudaGetLastError();
}

}  // namespace kvsel
