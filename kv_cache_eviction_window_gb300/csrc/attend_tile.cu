// Attention of many query rows (a chunk of new tokens) over a cache, on tcgen05:
//   S = Q K^T (fp32 in TMEM), P = exp2(s2 * S - ref) rounded to bf16 into TMEM, O += P V.
// The reference of a row stays within 8 of its running maximum (log2 units), so O, which stays
// in TMEM, is rescaled only when the maximum has grown by more; row sums are fp32 over the
// unrounded weights.  P is rounded to bf16 (2^-9 relative at most per weight): V is bf16 and
// both operands of the product need one type.
//
// A CTA works on two streams, each with 128 rows of S and O in TMEM (2 x 128 + 2 x 128 of 512
// columns; P overwrites the first half of its S):
//   SPLIT = false  an item has two blocks of query rows; both read the same K and V tiles
//   SPLIT = true   an item has one block; its even and odd key tiles are the two streams, whose
//                  results are added at the end
// While one stream's four warps form the weights of a tile, the tensor cores run the other
// stream's products.  A thread owns one query row, so a row's maximum and sum need no shuffle.
// Roles: warps 0-3 and 4-7 the streams' softmax, warp 8 issues the UMMAs, warp 9 the TMA loads.
//
// A block holds T = 128 / G tokens (T * G rows, the group's heads side by side), so that K and V
// tiles serve the whole group.  Items are cut along the cache as in attend_rows_kernel.
//
// Bound: the exponentials and the instructions around them (128 x 128 per tile and stream),
// then the tensor cores.
#include "attend.cuh"

namespace kvsel {
namespace {

constexpr int kTK = 128;                             // cached rows per tile
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kThreads = 384;                        // three warpgroups; warps 10 and 11 idle
// registers per thread: 168 at launch (3 x 168 x 32 per sub-partition), then 208 for the two
// softmax warpgroups, whose threads hold a row of S, and 88 for the third: 2 x 208 + 88 = 3 x 168
constexpr int kSoftRegs = 208, kOtherRegs = 88;
constexpr int kTile = 128 * 256;                     // bytes of one 128 x 128 bf16 tile
constexpr int kHalf = 128 * 128;                     // its 64-column half
constexpr int kStages = 5;
constexpr size_t kSmem = 1024 + 2 * kTile + kStages * kTile;

// A operand in TMEM
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// MN-major operand, 128-byte swizzle: stored [K rows][64 MN elements], 8-row atoms 1024 B apart, the
// next 64 MN elements one half tile further
__device__ __forceinline__ uint64_t sdesc_mnmajor(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kHalf >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* y) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3]), "=r"(y[4]), "=r"(y[5]), "=r"(y[6]), "=r"(y[7]), "=r"(y[8]),
        "=r"(y[9]), "=r"(y[10]), "=r"(y[11]), "=r"(y[12]), "=r"(y[13]), "=r"(y[14]), "=r"(y[15])
      : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The K or V rows of one tile into a 128B-swizzled stage, by the lanes of the load warp.
__device__ __forceinline__ void load_tile(const AttnArgs& a, const ItemRange& x, const CUtensorMap* map, int j0, int j1,
                                          uint8_t* dst, uint64_t* bar) {
  const int lane = lane_id();
  if (!a.src.paged) {
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, kTile);
      const int row = static_cast<int>(x.row0) + j0;
      const int h = a.offsets ? 0 : x.h, b = a.offsets ? 0 : x.b;
      tma_load_4d(dst, map, bar, 0, row, h, b);
      tma_load_4d(dst + kHalf, map, bar, 64, row, h, b);
    }
    return;
  }
  // lane i: page i of the tile; pages without a row that the item sees are not looked up
  const int bs = a.src.block_size, at = j0 + lane * bs;
  bool live = lane < kTK / bs && at < j1;
  if (live && a.window > 0 && at >= a.n_sink && at + bs - 1 <= x.p0 - a.window) live = false;
  int pb = 0;
  if (live) {
    pb = __ldg(a.src.block_table + static_cast<size_t>(x.b) * a.src.max_blocks + at / bs);
    if (pb < 0 || pb >= a.src.num_blocks) {
      atomicOr(a.wc.status, DEV_BAD_INDEX);
      pb = a.src.num_blocks;                         // outside the pool: zeros
    }
  }
  const unsigned pages = __popc(__ballot_sync(0xffffffffu, live));
  if (lane == 0) mbar_arrive_expect_tx(bar, pages * bs * 256);
  __syncwarp();
  if (live) {
    tma_load_4d(dst + lane * bs * 128, map, bar, 0, x.h, 0, pb);
    tma_load_4d(dst + kHalf + lane * bs * 128, map, bar, 64, x.h, 0, pb);
  }
}

template <bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tile_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const AttnArgs a, const int block) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align1024(smem_raw);
  uint8_t* sQ = smem;                                // two blocks (SPLIT: one, then the exchange buffer)
  uint8_t* sKV = smem + 2 * kTile;
  __shared__ __align__(8) uint64_t qfull, qempty, kvfull[kStages], kvempty[kStages], sfull[2], pfull[2], pv[2], done;
  __shared__ __align__(8) uint64_t xfull, xempty;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ float2 s_ml[128];

  const int warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    a.rec[blockIdx.x] = make_int4(-1, 0, 0, 0);
    mbar_init(&qfull, 1);
    mbar_init(&qempty, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&kvfull[s], 1);
      mbar_init(&kvempty[s], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&sfull[w], 1);
      mbar_init(&pfull[w], 4);
      mbar_init(&pv[w], 1);
    }
    mbar_init(&done, 1);
    mbar_init(&xfull, 4);
    mbar_init(&xempty, 4);
    s_abort = 0;
    fence_mbar_init();
  }
  const Share sh = share_of<kTK, kThreads>(a, blockIdx.x);
  if (static_cast<int>(blockIdx.x) >= sh.grid) return;   // the whole CTA
  if (warp == kMmaWarp) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = s_tmem;                     // S0, S1: columns 0, 128; O0, O1: 256, 384
  constexpr int nblk = SPLIT ? 1 : 2;                // query blocks per item

  if (warp >= kMmaWarp) regs_down<kOtherRegs>();
  if (warp == kLoadWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&tq);
      tma_prefetch_desc(&tk);
      tma_prefetch_desc(&tv);
    }
    int use = 0, piece = 0;                          // ring uses issued, pieces begun
    bool ok = true;                                  // the same in every lane
    long long base = sh.item_base, at = sh.begin;
    for (int item = sh.item; ok && at < sh.end; ++item) {
      const ItemRange x = item_range<kTK>(a, item);
      if (x.tiles == 0) continue;
      const int ta = static_cast<int>(at - base);
      const int cnt = static_cast<int>(min(static_cast<long long>(x.tiles), sh.end - base)) - ta;
      ok = __all_sync(0xffffffffu, mbar_wait(&qempty, (piece & 1) ^ 1, &s_abort, a.wc));
      if (!ok) break;
      if (lane == 0) {
        const int tok = block / a.G;                 // tokens per block
        mbar_arrive_expect_tx(&qfull, nblk * 2 * block * 128);
        for (int w = 0; w < nblk; ++w) {
          const int t0 = (x.rt * nblk + w) * tok;
          tma_load_4d(sQ + w * kTile, &tq, &qfull, 0, x.h * a.G, t0, x.b);
          tma_load_4d(sQ + w * kTile + kHalf, &tq, &qfull, 64, x.h * a.G, t0, x.b);
        }
      }
      ++piece;
      __syncwarp();
      auto load = [&](int ti, bool is_v) {
        const int s = use % kStages;
        ok = __all_sync(0xffffffffu, mbar_wait(&kvempty[s], ((use / kStages) & 1) ^ 1, &s_abort, a.wc));
        if (!ok) return;
        int j0, j1;
        tile_rows<kTK>(x, ta + ti, j0, j1);
        load_tile(a, x, is_v ? &tv : &tk, j0, j1, sKV + s * kTile, &kvfull[s]);
        ++use;
      };
      // the order in which the MMA warp takes the tiles
      constexpr int ahead = SPLIT ? 2 : 1;
      for (int i = 0; i < ahead && i < cnt && ok; ++i) load(i, false);
      for (int i = 0; i < cnt && ok; ++i) {
        load(i, true);
        if (ok && i + ahead < cnt) load(i + ahead, false);
      }
      base += x.tiles;
      at = base;
    }
    // copies in flight land, and the last releases arrive, before the CTA ends
    if (lane == 0) {
      for (int u = max(0, use - kStages); u < use; ++u) mbar_drain(&kvfull[u % kStages], (u / kStages) & 1, a.wc.status);
      if (piece) mbar_drain(&qfull, (piece - 1) & 1, a.wc.status);
      if (ok) {
        ring_tail(kvempty, kStages, use, &s_abort, a.wc);
        ring_tail(&qempty, 1, piece, &s_abort, a.wc);
      }
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, 128) | (1u << 16);   // B (V) MN-major
      int use = 0, piece = 0;
      int np[2] = {0, 0};                            // tiles of each stream so far
      bool ok = true;
      auto wait_stage = [&](int u) {
        ok = ok && mbar_wait(&kvfull[u % kStages], (u / kStages) & 1, &s_abort, a.wc);
        tc_fence_after();
      };
      auto qk = [&](int w, int u) {
        const uint64_t qd = sdesc_kmajor_sw128(smem_u32(sQ + (SPLIT ? 0 : w) * kTile));
        const uint64_t kd = sdesc_kmajor_sw128(smem_u32(sKV + (u % kStages) * kTile));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t off = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
          umma_bf16(tbase + w * 128, qd + off, kd + off, idesc_s, k ? 1u : 0u);
        }
        umma_commit(&sfull[w]);
      };
      // O_w (+)= P_w V once the weights are in TMEM
      auto pvm = [&](int w, int u, bool first) {
        ok = ok && mbar_wait(&pfull[w], np[w] & 1, &s_abort, a.wc);
        if (!ok) return;
        tc_fence_after();
        const uint32_t vb = smem_u32(sKV + (u % kStages) * kTile);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_bf16_ta(tbase + 256 + w * 128, tbase + w * 128 + k * 8, sdesc_mnmajor(vb + k * 2048), idesc_o,
                       (first && k == 0) ? 0u : 1u);
        umma_commit(&pv[w]);
        ++np[w];
      };
      // S_w is written again only after the product that reads P_w in its place
      auto wait_pv = [&](int w) {
        if (np[w]) ok = ok && mbar_wait(&pv[w], (np[w] - 1) & 1, &s_abort, a.wc);
        tc_fence_after();
      };
      auto release = [&](int u) { umma_commit(&kvempty[u % kStages]); };
      long long base = sh.item_base, at = sh.begin;
      for (int item = sh.item; ok && at < sh.end; ++item) {
        const ItemRange x = item_range<kTK>(a, item);
        if (x.tiles == 0) continue;
        const int cnt = static_cast<int>(min(static_cast<long long>(x.tiles), sh.end - base) - (at - base));
        ok = mbar_wait(&qfull, piece & 1, &s_abort, a.wc);
        if (!ok) break;
        tc_fence_after();
        ++piece;
        if (SPLIT) {
          for (int w = 0; w < 2 && w < cnt && ok; ++w) {
            wait_stage(use);
            wait_pv(w);
            if (!ok) break;
            qk(w, use);
            release(use++);
          }
          for (int i = 0; i < cnt && ok; ++i) {
            const int w = i & 1;
            wait_stage(use);
            pvm(w, use, i < 2);
            if (!ok) break;
            release(use++);
            if (i + 2 < cnt) {
              wait_stage(use);
              wait_pv(w);
              if (!ok) break;
              qk(w, use);
              release(use++);
            }
          }
        } else {
          wait_stage(use);
          for (int w = 0; w < 2 && ok; ++w) {
            wait_pv(w);
            if (ok) qk(w, use);
          }
          if (!ok) break;
          release(use++);
          for (int i = 0; i < cnt && ok; ++i) {
            const int uv = use;
            const bool more = i + 1 < cnt;
            wait_stage(uv);
            for (int w = 0; w < 2 && ok; ++w) {
              pvm(w, uv, i == 0);
              if (!ok) break;
              if (w == 1) release(uv);
              if (more) {
                if (w == 0) wait_stage(uv + 1);
                wait_pv(w);
                if (ok) qk(w, uv + 1);
              }
            }
            if (!ok) break;
            if (more) release(uv + 1);
            use += more ? 2 : 1;
          }
        }
        if (!ok) break;
        umma_commit(&qempty);
        base += x.tiles;
        at = base;
      }
      // every product issued has been done before TMEM is freed
      umma_commit(&done);
      mbar_drain(&done, 0, a.wc.status);
    }
  } else if (warp < kMmaWarp) {
    regs_up<kSoftRegs>();
    const int w = warp >> 2, row = threadIdx.x & 127;   // stream, query row within the block (TMEM lane)
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + w * 128 + lanes, tO = tbase + 256 + w * 128 + lanes;
    int np = 0, use = 0, nx = 0;                     // tiles of this stream; ring uses before this piece; exchanges
    bool ok = true;                                  // the same in every lane of a warp
    auto wait = [&](uint64_t* bar, int phase) {
      ok = __all_sync(0xffffffffu, ok && mbar_wait(bar, static_cast<uint32_t>(phase & 1), &s_abort, a.wc));
    };
    long long base = sh.item_base, at = sh.begin;
    for (int item = sh.item; ok && at < sh.end; ++item) {
      const ItemRange x = item_range<kTK>(a, item);
      if (x.tiles == 0) continue;
      const int ta = static_cast<int>(at - base);
      const int tb = static_cast<int>(min(static_cast<long long>(x.tiles), sh.end - base));
      const int cnt = tb - ta;
      const int first_row = SPLIT ? 0 : w * block;   // of the item
      const int rows = min(block, x.rows - first_row);
      const int rr = x.rt * a.tr + first_row + row;  // row of the segment
      const int p = a.causal ? x.n - x.m + rr / a.G : x.n - 1;
      // cache rows of the block's first and last token
      const int pa = a.causal ? x.n - x.m + (x.rt * a.tr + first_row) / a.G : x.n - 1;
      const int pb = a.causal ? x.n - x.m + (x.rt * a.tr + first_row + max(rows, 1) - 1) / a.G : x.n - 1;
      float ref = -INFINITY, sum = 0.f;
      int mine = 0;                                  // tiles of this piece so far
      for (int i = SPLIT ? w : 0; i < cnt; i += SPLIT ? 2 : 1) {
        int j0, j1;
        tile_rows<kTK>(x, ta + i, j0, j1);
        wait(&sfull[w], np);
        if (!ok) break;
        tc_fence_after();
        float s[128];
        tmem_ld32(tS, s);
        tmem_ld32(tS + 32, s + 32);
        tmem_ld32(tS + 64, s + 64);
        tmem_ld32(tS + 96, s + 96);
        tmem_ld_wait();
        const bool whole = j0 + kTK <= j1 && (!a.causal || (j0 + kTK <= pa + 1 &&
                                                            (a.window <= 0 || j0 > pb - a.window || j0 + kTK <= a.n_sink)));
        if (!whole) {
          // a row sees columns [0, hi) and, with a window, of these [lo, hi) and those below `first`
          const int hi = min(j1, a.causal ? p + 1 : j1) - j0;
          const int lo = a.window > 0 ? p - a.window + 1 - j0 : -1, first = a.window > 0 ? a.n_sink - j0 : 0;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= hi || (c < lo && c >= first)) s[c] = -INFINITY;
        }
        float t0 = s[0], t1 = s[1], t2 = s[2], t3 = s[3];
#pragma unroll
        for (int c = 4; c < 124; c += 8) {
          t0 = fmax3(t0, s[c], s[c + 1]);
          t1 = fmax3(t1, s[c + 2], s[c + 3]);
          t2 = fmax3(t2, s[c + 4], s[c + 5]);
          t3 = fmax3(t3, s[c + 6], s[c + 7]);
        }
        t0 = fmax3(t0, s[124], s[125]);
        t1 = fmax3(t1, s[126], s[127]);
        const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * a.s2;
        if (__any_sync(0xffffffffu, top > ref + 8.f)) {
          // each row by its own maximum: a result does not depend on the rows next to it
          const float r2 = top > ref + 8.f ? top : ref;
          const float f = ref == -INFINITY ? 0.f : exp2f(ref - r2);
          ref = r2;
          sum *= f;
          if (mine > 0) {
            // the products that wrote O are done: S of this tile was formed after them
#pragma unroll
            for (int c0 = 0; c0 < 128; c0 += 16) {
              uint32_t y[16];
              tmem_ld16(tO + c0, y);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 16; ++c) y[c] = __float_as_uint(__uint_as_float(y[c]) * f);
              tmem_st16(tO + c0, y);
            }
          }
        }
        const float off = ref == -INFINITY ? 0.f : -ref;
        const uint64_t sc2 = pack2(a.s2, a.s2), off2 = pack2(off, off);
        uint64_t acc0 = pack2(0.f, 0.f), acc1 = acc0;
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            float y0, y1;
            unpack2(ffma2(pack2(s[c0 + c], s[c0 + c + 1]), sc2, off2), y0, y1);
            y0 = ex2_approx(y0);
            y1 = ex2_approx(y1);
            if (c & 2)
              acc1 = fadd2(acc1, pack2(y0, y1));
            else
              acc0 = fadd2(acc0, pack2(y0, y1));
            pk[c >> 1] = pack_bf16(y0, y1);
          }
          tmem_st16(tS + (c0 >> 1), pk);
        }
        {
          float y0, y1;
          unpack2(fadd2(acc0, acc1), y0, y1);
          sum += y0 + y1;
        }
        // V rows that the item does not see may hold anything; their weights are zero, and the
        // rows become zero before the product reads them.  (!SPLIT: stream 0 does it for both,
        // its product is issued first.)
        if ((SPLIT || w == 0) &&
            (j0 + kTK > j1 || (a.window > 0 && j0 <= x.p0 - a.window && j0 + kTK > a.n_sink))) {
          // ring use of this tile's V
          const int uv = SPLIT ? use + min(cnt, 2) + i + max(0, min(i, cnt - 2)) : use + 1 + 2 * i;
          wait(&kvfull[uv % kStages], uv / kStages);
          if (!ok) break;
          if (unseen(a, x, j0 + row, j1)) {
            uint8_t* d = sKV + (uv % kStages) * kTile + row * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              *reinterpret_cast<uint4*>(d + c * 16) = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4*>(d + kHalf + c * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[w]);
        ++np;
        ++mine;
      }
      use += 2 * cnt;                                // a K and a V tile each

      // results of this piece
      const bool first = ta == 0, last = tb == x.tiles, direct = first && last;
      if (mine > 0) wait(&pv[w], np - 1);
      if (!ok) break;
      tc_fence_after();
      const bool live = row < rows && (!SPLIT || w == 0);
      const int slot = 2 * blockIdx.x + (first ? 1 : 0);
      float* po = a.part_o + (static_cast<long long>(slot) * a.tr + first_row + row) * kHeadDim;
      uint16_t* dst = live && direct ? out_row(a, x.b, x.h, rr) : nullptr;
      float f0 = 1.f, f1 = 0.f, inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int c0 = 0; c0 < 128; c0 += 32) {
        float y[32];
        if (mine > 0) {
          tmem_ld32(tO + c0, y);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) y[c] = 0.f;
        }
        if (SPLIT) {
          // stream 1 hands its rows over, 32 columns at a time (a row's 16-byte pieces rotated by
          // the row against bank conflicts), its references and sums with the first of them
          float4* ex = reinterpret_cast<float4*>(sQ + kTile) + row * 8;
          if (w == 1) {
            if (nx) wait(&xempty, nx - 1);
            if (!ok) break;
            if (c0 == 0) s_ml[row] = make_float2(ref, sum);
#pragma unroll
            for (int c = 0; c < 8; ++c)
              ex[(c + row) & 7] = make_float4(y[c * 4], y[c * 4 + 1], y[c * 4 + 2], y[c * 4 + 3]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&xfull);
          } else {
            wait(&xfull, nx);
            if (!ok) break;
            if (c0 == 0) {
              const float2 o = s_ml[row];
              const float M = fmaxf(ref, o.x);
              f0 = ref == -INFINITY ? 0.f : exp2f(ref - M);
              f1 = o.x == -INFINITY ? 0.f : exp2f(o.x - M);
              sum = sum * f0 + o.y * f1;
              ref = M;
              inv = sum > 0.f ? 1.f / sum : 0.f;
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float4 z = ex[(c + row) & 7];
              y[c * 4] = y[c * 4] * f0 + z.x * f1;
              y[c * 4 + 1] = y[c * 4 + 1] * f0 + z.y * f1;
              y[c * 4 + 2] = y[c * 4 + 2] * f0 + z.z * f1;
              y[c * 4 + 3] = y[c * 4 + 3] * f0 + z.w * f1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&xempty);
          }
          ++nx;
        }
        if (live) {
          if (direct) {
#pragma unroll
            for (int c = 0; c < 32; c += 8)
              *reinterpret_cast<uint4*>(dst + c0 + c) =
                  make_uint4(pack_bf16(y[c] * inv, y[c + 1] * inv), pack_bf16(y[c + 2] * inv, y[c + 3] * inv),
                             pack_bf16(y[c + 4] * inv, y[c + 5] * inv), pack_bf16(y[c + 6] * inv, y[c + 7] * inv));
          } else {
#pragma unroll
            for (int c = 0; c < 32; c += 4)
              *reinterpret_cast<float4*>(po + c0 + c) = make_float4(y[c], y[c + 1], y[c + 2], y[c + 3]);
          }
        }
      }
      if (!ok) break;
      if (live) {
        if (direct)
          write_lse(a, x.b, x.h, rr, ref, sum);
        else
          a.part_ml[static_cast<long long>(slot) * a.tr + first_row + row] = make_float2(ref, sum);
      }
      if (first && !last && threadIdx.x == 0)
        a.rec[blockIdx.x] = make_int4(item, last_cta(sh, base + x.tiles) - blockIdx.x, 0, 0);
      tc_fence_before();                             // O is read before the next piece's products
      base += x.tiles;
      at = base;
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

}  // namespace

int attend_tile_keys() { return kTK; }

cudaError_t launch_attend_tile(const AttnArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               int block, bool split, int grid, cudaStream_t st) {
  const auto kernel = split ? attend_tile_kernel<true> : attend_tile_kernel<false>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kernel), kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, kSmem, st>>>(tq, tk, tv, a, block);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_attend_join(a, grid, st);
}

}  // namespace kvsel
