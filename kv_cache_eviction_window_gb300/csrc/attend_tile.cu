// Attention of many query rows (a chunk of new tokens) over a cache, on tcgen05:
//   S = Q K^T (fp32 in TMEM), P = exp2(s2 * S - ref) rounded to bf16 into TMEM, O += P V.
// The reference of a row stays within kSlack = 16 of its running maximum (log2 units), so O, which
// stays in TMEM, is rescaled only when the maximum has grown by more; row sums are fp32 over the
// unrounded weights.  P is rounded to bf16 (2^-8 relative at most per weight): V is bf16 and
// both operands of the product need one type.
//
// A CTA works on two streams of 128 query rows.  Each has O in TMEM (128 columns) and two S
// buffers of 64 keys (P overwrites the first half of its S), 512 columns in all: a key tile of
// 128 is taken in two steps, and the tensor cores form the next step's S while the softmax warps
// work on this one.  (One buffer of 128 keys per stream had its next product wait for the last
// one's P: a dependent group of UMMAs costs about 480 cycles beyond its own 64 per UMMA, and a
// tile pair took 3700-4250 cycles for 2048 of tensor work.  At 64 keys Q K^T is bound by shared
// memory, 48 cycles per UMMA instead of 32, so a tile pair takes 2560 at least.)
//   SPLIT = false  an item has two blocks of query rows; both read the same K and V tiles
//   SPLIT = true   an item has one block; its even and odd key tiles are the two streams, whose
//                  results are added at the end.  Each stream has a K/V ring of its own: a wait for a
//                  phase of a stage is only sound for a warp that knows the phase before to be over,
//                  and with one ring that phase could be the other stream's, still on its way
// While one stream's four warps form the weights of a tile, the tensor cores run the other
// stream's products.  A thread owns one query row, so a row's maximum and sum need no shuffle.
// Roles: warps 0-3 and 4-7 the streams' softmax; warps 8 and 9 issue the streams' Q K^T, warps 10
// and 11 their P V; warp 12 the TMA loads.  (A wait behind a group of UMMAs returns only when the
// group has left its warp's issue queue, about 300 cycles: one warp for all products took 2800
// cycles per step of both streams, one per stream 2200.)
//
// A block holds T = 128 / G tokens (T * G rows, the group's heads side by side), so that K and V
// tiles serve the whole group.  Items are cut along the cache as in attend_rows_kernel.
//
// Bound: the latency of a softmax step (about 1500 cycles for 128 x 64: wait, TMEM load and maximum,
// exponentials, TMEM store), two streams at a time; then the tensor cores.  Measured, 8 KV heads:
// 2048 tokens of 4 query heads each over 32768 contiguous rows 714 us, 1492 TFLOP/s, 0.75 of
// cuBLAS in a burst; from pages of 16 rows 725 us (761-772 in a long run, under the power cap); over an
// empty cache 54 us; 2048 tokens of 8 query heads over 16384 rows, window of 4096, 254 us (tensor pipe
// 51% active, issue 47%).
#include "attend.cuh"

namespace kvsel {
namespace {

constexpr int kTK = 128;                             // cached rows per tile
constexpr int kQkWarp = 8, kPvWarp = 10, kLoadWarp = 12;   // + stream
constexpr int kThreads = 512;                        // four warpgroups; warps 13 (but for BOTH) to 15 idle
// registers per thread: 128 at launch (4 x 128 x 32 per sub-partition), then 184 for the two
// softmax warpgroups and 72 for the others: 2 x 184 + 2 x 72 = 4 x 128
constexpr int kSoftRegs = 184, kOtherRegs = 72;
constexpr int kTile = kTileBytes, kHalf = kHalfBytes;
constexpr int kStages = 5;                           // of 128 rows; SPLIT: per stream, of 64 rows
// What the start of an item costs, in tiles: results written, Q loaded, an empty pipeline, some 6000
// cycles.  (2048 tokens over an empty cache, whose first items have one tile: 75 us without it, 62
// at two tiles, 60 at three; six tokens of four requests over 4096 rows 25.8 and 22.3 us.  It loses
// where there is one tile for each CTA: six tokens over 4864 rows 14.1 and 15.7.)
constexpr int kStart = 3;
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
// Transposes four 16-byte words over four neighbouring lanes: lane q's v[k] becomes lane k's v[q].
__device__ __forceinline__ void quad_transpose(uint4 (&v)[4]) {
#pragma unroll
  for (int s = 1; s < 4; s <<= 1) {
    const bool up = lane_id() & s;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & s) continue;
      uint4 y = up ? v[k] : v[k | s];
      y.x = __shfl_xor_sync(0xffffffffu, y.x, s);
      y.y = __shfl_xor_sync(0xffffffffu, y.y, s);
      y.z = __shfl_xor_sync(0xffffffffu, y.z, s);
      y.w = __shfl_xor_sync(0xffffffffu, y.w, s);
      if (up)
        v[k] = y;
      else
        v[k | s] = y;
    }
  }
}
// MN-major operand in such a stage
__device__ __forceinline__ uint64_t sdesc_stage_v(uint32_t saddr, const StageLayout& l) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(l.half >> 4) << 16;
  d |= static_cast<uint64_t>(l.group >> 4) << 32;
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
// Pages of a 128-row tile of a piece of `cnt`: lane i gets the block of page i (rows of the pool in all, and a note, where
// the table's entry is out of range; -1: a page that no row is seen of).
__device__ __forceinline__ int page_of(const AttnArgs& a, const ItemRange& x, int ta, int ti, int cnt, bool note) {
  if (ti >= cnt) return -1;
  int j0, j1;
  tile_rows<kTK>(x, ta + ti, j0, j1);
  const int lane = lane_id(), bs = a.src.block_size, at = j0 + lane * bs;
  if (lane >= (kTK >> a.page_shift) || at >= j1 || (a.window > 0 && at >= a.n_sink && at + bs - 1 <= x.p0 - a.window)) return -1;
  int pb = __ldg(a.src.block_table + static_cast<size_t>(x.b) * a.src.max_blocks + (at >> a.page_shift));
  if (pb < 0 || pb >= a.src.num_blocks) {
    if (note) atomicOr(a.wc.status, DEV_BAD_INDEX);
    pb = a.src.num_blocks;                           // outside the pool: zeros
  }
  return pb;
}
// ROWS rows of it, half `sub` where that is 64, into a stage
template <int ROWS>
__device__ __forceinline__ void load_pages(const AttnArgs& a, const CUtensorMap* map, int h, int pb, int sub, uint8_t* dst,
                                           uint64_t* bar) {
  const int lane = lane_id(), bs = a.src.block_size, page = lane - (sub * 64 >> a.page_shift);
  const bool live = pb >= 0 && page >= 0 && page < (ROWS >> a.page_shift);
  const unsigned pages = __popc(__ballot_sync(0xffffffffu, live));
  if (lane == 0) mbar_arrive_expect_tx(bar, pages * bs * 256);
  __syncwarp();
  if (live) tma_load_5d(dst + page * bs * 256, map, bar, 0, 0, 0, 0, pb * (bs * a.H) + h);
  __syncwarp();
}

// V tiles of a paged cache by a warp of its own, in the order in which warp 12 loads K.  Warp 12, which sees every use of
// a stage, says where there is room: kvempty's phases pass for K's uses too, two of them look alike, and a warp that sees
// every other use would take one for the other.  (It is never four V tiles of a ring ahead: the stage of the fourth needs
// the first of them landed.)
template <bool SPLIT, int TREE, class Sh>
__device__ __forceinline__ void load_values(const AttnArgs& a, const Sh& sh, const CUtensorMap* tv, uint8_t* sKV,
                                            uint64_t (&kvfull)[2][kStages], uint64_t (&vroom)[2][4], int* s_abort) {
  constexpr int kRows = SPLIT ? 64 : 128;
  int use[2] = {1, 1};
  bool ok = true;                                    // the same in every lane
  long long base = sh.item_base;
  for (int item = sh.item; ok && base < sh.end; ++item) {
    const ItemRange x = item == sh.item ? sh.first : item_range<kTK, TREE>(a, item);
    int ta, tb;
    if (!next_piece(sh, item, x, base, ta, tb)) continue;
    const int cnt = tb - ta;
    auto load = [&](int ring, int sub, int page) {
      const int u = use[ring], s = u % kStages;
      ok = __all_sync(0xffffffffu, ok && mbar_wait(&vroom[ring][u >> 1 & 3], u >> 3 & 1, s_abort, a.wc));
      if (!ok) return;
      use[ring] += 2;
      load_pages<kRows>(a, tv, x.h, page, sub, sKV + (ring * kStages + s) * (kRows * 256), &kvfull[ring][s]);
    };
    // (looked up two tiles ahead of their use)
    int next0 = page_of(a, x, ta, 0, cnt, false), next1 = page_of(a, x, ta, 1, cnt, false);
    for (int i = 0; i < cnt && ok; i += 2) {
      const int page0 = next0, page1 = next1;
      next0 = page_of(a, x, ta, i + 2, cnt, false);
      next1 = page_of(a, x, ta, i + 3, cnt, false);
      if (SPLIT) {
        load(0, 0, page0);
        if (i + 1 < cnt && ok) load(1, 0, page1);
        if (ok) load(0, 1, page0);
        if (i + 1 < cnt && ok) load(1, 1, page1);
      } else {
        load(0, 0, page0);
        if (i + 1 < cnt && ok) load(0, 0, page1);
      }
    }
  }
  // copies in flight land before the CTA ends
  if (lane_id() == 0)
#pragma unroll
    for (int r = 0; r < (SPLIT ? 2 : 1); ++r)
      for (int u = max(1, use[r] - 6); u < use[r]; u += 2) mbar_drain(&kvfull[r][u % kStages], (u / kStages) & 1, a.wc.status);
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// BOTH: small pages by two warps, 12 for K and 13 for V, with the table looked up two tiles ahead.  A box takes its warp
// some 50 cycles beside its bytes.  8 segments of 8 requests of 2048 to 32768 rows, 32 nodes of 4 heads, pages of 16: one
// warp for both, which looks a page up when it loads it, 150 us; two 125; V by 16-byte copies of three warps 136 to 264.
template <bool SPLIT, int TREE, bool BOTH>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tile_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const AttnArgs a, const int block) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align1024(smem_raw);
  uint8_t* sQ = smem;                                // two blocks (SPLIT: one, then the exchange buffer)
  uint8_t* sKV = smem + 2 * kTile;
  __shared__ __align__(8) uint64_t qfull, qempty, kvfull[2][kStages], kvempty[2][kStages], sfull[2][2], pfull[2][2], pv[2][2], done;
  __shared__ __align__(8) uint64_t xfull, xempty, vfix[4], vroom[2][4];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ float2 s_ml[128];

  const int warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    rec_clear(a);
    mbar_init(&qfull, 1);
    mbar_init(&qempty, 2);
    for (int s = 0; s < kStages; ++s) {
      for (int w = 0; w < 2; ++w) {
        mbar_init(&kvfull[w][s], 1);
        mbar_init(&kvempty[w][s], SPLIT ? 1 : 2);    // both streams read a tile, or one
      }
    }
    for (int u = 0; u < 4; ++u) {
      mbar_init(&vfix[u], 4);
      if (BOTH) {
        mbar_init(&vroom[0][u], 1);
        mbar_init(&vroom[1][u], 1);
      }
    }
    for (int w = 0; w < 2; ++w)
      for (int u = 0; u < 2; ++u) {
        mbar_init(&sfull[w][u], 1);
        mbar_init(&pfull[w][u], 4);
        mbar_init(&pv[w][u], 1);
      }
    mbar_init(&done, 4);
    mbar_init(&xfull, 4);
    mbar_init(&xempty, 4);
    s_abort = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == kLoadWarp * 32) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  const auto& sh = share_of<kThreads>(a.B * a.H * a.rt, [&](int i) { return item_range<kTK, TREE>(a, i); }, blockIdx.x, kStart,
                                      a.whole);
  if (static_cast<int>(blockIdx.x) >= sh.grid) return;   // the whole CTA
  if (warp == kQkWarp) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = s_tmem;                     // S of stream w, buffer u: column 128 w + 64 u; O: 256 + 128 w
  constexpr int nblk = SPLIT ? 1 : 2;                // query blocks per item
  constexpr int nring = SPLIT ? 2 : 1;
  constexpr int kStageRows = SPLIT ? 64 : 128, kStageBytes = kStageRows * 256;
  auto stage = [&](int ring, int use) { return sKV + (ring * kStages + use % kStages) * kStageBytes; };

  __syncwarp();
  if (warp >= kQkWarp) regs_down<kOtherRegs>();
  if (warp == kLoadWarp) {
    int use[2] = {0, 0}, piece = 0;                  // ring uses issued, pieces begun
    bool ok = true;                                  // the same in every lane
    long long base = sh.item_base;
    for (int item = sh.item; ok && base < sh.end; ++item) {
      const ItemRange x = item == sh.item ? sh.first : item_range<kTK, TREE>(a, item);
      int ta, tb;
      if (!next_piece(sh, item, x, base, ta, tb)) continue;
      const int cnt = tb - ta;
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
      auto load = [&](int ring, int ti, int sub, bool is_v, int page = 0) {
        const int u = use[ring], s = u % kStages;
        ok = __all_sync(0xffffffffu, ok && mbar_wait(&kvempty[ring][s], ((u / kStages) & 1) ^ 1, &s_abort, a.wc));
        if (!ok) return;
        if (BOTH && is_v) {
          ++use[ring];
          if (lane == 0) mbar_arrive(&vroom[ring][u >> 1 & 3]);
          __syncwarp();
          return;
        }
        if (BOTH) {
          ++use[ring];
          load_pages<kStageRows>(a, &tk, x.h, page, sub, stage(ring, u), &kvfull[ring][s]);
          return;
        }
        int j0, j1;
        tile_rows<kTK>(x, ta + ti, j0, j1);
        load_rows<kStageRows>(a, x.b, x.h, x.row0, is_v ? &tv : &tk, j0 + sub * 64, j1, stage(ring, u), &kvfull[ring][s],
                              [&](int from, int to) { return a.window <= 0 || from < a.n_sink || to > x.p0 - a.window; });
        ++use[ring];
      };
      // K, then V, in the order in which the UMMA warps take them
      if constexpr (BOTH) {
        auto both = [&](int ring, int ti, int sub, int page) {
          load(ring, ti, sub, false, page);
          if (ok) load(ring, ti, sub, true);
        };
        int next0 = page_of(a, x, ta, 0, cnt, true), next1 = page_of(a, x, ta, 1, cnt, true);
        for (int i = 0; i < cnt && ok; i += 2) {
          const int page0 = next0, page1 = next1;
          next0 = page_of(a, x, ta, i + 2, cnt, true);
          next1 = page_of(a, x, ta, i + 3, cnt, true);
          if (SPLIT) {
            both(0, i, 0, page0);
            if (i + 1 < cnt && ok) both(1, i + 1, 0, page1);
            if (ok) both(0, i, 1, page0);
            if (i + 1 < cnt && ok) both(1, i + 1, 1, page1);
          } else {
            both(0, i, 0, page0);
            if (i + 1 < cnt && ok) both(0, i + 1, 0, page1);
          }
        }
      } else if (SPLIT) {
        for (int i = 0; i < cnt && ok; i += 2)
          for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              if (i + w >= cnt) break;
              load(w, i + w, sub, false);
              if (ok) load(w, i + w, sub, true);
            }
      } else {
        for (int i = 0; i < cnt && ok; ++i) {
          load(0, i, 0, false);
          if (ok) load(0, i, 0, true);
        }
      }
    }
    // copies in flight land, and the last releases arrive, before the CTA ends
    if (lane == 0) {
#pragma unroll
      for (int r = 0; r < nring; ++r)
        for (int u = max(0, use[r] - kStages); u < use[r]; ++u)
          if (!BOTH || (u & 1) == 0)                 // (V's are not this warp's)
            mbar_drain(&kvfull[r][u % kStages], (u / kStages) & 1, a.wc.status);
      if (piece) mbar_drain(&qfull, (piece - 1) & 1, a.wc.status);
      if (ok) {
#pragma unroll
        for (int r = 0; r < nring; ++r) ring_tail(kvempty[r], kStages, use[r], &s_abort, a.wc);
        ring_tail(&qempty, 1, piece, &s_abort, a.wc);
      }
    }
  } else if (BOTH && warp == kLoadWarp + 1) {
    load_values<SPLIT, TREE>(a, sh, &tv, sKV, kvfull, vroom, &s_abort);
  } else if (warp >= kQkWarp && warp < kLoadWarp) {
    // the whole warp follows the loop and one elected lane issues, so that descriptors stay in
    // uniform registers
    const int w = warp & 1;
    const bool is_qk = warp < kPvWarp;
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 64);
    constexpr uint32_t idesc_o = idesc_bf16_f32(128, 128) | (1u << 16);   // B (V) MN-major
    int use = 0, piece = 0, g = 0;                   // ring uses before this piece; pieces; steps
    bool ok = true;                                  // the same in every lane
    auto wait = [&](uint64_t* bar, int phase) {
      ok = __all_sync(0xffffffffu, ok && mbar_wait(bar, static_cast<uint32_t>(phase & 1), &s_abort, a.wc));
    };
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) umma_commit(bar);
      __syncwarp();
    };
    const uint64_t qd = sdesc_kmajor_sw128(smem_u32(sQ + (SPLIT ? 0 : w) * kTile));
    const int ring = SPLIT ? w : 0;
    const StageLayout lay = stage_layout(a, kStageRows);
    const uint32_t base0 = smem_u32(stage(ring, 0));
    const uint64_t kd0 = sdesc_stage_k(base0, lay), vd0 = sdesc_stage_v(base0, lay);
    const uint32_t sub_step = (8 * lay.group) >> 4, k_step = (2 * lay.group) >> 4, khalf = lay.half >> 4;   // 64 rows, 16 rows
    const uint32_t tS = tbase + w * 128, tO = tbase + 256 + w * 128;
    long long base = sh.item_base;
    for (int item = sh.item; ok && base < sh.end; ++item) {
      const ItemRange x = item == sh.item ? sh.first : item_range<kTK, TREE>(a, item);
      int ta, tb;
      if (!next_piece(sh, item, x, base, ta, tb)) continue;
      const int cnt = tb - ta;
      const int steps = 2 * (SPLIT ? (cnt + 1 - w) / 2 : cnt);   // of this stream: key tile n / 2, buffer n & 1
      if (is_qk) {
        wait(&qfull, piece);
        for (int n = 0; n < steps && ok; ++n, ++g) {
          const int u = n & 1, k = use + (SPLIT ? 2 * n : 2 * (n >> 1));   // ring use of the K rows
          if (SPLIT || u == 0) wait(&kvfull[ring][k % kStages], k / kStages);
          // the buffer is free when the product that read the last P in it is done
          if (g >= 2) wait(&pv[w][u], (g >> 1) - 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = kd0 + (k % kStages) * (kStageBytes >> 4) + (SPLIT ? 0 : u) * sub_step;
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t in = ((i & 3) * 32) >> 4;
              umma_bf16(tS + u * 64, qd + (i >> 2) * (kHalf >> 4) + in, kd + (i >> 2) * khalf + in, idesc_s, i ? 1u : 0u);
            }
            umma_commit(&sfull[w][u]);
            if (SPLIT || u == 1) umma_commit(&kvempty[ring][k % kStages]);
          }
          __syncwarp();
        }
        if (ok) commit(&qempty);
      } else {
        for (int n = 0; n < steps && ok; ++n, ++g) {
          const int u = n & 1, v = use + (SPLIT ? 2 * n : 2 * (n >> 1)) + 1;
          if (SPLIT || u == 0) wait(&kvfull[ring][v % kStages], v / kStages);
          wait(&pfull[w][u], g >> 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = vd0 + (v % kStages) * (kStageBytes >> 4) + (SPLIT ? 0 : u) * sub_step;
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              umma_bf16_ta(tO, tS + u * 64 + i * 8, vd + i * k_step, idesc_o, (n == 0 && i == 0) ? 0u : 1u);
            umma_commit(&pv[w][u]);
            if (SPLIT || u == 1) umma_commit(&kvempty[ring][v % kStages]);
          }
          __syncwarp();
        }
      }
      ++piece;
      use += SPLIT ? 2 * steps : 2 * cnt;
    }
    // every product issued has been done before TMEM is freed
    commit(&done);
    if (lane == 0 && warp == kQkWarp) mbar_drain(&done, 0, a.wc.status);
  } else if (warp < kQkWarp) {
    regs_up<kSoftRegs>();
    const int w = warp >> 2, row = threadIdx.x & 127;   // stream, query row within the block (TMEM lane)
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS0 = tbase + w * 128 + lanes, tO = tbase + 256 + w * 128 + lanes;
    // steps of this stream; ring uses before this piece; exchanges; tiles with unseen rows
    int g = 0, use = 0, nx = 0, nfix = 0;
    bool ok = true;                                  // the same in every lane of a warp
    auto wait = [&](uint64_t* bar, int phase) {
      // (the test alone is cheaper than a try_wait that succeeds)
      if (__all_sync(0xffffffffu, ok && mbar_test(bar, static_cast<uint32_t>(phase & 1)))) return;
      ok = __all_sync(0xffffffffu, ok && mbar_wait(bar, static_cast<uint32_t>(phase & 1), &s_abort, a.wc));
    };
    long long base = sh.item_base;
    for (int item = sh.item; ok && base < sh.end; ++item) {
      const ItemRange x = item == sh.item ? sh.first : item_range<kTK, TREE>(a, item);
      int ta, tb;
      if (!next_piece(sh, item, x, base, ta, tb)) continue;
      const int cnt = tb - ta;
      const int first_row = SPLIT ? 0 : w * block;   // of the item
      const int rows = min(block, x.rows - first_row);
      const int rr = x.rt * a.tr + first_row + row;  // row of the segment
      const int tree0 = x.n - x.m;                   // TREE: the first row of the tree
      const uint32_t* mask = TREE ? tree_mask(a, x.b, row < rows ? a.by_G(rr) : 0) : nullptr;
      const TreeRow node = TREE ? tree_row<TREE>(a, mask, x.m, tree0) : TreeRow{};
      const int p = TREE ? node.p : a.causal ? x.n - x.m + a.by_G(rr) : x.n - 1;
      // cache rows of the block's first and last token (TREE: all see the rows up to pa; none is behind pb)
      const int pa = TREE ? tree0 - 1 : a.causal ? x.n - x.m + a.by_G(x.rt * a.tr + first_row) : x.n - 1;
      const int pb = TREE ? x.p1 : a.causal ? x.n - x.m + a.by_G(x.rt * a.tr + first_row + max(rows, 1) - 1) : x.n - 1;
      float ref = -INFINITY, sum = 0.f;
      int mine = 0;                                  // steps of this piece so far
      const int steps = 2 * (SPLIT ? (cnt + 1 - w) / 2 : cnt);
      for (; mine < steps; ++mine, ++g) {
        const int u = mine & 1, i = SPLIT ? (mine & ~1) + w : mine >> 1;   // buffer; tile of the piece
        const uint32_t tS = tS0 + u * 64;
        int j0, j1;
        tile_rows<kTK>(x, ta + i, j0, j1);
        const int js = j0 + u * 64;                  // first key of the step
        wait(&sfull[w][u], g >> 1);
        if (!ok) break;
        tc_fence_after();
        __syncwarp();                                // (the TMEM instructions want a converged warp)
        float s[64];
        tmem_ld32(tS, s);
        tmem_ld32(tS + 32, s + 32);
        tmem_ld_wait();
        const bool whole = js + 64 <= j1 && (!a.causal || (js + 64 <= pa + 1 &&
                                                           (a.window <= 0 || js > pb - a.window || js + 64 <= a.n_sink)));
        if (TREE && !whole) {
          // columns before the tree: below `hi`, and not in [first, lo); the others by the node's mask, but for those that
          // the window hides
          const int hi = min(j1, tree0) - js;
          const int lo = a.window > 0 ? p - a.window + 1 - js : 0, first = a.window > 0 ? a.n_sink - js : 0;
          uint64_t see = (low_bits(hi) & ~(low_bits(lo) & ~low_bits(first))) |
                         (js + 64 > tree0 ? tree_bits(mask, x.m, js - tree0) & low_bits(j1 - js) : 0);
          if (TREE == kWindowed)                     // (columns before the tree are not among those)
            see &= ~(low_bits(node.from - (js - tree0)) & ~low_bits(node.first - (js - tree0))) | low_bits(tree0 - js);
          const uint32_t see0 = static_cast<uint32_t>(see), see1 = static_cast<uint32_t>(see >> 32);
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!((c < 32 ? see0 : see1) >> (c & 31) & 1u)) s[c] = -INFINITY;
        } else if (!whole) {
          // a row sees columns [0, hi) and, with a window, of these [lo, hi) and those below `first`
          const int hi = min(j1, a.causal ? p + 1 : j1) - js;
          const int lo = a.window > 0 ? p - a.window + 1 - js : -1, first = a.window > 0 ? a.n_sink - js : 0;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c >= hi || (c < lo && c >= first)) s[c] = -INFINITY;
        }
        float t0 = s[0], t1 = s[1], t2 = s[2], t3 = s[3];
#pragma unroll
        for (int c = 4; c < 60; c += 8) {
          t0 = fmax3(t0, s[c], s[c + 1]);
          t1 = fmax3(t1, s[c + 2], s[c + 3]);
          t2 = fmax3(t2, s[c + 4], s[c + 5]);
          t3 = fmax3(t3, s[c + 6], s[c + 7]);
        }
        t0 = fmax3(t0, s[60], s[61]);
        t1 = fmax3(t1, s[62], s[63]);
        const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * a.s2;
        if (__any_sync(0xffffffffu, top > ref + kSlack)) {
          // each row by its own maximum: a result does not depend on the rows next to it
          const float r2 = top > ref + kSlack ? top : ref;
          const float f = ref == -INFINITY ? 0.f : exp2f(ref - r2);
          ref = r2;
          sum *= f;
          if (mine > 0) {
            // after the product of the step before, the last that writes O until this P is there
            wait(&pv[w][u ^ 1], (g - 1) >> 1);
            if (!ok) break;
            tc_fence_after();
            __syncwarp();
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
        __syncwarp();
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 32) {
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
        // rows become zero before the tile's first product reads them.  Without SPLIT stream 0 does
        // it for both; it is at most two tiles ahead, so four barriers in turn tell stream 1.
        const int jv = SPLIT ? js : j0;              // rows of the V stage
        if ((SPLIT || u == 0) &&
            (jv + kStageRows > j1 || (a.window > 0 && jv <= x.p0 - a.window && jv + kStageRows > a.n_sink))) {
          if (SPLIT || w == 0) {
            const int ring = SPLIT ? w : 0, uv = use + (SPLIT ? 2 * mine : 2 * i) + 1;
            wait(&kvfull[ring][uv % kStages], uv / kStages);
            if (!ok) break;
            // a thread a row, or a column half of one
            const int r = row & (kStageRows - 1);
            if (unseen(a, x, jv + r, j1)) {
              const StageLayout lay = stage_layout(a, kStageRows);
              uint8_t* d = stage(ring, uv) + (r >> 3) * lay.group + (r & 7) * 128;
#pragma unroll
              for (int hf = 0; hf < 2; ++hf)
                if (!SPLIT || hf == row >> 6)
#pragma unroll
                  for (int c = 0; c < 8; ++c)
                    *reinterpret_cast<uint4*>(d + hf * lay.half + c * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (!SPLIT && lane == 0) mbar_arrive(&vfix[nfix & 3]);
          } else {
            wait(&vfix[nfix & 3], nfix >> 2);
            if (!ok) break;
            fence_proxy_async_smem();
          }
          ++nfix;
        }
        __syncwarp();
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[w][u]);
        __syncwarp();
      }
      use += SPLIT ? 2 * steps : 2 * cnt;                                // a K and a V tile each

      // results of this piece
      const bool first = ta == 0, last = tb == x.tiles, direct = first && last;
      if (mine > 0) wait(&pv[w][1], (g - 1) >> 1);
      if (!ok) break;
      tc_fence_after();
      const bool live = row < rows && (!SPLIT || w == 0);
      const int slot = 2 * blockIdx.x + (first ? 1 : 0);
      // Results leave by quads of lanes, 64 bytes of four rows in turn (a row per thread took 6000 to
      // 12000 cycles for a piece: 32 lines touched by each store)
      const int q0 = row & ~3;
      float* po = a.part_o + (static_cast<long long>(slot) * a.tr + first_row + q0) * kHeadDim + (lane & 3) * 4;
      uint16_t* dst[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        dst[k] = direct ? out_row(a, x.b, x.h, x.rt * a.tr + first_row + q0 + k) + (lane & 3) * 8 : nullptr;
      float f0 = 1.f, f1 = 0.f, inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll 1
      for (int c0 = 0; c0 < 128; c0 += 32) {
        float y[32];
        __syncwarp();
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
        if (!SPLIT || w == 0) {
          uint4 v[4];
          if (direct) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float* z = y + c * 8;
              v[c] = make_uint4(pack_bf16(z[0] * inv, z[1] * inv), pack_bf16(z[2] * inv, z[3] * inv),
                                pack_bf16(z[4] * inv, z[5] * inv), pack_bf16(z[6] * inv, z[7] * inv));
            }
            quad_transpose(v);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (q0 + k < rows) *reinterpret_cast<uint4*>(dst[k] + c0) = v[k];
          } else {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const float* z = y + hf * 16 + c * 4;
                v[c] = make_uint4(__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3]));
              }
              quad_transpose(v);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (q0 + k < rows) *reinterpret_cast<uint4*>(po + k * kHeadDim + c0 + hf * 16) = v[k];
            }
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
      if (first) rec_first(a, item, last ? 0 : last_cta(sh, base) - static_cast<int>(blockIdx.x));
      tc_fence_before();                             // O is read before the next piece's products
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kQkWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

}  // namespace

int attend_tile_rows(bool split) { return split ? 64 : 128; }

// Whether every item, of `tiles` tiles at most, goes to one CTA.  The plan, pieces of two kinds and the
// join cost 5 us with one block of query rows and 8 with two, and the work is cut over all CTAs;
// whole items take 2.45 us per two tiles (1.63 per tile), however few there are.  The rule follows
// these, with three quarters of the items counted (caches of one batch differ in length, and only a
// bound is known here).  Measured, group 4, plan and whole items, 6 tokens: 8 items of 256 rows 12.9
// and 10.4 us, of 1024 13.4 and 17.6; 128 items of 1024 29.2 and 18.2, of 3000 47 and 39.7; 512 tokens:
// 64 items of 768 rows 22.1 and 19.2, of 1536 26.1 and 29.1; 128 items of 1536 36.6 and 29.5.
bool attend_tile_whole(long long items, long long tiles, bool split, int grid) {
  if (items > grid) return false;
  const long long serial = split ? (tiles + 1) / 2 : tiles;
  return split ? serial <= 12 && serial * (100 - items * 7 / 10) <= 240
               : serial <= 32 && serial * (100 - items * 6 / 10) <= 550;
}

// Whether K and V come by a warp each: from pages of less than a stage's 64 rows.  The sizes above, two warps and one: pages
// of 8 133 and 151 us, of 16 125 and 150, of 32 126 and 127 (16 nodes 119 and 127), of 64 125 and 121 (contiguous rows, one
// warp, 115).
static bool attend_tile_both(const AttnArgs& a) { return a.src.paged && a.src.block_size < 64; }

template <int TREE>
static auto tree_kernel(bool split, bool both) {
  return both ? (split ? attend_tile_kernel<true, TREE, true> : attend_tile_kernel<false, TREE, true>)
              : (split ? attend_tile_kernel<true, TREE, false> : attend_tile_kernel<false, TREE, false>);
}

cudaError_t launch_attend_tile(const AttnArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               int block, bool split, int grid, cudaStream_t st) {
  const auto kernel = !a.tree         ? (split ? attend_tile_kernel<true, kCausal, false> : attend_tile_kernel<false, kCausal, false>)
                      : a.tree_window ? tree_kernel<kWindowed>(split, attend_tile_both(a))
                                      : tree_kernel<kMasks>(split, attend_tile_both(a));
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kernel), kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<a.whole ? a.B * a.H * a.rt : grid, kThreads, kSmem, st>>>(tq, tk, tv, a, block);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess || a.whole) return e;
  return launch_attend_join(a, grid, st);
}

}  // namespace kvsel
