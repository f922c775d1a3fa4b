// Shared by the kernels of kvsel_attend: the arguments, the key range that a block of query
// rows sees, and the division of all (block, key tile) pairs over the grid.
//
// Query rows of a segment (request b, KV head h) are numbered r = t * G + g: token t of the
// request's new tokens, member g of the head's group.  An item is a block of TR rows of one
// segment; it is worked through in tiles of TK cached rows.
#pragma once
#include "internal.cuh"

namespace kvsel {

// Division of 0 <= n < 2^31 by a number known at the launch: n * m >> p with p = 31 + ceil(log2 d) and
// m = ceil(2^p / d), exact for these n.  (The plan of a call is a chain of divisions.)
struct Div {
  unsigned int m;
  int p;
  __host__ static Div by(int d) {
    Div x;
    int k = 0;
    while ((1ll << k) < d) ++k;
    x.p = 31 + k;
    x.m = static_cast<unsigned int>(((1ull << x.p) + d - 1) / d);
    return x;
  }
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>((static_cast<unsigned long long>(n) * m) >> p);
  }
};

struct AttnArgs {
  int B, H, G, m;                 // requests, KV heads, group, new tokens of a request at most
  Div by_rt, by_H, by_G;          // items per segment, heads, group
  // weights_tile_kernel: blocks of 256 cached rows of a segment that some query row may see; with a window
  // that is shorter than a segment, first those of the first rows that stay visible (-1: all blocks)
  int kb, kb_sink;
  Div by_kb;
  int page_shift;                 // paged: log2 of the rows of a page
  int max_len;                    // rows of a segment at most
  int causal, window, n_sink;
  int per_head;                   // lens [B*H] instead of [B]
  float s2;                       // logit scale * log2(e)
  const int32_t* lens;
  const int32_t* new_lens;        // [B] or null: m for every request
  const int64_t* offsets;         // packed cache: first row of every segment
  long long n_rows;               // packed cache: rows in all
  const uint16_t* q;
  long long q_req, q_head, q_tok;
  uint16_t* out;
  long long o_req, o_head, o_tok;
  float* lse;                     // [B][H*G][m] natural log, or null
  float* lse2;                    // [B][H][m*G] log2 units, for the weights, or null
  float* logits;                  // [B*H][m*G][logit_stride], log2 units, masked: -inf (m*G <= 16), or null
  long long logit_stride;
  float* acc;                     // [B*H][acc_stride] or null
  long long acc_stride;
  KvSource src;
  const uint16_t* k;
  const uint16_t* v;
  long long stride_req, stride_head, stride_tok;
  int tr;                         // query rows of an item
  int rt;                         // items per segment
  // partial results of items that several CTAs share: two slots per CTA
  float* part_o;                  // [2 * grid][rows][128]
  float2* part_ml;                // [2 * grid][rows]: reference (log2 units) and sum
// who joins what.  by_item (fewer items than CTAs): rec[item] = {CTA of the first piece, or -1 when
  // the item is done, CTAs that follow}; else rec[CTA] = {item that starts there and goes on, or
  // -1, CTAs that follow}
  int2* rec;                      // [grid]
  int by_item;
  int whole;                      // attend_tile_kernel: a CTA per item, no plan, no join
  int grid;                       // CTAs of the kernel that works on the items
  WaitCtl wc;
};

// Whether rows [row0, row0 + n) lie in a packed cache of n_rows rows, whatever the caller's row0 is (the
// sum row0 + n could pass 64 bits).
__host__ __device__ constexpr bool segment_fits(long long row0, int n, long long n_rows) {
  return row0 >= 0 && row0 <= n_rows - n;
}
static_assert(segment_fits(0, 8, 8) && segment_fits(8, 0, 8) && !segment_fits(1, 8, 8) && !segment_fits(0, 9, 8));
static_assert(!segment_fits(-1, 0, 8) && !segment_fits(0x7FFFFFFFFFFFFFFFll, 1, 8));

// Rows of segment (b, h) and new tokens of request b, as the caller's device arrays give them;
// values out of range are flagged and clamped.
struct SegLen {
  int n, m;
  long long row0;                 // packed cache: first row
};
__device__ __forceinline__ SegLen seg_len(const AttnArgs& a, int b, int h) {
  SegLen s;
  const int raw = __ldg(a.lens + (a.per_head ? b * a.H + h : b));
  s.n = min(max(raw, 0), a.max_len);
  const int mr = a.new_lens ? __ldg(a.new_lens + b) : a.m;
  s.m = min(max(mr, 0), a.m);
  bool bad = s.n != raw || s.m != mr;
  s.row0 = 0;
  if (a.offsets) {
    s.row0 = __ldg(a.offsets + b * a.H + h);
    if (!segment_fits(s.row0, s.n, a.n_rows)) {
      bad = true;
      s.n = 0;
      s.row0 = 0;
    }
  }
  if (bad) atomicOr(a.wc.status, DEV_BAD_INDEX);
  return s;
}

// Key tiles of an item.  A row block sees [0, sink) and [lo, hi) of the cached rows (some row
// of it does); tiles [0, ns) cover the first range, the others [lo, hi).  Where the two
// meet, or without a window, lo = 0 and ns = 0.
struct ItemRange {
  int seg, b, h, rt;
  int n, m;                       // cached rows, new tokens
  int rows;                       // valid query rows of the block
  int p0, p1;                     // cache row of the block's first and last token
  int lo, hi, sink, ns, tiles;
  int skip;                       // the last of the segment's items where this and all behind it are empty, else the item
  long long row0;
};
template <int TK>
__device__ __forceinline__ ItemRange item_range(const AttnArgs& a, int item) {
  ItemRange x;
  const int TR = a.tr;
  x.seg = a.by_rt(item);
  x.rt = item - x.seg * a.rt;
  x.b = a.by_H(x.seg);
  x.h = x.seg - x.b * a.H;
  const SegLen s = seg_len(a, x.b, x.h);
  x.n = s.n;
  x.m = s.m;
  x.row0 = s.row0;
  const int R = s.m * a.G, r0 = x.rt * TR;
  x.rows = min(TR, R - r0);
  x.lo = x.ns = x.sink = x.hi = x.tiles = x.p0 = x.p1 = 0;
  x.skip = item;
  if (x.rows <= 0) {
    x.rows = 0;
    x.skip = item - x.rt + a.rt - 1;
    return x;
  }
  if (a.causal) {
    x.p0 = s.n - s.m + a.by_G(r0);
    x.p1 = s.n - s.m + a.by_G(r0 + x.rows - 1);
    x.hi = max(0, x.p1 + 1);
  } else {
    x.p0 = x.p1 = s.n - 1;
    x.hi = s.n;
  }
  if (a.window > 0) {
    const int lo = max(0, x.p0 - a.window + 1);
    // pages behind the window may be gone: a tile starts with the first page that is seen; at an
    // even row otherwise (two logits are kept at a time)
    const int al = lo & -(a.src.paged ? 1 << a.page_shift : 2);
    const int sink = min(a.n_sink, x.hi);
    const int ns = (sink + TK - 1) / TK;
    if (lo > sink && al > ns * TK) {
      x.lo = al;
      x.sink = sink;
      x.ns = ns;
    }
  }
  // a block that sees nothing (fewer rows than new tokens) still has its empty result to write
  x.tiles = max(1, x.ns + (x.hi - x.lo + TK - 1) / TK);
  return x;
}
// First row of tile ti and the end of the rows that it covers.
template <int TK>
__device__ __forceinline__ void tile_rows(const ItemRange& x, int ti, int& j0, int& j1) {
  if (ti < x.ns) {
    j0 = ti * TK;
    j1 = x.sink;
  } else {
    j0 = x.lo + (ti - x.ns) * TK;
    j1 = x.hi;
  }
}

// The share of CTA `cta` of the grid in all tiles of all items, in item order: units
// [total * cta / grid, total * (cta + 1) / grid).  An item has `start` units for what beginning it
// costs, then one per tile; a CTA whose share ends within the former leaves it to the next.
// Lengths live on the device, so every CTA adds up the items itself (a thread takes consecutive
// items, then a block-wide scan).
template <class Item>
struct Share {
  long long total;
  long long begin, end;           // this CTA's units
  int grid;                       // CTAs with work: min(gridDim.x, total)
  int start;
  int item;                       // item of unit `begin`
  long long item_base;            // its first unit
  Item first;                     // and its range
};
// SKIP: segments may end in many empty items (64 tokens of four requests of 2000 rows with weights, where
// max_len is 128000: 190 us without it, 68 with it; one item per segment: 0.3 us more).
// whole: item `cta` and nothing else.
// range(i): the range of item i, with its number of tiles.  The result stays in shared memory; kept in
// registers through attend_tile_kernel it costs the softmax warps' inner loop 2% (spills).
template <int THREADS, bool SKIP = true, class Range>
__device__ __forceinline__ auto share_of(int items, Range range, int cta, int start = 0, bool whole = false)
    -> const Share<decltype(range(0))>& {
  using Item = decltype(range(0));
  const auto units = [&](const Item& x) { return x.tiles > 0 ? x.tiles + start : 0; };
  __shared__ long long s_warp[THREADS / 32];
  __shared__ Share<Item> s_sh;
  if (whole) {
    if (threadIdx.x == 0) {
      const Item x = range(cta);
      s_sh.total = s_sh.end = x.tiles;
      s_sh.begin = s_sh.item_base = 0;
      s_sh.grid = gridDim.x;
      s_sh.start = 0;
      s_sh.item = cta;
      s_sh.first = x;
    }
    __syncthreads();
    return s_sh;
  }
  const int per = (items + THREADS - 1) / THREADS;
  const int i0 = min(items, static_cast<int>(threadIdx.x) * per), i1 = min(items, i0 + per);
  long long sum = 0;
  Item mine{};                                       // the last of this thread's items (the only one, as a rule)
  for (int i = i0; i < i1; ++i) {
    mine = range(i);
    sum += units(mine);
    if (SKIP) i = mine.skip;
  }
  long long inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if ((threadIdx.x & 31) >= o) inc += y;
  }
  if ((threadIdx.x & 31) == 31) s_warp[threadIdx.x >> 5] = inc;
  __syncthreads();
  long long before = inc - sum, total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < static_cast<int>(threadIdx.x >> 5)) before += s_warp[w];
    total += s_warp[w];
  }
  const int grid = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
  if (threadIdx.x == 0) s_sh.grid = grid;
  if (cta < grid) {
    const long long begin = total * cta / grid;
    if (sum > 0 && begin >= before && begin < before + sum) {
      long long at = before;
      int i = i0;
      if (per > 1) {
        for (; i < i1; ++i) {
          mine = range(i);
          if (begin < at + units(mine)) break;
          at += units(mine);
          if (SKIP) i = mine.skip;
        }
      }
      s_sh.total = total;
      s_sh.begin = begin;
      s_sh.end = total * (cta + 1) / grid;
      s_sh.start = start;
      s_sh.item = i;
      s_sh.item_base = at;
      s_sh.first = mine;
    }
  }
  __syncthreads();
  return s_sh;
}
// The tiles [ta, tb) of an item that this CTA works on; `base`, the item's first unit, moves to the next
// item's, and `item` over empty ones behind it.  False: none.
template <bool SKIP = true, class Item>
__device__ __forceinline__ bool next_piece(const Share<Item>& sh, int& item, const Item& x, long long& base, int& ta,
                                           int& tb) {
  if (x.tiles == 0) {
    if (SKIP) item = x.skip;
    return false;
  }
  ta = item == sh.item ? max(0, static_cast<int>(sh.begin - base) - sh.start) : 0;
  tb = static_cast<int>(min(static_cast<long long>(x.tiles), sh.end - base - sh.start));
  base += x.tiles + sh.start;
  return ta < tb;
}
// The last CTA with a unit of an item that ends before unit `e`.
template <class Item>
__device__ __forceinline__ int last_cta(const Share<Item>& sh, long long e) {
  return static_cast<int>((e * sh.grid - 1) / sh.total);
}

// Records for the join: at a kernel's start, and by the CTA that works on an item's first tile
// (`follow` CTAs work on the others).
__device__ __forceinline__ void rec_clear(const AttnArgs& a) {
  if (threadIdx.x == 0 && !a.by_item) a.rec[blockIdx.x] = make_int2(-1, 0);
}
__device__ __forceinline__ void rec_first(const AttnArgs& a, int item, int follow) {
  if (threadIdx.x != 0) return;
  if (a.by_item)
    a.rec[item] = make_int2(follow > 0 ? static_cast<int>(blockIdx.x) : -1, follow);
  else if (follow > 0)
    a.rec[blockIdx.x] = make_int2(item, follow);
}

// How far (log2 units) a row's running maximum may rise above the reference that its weights are
// scaled by before sum and accumulator are rescaled.  Floating point loses nothing by the scale; 16
// leaves 2^94 for the values at 2^17 rows.  (8 rescaled in one step of eight on keys of log-normal
// norms, 750 cycles each.)
constexpr float kSlack = 16.f;

// whether row p sees cached row j (j < hi of its tile)
__device__ __forceinline__ bool sees(const AttnArgs& a, int p, int j) {
  if (!a.causal) return true;
  return j <= p && (a.window <= 0 || j > p - a.window || j < a.n_sink);
}
// element offset of cached row j, or -1 (a block-table entry out of range)
__device__ __forceinline__ long long row_elem(const AttnArgs& a, int b, int h, long long row0, int j) {
  if (!a.src.paged)
    return b * a.stride_req + h * a.stride_head + (row0 + static_cast<long long>(j)) * a.stride_tok;
  const int page = j >> a.page_shift;
  const int pb = __ldg(a.src.block_table + static_cast<size_t>(b) * a.src.max_blocks + page);
  if (pb < 0 || pb >= a.src.num_blocks) return -1;
  return (((static_cast<long long>(pb) << a.page_shift) + (j - (page << a.page_shift))) * a.H + h) * kHeadDim;
}

// a row that no cached row is read for: behind the tile's end, or before the window of the
// item's first token (and not among the first rows that stay visible)
__device__ __forceinline__ bool unseen(const AttnArgs& a, const ItemRange& x, int j, int j1) {
  return j >= j1 || (a.window > 0 && j >= a.n_sink && j <= x.p0 - a.window);
}

// Log-sum-exp of query row rr of a segment from its reference M (log2 units) and sum L.
__device__ __forceinline__ void write_lse(const AttnArgs& a, int b, int h, int rr, float M, float L) {
  const int t = a.by_G(rr), g = rr - t * a.G;
  const float e2 = L > 0.f ? M + log2f(L) : -INFINITY;
  if (a.lse) a.lse[(static_cast<long long>(b) * a.H * a.G + h * a.G + g) * a.m + t] = e2 * 0.6931471805599453f;
  if (a.lse2) a.lse2[static_cast<long long>(b * a.H + h) * a.m * a.G + rr] = e2;
}
__device__ __forceinline__ uint16_t* out_row(const AttnArgs& a, int b, int h, int rr) {
  const int t = a.by_G(rr), g = rr - t * a.G;
  return a.out + b * a.o_req + static_cast<long long>(h * a.G + g) * a.o_head + static_cast<long long>(t) * a.o_tok;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// K and V stages of the UMMA kernels, 128-byte swizzle: atoms of 8 rows x 64 columns (1024 B).
// Contiguous and packed caches: the atoms of columns 0-63, then those of columns 64-127.
// Paged: the two atoms of 8 rows side by side, so that one box brings a page whole.  (A box costs
// about 53 cycles beyond 5 per 128-byte row: with a box per page and column half, 16-row pages
// came at 4300 cycles per K and V tile, and 16-byte copies by four warps at 4900.)
constexpr int kTileBytes = 128 * 256;                // one 128 x 128 bf16 tile
constexpr int kHalfBytes = 128 * 128;                // its 64-column half
struct StageLayout {
  uint32_t group, half;                              // bytes to the next 8 rows, to the other 64 columns
};
__device__ __forceinline__ StageLayout stage_layout(const AttnArgs& a, int rows) {
  return a.src.paged ? StageLayout{2048u, 1024u} : StageLayout{1024u, rows * 128u};
}
// K-major operand in such a stage
__device__ __forceinline__ uint64_t sdesc_stage_k(uint32_t saddr, const StageLayout& l) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1u) << 16;
  d |= static_cast<uint64_t>(l.group >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                            int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}
// ROWS (64 or 128) rows of a segment from row j0 (those below j1) into such a stage, by the lanes of
// a warp.  seen(first, last): whether any row of a page is seen; other pages are not looked up.
template <int ROWS, class Seen>
__device__ __forceinline__ void load_rows(const AttnArgs& a, int b, int h, long long row0, const CUtensorMap* map,
                                          int j0, int j1, uint8_t* dst, uint64_t* bar, Seen seen) {
  const int lane = lane_id();
  if (!a.src.paged) {
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, ROWS * 256);
      const int row = static_cast<int>(row0) + j0;
      tma_load_4d(dst, map, bar, 0, row, a.offsets ? 0 : h, a.offsets ? 0 : b);
      tma_load_4d(dst + ROWS * 128, map, bar, 64, row, a.offsets ? 0 : h, a.offsets ? 0 : b);
    }
    return;
  }
  const int bs = a.src.block_size, at = j0 + lane * bs;   // lane i: page i of the rows
  const bool live = lane < (ROWS >> a.page_shift) && at < j1 && seen(at, at + bs - 1);
  int pb = 0;
  if (live) {
    pb = __ldg(a.src.block_table + static_cast<size_t>(b) * a.src.max_blocks + (at >> a.page_shift));
    if (pb < 0 || pb >= a.src.num_blocks) {
      atomicOr(a.wc.status, DEV_BAD_INDEX);
      pb = a.src.num_blocks;                         // outside the pool: zeros
    }
  }
  const unsigned pages = __popc(__ballot_sync(0xffffffffu, live));
  if (lane == 0) mbar_arrive_expect_tx(bar, pages * bs * 256);
  __syncwarp();
  // the last dimension counts rows of the pool: (block, slot 0, head)
  if (live) tma_load_5d(dst + lane * bs * 256, map, bar, 0, 0, 0, 0, pb * (bs * a.H) + h);
  __syncwarp();
}
// one lane of a converged warp, the same one every time
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// a few rows per item (a.tr = attend_rows_tile())
cudaError_t launch_attend_rows(const AttnArgs& a, int grid, int cluster, cudaStream_t st);
int attend_rows_cluster(long long items, long long tiles, bool window, int grid);
int attend_rows_tile();
bool attend_tile_whole(long long items, long long tiles, bool split, int grid);
int attend_tile_rows(bool split);  // rows of a K/V stage, and of a box of its maps
int attend_rows_ctas_per_sm();
// tcgen05 tiles: two blocks of `block` query rows per item that share the cached rows, or, with
// `split`, one block whose even and odd key tiles run side by side
cudaError_t launch_attend_tile(const AttnArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               int block, bool split, int grid, cudaStream_t st);
// joins the pieces of items that several CTAs of either kernel share
cudaError_t launch_attend_join(const AttnArgs& a, int grid, cudaStream_t st);
// acc += the weights of every cached row: from the logits that attend_rows_kernel kept ...
cudaError_t launch_weights_kept(const AttnArgs& a, cudaStream_t st);
// ... or from Q K^T formed again on tcgen05 (rec, part_ml as for the tile kernel: they are free
// again; part: [2 * grid][256])
cudaError_t launch_weights_tile(const AttnArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, int block, float* part,
                                int grid, cudaStream_t st);

}  // namespace kvsel
