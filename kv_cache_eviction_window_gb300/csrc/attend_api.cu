// C-ABI host layer of the calls that use a cache after its compaction: attention of new
// tokens (kvsel_attend) and eviction by accumulated weight (kvsel_evict_append).  Argument
// validation, workspace layout and launches; nothing here allocates memory.
#include <algorithm>
#include <cmath>

#include "../../include/kvsel.h"
#include "attend.cuh"
#include "evict.cuh"

using namespace kvsel;

namespace {

constexpr unsigned long long kDefaultWaitCycles = 2000000000ull;   // ~1 s at the boost clock
constexpr long long kMaxRows = 1ll << 30;
constexpr int kMaxSegments = 65535;                  // a grid dimension

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int launch_rc(cudaError_t e) { return e == cudaSuccess ? KVSEL_OK : KVSEL_ECUDA; }

int device_sms(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KVSEL_ECUDA;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return KVSEL_ECUDA;
  return KVSEL_OK;
}

struct AttnPlan {
  int grid = 0, tr = 0, rt = 1;
  bool tiled = false, split = false;
  bool few = false;              // a tree: up to 16 query rows, cut over the grid
  int block = 0;                 // tiled: query rows per block, whole tokens of the group
  int cluster = 0;               // not tiled: attend_rows_cluster
  bool whole = false;            // tiled: attend_tile_whole
  int kb = 1, kb_sink = -1;      // tiled, with weights: blocks of 256 cached rows (attend.cuh)
  size_t rec = 0, ml = 0, o = 0, lse2 = 0, wpart = 0, logits = 0, total = 0;
  long long logit_stride = 0;
};

// a stride matters only where its dimension has more than one entry
bool bad_stride(long long s, long long extent) { return extent > 1 && (s <= 0 || s % 8 != 0); }

int check_attn(const kvsel_attn_params* p) {
  if (!p) return KVSEL_EINVAL;
  if (p->head_dim != kHeadDim) return KVSEL_EUNSUPPORTED;
  if (p->h_kv < 1 || p->h_kv > 64 || p->group < 1 || p->batch < 1 || p->n_new < 1 || p->max_len < 1) return KVSEL_EINVAL;
  if (p->group > KVSEL_MAX_ATTN_GROUP || p->batch > KVSEL_MAX_ATTN_BATCH) return KVSEL_EUNSUPPORTED;
  if (p->batch * p->h_kv > kMaxSegments) return KVSEL_EUNSUPPORTED;
  if (p->n_new > (1 << 20) || p->max_len > kMaxRows) return KVSEL_EUNSUPPORTED;
  if (static_cast<long long>(p->n_new) * p->group * p->h_kv * p->batch > kMaxRows) return KVSEL_EUNSUPPORTED;
  if (p->n_rows > (1ll << 31) - 1) return KVSEL_EUNSUPPORTED;
  if (p->causal < 0 || p->causal > 1 || p->lens_per_head < 0 || p->lens_per_head > 1) return KVSEL_EINVAL;
  if (p->window < 0 || p->window > kMaxRows || p->n_sink < 0 || p->n_sink > kMaxRows) return KVSEL_EINVAL;
  if (p->window > 0 && !p->causal) return KVSEL_EUNSUPPORTED;
  if (!(p->scale >= 0.f) || std::isinf(p->scale) || p->n_rows < 0 || p->acc_stride < 0) return KVSEL_EINVAL;
  const long long hq = static_cast<long long>(p->h_kv) * p->group;
  if (p->q_stride_req || p->q_stride_head || p->q_stride_tok)
    if (bad_stride(p->q_stride_req, p->batch) || bad_stride(p->q_stride_head, hq) || bad_stride(p->q_stride_tok, p->n_new))
      return KVSEL_EINVAL;
  if (p->o_stride_req || p->o_stride_head || p->o_stride_tok)
    if (bad_stride(p->o_stride_req, p->batch) || bad_stride(p->o_stride_head, hq) || bad_stride(p->o_stride_tok, p->n_new))
      return KVSEL_EINVAL;
  return KVSEL_OK;
}

int check_tree(const kvsel_attn_params* p) {
  const int rc = check_attn(p);
  if (rc) return rc;
  if (p->tree_window < 0 || p->tree_window > 1) return KVSEL_EINVAL;
  return !p->causal || p->n_new > KVSEL_MAX_TREE ? KVSEL_EUNSUPPORTED : KVSEL_OK;
}

// How the nodes of a tree go: in items of 16 rows by clusters of c CTAs (pl.cluster), each item of which reads the cache
// again, from L2; up to 16 rows cut over the grid and joined (pl.few); in items of 128 rows or two such blocks, whole ones
// to CTAs (pl.whole); or these cut over the grid and joined.  Up to 16 rows keep the softmax weights to 2^-16, as
// kvsel_attend's do, and so never go to the tile kernel, which rounds them to bf16 (384 segments of 8192 rows, 16 query rows:
// 203 us, whole items 268; of 800 rows with that max_len 34 and 55).  Otherwise the estimate, in tenths of a microsecond,
// follows what was measured (8 to 512 rows per segment, 1 to 128 segments of 128 to 4096 rows, pages of 16, masks included, us):
//   clusters  6.3 and 0.97 per tile of 64 rows, 7.8 and 1.06 where CTAs share an SM: 32 items of 1024 rows by clusters of
//             eight 10.0, of four 10.2, of two 14.6; 96 items by clusters of two 16.6; more clusters than fit at once lose
//   whole     8.4 and 2.45 per two tiles of 128 rows (one block), 8.6 and 1.7 per tile: 32 segments of 1024 rows 18.2
//   few       8.0 and the cache at 6.2 TB/s: 32 segments of 65536 rows 164.8
//   cut       17.0 and the cache at 6.3 TB/s or the products at 1.3 PFLOP/s: 8 segments of 1024 rows 15.5, 64 of 4096 43,
//             32 of 65536 182
// With more items than SMs whole ones go in waves, 3 us and the times above for each, and cut ones cost 8 us for each that a
// CTA has (5 for up to two tiles or of two blocks): 256 segments of 1024 rows, 32 query rows, 39.7 and 60.5; 512 of 256 rows
// 43.4 and 41.3; 176 of 4096 rows 89 and 79; 256 query rows 51.6 and 55.3, 54.4 and 50.5, 117 and 88.
// (Over those 210 shapes the calls take 1.11 times less than by the rules of kvsel_attend, and at most 15% more than by the
// best of the three.)
void plan_tree(const kvsel_attn_params* p, int sms, AttnPlan& pl) {
  const long long segs = static_cast<long long>(p->batch) * p->h_kv, R = static_cast<long long>(p->n_new) * p->group;
  // rows that a node may see, first ones and a window's apart
  long long rows = p->max_len;
  if (p->window > 0) rows = std::min(rows, p->n_sink + static_cast<long long>(p->window) + p->n_new + 128);
  double best;
  if (R <= attend_rows_tile()) {
    pl.few = true;
    best = 80.0 + segs * rows * 512.0 / 6.2e5;
  } else {
    const int block = 128 / p->group * p->group;
    const bool split = R <= block;
    const long long tiles = (rows + 127) / 128, items = segs * ((R + 2 * block - 1) / (2 * block));
    best = 170.0 + std::max(segs * rows * 512.0 / 6.3e5, segs * rows * R * 512.0 / 1.3e8);
    if (items > sms) best += (split && tiles > 2 ? 80.0 : 50.0) * items / sms;
    const double one = split ? 84.0 + 24.5 * ((tiles + 1) / 2) : 86.0 + 17.0 * tiles;
    const double each = items > sms ? 30.0 + one * ((items + sms - 1) / sms) : one;
    if (each < best) {
      best = each;
      pl.whole = true;
    }
  }
  const long long small = segs * ((R + attend_rows_tile() - 1) / attend_rows_tile()), steps = (rows + 63) / 64;
  for (int c = 8; c >= 1; c /= 2) {
    if (small * c > static_cast<long long>(sms) * attend_rows_ctas_per_sm() || small > attend_rows_clusters(c)) continue;
    const bool shared = small * c > sms;
    const double t = (shared ? 78.0 : 63.0) + (shared ? 10.6 : 9.7) * ((steps + c - 1) / c);
    if (t < best) {
      best = t;
      pl.cluster = c;
      pl.few = pl.whole = false;
    }
  }
}

int plan_attn(const kvsel_attn_params* p, bool with_acc, bool tree, AttnPlan& pl) {
  int rc = check_attn(p);
  if (rc) return rc;
  int sms = 0;
  if ((rc = device_sms(&sms))) return rc;
  const int R = p->n_new * p->group;
  const int tr = attend_rows_tile(), rt = (R + tr - 1) / tr;
  // up to 32 rows of few tiles go as two items (6 tokens of 8 segments of 512 rows, group 4: 6.5 us, as
  // chunks 12.7; 20 rows of 32 segments of 4096: 22.5 and 25.4; a CTA per item loses from 256 rows on).
  // (The weights' logits are kept for one item per segment.)
  if (tree) {
    plan_tree(p, sms, pl);
  } else if (rt == 1 || (rt == 2 && !with_acc)) {
    // tiles of 64 rows that an item may have: with a window some before it and some of the first rows
    long long tiles = (static_cast<long long>(p->max_len) + 63) / 64;
    const long long seen = (p->n_sink + 63ll) / 64 + (static_cast<long long>(p->window) + p->n_new + 126) / 64;
    const bool window = p->window > 0 && seen < tiles;
    if (window) tiles = seen;
    pl.cluster = attend_rows_cluster(static_cast<long long>(p->batch) * p->h_kv * rt, tiles, window,
                                     sms * attend_rows_ctas_per_sm());
    if (rt == 2 && tiles > (pl.cluster == 1 ? 2 : 16 * pl.cluster)) pl.cluster = 0;
  }
  if (tree ? pl.cluster || pl.few : rt == 1 || pl.cluster) {
    // single tokens and the like: HBM-bound, 16 query rows per item
    pl.tr = tr;
    pl.grid = sms * attend_rows_ctas_per_sm();
  } else {
    pl.tiled = true;
    pl.block = 128 / p->group * p->group;
    pl.split = R <= pl.block;
    pl.tr = pl.split ? pl.block : 2 * pl.block;
    pl.grid = sms;
  }
  pl.rt = (R + pl.tr - 1) / pl.tr;
  if (pl.tiled) {
    // tiles of 128 rows that an item may have
    long long tiles = (static_cast<long long>(p->max_len) + 127) / 128;
    if (p->window > 0)
      tiles = std::min(tiles, (p->n_sink + 127ll) / 128 + (static_cast<long long>(p->window) + pl.tr / p->group + 317) / 128);
    if (!tree) pl.whole = attend_tile_whole(static_cast<long long>(p->batch) * p->h_kv * pl.rt, tiles, pl.split, pl.grid);
  }
  // behind the status word and the counters that the scoring calls keep in a shared workspace
  size_t off = kStatusBytes + kCounterBytes;
  pl.rec = off;
  off = align256(off + sizeof(int2) * pl.grid);
  pl.ml = off;
  off = align256(off + sizeof(float2) * 2 * pl.grid * pl.tr);
  pl.o = off;
  off = align256(off + sizeof(float) * 2 * pl.grid * pl.tr * kHeadDim);
  if (with_acc) {
    pl.lse2 = off;
    const size_t rows = static_cast<size_t>(p->batch) * p->h_kv * R;
    off = align256(off + sizeof(float) * rows);
    if (pl.tiled) {
      const long long full = (static_cast<long long>(p->max_len) + 255) / 256, sinks = (p->n_sink + 255ll) / 256;
      const long long part = sinks + (static_cast<long long>(p->window) + p->n_new + 254) / 256 + 1;
      const bool few = p->causal && p->window > 0 && part < full;
      const long long kb = few ? part : full;
      if (kb * p->batch * p->h_kv > 1ll << 30) return KVSEL_EUNSUPPORTED;
      pl.kb = static_cast<int>(kb);
      pl.kb_sink = few ? static_cast<int>(sinks) : -1;
      pl.wpart = off;
      off = align256(off + sizeof(float) * 2 * pl.grid * 256);
    } else {
      pl.logits = off;
      pl.logit_stride = (static_cast<long long>(p->max_len) + 7) / 8 * 8;
      off = align256(off + sizeof(float) * rows * pl.logit_stride);
    }
  }
  pl.total = off;
  return KVSEL_OK;
}

// K/V views that the calls below read (and, for the eviction, write): `rows` per segment
int check_cache(const kvsel_kv* kv, int B, int H, long long rows, const int64_t* offsets, long long n_rows) {
  if (!kv || !kv->k || !kv->v || !aligned(kv->k, 16) || !aligned(kv->v, 16)) return KVSEL_EINVAL;
  if ((kv->layout == KVSEL_LAYOUT_PACKED) != (offsets != nullptr)) return KVSEL_EINVAL;
  if (kv->layout == KVSEL_LAYOUT_CONTIGUOUS) {
    if (kv->stride_tok < kHeadDim || kv->stride_tok % 8) return KVSEL_EINVAL;
    if (bad_stride(kv->stride_head, H) || bad_stride(kv->stride_req, B)) return KVSEL_EINVAL;
  } else if (kv->layout == KVSEL_LAYOUT_PACKED) {
    if (kv->stride_tok < kHeadDim || kv->stride_tok % 8 || n_rows < 1 || !aligned(offsets, 8)) return KVSEL_EINVAL;
  } else if (kv->layout == KVSEL_LAYOUT_PAGED) {
    const int bs = kv->block_size;
    if (!kv->block_table || !aligned(kv->block_table, 4) || !(bs == 8 || bs == 16 || bs == 32 || bs == 64)) return KVSEL_EINVAL;
    if (kv->num_blocks < 1 || kv->max_blocks < (rows + bs - 1) / bs) return KVSEL_EINVAL;
    // rows of the pool are counted in 32 bits
    if ((static_cast<long long>(kv->num_blocks) + 1) * bs * H > (1ll << 31) - 1) return KVSEL_EUNSUPPORTED;
  } else {
    return KVSEL_EINVAL;
  }
  return KVSEL_OK;
}

// Query tiles: 64 columns x the group's heads x whole tokens.
bool query_map(CUtensorMap* m, const AttnArgs& a, int block) {
  const cuuint64_t hq = static_cast<cuuint64_t>(a.H) * a.G;
  const cuuint64_t dims[4] = {kHeadDim, hq, static_cast<cuuint64_t>(a.m), static_cast<cuuint64_t>(a.B)};
  // the stride of a dimension with one entry is not used; any valid one will do
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(hq > 1 ? a.q_head : kHeadDim) * 2,
                                 static_cast<cuuint64_t>(a.m > 1 ? a.q_tok : kHeadDim) * 2,
                                 static_cast<cuuint64_t>(a.B > 1 ? a.q_req : kHeadDim) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(a.G), static_cast<cuuint32_t>(block / a.G), 1};
  return encode_bf16_map(m, a.q, 4, dims, strides, box);
}

// K or V tiles: 64 columns x `box_rows` rows of one segment (contiguous, packed) or a page.
bool cache_map(CUtensorMap* m, const void* base, const kvsel_kv* kv, const kvsel_attn_params* p, int box_rows) {
  const cuuint64_t H = p->h_kv, B = p->batch;
  if (kv->layout == KVSEL_LAYOUT_PAGED) {
    // a page whole, in atoms of 8 rows x 64 columns: columns, rows of an atom, column halves, atoms of
    // the page; the last dimension, rows of the pool, places the page and the head in one coordinate
    const cuuint64_t bs = kv->block_size, row = H * kHeadDim * 2;
    const cuuint64_t dims[5] = {64, 8, 2, bs / 8, static_cast<cuuint64_t>(kv->num_blocks) * bs * H};
    const cuuint64_t strides[4] = {row, 128, 8 * row, kHeadDim * 2};
    const cuuint32_t box[5] = {64, 8, 2, static_cast<cuuint32_t>(bs / 8), 1};
    return encode_bf16_map(m, base, 5, dims, strides, box);
  }
  const bool packed = kv->layout == KVSEL_LAYOUT_PACKED;
  const cuuint64_t rows = packed ? p->n_rows : p->max_len, tok = static_cast<cuuint64_t>(kv->stride_tok) * 2;
  const cuuint64_t dims[4] = {kHeadDim, rows, packed ? 1 : H, packed ? 1 : B};
  const cuuint64_t strides[3] = {tok, !packed && H > 1 ? static_cast<cuuint64_t>(kv->stride_head) * 2 : tok,
                                 !packed && B > 1 ? static_cast<cuuint64_t>(kv->stride_req) * 2 : tok};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), 1, 1};
  return encode_bf16_map(m, base, 4, dims, strides, box);
}

KvSource source_of(const kvsel_kv* kv) {
  KvSource s{};
  s.paged = kv->layout == KVSEL_LAYOUT_PAGED;
  s.block_size = s.paged ? kv->block_size : 1;
  s.max_blocks = kv->max_blocks;
  s.num_blocks = kv->num_blocks;
  s.block_table = kv->block_table;
  return s;
}

int check_ws(const void* ws, size_t have, size_t need) {
  return !ws || !aligned(ws, 256) || have < need ? KVSEL_EWORKSPACE : KVSEL_OK;
}

int check_evict(const kvsel_evict_params* p) {
  if (!p) return KVSEL_EINVAL;
  if (p->head_dim != kHeadDim) return KVSEL_EUNSUPPORTED;
  if (p->h_kv < 1 || p->h_kv > 64 || p->batch < 1 || p->n_new < 0 || p->capacity < 1 || p->budget < 1) return KVSEL_EINVAL;
  if (p->batch > KVSEL_MAX_ATTN_BATCH || p->batch * p->h_kv > kMaxSegments || p->capacity > kMaxRows)
    return KVSEL_EUNSUPPORTED;
  if (p->n_sink < 0 || p->n_recent < 0 || p->budget > p->capacity) return KVSEL_EINVAL;
  if (static_cast<long long>(p->n_sink) + std::max(p->n_recent, p->n_new) > p->budget) return KVSEL_EBUDGET;
  if (p->new_stride_req || p->new_stride_head || p->new_stride_tok)
    if (bad_stride(p->new_stride_req, p->batch) || bad_stride(p->new_stride_head, p->h_kv) ||
        bad_stride(p->new_stride_tok, p->n_new))
      return KVSEL_EINVAL;
  return KVSEL_OK;
}

struct EvictLayout {
  int most = 0;
  size_t head = 0, holes = 0, fills = 0, total = 0;
};
EvictLayout evict_layout(const kvsel_evict_params* p) {
  EvictLayout L;
  const size_t segs = static_cast<size_t>(p->batch) * p->h_kv;
  L.head = kStatusBytes + kCounterBytes;
  L.holes = align256(L.head + segs * sizeof(int4));
  // at most so many rows leave a segment, and so many slots lie behind its kept range
  L.most = p->capacity - p->budget + p->n_new;
  // (room for any budget, so that one workspace serves a cache for good)
  const size_t list = segs * p->capacity * sizeof(int32_t);
  L.fills = align256(L.holes + list);
  L.total = align256(L.fills + list);
  return L;
}

}  // namespace

// kvsel_attend, and with `tree` kvsel_attend_tree
static int attend(const kvsel_attn_params* p, const void* q, const kvsel_kv* kv, const int32_t* lens,
                  const int32_t* new_lens, const int64_t* offsets, const uint32_t* tree, void* out, float* lse, float* acc,
                  void* ws, size_t ws_bytes, void* stream) {
  int rc = check_attn(p);
  if (rc) return rc;
  if (!q || !aligned(q, 16) || !lens || !aligned(lens, 4) || !out || !aligned(out, 16)) return KVSEL_EINVAL;
  if (!aligned(new_lens, 4) || !aligned(lse, 4) || !aligned(acc, 4)) return KVSEL_EINVAL;
  if ((rc = check_cache(kv, p->batch, p->h_kv, p->max_len, offsets, p->n_rows))) return rc;
  if (acc && p->acc_stride < p->max_len) return KVSEL_EINVAL;
  AttnPlan pl;
  if ((rc = plan_attn(p, acc != nullptr, tree != nullptr, pl))) return rc;
  if ((rc = check_ws(ws, ws_bytes, pl.total))) return rc;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  AttnArgs a{};
  a.B = p->batch;
  a.H = p->h_kv;
  a.G = p->group;
  a.m = p->n_new;
  a.max_len = p->max_len;
  a.causal = p->causal;
  a.window = p->window;
  a.n_sink = p->n_sink;
  a.per_head = p->lens_per_head || offsets;
  const float scale = p->scale > 0.f ? p->scale : 1.f / std::sqrt(static_cast<float>(kHeadDim));
  a.s2 = scale * 1.4426950408889634f;
  a.lens = lens;
  a.new_lens = new_lens;
  a.offsets = offsets;
  a.n_rows = p->n_rows;
  const long long hq = static_cast<long long>(p->h_kv) * p->group, row = static_cast<long long>(p->n_new) * kHeadDim;
  const bool qd = !(p->q_stride_req || p->q_stride_head || p->q_stride_tok);
  const bool od = !(p->o_stride_req || p->o_stride_head || p->o_stride_tok);
  a.q = static_cast<const uint16_t*>(q);
  a.q_req = qd ? hq * row : p->q_stride_req;
  a.q_head = qd ? row : p->q_stride_head;
  a.q_tok = qd ? kHeadDim : p->q_stride_tok;
  a.out = static_cast<uint16_t*>(out);
  a.o_req = od ? hq * row : p->o_stride_req;
  a.o_head = od ? row : p->o_stride_head;
  a.o_tok = od ? kHeadDim : p->o_stride_tok;
  a.lse = lse;
  a.lse2 = acc ? reinterpret_cast<float*>(wsb + pl.lse2) : nullptr;
  a.logits = acc && !pl.tiled ? reinterpret_cast<float*>(wsb + pl.logits) : nullptr;
  a.logit_stride = pl.logit_stride;
  a.acc = acc;
  a.acc_stride = p->acc_stride;
  a.src = source_of(kv);
  a.k = static_cast<const uint16_t*>(kv->k);
  a.v = static_cast<const uint16_t*>(kv->v);
  a.stride_tok = kv->stride_tok;
  if (kv->layout == KVSEL_LAYOUT_CONTIGUOUS) {   // packed: rows follow each other, offsets place the segments
    a.stride_req = kv->stride_req;
    a.stride_head = kv->stride_head;
  }
  a.tree = tree;
  a.tree_words = (p->n_new + 31) / 32;
  a.tree_window = p->tree_window && p->window > 0 && p->window < p->n_new;
  a.by_rt = Div::by(pl.rt);
  a.by_H = Div::by(p->h_kv);
  a.by_G = Div::by(p->group);
  a.kb = pl.kb;
  a.kb_sink = pl.kb_sink;
  a.by_kb = Div::by(pl.kb);
  while (a.src.paged && (1 << a.page_shift) < a.src.block_size) ++a.page_shift;
  a.tr = pl.tr;
  a.rt = pl.rt;
  a.whole = pl.whole;
  a.part_o = reinterpret_cast<float*>(wsb + pl.o);
  a.part_ml = reinterpret_cast<float2*>(wsb + pl.ml);
  a.rec = reinterpret_cast<int2*>(wsb + pl.rec);
  a.grid = pl.grid;
  // A CTA for each row takes 2.2 us per 456 rows, eight rows per warp 0.4 us per piece of an item, of
  // which there are grid / items.  (16 items of 256 rows: 31 and 22 us for the whole call; 2 of 100, 76
  // pieces each: 20 and 43.)  A tree's rows go to a warp by eights, or to eight warps by eights from five
  // pieces an item on (join_trees_kernel: 19 pieces of 256 rows 16.6 and 5.2 us, two or three of 128 rows 6.6 and 9.6).
  const long long items = static_cast<long long>(p->batch) * p->h_kv * pl.rt;
  const int rows = std::min(pl.tr, p->n_new * p->group);
  a.by_item = tree ? items * 5 <= pl.grid : items <= pl.grid && items * items * rows <= 83ll * pl.grid;
  a.wc = WaitCtl{p->wait_cycles ? p->wait_cycles : kDefaultWaitCycles, static_cast<int*>(ws)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!pl.tiled) {
    rc = launch_rc(launch_attend_rows(a, pl.grid, pl.cluster, st));
    return rc || !acc ? rc : launch_rc(launch_weights_kept(a, st));
  }
  CUtensorMap tq, tk, tv;
  const int box = attend_tile_rows(pl.split);
  if (!query_map(&tq, a, pl.block) || !cache_map(&tk, kv->k, kv, p, box) || !cache_map(&tv, kv->v, kv, p, box))
    return KVSEL_EINVAL;
  rc = launch_rc(launch_attend_tile(a, tq, tk, tv, pl.block, pl.split, pl.grid, st));
  if (rc || !acc) return rc;
  if (pl.split && !cache_map(&tk, kv->k, kv, p, attend_tile_rows(false))) return KVSEL_EINVAL;
  return launch_rc(launch_weights_tile(a, tq, tk, pl.block, reinterpret_cast<float*>(wsb + pl.wpart), pl.grid, st));
}

extern "C" {

int kvsel_attend_workspace_size(const kvsel_attn_params* p, int with_acc, size_t* bytes) {
  if (!bytes) return KVSEL_EINVAL;
  AttnPlan pl;
  const int rc = plan_attn(p, with_acc != 0, false, pl);
  if (rc) return rc;
  *bytes = pl.total;
  return KVSEL_OK;
}

int kvsel_attend(const kvsel_attn_params* p, const void* q, const kvsel_kv* kv, const int32_t* lens,
                 const int32_t* new_lens, const int64_t* offsets, void* out, float* lse, float* acc, void* ws,
                 size_t ws_bytes, void* stream) {
  return attend(p, q, kv, lens, new_lens, offsets, nullptr, out, lse, acc, ws, ws_bytes, stream);
}

int kvsel_attend_tree_workspace_size(const kvsel_attn_params* p, size_t* bytes) {
  if (!bytes) return KVSEL_EINVAL;
  int rc = check_tree(p);
  if (rc) return rc;
  AttnPlan pl;
  if ((rc = plan_attn(p, false, true, pl))) return rc;
  *bytes = pl.total;
  return KVSEL_OK;
}

int kvsel_attend_tree(const kvsel_attn_params* p, const void* q, const kvsel_kv* kv, const int32_t* lens,
                      const int32_t* new_lens, const int64_t* offsets, const uint32_t* tree, void* out, float* lse,
                      void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_tree(p);
  if (rc) return rc;
  if (!tree || !aligned(tree, 4)) return KVSEL_EINVAL;
  return attend(p, q, kv, lens, new_lens, offsets, tree, out, lse, nullptr, ws, ws_bytes, stream);
}

int kvsel_evict_append_workspace_size(const kvsel_evict_params* p, size_t* bytes) {
  if (!bytes) return KVSEL_EINVAL;
  const int rc = check_evict(p);
  if (rc) return rc;
  *bytes = evict_layout(p).total;
  return KVSEL_OK;
}

int kvsel_evict_append(const kvsel_evict_params* p, const kvsel_kv* kv, int32_t* lens, int32_t* seen, int32_t* pos,
                       float* acc, const void* k_new, const void* v_new, const int32_t* new_lens, void* ws,
                       size_t ws_bytes, void* stream) {
  int rc = check_evict(p);
  if (rc) return rc;
  if (!lens || !seen || !pos || !acc || !aligned(lens, 4) || !aligned(seen, 4) || !aligned(pos, 4) || !aligned(acc, 4))
    return KVSEL_EINVAL;
  if (!aligned(new_lens, 4) || (p->n_new > 0 && (!k_new || !v_new || !aligned(k_new, 16) || !aligned(v_new, 16))))
    return KVSEL_EINVAL;
  if ((rc = check_cache(kv, p->batch, p->h_kv, p->capacity, nullptr, 0))) return rc;
  const EvictLayout L = evict_layout(p);
  if ((rc = check_ws(ws, ws_bytes, L.total))) return rc;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  EvictArgs a{};
  a.B = p->batch;
  a.H = p->h_kv;
  a.m = p->n_new;
  a.capacity = p->capacity;
  a.budget = p->budget;
  a.n_sink = p->n_sink;
  a.n_recent = p->n_recent;
  a.src = source_of(kv);
  a.k = static_cast<uint16_t*>(const_cast<void*>(kv->k));
  a.v = static_cast<uint16_t*>(const_cast<void*>(kv->v));
  a.stride_req = kv->stride_req;
  a.stride_head = kv->stride_head;
  a.stride_tok = kv->stride_tok;
  a.lens = lens;
  a.seen = seen;
  a.pos = pos;
  a.acc = acc;
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  const bool dense = !(p->new_stride_req || p->new_stride_head || p->new_stride_tok);
  const long long row = static_cast<long long>(p->n_new) * kHeadDim;
  a.new_req = dense ? p->h_kv * row : p->new_stride_req;
  a.new_head = dense ? row : p->new_stride_head;
  a.new_tok = dense ? kHeadDim : p->new_stride_tok;
  a.new_lens = new_lens;
  a.head = reinterpret_cast<int4*>(wsb + L.head);
  a.holes = reinterpret_cast<int32_t*>(wsb + L.holes);
  a.fills = reinterpret_cast<int32_t*>(wsb + L.fills);
  a.most = L.most;
  if ((rc = device_sms(&a.sms))) return rc;
  a.status = static_cast<int*>(ws);
  return launch_rc(launch_evict(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
