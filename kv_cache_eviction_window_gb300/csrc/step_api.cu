// C-ABI host layer of a step of drafted tokens: masks and verification of trees, pages that requests share,
// rotary positions.  Argument validation, workspace layout and launches; nothing here allocates memory.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/kvsel.h"
#include "step.cuh"

using namespace kvsel;

namespace {

constexpr unsigned long long kDefaultWaitCycles = 2000000000ull;   // ~1 s at the boost clock

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int launch_rc(cudaError_t e) { return e == cudaSuccess ? KVSEL_OK : KVSEL_ECUDA; }
bool bad_stride(long long s, long long extent) { return extent > 1 && (s <= 0 || s % 8 != 0); }
bool other(long long a, long long b, long long extent) { return extent > 1 && a != b; }
int check_ws(const void* ws, size_t have, size_t need) {
  return !ws || !aligned(ws, 256) || have < need ? KVSEL_EWORKSPACE : KVSEL_OK;
}
int device_sms(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KVSEL_ECUDA;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return KVSEL_ECUDA;
  return KVSEL_OK;
}

int check_verify(const kvsel_verify_params* p) {
  if (!p) return KVSEL_EINVAL;
  if (p->batch < 1 || p->n_new < 1 || p->vocab < 1) return KVSEL_EINVAL;
  if (p->batch > KVSEL_MAX_ATTN_BATCH || p->n_new > KVSEL_MAX_TREE || p->vocab > KVSEL_MAX_VOCAB) return KVSEL_EUNSUPPORTED;
  if (p->mode < 0 || p->mode > 2 || p->dtype < 0 || p->dtype > 1) return KVSEL_EINVAL;
  if (p->stride_req || p->stride_node)
    if ((p->n_new > 1 && p->stride_node < p->vocab) || (p->batch > 1 && p->stride_req < p->vocab)) return KVSEL_EINVAL;
  return KVSEL_OK;
}

// table entries that the new rows of a request may touch
long long reserve_entries(const kvsel_pages_params* p) { return p->n_new / p->block_size + 2ll; }

// elements of a layer's pool
long long layer_elems(const kvsel_pages_params* p) {
  return static_cast<long long>(p->num_blocks) * p->block_size * p->h_kv * kHeadDim;
}

int check_pages(const kvsel_pages_params* p) {
  if (!p) return KVSEL_EINVAL;
  if (p->head_dim != kHeadDim) return KVSEL_EUNSUPPORTED;
  if (p->h_kv < 1 || p->h_kv > 64 || p->batch < 1 || p->max_blocks < 1 || p->num_blocks < 1 || p->layers < 1 || p->n_new < 0)
    return KVSEL_EINVAL;
  const int bs = p->block_size;
  if (!(bs == 8 || bs == 16 || bs == 32 || bs == 64) || p->lens_per_head < 0 || p->lens_per_head > 1) return KVSEL_EINVAL;
  if (p->batch > KVSEL_MAX_ATTN_BATCH || p->max_blocks > (1 << 20) || p->num_blocks > (1 << 28) || p->layers > 1024 ||
      p->n_new > (1 << 20) || p->batch * reserve_entries(p) > (1 << 20))
    return KVSEL_EUNSUPPORTED;
  // (pools of layers do not overlap)
  if (p->stride_layer && p->layers > 1 && (p->stride_layer < layer_elems(p) || p->stride_layer % 8)) return KVSEL_EINVAL;
  return KVSEL_OK;
}

struct PagesLayout {
  size_t need = 0, pages = 0, list = 0, copies = 0, seats = 0, total = 0;
};
PagesLayout pages_layout(const kvsel_pages_params* p) {
  PagesLayout L;
  const size_t items = static_cast<size_t>(p->batch) * reserve_entries(p);
  // behind the status word and the counters that other calls keep in a shared workspace
  L.need = kStatusBytes + kCounterBytes;
  L.pages = align256(L.need + items * sizeof(int32_t));
  L.list = align256(L.pages + items * sizeof(int32_t));
  L.copies = align256(L.list + items * sizeof(int32_t));
  L.seats = align256(L.copies + (items + 1) * sizeof(int4));
  size_t slots = 64;
  while (slots < 2 * items) slots *= 2;
  L.total = align256(L.seats + 3 * slots * sizeof(int32_t));
  return L;
}

PagesArgs pages_args(const kvsel_pages_params* p, void* ws) {
  PagesArgs a{};
  a.H = p->h_kv;
  a.B = p->batch;
  a.block_size = p->block_size;
  while ((1 << a.shift) < p->block_size) ++a.shift;
  a.max_blocks = p->max_blocks;
  a.num_blocks = p->num_blocks;
  a.layers = p->layers;
  a.m = p->n_new;
  a.per = static_cast<int>(reserve_entries(p));
  a.per_head = p->lens_per_head;
  a.stride_layer = p->stride_layer ? p->stride_layer : layer_elems(p);
  a.status = static_cast<int*>(ws);
  return a;
}
bool words(std::initializer_list<const void*> list) {
  for (const void* x : list)
    if (!x || !aligned(x, 4)) return false;
  return true;
}

RopeTable rope_table(const kvsel_rope_angles* t) {
  RopeTable r;
  for (int i = 0; i < 64; ++i) r.turns[i] = t->back ? 0 - t->turns[i] : t->turns[i];
  r.rot = t->rot_dim;
  r.interleaved = t->layout == KVSEL_ROPE_INTERLEAVED;
  r.scale = t->scale;
  return r;
}
bool bad_table(const kvsel_rope_angles* t) {
  return !t || t->rot_dim < 16 || t->rot_dim > kHeadDim || t->rot_dim % 16 || t->layout < 0 || t->layout > 1 || t->back < 0 ||
         t->back > 1 || !std::isfinite(t->scale);
}

}  // namespace

extern "C" {

int kvsel_tree_masks(const int32_t* parents, const int32_t* new_lens, const int32_t* first, int32_t batch, int32_t n_new,
                     uint32_t* tree, int32_t* pos, void* stream) {
  if (batch < 1 || n_new < 1) return KVSEL_EINVAL;
  if (batch > KVSEL_MAX_ATTN_BATCH || n_new > KVSEL_MAX_TREE) return KVSEL_EUNSUPPORTED;
  if (!words({parents, tree}) || !aligned(new_lens, 4) || !aligned(first, 4) || !aligned(pos, 4) || (pos && !first))
    return KVSEL_EINVAL;
  return launch_rc(launch_tree_masks(parents, new_lens, first, batch, n_new, tree, pos, static_cast<cudaStream_t>(stream)));
}

int kvsel_verify_workspace_size(const kvsel_verify_params* p, size_t* bytes) {
  if (!bytes) return KVSEL_EINVAL;
  const int rc = check_verify(p);
  if (rc) return rc;
  *bytes = kStatusBytes;
  return KVSEL_OK;
}

int kvsel_verify(const kvsel_verify_params* p, const int32_t* tokens, const int32_t* parents, const void* target,
                 const void* draft, const float* u, const int32_t* new_lens, int32_t* path, int32_t* counts,
                 int32_t* next, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_verify(p);
  if (rc) return rc;
  const unsigned size = p->dtype == KVSEL_DTYPE_FP32 ? 4 : 2;
  if (!words({tokens, parents, path, counts, next}) || !aligned(new_lens, 4) || !aligned(u, 4)) return KVSEL_EINVAL;
  if (!target || !aligned(target, size) || !aligned(draft, size)) return KVSEL_EINVAL;
  if ((draft != nullptr) != (p->mode == KVSEL_VERIFY_SAMPLED) || (!u && p->mode != KVSEL_VERIFY_GREEDY)) return KVSEL_EINVAL;
  if ((rc = check_ws(ws, ws_bytes, kStatusBytes))) return rc;
  VerifyArgs a{};
  a.m = p->n_new;
  a.vocab = p->vocab;
  a.mode = p->mode;
  const bool dense = !(p->stride_req || p->stride_node);
  a.stride_node = dense ? p->vocab : p->stride_node;
  a.stride_req = dense ? static_cast<long long>(p->n_new) * p->vocab : p->stride_req;
  a.tokens = tokens;
  a.parents = parents;
  a.target = target;
  a.draft = draft;
  a.u = u;
  a.new_lens = new_lens;
  a.path = path;
  a.counts = counts;
  a.next = next;
  a.wait_cycles = p->wait_cycles ? p->wait_cycles : kDefaultWaitCycles;
  a.status = static_cast<int*>(ws);
  int sms = 0;
  if ((rc = device_sms(&sms))) return rc;
  return launch_rc(launch_verify(a, p->batch, p->dtype == KVSEL_DTYPE_BF16, sms, static_cast<cudaStream_t>(stream)));
}

int kvsel_pages_workspace_size(const kvsel_pages_params* p, size_t* bytes) {
  if (!bytes) return KVSEL_EINVAL;
  const int rc = check_pages(p);
  if (rc) return rc;
  *bytes = pages_layout(p).total;
  return KVSEL_OK;
}

int kvsel_pages_fork(const kvsel_pages_params* p, const int32_t* table_in, const int32_t* lens_in, const int32_t* src,
                     int32_t* table_out, int32_t* lens_out, int32_t* ref, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_pages(p);
  if (rc) return rc;
  if (!words({table_in, lens_in, src, table_out, lens_out, ref})) return KVSEL_EINVAL;
  const long long entries = static_cast<long long>(p->batch) * p->max_blocks;
  const int segs = p->lens_per_head ? p->batch * p->h_kv : p->batch;
  if ((table_in < table_out + entries && table_out < table_in + entries) || (lens_in < lens_out + segs && lens_out < lens_in + segs))
    return KVSEL_EINVAL;
  if ((rc = check_ws(ws, ws_bytes, pages_layout(p).total))) return rc;
  PagesArgs a = pages_args(p, ws);
  a.table_in = table_in;
  a.lens_in = lens_in;
  a.src = src;
  a.table = table_out;
  a.lens_out = lens_out;
  a.ref = ref;
  return launch_rc(launch_pages_fork(a, static_cast<cudaStream_t>(stream)));
}

int kvsel_pages_reserve(const kvsel_pages_params* p, void* k, void* v, int32_t* table, int32_t* ref, const int32_t* lens,
                        const int32_t* new_lens, int32_t* granted, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_pages(p);
  if (rc) return rc;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !words({table, ref, lens, granted}) || !aligned(new_lens, 4))
    return KVSEL_EINVAL;
  const PagesLayout L = pages_layout(p);
  if ((rc = check_ws(ws, ws_bytes, L.total))) return rc;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  PagesArgs a = pages_args(p, ws);
  a.k = static_cast<uint16_t*>(k);
  a.v = static_cast<uint16_t*>(v);
  a.table = table;
  a.ref = ref;
  a.lens = lens;
  a.new_lens = new_lens;
  a.granted = granted;
  a.need = reinterpret_cast<int32_t*>(wsb + L.need);
  a.pages = reinterpret_cast<int32_t*>(wsb + L.pages);
  a.list = reinterpret_cast<int32_t*>(wsb + L.list);
  a.copies = reinterpret_cast<int4*>(wsb + L.copies);
  a.seats = reinterpret_cast<int32_t*>(wsb + L.seats);
  a.ticket = reinterpret_cast<int*>(wsb + kStatusBytes);   // one of the counters that kvsel_workspace_init zeroes
  int sms = 0;
  if ((rc = device_sms(&sms))) return rc;
  return launch_rc(launch_pages_reserve(a, sms, static_cast<cudaStream_t>(stream)));
}

int kvsel_pages_trim(const kvsel_pages_params* p, int32_t* table, int32_t* ref, const int32_t* lens, void* ws,
                     size_t ws_bytes, void* stream) {
  int rc = check_pages(p);
  if (rc) return rc;
  if (!words({table, ref, lens})) return KVSEL_EINVAL;
  if ((rc = check_ws(ws, ws_bytes, pages_layout(p).total))) return rc;
  PagesArgs a = pages_args(p, ws);
  a.table = table;
  a.ref = ref;
  a.lens = lens;
  return launch_rc(launch_pages_trim(a, static_cast<cudaStream_t>(stream)));
}

int kvsel_pages_accept(const kvsel_pages_params* p, void* k, void* v, const int32_t* table, const int32_t* lens,
                       const int32_t* new_lens, const int32_t* path, const int32_t* counts, int32_t* lens_out, void* ws,
                       size_t ws_bytes, void* stream) {
  int rc = check_pages(p);
  if (rc) return rc;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !words({table, lens, path, counts, lens_out}) || !aligned(new_lens, 4))
    return KVSEL_EINVAL;
  if (p->n_new < 1) return KVSEL_EINVAL;
  if ((rc = check_ws(ws, ws_bytes, pages_layout(p).total))) return rc;
  PagesArgs a = pages_args(p, ws);
  a.k = static_cast<uint16_t*>(k);
  a.v = static_cast<uint16_t*>(v);
  a.table = const_cast<int32_t*>(table);
  a.lens = lens;
  a.new_lens = new_lens;
  a.path = path;
  a.counts = counts;
  a.lens_out = lens_out;
  return launch_rc(launch_pages_accept(a, static_cast<cudaStream_t>(stream)));
}

int kvsel_rope_table(const kvsel_rope_params* p, kvsel_rope_angles* t) {
  if (!p || !t) return KVSEL_EINVAL;
  const int rot = p->rot_dim;
  if (rot < 1 || p->layout < 0 || p->layout > 1 || p->direction < 0 || p->direction > 2 || p->scaling < 0 || p->scaling > 4)
    return KVSEL_EINVAL;
  if (rot % 16 || rot > kHeadDim || (p->scaling == KVSEL_ROPE_NTK && rot < 32)) return KVSEL_EUNSUPPORTED;
  if (!(p->theta > 1.0) || !std::isfinite(p->theta) || !(p->value_scale >= 0.0) || !std::isfinite(p->value_scale))
    return KVSEL_EINVAL;
  const double two_pi = 6.283185307179586, f = p->scaling == KVSEL_ROPE_NONE ? 1.0 : p->factor;
  if (!(f >= 1.0) || !std::isfinite(f)) return KVSEL_EINVAL;
  double theta = p->theta, scale = 1.0, low = 0.0, high = 0.0;
  if (p->scaling == KVSEL_ROPE_NTK) theta *= std::pow(f, rot / (rot - 2.0));
  if (p->scaling == KVSEL_ROPE_YARN) {
    if (p->orig_len < 1 || !(p->beta_slow > 0.0) || !(p->beta_fast > p->beta_slow) || !std::isfinite(p->beta_fast)) return KVSEL_EINVAL;
    // the pair that turns beta times in orig_len
    const double per = rot / (2.0 * std::log(theta));
    low = std::max(std::floor(per * std::log(p->orig_len / (p->beta_fast * two_pi))), 0.0);
    high = std::min(std::ceil(per * std::log(p->orig_len / (p->beta_slow * two_pi))), rot - 1.0);
    scale = 0.1 * std::log(f) + 1.0;
  }
  if (p->scaling == KVSEL_ROPE_BANDS &&
      (p->orig_len < 1 || !(p->low_freq > 0.0) || !(p->high_freq > p->low_freq) || !std::isfinite(p->high_freq)))
    return KVSEL_EINVAL;
  std::memset(t, 0, sizeof(*t));
  for (int i = 0; i < rot / 2; ++i) {
    double w = std::pow(theta, -2.0 * i / rot);
    if (p->scaling == KVSEL_ROPE_LINEAR) w /= f;
    if (p->scaling == KVSEL_ROPE_YARN) {
      const double g = std::min(std::max((i - low) / std::max(high - low, 0.001), 0.0), 1.0);
      w *= g / f + 1.0 - g;
    }
    if (p->scaling == KVSEL_ROPE_BANDS) {
      const double s = std::min(std::max((p->orig_len * w / two_pi - p->low_freq) / (p->high_freq - p->low_freq), 0.0), 1.0);
      w *= s + (1.0 - s) / f;
    }
    t->turns[i] = static_cast<uint64_t>(std::ldexp(w / two_pi, 64));
  }
  if (p->value_scale > 0.0) scale = p->value_scale;
  t->rot_dim = rot;
  t->layout = p->layout;
  t->scale = static_cast<float>(p->direction == KVSEL_ROPE_INVERSE ? 1.0 / scale : scale);
  t->back = p->direction != KVSEL_ROPE_FORWARD;
  return KVSEL_OK;
}

int kvsel_rope(const kvsel_rope_angles* table, const kvsel_rope_rows* p, const void* q, void* q_out, const void* k,
               void* k_out, const int32_t* pos, const int32_t* new_lens, void* stream) {
  if (bad_table(table) || !p) return KVSEL_EINVAL;
  if (p->batch < 1 || p->n_tok < 1 || p->heads < 1 || p->k_heads < 0 || p->pos_req < 0) return KVSEL_EINVAL;
  if (p->batch > 65535 || p->n_tok > (1 << 20) || static_cast<long long>(p->batch) * p->n_tok > (1ll << 31) - 64 || p->heads > 8192 || p->k_heads > 8192 || p->heads + p->k_heads > 8192)
    return KVSEL_EUNSUPPORTED;
  if (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16) || !pos || !aligned(pos, 4) || !aligned(new_lens, 4)) return KVSEL_EINVAL;
  if (p->k_heads && (!k || !k_out || !aligned(k, 16) || !aligned(k_out, 16))) return KVSEL_EINVAL;
  const long long B = p->batch, n = p->n_tok;
  if (bad_stride(p->q_req, B) || bad_stride(p->q_head, p->heads) || bad_stride(p->q_tok, n) || bad_stride(p->qo_req, B) ||
      bad_stride(p->qo_head, p->heads) || bad_stride(p->qo_tok, n))
    return KVSEL_EINVAL;
  if (p->k_heads && (bad_stride(p->k_req, B) || bad_stride(p->k_head, p->k_heads) || bad_stride(p->k_tok, n) ||
                     bad_stride(p->ko_req, B) || bad_stride(p->ko_head, p->k_heads) || bad_stride(p->ko_tok, n)))
    return KVSEL_EINVAL;
  // in place: a row goes where it came from
  if (q == q_out && (other(p->q_req, p->qo_req, B) || other(p->q_head, p->qo_head, p->heads) || other(p->q_tok, p->qo_tok, n)))
    return KVSEL_EINVAL;
  if (p->k_heads && k == k_out &&
      (other(p->k_req, p->ko_req, B) || other(p->k_head, p->ko_head, p->k_heads) || other(p->k_tok, p->ko_tok, n)))
    return KVSEL_EINVAL;
  RopeArgs a{};
  a.t = rope_table(table);
  a.B = p->batch;
  a.n_tok = p->n_tok;
  a.heads = p->heads;
  a.k_heads = p->k_heads;
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k = static_cast<const uint16_t*>(k);
  a.k_out = static_cast<uint16_t*>(k_out);
  a.q_req = p->q_req;
  a.q_head = p->q_head;
  a.q_tok = p->q_tok;
  a.qo_req = p->qo_req;
  a.qo_head = p->qo_head;
  a.qo_tok = p->qo_tok;
  a.k_req = p->k_req;
  a.k_head = p->k_head;
  a.k_tok = p->k_tok;
  a.ko_req = p->ko_req;
  a.ko_head = p->ko_head;
  a.ko_tok = p->ko_tok;
  a.pos = pos;
  a.pos_req = p->pos_req;
  a.new_lens = new_lens;
  int sms = 0;
  const int rc = device_sms(&sms);
  return rc ? rc : launch_rc(launch_rope(a, sms, static_cast<cudaStream_t>(stream)));
}

int kvsel_rope_cache(const kvsel_rope_angles* table, const kvsel_rope_cache_params* p, const kvsel_kv* kv,
                     const int32_t* lens, const int32_t* pos, void* k_out, void* ws, size_t ws_bytes, void* stream) {
  if (bad_table(table) || !p || !kv || !kv->k || !aligned(kv->k, 16)) return KVSEL_EINVAL;
  if (p->h_kv < 1 || p->h_kv > 64 || p->batch < 1 || p->max_len < 1 || p->lens_per_head < 0 || p->lens_per_head > 1)
    return KVSEL_EINVAL;
  if (p->batch > KVSEL_MAX_ATTN_BATCH || p->batch * p->h_kv > 65535 || p->max_len > (1 << 30)) return KVSEL_EUNSUPPORTED;
  if (!lens || !aligned(lens, 4) || !aligned(pos, 4) || !aligned(k_out, 16)) return KVSEL_EINVAL;
  if ((pos != nullptr) != (p->pos_stride != 0) || (pos && p->pos_stride < p->max_len)) return KVSEL_EINVAL;
  if (k_out && (bad_stride(p->o_req, p->batch) || bad_stride(p->o_head, p->h_kv) || bad_stride(p->o_tok, p->max_len)))
    return KVSEL_EINVAL;
  if (ws && (!aligned(ws, 16) || ws_bytes < kStatusBytes)) return KVSEL_EWORKSPACE;
  RopeCacheArgs a{};
  if (kv->layout == KVSEL_LAYOUT_CONTIGUOUS) {
    if (kv->stride_tok < kHeadDim || kv->stride_tok % 8 || bad_stride(kv->stride_head, p->h_kv) || bad_stride(kv->stride_req, p->batch))
      return KVSEL_EINVAL;
    a.stride_req = kv->stride_req;
    a.stride_head = kv->stride_head;
    a.stride_tok = kv->stride_tok;
  } else if (kv->layout == KVSEL_LAYOUT_PAGED) {
    const int bs = kv->block_size;
    if (!words({kv->block_table}) || !(bs == 8 || bs == 16 || bs == 32 || bs == 64) || kv->num_blocks < 1 ||
        kv->max_blocks < (p->max_len + bs - 1) / bs)
      return KVSEL_EINVAL;
    a.src.paged = 1;
    a.src.block_size = bs;
    a.src.max_blocks = kv->max_blocks;
    a.src.num_blocks = kv->num_blocks;
    a.src.block_table = kv->block_table;
    while ((1 << a.page_shift) < bs) ++a.page_shift;
  } else {
    return KVSEL_EINVAL;
  }
  a.t = rope_table(table);
  a.B = p->batch;
  a.H = p->h_kv;
  a.max_len = p->max_len;
  a.per_head = p->lens_per_head;
  a.k = static_cast<uint16_t*>(const_cast<void*>(kv->k));
  a.lens = lens;
  a.pos = pos;
  a.pos_stride = p->pos_stride;
  a.out = static_cast<uint16_t*>(k_out);
  a.o_req = p->o_req;
  a.o_head = p->o_head;
  a.o_tok = p->o_tok;
  a.status = static_cast<int*>(ws);
  int sms = 0;
  const int rc = device_sms(&sms);
  return rc ? rc : launch_rc(launch_rope_cache(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
