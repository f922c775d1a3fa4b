// Shared by the kernels of a step of drafted tokens: masks and verification of trees, pages that requests
// share, rotary positions, kept rows left in their cache.
#pragma once
#include "internal.cuh"

namespace kvsel {

cudaError_t launch_tree_masks(const int32_t* parents, const int32_t* new_lens, const int32_t* first, int batch, int n_new,
                              uint32_t* tree, int32_t* pos, cudaStream_t st);

struct VerifyArgs {
  int m, vocab, mode;
  long long stride_req, stride_node;
  const int32_t* tokens;
  const int32_t* parents;
  const void* target;
  const void* draft;
  const float* u;
  const int32_t* new_lens;
  int32_t* path;
  int32_t* counts;
  int32_t* next;
  unsigned long long wait_cycles;
  int* status;
};
cudaError_t launch_verify(const VerifyArgs& a, int batch, bool bf16, int sms, cudaStream_t st);

struct PagesArgs {
  int H, B, block_size, shift, max_blocks, num_blocks, layers;
  int m, per;                     // new rows of a request at most; table entries that they may touch
  int per_head;                   // lens [B*H] instead of [B]
  long long stride_layer;
  uint16_t* k;
  uint16_t* v;
  const int32_t* table_in;        // fork: the rows before
  const int32_t* lens_in;
  const int32_t* src;
  int32_t* table;
  int32_t* ref;
  const int32_t* lens;
  int32_t* lens_out;
  const int32_t* new_lens;
  int32_t* granted;
  const int32_t* path;
  const int32_t* counts;
  // workspace of a reservation: what each touched entry needs, the pages that are handed out, and the copies
  // {from, to, rows, 0}, their number in copies[0].x
  int32_t* need;                  // [B*per]
  int32_t* pages;                 // [B*per]
  int32_t* list;                  // [B*per]
  int32_t* seats;                 // [3 * at least 2*B*per, a power of two]: shared pages and who writes to them
  int4* copies;                   // [1 + B*per]
  int* ticket;                    // zero between calls
  int* status;
};
cudaError_t launch_pages_fork(const PagesArgs& a, cudaStream_t st);
cudaError_t launch_pages_reserve(const PagesArgs& a, int sms, cudaStream_t st);
cudaError_t launch_pages_trim(const PagesArgs& a, cudaStream_t st);
cudaError_t launch_pages_accept(const PagesArgs& a, cudaStream_t st);

struct RopeTable {
  unsigned long long turns[64];   // of one position, in units of 2^-64 turns; turned back: their negatives
  int rot, interleaved;
  float scale;
};
struct RopeArgs {
  RopeTable t;
  int B, n_tok, heads, k_heads;
  const uint16_t* q;
  uint16_t* q_out;
  const uint16_t* k;
  uint16_t* k_out;
  long long q_req, q_head, q_tok, qo_req, qo_head, qo_tok, k_req, k_head, k_tok, ko_req, ko_head, ko_tok;
  const int32_t* pos;
  long long pos_req;
  const int32_t* new_lens;
};
cudaError_t launch_rope(const RopeArgs& a, int sms, cudaStream_t st);
struct RopeCacheArgs {
  RopeTable t;
  int B, H, max_len, per_head, page_shift;
  KvSource src;
  uint16_t* k;
  long long stride_req, stride_head, stride_tok;
  const int32_t* lens;
  const int32_t* pos;
  long long pos_stride;
  uint16_t* out;                  // null: in place
  long long o_req, o_head, o_tok;
  int* status;                    // may be null
};
cudaError_t launch_rope_cache(const RopeCacheArgs& a, int sms, cudaStream_t st);

struct KeepArgs {
  ReqTable rq;
  KvSource src;
  uint16_t* k;
  uint16_t* v;
  long long stride_req, stride_head, stride_tok;
  const int32_t* idx;
  const int32_t* counts;
  const int64_t* offsets;
  long long n_kept;
  const float* scores;            // may be null
  int32_t* lens;
  int32_t* seen;                  // may be null
  int32_t* pos;
  float* acc;                     // may be null
  long long capacity;
  int* status;                    // may be null
};
cudaError_t launch_keep(const KeepArgs& a, int max_count, cudaStream_t st);

}  // namespace kvsel
