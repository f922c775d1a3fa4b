// Shared by the kernels of kvsel_evict_append.
#pragma once
#include "internal.cuh"

namespace kvsel {

struct EvictArgs {
  int B, H, m;                    // requests, KV heads, new rows of a segment at most
  int capacity, budget, n_sink, n_recent;
  KvSource src;
  uint16_t* k;
  uint16_t* v;
  long long stride_req, stride_head, stride_tok;
  int32_t* lens;                  // [B*H]
  int32_t* seen;                  // [B*H]
  int32_t* pos;                   // [B*H][capacity]
  float* acc;                     // [B*H][capacity]
  const uint16_t* k_new;
  const uint16_t* v_new;
  long long new_req, new_head, new_tok;
  const int32_t* new_lens;        // [B] or null
  // workspace: the segment's numbers for the second launch, its holes, and the rank among the
  // kept ones (or -1) of every slot behind the kept range
  int4* head;                     // [B*H]: rows kept, rows before, new rows, tokens seen before
  int sms;                        // of the device
  int most;                       // rows to evict, and slots behind the kept range, at most
  int32_t* holes;                 // [B*H][most]
  int32_t* fills;                 // [B*H][most]
  int* status;
};
bool evict_in_one_launch(int most);   // then holes and fills are not used
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st);

}  // namespace kvsel
