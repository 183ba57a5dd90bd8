// Host side that the cache, attention, block and page calls share: checks of
// arguments, and where a call's status goes.
#pragma once

#include <cuda_runtime.h>

#include <memory>
#include <mutex>

#include "tks_attention.h"
#include "tks_blocks.h"

namespace tks {
namespace attn {

inline bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool strides_ok(int64_t size, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2 = 0, int64_t s2 = 0);
int check_cache(const tks_cache* c);
int check_q(int32_t kv_heads, const tks_queries* q);  // without out, lse and softmax_scale
int log2_of(int32_t n);
int check_bounds(const tks_bounds* b);
bool bounds_of(const tks_bounds* b, const tks_cache* c);  // whether they have the cache's sizes

// The current device, and a stream's status word.
struct Place {
  int sms;
  unsigned* status;
  std::shared_ptr<std::mutex> order;  // held while a call is queued
};
int place_of(void* stream, Place* place);
cudaError_t setup_pages();  // (tks_pages.cu)

}  // namespace attn
}  // namespace tks
