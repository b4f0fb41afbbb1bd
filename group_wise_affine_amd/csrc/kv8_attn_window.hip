// Attention over the paged 8-bit cache, a sliding window with sinks: a query at
// position p sees the positions above p - window up to its own, and those below
// `sinks` up to its own. Tiles that no row of a workgroup sees are not read.
#include "kv8_attn_impl.hpp"

namespace qmm {

int64_t kv8_attention_window_work(const Kv8& c, int64_t T, int64_t Hq, int64_t S, int64_t W,
                                  int64_t window, int64_t sinks) {
  return attention_work<Mask::kWindow>(c, T, Hq, S, W, window, sinks);
}

hipError_t launch_kv8_attention_window(const Kv8& c, int dt, const void* q, int64_t ldq, int64_t T,
                                       int64_t Hq, const int32_t* table, const int32_t* lens,
                                       const int32_t* cu, int64_t S, int64_t W, int64_t window,
                                       int64_t sinks, float scale, void* out, float* lse, float* ws,
                                       hipStream_t st) {
  return launch_attention<Mask::kWindow>(c, dt, q, ldq, T, Hq, table, lens, cu, S, W, window, sinks,
                                         nullptr, scale, out, lse, ws, st);
}

}  // namespace qmm
