// Attention over the paged 8-bit cache, causal.
#include "kv8_attn_impl.hpp"

namespace qmm {

int64_t kv8_attention_work(const Kv8& c, int64_t T, int64_t Hq, int64_t S, int64_t W) {
  return attention_work<Mask::kCausal>(c, T, Hq, S, W);
}

hipError_t launch_kv8_attention(const Kv8& c, int dt, const void* q, int64_t ldq, int64_t T,
                                int64_t Hq, const int32_t* table, const int32_t* lens,
                                const int32_t* cu, int64_t S, int64_t W, float scale, void* out,
                                float* lse, float* ws, hipStream_t st) {
  return launch_attention<Mask::kCausal>(c, dt, q, ldq, T, Hq, table, lens, cu, S, W, 0, 0, nullptr,
                                         scale, out, lse, ws, st);
}

}  // namespace qmm
