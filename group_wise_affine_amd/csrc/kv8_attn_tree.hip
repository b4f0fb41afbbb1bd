// Attention over the paged 8-bit cache for a tree of drafted tokens: a sequence's
// last new tokens, up to 64, form a tree; each sees what precedes the tree, its
// ancestors and itself. New tokens before the tree are causal.
#include "kv8_attn_impl.hpp"

namespace qmm {

int64_t kv8_attention_tree_work(const Kv8& c, int64_t T, int64_t Hq, int64_t S, int64_t W) {
  return attention_work<Mask::kTree>(c, T, Hq, S, W);
}

hipError_t launch_kv8_attention_tree(const Kv8& c, int dt, const void* q, int64_t ldq, int64_t T,
                                     int64_t Hq, const int32_t* table, const int32_t* lens,
                                     const int32_t* cu, int64_t S, int64_t W, const int32_t* parent,
                                     float scale, void* out, float* lse, float* ws, hipStream_t st) {
  return launch_attention<Mask::kTree>(c, dt, q, ldq, T, Hq, table, lens, cu, S, W, 0, 0, parent,
                                       scale, out, lse, ws, st);
}

}  // namespace qmm
