// The paged 8-bit key/value cache as the kernels see it. Page p holds, for
// each head, B consecutive tokens of one sequence: keys as [B][D] codes,
// values transposed as [D][B] codes (so that both are read with 16-byte loads
// in the order in which the attention's matrix instructions take them), and
// one fp32 scale for the keys and one for the values.
#pragma once

#include "int8_common.hpp"

namespace qmm {

struct Kv8 {
  int8_t* k;
  int8_t* v;
  float* ks;
  float* vs;
  int pages, heads, bt_log2, dim;   // tokens per page = 1 << bt_log2
  __host__ __device__ int64_t block(int64_t page, int head) const {   // codes before (page, head)
    return (page * heads + head) * ((int64_t)dim << bt_log2);
  }
};

// The new tokens of sequence s are rows cu[s] .. cu[s+1] of the packed batch;
// lens[s] counts the sequence's tokens with them. Values that cannot be are
// brought into range, so that no access leaves an array.
struct Kv8Seqs {
  const int32_t* table;   // [S][W] page numbers
  const int32_t* lens;    // [S]
  const int32_t* cu;      // [S + 1]
  int S, W, T;            // T <= 2^24
  // (values of one sequence are the same in every lane: they belong in scalar
  // registers, which the compiler does not see through the loads)
  __device__ int first(int s) const {
    const int c = __builtin_amdgcn_readfirstlane(cu[s]);
    return c < 0 ? 0 : c > T ? T : c;
  }
  __device__ int count(int s) const {
    const int n = first(s + 1) - first(s);
    return n < 0 ? 0 : n;
  }
  __device__ int length(int s, int bt_log2) const {
    const int64_t most = (int64_t)W << bt_log2;
    const int n = __builtin_amdgcn_readfirstlane(lens[s]);
    return n < 0 ? 0 : n > most ? (int)most : n;
  }
};

// Work items of a ragged batch, `unit` new tokens each: sequence s owns items
// cu[s] / unit + extra * s .. cu[s+1] / unit + extra * (s+1), at least count /
// unit + extra of them. Returns the sequence that owns item i (binary search).
__device__ __forceinline__ int first_item(const Kv8Seqs& q, int s, int unit, int extra) {
  return (uint32_t)q.first(s) / (uint32_t)unit + extra * s;
}
__device__ __forceinline__ int find_seq(const Kv8Seqs& q, int i, int unit, int extra) {
  int lo = 0, hi = q.S;   // the item belongs to a sequence in [lo, hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first_item(q, mid, unit, extra) <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Copies part `part` of `parts` of a page (codes, and with part 0 the scales)
// with 256 threads, four 16-byte pieces in flight per thread.
constexpr int kCopyBytes = 16384;   // of keys and of values each, per part
__host__ __device__ inline int copy_parts(const Kv8& c) {
  const int64_t bytes = c.block(1, 0);
  return (int)((bytes + kCopyBytes - 1) / kCopyBytes);
}
__device__ __forceinline__ void copy_page(const Kv8& to, int64_t d, const Kv8& from, int64_t s,
                                          int part, int parts) {
  const int64_t page = to.block(1, 0) / 16;   // pieces of a page
  const int64_t per = (page + parts - 1) / parts, begin = part * per;
  const int64_t end = begin + per < page ? begin + per : page;
  const uint4* ks = reinterpret_cast<const uint4*>(from.k) + s * page;
  const uint4* vs = reinterpret_cast<const uint4*>(from.v) + s * page;
  uint4* kd = reinterpret_cast<uint4*>(to.k) + d * page;
  uint4* vd = reinterpret_cast<uint4*>(to.v) + d * page;
  for (int64_t i = begin + threadIdx.x; i < end; i += 512) {
    const bool two = i + 256 < end;
    const int64_t j = two ? i + 256 : i;
    const uint4 a = ks[i], b = vs[i], e = ks[j], f = vs[j];
    kd[i] = a;
    vd[i] = b;
    if (two) {
      kd[j] = e;
      vd[j] = f;
    }
  }
  if (part == 0)
    for (int h = threadIdx.x; h < to.heads; h += 256) {
      to.ks[d * to.heads + h] = from.ks[s * from.heads + h];
      to.vs[d * to.heads + h] = from.vs[s * from.heads + h];
    }
}

}  // namespace qmm
