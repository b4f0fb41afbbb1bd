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
  __device__ int clip_row(int c) const { return c < 0 ? 0 : c > T ? T : c; }
};

// Work items of a ragged batch, `unit` new tokens each: sequence s owns items
// cu[s] / unit + extra * s .. cu[s+1] / unit + extra * (s+1), at least count /
// unit + extra of them. locate() finds the sequence that owns item i (the last
// one whose items start at or before i) and what a workgroup needs to know
// of it. It is the first link of a chain of dependent loads (sequence, pages,
// codes), so the lanes look at 64 boundaries at once: one round trip up to 64
// sequences, two up to 4096.
struct SeqAt {
  int s, first, count, len;   // new tokens are rows first .. first + count
  int item;                   // index of the work item in the sequence
};
__device__ __forceinline__ SeqAt locate(const Kv8Seqs& q, int i, int unit, int extra, int bt_log2) {
  const int lane = threadIdx.x % 64;
  auto starts = [&](int c, int j) QMM_INLINE {
    return (int)((uint32_t)q.clip_row(c) / (uint32_t)unit) + extra * j <= i;
  };
  int lo = 0, n = q.S;   // the sequence is one of lo .. lo + n
  while (n > 64) {
    const int step = (n + 63) / 64, j = lo + lane * step;
    const bool at = j < lo + n && starts(q.cu[min(j, q.S)], j);
    const int c = max(__builtin_popcountll(__ballot(at)), 1) - 1;
    n = min(step, n - c * step);
    lo += c * step;
  }
  const int j = min(lo + lane, q.S);
  const int c = q.cu[j], l = q.lens[min(j, q.S - 1)];
  const int k = max(__builtin_popcountll(__ballot(lane < n && starts(c, j))), 1) - 1;
  const int next = __shfl(c, (k + 1) & 63), past = q.cu[min(lo + 64, q.S)];
  const int first = q.clip_row(__shfl(c, k)), len = max(__shfl(l, k), 0);
  const int64_t most = (int64_t)q.W << bt_log2;
  // (the same in every lane, which the compiler cannot see: made scalar, or
  // every loop over the sequence would be one over lanes)
  SeqAt r;
  r.s = __builtin_amdgcn_readfirstlane(lo + k);
  r.first = __builtin_amdgcn_readfirstlane(first);
  r.count = __builtin_amdgcn_readfirstlane(max(q.clip_row(k < 63 ? next : past) - first, 0));
  r.len = __builtin_amdgcn_readfirstlane(len > most ? (int)most : len);
  r.item = i - ((int)((uint32_t)r.first / (uint32_t)unit) + extra * r.s);
  return r;
}

// Copies part `part` of `parts` of a page (codes, and with part 0 the scales)
// with 256 threads, eight 16-byte pieces in flight per thread.
constexpr int kCopyBytes = 16384;   // of keys and of values each, per part
__host__ __device__ inline int copy_parts(const Kv8& c) {
  const int64_t bytes = c.block(1, 0);
  return (int)((bytes + kCopyBytes - 1) / kCopyBytes);
}
__device__ __forceinline__ void copy_page(const Kv8& to, int64_t d, const Kv8& from, int64_t s,
                                          int part, int parts) {
  const int page = (int)(to.block(1, 0) / 16);   // pieces of a page
  const int per = (page + parts - 1) / parts, begin = part * per;
  const int end = begin + per < page ? begin + per : page;
  const u32x4_t* ks = reinterpret_cast<const u32x4_t*>(from.k) + s * page;
  const u32x4_t* vs = reinterpret_cast<const u32x4_t*>(from.v) + s * page;
  u32x4_t* kd = reinterpret_cast<u32x4_t*>(to.k) + d * page;
  u32x4_t* vd = reinterpret_cast<u32x4_t*>(to.v) + d * page;
  int i = begin + threadIdx.x;
  for (; i + 768 < end; i += 1024) {
    const u32x4_t a0 = ks[i], a1 = ks[i + 256], a2 = ks[i + 512], a3 = ks[i + 768];
    const u32x4_t b0 = vs[i], b1 = vs[i + 256], b2 = vs[i + 512], b3 = vs[i + 768];
    kd[i] = a0;
    kd[i + 256] = a1;
    kd[i + 512] = a2;
    kd[i + 768] = a3;
    vd[i] = b0;
    vd[i + 256] = b1;
    vd[i + 512] = b2;
    vd[i + 768] = b3;
  }
  for (; i < end; i += 256) {
    const u32x4_t a = ks[i], b = vs[i];
    kd[i] = a;
    vd[i] = b;
  }
  if (part == 0)
    for (int h = threadIdx.x; h < to.heads; h += 256) {
      to.ks[d * to.heads + h] = from.ks[s * from.heads + h];
      to.vs[d * to.heads + h] = from.vs[s * from.heads + h];
    }
}

}  // namespace qmm
