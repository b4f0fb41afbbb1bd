// 8-bit cache: append new tokens, read pages back as values, copy pages.
#include "kernels.hpp"
#include "kv8_common.hpp"

namespace qmm {
namespace {

// ------------------------------------------------------------------- append
// One workgroup per (sequence, page that gets tokens, head). The block's new
// scale is fl32(amax of its new values / 127), and not below the old scale
// when the page holds earlier tokens; the earlier codes are then brought to
// the new scale, rint(fl32(fl32(c * old) / new)). Slots behind the last token
// become zero. Bound by memory: the new values are read once (the second look
// at them, for the codes, hits the caches), the codes written once.
template <class T>
__global__ __launch_bounds__(256) void kv8_append_kernel(Kv8 c, Kv8Seqs q,
                                                         const uint16_t* __restrict__ kx,
                                                         int64_t ldk,
                                                         const uint16_t* __restrict__ vx,
                                                         int64_t ldv) {
  extern __shared__ __attribute__((aligned(16))) uint8_t vt[];   // new value codes, [D][B + 4]
  __shared__ uint32_t top_k[4], top_v[4];
  const int tid = threadIdx.x, head = blockIdx.y;
  const int B = 1 << c.bt_log2, D = c.dim, D8 = D / 8;
  const SeqAt at_seq = locate(q, blockIdx.x, B, 2, c.bt_log2);
  const int s = at_seq.s, t0 = at_seq.first, n = at_seq.count, len = at_seq.len, item = at_seq.item;
  // a sequence whose tokens cannot be placed (fewer places than tokens) gets
  // its last `len` ones
  const int begin = len - n > 0 ? len - n : 0;
  const int pi = (begin >> c.bt_log2) + item;
  if (n <= 0 || item < 0 || (int64_t)pi * B >= len || pi >= q.W) return;
  const int page = __builtin_amdgcn_readfirstlane(q.table[(int64_t)s * q.W + pi]);
  if (page < 0 || page >= c.pages) return;
  const int o0 = begin > pi * B ? begin - pi * B : 0;                     // first new slot
  const int o1 = len - pi * B < B ? len - pi * B : B;                     // end of the tokens
  const int64_t row0 = t0 + n - len + pi * B;                             // row of slot 0
  const uint16_t* kr = kx + (int64_t)head * D;
  const uint16_t* vr = vx + (int64_t)head * D;
  const int units = (o1 - o0) * D8;

  uint32_t mk = 0, mv = 0;
  for (int u = tid; u < units; u += 256) {
    const int64_t row = row0 + o0 + u / D8;
    const int d = (u % D8) * 8;
    const uint4 a = *reinterpret_cast<const uint4*>(kr + row * ldk + d);
    const uint4 b = *reinterpret_cast<const uint4*>(vr + row * ldv + d);
    mk = amax_pair(amax_pair(amax_pair(amax_pair(mk, a.x), a.y), a.z), a.w);
    mv = amax_pair(amax_pair(amax_pair(amax_pair(mv, b.x), b.y), b.z), b.w);
  }
  mk = wave_umax(amax_halves(mk));
  mv = wave_umax(amax_halves(mv));
  if (tid % 64 == 0) {
    top_k[tid / 64] = mk;
    top_v[tid / 64] = mv;
  }
  const int64_t at = (int64_t)page * c.heads + head;
  const float old_k = c.ks[at], old_v = c.vs[at];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; i++) {
    mk = top_k[i] > mk ? top_k[i] : mk;
    mv = top_v[i] > mv ? top_v[i] : mv;
  }
  auto raise = [&](float was, float now) QMM_INLINE {   // a NaN on either side stays
    return o0 == 0 ? now : was > now || was != was ? was : now;
  };
  const Divisor dk = divisor(raise(old_k, amax_scale<T>(mk)));
  const Divisor dv = divisor(raise(old_v, amax_scale<T>(mv)));
  if (tid == 0) {
    c.ks[at] = dk.s;
    c.vs[at] = dv.s;
  }
  int8_t* kc = c.k + c.block(page, head);
  int8_t* vc = c.v + c.block(page, head);
  // four codes of the earlier tokens at the new scale
  auto again = [&](uint32_t w, float old, const Divisor& d) QMM_INLINE {
    float f[4], r[4];
#pragma unroll
    for (int i = 0; i < 4; i++) f[i] = code_f32(w, i) * old;
    divide_round<4>(f, d, r);
    return pack_codes(r[0], r[1], r[2], r[3]);
  };
  // keys: 8 codes of one token at a time
  const bool same_k = old_k == dk.s, same_v = old_v == dv.s;
  for (int u = tid; u < B * D8; u += 256) {
    const int slot = u / D8, d = (u % D8) * 8;
    uint2* p = reinterpret_cast<uint2*>(kc + slot * D + d);
    if (slot < o0) {
      if (same_k) continue;
      const uint2 w = *p;
      *p = make_uint2(again(w.x, old_k, dk), again(w.y, old_k, dk));
    } else if (slot < o1) {
      float f[8], r[8];
      unpack8(T{}, *reinterpret_cast<const uint4*>(kr + (row0 + slot) * ldk + d), f);
      divide_round<8>(f, dk, r);
      *p = make_uint2(pack_codes(r[0], r[1], r[2], r[3]), pack_codes(r[4], r[5], r[6], r[7]));
    } else {
      *p = make_uint2(0, 0);
    }
  }
  // values: codes to LDS by column, then whole words of four tokens
  const int ldt = B + 4;
  for (int u = tid; u < units; u += 256) {
    const int slot = o0 + u / D8, d = (u % D8) * 8;
    float f[8], r[8];
    unpack8(T{}, *reinterpret_cast<const uint4*>(vr + (row0 + slot) * ldv + d), f);
    divide_round<8>(f, dv, r);
#pragma unroll
    for (int i = 0; i < 8; i++) vt[(d + i) * ldt + slot] = (uint8_t)(int)r[i];
  }
  __syncthreads();
  const int B4 = B / 4;
  for (int u = tid; u < D * B4; u += 256) {
    const int d = u / B4, slot = (u % B4) * 4;
    if (same_v && slot + 4 <= o0) continue;
    uint32_t* p = reinterpret_cast<uint32_t*>(vc + d * B + slot);
    uint32_t was = 0;
    if (slot < o0) {
      was = *p;
      if (!same_v) was = again(was, old_v, dv);
    }
    const uint32_t now = *reinterpret_cast<const uint32_t*>(vt + d * ldt + slot);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t m = 0xffu << (8 * i);
      w |= slot + i < o0 ? was & m : slot + i < o1 ? now & m : 0u;
    }
    *p = w;
  }
}

// --------------------------------------------------------------------- read
// One workgroup per (listed page, head): T(fl32(scale * code)) as [B][D].
template <class T>
__global__ __launch_bounds__(256) void kv8_read_kernel(Kv8 c, const int32_t* __restrict__ pages,
                                                       uint16_t* __restrict__ ko,
                                                       uint16_t* __restrict__ vo) {
  extern __shared__ __attribute__((aligned(16))) uint8_t vt[];   // value codes, [D][B + 4]
  const int tid = threadIdx.x, head = blockIdx.y;
  const int B = 1 << c.bt_log2, D = c.dim, D8 = D / 8, B4 = B / 4, ldt = B + 4;
  const int page = pages[blockIdx.x];
  const bool live = page >= 0 && page < c.pages;   // other numbers read as zeros
  const int64_t at = live ? (int64_t)page * c.heads + head : 0;
  const float sk = c.ks[at], sv = c.vs[at];
  const int8_t* kc = c.k + (live ? c.block(page, head) : 0);
  const int8_t* vc = c.v + (live ? c.block(page, head) : 0);
  const int64_t out = ((int64_t)blockIdx.x * c.heads + head) * B * D;
  for (int u = tid; u < D * B4; u += 256) {
    const int d = u / B4, slot = (u % B4) * 4;
    *reinterpret_cast<uint32_t*>(vt + d * ldt + slot) =
        *reinterpret_cast<const uint32_t*>(vc + d * B + slot);
  }
  for (int u = tid; u < B * D8; u += 256) {
    const uint2 w = *reinterpret_cast<const uint2*>(kc + u * 8);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = live ? code_f32(i < 4 ? w.x : w.y, i % 4) * sk : 0.0f;
    *reinterpret_cast<uint4*>(ko + out + u * 8) = pack8(T{}, f);
  }
  __syncthreads();
  for (int u = tid; u < B * D8; u += 256) {
    const int slot = u / D8, d = (u % D8) * 8;
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; i++)
      f[i] = live ? (float)(int8_t)vt[(d + i) * ldt + slot] * sv : 0.0f;
    *reinterpret_cast<uint4*>(vo + out + u * 8) = pack8(T{}, f);
  }
}

// --------------------------------------------------------------------- copy
// Pages src[i] -> dst[i], between two caches of one shape or within one.
__global__ __launch_bounds__(256) void kv8_copy_kernel(Kv8 to, Kv8 from,
                                                       const int32_t* __restrict__ dst,
                                                       const int32_t* __restrict__ src,
                                                       int parts) {
  const int d = dst[blockIdx.x], s = src[blockIdx.x];
  if (d < 0 || d >= to.pages || s < 0 || s >= from.pages) return;
  copy_page(to, d, from, s, blockIdx.y, parts);
}

Kv8Seqs seqs(const int32_t* table, const int32_t* lens, const int32_t* cu, int64_t S, int64_t W,
             int64_t T) {
  return {table, lens, cu, (int)S, (int)W, (int)T};
}

}  // namespace

hipError_t launch_kv8_append(const Kv8& c, int dt, const void* k, int64_t ldk, const void* v,
                             int64_t ldv, int64_t T, const int32_t* table, const int32_t* lens,
                             const int32_t* cu, int64_t S, int64_t W, hipStream_t st) {
  const dim3 grid((unsigned)((T >> c.bt_log2) + 2 * S), (unsigned)c.heads);
  const size_t lds = (size_t)c.dim * ((1 << c.bt_log2) + 4);
  const Kv8Seqs q = seqs(table, lens, cu, S, W, T);
  const uint16_t *kx = static_cast<const uint16_t*>(k), *vx = static_cast<const uint16_t*>(v);
  if (dt == 0)
    hipLaunchKernelGGL(kv8_append_kernel<F16>, grid, dim3(256), lds, st, c, q, kx, ldk, vx, ldv);
  else
    hipLaunchKernelGGL(kv8_append_kernel<BF16>, grid, dim3(256), lds, st, c, q, kx, ldk, vx, ldv);
  return hipGetLastError();
}

hipError_t launch_kv8_read(const Kv8& c, int dt, const int32_t* pages, int64_t n, void* k, void* v,
                           hipStream_t st) {
  const dim3 grid((unsigned)n, (unsigned)c.heads);
  const size_t lds = (size_t)c.dim * ((1 << c.bt_log2) + 4);
  uint16_t *ko = static_cast<uint16_t*>(k), *vo = static_cast<uint16_t*>(v);
  if (dt == 0)
    hipLaunchKernelGGL(kv8_read_kernel<F16>, grid, dim3(256), lds, st, c, pages, ko, vo);
  else
    hipLaunchKernelGGL(kv8_read_kernel<BF16>, grid, dim3(256), lds, st, c, pages, ko, vo);
  return hipGetLastError();
}

hipError_t launch_kv8_copy(const Kv8& to, const Kv8& from, const int32_t* dst, const int32_t* src,
                           int64_t n, hipStream_t st) {
  const int parts = copy_parts(to);
  hipLaunchKernelGGL(kv8_copy_kernel, dim3((unsigned)n, (unsigned)parts), dim3(256), 0, st, to,
                     from, dst, src, parts);
  return hipGetLastError();
}

}  // namespace qmm
