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
// become zero. Bound by memory: new values are read once, codes written once
// (20278 tokens of 8 x 128, f16: 31 us, 4.0 TB/s; 64 single tokens: 7 us, the
// chain of loads from the sequence to the page's old codes).
//
// A thread's unit is 4 slots by 8 columns of the keys or of the values: four
// 16-byte loads, held in registers between the maximum and the codes; the key
// codes go out as 8 bytes per slot, the value codes, transposed by the packing,
// as a word of four slots per column. The lanes of key units run along the
// columns, those of value units along the slots, so that both write runs.
template <class T, int U>   // U units per thread
__global__ __launch_bounds__(256) void kv8_append_kernel(Kv8 c, Kv8Seqs q,
                                                         const uint16_t* __restrict__ kx,
                                                         int64_t ldk,
                                                         const uint16_t* __restrict__ vx,
                                                         int64_t ldv) {
  __shared__ uint32_t top_k[4], top_v[4];
  const int tid = threadIdx.x, head = blockIdx.y;
  const int B = 1 << c.bt_log2, D = c.dim;
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
  const int64_t row0 = (int64_t)t0 + n - len + (int64_t)pi * B;           // row of slot 0
  const int64_t at = (int64_t)page * c.heads + head;
  const float old_k = c.ks[at], old_v = c.vs[at];
  const int half = (B / 4) * (D / 8);   // key units, then as many value units

  struct Unit {
    bool value, live;
    int slot, d;   // first of 4 slots, first of 8 columns
  };
  auto unit = [&](int i) QMM_INLINE {
    const int u = i * 256 + tid;
    Unit x;
    x.value = u >= half;
    x.live = u < 2 * half;
    if (x.value) {
      x.slot = (u - half) % (B / 4) * 4;
      x.d = (u - half) / (B / 4) * 8;
    } else {
      x.slot = u / (D / 8) * 4;
      x.d = u % (D / 8) * 8;
    }
    return x;
  };
  uint4 w[U][4];
  uint32_t mk = 0, mv = 0;
#pragma unroll
  for (int i = 0; i < U; i++) {
    const Unit x = unit(i);
    const uint16_t* p = (x.value ? vx : kx) + (int64_t)head * D + x.d;
    const int64_t ld = x.value ? ldv : ldk;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const bool in = x.live && x.slot + j >= o0 && x.slot + j < o1;
      w[i][j] = in ? *reinterpret_cast<const uint4*>(p + (row0 + x.slot + j) * ld)
                   : make_uint4(0, 0, 0, 0);
      m = amax_pair(amax_pair(amax_pair(amax_pair(m, w[i][j].x), w[i][j].y), w[i][j].z), w[i][j].w);
    }
    m = amax_halves(m);
    mk = !x.value && m > mk ? m : mk;
    mv = x.value && m > mv ? m : mv;
  }
  mk = wave_umax(mk);
  mv = wave_umax(mv);
  if (tid % 64 == 0) {
    top_k[tid / 64] = mk;
    top_v[tid / 64] = mv;
  }
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
  // four codes of the earlier tokens at the new scale
  auto again = [&](uint32_t word, float old, const Divisor& d) QMM_INLINE {
    float f[4], r[4];
#pragma unroll
    for (int i = 0; i < 4; i++) f[i] = code_f32(word, i) * old;
    divide_round<4>(f, d, r);
    return pack_codes(r[0], r[1], r[2], r[3]);
  };
#pragma unroll
  for (int i = 0; i < U; i++) {
    const Unit x = unit(i);
    if (!x.live) continue;
    const float old = x.value ? old_v : old_k;
    const Divisor d = x.value ? dv : dk;
    const bool same = old == d.s;
    if (same && x.slot + 4 <= o0) continue;   // earlier tokens, as they were
    float r[4][8];
#pragma unroll
    for (int j = 0; j < 4; j++) {
#pragma unroll
      for (int e = 0; e < 8; e++) r[j][e] = 0.0f;
      if (x.slot + j >= o0 && x.slot + j < o1) {
        float f[8];
        unpack8(T{}, w[i][j], f);
        divide_round<8>(f, d, r[j]);
      }
    }
    if (!x.value) {
      int8_t* p = c.k + c.block(page, head) + x.slot * D + x.d;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        uint2* to = reinterpret_cast<uint2*>(p + j * D);
        uint2 code = make_uint2(pack_codes(r[j][0], r[j][1], r[j][2], r[j][3]),
                                pack_codes(r[j][4], r[j][5], r[j][6], r[j][7]));
        if (x.slot + j < o0) {
          if (same) continue;
          code = *to;
          code = make_uint2(again(code.x, old, d), again(code.y, old, d));
        }
        *to = code;
      }
    } else {
      int8_t* p = c.v + c.block(page, head) + x.d * B + x.slot;
      const int kept = o0 - x.slot;   // slots of the word with earlier tokens
      const uint32_t mask = kept <= 0 ? 0u : kept >= 4 ? ~0u : (1u << (8 * kept)) - 1u;
#pragma unroll
      for (int e = 0; e < 8; e++) {
        uint32_t* to = reinterpret_cast<uint32_t*>(p + e * B);
        uint32_t code = pack_codes(r[0][e], r[1][e], r[2][e], r[3][e]);
        if (mask) {
          const uint32_t was = same ? *to : again(*to, old, d);
          code = (code & ~mask) | (was & mask);
        }
        *to = code;
      }
    }
  }
}

// --------------------------------------------------------------------- read
// One workgroup per (listed page, head): T(fl32(scale * code)) as [B][D]. Bound by
// memory (20352 tokens of 8 x 128: 21 us).
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
  const Kv8Seqs q = seqs(table, lens, cu, S, W, T);
  const uint16_t *kx = static_cast<const uint16_t*>(k), *vx = static_cast<const uint16_t*>(v);
  const int units = (2 * (c.dim << c.bt_log2) / 32 + 255) / 256;   // per thread: 1, 2 or 4
  auto go = [&]<class T_>() {
    auto each = [&]<int U>() {
      hipLaunchKernelGGL((kv8_append_kernel<T_, U>), grid, dim3(256), 0, st, c, q, kx, ldk, vx, ldv);
    };
    if (units == 1) each.template operator()<1>();
    else if (units == 2) each.template operator()<2>();
    else each.template operator()<4>();
  };
  if (dt == 0) go.template operator()<F16>();
  else go.template operator()<BF16>();
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
