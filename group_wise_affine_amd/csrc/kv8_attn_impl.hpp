// Attention over the paged 8-bit cache, causal from the end: the i-th of a
// sequence's n new tokens sits at position len - n + i and sees the positions
// up to its own. Grouped heads: query heads h*G .. h*G + G read cache head h.
//
//   x_j = scale * ks(page of j) * (q . kcode_j),   m = max x_j,
//   out = sum_j exp(x_j - m) * vs(page of j) * vcode_j / sum_j exp(x_j - m)
//
// A row that sees no key gives zeros and a logarithm of -inf. Places whose
// page number is outside the pool are not seen.
//
// Both products run on the f16 matrix units: codes are exact in f16, queries
// too (bf16 rows are first scaled by a power of two), so only the weights
// exp(x - m) * vs are rounded on their way into the second product, relative
// to the row's largest (to 11 bits for bf16 results, to two f16 terms for f16
// ones); sums, maxima and the normaliser stay in fp32.
//
// Three masks: causal alone; a sliding window with the first tokens visible
// (sinks); and a tree of drafted tokens. Each is an instance of its own of the
// same kernels (the sources that include this file), so that a mask costs the
// others nothing.
#pragma once

#include "kernels.hpp"
#include "kv8_common.hpp"

namespace qmm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTile = 64;   // tokens per step of a wavefront
constexpr int kMaxSplits = 128;   // parts of a sequence

// What a query at position p of its sequence sees of the positions up to p:
// everything; those above p - window and those below sinks; or, where the last
// new tokens (at most kTreeTokens) are a tree of drafts, what precedes the tree
// and the token's ancestors in it.
enum class Mask { kCausal, kWindow, kTree };
constexpr int kTreeTokens = 64;

struct AttnArgs {
  Kv8 c;
  Kv8Seqs q;
  const uint16_t* x;   // queries, row t at x + t * ldq
  int64_t ldq;
  int G;               // query heads per cache head, 16 at a time
  int unit;            // new tokens per workgroup
  int step, extra;     // items of a sequence: one for each `step` new tokens, and so many
  int items;           // of the batch
  int bundle_log2;     // draft kernel: items that follow each other on one XCD
  int many;            // sequences with more query rows than this are the prompt kernel's
  float scale;         // magnitude of the scores' scale, times log2 e
  uint32_t flip;       // its sign, as the sign bits of two queries
  uint16_t* out;       // [T][heads * G][D]
  float* lse;          // [T][heads * G] or null
  int splits, per;     // workgroups of a sequence (gridDim.z), tiles of each
  float* ws;
  int window, sinks;       // kWindow; sinks <= 2^30
  const int32_t* parent;   // kTree: [T]
};

// The tiles that an item looks at: those of its sequence up to `most`, without
// the ones that lie between the sinks and the window of its first row (at
// position `low`). The t-th of them is tile t, and from `near` on t + gap.
struct Walk {
  int tiles, near, gap;
  __device__ __forceinline__ int real(int t) const { return t + (t >= near ? gap : 0); }
};
template <Mask M>
__device__ __forceinline__ Walk walk(const AttnArgs& a, int most, int low) {
  Walk w{most > 0 ? (most + kTile - 1) / kTile : 0, 0, 0};
  if constexpr (M == Mask::kWindow) {
    const int lo = max(low - a.window + 1, 0);   // (low > -2^24, window >= 1)
    const int near = (min(a.sinks, lo) + kTile - 1) / kTile, gap = lo / kTile - near;
    if (gap > 0 && w.tiles > 0) {
      w.near = near;
      w.gap = gap;
      w.tiles -= gap;
    }
  }
  return w;
}

// What the lanes' rows see, as bits: of the new tokens that are a tree, those on
// the way from this row's token `i` (of n new ones) to its root, the token itself
// among them. Every wavefront finds its rows' by itself: a lane holds the parent
// of each of the at most 64 tokens, and the rows walk up together. A parent that
// is not an earlier token of the tree makes the token a root, so that every walk
// ends.
__device__ __forceinline__ int tree_parent(const AttnArgs& a, int t0, int n) {
  const int lane = threadIdx.x % 64, b = max(n - kTreeTokens, 0);
  return b + lane < n ? a.parent[t0 + b + lane] : -1;
}
__device__ __forceinline__ uint64_t tree_path(int parent, int n, int i) {
  const int lane = threadIdx.x % 64, b = max(n - kTreeTokens, 0);
  // (unsigned: any number may stand there, and one below b becomes a large one)
  const uint32_t earlier = (uint32_t)parent - (uint32_t)b;
  parent = earlier < (uint32_t)lane ? (int)earlier : -1;
  int at = i - b;
  uint64_t path = 0;
  while (__any(at >= 0)) {
    path |= at >= 0 ? 1ull << at : 0;
    const int up = __shfl(parent, at & 63);
    at = at >= 0 ? up : -1;
  }
  return path;
}

// bits 0 .. n - 1, for any n
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1;
}
// The tokens of the tile at `base` that a row at position `limit` sees; the tree
// starts at position `tree`.
template <Mask M>
__device__ __forceinline__ uint64_t seen_bits(const AttnArgs& a, int base, int limit, int tree,
                                              uint64_t path) {
  uint64_t seen = low_bits(limit - base + 1);
  if constexpr (M == Mask::kWindow)
    seen &= ~low_bits(limit - a.window + 1 - base) | low_bits(a.sinks - base);
  if constexpr (M == Mask::kTree) {
    const int t = tree - base;
    seen &= t >= 64 ? ~0ull : t >= 0 ? low_bits(t) | path << t : t > -64 ? path >> -t : 0;
  }
  return seen;
}
// Whether every row at positions low .. high sees the whole tile
template <Mask M>
__device__ __forceinline__ bool all_seen(const AttnArgs& a, int base, int low, int high, int tree) {
  const int last = base + kTile - 1;
  if constexpr (M == Mask::kWindow)
    return last <= low && (base > high - a.window || last < a.sinks);
  if constexpr (M == Mask::kTree) return last <= low && last < tree;
  return last <= low;
}

// eight signed codes (two words) as f16: 1024 + (code + 128) - 1152, exact
__device__ __forceinline__ half8_t codes_f16(uint32_t a, uint32_t b) {
  const uint32_t m = 0x64646464u;
  a ^= 0x80808080u;
  b ^= 0x80808080u;
  const half2_t off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
  uint32_t r[4] = {__builtin_amdgcn_perm(m, a, 0x04010400u), __builtin_amdgcn_perm(m, a, 0x04030402u),
                   __builtin_amdgcn_perm(m, b, 0x04010400u), __builtin_amdgcn_perm(m, b, 0x04030402u)};
#pragma unroll
  for (int i = 0; i < 4; i++)
    r[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, r[i]) + off);
  return __builtin_bit_cast(half8_t, make_uint4(r[0], r[1], r[2], r[3]));
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint4 load_q(const uint16_t* p, uint32_t flip) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  return make_uint4(u.x ^ flip, u.y ^ flip, u.z ^ flip, u.w ^ flip);
}
// bf16 queries: a row times 2^-e, 2^e the power of two below its largest
// magnitude (bits m), is exact in f16 down to 2^-14 of that (fewer bits below)
struct Pow2 {
  float up, down;
};
__device__ __forceinline__ Pow2 row_power(uint32_t m) {
  int e = (int)(m >> 7) - 127;
  e = e < -126 ? -126 : e > 126 ? 126 : e;   // both powers are finite and normal
  return {__builtin_bit_cast(float, (uint32_t)(127 + e) << 23),
          __builtin_bit_cast(float, (uint32_t)(127 - e) << 23)};
}
__device__ __forceinline__ half8_t bf16_to_f16(const uint4& u, float down) {
  float f[8];
  unpack8(BF16{}, u, f);
  half8_t r;
#pragma unroll
  for (int i = 0; i < 8; i++) r[i] = (_Float16)(f[i] * down);
  return r;
}

// The weights 2^x * vs (x a score times log2 e) go into the second product as
// f16 relative to 2^w, w the largest x + log2 vs that the row has seen: the
// page that carries a result keeps its bits, however small its scale beside
// others of no weight. The sum of 2^x is held relative to 2^base, base the
// largest x, or up to 2^64 below it where w lies far below (the keys of weight
// have values of nearly no scale): the exponentials that then matter stay within
// fp32. Both only rise as a row goes on.
struct Refs {
  float w, base;
};
constexpr float kNone = -0x1.fffffep+127f;   // before a row's first key
// from tokens whose largest x is m and whose largest x + log2 vs is w
__device__ __forceinline__ Refs rise(Refs r, float m, float w) {
  Refs n;
  n.w = fmaxf(r.w, w);
  n.base = fmaxf(r.base, fmaxf(m - 64.0f, fminf(m, n.w + 64.0f)));
  n.w = fmaxf(n.w, n.base - 126.0f);
  return n;
}
// vs * 2^(base - w), finite for a finite scale (where the product would not be,
// 2^(x - base) is 0); a NaN stays
__device__ __forceinline__ float weight_scale(float vs, const Refs& at) {
  const float r = vs * __builtin_amdgcn_exp2f(at.base - at.w);
  return r > 0x1.fffffep+127f ? 0x1.fffffep+127f : r;
}

// Two weights as two f16 terms each, the rounding and what it leaves. The compiler is not
// to know how the first came to be: it would round the product that a weight is once more
// for the second, by v_fma_mix of the exact product where the first is v_cvt of the one
// rounded to fp32, and where these differ (one weight in 2^13) a bit of eleven is lost.
struct Terms {
  half2_t hi, lo;
};
__device__ __forceinline__ Terms two_terms(float w0, float w1) {
  uint32_t h = __builtin_bit_cast(uint32_t, half2_t{(_Float16)w0, (_Float16)w1});
  asm("" : "+v"(h));
  const half2_t hi = __builtin_bit_cast(half2_t, h);
  return {hi, half2_t{(_Float16)(w0 - (float)hi[0]), (_Float16)(w1 - (float)hi[1])}};
}
// weight i of eight, in two terms when the next one is there too
template <bool TWO>
__device__ __forceinline__ void put_weight(half8_t& hi, half8_t& lo, int i, float w, float& before) {
  if constexpr (!TWO) {
    hi[i] = (_Float16)w;
  } else if (i % 2 == 0) {
    before = w;
  } else {
    const Terms t = two_terms(before, w);
    hi[i - 1] = t.hi[0];
    hi[i] = t.hi[1];
    lo[i - 1] = t.lo[0];
    lo[i] = t.lo[1];
  }
}

// two outputs of a row, and whether it has seen a key at all
struct Share {
  uint32_t pair;
  bool any;
};
template <class T>
__device__ __forceinline__ Share share(float v0, float v1, float l) {
  Share s;
  s.any = l > 0.0f || l != l;
  const float back = s.any ? 1.0f / l : 0.0f;
  s.pair = from_f32(T{}, s.any ? v0 * back : 0.0f) |
           (uint32_t)from_f32(T{}, s.any ? v1 * back : 0.0f) << 16;
  return s;
}
// A part in the scratch buffer: R rows' maxima and sums, then the rows. R is 16
// for the decode kernel, kDraftRows for the draft kernel and kPromptRows for the
// prompt kernel.
constexpr int kDraftRows = 32;
constexpr int kPromptRows = 128;
template <int D, int R>
constexpr int kPart = R * (D + 2);

// the value of the lane 32 away
__device__ __forceinline__ float other_half(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, threadIdx.x & 32 ? r[0] : r[1]);
}

// ------------------------------------------------------------------- decode
// Up to 16 query rows (tokens x heads of one group) per workgroup, NW
// wavefronts. A wavefront takes every NW-th tile of 64 tokens and holds its
// whole state in registers; no shared memory until the wavefronts' results
// are joined at the end.
//
// S^T = K Q^T with v_mfma_f32_16x16x32_f16: row i of the A operand of the j-th
// of four products is token 16 * (i/4) + 4 * j + i%4 of the tile, so that lane
// group g = lane/16 gets the scores of tokens 16 g .. 16 g + 16 of query
// lane%16: exactly the order in which the B operand of O^T = V^T P^T wants
// the weights, and in which V^T is read (16 tokens of one column per 16-byte
// load). Nothing moves between lanes but the maximum.
//
// Bound by reading codes once: 48 contexts of up to 8192 tokens, 8 heads of
// 128, 414 MB, in 105 us, 3.9 TB/s (the same loads alone: 95 us); one context of
// 131071 tokens, 2 heads, 67 MB, in 16.8.
template <Mask M, class T, int D, int BT, int NW>   // pages of 1 << BT tokens
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : D == 128 ? 2 : 3) void kv8_decode_kernel(AttnArgs a) {
  constexpr int KD = D / 64, VD = D / 16;
  // f16 results: the weights go in as two f16 terms, since 11 bits of them would
  // cost as much as rounding the result
  constexpr bool kTwo = __is_same(T, F16);
  const int tid = threadIdx.x, lane = tid % 64;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);   // uniform: scalar
  const int col = lane % 16, g = lane / 16;
  const int blocks = (a.G + 15) / 16;   // of heads in a group
  const int head = blockIdx.y / blocks, h0 = blockIdx.y % blocks * 16, split = blockIdx.z;
  const int G = min(16, a.G - h0);
  const Kv8& c = a.c;
  const SeqAt seq = locate(a.q, blockIdx.x, a.step, a.extra, BT);
  const int s = seq.s, t0 = seq.first, n = seq.count, len = seq.len, item = seq.item;
  const int i0 = item * a.unit;
  if (item < 0 || i0 >= n || (int64_t)n * a.G > a.many) return;
  const int ntok = min(n - i0, a.unit);
  const int rows = ntok * G;                 // <= 16
  // positions that the last row sees, tiles of them, this workgroup's share
  const int most = len - n + i0 + ntok;
  const Walk path = walk<M>(a, most, len - n + i0);
  const int tiles = path.tiles;
  const int per = a.per;
  const int parts = tiles > 0 ? (tiles + per - 1) / per : 1;
  if (split >= parts) return;
  const int first = split * per, last = min(first + per, tiles);

  // this lane's query row: token col / G, head col % G (columns past the rows
  // repeat the first one, and nothing reads them)
  const int ct = col < rows ? col / G : 0, ch = col < rows ? col % G : 0;
  const int64_t trow = t0 + i0 + ct;
  const int qh = head * a.G + h0 + ch;
  const int min_limit = len - n + i0;   // last position that every row sees
  const int limit = min_limit + ct;     // that this one sees
  const int tree = len - min(n, kTreeTokens);
  int parent = -1;
  if constexpr (M == Mask::kTree) parent = tree_parent(a, t0, n);
  uint4 u[KD][2];   // asked for first, looked at when the codes are on their way
  {
    const uint16_t* qr = a.x + trow * a.ldq + (int64_t)qh * D + g * 16;
#pragma unroll
    for (int b = 0; b < KD; b++)
#pragma unroll
      for (int h = 0; h < 2; h++) u[b][h] = load_q(qr + b * 64 + h * 8, a.flip);
  }
  half8_t qf[KD][2];
  float qs = a.scale;
  auto take_queries = [&]() QMM_INLINE {
    if constexpr (__is_same(T, F16)) {
#pragma unroll
      for (int b = 0; b < KD; b++)
#pragma unroll
        for (int h = 0; h < 2; h++) qf[b][h] = __builtin_bit_cast(half8_t, u[b][h]);
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int b = 0; b < KD; b++)
#pragma unroll
        for (int h = 0; h < 2; h++)
          m = amax_pair(amax_pair(amax_pair(amax_pair(m, u[b][h].x), u[b][h].y), u[b][h].z), u[b][h].w);
      m = amax_halves(m);
      m = umax(m, (uint32_t)__shfl_xor((int)m, 16));
      m = umax(m, (uint32_t)__shfl_xor((int)m, 32));
      const Pow2 e = row_power(m);
      qs *= e.up;
#pragma unroll
      for (int b = 0; b < KD; b++)
#pragma unroll
        for (int h = 0; h < 2; h++) qf[b][h] = bf16_to_f16(u[b][h], e.down);
    }
  };

  float4_t o[VD];
#pragma unroll
  for (int i = 0; i < VD; i++) o[i] = float4_t{0, 0, 0, 0};
  Refs at{kNone, kNone};   // O relative to 2^at.w, l to 2^at.base
  float l_run = 0.0f;

  const int32_t* row = a.q.table + (int64_t)s * a.q.W;
  // Every wavefront walks a run of tiles. The numbers and scales of the next 64
  // pages sit one per lane, so that nothing but the codes is loaded in the
  // loop, and the loads run ahead of their use: a tile's keys are asked for
  // when those of the tile before have been multiplied, its values when those
  // of the tile before are spent.
  constexpr int kPer = kTile >> BT;   // pages of a tile
  const int kg = (col / 4) * 16;      // first token of this lane's K rows in a tile
  int pages = -1;                     // page `lane` of the chunk of 64
  float pages_ks = 0.0f, pages_vs = 0.0f;
  auto chunk = [&](int tile) QMM_INLINE {   // pages from this tile's first on
    const int t = path.real(tile) * kTile + (lane << BT);
    const int p = t < most ? row[t >> BT] : -1;   // most <= W << BT
    pages = p < c.pages ? p : -1;
    const int64_t blk = (int64_t)(pages < 0 ? 0 : pages) * c.heads + head;
    pages_ks = c.ks[blk];
    pages_vs = c.vs[blk];
  };
  int pk, pv;      // this lane's pages of keys and values in a tile
  auto look_up = [&](int i) QMM_INLINE {   // the chunk's i-th tile
    pk = __shfl(pages, i * kPer + (kg >> BT));
    pv = __shfl(pages, i * kPer + (g * 16 >> BT));
  };
  u32x4_t kw[4][KD], vw[VD];
  auto fetch_keys = [&]() QMM_INLINE {
    const int8_t* kp = c.k + c.block(pk < 0 ? 0 : pk, head) +
                       ((kg & ((1 << BT) - 1)) + col % 4) * D + g * 16;
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int b = 0; b < KD; b++)
        kw[j][b] = *(
            reinterpret_cast<const u32x4_t*>(kp + j * 4 * D + b * 64));
  };
  auto fetch_values = [&](int page) QMM_INLINE {
    const int8_t* vp = c.v + c.block(page < 0 ? 0 : page, head) + (col << BT) +
                       ((g * 16) & ((1 << BT) - 1));
#pragma unroll
    for (int i = 0; i < VD; i++)
      vw[i] = *(
          reinterpret_cast<const u32x4_t*>(vp + ((i * 16) << BT)));
  };
  const int run = per / NW;   // tiles of a wavefront
  const int w_first = first + wave * run, w_last = min(w_first + run, last);
  auto begin = [&](int tile) QMM_INLINE {
    chunk(tile);
    look_up(0);
    fetch_keys();
    fetch_values(pv);
    // an (empty) use: the wait for the scales belongs here, and not in the
    // loop, where it would take the code loads in flight with it
    asm volatile("" : "+v"(pages), "+v"(pages_ks), "+v"(pages_vs));
  };
  if (w_first < w_last) begin(w_first);
  take_queries();
  uint64_t line = 0;
  if constexpr (M == Mask::kTree) line = tree_path(parent, n, i0 + ct);
  // (a step that is a constant keeps the loop's counter scalar: 21.4 us for one context of
  // 131071 tokens, 2 heads, 21.8 with a step of `count`)
  int short_of = 0;   // a chunk's 64 pages: it ends where the sinks do
  for (int from = w_first; from < w_last; from += (1 << BT) - short_of) {
   int count = min(w_last - from, 1 << BT);
   if constexpr (M == Mask::kWindow) {
     if (from < path.near) count = min(count, path.near - from);
     short_of = (1 << BT) - count;
   }
   if (from != w_first) begin(from);
   for (int i = 0; i < count; i++) {
    const int base = (path.real(from) + i) * kTile;
    const int page = pv;
    const float ks = __shfl(pages_ks, i * kPer + (g * 16 >> BT));
    const float vs_now = __shfl(pages_vs, i * kPer + (g * 16 >> BT));
    const bool more = i + 1 < count;
    if (more) look_up(i + 1);
    float4_t sc[4];
#pragma unroll
    for (int j = 0; j < 4; j++) sc[j] = float4_t{0, 0, 0, 0};
#pragma unroll
    for (int b = 0; b < KD; b++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
#pragma unroll
        for (int j = 0; j < 4; j++)
          sc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
              codes_f16(kw[j][b][2 * h], kw[j][b][2 * h + 1]), qf[b][h], sc[j], 0, 0, 0);
        // (the compiler would convert the whole tile first and run out of registers)
        __builtin_amdgcn_sched_barrier(0);
      }
    const float f = ks * qs;
    if (more) fetch_keys();
    __builtin_amdgcn_sched_barrier(0);
    float p[16];
#pragma unroll
    for (int i = 0; i < 16; i++) p[i] = sc[i / 4][i % 4] * f;
    float r = vs_now;
    if (!(all_seen<M>(a, base, min_limit, min_limit + ntok - 1, tree) && __all(page >= 0))) {
      // what is not seen weighs nothing, whatever its scale
      if constexpr (M == Mask::kCausal) {   // tokens 0 .. left of this lane's 16 are seen
        const int left = page < 0 ? -1 : limit - (base + g * 16);
#pragma unroll
        for (int i = 0; i < 16; i++) p[i] = i <= left ? p[i] : -__builtin_inff();
        r = left < 0 ? 0.0f : r;
      } else {
        const uint32_t seen =
            page < 0 ? 0 : (uint32_t)(seen_bits<M>(a, base, limit, tree, line) >> (g * 16)) & 0xffffu;
#pragma unroll
        for (int i = 0; i < 16; i++) p[i] = seen >> i & 1 ? p[i] : -__builtin_inff();
        r = seen == 0 ? 0.0f : r;
      }
    }
    float mx = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < 16; i++) mx = fmaxf(mx, p[i]);
    // (an infinite or NaN scale leaves the reference, a zero's logarithm is -inf)
    float wx = r < __builtin_inff() ? mx + __builtin_amdgcn_logf(r) : -__builtin_inff();
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    wx = fmaxf(wx, __shfl_xor(wx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    wx = fmaxf(wx, __shfl_xor(wx, 32));
    const Refs to = rise(at, mx, wx);
    const float down = __builtin_amdgcn_exp2f(at.w - to.w);   // what the values so far shrink by
    l_run *= __builtin_amdgcn_exp2f(at.base - to.base);
    at = to;
    r = weight_scale(r, at);
    // (always: a branch around it costs more registers than it saves cycles)
#pragma unroll
    for (int i = 0; i < VD; i++) o[i] *= down;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      half8_t pf, pl;
      float before;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float e = __builtin_amdgcn_exp2f(p[8 * h + i] - at.base);
        l_run += e;
        put_weight<kTwo>(pf, pl, i, e * r, before);
      }
#pragma unroll
      for (int i = 0; i < VD; i++) {
        const half8_t vf = codes_f16(vw[i][2 * h], vw[i][2 * h + 1]);
        o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf, o[i], 0, 0, 0);
        if constexpr (kTwo) o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pl, o[i], 0, 0, 0);
        if (i % 2 == 1) __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (more) fetch_values(pv);
    __builtin_amdgcn_sched_barrier(0);
   }
  }
  l_run += __shfl_xor(l_run, 16);
  l_run += __shfl_xor(l_run, 32);

  // join the wavefronts: column (query row) col, o[i][e] is value column
  // 16 i + 4 g + e
  __shared__ float jm[NW][16], jl[NW][16];
  extern __shared__ __attribute__((aligned(16))) float jo[];   // [NW][16][D]
  if (g == 0) {
    jm[wave][col] = at.base;
    jl[wave][col] = l_run;
  }
  const float vref = __builtin_amdgcn_exp2f(at.w - at.base);
#pragma unroll
  for (int i = 0; i < VD; i++)
    *reinterpret_cast<float4_t*>(jo + ((wave * 16 + col) * D + i * 16 + g * 4)) = o[i] * vref;
  __syncthreads();
  // (gridDim.y, computed: it lies behind the arguments, on a line of its own, and a load
  // of it takes 0.2 us)
  const int columns = c.heads * blocks;
  float* part = a.ws + (((int64_t)blockIdx.x * columns + blockIdx.y) * a.splits + split) * kPart<D, 16>;
  for (int i = tid; i < rows * (D / 2); i += 64 * NW) {
    const int r = i / (D / 2), d = i % (D / 2) * 2;
    float m = kNone;
#pragma unroll
    for (int w = 0; w < NW; w++) m = fmaxf(m, jm[w][r]);
    float l = 0.0f, v0 = 0.0f, v1 = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; w++) {
      const float e = __builtin_amdgcn_exp2f(jm[w][r] - m);
      const float2 v = *reinterpret_cast<const float2*>(jo + (w * 16 + r) * D + d);
      l += jl[w][r] * e;
      v0 += v.x * e;
      v1 += v.y * e;
    }
    if (parts == 1) {
      const int64_t at = (int64_t)(t0 + i0 + r / G) * (c.heads * a.G) + head * a.G + h0 + r % G;
      const Share sh = share<T>(v0, v1, l);
      *reinterpret_cast<uint32_t*>(a.out + at * D + d) = sh.pair;
      if (d == 0 && a.lse) a.lse[at] = sh.any ? fmaf(m, kLn2, logf(l)) : -__builtin_inff();
    } else {
      *reinterpret_cast<float2*>(part + 32 + r * D + d) = make_float2(v0, v1);
      if (d == 0) *reinterpret_cast<float2*>(part + 2 * r) = make_float2(m, l);
    }
  }
}

// Where a workgroup of a join kernel works: the query row `at` of the outputs
// and the number of parts of its sequence (at most 1: nothing to join).
struct JoinAt {
  int64_t at;
  int parts;
};
template <Mask M, int R>
__device__ __forceinline__ JoinAt join_at(const AttnArgs& a, int unit, int r) {
  constexpr bool PROMPT = R == kPromptRows;
  const int blocks = PROMPT ? 1 : (a.G + R - 1) / R, columns = a.c.heads * blocks;
  const int index = unit / columns, column = unit % columns;
  const int head = column / blocks, h0 = column % blocks * R;
  const int G = PROMPT ? a.G : min(R, a.G - h0);
  const SeqAt q = locate(a.q, index, a.step, a.extra, a.c.bt_log2);
  const int i0 = q.item * a.unit;
  JoinAt j{0, 0};
  if (q.item < 0 || i0 >= q.count || ((int64_t)q.count * a.G > a.many) != PROMPT) return j;
  const int ntok = min(q.count - i0, a.unit);
  if (r >= ntok * G) return j;
  const int most = q.len - q.count + i0 + ntok;
  j.parts = (walk<M>(a, most, q.len - q.count + i0).tiles + a.per - 1) / a.per;
  j.at = (int64_t)(q.first + i0 + r / G) * (a.c.heads * a.G) + head * a.G + h0 + r % G;
  return j;
}
template <class T>
__device__ __forceinline__ void join_out(const AttnArgs& a, int64_t at, int D, int d, float v0,
                                         float v1, float m, float l) {
  const Share sh = share<T>(v0, v1, l);
  *reinterpret_cast<uint32_t*>(a.out + at * D + d) = sh.pair;
  if (d == 0 && a.lse) a.lse[at] = sh.any ? fmaf(m, kLn2, logf(l)) : -__builtin_inff();
}

// Few parts (at most kFewParts): a thread joins two values of a row by itself.
// (48 contexts of up to 6 parts: 8.5 us with the kernel below, 4.9 with this.)
constexpr int kFewParts = 16;
constexpr int few_parts(int R) { return R == kDraftRows ? 32 : kFewParts; }
template <Mask M, class T, int D, int R>
__global__ __launch_bounds__(256) void kv8_join_few_kernel(AttnArgs a) {
  constexpr int kFloats = kPart<D, R>, kFew = few_parts(R);
  const int r = blockIdx.y * (512 / D) + threadIdx.x / (D / 2), d = threadIdx.x % (D / 2) * 2;
  const float* part = a.ws + (int64_t)blockIdx.x * a.splits * kFloats;
  float2 v[kFew], ml[kFew];
#pragma unroll
  for (int w = 0; w < kFew; w++)
    if (w < a.splits) {
      ml[w] = *reinterpret_cast<const float2*>(part + w * kFloats + 2 * r);
      v[w] = *reinterpret_cast<const float2*>(part + w * kFloats + 2 * R + r * D + d);
    }
  const JoinAt j = join_at<M, R>(a, blockIdx.x, r);
  if (j.parts <= 1) return;
  float m = kNone, l = 0.0f, v0 = 0.0f, v1 = 0.0f;
#pragma unroll
  for (int w = 0; w < kFew; w++)
    if (w < j.parts) m = fmaxf(m, ml[w].x);
#pragma unroll
  for (int w = 0; w < kFew; w++)
    if (w < j.parts) {
      const float e = __builtin_amdgcn_exp2f(ml[w].x - m);
      l += ml[w].y * e;
      v0 = fmaf(v[w].x, e, v0);
      v1 = fmaf(v[w].y, e, v1);
    }
  join_out<T>(a, j.at, D, d, v0, v1, m, l);
}

// Joins the parts of one query row (blockIdx.y of the rows of item
// blockIdx.x / columns): a thread per two of its D values and 1/kSub of the
// parts. All loads are asked for at once, before anything is known of the
// sequence: the scratch buffer was written from all over the chip, so each of
// them takes as long as memory does, and what lies past the sequence's parts
// is not used. A kernel of its own: its launch costs less than a counter that
// every workgroup waits for.
template <Mask M, class T, int D, int R>
__global__ __launch_bounds__(256) void kv8_join_kernel(AttnArgs a) {
  static_assert(R == 16, "only the decode kernel's parts are many");
  constexpr int kFloats = kPart<D, R>;
  constexpr int kSub = 512 / D, kEach = kMaxSplits / kSub;
  __shared__ float fac[kMaxSplits], half[256][2];
  const int tid = threadIdx.x, lane = tid % 64, r = blockIdx.y;
  const int sub = tid / (D / 2), d = tid % (D / 2) * 2;
  const float* part = a.ws + (int64_t)blockIdx.x * a.splits * kFloats;
  float2 v[kEach], ml[kMaxSplits / 64];
#pragma unroll
  for (int k = 0; k < kMaxSplits / 64; k++)
    if (k * 64 + lane < a.splits)
      ml[k] = *reinterpret_cast<const float2*>(part + (k * 64 + lane) * kFloats + 2 * r);
#pragma unroll
  for (int k = 0; k < kEach; k++)
    if (k * kSub + sub < a.splits)
      v[k] = *reinterpret_cast<const float2*>(part + (k * kSub + sub) * kFloats + 2 * R + r * D + d);
  const JoinAt j = join_at<M, R>(a, blockIdx.x, r);
  const int parts = j.parts;
  if (parts <= 1) return;   // written already
  // the parts' factors exp2(m - max) and the sum, by every wavefront
  float m = kNone, l = 0.0f;
#pragma unroll
  for (int k = 0; k < kMaxSplits / 64; k++)
    if (k * 64 + lane < parts) m = fmaxf(m, ml[k].x);
#pragma unroll
  for (int x = 32; x >= 1; x >>= 1) m = fmaxf(m, __shfl_xor(m, x));
#pragma unroll
  for (int k = 0; k < kMaxSplits / 64; k++)
    if (k * 64 + lane < parts) {
      const float e = __builtin_amdgcn_exp2f(ml[k].x - m);
      l += ml[k].y * e;
      if (tid < 64) fac[k * 64 + lane] = e;
    }
#pragma unroll
  for (int x = 32; x >= 1; x >>= 1) l += __shfl_xor(l, x);
  __syncthreads();
  float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
  for (int k = 0; k < kEach; k++) {
    const int w = k * kSub + sub;
    if (w < parts) {
      v0 = fmaf(v[k].x, fac[w], v0);
      v1 = fmaf(v[k].y, fac[w], v1);
    }
  }
  half[tid][0] = v0;
  half[tid][1] = v1;
  __syncthreads();
  if (sub > 0) return;
#pragma unroll
  for (int k = 1; k < kSub; k++) {
    v0 += half[tid + k * (D / 2)][0];
    v1 += half[tid + k * (D / 2)][1];
  }
  join_out<T>(a, j.at, D, d, v0, v1, m, l);
}

// ------------------------------------------------------------------- drafts
// Some drafted tokens per sequence: up to 32 query rows (tokens x heads of one
// group) per workgroup, NW wavefronts. As in the decode kernel a wavefront takes
// tiles of 64 tokens for itself and holds its whole state in registers, but
// the products are v_mfma_f32_32x32x16_f16, so that a code is read and turned into
// f16 once for 32 rows.
//
// S^T = K Q^T: row 8 (e/4) + 4 h + e%4 of the A operand is token 16 h + e of 32, so
// that lane half h gets the scores of 16 tokens in a row, which lie in one page, and
// its registers are eight by eight the B operand of O^T = V^T P^T, whose A operand is
// V^T as it is read (16 tokens of one column per 16-byte load). The order of the
// sum over D is that of 16-byte loads of keys and queries.
//
// Row groups of a sequence read the same codes: up to four that follow each other
// are numbered eight apart, which puts them on one XCD and its L2 (62 % of the requests
// hit it).
//
// Bound: no unit. With two wavefronts to a SIMD a wavefront waits for its loads 41 % of
// its time and for its turn 22 %; the vector unit (conversions and exponentials, 580
// instructions per tile and wavefront) is busy 37 % of the cycles, the matrix unit 12 %.
// A tile of 64 tokens takes 3.0 us, and 11 us of a workgroup's 40 are its start and its
// end. 16 trees of up to 26 tokens behind up to 8166, 8 heads of 4 of 128, bf16: 856
// parts on 512 places, 86 us and 15 to join them, 1.9 TB/s of the codes (the prompt
// kernel 124 us and, for the smaller trees, the decode kernel 49 more).
// floats from one row to the next where the wavefronts' results are joined: rows
// start in other banks
constexpr int draft_row(int D) { return D + 4; }
template <class T, int D, int BT, int NW>   // pages of 1 << BT tokens
__global__ __launch_bounds__(64 * NW, 2) void kv8_draft_kernel(AttnArgs a) {
  constexpr Mask M = Mask::kTree;
  constexpr int KD = D / 32, VD = D / 32, R = kDraftRows, kRow = draft_row(D);
  constexpr bool kTwo = __is_same(T, F16);   // two f16 terms of the weights, as in the decode kernel
  const int tid = threadIdx.x, lane = tid % 64;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);   // uniform: scalar
  const int col = lane % 32, h = lane / 32;
  const Kv8& c = a.c;
  const int blocks = (a.G + R - 1) / R, columns = c.heads * blocks;
  const int id = blockIdx.y * gridDim.x + blockIdx.x, log2 = a.bundle_log2;
  const int at_unit = (id >> (3 + log2)) * 8 + id % 8;   // (bundle, column, part)
  const int bundles = (a.items + (1 << log2) - 1) >> log2;
  const int column = at_unit % columns, split = at_unit / columns / bundles;
  const int index = ((at_unit / columns % bundles) << log2) + (id >> 3 & ((1 << log2) - 1));
  if (split >= a.splits || index >= a.items) return;
  const int head = column / blocks, h0 = column % blocks * R;
  const int G = min(R, a.G - h0);
  const SeqAt seq = locate(a.q, index, a.step, a.extra, BT);
  const int s = seq.s, t0 = seq.first, n = seq.count, len = seq.len, i0 = seq.item * a.unit;
  if (seq.item < 0 || i0 >= n || (int64_t)n * a.G > a.many) return;
  const int ntok = min(n - i0, a.unit);
  const int rows = ntok * G;                 // <= 32
  const int most = len - n + i0 + ntok;
  const int tiles = walk<M>(a, most, len - n + i0).tiles, per = a.per;
  const int parts = tiles > 0 ? (tiles + per - 1) / per : 1;
  if (split >= parts) return;
  const int first = split * per, last = min(first + per, tiles);

  // this lane's query row (columns past the rows repeat the first one)
  const int ct = col < rows ? col / G : 0, ch = col < rows ? col % G : 0;
  const int min_limit = len - n + i0, limit = min_limit + ct;
  const int tree = len - min(n, kTreeTokens);
  const int parent = tree_parent(a, t0, n);
  uint4 u[KD][2];
  {
    const uint16_t* qr = a.x + (int64_t)(t0 + i0 + ct) * a.ldq + (int64_t)(head * a.G + h0 + ch) * D + h * 16;
#pragma unroll
    for (int b = 0; b < KD; b++)
#pragma unroll
      for (int m = 0; m < 2; m++) u[b][m] = load_q(qr + b * 32 + m * 8, a.flip);
  }
  // the queries wait in the part of the shared memory where this wavefront's result
  // goes at the end, a lane's pieces 64 pieces apart
  extern __shared__ __attribute__((aligned(16))) float jo[];   // [NW][R][kRow]
  half8_t* const qf = reinterpret_cast<half8_t*>(jo + wave * R * kRow) + lane;
  float qs = a.scale;
  auto take_queries = [&]() QMM_INLINE {
    if constexpr (__is_same(T, F16)) {
#pragma unroll
      for (int b = 0; b < KD; b++)
#pragma unroll
        for (int m = 0; m < 2; m++) qf[(b * 2 + m) * 64] = __builtin_bit_cast(half8_t, u[b][m]);
    } else {
      uint32_t top = 0;
#pragma unroll
      for (int b = 0; b < KD; b++)
#pragma unroll
        for (int m = 0; m < 2; m++)
          top = amax_pair(amax_pair(amax_pair(amax_pair(top, u[b][m].x), u[b][m].y), u[b][m].z), u[b][m].w);
      top = amax_halves(top);
      top = umax(top, (uint32_t)__shfl_xor((int)top, 32));
      const Pow2 e = row_power(top);
      qs *= e.up;
#pragma unroll
      for (int b = 0; b < KD; b++)
#pragma unroll
        for (int m = 0; m < 2; m++) qf[(b * 2 + m) * 64] = bf16_to_f16(u[b][m], e.down);
    }
  };

  float16_t o[VD];
#pragma unroll
  for (int i = 0; i < VD; i++)
#pragma unroll
    for (int e = 0; e < 16; e++) o[i][e] = 0.0f;
  Refs at{kNone, kNone};   // O relative to 2^at.w, l to 2^at.base
  float l_run = 0.0f;

  const int32_t* row = a.q.table + (int64_t)s * a.q.W;
  // pages one per lane, loads ahead of their use: as in the decode kernel
  constexpr int kPer = kTile >> BT, kIn = (1 << BT) - 1;
  const int tk = 16 * (col >> 2 & 1) + 4 * (col >> 3) + (col & 3);   // this lane's key row of 32
  int pages = -1;
  float pages_ks = 0.0f, pages_vs = 0.0f;
  auto chunk = [&](int tile) QMM_INLINE {   // pages from this tile's first on
    const int t = tile * kTile + (lane << BT);
    const int p = t < most ? row[t >> BT] : -1;   // most <= W << BT
    pages = p < c.pages ? p : -1;
    const int64_t blk = (int64_t)(pages < 0 ? 0 : pages) * c.heads + head;
    pages_ks = c.ks[blk];
    pages_vs = c.vs[blk];
  };
  int pk[2], pv[2];   // this lane's pages of keys and values in a tile's halves
  auto look_up = [&](int i) QMM_INLINE {   // the chunk's i-th tile
#pragma unroll
    for (int j = 0; j < 2; j++) {
      pk[j] = __shfl(pages, i * kPer + ((32 * j + (tk & 16)) >> BT));
      pv[j] = __shfl(pages, i * kPer + ((32 * j + 16 * h) >> BT));
    }
  };
  u32x4_t kw[2][KD], vw[2][VD];
  auto key_at = [&](int j) QMM_INLINE {
    return c.k + c.block(pk[j] < 0 ? 0 : pk[j], head) + ((32 * j + tk) & kIn) * D + h * 16;
  };
  auto fetch_values = [&](int j) QMM_INLINE {
    const int8_t* vp = c.v + c.block(pv[j] < 0 ? 0 : pv[j], head) + (col << BT) + ((32 * j + 16 * h) & kIn);
#pragma unroll
    for (int i = 0; i < VD; i++) vw[j][i] = *reinterpret_cast<const u32x4_t*>(vp + ((i * 32) << BT));
  };
  const int run = per / NW;   // tiles of a wavefront
  const int w_first = first + wave * run, w_last = min(w_first + run, last);
  auto begin = [&](int tile) QMM_INLINE {
    chunk(tile);
    look_up(0);
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const int8_t* kp = key_at(j);
#pragma unroll
      for (int b = 0; b < KD; b++) kw[j][b] = *reinterpret_cast<const u32x4_t*>(kp + b * 32);
    }
    fetch_values(0);
    fetch_values(1);
    // an (empty) use: the wait for the scales belongs here, and not in the loop
    asm volatile("" : "+v"(pages), "+v"(pages_ks), "+v"(pages_vs));
  };
  if (w_first < w_last) begin(w_first);
  take_queries();
  const uint64_t line = last * kTile > tree ? tree_path(parent, n, i0 + ct) : 0;   // (no tile before is masked)
  for (int from = w_first; from < w_last; from += 1 << BT) {   // a chunk: 64 pages
   const int count = min(w_last - from, 1 << BT);
   if (from != w_first) begin(from);
   for (int i = 0; i < count; i++) {
    const int base = (from + i) * kTile;
    int page[2];
    float ks[2], r[2];
#pragma unroll
    for (int j = 0; j < 2; j++) {
      page[j] = pv[j];
      ks[j] = __shfl(pages_ks, i * kPer + ((32 * j + 16 * h) >> BT)) * qs;
      r[j] = __shfl(pages_vs, i * kPer + ((32 * j + 16 * h) >> BT));
    }
    const bool more = i + 1 < count;
    if (more) look_up(i + 1);
    float16_t sc[2];
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int e = 0; e < 16; e++) sc[j][e] = 0.0f;
    const int8_t *k0 = key_at(0), *k1 = key_at(1);   // of the next tile
#pragma unroll
    for (int b = 0; b < KD; b++) {
#pragma unroll
      for (int m = 0; m < 2; m++) {
        const half8_t q = qf[(b * 2 + m) * 64];
#pragma unroll
        for (int j = 0; j < 2; j++)
          sc[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(codes_f16(kw[j][b][2 * m], kw[j][b][2 * m + 1]), q, sc[j], 0, 0, 0);
        // (the compiler would convert the whole tile first and run out of registers)
        __builtin_amdgcn_sched_barrier(0);
      }
      if (more) {
        kw[0][b] = *reinterpret_cast<const u32x4_t*>(k0 + b * 32);
        kw[1][b] = *reinterpret_cast<const u32x4_t*>(k1 + b * 32);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (!(all_seen<M>(a, base, min_limit, min_limit + ntok - 1, tree) && __all(page[0] >= 0 && page[1] >= 0))) {
      // what is not seen weighs nothing, whatever its scale
      const uint64_t tokens = seen_bits<M>(a, base, limit, tree, line) >> (h * 16);
#pragma unroll
      for (int j = 0; j < 2; j++) {
        const uint32_t seen = page[j] < 0 ? 0 : (uint32_t)(tokens >> (32 * j)) & 0xffffu;
#pragma unroll
        for (int e = 0; e < 16; e++) sc[j][e] = seen >> e & 1 ? sc[j][e] * ks[j] : -__builtin_inff();
        r[j] = seen == 0 ? 0.0f : r[j];
        ks[j] = 1.0f;
      }
    }
    float mx = -__builtin_inff(), wx = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < 2; j++) {
      float top = sc[j][0];
#pragma unroll
      for (int e = 1; e < 16; e++) top = fmaxf(top, sc[j][e]);
      top *= ks[j];   // (no scale is negative)
      mx = fmaxf(mx, top);
      // (an infinite or NaN scale leaves the reference, a zero's logarithm is -inf)
      if (r[j] < __builtin_inff()) wx = fmaxf(wx, top + __builtin_amdgcn_logf(r[j]));
    }
    mx = fmaxf(mx, other_half(mx));
    wx = fmaxf(wx, other_half(wx));
    // raised when one grows by more than 2^8, as in the prompt kernel
    const bool raise = mx > at.base + 8.0f || wx > at.w + 8.0f;
    if (__any(raise)) {   // (a row's results do not depend on the other rows')
      const Refs to = rise(at, raise ? mx : kNone, raise ? wx : kNone);
      const float down = __builtin_amdgcn_exp2f(at.w - to.w);   // what the values so far shrink by
      l_run *= __builtin_amdgcn_exp2f(at.base - to.base);
      at = to;
#pragma unroll
      for (int i = 0; i < VD; i++) o[i] *= down;
    }
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const float f = weight_scale(r[j], at);
#pragma unroll
      for (int m = 0; m < 2; m++) {
        half8_t pf, pl;
        float before;
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const float x = __builtin_amdgcn_exp2f(fmaf(sc[j][8 * m + e], ks[j], -at.base));
          l_run += x;
          put_weight<kTwo>(pf, pl, e, x * f, before);
        }
#pragma unroll
        for (int i = 0; i < VD; i++) {
          const half8_t vf = codes_f16(vw[j][i][2 * m], vw[j][i][2 * m + 1]);
          o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, pf, o[i], 0, 0, 0);
          if constexpr (kTwo) o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, pl, o[i], 0, 0, 0);
          if (i % 2 == 1) __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (more) fetch_values(j);
      __builtin_amdgcn_sched_barrier(0);
    }
   }
  }
  l_run += other_half(l_run);

  // join the wavefronts: o[i][4 q + e] is value column 32 i + 8 q + 4 h + e
  __shared__ float jm[NW][R], jl[NW][R];
  if (h == 0) {
    jm[wave][col] = at.base;
    jl[wave][col] = l_run;
  }
  const float vref = __builtin_amdgcn_exp2f(at.w - at.base);
#pragma unroll
  for (int i = 0; i < VD; i++)
#pragma unroll
    for (int q = 0; q < 4; q++)
      *reinterpret_cast<float4_t*>(jo + ((wave * R + col) * kRow + i * 32 + q * 8 + h * 4)) =
          float4_t{o[i][q * 4], o[i][q * 4 + 1], o[i][q * 4 + 2], o[i][q * 4 + 3]} * vref;
  __syncthreads();
  float* part = a.ws + (((int64_t)index * columns + column) * a.splits + split) * kPart<D, R>;
  for (int i = tid; i < rows * (D / 2); i += 64 * NW) {
    const int q = i / (D / 2), d = i % (D / 2) * 2;
    float m = kNone;
#pragma unroll
    for (int w = 0; w < NW; w++) m = fmaxf(m, jm[w][q]);
    float l = 0.0f, v0 = 0.0f, v1 = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; w++) {
      const float e = __builtin_amdgcn_exp2f(jm[w][q] - m);
      const float2 v = *reinterpret_cast<const float2*>(jo + (w * R + q) * kRow + d);
      l += jl[w][q] * e;
      v0 += v.x * e;
      v1 += v.y * e;
    }
    if (parts == 1) {
      join_out<T>(a, (int64_t)(t0 + i0 + q / G) * (c.heads * a.G) + head * a.G + h0 + q % G, D, d, v0, v1, m, l);
    } else {
      *reinterpret_cast<float2*>(part + 2 * R + q * D + d) = make_float2(v0, v1);
      if (d == 0) *reinterpret_cast<float2*>(part + 2 * q) = make_float2(m, l);
    }
  }
}

// ------------------------------------------------------------------ prompts
// The work items of a prompt batch differ in length by as much as the contexts
// do, and there are only a few of them per CU: the longest come first. Returns
// the item of rank `rank` (every workgroup finds the ranks by itself: a few
// hundred comparisons per thread). Batches of more items or sequences than a
// workgroup has threads go from the last item of the last sequence to the first.
template <int N>
__device__ __forceinline__ int longest_first(const AttnArgs& a, int rank, int items) {
  __shared__ int cu[N + 1], begin[N], len[N], most[N], found;
  const int tid = threadIdx.x, S = a.q.S;
  if (items > N || S >= N) return items - 1 - rank;
  if (tid <= S) cu[tid] = a.q.clip_row(a.q.cu[tid]);
  if (tid < S) {
    begin[tid] = (int)((uint32_t)a.q.clip_row(a.q.cu[tid]) / (uint32_t)a.unit) + a.extra * tid;
    len[tid] = a.q.lens[tid];
  }
  if (tid == 0) found = 0;
  __syncthreads();
  if (tid < items) {
    int s = 0;
    for (int j = 1; j < S; j++)
      if (begin[j] <= tid) s = j;
    const int n = cu[s + 1] - cu[s], i0 = (tid - begin[s]) * a.unit;
    // (a length past the table is cut later: it only costs order here)
    most[tid] = i0 < 0 || i0 >= n ? -1 : len[s] - n + min(i0 + a.unit, n);
  }
  __syncthreads();
  if (tid < items) {
    const int mine = most[tid];
    int before = 0;
    for (int j = 0; j < items; j++) before += most[j] > mine || (most[j] == mine && j < tid);
    if (before == rank) found = tid;
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(found);
}

// 32 query rows per wavefront, four wavefronts, tiles of 64 tokens through two
// LDS buffers. The codes are turned into f16 once per workgroup on their way
// into LDS (keys [64][D], rows in the order in which the products want them;
// values [D][64]); the 16-byte pieces of a row are permuted by an exclusive-or
// with the row number, so that the 16 rows that are read together touch all
// banks.
//
// S^T = K Q^T with v_mfma_f32_32x32x16_f16; D row 8 i + 4 h + r of lane half h
// is made token 16 (i/2) + 8 h + 4 (i%2) + r, so that a lane's registers are,
// eight by eight, the B operand of O^T = V^T P^T. A page's scales are uniform
// over groups of 16 tokens, hence scalars. The running maxima (of the scores
// and of the weights with their scales) are only raised when one grows by more
// than 2^8: until then weights reach 256, which f16 and the fp32 sums hold as
// well, and nothing is rescaled.
//
// Bound: the vector unit (conversions, exponentials, maxima: 61 % of the cycles)
// and after it the matrix unit (34 %). Of visible pairs, four chunks of 2048 tokens
// behind 3952, 8 heads of 4: 760 to 830 TFLOP/s for D = 128 in bf16, 645 in f16 (two
// products per value), 660 and 530 for D = 64; 580 to 605 and 535 for D = 256 (two
// chunks of 1024 behind 4976). Eight wavefronts that share a tile, and two
// groups of wavefronts of which one multiplies while the other weighs, took the
// same time. The references of the weights and of the sum that follow each row by
// itself cost 2 % (822 us, 806 with the largest value scale of a tile as the only
// one, which loses bits: four chunks of up to 2048 tokens behind up to 8000).
//
// No variant may need scratch memory: the compiler has put the stores of
// spilled registers between a branch that some lanes take and its end, where the
// other lanes store nothing; the build refuses a kernel here that does. Hence the
// places that are computed again rather than kept, and the scalar branches. (30
// to 38 scalar registers do not fit and wait in lanes of a vector register,
// which needs no memory.)
template <Mask M, class T, int D>
__global__ __launch_bounds__(2 * kPromptRows, D == 256 ? 1 : 2) void kv8_prompt_kernel(AttnArgs a) {
  constexpr int NW = kPromptRows / 32;
  constexpr int KS = D / 16, VD = D / 32, kThreads = 64 * NW;
  constexpr int kUnits = kTile * D / 16 / kThreads;   // 16 codes per unit
  // f16 results: the weights go in as two f16 terms, since 11 bits of them would
  // cost as much as rounding the result
  constexpr bool kTwo = __is_same(T, F16);
  static_assert(kUnits >= 1, "a unit per thread");
  __shared__ __attribute__((aligned(16))) uint16_t lk[2][kTile * D], lv[2][kTile * D];
  __shared__ float lsk[2][4], lsv[2][4], lsw[2][4];   // scales; log2 of the values'
  // position of 16-byte piece p of key row r (rows of D * 2 bytes)
  auto key_piece = [](int r, int p) QMM_INLINE {
    return (p ^ (D == 64 ? r >> 1 : r)) & (D / 8 - 1);
  };
  const int tid = threadIdx.x, lane = tid % 64;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);   // uniform: scalar
  const int col = lane % 32, h = lane / 32;
  const Kv8& c = a.c;
  const int head = blockIdx.x % c.heads, items = gridDim.x / c.heads, split = blockIdx.y;
  // (Under a window items differ little in length, and neighbours share tiles, in
  // their L2 when they run together: four chunks of up to 2048 under 1024 tokens, 213 us
  // sorted, 190 in order.)
  const int rank = blockIdx.x / c.heads;
  const int index = M == Mask::kWindow ? rank : longest_first<kThreads>(a, rank, items);
  const SeqAt seq = locate(a.q, index, a.step, a.extra, c.bt_log2);
  const int s = seq.s, t0 = seq.first, n = seq.count, len = seq.len, item = seq.item;
  const int i0 = item * a.unit;
  if (item < 0 || i0 >= n || (int64_t)n * a.G <= a.many) return;
  const int ntok = min(n - i0, a.unit);
  const int rows = ntok * a.G;
  const int most = len - n + i0 + ntok;
  const Walk path = walk<M>(a, most, len - n + i0);
  const int tiles = path.tiles;
  const int parts = tiles > 0 ? (tiles + a.per - 1) / a.per : 1;
  if (split >= parts) return;
  const int first = split * a.per;
  const int last = __builtin_amdgcn_readfirstlane(min(first + a.per, tiles));   // scalar

  // this lane's query row; rows past the last repeat it, and nothing reads them
  const int rr = min(wave * 32 + col, rows - 1);
  const int ct = rr / a.G, ch = rr % a.G;
  const int limit = len - n + i0 + ct;
  const int wave_min = len - n + i0 + min(wave * 32, rows - 1) / a.G;
  const int wave_max = len - n + i0 + min(wave * 32 + 31, rows - 1) / a.G;
  const int tree = len - min(n, kTreeTokens);
  uint64_t line = 0;
  if constexpr (M == Mask::kTree) line = tree_path(tree_parent(a, t0, n), n, i0 + ct);
  half8_t qf[KS];
  float qs = a.scale;
  {
    const uint16_t* qr = a.x + (int64_t)(t0 + i0 + ct) * a.ldq + (int64_t)(head * a.G + ch) * D + h * 8;
    uint4 u[KS];
#pragma unroll
    for (int i = 0; i < KS; i++) u[i] = load_q(qr + i * 16, a.flip);
    if constexpr (__is_same(T, F16)) {
#pragma unroll
      for (int i = 0; i < KS; i++) qf[i] = __builtin_bit_cast(half8_t, u[i]);
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < KS; i++)
        m = amax_pair(amax_pair(amax_pair(amax_pair(m, u[i].x), u[i].y), u[i].z), u[i].w);
      m = amax_halves(m);
      m = umax(m, (uint32_t)__shfl_xor((int)m, 32));
      const Pow2 e = row_power(m);
      qs *= e.up;
#pragma unroll
      for (int i = 0; i < KS; i++) qf[i] = bf16_to_f16(u[i], e.down);
    }
  }
  float16_t o[VD];
#pragma unroll
  for (int i = 0; i < VD; i++)
#pragma unroll
    for (int e = 0; e < 16; e++) o[i][e] = 0.0f;
  Refs at{kNone, kNone};   // O relative to 2^at.w, l to 2^at.base
  float l_run = 0.0f;

  const int32_t* row = a.q.table + (int64_t)s * a.q.W;
  const int bt = c.bt_log2;
  // Each tile's pages are looked up two tiles ahead and its codes and scales
  // loaded one tile ahead, and nothing touches them before the next step (the
  // page numbers are checked when they are used), so that no step waits for a
  // load it has just asked for (783 us; 819 with the numbers checked as they
  // came: four chunks of up to 2048 tokens behind up to 8000, 8 heads of 4,
  // D = 128). Unit i of a thread: 16 columns of key token tk + i * kStep, 16
  // tokens of value column vd + 64 i; the first wavefront carries the scales,
  // its lane the ones of group lane modulo 4. Past the last token any page of
  // the sequence will do.
  constexpr int kStep = kThreads / (D / 16);   // tokens from one key unit to the next
  const int tk = tid / (D / 16), vd = tid / 4, vc = tid % 4 * 16;
  const uint32_t page_bytes = (uint32_t)c.block(1, 0);   // <= 2^24
  const int in = (1 << bt) - 1;   // (bits of tk and of i * kStep do not overlap)
  const int8_t* const kb = c.k + c.block(0, head) + (tk & in) * D + tid % (D / 16) * 16;
  const int8_t* const vb = c.v + c.block(0, head) + (vd << bt) + (vc & in);
  int kp[kUnits], vp;
  auto look_up = [&](int tile) QMM_INLINE {   // most <= W << bt
    tile = path.real(tile);
#pragma unroll
    for (int i = 0; i < kUnits; i++)
      kp[i] = row[min(tile * kTile + tk + i * kStep, most - 1) >> bt];
    vp = row[min(tile * kTile + vc, most - 1) >> bt];
  };
  // rows of keys in LDS, and where this thread's first units go
  auto key_row = [](int t) QMM_INLINE {
    return (t & 32) + 8 * ((t >> 4 & 1) * 2 + (t >> 2 & 1)) + 4 * (t >> 3 & 1) + (t & 3);
  };
  const int to_k = key_row(tk) * D + key_piece(key_row(tk), tid % (D / 16) * 2) * 8;
  const int to_v = vd * kTile + ((vc / 8 ^ vd >> 1) & 7) * 8;
  u32x4_t kw[kUnits], vw[kUnits];
  float sk = 0, sv = 0;
  bool miss = false;
  auto fetch = [&]() QMM_INLINE {
    auto page = [&](int p) QMM_INLINE {
      return (uint64_t)((uint32_t)p < (uint32_t)c.pages ? (uint32_t)p : 0);
    };
    if (wave == 0) {
      miss = (uint32_t)vp >= (uint32_t)c.pages;
      const int64_t blk = (int64_t)page(vp) * c.heads + head;
      sk = c.ks[blk];
      sv = c.vs[blk];
    }
#pragma unroll
    for (int i = 0; i < kUnits; i++) {
      kw[i] = *reinterpret_cast<const u32x4_t*>(kb + (page(kp[i]) * page_bytes +
                                                      (uint32_t)((i * kStep & in) * D)));
      vw[i] = *reinterpret_cast<const u32x4_t*>(vb + (page(vp) * page_bytes +
                                                      (uint32_t)(i * (kThreads / 4) << bt)));
    }
  };
  auto put = [&](int buf) QMM_INLINE {
    if (wave == 0) {
      lsk[buf][lane % 4] = sk;
      lsv[buf][lane % 4] = miss ? -1.0f : sv;   // no scale is negative: not seen
      // (an infinite or NaN scale leaves the reference of the weights)
      lsw[buf][lane % 4] = !miss && sv < __builtin_inff() ? __builtin_amdgcn_logf(sv) : -__builtin_inff();
    }
#pragma unroll
    for (int i = 0; i < kUnits; i++) {
      const int r = key_row(i * kStep);
      uint16_t* kt = &lk[buf][(to_k ^ (r & (D / 8 - 1)) * 8) + r * D];
      uint16_t* vt = &lv[buf][to_v + i * (kThreads / 4) * kTile];
      const int odd = (to_k & 8) ? -8 : 8, odd_v = (to_v & 8) ? -8 : 8;   // the other piece
      *reinterpret_cast<half8_t*>(kt) = codes_f16(kw[i][0], kw[i][1]);
      *reinterpret_cast<half8_t*>(kt + odd) = codes_f16(kw[i][2], kw[i][3]);
      *reinterpret_cast<half8_t*>(vt) = codes_f16(vw[i][0], vw[i][1]);
      *reinterpret_cast<half8_t*>(vt + odd_v) = codes_f16(vw[i][2], vw[i][3]);
    }
  };
  // one tile's softmax and second product; MASK: some of its tokens are not
  // seen by some of the wavefront's rows
  auto weigh = [&]<bool MASK>(float16_t* sc, const float* f, const float* vs, int left,
                              uint32_t missing, uint32_t seen, int buf) QMM_INLINE {
    // whether a token of a masked tile is seen: element e of group g
    auto sees = [&](int g, int e) QMM_INLINE {
      if constexpr (M == Mask::kCausal) return g * 16 + e <= left && !(missing >> g & 1);
      else return (seen >> (g * 8 + e) & 1) != 0;
    };
    // element e of sc[j]: token 32 j + 16 (e/8) + 8 h + e%8
    float mx = -__builtin_inff(), wx = -__builtin_inff();
#pragma unroll
    for (int g = 0; g < 4; g++) {
      float top = -__builtin_inff();
#pragma unroll
      for (int e = 0; e < 8; e++) {
        float x = sc[g / 2][g % 2 * 8 + e];
        if constexpr (MASK) {
          x = sees(g, e) ? x * f[g] : -__builtin_inff();
          sc[g / 2][g % 2 * 8 + e] = x;
        }
        top = fmaxf(top, x);
      }
      if constexpr (!MASK) top *= f[g];
      mx = fmaxf(mx, top);
      wx = fmaxf(wx, top + lsw[buf][g]);
    }
    mx = fmaxf(mx, other_half(mx));
    wx = fmaxf(wx, other_half(wx));
    const bool raise = mx > at.base + 8.0f || wx > at.w + 8.0f;
    if (__any(raise)) {   // (a row's results do not depend on the other rows')
      const Refs to = rise(at, raise ? mx : kNone, raise ? wx : kNone);
      const float down = __builtin_amdgcn_exp2f(at.w - to.w);
      l_run *= __builtin_amdgcn_exp2f(at.base - to.base);
#pragma unroll
      for (int i = 0; i < VD; i++) o[i] *= down;
      at = to;
    }
    int piece = col * kTile + ((h ^ col >> 1) & 7) * 8;
    asm volatile("" : "+v"(piece));
#pragma unroll
    for (int g = 0; g < 4; g++) {
      float r = weight_scale(vs[g], at);
      // (of a page that the row does not see a scale may be anything; seen in part, its
      // scale is the row's too, and the exponentials of the rest are 0)
      if constexpr (MASK && M != Mask::kCausal) r = seen >> (g * 8) & 0xff ? r : 0.0f;
      half8_t hi, lo;
      float before;
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const float x = sc[g / 2][g % 2 * 8 + e];
        const float p = __builtin_amdgcn_exp2f(MASK ? x - at.base : fmaf(x, f[g], -at.base));
        l_run += p;
        float w = p * r;
        if constexpr (MASK && M == Mask::kCausal) w = sees(g, e) ? w : 0.0f;
        put_weight<kTwo>(hi, lo, e, w, before);
      }
#pragma unroll
      for (int i = 0; i < VD; i++) {
        const half8_t vf =
            *reinterpret_cast<const half8_t*>(&lv[buf][(piece ^ g * 16) + i * 32 * kTile]);
        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, hi, o[i], 0, 0, 0);
        if constexpr (kTwo) o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, lo, o[i], 0, 0, 0);
      }
      // (operands of the product after next are asked for before the present one,
      // for which the compiler finds no registers by itself: 634 us, 725 without)
      if constexpr (D == 256) {
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
        for (int i = 0; i < VD; i++) {
          __builtin_amdgcn_sched_group_barrier(0x008, kTwo ? 2 : 1, 0);
          if (i < VD - 2) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
      }
    }
  };
  if (first < last) {
    look_up(first);
    fetch();
    look_up(first + 1);
    put(first & 1);
  }
  for (int tile = first; tile < last; tile++) {
    const int buf = tile & 1;
    __syncthreads();
    if (tile + 1 < last) {
      fetch();
      look_up(tile + 2);
    }
    const int base = path.real(tile) * kTile;
    if (base <= wave_max && wave * 32 < rows) {   // (a wavefront without rows only carries codes)
      float f[4], vs[4];
      uint32_t missing = 0;
#pragma unroll
      for (int g = 0; g < 4; g++) {
        f[g] = lsk[buf][g] * qs;
        vs[g] = lsv[buf][g];
        const bool gone = __builtin_bit_cast(uint32_t, vs[g]) == 0xbf800000u;
        missing |= gone ? 1u << g : 0u;
      }
      int piece = col * D + key_piece(col, h) * 8;
      asm volatile("" : "+v"(piece));   // (places of operands are not kept either)
      float16_t sc[2];
#pragma unroll
      for (int j = 0; j < 2; j++)
#pragma unroll
        for (int e = 0; e < 16; e++) sc[j][e] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const half8_t kf = *reinterpret_cast<const half8_t*>(&lk[buf][(piece ^ ks * 16) + j * 32 * D]);
          sc[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[ks], sc[j], 0, 0, 0);
        }
      const int left = limit - base - h * 8;   // tokens g * 16 + e up to this are seen
      if (all_seen<M>(a, base, wave_min, wave_max, tree) && missing == 0) {
        weigh.template operator()<false>(sc, f, vs, left, missing, 0, buf);
      } else {
        uint32_t seen = 0;   // eight bits for each group's tokens 8 h .. 8 h + 7
        if constexpr (M != Mask::kCausal) {
          const uint64_t tokens = seen_bits<M>(a, base, limit, tree, line) >> (h * 8);
#pragma unroll
          for (int g = 0; g < 4; g++)
            seen |= missing >> g & 1 ? 0 : (uint32_t)(tokens >> (g * 16) & 0xff) << (g * 8);
        }
        weigh.template operator()<true>(sc, f, vs, left, missing, seen, buf);
      }
    }
    if (tile + 1 < last) put(buf ^ 1);
  }
  if (wave * 32 + col >= rows) return;
  l_run += __shfl_xor(l_run, 32);
  if (parts > 1) {   // kv8_join_few_kernel adds them up
    const int64_t unit = (int64_t)index * c.heads + head;
    float* part = a.ws + (unit * a.splits + split) * kPart<D, kPromptRows>;
    const float vref = __builtin_amdgcn_exp2f(at.w - at.base);
    if (h == 0) *reinterpret_cast<float2*>(part + 2 * (wave * 32 + col)) = make_float2(at.base, l_run);
    float* mine = part + 2 * kPromptRows + (wave * 32 + col) * D + h * 4;
#pragma unroll
    for (int i = 0; i < VD; i++)
#pragma unroll
      for (int q = 0; q < 4; q++)
        *reinterpret_cast<float4_t*>(mine + i * 32 + q * 8) =
            float4_t{o[i][q * 4], o[i][q * 4 + 1], o[i][q * 4 + 2], o[i][q * 4 + 3]} * vref;
    return;
  }
  int r_out = wave * 32 + col;   // (not kept through the loop: registers are short)
  asm volatile("" : "+v"(r_out));
  const int64_t to = (int64_t)(t0 + i0 + r_out / a.G) * (c.heads * a.G) + head * a.G + r_out % a.G;
  const bool any = l_run > 0.0f || l_run != l_run;
  const float back = any ? __builtin_amdgcn_exp2f(at.w - at.base) / l_run : 0.0f;
#pragma unroll
  for (int i = 0; i < VD; i++)
#pragma unroll
    for (int q = 0; q < 4; q++) {
      uint16_t w[4];
#pragma unroll
      for (int e = 0; e < 4; e++) w[e] = from_f32(T{}, any ? o[i][q * 4 + e] * back : 0.0f);
      *reinterpret_cast<uint2*>(a.out + to * D + i * 32 + q * 8 + h * 4) =
          make_uint2(w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16);
    }
  if (h == 0 && a.lse) a.lse[to] = any ? fmaf(at.base, kLn2, logf(l_run)) : -__builtin_inff();
}

// Sequences with at most this many query rows (new tokens x heads of a group) go
// to the decode kernel, 16 rows at a time; the others to the prompt kernel.
constexpr int kFewRows = 64;

struct Plan {
  int unit, step, extra, bundle_log2, splits, per, nw, many, most_rows;
  int64_t items, columns;   // grid: items x heads and blocks of a group's heads
  bool prompts, drafts;     // drafts: the draft kernel in the decode kernel's place
  int p_unit, p_splits, p_per;
  int64_t p_items;
};

// window > 0: an item whose rows span `rows` positions looks at no more tiles
// than their windows and the sinks touch
int64_t most_tiles(int64_t tiles, int64_t rows, int64_t window, int64_t sinks) {
  if (window <= 0) return tiles;
  const int64_t n = (window + rows - 2 + kTile - 1) / kTile + 1 + (sinks + kTile - 1) / kTile;
  return n < tiles ? n : tiles;
}

template <Mask M>
Plan plan(const Kv8& c, int64_t T, int64_t Hq, int64_t S, int64_t W, int64_t window = 0,
          int64_t sinks = 0) {
  Plan p{};
  const int64_t G = Hq / c.heads;
  // the packed batch says how many new tokens a sequence can have at most
  const int64_t longest = T;
  // (For large batches of few rows the decode kernel is quicker: 48 trees of up to 4
  // tokens, 8 heads of 4, 113 us, 128 with the draft kernel; 16 of up to 5, 39 and 31; one
  // of 4 behind 31996, 44 and 24. D = 256: its state does not fit the registers.)
  p.drafts = M == Mask::kTree && T > S && G <= kDraftRows && c.dim <= 128 &&
             (T * G > 13 * S || S * c.heads < 128);
  p.prompts = longest * G > kFewRows && T > S && G <= kPromptRows;
  // Trees go to the draft kernel whole (the two kernels one after the other, each for
  // some of the sequences, take longer than either: 215 us for 16 trees of up to 64
  // tokens behind up to 8128, 8 heads of 4, 153 and 178 by themselves), unless they
  // are so large that what the prompt kernel's four wavefronts share outweighs its
  // barriers: from 256 rows (16 trees of up to 64, 8 heads of 8: 238 us, 397; one
  // of 32 behind 31968, 256 rows: 101 us, 83), from 160 where they fill the chip.
  if (p.drafts) p.prompts = T * G > 256 * S || (T * G > 160 * S && S * c.heads >= 128);
  p.many = p.prompts ? kFewRows : INT32_MAX;
  const int64_t all = ((W << c.bt_log2) + kTile - 1) / kTile;
  if (p.drafts) {
    p.unit = (int)(kDraftRows / G);
    p.columns = c.heads;
    p.most_rows = (int)(p.unit * G);
    p.extra = 1;
    p.items = T / p.unit + S;
    p.step = p.unit;
    if (S == 1) {   // all the tokens are its
      p.step = INT32_MAX;
      p.items = p.extra = (int)((T + p.unit - 1) / p.unit);
    }
    p.bundle_log2 = p.items >= 3 * S ? 2 : p.items >= 2 * S ? 1 : 0;
    p.nw = 4;
    // A workgroup's start and end take as long as 16 tiles, so that parts are 32 tiles
    // where that leaves one for each CU, more where it makes over 1024 of them (two
    // rounds) of contexts as long as the table, and no more than 32 of a context. (16
    // trees of up to 26 tokens behind up to 8166, 8 heads of 4: 97 us with parts of 40
    // tiles, 114 with 80; 4 of 12 behind 7988: 33 us with 20, 39 with 8; one of 8 behind
    // 31992: 26 us in 32 parts, 30 in 16, 36 in 126.)
    const int64_t tiles = most_tiles(all, p.unit, window, sinks);
    const int64_t work = (S > T / p.unit ? S : T / p.unit) * p.columns * tiles;
    const int64_t cut = (tiles + few_parts(kDraftRows) - 1) / few_parts(kDraftRows);
    int64_t per = work / 256 < 32 ? work / 256 : 32;
    const int64_t least = tiles < 64 ? 4 : 8;
    per = per > least ? per : least;
    per = per > work / 1024 ? per : work / 1024;
    per = per > cut ? per : cut;
    if (p.items * p.columns * cut > (1 << 20)) per = tiles;
    p.per = (int)((per + p.nw - 1) / p.nw * p.nw);
    p.splits = (int)((tiles + p.per - 1) / p.per);
  } else {
    p.unit = T > S && G <= 8 ? (int)(16 / G) : 1;
    p.step = p.unit;
    p.extra = p.unit > 1 ? 1 : 0;
    p.items = T / p.unit + p.extra * S;
    p.columns = c.heads * ((G + 15) / 16);
    p.most_rows = (int)(p.unit * (G < 16 ? G : 16));
    const int64_t units = (T < p.items ? T : p.items) * p.columns;
    const int64_t tiles = most_tiles(all, p.unit, window, sinks);
    // Every workgroup takes the same number of tiles, so that ragged sequences
    // load the chip evenly: as many as make 2048 workgroups of sequences that
    // fill their table rows (1024 for D = 256, whose registers leave room for half
    // as many wavefronts: 121 against 140 us for 48 contexts to 4096), and no more
    // than kMaxSplits parts of a sequence.
    // Contexts of up to 24 tiles are not cut: eight wavefronts walk them in
    // three steps, which costs less than the second launch that joins parts.
    // (48 contexts to 8192 tokens, 8 heads: 111 us with parts of 24 tiles and 4
    // wavefronts, 134 us with 8, 119 us with 10 tiles and 1; one context of
    // 131071 tokens, 2 heads: 23.8 us with 128 parts, 26.7 with 64, 37 with 1
    // wavefront.)
    const int64_t cut = (tiles + kMaxSplits - 1) / kMaxSplits;
    const int64_t wanted = c.dim == 256 ? 1024 : 2048;
    int64_t per = (units * tiles + wanted - 1) / wanted;
    per = per > cut ? per : cut;
    p.nw = 4;
    if (tiles <= 24) {
      p.nw = c.dim == 256 ? 4 : 8;
      per = tiles;
    }
    if (p.items * p.columns * cut > (1 << 20)) per = tiles;
    per = (per + p.nw - 1) / p.nw * p.nw;
    p.per = (int)per;
    p.splits = (int)((tiles + per - 1) / per);
  }
  if (p.prompts) {
    // The sequences of the decode or draft kernel have few tokens then, so that their
    // items can be counted by sequence: a workgroup for every token of the prompts, to
    // find that it has nothing to do, takes as long as some prompts' attention (33 us
    // of 245 under a window of 1024).
    const int64_t each = (kFewRows / G + p.unit - 1) / p.unit;
    if (S * each < p.items) {
      p.step = INT32_MAX;   // (no sequence has so many tokens)
      p.extra = (int)each;
      p.items = S * each;
    }
  }
  p.p_unit = (int)(kPromptRows / (G < kPromptRows ? G : kPromptRows));
  p.p_items = T / p.p_unit + S;
  // Prompts: where the items do not fill the chip (two workgroups per CU), the
  // tiles of each are cut, into parts of at least 16 tiles: a part costs a pass
  // over its rows in fp32, there and back. (A chunk of 600 tokens behind 29400,
  // 8 heads of 4: 535 us cut, 949 us whole.)
  const int64_t work = p.p_items * c.heads;
  // Trees hardly ever fill their last item and are few, so that they are cut finer, into
  // parts of at least 8 tiles (4 of up to 40 tokens behind 3960, D = 256: 65 us, 98 with 16;
  // 3 of up to 200 behind 2800, D = 128: 36 us, 47), and for D = 256, of which a CU holds
  // one, fewer (5 of up to 118 behind 7160, one head of 8: 96 us in 7 parts, 125 in 9).
  // Small trees are not theirs, and would only wait for more of them to leave.
  const bool trees = M == Mask::kTree && T * G > kFewRows * S;
  const int64_t least = trees ? 8 : 16;
  const int64_t wanted = !trees ? 512 : c.dim == 256 ? 288 : 1024;
  int64_t ps = wanted / (work < 1 ? 1 : work);
  const int64_t p_tiles = most_tiles(all, p.p_unit, window, sinks);
  ps = ps < p_tiles / least ? ps : p_tiles / least;
  ps = ps < 1 ? 1 : ps > kFewParts ? kFewParts : ps;
  p.p_per = (int)((p_tiles + ps - 1) / ps);
  p.p_splits = (int)((p_tiles + p.p_per - 1) / p.p_per);
  return p;
}

// bytes of the decode or draft kernel's parts, then of the prompt kernel's
int64_t decode_bytes(const Plan& p, const Kv8& c) {
  return p.splits > 1 ? p.items * p.columns * p.splits * (p.drafts ? kDraftRows : 16) * (c.dim + 2) * 4 : 0;
}
int64_t prompt_bytes(const Plan& p, const Kv8& c) {
  return p.prompts && p.p_splits > 1
             ? p.p_items * c.heads * p.p_splits * kPromptRows * (c.dim + 2) * 4 : 0;
}

template <Mask M>
int64_t attention_work(const Kv8& c, int64_t T, int64_t Hq, int64_t S, int64_t W, int64_t window = 0,
                       int64_t sinks = 0) {
  const Plan p = plan<M>(c, T, Hq, S, W, window, sinks);
  return decode_bytes(p, c) + prompt_bytes(p, c);
}

template <Mask M>
hipError_t launch_attention(const Kv8& c, int dt, const void* q, int64_t ldq, int64_t T, int64_t Hq,
                            const int32_t* table, const int32_t* lens, const int32_t* cu, int64_t S,
                            int64_t W, int64_t window, int64_t sinks, const int32_t* parent,
                            float scale, void* out, float* lse, float* ws, hipStream_t st) {
  const Plan p = plan<M>(c, T, Hq, S, W, window, sinks);
  AttnArgs a{c, {table, lens, cu, (int)S, (int)W, (int)T}, static_cast<const uint16_t*>(q), ldq,
             (int)(Hq / c.heads), p.unit, p.step, p.extra, (int)p.items, p.bundle_log2, p.many, fabsf(scale) * kLog2e,
             scale < 0 ? 0x80008000u : 0u, static_cast<uint16_t*>(out), lse, p.splits, p.per, ws,
             (int)window, (int)sinks, parent};
  const dim3 grid((unsigned)p.items, (unsigned)p.columns, (unsigned)p.splits);
  auto join = [&]<class T_, int D, int R>(const AttnArgs& x, unsigned units, int rows) {
    auto few = [&]() {
      hipLaunchKernelGGL((kv8_join_few_kernel<M, T_, D, R>),
                         dim3(units, (unsigned)((rows + 512 / D - 1) / (512 / D))), dim3(256), 0, st, x);
    };
    if constexpr (R == 16) {
      if (x.splits > few_parts(R)) {
        hipLaunchKernelGGL((kv8_join_kernel<M, T_, D, R>), dim3(units, (unsigned)rows), dim3(256), 0, st, x);
        return;
      }
    }
    few();   // (plan() cuts drafts and prompts into no more parts than that)
  };
  auto go = [&]<class T_, int D>() {
    auto decode = [&]<int BT>() {
      if constexpr (M == Mask::kTree && D <= 128)
        if (p.drafts) {
          const int64_t bundle = 1 << p.bundle_log2;
          const int64_t units = (p.items + bundle - 1) / bundle * p.columns * p.splits;
          const int64_t ids = (units + 7) / 8 * 8 * bundle;
          const unsigned wide = (unsigned)(ids < (1 << 20) ? ids : 1 << 20);   // (a row of a grid is short of 2^32 threads)
          hipLaunchKernelGGL((kv8_draft_kernel<T_, D, BT, 4>), dim3(wide, (unsigned)((ids + wide - 1) / wide)), dim3(256),
                             4 * kDraftRows * draft_row(D) * 4, st, a);
          if (p.splits > 1)
            join.template operator()<T_, D, kDraftRows>(a, (unsigned)(p.items * p.columns), p.most_rows);
          return;
        }
      auto waves = [&]<int NW>() {
        hipLaunchKernelGGL((kv8_decode_kernel<M, T_, D, BT, NW>), grid, dim3(64 * NW), NW * 16 * D * 4,
                           st, a);
      };
      if (p.items == 0) return;
      if (p.nw == 4) waves.template operator()<4>();
      else waves.template operator()<D == 256 ? 4 : 8>();
      if (p.splits > 1)
        join.template operator()<T_, D, 16>(a, (unsigned)(p.items * p.columns), p.most_rows);
    };
    if (c.bt_log2 == 4) decode.template operator()<4>();
    else if (c.bt_log2 == 5) decode.template operator()<5>();
    else decode.template operator()<6>();
    if (!p.prompts) return;
    AttnArgs b = a;
    b.unit = b.step = p.p_unit;
    b.extra = 1;
    b.items = (int)p.p_items;
    b.splits = p.p_splits;
    b.per = p.p_per;
    b.ws = ws + decode_bytes(p, c) / 4;
    const unsigned units = (unsigned)(p.p_items * c.heads);
    hipLaunchKernelGGL((kv8_prompt_kernel<M, T_, D>), dim3(units, (unsigned)p.p_splits), dim3(256), 0,
                       st, b);
    if (p.p_splits > 1)
      join.template operator()<T_, D, kPromptRows>(b, units, kPromptRows);
  };
  auto by_dim = [&]<class T_>() {
    if (c.dim == 64) go.template operator()<T_, 64>();
    else if (c.dim == 128) go.template operator()<T_, 128>();
    else go.template operator()<T_, 256>();
  };
  if (dt == 0) by_dim.template operator()<F16>();
  else by_dim.template operator()<BF16>();
  return hipGetLastError();
}

}  // namespace
}  // namespace qmm
