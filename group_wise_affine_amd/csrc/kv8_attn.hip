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
// exp(x - m) * vs are rounded on their way into the second product (to 11
// bits for bf16 results, to two f16 terms for f16 ones); sums, maxima and the
// normaliser stay in fp32.
#include "kernels.hpp"
#include "kv8_common.hpp"

namespace qmm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTile = 64;   // tokens per step of a wavefront
constexpr int kDecodeWaves = 4;
constexpr int kMaxSplits = 64;   // parts of a sequence that one workgroup joins

struct AttnArgs {
  Kv8 c;
  Kv8Seqs q;
  const uint16_t* x;   // queries, row t at x + t * ldq
  int64_t ldq;
  int G;               // query heads per cache head, 16 at a time
  int unit, extra;     // new tokens per workgroup, spare items per sequence
  int many;            // sequences with more query rows than this are the prompt kernel's
  float scale;         // magnitude of the scores' scale, times log2 e
  uint32_t flip;       // its sign, as the sign bits of two queries
  uint16_t* out;       // [T][heads * G][D]
  float* lse;          // [T][heads * G] or null
  int splits, per;     // workgroups of a sequence (gridDim.z), tiles of each
  float* ws;
  unsigned* cnt;
};

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
  e = e < -100 ? -100 : e > 100 ? 100 : e;
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
template <class T, int D, int BT, int NW>   // pages of 1 << BT tokens
__global__ __launch_bounds__(64 * NW, D == 64 ? 4 : D == 128 ? 3 : 1) void kv8_decode_kernel(AttnArgs a) {
  constexpr int KD = D / 64, VD = D / 16;
  // f16 results: the weights go in as two f16 terms, since 11 bits of them would
  // cost as much as rounding the result
  constexpr bool kTwo = __is_same(T, F16);
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int col = lane % 16, g = lane / 16;
  const int blocks = (a.G + 15) / 16;   // of heads in a group
  const int head = blockIdx.y / blocks, h0 = blockIdx.y % blocks * 16, split = blockIdx.z;
  const int G = min(16, a.G - h0);
  const Kv8& c = a.c;
  const int s = find_seq(a.q, blockIdx.x, a.unit, a.extra);
  const int t0 = a.q.first(s), n = a.q.count(s), len = a.q.length(s, BT);
  const int item = blockIdx.x - first_item(a.q, s, a.unit, a.extra);
  const int i0 = item * a.unit;
  if (item < 0 || i0 >= n || (int64_t)n * a.G > a.many) return;
  const int ntok = min(n - i0, a.unit);
  const int rows = ntok * G;                 // <= 16
  // positions that the last row sees, tiles of them, this workgroup's share
  const int most = len - n + i0 + ntok;
  const int tiles = most > 0 ? (most + kTile - 1) / kTile : 0;
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
  half8_t qf[KD][2];
  float qs = a.scale;
  {
    const uint16_t* qr = a.x + trow * a.ldq + (int64_t)qh * D + g * 16;
    uint4 u[KD][2];
    uint32_t m = 0;
#pragma unroll
    for (int b = 0; b < KD; b++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        u[b][h] = load_q(qr + b * 64 + h * 8, a.flip);
        m = amax_pair(amax_pair(amax_pair(amax_pair(m, u[b][h].x), u[b][h].y), u[b][h].z), u[b][h].w);
      }
    if constexpr (__is_same(T, F16)) {
#pragma unroll
      for (int b = 0; b < KD; b++)
#pragma unroll
        for (int h = 0; h < 2; h++) qf[b][h] = __builtin_bit_cast(half8_t, u[b][h]);
    } else {
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
  }

  float4_t o[VD];
#pragma unroll
  for (int i = 0; i < VD; i++) o[i] = float4_t{0, 0, 0, 0};
  float m_run = -__builtin_inff(), l_run = 0.0f;
  // O holds sums of codes weighted with p * vs / vref, vref = 2^v_exp a power
  // of two that follows the largest value scale seen
  int v_exp = -126;

  const int32_t* row = a.q.table + (int64_t)s * a.q.W;
  // page of token t of the sequence (-1: none, its tokens are not seen)
  auto page_at = [&](int t) QMM_INLINE {
    const int j = t >> BT;
    const int p = t < most ? row[j] : -1;   // most <= W << BT
    return p < c.pages ? p : -1;
  };
  // The loads run ahead of their use: a tile's pages are looked up one tile
  // before its codes are asked for, its key codes while the tile before is
  // weighed, its value codes once the values of the tile before are spent.
  const int kg = (col / 4) * 16;   // first token of this lane's K rows in a tile
  int pk, pv;
  auto look_up = [&](int tile) QMM_INLINE {
    pk = page_at(tile * kTile + kg);
    pv = page_at(tile * kTile + g * 16);
  };
  u32x4_t kw[4][KD], vw[VD];
  auto fetch_keys = [&]() QMM_INLINE {
    const int8_t* kp = c.k + c.block(pk < 0 ? 0 : pk, head) +
                       ((kg & ((1 << BT) - 1)) + col % 4) * D + g * 16;
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int b = 0; b < KD; b++)
        kw[j][b] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4_t*>(kp + j * 4 * D + b * 64));
  };
  auto fetch_values = [&](int page) QMM_INLINE {
    const int8_t* vp = c.v + c.block(page < 0 ? 0 : page, head) + (col << BT) +
                       ((g * 16) & ((1 << BT) - 1));
#pragma unroll
    for (int i = 0; i < VD; i++)
      vw[i] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4_t*>(vp + ((i * 16) << BT)));
  };
  float ks = 0.0f, vs = 0.0f;   // scales of this lane's 16 tokens
  auto fetch_scales = [&](int page) QMM_INLINE {
    const int64_t blk = (int64_t)(page < 0 ? 0 : page) * c.heads + head;
    ks = c.ks[blk];
    vs = c.vs[blk];
  };
  // one tile's weights; MASK: some of its tokens are not seen by some row
  half8_t pf[2], pl[2];
  auto weigh = [&]<bool MASK>(const float4_t* sc, float f, float vs, int ve, int left) QMM_INLINE {
    float p[16];
    float mx = m_run;
#pragma unroll
    for (int i = 0; i < 16; i++) {
      p[i] = sc[i / 4][i % 4] * f;
      if constexpr (MASK) p[i] = i <= left ? p[i] : -__builtin_inff();
      mx = fmaxf(mx, p[i]);
    }
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float mu = mx == -__builtin_inff() ? 0.0f : mx;
    if (__any(mx != m_run || ve != v_exp)) {
      const float al = __builtin_amdgcn_exp2f(m_run - mu);
      const float down = ldexpf(al, v_exp - ve);
      l_run *= al;
#pragma unroll
      for (int i = 0; i < VD; i++) o[i] *= down;
      m_run = mx;
      v_exp = ve;
    }
    const float r = ldexpf(vs, -v_exp);
#pragma unroll
    for (int i = 0; i < 16; i++) {
      const float e = __builtin_amdgcn_exp2f(p[i] - mu);
      l_run += e;
      float w = e * r;
      if constexpr (MASK) w = i <= left ? w : 0.0f;
      pf[i / 8][i % 8] = (_Float16)w;
      if constexpr (kTwo) pl[i / 8][i % 8] = (_Float16)(w - (float)pf[i / 8][i % 8]);
    }
  };
  int tile = first + wave;
  if (tile < last) {
    look_up(tile);
    fetch_keys();
    fetch_values(pv);
    fetch_scales(pv);
  }
  for (; tile < last; tile += NW) {
    const int base = tile * kTile;
    const int page = pv;
    const bool more = tile + NW < last;
    if (more) look_up(tile + NW);
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
    const float f = ks * qs, vs_now = vs;
    if (more) {
      fetch_keys();
      fetch_scales(pv);
    }
    __builtin_amdgcn_sched_barrier(0);
    // the largest value scale's exponent (NaN and infinity leave it)
    int ve = (int)(__builtin_bit_cast(uint32_t, vs_now) >> 23 & 255) - 127;
    if (ve > 127 || page < 0) ve = -126;
    ve = max(ve, __shfl_xor(ve, 16));
    ve = max(max(ve, __shfl_xor(ve, 32)), v_exp);
    if (base + kTile - 1 <= min_limit && __all(page >= 0)) {
      weigh.template operator()<false>(sc, f, vs_now, ve, 0);
    } else {   // tokens 0 .. left of this lane's 16 are seen
      const int left = page < 0 ? -1 : limit - (base + g * 16);
      weigh.template operator()<true>(sc, f, vs_now, ve, left);
    }
#pragma unroll
    for (int i = 0; i < VD; i++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const half8_t vf = codes_f16(vw[i][2 * h], vw[i][2 * h + 1]);
        o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf[h], o[i], 0, 0, 0);
        if constexpr (kTwo) o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pl[h], o[i], 0, 0, 0);
        if (h == 1 && i % 2 == 1) __builtin_amdgcn_sched_barrier(0);
      }
    if (more) fetch_values(pv);
    __builtin_amdgcn_sched_barrier(0);
  }
  l_run += __shfl_xor(l_run, 16);
  l_run += __shfl_xor(l_run, 32);

  // join the wavefronts: column (query row) col, o[i][e] is value column
  // 16 i + 4 g + e
  __shared__ float jm[NW][16], jl[NW][16];
  extern __shared__ __attribute__((aligned(16))) float jo[];   // [NW][16][D]
  if (g == 0) {
    jm[wave][col] = m_run;
    jl[wave][col] = l_run;
  }
  const float vref = ldexpf(1.0f, v_exp);
#pragma unroll
  for (int i = 0; i < VD; i++)
    *reinterpret_cast<float4_t*>(jo + ((wave * 16 + col) * D + i * 16 + g * 4)) = o[i] * vref;
  __syncthreads();
  const int Hq = c.heads * a.G;
  auto finish = [&](int r, int d, float v0, float v1, float m, float l) QMM_INLINE {
    const int64_t at = (int64_t)(t0 + i0 + r / G) * Hq + head * a.G + h0 + r % G;
    const bool any = l > 0.0f || l != l;
    const float back = any ? 1.0f / l : 0.0f;
    *reinterpret_cast<uint32_t*>(a.out + at * D + d) =
        from_f32(T{}, any ? v0 * back : 0.0f) | (uint32_t)from_f32(T{}, any ? v1 * back : 0.0f) << 16;
    if (d == 0 && a.lse) a.lse[at] = any ? fmaf(m, kLn2, logf(l)) : -__builtin_inff();
  };
  // a part in the workspace: per row the maximum and the sum, then the rows
  constexpr int kPart = 16 * (D + 2);
  const int64_t unit = (int64_t)blockIdx.x * gridDim.y + blockIdx.y;
  float* part = a.ws + unit * a.splits * kPart;
  auto put2 = [&](float* p, float x, float y) QMM_INLINE {
    const uint64_t w = __builtin_bit_cast(uint32_t, x) | (uint64_t)__builtin_bit_cast(uint32_t, y) << 32;
    __hip_atomic_store(reinterpret_cast<uint64_t*>(p), w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  auto get2 = [&](const float* p) QMM_INLINE {
    const uint64_t w = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
    return make_float2(__builtin_bit_cast(float, (uint32_t)w), __builtin_bit_cast(float, (uint32_t)(w >> 32)));
  };
  for (int i = tid; i < rows * (D / 2); i += 64 * NW) {
    const int r = i / (D / 2), d = i % (D / 2) * 2;
    float m = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < NW; w++) m = fmaxf(m, jm[w][r]);
    const float mu = m == -__builtin_inff() ? 0.0f : m;
    float l = 0.0f, v0 = 0.0f, v1 = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; w++) {
      const float e = __builtin_amdgcn_exp2f(jm[w][r] - mu);
      const float2 v = *reinterpret_cast<const float2*>(jo + (w * 16 + r) * D + d);
      l += jl[w][r] * e;
      v0 += v.x * e;
      v1 += v.y * e;
    }
    if (parts == 1) {
      finish(r, d, v0, v1, m, l);
    } else {
      float* mine = part + split * kPart;
      put2(mine + 32 + r * D + d, v0, v1);
      if (d == 0) put2(mine + 2 * r, m, l);
    }
  }
  if (parts == 1) return;
  // several workgroups share the rows: the last to arrive joins their parts,
  // in order. Relaxed agent-scope accesses are coherent across the XCDs' L2
  // caches; the stores have completed before the counter is touched, and the
  // wrapping increment leaves it at zero.
  __shared__ unsigned is_last;
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (tid == 0)
    is_last = __builtin_amdgcn_atomic_inc32(a.cnt + unit, (unsigned)(parts - 1), __ATOMIC_RELAXED,
                                            "agent") == (unsigned)(parts - 1);
  __syncthreads();
  if (!is_last) return;
  // every part's factor exp2(m - max) per row, and the rows' sums
  float* fac = jo;                       // [parts][16]; parts <= kMaxSplits
  for (int i = tid; i < parts * rows; i += 64 * NW) {
    const float2 ml = get2(part + i / rows * kPart + 2 * (i % rows));
    fac[i / rows * 16 + i % rows] = ml.x;
    fac[(kMaxSplits + i / rows) * 16 + i % rows] = ml.y;
  }
  __syncthreads();
  for (int r = wave; r < rows; r += NW) {   // a wavefront per row
    float m = -__builtin_inff();
    for (int w = lane; w < parts; w += 64) m = fmaxf(m, fac[w * 16 + r]);
#pragma unroll
    for (int x = 32; x >= 1; x >>= 1) m = fmaxf(m, __shfl_xor(m, x));
    const float mu = m == -__builtin_inff() ? 0.0f : m;
    float l = 0.0f;
    for (int w = lane; w < parts; w += 64) {
      const float e = __builtin_amdgcn_exp2f(fac[w * 16 + r] - mu);
      fac[w * 16 + r] = e;
      l += fac[(kMaxSplits + w) * 16 + r] * e;
    }
#pragma unroll
    for (int x = 32; x >= 1; x >>= 1) l += __shfl_xor(l, x);
    if (lane == 0) {
      jm[0][r] = m;
      jl[0][r] = l;
    }
  }
  __syncthreads();
  for (int i = tid; i < rows * (D / 2); i += 64 * NW) {
    const int r = i / (D / 2), d = i % (D / 2) * 2;
    float v0 = 0.0f, v1 = 0.0f;
    const float* p = part + 32 + r * D + d;
    int w = 0;
    for (; w + 8 <= parts; w += 8) {   // eight loads in flight
      float2 v[8];
#pragma unroll
      for (int x = 0; x < 8; x++) v[x] = get2(p + (w + x) * kPart);
#pragma unroll
      for (int x = 0; x < 8; x++) {
        const float e = fac[(w + x) * 16 + r];
        v0 = fmaf(v[x].x, e, v0);
        v1 = fmaf(v[x].y, e, v1);
      }
    }
    for (; w < parts; w++) {
      const float2 v = get2(p + w * kPart);
      const float e = fac[w * 16 + r];
      v0 = fmaf(v.x, e, v0);
      v1 = fmaf(v.y, e, v1);
    }
    finish(r, d, v0, v1, jm[0][r], jl[0][r]);
  }
}

// ------------------------------------------------------------------ prompts
// 32 query rows per wavefront, NW wavefronts, tiles of 64 tokens through two
// LDS buffers. The codes are turned into f16 once per workgroup on their way
// into LDS (keys [64][D], rows in the order in which the products want them;
// values [D][64]); the 16-byte pieces of a row are permuted by an exclusive-or
// with the row number, so that the 16 rows that are read together touch all
// banks.
//
// S^T = K Q^T with v_mfma_f32_32x32x16_f16; D row 8 i + 4 h + r of lane half h
// is made token 16 (i/2) + 8 h + 4 (i%2) + r, so that a lane's registers are,
// eight by eight, the B operand of O^T = V^T P^T. A page's scales are uniform
// over groups of 16 tokens, hence scalars. The running maximum is only raised
// when it grows by more than 2^8: until then weights reach 256, which f16 and
// the fp32 sums hold as well, and nothing is rescaled.
template <class T, int D, int NW>
__global__ __launch_bounds__(64 * NW) void kv8_prompt_kernel(AttnArgs a) {
  constexpr int KS = D / 16, VD = D / 32, kThreads = 64 * NW;
  constexpr int kUnits = kTile * D / 16 / kThreads;   // 16 codes per unit
  // f16 results: the weights go in as two f16 terms, since 11 bits of them would
  // cost as much as rounding the result
  constexpr bool kTwo = __is_same(T, F16);
  static_assert(kUnits >= 1, "a unit per thread");
  __shared__ __attribute__((aligned(16))) uint16_t lk[2][kTile * D], lv[2][kTile * D];
  __shared__ float lsk[2][4], lsv[2][4];
  // position of 16-byte piece p of key row r (rows of D * 2 bytes)
  auto key_piece = [](int r, int p) QMM_INLINE {
    return (p ^ (D == 64 ? r >> 1 : r)) & (D / 8 - 1);
  };
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int col = lane % 32, h = lane / 32;
  const int head = blockIdx.y;
  const Kv8& c = a.c;
  // long sequences' last items have most to do: they come first
  const int index = gridDim.x - 1 - blockIdx.x;
  const int s = find_seq(a.q, index, a.unit, a.extra);
  const int t0 = a.q.first(s), n = a.q.count(s), len = a.q.length(s, c.bt_log2);
  const int item = index - first_item(a.q, s, a.unit, a.extra);
  const int i0 = item * a.unit;
  if (item < 0 || i0 >= n || (int64_t)n * a.G <= a.many) return;
  const int ntok = min(n - i0, a.unit);
  const int rows = ntok * a.G;
  const int most = len - n + i0 + ntok;
  const int tiles = most > 0 ? (most + kTile - 1) / kTile : 0;

  // this lane's query row; rows past the last repeat it, and nothing reads them
  const int rr = min(wave * 32 + col, rows - 1);
  const int ct = rr / a.G, ch = rr % a.G;
  const int limit = len - n + i0 + ct;
  const int wave_min = len - n + i0 + min(wave * 32, rows - 1) / a.G;
  const int wave_max = len - n + i0 + min(wave * 32 + 31, rows - 1) / a.G;
  const int64_t at = (int64_t)(t0 + i0 + ct) * (c.heads * a.G) + head * a.G + ch;
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
  float m_run = -__builtin_inff(), l_run = 0.0f;
  int v_exp = -126;   // O holds sums of codes weighted with p * vs / 2^v_exp

  const int32_t* row = a.q.table + (int64_t)s * a.q.W;
  const int bt = c.bt_log2;
  auto page_at = [&](int t) QMM_INLINE {
    const int p = t < most ? row[t >> bt] : -1;   // most <= W << bt
    return p < c.pages ? p : -1;
  };
  // Each tile's pages are looked up two tiles ahead and its codes and scales
  // loaded one tile ahead, so that no step waits for a load it has just asked
  // for. Unit u of a thread: 16 columns of key token u / (D/16), 16 tokens of
  // value column u / 4; threads 0 .. 3 carry the scales of their 16 tokens.
  int kp[kUnits], vp[kUnits];
  auto look_up = [&](int tile) QMM_INLINE {
#pragma unroll
    for (int i = 0; i < kUnits; i++) {
      const int u = i * kThreads + tid;
      kp[i] = page_at(tile * kTile + u / (D / 16));
      vp[i] = page_at(tile * kTile + u % 4 * 16);
    }
  };
  u32x4_t kw[kUnits], vw[kUnits];
  float sk = 0, sv = 0;
  bool miss = false;
  auto fetch = [&]() QMM_INLINE {
    if (tid < 4) {
      miss = vp[0] < 0;
      const int64_t blk = (int64_t)(miss ? 0 : vp[0]) * c.heads + head;
      sk = c.ks[blk];
      sv = c.vs[blk];
    }
#pragma unroll
    for (int i = 0; i < kUnits; i++) {
      const int u = i * kThreads + tid;
      const int tk = u / (D / 16), kc = u % (D / 16), vd = u / 4, vc = u % 4 * 16;
      kw[i] = *reinterpret_cast<const u32x4_t*>(c.k + c.block(kp[i] < 0 ? 0 : kp[i], head) +
                                                (tk & ((1 << bt) - 1)) * D + kc * 16);
      vw[i] = *reinterpret_cast<const u32x4_t*>(c.v + c.block(vp[i] < 0 ? 0 : vp[i], head) +
                                                ((int64_t)vd << bt) + (vc & ((1 << bt) - 1)));
    }
  };
  auto put = [&](int buf) QMM_INLINE {
    if (tid < 4) {
      lsk[buf][tid] = sk;
      lsv[buf][tid] = miss ? -1.0f : sv;   // no scale is negative: not seen
    }
#pragma unroll
    for (int i = 0; i < kUnits; i++) {
      const int u = i * kThreads + tid;
      const int tk = u / (D / 16), kc = u % (D / 16);
      const int kr = (tk & 32) + 8 * ((tk >> 4 & 1) * 2 + (tk >> 2 & 1)) + 4 * (tk >> 3 & 1) + (tk & 3);
      const int vd = u / 4, vc = u % 4;
#pragma unroll
      for (int j = 0; j < 2; j++) {
        *reinterpret_cast<half8_t*>(&lk[buf][kr * D + key_piece(kr, kc * 2 + j) * 8]) =
            codes_f16(kw[i][2 * j], kw[i][2 * j + 1]);
        *reinterpret_cast<half8_t*>(&lv[buf][vd * kTile + (((vc * 2 + j) ^ vd >> 1) & 7) * 8]) =
            codes_f16(vw[i][2 * j], vw[i][2 * j + 1]);
      }
    }
  };
  // one tile's softmax and second product; MASK: some of its tokens are not
  // seen by some of the wavefront's rows
  auto weigh = [&]<bool MASK>(float16_t* sc, const float* f, const float* vs, int ve, int left,
                              uint32_t missing, int buf) QMM_INLINE {
    // element e of sc[j]: token 32 j + 16 (e/8) + 8 h + e%8
    float mx = -__builtin_inff();
#pragma unroll
    for (int g = 0; g < 4; g++) {
      float top = -__builtin_inff();
#pragma unroll
      for (int e = 0; e < 8; e++) {
        float x = sc[g / 2][g % 2 * 8 + e];
        if constexpr (MASK) {
          x = g * 16 + e <= left && !(missing >> g & 1) ? x * f[g] : -__builtin_inff();
          sc[g / 2][g % 2 * 8 + e] = x;
        }
        top = fmaxf(top, x);
      }
      mx = fmaxf(mx, MASK ? top : top * f[g]);
    }
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    if (__any(mx > m_run + 8.0f || ve != v_exp)) {
      const float mn = fmaxf(m_run, mx);
      const float al = mn == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m_run - mn);
      const float down = ldexpf(al, v_exp - ve);
      l_run *= al;
#pragma unroll
      for (int i = 0; i < VD; i++) o[i] *= down;
      m_run = mn;
      v_exp = ve;
    }
    const float mu = m_run == -__builtin_inff() ? 0.0f : m_run;
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const float r = ldexpf(vs[g], -v_exp);
      half8_t hi, lo;
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const float x = sc[g / 2][g % 2 * 8 + e];
        const float p = __builtin_amdgcn_exp2f(MASK ? x - mu : fmaf(x, f[g], -mu));
        l_run += p;
        float w = p * r;
        if constexpr (MASK) w = g * 16 + e <= left && !(missing >> g & 1) ? w : 0.0f;
        hi[e] = (_Float16)w;
        if constexpr (kTwo) lo[e] = (_Float16)(w - (float)hi[e]);
      }
#pragma unroll
      for (int i = 0; i < VD; i++) {
        const int d = i * 32 + col;
        const half8_t vf = *reinterpret_cast<const half8_t*>(
            &lv[buf][d * kTile + (((g * 2 + h) ^ d >> 1) & 7) * 8]);
        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, hi, o[i], 0, 0, 0);
        if constexpr (kTwo) o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, lo, o[i], 0, 0, 0);
      }
    }
  };
  if (tiles > 0) {
    look_up(0);
    fetch();
    look_up(1);
    put(0);
  }
  for (int tile = 0; tile < tiles; tile++) {
    const int buf = tile & 1;
    __syncthreads();
    if (tile + 1 < tiles) {
      fetch();
      look_up(tile + 2);
    }
    const int base = tile * kTile;
    if (base <= wave_max) {
      float f[4], vs[4];
      int ve = v_exp;
      uint32_t missing = 0;
#pragma unroll
      for (int g = 0; g < 4; g++) {
        f[g] = lsk[buf][g] * qs;
        vs[g] = lsv[buf][g];
        const int e = (int)(__builtin_bit_cast(uint32_t, vs[g]) >> 23 & 255) - 127;
        const bool gone = __builtin_bit_cast(uint32_t, vs[g]) == 0xbf800000u;
        if (!gone && e <= 127) ve = max(ve, e);   // NaN and infinity leave it
        missing |= gone ? 1u << g : 0u;
      }
      float16_t sc[2];
#pragma unroll
      for (int j = 0; j < 2; j++)
#pragma unroll
        for (int e = 0; e < 16; e++) sc[j][e] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const int r = j * 32 + col;
          const half8_t kf =
              *reinterpret_cast<const half8_t*>(&lk[buf][r * D + key_piece(r, ks * 2 + h) * 8]);
          sc[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[ks], sc[j], 0, 0, 0);
        }
      const int left = limit - base - h * 8;   // tokens g * 16 + e up to this are seen
      if (base + kTile - 1 <= wave_min && missing == 0)
        weigh.template operator()<false>(sc, f, vs, ve, left, missing, buf);
      else
        weigh.template operator()<true>(sc, f, vs, ve, left, missing, buf);
    }
    if (tile + 1 < tiles) put(buf ^ 1);
  }
  if (wave * 32 + col >= rows) return;
  l_run += __shfl_xor(l_run, 32);
  const bool any = l_run > 0.0f || l_run != l_run;
  const float back = any ? ldexpf(1.0f, v_exp) / l_run : 0.0f;
#pragma unroll
  for (int i = 0; i < VD; i++)
#pragma unroll
    for (int q = 0; q < 4; q++) {
      uint16_t w[4];
#pragma unroll
      for (int e = 0; e < 4; e++) w[e] = from_f32(T{}, any ? o[i][q * 4 + e] * back : 0.0f);
      *reinterpret_cast<uint2*>(a.out + at * D + i * 32 + q * 8 + h * 4) =
          make_uint2(w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16);
    }
  if (h == 0 && a.lse) a.lse[at] = any ? fmaf(m_run, kLn2, logf(l_run)) : -__builtin_inff();
}

// Sequences with at most this many query rows (new tokens x heads of a group)
// go to the decode kernel, 16 rows at a time; the others to the prompt kernel.
constexpr int kFewRows = 64;

struct Plan {
  int unit, extra, splits, per, nw, many;
  int64_t items, columns;   // grid: items x heads and blocks of a group's heads
  bool prompts;
  int p_unit;
  int64_t p_items;
};

Plan plan(const Kv8& c, int64_t T, int64_t Hq, int64_t S, int64_t W) {
  Plan p{};
  const int64_t G = Hq / c.heads;
  const int prompt_rows = c.dim == 128 ? 256 : 128;
  // the packed batch says how many new tokens a sequence can have at most
  const int64_t longest = T;
  p.prompts = longest * G > kFewRows && T > S && G <= prompt_rows;
  p.many = p.prompts ? kFewRows : INT32_MAX;
  p.unit = T > S && G <= 8 ? (int)(16 / G) : 1;
  p.extra = p.unit > 1 ? 1 : 0;
  p.items = T / p.unit + p.extra * S;
  p.columns = c.heads * ((G + 15) / 16);
  p.p_unit = (int)(prompt_rows / (G < prompt_rows ? G : prompt_rows));
  p.p_items = T / p.p_unit + S;
  p.nw = kDecodeWaves;
  const int64_t units = (T < p.items ? T : p.items) * p.columns;
  const int64_t tiles = ((W << c.bt_log2) + kTile - 1) / kTile;
  // Every workgroup takes the same number of tiles (a multiple of the
  // wavefronts), so that ragged sequences load the chip evenly: as many as
  // make about 2048 workgroups of sequences that fill their table rows, and
  // no sequence is cut into more parts than one workgroup joins.
  int64_t per = (units * tiles + 2047) / 2048;
  per = per > (tiles + kMaxSplits - 1) / kMaxSplits ? per : (tiles + kMaxSplits - 1) / kMaxSplits;
  if (p.items * p.columns > kScratchCounters) per = tiles;
  per = (per + p.nw - 1) / p.nw * p.nw;
  p.per = (int)per;
  const int64_t sp = (tiles + per - 1) / per;
  p.splits = (int)sp;
  return p;
}

}  // namespace

int64_t kv8_attention_work(const Kv8& c, int64_t T, int64_t Hq, int64_t S, int64_t W) {
  const Plan p = plan(c, T, Hq, S, W);
  return p.splits > 1 ? p.items * p.columns * p.splits * 16 * (c.dim + 2) * 4 : 0;
}

hipError_t launch_kv8_attention(const Kv8& c, int dt, const void* q, int64_t ldq, int64_t T,
                                int64_t Hq, const int32_t* table, const int32_t* lens,
                                const int32_t* cu, int64_t S, int64_t W, float scale, void* out,
                                float* lse, unsigned* cnt, float* ws, hipStream_t st) {
  const Plan p = plan(c, T, Hq, S, W);
  AttnArgs a{c, {table, lens, cu, (int)S, (int)W, (int)T}, static_cast<const uint16_t*>(q), ldq,
             (int)(Hq / c.heads), p.unit, p.extra, p.many, fabsf(scale) * kLog2e,
             scale < 0 ? 0x80008000u : 0u, static_cast<uint16_t*>(out), lse, p.splits, p.per, ws, cnt};
  const dim3 grid((unsigned)p.items, (unsigned)p.columns, (unsigned)p.splits);
  auto go = [&]<class T_, int D>() {
    constexpr int NW = kDecodeWaves;
    const size_t lds = (size_t)NW * 16 * D * 4;
    auto decode = [&]<int BT>() {
      hipLaunchKernelGGL((kv8_decode_kernel<T_, D, BT, NW>), grid, dim3(64 * NW), lds, st, a);
    };
    if (c.bt_log2 == 4) decode.template operator()<4>();
    else if (c.bt_log2 == 5) decode.template operator()<5>();
    else decode.template operator()<6>();
    if (!p.prompts) return;
    AttnArgs b = a;
    b.unit = p.p_unit;
    b.extra = 1;
    hipLaunchKernelGGL((kv8_prompt_kernel<T_, D, D == 256 ? 4 : D == 128 ? 8 : 4>),
                       dim3((unsigned)p.p_items, (unsigned)c.heads), dim3(D == 128 ? 512 : 256), 0,
                       st, b);
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

}  // namespace qmm
