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
// exp(x - m) * vs are rounded to 11 bits on their way into the second
// product; sums, maxima and the normaliser stay in fp32.
#include "kernels.hpp"
#include "kv8_common.hpp"

namespace qmm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTile = 64;   // tokens per step of a wavefront

struct AttnArgs {
  Kv8 c;
  Kv8Seqs q;
  const uint16_t* x;   // queries, row t at x + t * ldq
  int64_t ldq;
  int G;               // query heads per cache head, 16 at a time
  int rows_log2, extra;   // new tokens per workgroup, spare items per sequence
  float scale;         // of the scores, times log2 e
  uint16_t* out;       // [T][heads * G][D]
  float* lse;          // [T][heads * G] or null
  int splits;          // of a sequence's tiles, over gridDim.z workgroups
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

__device__ __forceinline__ uint32_t max3(uint32_t a, uint32_t b) { return a > b ? a : b; }

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
template <class T, int D, int NW>
__global__ __launch_bounds__(64 * NW) void kv8_decode_kernel(AttnArgs a) {
  constexpr int KD = D / 64, VD = D / 16;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int col = lane % 16, g = lane / 16;
  const int blocks = (a.G + 15) / 16;   // of heads in a group
  const int head = blockIdx.y / blocks, h0 = blockIdx.y % blocks * 16, split = blockIdx.z;
  const int G = min(16, a.G - h0);
  const Kv8& c = a.c;
  const int s = find_seq(a.q, blockIdx.x, a.rows_log2, a.extra);
  const int64_t t0 = a.q.first(s), n = a.q.count(s), len = a.q.length(s, c.bt_log2);
  const int64_t item = blockIdx.x - ((t0 >> a.rows_log2) + (int64_t)a.extra * s);
  const int tok = 1 << a.rows_log2;          // new tokens per workgroup
  const int64_t i0 = item << a.rows_log2;
  if (item < 0 || i0 >= n) return;
  const int ntok = n - i0 < tok ? (int)(n - i0) : tok;
  const int rows = ntok * G;                 // <= 16
  // positions that the last row sees, tiles of them, this workgroup's share
  const int64_t most = len - n + i0 + ntok;
  const int tiles = most > 0 ? (int)((most + kTile - 1) / kTile) : 0;
  const int per = max((tiles + a.splits - 1) / a.splits, NW);   // tiles per workgroup
  const int parts = tiles > 0 ? (tiles + per - 1) / per : 1;
  if (split >= parts) return;
  const int first = split * per, last = min(first + per, tiles);

  // this lane's query row: token col / G, head col % G (columns past the rows
  // repeat the first one, and nothing reads them)
  const int ct = col < rows ? col / G : 0, ch = col < rows ? col % G : 0;
  const int64_t trow = t0 + i0 + ct;
  const int qh = head * a.G + h0 + ch;
  const int64_t min_limit = len - n + i0;   // last position that every row sees
  const int64_t limit = min_limit + ct;     // that this one sees
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
        u[b][h] = *reinterpret_cast<const uint4*>(qr + b * 64 + h * 8);
        m = amax_pair(amax_pair(amax_pair(amax_pair(m, u[b][h].x), u[b][h].y), u[b][h].z), u[b][h].w);
      }
    if constexpr (__is_same(T, F16)) {
#pragma unroll
      for (int b = 0; b < KD; b++)
#pragma unroll
        for (int h = 0; h < 2; h++) qf[b][h] = __builtin_bit_cast(half8_t, u[b][h]);
    } else {
      // bf16: times 2^-e with 2^e the row's largest power of two, exact in
      // f16 down to 2^-14 of it (and to 2^-24 with fewer bits)
      m = amax_halves(m);
      m = max3(m, (uint32_t)__shfl_xor((int)m, 16));
      m = max3(m, (uint32_t)__shfl_xor((int)m, 32));
      int e = (int)(m >> 7) - 127;
      e = e < -100 ? -100 : e > 100 ? 100 : e;
      const float down = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
      qs *= __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
#pragma unroll
      for (int b = 0; b < KD; b++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
          float f[8];
          unpack8(BF16{}, u[b][h], f);
#pragma unroll
          for (int i = 0; i < 8; i++) qf[b][h][i] = (_Float16)(f[i] * down);
        }
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
  const int bt = c.bt_log2;
  // page of token t of the sequence; tokens past the row's pages read page 0
  auto page_at = [&](int64_t t) QMM_INLINE {
    const int64_t j = t >> bt;
    const int p = j < a.q.W && t < most ? row[j] : -1;
    return p < c.pages ? p : -1;
  };
  const int kg = (col / 4) * 16;   // first token of this lane's K rows in a tile
  for (int tile = first + wave; tile < last; tile += NW) {
    const int64_t base = (int64_t)tile * kTile;
    const int pk = page_at(base + kg), pv = page_at(base + g * 16);
    const int8_t* kp = c.k + c.block(pk < 0 ? 0 : pk, head) +
                       ((kg & ((1 << bt) - 1)) + col % 4) * D + g * 16;
    const int8_t* vp = c.v + c.block(pv < 0 ? 0 : pv, head) + ((int64_t)col << bt) +
                       ((g * 16) & ((1 << bt) - 1));
    u32x4_t kw[4][KD], vw[VD];
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int b = 0; b < KD; b++)
        kw[j][b] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4_t*>(kp + j * 4 * D + b * 64));
#pragma unroll
    for (int i = 0; i < VD; i++)
      vw[i] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4_t*>(vp + ((int64_t)(i * 16) << bt)));
    const int64_t blk = (int64_t)(pv < 0 ? 0 : pv) * c.heads + head;
    const float ks = c.ks[blk], vs = c.vs[blk];

    float4_t sc[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      sc[j] = float4_t{0, 0, 0, 0};
#pragma unroll
      for (int b = 0; b < KD; b++)
#pragma unroll
        for (int h = 0; h < 2; h++)
          sc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
              codes_f16(kw[j][b][2 * h], kw[j][b][2 * h + 1]), qf[b][h], sc[j], 0, 0, 0);
    }
    const float f = ks * qs;
    float p[16];
    float mx = m_run;
    // every token of the tile seen by every row? (then nothing is masked)
    const bool whole = base + kTile - 1 <= min_limit && __all(pv >= 0);
    const int64_t left = pv < 0 ? -1 : limit - (base + g * 16);   // tokens 0 .. left are seen
#pragma unroll
    for (int i = 0; i < 16; i++) {
      p[i] = sc[i / 4][i % 4] * f;
      if (!whole) p[i] = i <= left ? p[i] : -__builtin_inff();
      mx = fmaxf(mx, p[i]);
    }
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float mu = mx == -__builtin_inff() ? 0.0f : mx;
    // the largest value scale's exponent (NaN and infinity leave it)
    int ve = (int)(__builtin_bit_cast(uint32_t, vs) >> 23 & 255) - 127;
    if (ve > 127 || pv < 0) ve = -126;
    ve = max(ve, __shfl_xor(ve, 16));
    ve = max(max(ve, __shfl_xor(ve, 32)), v_exp);
    if (__any(mx != m_run || ve != v_exp)) {
      const float al = __builtin_amdgcn_exp2f(m_run - mu) ;
      const float down = ldexpf(al, v_exp - ve);
      l_run *= al;
#pragma unroll
      for (int i = 0; i < VD; i++) o[i] *= down;
      m_run = mx;
      v_exp = ve;
    }
    const float r = ldexpf(vs, -v_exp);
    half8_t pf[2];
#pragma unroll
    for (int i = 0; i < 16; i++) {
      const float e = __builtin_amdgcn_exp2f(p[i] - mu);
      l_run += e;
      float w = e * r;
      if (!whole) w = i <= left ? w : 0.0f;
      pf[i / 8][i % 8] = (_Float16)w;
    }
#pragma unroll
    for (int i = 0; i < VD; i++)
#pragma unroll
      for (int h = 0; h < 2; h++)
        o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16(vw[i][2 * h], vw[i][2 * h + 1]),
                                                      pf[h], o[i], 0, 0, 0);
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
  auto finish = [&](int r, int d, float v, float m, float l) QMM_INLINE {
    const int64_t at = (t0 + i0 + r / G) * Hq + head * a.G + h0 + r % G;
    a.out[at * D + d] = from_f32(T{}, l > 0.0f || l != l ? v / l : 0.0f);
    if (d == 0 && a.lse)
      a.lse[at] = l > 0.0f || l != l ? fmaf(m, kLn2, logf(l)) : -__builtin_inff();
  };
  const int64_t unit = (int64_t)blockIdx.x * gridDim.y + blockIdx.y;
  float* part = a.ws + unit * a.splits * (16 * (D + 2));
  for (int i = tid; i < rows * D; i += 64 * NW) {
    const int r = i / D, d = i % D;
    float m = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < NW; w++) m = fmaxf(m, jm[w][r]);
    const float mu = m == -__builtin_inff() ? 0.0f : m;
    float l = 0.0f, v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; w++) {
      const float e = __builtin_amdgcn_exp2f(jm[w][r] - mu);
      l += jl[w][r] * e;
      v += jo[(w * 16 + r) * D + d] * e;
    }
    if (parts == 1) {
      finish(r, d, v, m, l);
    } else {
      float* mine = part + split * (16 * (D + 2));
      __hip_atomic_store(mine + 32 + r * D + d, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (d == 0) {
        __hip_atomic_store(mine + r, m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(mine + 16 + r, l, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
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
  auto get = [&](const float* p) QMM_INLINE {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  for (int i = tid; i < rows * D; i += 64 * NW) {
    const int r = i / D, d = i % D;
    float m = -__builtin_inff(), l = 0.0f, v = 0.0f;
    for (int w = 0; w < parts; w++) {
      const float* p = part + w * (16 * (D + 2));
      const float mw = get(p + r), lw = get(p + 16 + r), vw = get(p + 32 + r * D + d);
      const float mn = fmaxf(m, mw), mu = mn == -__builtin_inff() ? 0.0f : mn;
      const float ea = __builtin_amdgcn_exp2f(m - mu), eb = __builtin_amdgcn_exp2f(mw - mu);
      l = l * ea + lw * eb;
      v = v * ea + vw * eb;
      m = mn;
    }
    finish(r, d, v, m, l);
  }
}

struct Plan {
  int rows_log2, extra, splits, nw;
  int64_t items, columns;   // grid: items x heads and blocks of a group's heads
};

Plan plan(const Kv8& c, int64_t T, int64_t Hq, int64_t S, int64_t W) {
  Plan p{};
  const int64_t G = Hq / c.heads;
  p.rows_log2 = 0;
  while (2 * G << p.rows_log2 <= 16 && (T >> p.rows_log2) > S) p.rows_log2++;
  p.extra = p.rows_log2 > 0 ? 1 : 0;
  p.items = (T >> p.rows_log2) + p.extra * S;
  p.columns = c.heads * ((G + 15) / 16);
  p.nw = c.dim == 256 ? 4 : 8;
  const int64_t units = (T < p.items ? T : p.items) * p.columns;
  const int64_t tiles = ((W << c.bt_log2) + kTile - 1) / kTile;
  // enough workgroups to fill the chip several times over, each with at least
  // one tile per wavefront
  int64_t sp = 1024 / (units < 1 ? 1 : units);
  sp = sp < 1 ? 1 : sp;
  sp = sp < tiles / p.nw ? sp : tiles / p.nw;
  sp = sp < 1 ? 1 : sp > 128 ? 128 : sp;
  if (p.items * p.columns > kScratchCounters) sp = 1;
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
  AttnArgs a{c, {table, lens, cu, (int)S, (int)W, T}, static_cast<const uint16_t*>(q), ldq,
             (int)(Hq / c.heads), p.rows_log2, p.extra, scale * kLog2e, static_cast<uint16_t*>(out), lse,
             p.splits, ws, cnt};
  const dim3 grid((unsigned)p.items, (unsigned)p.columns, (unsigned)p.splits);
  auto go = [&]<class T_, int D, int NW>() {
    const size_t lds = (size_t)NW * 16 * D * 4;
    hipLaunchKernelGGL((kv8_decode_kernel<T_, D, NW>), grid, dim3(64 * NW), lds, st, a);
  };
  auto by_dim = [&]<class T_>() {
    if (c.dim == 64) go.template operator()<T_, 64, 8>();
    else if (c.dim == 128) go.template operator()<T_, 128, 8>();
    else go.template operator()<T_, 256, 4>();
  };
  if (dt == 0) by_dim.template operator()<F16>();
  else by_dim.template operator()<BF16>();
  return hipGetLastError();
}

}  // namespace qmm
