// 8-bit integer products with one scale per token (row of x) and per channel
// (row of W):  y[m,n] = T(fl32(sx[m] * sw[n]) * sum_k xq[m,k] * wq[n,k] + bias[n]),
// the integer sum exact in 32 bits (K < 2^17), and the row quantizer
// sx[m] = fl32(max_k |x[m,k]| / 127), xq = clamp(rint(fl32(x / sx)), -127, 127).
//
// Kernels: the quantizer; a GEMV for a few rows of x, bound by reading W
// once; a tile GEMM, bound by the matrix units (v_mfma_i32_32x32x32_i8 takes
// 16 bytes of each operand per lane, twice the multiply-adds of the 16-bit
// form in the same cycles).
#include "int8_common.hpp"
#include "kernels.hpp"

namespace qmm {
namespace {

// ------------------------------------------------------------ row quantizer
// NT threads per row, each holding up to 4 chunks of 8 elements in registers
// (rows longer than 32 * NT are read a second time). Bound by memory, x read
// once: 8192 x 4096 in 27 us, 3.7 TB/s of what is read and written; a few rows by
// the chain of load, maximum and store (13 x 2048: 3.4 us).
template <class T, int NT>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void i8_quantize_kernel(const uint16_t* __restrict__ x,
                                                          int64_t ldx, int64_t rows, int K,
                                                          int8_t* __restrict__ xq,
                                                          float* __restrict__ sx) {
  constexpr int kHold = 4, kBlock = NT < 256 ? 256 : NT;
  const int64_t row = (int64_t)blockIdx.x * (kBlock / NT) + threadIdx.x / NT;
  const int t = threadIdx.x % NT;
  const bool live = row < rows;
  const uint16_t* xr = x + (live ? row : 0) * ldx;
  uint4 u[kHold];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kHold; i++) {
    const int k = (i * NT + t) * 8;
    u[i] = live && k < K ? *reinterpret_cast<const uint4*>(xr + k) : make_uint4(0, 0, 0, 0);
    m = amax_pair(amax_pair(amax_pair(amax_pair(m, u[i].x), u[i].y), u[i].z), u[i].w);
  }
  if (live)
    for (int k = (kHold * NT + t) * 8; k < K; k += NT * 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(xr + k);
      m = amax_pair(amax_pair(amax_pair(amax_pair(m, v.x), v.y), v.z), v.w);
    }
  uint32_t top = wave_umax(amax_halves(m));
  if constexpr (NT > 64) {
    __shared__ uint32_t part[kBlock / 64];   // of the row's NT / 64 wavefronts
    const int wave = threadIdx.x / 64, w0 = wave - t / 64;
    if (t % 64 == 0) part[wave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 64; i++) top = part[w0 + i] > top ? part[w0 + i] : top;
  }
  if (!live) return;
  const float s = amax_scale<T>(top);
  const Divisor d = divisor(s);
  if (t == 0) sx[row] = s;
  int8_t* qr = xq + row * K;
  auto put = [&](int k, const uint4& v) QMM_INLINE {
    float f[8], q[8];
    unpack8(T{}, v, f);
    divide_round<8>(f, d, q);
    *reinterpret_cast<uint2*>(qr + k) =
        make_uint2(pack_codes(q[0], q[1], q[2], q[3]), pack_codes(q[4], q[5], q[6], q[7]));
  };
#pragma unroll
  for (int i = 0; i < kHold; i++) {
    const int k = (i * NT + t) * 8;
    if (k < K) put(k, u[i]);
  }
  for (int k = (kHold * NT + t) * 8; k < K; k += NT * 8)
    put(k, *reinterpret_cast<const uint4*>(xr + k));
}

// --------------------------------------------------------------------- GEMV
// 16 rows of W and up to 16 * MT rows of x per workgroup; its NW wavefronts
// take 128-byte pieces of K in turn and their integer sums are
// added in LDS. v_mfma_i32_16x16x64_i8: A (W) row lane%16, B (x) column
// lane%16, both k = 16 * (lane/16) .. +16; D column lane%16, rows
// 4 * (lane/16) .. +4. Bound by reading W: 1 x 4096 x 4096 in 5.7 us, back to back
// with its weights among others, of which 3.3 are the bytes at a copy's rate; 64 x
// 4096 x 4096 in 13.2.

template <class T>
__device__ __forceinline__ uint16_t i8_out(int acc, float sx, float sw, const uint16_t* bias,
                                           int64_t n) {
  float v = sx * sw * (float)acc;
  if (bias) v = fmaf(sx * sw, (float)acc, to_f32(T{}, bias[n]));
  return from_f32(T{}, v);
}

// FUSED: x itself (at most kGvChunks * 512 pieces of 8, at most 16 rows) comes
// in, and every workgroup quantizes it into LDS while its first pieces of W
// are on their way; otherwise codes and scales come in.
// (13 x 2048: 14.2 us fused, 10.6 us in two launches; 1 x 4096: 5.7 and 10.0.)
constexpr int kGvChunks = 2, kGvFused = 8;   // (wavefronts)

template <class T, int MT, int NW, bool FUSED>
__global__ __launch_bounds__(64 * NW) void i8_gemv_kernel(
    const uint16_t* __restrict__ x, int64_t ldx, const int8_t* __restrict__ xq,
    const float* __restrict__ sx, const int8_t* __restrict__ wq, const float* __restrict__ sw,
    const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int M, int N, int K) {
  constexpr int kThreads = 64 * NW;
  constexpr int kGvHold = MT <= 2 ? 4 : 2;   // pieces in flight per wavefront
  __shared__ int part[NW][MT * 256];
  __shared__ uint32_t top[16];
  extern __shared__ __attribute__((aligned(16))) uint8_t codes[];   // FUSED: [M][K + 16]
  const int tid = threadIdx.x, lane = tid % 64;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int r = lane % 16, g = lane / 16;
  const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * 16 * MT;
  const int wrows = (int)(N - n0 < 16 ? N - n0 : 16);
  const int xrows = (int)(M - m0 < 16 * MT ? M - m0 : 16 * MT);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(wq + n0 * K, (uint32_t)wrows * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(xq + m0 * K, FUSED ? 0u : (uint32_t)xrows * (uint32_t)K);
  int4_t acc[MT];
#pragma unroll
  for (int i = 0; i < MT; i++) acc[i] = int4_t{0, 0, 0, 0};
  const uint32_t row = (uint32_t)r * (uint32_t)K;
  // out-of-range pieces and rows load zeros
  auto at = [&](uint32_t base, int k) QMM_INLINE { return base + (k < K ? (uint32_t)k : kOob); };
  u32x4_t w[kGvHold][2];
  auto fetch = [&](int k0) QMM_INLINE {
#pragma unroll
    for (int i = 0; i < kGvHold; i++)
#pragma unroll
      for (int h = 0; h < 2; h++)
        w[i][h] = __builtin_amdgcn_raw_buffer_load_b128(
            rw, (int)at(row, k0 + i * NW * 128 + h * 64 + g * 16), 0, 0);
  };
  fetch(wave * 128);
  const int ldc = K + 16;   // (16 rows' pieces fall on different banks)
  if constexpr (FUSED) {
    const int per = K / 8, pieces = M * per;
    uint4 u[kGvChunks];
    if (tid < 16) top[tid] = 0;
#pragma unroll
    for (int i = 0; i < kGvChunks; i++) {
      const int c = i * kThreads + tid, m = c / per;
      if (c < pieces) u[i] = *reinterpret_cast<const uint4*>(x + m * ldx + (c - m * per) * 8);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGvChunks; i++) {
      const int c = i * kThreads + tid;
      if (i * kThreads + wave * 64 >= pieces) break;
      const int m = min(c, pieces - 1) / per;
      const uint32_t v = c < pieces ? amax_halves(amax_pair(amax_pair(amax_pair(amax_pair(0, u[i].x), u[i].y), u[i].z), u[i].w)) : 0;
      if (__all(m == __builtin_amdgcn_readfirstlane(m))) {   // one row: one update
        const uint32_t a = wave_umax(v);
        if (lane == 0) atomicMax(&top[m], a);
      } else if (c < pieces) {
        atomicMax(&top[m], v);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGvChunks; i++) {
      const int c = i * kThreads + tid, m = c / per;
      if (c < pieces) {
        const Divisor d = divisor(amax_scale<T>(top[m]));
        float f[8], q[8];
        unpack8(T{}, u[i], f);
        divide_round<8>(f, d, q);
        *reinterpret_cast<uint2*>(codes + m * ldc + (c - m * per) * 8) =
            make_uint2(pack_codes(q[0], q[1], q[2], q[3]), pack_codes(q[4], q[5], q[6], q[7]));
      }
    }
    __syncthreads();
  }
  for (int k0 = wave * 128; k0 < K; k0 += NW * 128 * kGvHold) {
    if (k0 > wave * 128) fetch(k0);
    // x comes from the L2 (or LDS); all of it is asked for before its first use
    u32x4_t xv[MT][kGvHold][2];
#pragma unroll
    for (int i = 0; i < kGvHold; i++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int k = k0 + i * NW * 128 + h * 64 + g * 16;
#pragma unroll
        for (int t = 0; t < MT; t++) {
          if constexpr (FUSED)   // (past K: the last piece again, W is zero there)
            xv[t][i][h] = *reinterpret_cast<const u32x4_t*>(codes + min(r, M - 1) * ldc + min(k, K - 16));
          else
            xv[t][i][h] = __builtin_amdgcn_raw_buffer_load_b128(
                rx, (int)at(row + (uint32_t)(t * 16) * (uint32_t)K, k), 0, 0);
        }
      }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kGvHold; i++)
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int t = 0; t < MT; t++)
          acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
              __builtin_bit_cast(int4_t, w[i][h]), __builtin_bit_cast(int4_t, xv[t][i][h]), acc[t],
              0, 0, 0);
  }
#pragma unroll
  for (int t = 0; t < MT; t++)
#pragma unroll
    for (int e = 0; e < 4; e++) part[wave][t * 256 + r * 16 + g * 4 + e] = acc[t][e];
  __syncthreads();
  for (int i = tid; i < MT * 256; i += kThreads) {
    const int64_t m = m0 + i / 16, n = n0 + i % 16;
    if (m >= M || n >= N) continue;
    int s = 0;
#pragma unroll
    for (int v = 0; v < NW; v++) s += part[v][i];
    const float sm = FUSED ? amax_scale<T>(top[i / 16]) : sx[m];
    y[m * N + n] = i8_out<T>(s, sm, sw[n], bias, n);
  }
}

// ---------------------------------------------------------------- tile GEMM
// BM rows of x by BN rows of W per workgroup, WM x WN wavefronts. K advances
// in steps of 128 bytes (whole cache lines of every row: steps of 64 in twice
// as many slots cost 52 instead of 42 us at 2048 x 4096 x 4096) through a ring of
// NS LDS slots filled by direct global-to-LDS copies, NS - 1 steps ahead. Inside
// a slot row r's 16-byte piece c sits at position c ^ (r / 2 & 7), so the 16
// rows that are read together touch all banks. W is the A operand, so a lane
// ends up with runs of four consecutive n of one row of y.
// Bound by the matrix units and the clock that their power leaves (1.65 to 1.9
// GHz): 8192 x 8192 x 4096 in 268 to 290 us, 1.9 to 2.05 Pop/s, 16384 x 8192 x
// 8192 in 990, 2.2; the library's product of 8192^3 reaches 2.04. Small tiles, whose
// wavefronts share less, are bound by LDS: 777 x 2050 x 8192 in 31 us, two parts of
// K, of which a third is the exchange of the parts (a ticket and a wait in place
// of the last to arrive, and 16-byte accesses, cost the same).
struct I8Args {
  const int8_t* xq;
  const float* sx;
  const int8_t* wq;
  const float* sw;
  const uint16_t* bias;
  uint16_t* y;
  int M, N, K;
  int ks, steps;    // K splits and K steps per split
  int* ws;          // split > 1: partial tiles [tile][split][BM * BN]
  unsigned* cnt;    //            arrival counters, zero between calls
};

typedef __attribute__((address_space(3))) void lds_ptr_t;

template <int N>
__device__ __forceinline__ void ring_wait() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));   // vmcnt(N) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Operand reads of one 32-byte K piece: TN pieces of W and TM of x, 32 rows
// (4096 bytes) apart in LDS.
//
// The reads are assembly, because before any LDS read of its own the compiler
// waits for every global-to-LDS copy in flight, which the ring is there to keep
// flying. Each block waits for what it reads. multiply_read() puts the reads
// of the next piece between the products of the present one, so that their
// wait at the block's end finds them done.
template <int R>
struct Operands {
  u32x4_t a[R], b[R];
};
#define QMM_LD(d, p, o) "ds_read_b128 %[" #d "], %[" #p "] offset:" #o "\n\t"
#define QMM_MM(i, j) "v_mfma_i32_32x32x32_i8 %[c" #i #j "], %[a" #i "], %[b" #j "], %[c" #i #j "]\n\t"
// The compiler does not see the products and leaves no cycles around them: it
// would give them 2 between a write of an operand and the product, with which
// each block therefore begins, and 12 before a result is read or moved. Where no
// further block follows (left is 0) the block itself ends with more than that;
// between blocks nothing but the next one touches the sums, which the build
// checks.
#define QMM_BEGIN "s_nop 1\n\t"
#define QMM_SETTLE                                                    \
  "s_cmp_lg_u32 %[left], 0\n\ts_cbranch_scc1 .Lgo%=\n\t"            \
  "s_nop 15\n\ts_nop 15\n.Lgo%=:"
__device__ __forceinline__ void read_operands(uint32_t pa, uint32_t pb, Operands<2>& n) {
  asm volatile(QMM_LD(na0, pa, 0) QMM_LD(nb0, pb, 0) QMM_LD(na1, pa, 4096) QMM_LD(nb1, pb, 4096)
               "s_waitcnt lgkmcnt(0)"
               : [na0] "=&v"(n.a[0]), [na1] "=&v"(n.a[1]), [nb0] "=&v"(n.b[0]), [nb1] "=&v"(n.b[1])
               : [pa] "v"(pa), [pb] "v"(pb)
               : "memory");
}
__device__ __forceinline__ void read_operands(uint32_t pa, uint32_t pb, Operands<4>& n) {
  asm volatile(QMM_LD(na0, pa, 0) QMM_LD(nb0, pb, 0) QMM_LD(na1, pa, 4096) QMM_LD(nb1, pb, 4096)
               QMM_LD(na2, pa, 8192) QMM_LD(nb2, pb, 8192) QMM_LD(na3, pa, 12288)
               QMM_LD(nb3, pb, 12288) "s_waitcnt lgkmcnt(0)"
               : [na0] "=&v"(n.a[0]), [na1] "=&v"(n.a[1]), [na2] "=&v"(n.a[2]), [na3] "=&v"(n.a[3]),
                 [nb0] "=&v"(n.b[0]), [nb1] "=&v"(n.b[1]), [nb2] "=&v"(n.b[2]), [nb3] "=&v"(n.b[3])
               : [pa] "v"(pa), [pb] "v"(pb)
               : "memory");
}
// LAST: of a step; `left` steps follow
#define QMM_MULTIPLY_READ(body, sums, next, operands)                                             \
  if constexpr (LAST)                                                                             \
    asm volatile(QMM_BEGIN body "s_waitcnt lgkmcnt(0)\n\t" QMM_SETTLE                            \
                 : sums, next : operands, [pa] "v"(pa), [pb] "v"(pb), [left] "s"(left)             \
                 : "memory", "scc");                                                              \
  else                                                                                            \
    asm volatile(QMM_BEGIN body "s_waitcnt lgkmcnt(0)"                                            \
                 : sums, next : operands, [pa] "v"(pa), [pb] "v"(pb) : "memory")
#define QMM_LIST(...) __VA_ARGS__
template <bool LAST>
__device__ __forceinline__ void multiply_read(int16v_t (&c)[2][2], const Operands<2>& u,
                                              uint32_t pa, uint32_t pb, Operands<2>& n, int left) {
  QMM_MULTIPLY_READ(
      QMM_MM(0, 0) QMM_LD(na0, pa, 0) QMM_LD(nb0, pb, 0)
      QMM_MM(0, 1) QMM_LD(na1, pa, 4096) QMM_LD(nb1, pb, 4096)
      QMM_MM(1, 0) QMM_MM(1, 1),
      QMM_LIST([c00] "+a"(c[0][0]), [c01] "+a"(c[0][1]), [c10] "+a"(c[1][0]), [c11] "+a"(c[1][1])),
      QMM_LIST([na0] "=&v"(n.a[0]), [na1] "=&v"(n.a[1]), [nb0] "=&v"(n.b[0]), [nb1] "=&v"(n.b[1])),
      QMM_LIST([a0] "v"(u.a[0]), [a1] "v"(u.a[1]), [b0] "v"(u.b[0]), [b1] "v"(u.b[1])));
}
template <bool LAST>
__device__ __forceinline__ void multiply_read(int16v_t (&c)[4][4], const Operands<4>& u,
                                              uint32_t pa, uint32_t pb, Operands<4>& n, int left) {
  QMM_MULTIPLY_READ(
      QMM_MM(0, 0) QMM_LD(na0, pa, 0) QMM_MM(0, 1) QMM_LD(nb0, pb, 0)
      QMM_MM(0, 2) QMM_LD(nb1, pb, 4096) QMM_MM(0, 3) QMM_LD(nb2, pb, 8192)
      QMM_MM(1, 0) QMM_LD(nb3, pb, 12288) QMM_MM(1, 1) QMM_LD(na1, pa, 4096)
      QMM_MM(1, 2) QMM_LD(na2, pa, 8192) QMM_MM(1, 3) QMM_LD(na3, pa, 12288)
      QMM_MM(2, 0) QMM_MM(2, 1) QMM_MM(2, 2) QMM_MM(2, 3)
      QMM_MM(3, 0) QMM_MM(3, 1) QMM_MM(3, 2) QMM_MM(3, 3),
      QMM_LIST([c00] "+a"(c[0][0]), [c01] "+a"(c[0][1]), [c02] "+a"(c[0][2]), [c03] "+a"(c[0][3]),
               [c10] "+a"(c[1][0]), [c11] "+a"(c[1][1]), [c12] "+a"(c[1][2]), [c13] "+a"(c[1][3]),
               [c20] "+a"(c[2][0]), [c21] "+a"(c[2][1]), [c22] "+a"(c[2][2]), [c23] "+a"(c[2][3]),
               [c30] "+a"(c[3][0]), [c31] "+a"(c[3][1]), [c32] "+a"(c[3][2]), [c33] "+a"(c[3][3])),
      QMM_LIST([na0] "=&v"(n.a[0]), [na1] "=&v"(n.a[1]), [na2] "=&v"(n.a[2]), [na3] "=&v"(n.a[3]),
               [nb0] "=&v"(n.b[0]), [nb1] "=&v"(n.b[1]), [nb2] "=&v"(n.b[2]), [nb3] "=&v"(n.b[3])),
      QMM_LIST([a0] "v"(u.a[0]), [a1] "v"(u.a[1]), [a2] "v"(u.a[2]), [a3] "v"(u.a[3]),
               [b0] "v"(u.b[0]), [b1] "v"(u.b[1]), [b2] "v"(u.b[2]), [b3] "v"(u.b[3])));
}
#undef QMM_LIST
#undef QMM_MULTIPLY_READ
#undef QMM_SETTLE
#undef QMM_BEGIN
#undef QMM_LD
#undef QMM_MM

template <class T, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(64 * WM * WN, BM * BN == 65536 || NS > 2 ? 1 : 2) void i8_tile_kernel(I8Args a) {
  constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32;   // 32x32 tiles per wavefront
  constexpr int kRows = BM + BN;
  constexpr int kLoads = kRows * 8 / kThreads;          // 16-byte pieces per thread and step
  constexpr int kSlot = kRows * 128;
  static_assert(BM * 8 % kThreads == 0 && BN * 8 % kThreads == 0 && TM == TN, "shape");
  __shared__ __attribute__((aligned(128))) uint8_t lds[NS * kSlot];
  const int tid = threadIdx.x, lane = tid % 64;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);   // uniform: scalar
  const int tiles_n = (a.N + BN - 1) / BN, tiles_m = (a.M + BM - 1) / BM;
  // The eight XCDs take workgroups in turn: give each a run of consecutive
  // tiles, walked in bands of 8 row tiles, so that the tiles an XCD works on
  // together share rows of x and W in its L2.
  const int tiles = tiles_m * tiles_n;
  int tile = blockIdx.x;   // of all splits
  {
    const int per = tiles * a.ks / 8, rem = tiles * a.ks % 8;
    const int xcd = tile % 8, i = tile / 8;
    tile = xcd * per + (xcd < rem ? xcd : rem) + i;
  }
  const int split = tile / tiles;
  tile %= tiles;
  constexpr int kBand = 8;
  const int band = tile / (kBand * tiles_n), first = band * kBand;
  const int high = tiles_m - first < kBand ? tiles_m - first : kBand;
  const int in = tile - first * tiles_n;
  const int64_t m0 = (int64_t)(first + in % high) * BM, n0 = (int64_t)(in / high) * BN;
  const int xrows = (int)(a.M - m0 < BM ? a.M - m0 : BM);
  const int wrows = (int)(a.N - n0 < BN ? a.N - n0 : BN);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.xq + m0 * a.K, (uint32_t)xrows * (uint32_t)a.K);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.wq + n0 * a.K, (uint32_t)wrows * (uint32_t)a.K);
  const int k_begin = split * a.steps * 128;
  const int total = (a.K + 127) / 128;
  const int steps = total - split * a.steps < a.steps ? total - split * a.steps : a.steps;

  // piece i of this thread: row (i * kThreads + tid) / 8 of [x rows | W rows];
  // pieces past K are out of every row's range and become zeros
  const int c = (tid % 8) ^ (tid / 16 % 8);
  auto copy = [&](int step, int at) QMM_INLINE {
    const uint32_t k = (uint32_t)(k_begin + step * 128 + c * 16);
    const uint32_t off = (tid / 8) * (uint32_t)a.K + (k < (uint32_t)a.K ? k : kOob);
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      constexpr int kX = BM * 8 / kThreads;
      const int row = (i < kX ? i : i - kX) * (kThreads / 8);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          i < kX ? rx : rw, (lds_ptr_t*)(lds + at + (i * kThreads + wave * 64) * 16), 16,
          (int)(off + (uint32_t)row * (uint32_t)a.K), 0, 0, 0);
    }
  };
  int16v_t acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; i++)
#pragma unroll
    for (int j = 0; j < TM; j++)
#pragma unroll
      for (int e = 0; e < 16; e++) acc[i][j][e] = 0;
  const int wm = wave % WM, wn = wave / WM;
  const int lr = lane % 32, lh = lane / 32;
  // LDS byte addresses of this lane's operand rows; the permuted position of
  // a K piece depends on the row's low bits only, which are the same for all
  // of a wavefront's tiles
  const uint32_t base = (uint32_t)(uintptr_t)(lds_ptr_t*)&lds[0];
  const uint32_t at_x = base + (uint32_t)(wm * TM * 32 + lr) * 128;
  const uint32_t at_w = base + (uint32_t)(BM + wn * TN * 32 + lr) * 128;
  auto piece = [&](int ks) QMM_INLINE { return (uint32_t)(((ks * 2 + lh) ^ (lr >> 1)) & 7) * 16; };
  // copies past the last step bring zeros, or the next split's data, unused
#pragma unroll
  for (int s = 0; s < NS - 1; s++) copy(s, s * kSlot);
  ring_wait<(NS - 2) * kLoads>();
  copy(NS - 1, (NS - 1) * kSlot);
  Operands<TN> u[2];
  read_operands(at_w + piece(0), at_x + piece(0), u[0]);
  int slot = 0;
  for (int step = 0; step < steps; step++) {
    auto next = [&](int ks) QMM_INLINE { return (uint32_t)slot + piece(ks); };
    multiply_read<false>(acc, u[0], at_w + next(1), at_x + next(1), u[1], 0);
    multiply_read<false>(acc, u[1], at_w + next(2), at_x + next(2), u[0], 0);
    multiply_read<false>(acc, u[0], at_w + next(3), at_x + next(3), u[1], 0);
    // every wavefront has read the last piece of this step's slot, and this
    // wavefront's copies of the next step have landed
    ring_wait<(NS - 2) * kLoads>();
    copy(step + NS, slot);
    slot = slot + kSlot < NS * kSlot ? slot + kSlot : 0;
    multiply_read<true>(acc, u[1], at_w + next(0), at_x + next(0), u[0], steps - 1 - step);
  }
  __builtin_amdgcn_s_waitcnt(0);   // no copy is left in flight when LDS is given up

  // acc[i][j][e]: n = n0 + 32 * (wn * TN + i) + 8 * (e / 4) + 4 * lh + e % 4,
  //               m = m0 + 32 * (wm * TM + j) + lr
  if (BM * BN < 65536 && a.ks > 1) {   // (many large tiles: never split)
    // every split leaves its tile in the workspace; the last to arrive adds
    // them (integer sums: the order does not matter). Relaxed agent-scope
    // accesses are coherent across the XCDs' L2 caches; the stores have
    // completed before the counter is touched.
    __shared__ unsigned last;
    const int64_t t = tile;
    int* mine = a.ws + (t * a.ks + split) * (BM * BN);
#pragma unroll
    for (int i = 0; i < TN; i++)
#pragma unroll
      for (int j = 0; j < TM; j++)
#pragma unroll
        for (int e = 0; e < 16; e++)
          __hip_atomic_store(mine + ((i * TM + j) * 16 + e) * kThreads + tid, acc[i][j][e],
                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (tid == 0)
      last = __builtin_amdgcn_atomic_inc32(a.cnt + t, (unsigned)(a.ks - 1), __ATOMIC_RELAXED,
                                           "agent") == (unsigned)(a.ks - 1);
    __syncthreads();
    if (!last) return;
    for (int s = 0; s < a.ks; s++) {
      if (s == split) continue;
      const int* other = a.ws + (t * a.ks + s) * (BM * BN);
#pragma unroll
      for (int i = 0; i < TN; i++)
#pragma unroll
        for (int j = 0; j < TM; j++)
#pragma unroll
          for (int e = 0; e < 16; e++)
            acc[i][j][e] += __hip_atomic_load(other + ((i * TM + j) * 16 + e) * kThreads + tid,
                                              __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  // Each wavefront turns its outputs round in LDS (its own TM * 32 rows of m
  // by TN * 32 columns of n; the copies have drained), so that y is written in
  // whole rows: 16-byte piece p of row r sits at p ^ r modulo the row's pieces.
  constexpr int kRow = TN * 64, kPieces = kRow / 16;   // bytes, pieces of a row
  __syncthreads();
  uint8_t* mine = &lds[0] + wave * (TM * 32 * kRow);
  auto at = [&](int r, int p) QMM_INLINE {
    return mine + r * kRow + ((p ^ (kPieces == 8 ? r >> 1 : r)) & (kPieces - 1)) * 16;
  };
  const int nw = wn * TN * 32, mw = wm * TM * 32;   // within the tile
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.sw + n0, (uint32_t)wrows * 4);
  float sm[TM];
#pragma unroll
  for (int j = 0; j < TM; j++) {
    const int64_t m = m0 + mw + 32 * j + lr;
    sm[j] = a.sx[m < a.M ? m : a.M - 1];
  }
#pragma unroll
  for (int i = 0; i < TN; i++) {
#pragma unroll
    for (int q = 0; q < 4; q++) {
      const int n = nw + 32 * i + 8 * q + 4 * lh;
      const float4_t sn = __builtin_bit_cast(
          float4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, n * 4, 0, 0));   // 0 past N
      float bn[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (a.bias)
#pragma unroll
        for (int e = 0; e < 4; e++)
          bn[e] = to_f32(T{}, a.bias[n0 + n + e < a.N ? n0 + n + e : a.N - 1]);
#pragma unroll
      for (int j = 0; j < TM; j++) {
        uint16_t o[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float s = sm[j] * sn[e], v = (float)acc[i][j][q * 4 + e];
          o[e] = from_f32(T{}, a.bias ? fmaf(s, v, bn[e]) : s * v);
        }
        *reinterpret_cast<uint2*>(at(32 * j + lr, i * 4 + q) + lh * 8) =
            make_uint2(o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16);
      }
    }
  }
  // rows of y start on 16, 4 or 2 bytes, as N allows
  const int64_t n = n0 + nw + lane % kPieces * 8;
  const int left = (int)(a.N - n < 8 ? a.N - n : 8);
#pragma unroll 4
  for (int r = lane / kPieces; r < TM * 32; r += 64 / kPieces) {
    const int64_t m = m0 + mw + r;
    if (m >= a.M || left <= 0) break;
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(at(r, lane % kPieces));
    uint16_t* yr = a.y + m * a.N + n;
    if (a.N % 8 == 0) {
      *reinterpret_cast<u32x4_t*>(yr) = w;
    } else if (a.N % 2 == 0) {
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (2 * e < left) reinterpret_cast<uint32_t*>(yr)[e] = w[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (e < left) yr[e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
    }
  }
}

}  // namespace

hipError_t launch_i8_quantize(int dt, const void* x, int64_t ldx, int64_t rows, int64_t K,
                              int8_t* xq, float* sx, hipStream_t st) {
  auto go = [&]<class T>() {
    const uint16_t* p = static_cast<const uint16_t*>(x);
    auto threads = [&]<int NT>() {   // per row: they hold 32 * NT elements
      constexpr int block = NT < 256 ? 256 : NT, per = block / NT;
      hipLaunchKernelGGL((i8_quantize_kernel<T, NT>), dim3((unsigned)((rows + per - 1) / per)),
                         dim3(block), 0, st, p, ldx, rows, (int)K, xq, sx);
    };
    // few rows: the latency counts (13 x 2048: 3.6 us with 256 threads, 4.8 with
    // 64; 13 x 8192: 4.2 with 512, 5.1 with 256); many: the fewer the better
    // (777 x 8192: 10.0 with 512, 9.8 with 256)
    if (rows <= 256 && K > 4096) threads.template operator()<512>();
    else if (rows <= 256 && K > 512) threads.template operator()<256>();
    else if (K <= 2048) threads.template operator()<64>();
    else if (K <= 4096) threads.template operator()<128>();
    else threads.template operator()<256>();
  };
  if (dt == 0) go.template operator()<F16>();
  else go.template operator()<BF16>();
  return hipGetLastError();
}

bool i8_fused(int64_t M, int64_t K) {
  return M <= 16 && M * K <= kGvChunks * 64 * kGvFused * 8;
}

hipError_t launch_i8_fused(int dt, const void* x, int64_t ldx, const int8_t* wq, const float* sw,
                           const void* bias, int64_t M, int64_t N, int64_t K, void* y,
                           hipStream_t st) {
  auto go = [&]<class T>() {
    hipLaunchKernelGGL((i8_gemv_kernel<T, 1, kGvFused, true>), dim3((unsigned)((N + 15) / 16)),
                       dim3(64 * kGvFused), (size_t)(M * (K + 16)), st,
                       static_cast<const uint16_t*>(x), ldx, nullptr, nullptr, wq, sw,
                       static_cast<const uint16_t*>(bias), static_cast<uint16_t*>(y), (int)M,
                       (int)N, (int)K);
  };
  if (dt == 0) go.template operator()<F16>();
  else go.template operator()<BF16>();
  return hipGetLastError();
}

// Whether the GEMV takes the product. Beyond kI8GemvMaxM rows it reads W once
// per 64 of them, which it pays 9 us per 2^30 multiply-adds for; the tile kernel's
// start, end and exchange of K parts cost more than that where there is little
// to do (512 x 512 x 2048: 7.5 us against 13.8; 300 x 1000 x 1504: 7.5 and 10.8;
// 1024 x 512 x 2048: 12.6 and 15.1; but 1024 x 1024 x 1024: 12.9 and 9.5, 2048 x
// 2048 x 128: 14.3 and 7.4).
static bool i8_few(int64_t M, int64_t N, int64_t K) {
  if (M <= kI8GemvMaxM) return true;
  if (M > 8192 || K <= 512) return false;
  return (M + 63) / 64 * 64 * N * K <= (int64_t)1 << (K >= 2048 ? 30 : 29);
}

I8Plan i8_plan(int64_t M, int64_t N, int64_t K) {
  I8Plan p{};
  if (i8_few(M, N, K)) {
    p.gemv = true;
    p.ks = 1;
    return p;
  }
  // A round of 256 large tiles takes 1.8 times as long as one of 512 small ones
  // (4096 x 4096 x 4096: 75 against 41 us per round), and small tiles end in
  // smaller steps: the large ones run where their rounds are full enough.
  auto tiles = [&](int64_t b) { return ((M + b - 1) / b) * ((N + b - 1) / b); };
  p.bm = p.bn = (tiles(256) + 255) / 256 * 9 * 512 <= tiles(128) * 5 ? 256 : 128;
  p.ks = 1;
  p.tiles = tiles(p.bm);
  const int64_t steps = (K + 127) / 128;
  // A few tiles: K over up to 4 workgroups, at least 8 steps each, while they
  // fit the chip once. (512 x 4096 x 4096: 24.3 / 21.0 / 25.7 us for 1 / 2 / 4
  // parts, 128 tiles; 128 x 4096 x 4096: 23.3 / 17.6 / 16.2 / 20.2 for 1 / 2 / 4
  // / 8, 32 tiles.)
  if (p.bm == 128)
    while (p.tiles * p.ks * 2 <= 256 && steps / (p.ks * 2) >= 8 && p.ks < (p.tiles <= 32 ? 4 : 2))
      p.ks *= 2;
  p.steps = (steps + p.ks - 1) / p.ks;
  p.ks = (steps + p.steps - 1) / p.steps;
  p.ws_bytes = p.ks > 1 ? p.tiles * p.ks * p.bm * p.bn * 4 : 0;
  return p;
}

hipError_t launch_i8_t(int dt, const int8_t* xq, const float* sx, const int8_t* wq,
                       const float* sw, const void* bias, int64_t M, int64_t N, int64_t K, void* y,
                       unsigned* cnt, int* ws, hipStream_t st) {
  const I8Plan p = i8_plan(M, N, K);
  const uint16_t* b = static_cast<const uint16_t*>(bias);
  uint16_t* yo = static_cast<uint16_t*>(y);
  auto go = [&]<class T>() {
    if (p.gemv) {
      const unsigned nb = (unsigned)((N + 15) / 16);
      auto waves = [&]<int MT, int NW>() {
        hipLaunchKernelGGL((i8_gemv_kernel<T, MT, NW, false>),
                           dim3(nb, (unsigned)((M + 16 * MT - 1) / (16 * MT))), dim3(64 * NW), 0,
                           st, nullptr, 0, xq, sx, wq, sw, b, yo, (int)M, (int)N, (int)K);
      };
      auto mv = [&]<int MT>() {
        // (13 x 8192 x 2048: 6.5 us with 4 wavefronts, 7.2 with 8; at K = 4096 four
        // would make two passes)
        if (K <= 2048) waves.template operator()<MT, 4>();
        else waves.template operator()<MT, 8>();
      };
      if (M <= 16) mv.template operator()<1>();
      else if (M <= 32) mv.template operator()<2>();
      else mv.template operator()<4>();
      return;
    }
    I8Args a{xq, sx, wq, sw, b, yo, (int)M, (int)N, (int)K, (int)p.ks, (int)p.steps, ws, cnt};
    const dim3 grid((unsigned)(p.tiles * p.ks));
    if (p.bm == 256)
      hipLaunchKernelGGL((i8_tile_kernel<T, 256, 256, 2, 2, 2>), grid, dim3(256), 0, st, a);
    else if (p.tiles * p.ks <= 256)   // one workgroup per CU: the LDS is its own
      hipLaunchKernelGGL((i8_tile_kernel<T, 128, 128, 2, 2, 4>), grid, dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((i8_tile_kernel<T, 128, 128, 2, 2, 2>), grid, dim3(256), 0, st, a);
  };
  if (dt == 0) go.template operator()<F16>();
  else go.template operator()<BF16>();
  return hipGetLastError();
}

}  // namespace qmm
