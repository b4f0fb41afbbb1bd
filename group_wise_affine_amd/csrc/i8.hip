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
// (rows longer than 32 * NT are read a second time).
template <class T, int NT>
__global__ __launch_bounds__(256) void i8_quantize_kernel(const uint16_t* __restrict__ x,
                                                          int64_t ldx, int64_t rows, int K,
                                                          int8_t* __restrict__ xq,
                                                          float* __restrict__ sx) {
  constexpr int kHold = 4;
  const int64_t row = (int64_t)blockIdx.x * (256 / NT) + threadIdx.x / NT;
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
    __shared__ uint32_t part[NT / 64];
    if (t % 64 == 0) part[t / 64] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 64; i++) top = part[i] > top ? part[i] : top;
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
// 16 rows of W and up to 16 * MT rows of x per workgroup; the eight
// wavefronts take 128-byte pieces of K in turn and their integer sums are
// added in LDS. v_mfma_i32_16x16x64_i8: A (W) row lane%16, B (x) column
// lane%16, both k = 16 * (lane/16) .. +16; D column lane%16, rows
// 4 * (lane/16) .. +4.
constexpr int kGvWaves = 8;
constexpr int kGvHold = 4;   // pieces in flight per wavefront

template <class T>
__device__ __forceinline__ uint16_t i8_out(int acc, float sx, float sw, const uint16_t* bias,
                                           int64_t n) {
  float v = sx * sw * (float)acc;
  if (bias) v = fmaf(sx * sw, (float)acc, to_f32(T{}, bias[n]));
  return from_f32(T{}, v);
}

template <class T, int MT>
__global__ __launch_bounds__(64 * kGvWaves) void i8_gemv_kernel(
    const int8_t* __restrict__ xq, const float* __restrict__ sx, const int8_t* __restrict__ wq,
    const float* __restrict__ sw, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y,
    int M, int N, int K) {
  __shared__ int part[kGvWaves][MT * 256];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int r = lane % 16, g = lane / 16;
  const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * 16 * MT;
  const int wrows = (int)(N - n0 < 16 ? N - n0 : 16);
  const int xrows = (int)(M - m0 < 16 * MT ? M - m0 : 16 * MT);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(wq + n0 * K, (uint32_t)wrows * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(xq + m0 * K, (uint32_t)xrows * (uint32_t)K);
  int4_t acc[MT];
#pragma unroll
  for (int i = 0; i < MT; i++) acc[i] = int4_t{0, 0, 0, 0};
  const uint32_t row = (uint32_t)r * (uint32_t)K;
  // out-of-range pieces and rows load zeros
  auto at = [&](uint32_t base, int k) QMM_INLINE { return k < K ? base + (uint32_t)k : kOob; };
  for (int k0 = wave * 128; k0 < K; k0 += kGvWaves * 128 * kGvHold) {
    u32x4_t w[kGvHold][2];
#pragma unroll
    for (int i = 0; i < kGvHold; i++)
#pragma unroll
      for (int h = 0; h < 2; h++)
        w[i][h] = __builtin_amdgcn_raw_buffer_load_b128(
            rw, (int)at(row, k0 + i * kGvWaves * 128 + h * 64 + g * 16), 0, 0);
#pragma unroll
    for (int i = 0; i < kGvHold; i++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int k = k0 + i * kGvWaves * 128 + h * 64 + g * 16;
#pragma unroll
        for (int t = 0; t < MT; t++) {
          const u32x4_t xv = __builtin_amdgcn_raw_buffer_load_b128(
              rx, (int)at(row + (uint32_t)(t * 16) * (uint32_t)K, k), 0, 0);
          acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(int4_t, w[i][h]),
                                                         __builtin_bit_cast(int4_t, xv), acc[t],
                                                         0, 0, 0);
        }
      }
  }
#pragma unroll
  for (int t = 0; t < MT; t++)
#pragma unroll
    for (int e = 0; e < 4; e++) part[wave][t * 256 + r * 16 + g * 4 + e] = acc[t][e];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * 256; i += 64 * kGvWaves) {
    const int64_t m = m0 + i / 16, n = n0 + i % 16;
    if (m >= M || n >= N) continue;
    int s = 0;
#pragma unroll
    for (int v = 0; v < kGvWaves; v++) s += part[v][i];
    y[m * N + n] = i8_out<T>(s, sx[m], sw[n], bias, n);
  }
}

// ---------------------------------------------------------------- tile GEMM
// BM rows of x by BN rows of W per workgroup, WM x WN wavefronts. K advances
// in steps of 128 bytes through a ring of NS LDS slots filled by direct
// global-to-LDS copies; inside a slot row r's 16-byte piece c sits at
// position c ^ (r & 7), so the eight rows that are read together touch all
// banks. W is the A operand, so a lane ends up with runs of four consecutive
// n of one row of y.
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

template <class T, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(64 * WM * WN) void i8_tile_kernel(I8Args a) {
  constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32;   // 32x32 tiles per wavefront
  constexpr int kRows = BM + BN;
  constexpr int kLoads = kRows * 8 / kThreads;          // 16-byte pieces per thread and step
  static_assert(BM * 8 % kThreads == 0 && BN * 8 % kThreads == 0, "copy shape");
  __shared__ __attribute__((aligned(128))) uint8_t lds[NS][kRows * 128];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int tiles_n = (a.N + BN - 1) / BN, tiles_m = (a.M + BM - 1) / BM;
  // The eight XCDs take workgroups in turn: give each a run of consecutive
  // tiles, walked in bands of 8 row tiles, so that the tiles an XCD works on
  // together share rows of x and W in its L2.
  int tile = blockIdx.x;
  {
    const int tiles = tiles_m * tiles_n, per = tiles / 8, rem = tiles % 8;
    const int xcd = tile % 8, i = tile / 8;
    tile = xcd * per + (xcd < rem ? xcd : rem) + i;
  }
  constexpr int kBand = 8;
  const int band = tile / (kBand * tiles_n), first = band * kBand;
  const int high = tiles_m - first < kBand ? tiles_m - first : kBand;
  const int in = tile - first * tiles_n;
  const int64_t m0 = (int64_t)(first + in % high) * BM, n0 = (int64_t)(in / high) * BN;
  const int split = blockIdx.y;
  const int xrows = (int)(a.M - m0 < BM ? a.M - m0 : BM);
  const int wrows = (int)(a.N - n0 < BN ? a.N - n0 : BN);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.xq + m0 * a.K, (uint32_t)xrows * (uint32_t)a.K);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.wq + n0 * a.K, (uint32_t)wrows * (uint32_t)a.K);
  const int k_begin = split * a.steps * 128;
  const int total = (a.K + 127) / 128;
  const int steps = total - split * a.steps < a.steps ? total - split * a.steps : a.steps;

  // piece i of this thread: row (i * kThreads + tid) / 8 of [x rows | W rows]
  const int c = (tid % 8) ^ (tid / 8 % 8);
  auto copy = [&](int step) QMM_INLINE {
    uint8_t* slot = lds[step % NS];
    const int k = k_begin + step * 128 + c * 16;
    const bool in_k = k < a.K;
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      constexpr int kX = BM * 8 / kThreads;
      const int rr = (i * kThreads + tid) / 8 - (i < kX ? 0 : BM);
      const uint32_t off = in_k ? (uint32_t)rr * (uint32_t)a.K + (uint32_t)k : kOob;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          i < kX ? rx : rw, (lds_ptr_t*)(slot + (i * kThreads + wave * 64) * 16), 16, (int)off, 0,
          0, 0);
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
#pragma unroll
  for (int s = 0; s < NS - 1; s++) copy(s);   // past the last step: zeros or unused
  for (int step = 0; step < steps; step++) {
    // the copies of the NS - 2 later steps may still be in flight
    ring_wait<(NS - 2) * kLoads>();
    copy(step + NS - 1);
    const uint8_t* slot = lds[step % NS];
#pragma unroll
    for (int ks = 0; ks < 4; ks++) {
      u32x4_t fa[TN], fb[TM];
      auto frag = [&](int row) QMM_INLINE {
        return *reinterpret_cast<const u32x4_t*>(slot + row * 128 +
                                                 (((ks * 2 + lh) ^ (row & 7)) * 16));
      };
#pragma unroll
      for (int j = 0; j < TM; j++) fb[j] = frag((wm * TM + j) * 32 + lr);
#pragma unroll
      for (int i = 0; i < TN; i++) fa[i] = frag(BM + (wn * TN + i) * 32 + lr);
#pragma unroll
      for (int i = 0; i < TN; i++)
#pragma unroll
        for (int j = 0; j < TM; j++)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
              __builtin_bit_cast(int4_t, fa[i]), __builtin_bit_cast(int4_t, fb[j]), acc[i][j], 0,
              0, 0);
    }
  }
  __builtin_amdgcn_s_waitcnt(0);   // no copy is left in flight when LDS is given up

  // acc[i][j][e]: n = n0 + 32 * (wn * TN + i) + 8 * (e / 4) + 4 * lh + e % 4,
  //               m = m0 + 32 * (wm * TM + j) + lr
  if (a.ks > 1) {
    // every split leaves its tile in the workspace; the last to arrive adds
    // them (integer sums: the order does not matter). Relaxed agent-scope
    // accesses are coherent across the XCDs' L2 caches; the stores have
    // completed before the counter is touched.
    __shared__ unsigned last;
    const int64_t t = blockIdx.x;
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
  const bool quad = a.N % 4 == 0;   // four outputs start on 8 bytes
#pragma unroll
  for (int j = 0; j < TM; j++) {
    const int64_t m = m0 + 32 * (wm * TM + j) + lr;
    if (m >= a.M) continue;
    const float sm = a.sx[m];
    uint16_t* yr = a.y + m * a.N;
#pragma unroll
    for (int i = 0; i < TN; i++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int64_t n = n0 + 32 * (wn * TN + i) + 8 * q + 4 * lh;
        if (quad) {
          if (n >= a.N) continue;
          uint16_t o[4];
#pragma unroll
          for (int e = 0; e < 4; e++)
            o[e] = i8_out<T>(acc[i][j][q * 4 + e], sm, a.sw[n + e], a.bias, n + e);
          *reinterpret_cast<uint2*>(yr + n) =
              make_uint2(o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16);
        } else {
#pragma unroll
          for (int e = 0; e < 4; e++)
            if (n + e < a.N) yr[n + e] = i8_out<T>(acc[i][j][q * 4 + e], sm, a.sw[n + e], a.bias, n + e);
        }
      }
  }
}

}  // namespace

hipError_t launch_i8_quantize(int dt, const void* x, int64_t ldx, int64_t rows, int64_t K,
                              int8_t* xq, float* sx, hipStream_t st) {
  auto go = [&]<class T>() {
    const uint16_t* p = static_cast<const uint16_t*>(x);
    if (K <= 2048)   // a wavefront holds the whole row
      hipLaunchKernelGGL((i8_quantize_kernel<T, 64>), dim3((unsigned)((rows + 3) / 4)), dim3(256),
                         0, st, p, ldx, rows, (int)K, xq, sx);
    else
      hipLaunchKernelGGL((i8_quantize_kernel<T, 256>), dim3((unsigned)rows), dim3(256), 0, st, p,
                         ldx, rows, (int)K, xq, sx);
  };
  if (dt == 0) go.template operator()<F16>();
  else go.template operator()<BF16>();
  return hipGetLastError();
}

I8Plan i8_plan(int64_t M, int64_t N, int64_t K) {
  I8Plan p{};
  if (M <= kI8GemvMaxM) {
    p.gemv = true;
    p.ks = 1;
    return p;
  }
  p.bm = p.bn = M > 1024 && N >= 256 ? 256 : 128;
  p.ks = 1;
  p.tiles = ((M + p.bm - 1) / p.bm) * ((N + p.bn - 1) / p.bn);
  const int64_t steps = (K + 127) / 128;
  if (p.bm == 128)   // a few tiles: K over several workgroups, at least 8 steps each
    while (p.tiles * p.ks * 2 <= 512 && steps / (p.ks * 2) >= 8 && p.ks < 16 &&
           p.tiles <= kScratchCounters)
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
      auto mv = [&]<int MT>() {
        hipLaunchKernelGGL((i8_gemv_kernel<T, MT>), dim3(nb, (unsigned)((M + 16 * MT - 1) / (16 * MT))),
                           dim3(64 * kGvWaves), 0, st, xq, sx, wq, sw, b, yo, (int)M, (int)N, (int)K);
      };
      if (M <= 16) mv.template operator()<1>();
      else mv.template operator()<2>();
      return;
    }
    I8Args a{xq, sx, wq, sw, b, yo, (int)M, (int)N, (int)K, (int)p.ks, (int)p.steps, ws, cnt};
    const dim3 grid((unsigned)p.tiles, (unsigned)p.ks);
    if (p.bm == 256)
      hipLaunchKernelGGL((i8_tile_kernel<T, 256, 256, 2, 4, 2>), grid, dim3(512), 0, st, a);
    else
      hipLaunchKernelGGL((i8_tile_kernel<T, 128, 128, 2, 2, 2>), grid, dim3(256), 0, st, a);
  };
  if (dt == 0) go.template operator()<F16>();
  else go.template operator()<BF16>();
  return hipGetLastError();
}

}  // namespace qmm
