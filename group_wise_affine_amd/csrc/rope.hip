// Norm and rotation of queries and keys, head by head, in one pass:
//
//   y = x * rsqrt(sum x^2 / D + eps) * w          (where there is a weight)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position * freq[i]
//
// for the i-th pair of a head's first R elements, (i, i + R/2) or (2i, 2i + 1);
// the elements past R keep their places. One rounding, at the end.
//
// The angle is a product in 64 bits, reduced there to a fraction of a turn (in 32
// bits a position of 10^5 leaves an error of 0.004), its sine and cosine are
// polynomials in 32 bits.
//
// Bound: memory (8192 tokens, 40 heads of 128, bf16: 168 MB in 34 to 37 us, 4.5 to 4.9
// TB/s), for few tokens the launch (1 token: 2.5 us; a call of it from Python takes the
// host 6).
#include "int8_common.hpp"
#include "kernels.hpp"

namespace qmm {
namespace {

struct RopeArgs {
  const uint16_t *q, *k, *wq, *wk;   // weights or null
  int64_t ldq, ldk;
  uint16_t *qo, *ko;
  int64_t ldqo, ldko;
  const int32_t* pos;
  const float* freq;
  int64_t T;
  int hq, heads, D, half;   // query heads, all heads; half = R / 2
  float eps;
};

// sine and cosine of 2 pi r, |r| <= 1/2: to the nearest quarter turn, then the
// Taylor series on [-pi/4, pi/4] to the powers 9 and 10 (2e-9 and 2e-10 off)
__device__ __forceinline__ void turn(float r, float& s, float& c) {
  const float n = __builtin_rintf(4.0f * r);
  const float t = fmaf(n, -0.25f, r) * 6.283185307179586f, z = t * t;
  const float ps = fmaf(z * t, fmaf(z, fmaf(z, fmaf(z, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), t);
  const float pc = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720),
                                             1.0f / 24), -0.5f), 1.0f);
  const int i = (int)n & 3;
  const float a = i & 1 ? pc : ps, b = i & 1 ? ps : pc;
  s = i & 2 ? -a : a;
  c = (i + 1) & 2 ? -b : b;
}

// A lane's eight elements of a row are four pairs: two runs of four, half a
// rotation (or half of what is not turned) apart, or one run of eight.
template <bool NEIGHBOURS>
__device__ __forceinline__ uint4 load_pairs(const uint16_t* p, int a, int b) {
  if constexpr (NEIGHBOURS) return *reinterpret_cast<const uint4*>(p + a);
  const uint2 u = *reinterpret_cast<const uint2*>(p + a), v = *reinterpret_cast<const uint2*>(p + b);
  return make_uint4(u.x, u.y, v.x, v.y);
}
template <bool NEIGHBOURS>
__device__ __forceinline__ void store_pairs(uint16_t* p, int a, int b, const uint4& u) {
  if constexpr (NEIGHBOURS) {
    *reinterpret_cast<uint4*>(p + a) = u;
  } else {
    *reinterpret_cast<uint2*>(p + a) = make_uint2(u.x, u.y);
    *reinterpret_cast<uint2*>(p + b) = make_uint2(u.z, u.w);
  }
}
// where the i-th pair's two elements stand among a lane's eight
template <bool NEIGHBOURS>
constexpr int first_of(int i) { return NEIGHBOURS ? 2 * i : i; }
template <bool NEIGHBOURS>
constexpr int second_of(int i) { return NEIGHBOURS ? 2 * i + 1 : i + 4; }

// A wavefront takes one token and PASSES times 64 / L of its heads, L lanes to a
// head (the power of two from D / 8 on): the sines are computed once for all of
// them, and every load is asked for before the first is used.
template <class T, bool NEIGHBOURS, int L, int PASSES>
__global__ __launch_bounds__(256) void qk_rope_kernel(RopeArgs a) {
  constexpr int kRows = 64 / L;
  const int lane = threadIdx.x % 64, li = lane % L;
  const int blocks = (a.heads + kRows * PASSES - 1) / (kRows * PASSES);
  // (T * heads < 2^31)
  const uint32_t unit = (blockIdx.y * gridDim.x + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t t = unit / (uint32_t)blocks;
  if (t >= a.T) return;
  const int h0 = (int)(unit % (uint32_t)blocks) * (kRows * PASSES) + lane / L;
  const bool mine = li * 8 < a.D;
  const int turned = a.half / 4;   // lanes of a row whose elements turn
  const bool turns = li < turned;
  int e0, e1;
  if constexpr (NEIGHBOURS) {
    e0 = e1 = li * 8;
  } else {
    const int rest = 2 * a.half;   // first element that does not turn
    e0 = turns ? li * 4 : rest + (li - turned) * 4;
    e1 = e0 + (turns ? a.half : (a.D - rest) / 2);
  }
  uint4 u[PASSES], w[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; i++) {
    const int h = h0 + i * kRows;
    if (!mine || h >= a.heads) continue;
    const bool key = h >= a.hq;
    const uint16_t* p = key ? a.k + t * a.ldk + (int64_t)(h - a.hq) * a.D : a.q + t * a.ldq + (int64_t)h * a.D;
    u[i] = load_pairs<NEIGHBOURS>(p, e0, e1);
    const uint16_t* wp = key ? a.wk : a.wq;
    if (wp) w[i] = load_pairs<NEIGHBOURS>(wp, e0, e1);
  }
  float s[4] = {0, 0, 0, 0}, c[4] = {1, 1, 1, 1};
  if (turns) {
    const float4 f = *reinterpret_cast<const float4*>(a.freq + li * 4);
    const float fs[4] = {f.x, f.y, f.z, f.w};
    const double pos = a.pos[t] * 0.15915494309189535;   // 1 / (2 pi)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const double r = pos * (double)fs[i];
      turn((float)(r - __builtin_rint(r)), s[i], c[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < PASSES; i++) {
    const int h = h0 + i * kRows;
    const bool key = h >= a.hq, here = mine && h < a.heads;
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (here) unpack8(T{}, u[i], x);
    if (here && (key ? a.wk : a.wq) == nullptr) {
      // (no norm)
    } else {
      auto squares = [&]() QMM_INLINE {
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++) ss = fmaf(x[j], x[j], ss);
#pragma unroll
        for (int o = L / 2; o >= 1; o >>= 1) ss += __shfl_xor(ss, o);
        return ss;
      };
      float ss = squares(), eps = a.eps;
      if constexpr (__is_same(T, BF16)) {
        // squares that leave the range of 32 bits: the row by a power of two (where eps
        // outweighs small ones, they need no bits). Up by 2^92: the square of 2^-133 is then
        // far from the subnormal numbers, of which the reciprocal root would be infinite,
        // and 2^-90 or an eps of 2^-60 still finite
        const float f = h >= a.heads ? 1.0f : ss > 0x1p100f ? 0x1p-70f : ss < 0x1p-90f && eps < 0x1p-60f ? 0x1p92f : 1.0f;
        if (__any(f != 1.0f)) {
#pragma unroll
          for (int j = 0; j < 8; j++) x[j] *= f;
          ss = squares();
          eps = eps * f * f;   // (f * f leaves the range)
        }
      }
      const float inv = __builtin_amdgcn_rsqf(ss / (float)a.D + eps);
      if (here) {
        float g[8];
        unpack8(T{}, w[i], g);
#pragma unroll
        for (int j = 0; j < 8; j++) x[j] = x[j] * inv * g[j];
      }
    }
    if (!here) continue;
    float y[8];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const float p = x[first_of<NEIGHBOURS>(j)], q = x[second_of<NEIGHBOURS>(j)];
      y[first_of<NEIGHBOURS>(j)] = turns ? fmaf(p, c[j], -(q * s[j])) : p;
      y[second_of<NEIGHBOURS>(j)] = turns ? fmaf(q, c[j], p * s[j]) : q;
    }
    uint16_t* to = key ? a.ko + t * a.ldko + (int64_t)(h - a.hq) * a.D : a.qo + t * a.ldqo + (int64_t)h * a.D;
    store_pairs<NEIGHBOURS>(to, e0, e1, pack8(T{}, y));
  }
}

}  // namespace

hipError_t launch_qk_norm_rope(int dt, const void* q, int64_t ldq, const void* k, int64_t ldk,
                               int64_t T, int64_t hq, int64_t hk, int64_t D, const int32_t* pos,
                               const float* freq, int64_t rot, bool neighbours, const void* wq,
                               const void* wk, float eps, void* qo, int64_t ldqo, void* ko,
                               int64_t ldko, hipStream_t st) {
  RopeArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
             static_cast<const uint16_t*>(wq), static_cast<const uint16_t*>(wk), ldq, ldk,
             static_cast<uint16_t*>(qo), static_cast<uint16_t*>(ko), ldqo, ldko, pos, freq, T,
             (int)hq, (int)(hq + hk), (int)D, (int)(rot / 2), eps};
  // (an f16 head that is not all zeros has a mean square above 2^-58, and of zeros the result
  // is 0 for any eps but 0: a subnormal one, of which the reciprocal root would be infinite,
  // need not be met)
  if (dt == 0 && eps > 0.0f && eps < 0x1p-126f) a.eps = 0x1p-126f;
  auto go = [&]<class T_, bool N, int L, int PASSES>() {
    const int64_t per = 64 / L * PASSES, units = T * ((a.heads + per - 1) / per), groups = (units + 3) / 4;
    // (a row of a grid is short of 2^32 threads)
    const unsigned wide = (unsigned)(groups < (1 << 20) ? groups : 1 << 20);
    hipLaunchKernelGGL((qk_rope_kernel<T_, N, L, PASSES>), dim3(wide, (unsigned)((groups + wide - 1) / wide)),
                       dim3(256), 0, st, a);
  };
  auto passes = [&]<class T_, bool N, int L>() {
    // wavefronts of one pass: the chip holds 8192. (Rows of 40 heads of 128 in bf16, 1, 2
    // and 4 passes: 512 tokens, 5120 wavefronts, 5.2, 5.5 and 6.5 us; 1024: 8.1, 7.4 and
    // 8.2; 8192: 45.4, 37.0 and 35.4.)
    const int64_t waves = T * ((a.heads + 64 / L - 1) / (64 / L));
    if (waves <= 6144) go.template operator()<T_, N, L, 1>();
    else if (waves <= 32768) go.template operator()<T_, N, L, 2>();
    else go.template operator()<T_, N, L, 4>();
  };
  auto lanes = [&]<class T_, bool N>() {
    if (D <= 64) passes.template operator()<T_, N, 8>();
    else if (D <= 128) passes.template operator()<T_, N, 16>();
    else if (D <= 256) passes.template operator()<T_, N, 32>();
    else passes.template operator()<T_, N, 64>();
  };
  auto pairs = [&]<class T_>() {
    if (neighbours) lanes.template operator()<T_, true>();
    else lanes.template operator()<T_, false>();
  };
  if (dt == 0) pairs.template operator()<F16>();
  else pairs.template operator()<BF16>();
  return hipGetLastError();
}

}  // namespace qmm
