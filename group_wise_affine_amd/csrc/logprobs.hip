// Log probabilities of given tokens, the entropy and the K most likely tokens of
// each row of logits, in one pass over the logits:
//
//   lse = ln sum exp x,  logprob = x[token] - lse,  entropy = lse - sum p x
//
// A lane holds the running maximum m of what it has seen, S = sum 2^y and
// Y = sum y 2^y with y = (x - m) log2 e, so that entropy = ln 2 (log2 S - Y / S)
// and a logarithm of a probability is (x - m) - ln 2 log2 S: no difference of large
// numbers.
//
// The K most likely (K <= 64) are a sorted list, one entry per lane of a
// wavefront: 64-bit keys of the value, ordered as an unsigned number, and the
// complement of the index, so that among equal values the lowest index comes
// first. Each wavefront keeps the list of what it has seen; elements above the
// list's K-th value go to a buffer, and 64 of them at a time are sorted and merged
// in (bitonic networks over the lanes). A first bound is the K-th largest of the
// lanes' maxima.
//
// A row's elements are cut over wavefronts, and over workgroups where there are
// few rows; their sums and lists are joined in their order.
#include "int8_common.hpp"
#include "kernels.hpp"

namespace qmm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWaves = 4;   // of a workgroup
constexpr int kAhead = 4;   // loads in flight per lane

struct LogprobArgs {
  const void* x;
  int64_t ld, M, V;
  const int32_t* tokens;
  int top, parts;
  float *logprob, *entropy;
  int32_t* ids;
  float* top_lp;
  float4* sums;      // [M][parts] m, S, Y
  uint64_t* lists;   // [M][parts][top]
};

// ------------------------------------------------------- lists over 64 lanes
// the value of the lane whose number differs in the bits X
template <int X>
__device__ __forceinline__ uint32_t across(uint32_t v) {
  auto dpp = [](uint32_t u, auto ctrl) QMM_INLINE {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, decltype(ctrl)::value, 0xf, 0xf, true);
  };
  if constexpr ((X & 32) != 0) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = threadIdx.x & 32 ? r[0] : r[1];
  }
  if constexpr ((X & 16) != 0) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = threadIdx.x & 16 ? r[0] : r[1];
  }
  constexpr int Y = X & 15;
  if constexpr (Y == 1) v = dpp(v, std::integral_constant<int, 0xb1>{});         // quads 1 0 3 2
  else if constexpr (Y == 2) v = dpp(v, std::integral_constant<int, 0x4e>{});    // quads 2 3 0 1
  else if constexpr (Y == 3) v = dpp(v, std::integral_constant<int, 0x1b>{});    // quads 3 2 1 0
  else if constexpr (Y == 7) v = dpp(v, std::integral_constant<int, 0x141>{});   // halves of a row reversed
  else if constexpr (Y == 15) v = dpp(v, std::integral_constant<int, 0x140>{});  // rows reversed
  else if constexpr (Y == 8) v = dpp(v, std::integral_constant<int, 0x128>{});   // rows turned by 8
  else if constexpr (Y == 4) v = across<3>(across<7>(v));
  else static_assert(Y == 0, "a pattern of the networks below");
  return v;
}
template <int X>
__device__ __forceinline__ uint64_t across(uint64_t v) {
  return across<X>((uint32_t)v) | (uint64_t)across<X>((uint32_t)(v >> 32)) << 32;
}
// lanes that differ in X: the one without the highest bit of X keeps the larger
template <int X, class K>
__device__ __forceinline__ K exchange(K v) {
  constexpr int kHigh = X >= 32 ? 32 : X >= 16 ? 16 : X >= 8 ? 8 : X >= 4 ? 4 : X >= 2 ? 2 : 1;
  const K p = across<X>(v);
  return (p > v) != ((threadIdx.x & kHigh) != 0) ? p : v;
}
// any 64 keys, largest first
template <class K>
__device__ __forceinline__ K sort64(K v) {
  v = exchange<1>(v);
  v = exchange<1>(exchange<3>(v));
  v = exchange<1>(exchange<2>(exchange<7>(v)));
  v = exchange<1>(exchange<2>(exchange<4>(exchange<15>(v))));
  v = exchange<1>(exchange<2>(exchange<4>(exchange<8>(exchange<31>(v)))));
  return exchange<1>(exchange<2>(exchange<4>(exchange<8>(exchange<16>(exchange<63>(v))))));
}
// the 64 largest of two sorted lists
__device__ __forceinline__ uint64_t merge64(uint64_t a, uint64_t b) {
  b = across<63>(b);
  a = a > b ? a : b;
  return exchange<1>(exchange<2>(exchange<4>(exchange<8>(exchange<16>(exchange<32>(a))))));
}

// numbers in the order of the floats (-0 as 0); 0 stands for none
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __builtin_bit_cast(float, o ^ ((uint32_t)((int32_t)~o >> 31) | 0x80000000u));
}

__device__ __forceinline__ float max_or_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// ------------------------------------------------------------- running sums
struct Sums {
  float m, s, y;   // m: NaN once a NaN was seen
};
// (differences first: a product with log2 e may leave the range)
__device__ __forceinline__ float shift(float from, float to) {
  return from == to ? 0.0f : (from - to) * kLog2e;
}
__device__ __forceinline__ Sums raised(Sums a, float m) {
  const float d = fmaxf(shift(a.m, m), -200.0f), f = __builtin_amdgcn_exp2f(d);
  return {m, a.s * f, f * fmaf(a.s, d, a.y)};
}
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
  const float m = max_or_nan(a.m, b.m);
  const Sums p = raised(a, m), q = raised(b, m);
  return {m, p.s + q.s, p.y + q.y};
}
template <int X>
__device__ __forceinline__ Sums join_across(const Sums& a) {
  const Sums b = {__builtin_bit_cast(float, across<X>(__builtin_bit_cast(uint32_t, a.m))),
                  __builtin_bit_cast(float, across<X>(__builtin_bit_cast(uint32_t, a.s))),
                  __builtin_bit_cast(float, across<X>(__builtin_bit_cast(uint32_t, a.y)))};
  return join(a, b);
}

template <class T>
__device__ __forceinline__ float element(const void* x, int64_t i) {
  return to_f32(T{}, static_cast<const typename T::word*>(x)[i]);
}
template <class T>
__device__ __forceinline__ void unpack(const u32x4_t& u, float* v) {
  if constexpr (__is_same(T, F32)) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t w = u[i];   // (of the element itself the compiler casts the last one)
      v[i] = __builtin_bit_cast(float, w);
    }
  } else {
    unpack8(T{}, make_uint4(u[0], u[1], u[2], u[3]), v);
  }
}

// What a wavefront knows of the elements it has seen, in order of their indexes
template <bool TOP>
struct Seen {
  Sums sums{-__builtin_inff(), 0.0f, 0.0f};
  uint64_t list = 0;
  float above = __builtin_nanf("");   // only larger ones may enter the list (NaN: any)
  int held = 0;                       // elements in the buffer, below 64
  uint64_t* buffer;                   // [128], the wavefront's
  int top;

  __device__ __forceinline__ void flush() {   // the first 64 of the buffer
    const int lane = threadIdx.x % 64;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const uint64_t k = lane < held ? buffer[lane] : 0, rest = buffer[64 + lane];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    buffer[lane] = rest;
    held = max(held - 64, 0);
    list = merge64(list, sort64(k));
    bound(__builtin_amdgcn_readlane((uint32_t)(list >> 32), top - 1));
  }
  // elements equal to the K-th of the list come later than it
  __device__ __forceinline__ void bound(uint32_t kth) {
    if (kth != 0) above = from_ordered(kth);
  }
  // N elements of each lane, the first with index i; none where !valid
  template <int N>
  __device__ __forceinline__ void take(const float* x, uint32_t i, bool valid) {
    float mx = x[0];
    if constexpr (N == 4) mx = max_or_nan(max_or_nan(x[0], x[1]), max_or_nan(x[2], x[3]));
    if constexpr (N == 8)
      mx = max_or_nan(max_or_nan(max_or_nan(max_or_nan(x[0], x[1]), x[2]), max_or_nan(max_or_nan(x[3], x[4]), x[5])),
                      max_or_nan(x[6], x[7]));
    if (__any(valid && !(mx <= sums.m))) {
      const float m = valid ? max_or_nan(sums.m, mx) : sums.m;
      sums = raised(sums, m);
    }
#pragma unroll
    for (int j = 0; j < N; j++) {
      // (what is -inf weighs nothing; 2^-200 is 0)
      const float y = valid ? fmaxf((x[j] - sums.m) * kLog2e, -200.0f) : -200.0f, e = __builtin_amdgcn_exp2f(y);
      sums.s += e;
      sums.y = fmaf(e, y, sums.y);
    }
    if constexpr (!TOP) return;
    if (__any(valid && !(mx <= above))) {
      const float at = above;   // (the same for all, in whatever order they come)
#pragma unroll
      for (int j = 0; j < N; j++) {
        const bool in = valid && !(x[j] <= at);
        const uint64_t who = __ballot(in);
        if (who != 0) {
          const int to = held + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
          if (in) buffer[to] = (uint64_t)ordered(x[j]) << 32 | (uint32_t)~(i + j);
          held += __builtin_popcountll(who);
          if (held >= 64) flush();
        }
      }
    }
  }
  // a first bound: the K-th largest of the lanes' maxima (0: a lane without any)
  __device__ __forceinline__ void first_bound(uint32_t largest) {
    const uint32_t kth = __builtin_amdgcn_readlane(sort64(largest), top - 1);
    if (kth == 0) return;
    // from it on: above the number before it, which is not -0
    above = from_ordered(kth - (kth == 0x80000000u ? 2 : 1));
  }
};

__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t row, const Sums& r, uint64_t list, float x_token) {
  const int lane = threadIdx.x % 64;
  const bool bad = !(r.m < __builtin_inff()), none = r.s == 0.0f;
  const float nan = __builtin_nanf(""), ls = none ? 0.0f : __log2f(r.s);
  auto lp = [&](float x) QMM_INLINE {
    return bad ? nan : x == -__builtin_inff() ? x : fmaf(-kLn2, ls, x - r.m);
  };
  if (lane == 0) {
    a.logprob[row] = lp(x_token);
    a.entropy[row] = bad ? nan : none ? 0.0f : fmaxf(kLn2 * (ls - r.y / r.s), 0.0f);
  }
  if (lane < a.top) {
    a.ids[row * a.top + lane] = bad ? -1 : (int32_t)~(uint32_t)list;
    a.top_lp[row * a.top + lane] = lp(from_ordered((uint32_t)(list >> 32)));
  }
}

// One part of a row. Wavefronts take steps of kAhead loads in turn.
template <class T, bool TOP>
__global__ __launch_bounds__(64 * kWaves) void logprobs_kernel(LogprobArgs a) {
  constexpr int N = __is_same(T, F32) ? 4 : 8;   // elements of a load
  constexpr int kStep = 64 * kAhead;             // loads of a wavefront's step
  __shared__ uint64_t buffers[kWaves][128];
  __shared__ Sums sums[kWaves];
  const int tid = threadIdx.x, lane = tid % 64;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int64_t row = blockIdx.x / a.parts;
  const int part = blockIdx.x % a.parts;
  using W = typename T::word;
  const W* x = static_cast<const W*>(a.x) + row * a.ld;
  // elements before the first whole 16 bytes, loads, elements after the last
  const int V = (int)a.V;
  const int head = min(V, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(W));
  const int loads = (V - head) / N, tail = V - head - loads * N;
  const u32x4_t* body = reinterpret_cast<const u32x4_t*>(x + head);
  const int steps = (loads + kStep - 1) / kStep, per = (steps + a.parts - 1) / a.parts;
  const int first = part * per, last = min(first + per, steps);
  const int32_t token = a.tokens[row];
  float x_token = -__builtin_inff();
  if (a.parts == 1 && token >= 0 && token < V) x_token = element<T>(x, token);

  Seen<TOP> seen;
  seen.buffer = buffers[wave];
  seen.top = a.top;
  if (part == 0 && wave == 0 && head > 0) {
    const float e = element<T>(x, lane < head ? lane : 0);
    seen.template take<1>(&e, lane, lane < head);
  }
  bool fresh = true;
  for (int step = first + wave; step < last; step += kWaves) {
    u32x4_t u[kAhead];
    const int at = step * kStep + lane;
    const bool whole = (step + 1) * kStep <= loads;
#pragma unroll
    for (int i = 0; i < kAhead; i++) u[i] = body[whole ? at + i * 64 : min(at + i * 64, loads - 1)];
    if (TOP && fresh) {
      fresh = false;
      uint32_t largest = 0;
#pragma unroll
      for (int i = 0; i < kAhead; i++) {
        float v[N];
        unpack<T>(u[i], v);
#pragma unroll
        for (int j = 0; j < N; j++) {
          const uint32_t o = ordered(v[j]);
          if (at + i * 64 < loads && o > largest) largest = o;
        }
      }
      if (!(seen.above == seen.above)) seen.first_bound(largest);
    }
#pragma unroll
    for (int i = 0; i < kAhead; i++) {
      float v[N];
      unpack<T>(u[i], v);
      seen.template take<N>(v, (uint32_t)(head + (at + i * 64) * N), whole || at + i * 64 < loads);
    }
  }
  if (part == a.parts - 1 && wave == kWaves - 1 && tail > 0) {
    const int i = V - tail + lane;
    const float e = element<T>(x, lane < tail ? i : 0);
    seen.template take<1>(&e, i, lane < tail);
  }
  if (TOP && seen.held > 0) seen.flush();
  Sums s = join_across<32>(join_across<16>(join_across<8>(join_across<4>(join_across<2>(join_across<1>(seen.sums))))));
  if (lane == 0) sums[wave] = s;
  if (TOP) buffers[wave][lane] = seen.list;
  __syncthreads();
  if (wave > 0) return;
  s = sums[0];
  uint64_t list = seen.list;
#pragma unroll
  for (int w = 1; w < kWaves; w++) {
    s = join(s, sums[w]);
    if (TOP) list = merge64(list, buffers[w][lane]);
  }
  if (a.parts == 1) {
    write_row(a, row, s, list, x_token);
  } else {
    if (lane == 0) a.sums[blockIdx.x] = make_float4(s.m, s.s, s.y, 0.0f);
    if (lane < a.top) a.lists[(int64_t)blockIdx.x * a.top + lane] = list;
  }
}

// Joins a row's parts.
constexpr int kJoinWaves = 8;
template <class T>
__global__ __launch_bounds__(64 * kJoinWaves) void logprobs_join_kernel(LogprobArgs a) {
  __shared__ uint64_t lists[kJoinWaves][64];
  __shared__ Sums sums[kJoinWaves];
  const int tid = threadIdx.x, lane = tid % 64;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int64_t row = blockIdx.x;
  const int32_t token = a.tokens[row];
  float x_token = -__builtin_inff();
  if (token >= 0 && token < a.V) x_token = element<T>(a.x, row * a.ld + token);
  Sums s{-__builtin_inff(), 0.0f, 0.0f};
  uint64_t list = 0;
  for (int p = wave; p < a.parts; p += kJoinWaves) {
    const float4 v = a.sums[row * a.parts + p];
    const uint64_t k = lane < a.top ? a.lists[(row * a.parts + p) * a.top + lane] : 0;
    s = join(s, Sums{v.x, v.y, v.z});
    if (a.top > 0) list = merge64(list, k);
  }
  if (lane == 0) sums[wave] = s;
  lists[wave][lane] = list;
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int w = 1; w < kJoinWaves; w++) {
    s = join(s, sums[w]);
    if (a.top > 0) list = merge64(list, lists[w][lane]);
  }
  write_row(a, row, s, list, x_token);
}

// Parts of a row: enough workgroups for the chip (1024), a step at least for each
// wavefront of a part, and no more parts than the join takes well.
int parts_of(int dt, int64_t M, int64_t V) {
  const int64_t step = (int64_t)64 * kAhead * (dt == 2 ? 4 : 8);
  int64_t p = (1024 + M - 1) / M, most = V / (step * kWaves);
  p = p < most ? p : most;
  return (int)(p < 1 ? 1 : p > 64 ? 64 : p);
}

}  // namespace

int64_t logprobs_work(int dt, int64_t M, int64_t V, int64_t top) {
  const int64_t p = parts_of(dt, M, V);
  return p > 1 ? M * p * (16 + 8 * top) : 0;
}

hipError_t launch_logprobs(int dt, const void* x, int64_t ld, int64_t M, int64_t V,
                           const int32_t* tokens, int64_t top, float* logprob, float* entropy,
                           int32_t* ids, float* top_lp, void* work, hipStream_t st) {
  LogprobArgs a{x, ld, M, V, tokens, (int)top, parts_of(dt, M, V), logprob, entropy, ids, top_lp,
                static_cast<float4*>(work), nullptr};
  a.lists = reinterpret_cast<uint64_t*>(a.sums + M * a.parts);
  auto go = [&]<class T>() {
    const dim3 grid((unsigned)(M * a.parts));
    if (top > 0) hipLaunchKernelGGL((logprobs_kernel<T, true>), grid, dim3(64 * kWaves), 0, st, a);
    else hipLaunchKernelGGL((logprobs_kernel<T, false>), grid, dim3(64 * kWaves), 0, st, a);
    if (a.parts > 1)
      hipLaunchKernelGGL((logprobs_join_kernel<T>), dim3((unsigned)M), dim3(64 * kJoinWaves), 0, st, a);
  };
  if (dt == 0) go.template operator()<F16>();
  else if (dt == 1) go.template operator()<BF16>();
  else go.template operator()<F32>();
  return hipGetLastError();
}

}  // namespace qmm
