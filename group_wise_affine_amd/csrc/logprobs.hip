// Log probabilities of given tokens, the entropy and the K most likely tokens of
// each row of logits, in one pass over the logits:
//
//   lse = ln sum exp x,  logprob = x[token] - lse,  entropy = lse - sum p x
//
// A lane holds the running maximum m of what it has seen, S = sum 2^y and
// Y = sum y 2^y with y = (x - m) log2 e, so that entropy = ln 2 (log2 S - Y / S)
// and a logarithm of a probability is ln 2 (y - log2 S): no difference of large
// numbers.
//
// The K most likely (K <= 64) are a sorted list, one entry per lane of a
// wavefront: 64-bit keys of the value, ordered as an unsigned number, and the
// complement of the index, so that among equal values the lowest index comes
// first. Each wavefront keeps the list of what it has seen; elements above the
// list's K-th value go to a buffer, and 64 of them at a time are sorted and merged
// in (bitonic networks over the lanes). A first bound is the K-th largest of the
// lanes' maxima; of the elements that equal it only the first ones are taken, so
// that a plateau (a mask of the type's lowest value) does not fill the buffer.
//
// A row's elements are cut over wavefronts, and over workgroups where there are
// few rows; their sums and lists are joined in their order.
#include "int8_common.hpp"
#include "kernels.hpp"

namespace qmm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kAhead = 4;   // loads in flight per lane
constexpr int kBuffer = 32 + 512;   // keys of a wavefront's buffer: what is left, and a load of each lane

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
// m: the largest, NaN once a NaN was seen; s and y relative to m log2 e. Below kBig that is
// c = fl(m log2 e), so that an element costs one product and addition; the difference
// y - (x - m) log2 e, half an ulp of c, is at most 2^-8 there, and the same in every term.
// From kBig on (masks of -1e9 or of a type's lowest value, of f16 none) it would not stay
// small (440 for -1e10), and differences come before the product.
struct Sums {
  float m, s, y;
};
constexpr float kBig = 65536.0f;
// y of an element
__device__ __forceinline__ float power(float x, float m) {
  const float c = m * kLog2e;
  return fabsf(m) < kBig ? fmaf(x, kLog2e, -c) : (x - m) * kLog2e;
}
// what y changes by when m goes from `from` to `to`: each one's reference is the rounded
// product below kBig, the exact one from there on
__device__ __forceinline__ float shift(float from, float to) {
#pragma clang fp contract(off)
  const float a = from * kLog2e, b = to * kLog2e;   // (fused, the two would not be those that were taken)
  const bool ra = fabsf(from) < kBig, rb = fabsf(to) < kBig;
  if (from == to) return 0.0f;
  if (ra && rb) return a - b;
  return ra ? fmaf(-to, kLog2e, a) : rb ? fmaf(from, kLog2e, -b) : (from - to) * kLog2e;
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
// the lanes' sums joined: the largest first, so that each lane's are scaled once
template <class F>
__device__ __forceinline__ float fold(float v, F f) {
  auto step = [&]<int X>() QMM_INLINE {
    v = f(v, __builtin_bit_cast(float, across<X>(__builtin_bit_cast(uint32_t, v))));
  };
  step.template operator()<1>();
  step.template operator()<2>();
  step.template operator()<7>();
  step.template operator()<15>();
  step.template operator()<16>();
  step.template operator()<32>();
  return v;
}
__device__ __forceinline__ Sums join_lanes(const Sums& a) {
  const Sums b = raised(a, fold(a.m, max_or_nan));
  auto add = [](float x, float y) QMM_INLINE { return x + y; };
  return {b.m, fold(b.s, add), fold(b.y, add)};
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
  bool big = false;                   // some lane's largest is kBig or more
  uint64_t list = 0;                  // (-inf never enters: write_row() puts it in where it is needed)
  float above = -__builtin_inff();    // only larger ones may enter the list,
  float from = 0.0f;                  // and while `open` the first ones that equal this, the next number
  bool open = false;
  int ties = 0;                       // of those seen
  int held = 0;                       // elements in the buffer, below 32 between loads
  uint64_t* buffer;                   // [kBuffer], the wavefront's
  int top;

  __device__ __forceinline__ void flush() {   // the last 64 of the buffer
    const int lane = threadIdx.x % 64, first = max(held - 64, 0);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const uint64_t k = sort64(first + lane < held ? buffer[first + lane] : 0);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    held = first;
    list = merge64(list, k);
    const uint32_t kth = __builtin_amdgcn_readlane((uint32_t)(list >> 32), top - 1);
    if (kth != 0) {   // (what equals it and comes with a later load comes later than it)
      above = from_ordered(kth);
      open = false;
    }
  }
  // A first bound: the K-th largest of the lanes' maxima, bit by bit from the top: the
  // largest number that K of them reach. The BITS high bits tell the type's values
  // apart; those below are a negative number's ones.
  template <int BITS>
  __device__ __forceinline__ void first_bound(float largest) {
    const uint32_t mine = ordered(largest);
    uint32_t kth = 0;
#pragma unroll
    for (int i = 31; i >= 32 - BITS; i--) {
      const uint32_t next = kth | 1u << i;
      if (__builtin_popcountll(__ballot(mine >= next)) >= top) kth = next;
    }
    if constexpr (BITS < 32)
      if (kth < 0x80000000u) kth |= (1u << (32 - BITS)) - 1;
    if (kth <= 0x007fffffu) return;   // -inf
    from = from_ordered(kth);
    above = from_ordered(kth - (kth == 0x80000000u ? 2 : 1));   // (the number before 0 is not -0)
    open = true;
  }
  // the sums of N elements of each lane, -inf where there is none; whether some may
  // enter the list
  template <int N>
  __device__ __forceinline__ bool take(const float* x) {
    float mx = max_or_nan(max_or_nan(max_or_nan(x[0], x[1]), x[2]), x[3]);
    if constexpr (N == 8) mx = max_or_nan(max_or_nan(mx, max_or_nan(max_or_nan(x[4], x[5]), x[6])), x[7]);
    if (__any(!(mx <= sums.m))) {
      sums = raised(sums, max_or_nan(sums.m, mx));
      big = __any(fabsf(sums.m) >= kBig && sums.m > -__builtin_inff());
    }
    // A load's terms are added up first: one by one, those of a plateau would be rounded the
    // same way at each step of a long row (1.4e-5 off in a sum of 1000, 2.7e-6 so).
    // (what is -inf weighs nothing; 2^-200 is 0)
    float s = 0.0f, t = 0.0f;
    auto add = [&](float p) QMM_INLINE {
      const float y = fmaxf(p, -200.0f), e = __builtin_amdgcn_exp2f(y);
      s += e;
      t = fmaf(e, y, t);
    };
    if (!big) {
      const float c = -sums.m * kLog2e;
#pragma unroll
      for (int j = 0; j < N; j++) add(fmaf(x[j], kLog2e, c));
    } else {
#pragma unroll
      for (int j = 0; j < N; j++) add(power(x[j], sums.m));
    }
    sums.s += s;
    sums.y += t;
    return TOP && __any(mx > above);
  }
  // the first element's index is i
  template <int N>
  __device__ __forceinline__ void push(const float* x, uint32_t i) {
    auto enter = [&](int j, bool in) QMM_INLINE {
      const uint64_t who = __ballot(in);
      if (who == 0) return;
      if (in) buffer[held + below(who)] = (uint64_t)ordered(x[j]) << 32 | (uint32_t)~(i + j);
      held += __builtin_popcountll(who);
    };
    if (!open) {
#pragma unroll
      for (int j = 0; j < N; j++) enter(j, x[j] > above);
    } else {
      // of many equal ones the first lanes' are enough
      bool any = false;
#pragma unroll
      for (int j = 0; j < N; j++) any |= x[j] == from;
      const bool mine = (int)below(__ballot(any)) < top;
#pragma unroll
      for (int j = 0; j < N; j++) {
        ties += __builtin_popcountll(__ballot(mine && x[j] == from));
        enter(j, x[j] > above && (mine || x[j] != from));
      }
      if (ties >= top) {
        above = from;
        open = false;
      }
    }
    // (an old bound lets more in than a new one costs: 32 rather than 64)
    while (held >= 32) flush();
  }
  static __device__ __forceinline__ uint32_t below(uint64_t who) {   // how many of them are lanes before this one
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
  }
};

template <class T>
__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t row, const Sums& r, uint64_t list, float x_token) {
  const int lane = threadIdx.x % 64;
  const float inf = __builtin_inff(), nan = __builtin_nanf("");
  const bool bad = !(r.m < inf), none = r.s == 0.0f;
  const float ls = none ? 0.0f : __log2f(r.s);
  // (of a mask near the type's lowest value only the difference stays in range: times log2 e
  // it need not, and what the sum adds, below 30, is no bit of it)
  auto lp = [&](float x) QMM_INLINE {
    const float d = x - r.m;
    return bad ? nan : x == -inf ? x : d < -1e30f ? d : kLn2 * (power(x, r.m) - ls);
  };
  if (lane == 0) {
    a.logprob[row] = lp(x_token);
    a.entropy[row] = bad ? nan : none ? 0.0f : max_or_nan(kLn2 * (ls - r.y / r.s), 0.0f);
  }
  const bool there = lane < a.top && (bad || list != 0);
  if (there) {
    a.ids[row * a.top + lane] = bad ? -1 : (int32_t)~(uint32_t)list;
    a.top_lp[row * a.top + lane] = lp(from_ordered((uint32_t)(list >> 32)));
  }
  // fewer than K that can be: the first of the others, which are as many as it takes
  int have = __builtin_popcountll(__ballot(there));
  for (int i = lane; have < a.top && __any(i < a.V); i += 64) {
    const bool in = i < a.V && element<T>(a.x, row * a.ld + i) == -inf;
    const uint64_t who = __ballot(in);
    const int to = have + (int)Seen<true>::below(who);
    if (in && to < a.top) {
      a.ids[row * a.top + to] = i;
      a.top_lp[row * a.top + to] = -inf;
    }
    have += __builtin_popcountll(who);
  }
}

// Joins W wavefronts' sums and lists in pairs; the first one has the result. Lists
// go through lists, `stride` keys per wavefront.
template <int W, bool TOP>
__device__ __forceinline__ void join_waves(Sums& s, uint64_t& list, Sums* sums, uint64_t* lists, int stride, int wave) {
  const int lane = threadIdx.x % 64;
#pragma unroll
  for (int d = W / 2; d >= 1; d >>= 1) {
    if (wave >= d && wave < 2 * d) {
      if (lane == 0) sums[wave] = s;
      if (TOP) lists[wave * stride + lane] = list;
    }
    __syncthreads();
    if (wave < d) {
      s = join(s, sums[wave + d]);
      if (TOP) list = merge64(list, lists[(wave + d) * stride + lane]);
    }
  }
}

// One part of a row; each wavefront takes a run of loads, kAhead of them in flight.
template <class T, bool TOP, int kWaves>
__global__ __launch_bounds__(64 * kWaves, 8) void logprobs_kernel(LogprobArgs a) {
  constexpr int N = __is_same(T, F32) ? 4 : 8;   // elements of a load
  __shared__ uint64_t buffers[TOP ? kWaves * kBuffer : 1];
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
  // the part's loads; the wavefronts take 64 of them in turn
  const int run = ((loads + a.parts - 1) / a.parts + 63) / 64 * 64;
  const int first = min(part * run, loads), last = min(first + run, loads);
  const int turns = max(((last - first + 63) / 64 - wave + kWaves - 1) / kWaves, 0);
  const int batches = (turns + kAhead - 1) / kAhead;
  const bool has_head = part == 0 && wave == 0 && head > 0;
  const bool has_tail = part == a.parts - 1 && wave == kWaves - 1 && tail > 0;
  const int32_t token = a.tokens[row];
  float x_token = -__builtin_inff();
  if (a.parts == 1 && token >= 0 && token < V) x_token = element<T>(x, token);

  constexpr uint32_t kNone = __is_same(T, F16) ? 0xfc00fc00u : __is_same(T, BF16) ? 0xff80ff80u : 0xff800000u;   // -inf
  const u32x4_t none = {kNone, kNone, kNone, kNone};
  Seen<TOP> seen;
  seen.buffer = buffers + wave * kBuffer;
  seen.top = a.top;
  // the elements before, the loads, the elements after, in one loop: the code that
  // enters elements into the list stands once (as often as there are loads ahead, it
  // does not fit the instruction cache: 167 us for 2048 rows of 128000, 131 so)
  for (int b = has_head ? -1 : 0; b < batches + (has_tail ? 1 : 0); b++) {
    u32x4_t u[kAhead];
    int count = 1, at = 0, next = 0;   // loads, the first one's first element, from one to the next
    if (b >= 0 && b < batches) {
      constexpr int kTurn = 64 * kWaves;
      const int from = first + b * (kTurn * kAhead) + wave * 64 + lane;
      count = min(turns - b * kAhead, kAhead);
      at = head + from * N;
      next = kTurn * N;
#pragma unroll
      for (int i = 0; i < kAhead; i++)
        if (i < count) u[i] = body[min(from + i * kTurn, last - 1)];
      if (b == batches - 1)
#pragma unroll
        for (int i = 0; i < kAhead; i++)
          if (from + i * kTurn >= last) u[i] = none;
      if (TOP && b == 0) {
        float largest = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < kAhead; i++)
          if (i < count) {
            float v[N];
            unpack<T>(u[i], v);
#pragma unroll
            for (int j = 0; j < N; j += 2) largest = max_or_nan(max_or_nan(largest, v[j]), v[j + 1]);
          }
        seen.template first_bound<__is_same(T, F32) ? 32 : __is_same(T, F16) ? 19 : 16>(largest);
      }
    } else {
      const int edge = b < 0 ? lane : V - tail + lane;
      at = edge;
      u[0] = none;
      if (lane < (b < 0 ? head : tail)) {
        if constexpr (__is_same(T, F32)) u[0][0] = __builtin_bit_cast(uint32_t, x[edge]);
        else u[0][0] = x[edge] | (kNone & 0xffff0000u);
      }
    }
    uint32_t enter = 0;   // loads with elements for the list
#pragma unroll
    for (int i = 0; i < kAhead; i++)
      if (i < count) {
        float v[N];
        unpack<T>(u[i], v);
        enter |= seen.template take<N>(v) ? 1u << i : 0;
      }
    while (enter != 0) {
      const int i = __builtin_ctz(enter);
      enter &= enter - 1;
      u32x4_t w = u[0];
#pragma unroll
      for (int j = 1; j < kAhead; j++)
        if (i == j) {
          w = u[j];
          asm volatile("" : "+v"(w));   // (moved where it is, rather than chosen lane by lane)
        }
      float v[N];
      unpack<T>(w, v);
      seen.template push<N>(v, (uint32_t)(at + i * next));
    }
  }
  if (TOP && seen.held > 0) seen.flush();
  Sums s = join_lanes(seen.sums);
  uint64_t list = seen.list;
  join_waves<kWaves, TOP>(s, list, sums, buffers, kBuffer, wave);
  if (wave > 0) return;
  if (a.parts == 1) {
    write_row<T>(a, row, s, list, x_token);
  } else {
    if (lane == 0) a.sums[blockIdx.x] = make_float4(s.m, s.s, s.y, 0.0f);
    if (lane < a.top) a.lists[(int64_t)blockIdx.x * a.top + lane] = list;
  }
}

// Joins a row's parts: all of them are asked for at once.
constexpr int kJoinWaves = 8, kMaxParts = 16;
template <class T, bool TOP>
__global__ __launch_bounds__(64 * kJoinWaves) void logprobs_join_kernel(LogprobArgs a) {
  constexpr int kEach = kMaxParts / kJoinWaves;
  __shared__ uint64_t lists[kJoinWaves * 64];
  __shared__ Sums sums[kJoinWaves];
  const int tid = threadIdx.x, lane = tid % 64;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int64_t row = blockIdx.x;
  float4 v[kEach];
  uint64_t k[kEach];
#pragma unroll
  for (int i = 0; i < kEach; i++) {
    const int p = i * kJoinWaves + wave;
    if (p < a.parts) {
      v[i] = a.sums[row * a.parts + p];
      if (TOP) k[i] = lane < a.top ? a.lists[(row * a.parts + p) * a.top + lane] : 0;
    }
  }
  const int32_t token = a.tokens[row];
  float x_token = -__builtin_inff();
  if (token >= 0 && token < a.V) x_token = element<T>(a.x, row * a.ld + token);
  Sums s{-__builtin_inff(), 0.0f, 0.0f};
  uint64_t list = 0;
#pragma unroll
  for (int i = 0; i < kEach; i++)
    if (i * kJoinWaves + wave < a.parts) {
      s = join(s, Sums{v[i].x, v[i].y, v[i].z});
      if (TOP) list = i == 0 ? k[i] : merge64(list, k[i]);
    }
  join_waves<kJoinWaves, TOP>(s, list, sums, lists, 64, wave);
  if (wave == 0) write_row<T>(a, row, s, list, x_token);
}

// A row is a workgroup's where there are many, and cut into parts where there are
// few: up to 512 workgroups of 16 parts at most, and a load at least for each lane of
// them. (64 rows of 128000 in bf16, 20 tokens: 20 us with 8 parts, 29 with 2, 38 whole;
// 256 rows: 39 with 2, 40 whole, 46 with 8.)
constexpr int kSomeWaves = 8;
int parts_of(int dt, int64_t M, int64_t V) {
  const int64_t each = (int64_t)64 * (dt == 2 ? 4 : 8) * kSomeWaves;
  int64_t p = 512 / M, most = V / each;
  p = p < most ? p : most;
  return (int)(p < 1 ? 1 : p > kMaxParts ? kMaxParts : p);
}
// Eight wavefronts of a workgroup, fewer where the rows fill the chip: two with a list, of
// which each wavefront pays the start and the end, and four without. (bf16, few and eight
// wavefronts, us:
//   rows            1024      1280      1536      1800      2048      2560      4096
//   V 32000,  20   39, 37    44, 44    49, 50    50, 62    51, 63    63, 75    78, 114
//   V 128000, 20   97, 78   109, 94   122, 108  124, 133  126, 138  158, 167  218, 255
//   V 200064, 20  134, 105  149, 127  168, 147  171, 181  177, 190  222, 231  319, 358
//   V 128000, 0    61, 52    68, 73    75, 79    88, 90    98, 98   137, 120  187, 186
// and with 5 or 64 tokens as with 20.)
constexpr int64_t kManyRows = 1537;

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
    auto rows = [&]<bool TOP, int W>() {
      hipLaunchKernelGGL((logprobs_kernel<T, TOP, W>), grid, dim3(64 * W), 0, st, a);
    };
    if (M < kManyRows && top > 0) rows.template operator()<true, kSomeWaves>();
    else if (M < kManyRows) rows.template operator()<false, kSomeWaves>();
    else if (top > 0) rows.template operator()<true, 2>();
    else rows.template operator()<false, 4>();
    if (a.parts == 1) return;
    if (top > 0) hipLaunchKernelGGL((logprobs_join_kernel<T, true>), dim3((unsigned)M), dim3(64 * kJoinWaves), 0, st, a);
    else hipLaunchKernelGGL((logprobs_join_kernel<T, false>), dim3((unsigned)M), dim3(64 * kJoinWaves), 0, st, a);
  };
  if (dt == 0) go.template operator()<F16>();
  else if (dt == 1) go.template operator()<BF16>();
  else go.template operator()<F32>();
  return hipGetLastError();
}

}  // namespace qmm
