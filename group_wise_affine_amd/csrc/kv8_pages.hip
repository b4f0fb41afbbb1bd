// Page bookkeeping of the 8-bit cache, all on the device: one call that
// re-orders, forks, truncates, grows, starts and drops sequences, and one
// that packs the pages in use to the front of the pool. Whole numbers
// throughout; the results do not depend on the order in which workgroups run.
#include "kernels.hpp"
#include "kv8_common.hpp"

namespace qmm {
namespace {

constexpr int kChunk = 1024;   // pages per count

// exclusive prefix sum of one int per thread over 256 threads; `total` gets
// the sum
__device__ __forceinline__ int scan256(int v, int* total) {
  __shared__ int wave_sum[4];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  int s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();   // wave_sum of an earlier call has been read
  if (lane == 63) wave_sum[wave] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    before += i < wave ? wave_sum[i] : 0;
    all += wave_sum[i];
  }
  *total = all;
  return before + s - v;
}

struct Update {
  const int32_t *ref, *table, *lens, *parent, *new_lens;
  int32_t *ref_out, *table_out, *shortage;
  int32_t *shared, *free_in;   // scratch: [P] shares by other slots, [chunks] free pages
  int S, W, P, bt_log2;
  __device__ int64_t clip(int64_t n) const {
    const int64_t most = (int64_t)W << bt_log2;
    return n < 0 ? 0 : n > most ? most : n;
  }
  __device__ int pages(int64_t n) const { return (int)((n + (1 << bt_log2) - 1) >> bt_log2); }
  __device__ int par(int s) const {
    const int p = parent[s];
    return p >= 0 && p < S ? p : -1;
  }
  __device__ int64_t keep(int s) const {   // tokens that slot s takes over
    const int p = par(s);
    if (p < 0) return 0;
    const int64_t a = clip(lens[p]), b = clip(new_lens[s]);
    return a < b ? a : b;
  }
  __device__ int entry(int s, int j) const {   // -1 for what is no page
    const int e = table[(int64_t)s * W + j];
    return e >= 0 && e < P ? e : -1;
  }
};

// counts start from the old ones; free pages are counted by chunk
__global__ __launch_bounds__(256) void update_begin_kernel(Update u) {
  const int base = blockIdx.x * kChunk;
  int free = 0;
#pragma unroll
  for (int i = 0; i < kChunk / 256; i++) {
    const int p = base + i * 256 + threadIdx.x;
    if (p < u.P) {
      const int r = u.ref[p];
      u.ref_out[p] = r;
      u.shared[p] = 0;
      free += r == 0;
    }
  }
  int total;
  scan256(free, &total);
  if (threadIdx.x == 0) u.free_in[blockIdx.x] = total;
  if (blockIdx.x == 0 && threadIdx.x == 0) *u.shortage = 0;
}

// the old rows' references go, the whole pages that another slot's new row
// shares come (integer sums; a slot that keeps its own pages changes nothing)
__global__ __launch_bounds__(256) void update_count_kernel(Update u) {
  const int s = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x;
  if (j >= u.W) return;
  const int p = u.par(s);
  const int full = (int)(u.keep(s) >> u.bt_log2);
  const bool own = p == s && j < full;
  if (j < u.pages(u.clip(u.lens[s])) && !own) {
    const int e = u.entry(s, j);
    if (e >= 0) atomicAdd(u.ref_out + e, -1);
  }
  if (j < full && !own) {
    const int e = u.entry(p, j);
    if (e >= 0) {
      atomicAdd(u.ref_out + e, 1);
      atomicAdd(u.shared + e, 1);
    }
  }
}

// what slot s does with the page that its kept tokens fill in part: keeps it
// in place when it is the slot's own and nobody else will read it, else
// copies it to a fresh page
struct Last {
  int page;     // the old page, -1: none
  bool copied;
};
__device__ __forceinline__ Last last_page(const Update& u, int s, int64_t keep) {
  Last l{-1, false};
  if ((keep & ((1 << u.bt_log2) - 1)) == 0) return l;
  const int p = u.par(s);
  l.page = u.entry(p, (int)(keep >> u.bt_log2));
  l.copied = l.page >= 0 && !(p == s && u.ref[l.page] == 1 && u.shared[l.page] == 0);
  return l;
}
// One slot per blockIdx.x: its fresh pages are the free pages of rank r0 ..
// r0 + need, r0 the pages that the slots before it take. The workgroups of
// blockIdx.y > 0 find the same numbers and help to copy the last page. What
// bounds it is the chain of dependent loads, so a thread looks at each slot up
// to this one, this one among them, and the first counts of free pages are
// asked for before that. (64 slots: 6.6 us, after 2.8 and 3.1 for the two above.)
__global__ __launch_bounds__(256) void update_assign_kernel(Update u, Kv8 c) {
  const int s = blockIdx.x, tid = threadIdx.x;
  const bool writer = blockIdx.y == 0;
  const int chunks = (u.P + kChunk - 1) / kChunk;
  const int free0 = tid < chunks ? u.free_in[tid] : 0;
  __shared__ int own_page, own_copied, own_need, own_full, own_kept;
  int sum = 0, r0 = 0;
  for (int t = tid; t <= s; t += 256) {
    const int64_t keep = u.keep(t);
    const Last l = last_page(u, t, keep);
    const int grow = u.pages(u.clip(u.new_lens[t])) - u.pages(keep);
    const int need = (grow > 0 ? grow : 0) + (l.copied ? 1 : 0);
    if (t < s) {
      sum += need;
    } else {
      own_page = l.page;
      own_copied = l.copied;
      own_need = need;
      own_full = (int)(keep >> u.bt_log2);
      own_kept = u.pages(keep);
    }
  }
  scan256(sum, &r0);   // (and a barrier)
  const Last last{own_page, own_copied != 0};
  if (!writer && !last.copied) return;
  const int need = own_need, full = own_full, kept = own_kept;
  const int j0 = last.copied ? full : kept;   // fresh pages take columns j0 ..
  int32_t* row = u.table_out + (int64_t)s * u.W;
  __shared__ int copy_to, hit[256], start[256];   // chunks that hold wanted ranks
  if (tid == 0) copy_to = -1;
  if (writer) {
    const int p = u.par(s);
    for (int j = tid; j < u.W; j += 256)
      if (j < j0 || j >= j0 + need) row[j] = j < kept ? u.entry(p, j) : -1;
    if (tid == 0 && last.page >= 0 && !last.copied) atomicAdd(u.ref_out + last.page, 1);
  }
  // free pages by rank
  int seen = 0;
  const int want = writer ? need : 1;
  for (int b = 0; b < chunks && seen < r0 + want; b += 256) {
    const int mine = b == 0 ? free0 : b + tid < chunks ? u.free_in[b + tid] : 0;
    int all;
    const int before = seen + scan256(mine, &all);
    // this thread's chunk holds ranks before .. before + mine
    const bool touch = mine > 0 && before < r0 + want && before + mine > r0;
    int n_hit;
    const int slot = scan256(touch ? 1 : 0, &n_hit);
    if (touch) {
      hit[slot] = b + tid;
      start[slot] = before;
    }
    __syncthreads();
    for (int h = 0; h < n_hit; h++) {
      const int base = hit[h] * kChunk + tid * (kChunk / 256);
      int flags = 0, cnt = 0;
#pragma unroll
      for (int i = 0; i < kChunk / 256; i++)
        if (base + i < u.P && u.ref[base + i] == 0) {
          flags |= 1 << i;
          cnt++;
        }
      int chunk_all;
      int rank = start[h] + scan256(cnt, &chunk_all);
#pragma unroll
      for (int i = 0; i < kChunk / 256; i++)
        if (flags >> i & 1) {
          if (rank >= r0 && rank < r0 + want) {
            if (rank == r0) copy_to = base + i;
            if (writer) {
              row[j0 + rank - r0] = base + i;
              u.ref_out[base + i] = 1;
            }
          }
          rank++;
        }
    }
    seen += all;
  }
  __syncthreads();
  // fewer free pages than asked for: the places stay empty and are counted
  if (writer) {
    const int got = seen - r0 < 0 ? 0 : seen - r0;
    if (got < need) {
      for (int i = got + tid; i < need; i += 256) row[j0 + i] = -1;
      if (tid == 0) atomicAdd(u.shortage, need - got);
    }
  }
  if (last.copied && copy_to >= 0) copy_page(c, copy_to, c, last.page, blockIdx.y, gridDim.y);
}

// ------------------------------------------------------------------ compact
struct Compact {
  const int32_t *ref, *table;
  int32_t *ref_out, *table_out, *remap, *used;
  int32_t *used_in, *holes, *movers, *rank;   // scratch: [chunks], [P], [P], [P]
  int64_t entries;
  int P;
};

__global__ __launch_bounds__(256) void compact_count_kernel(Compact u) {
  int n = 0, total;
#pragma unroll
  for (int i = 0; i < kChunk / 256; i++) {
    const int p = blockIdx.x * kChunk + i * 256 + threadIdx.x;
    n += p < u.P && u.ref[p] > 0;
  }
  scan256(n, &total);
  if (threadIdx.x == 0) u.used_in[blockIdx.x] = total;
}

// With n pages in use, the i-th used page at or past n moves into the i-th
// hole below n: lists both, in order.
__global__ __launch_bounds__(256) void compact_list_kernel(Compact u) {
  const int tid = threadIdx.x, chunks = (u.P + kChunk - 1) / kChunk;
  int a = 0, b = 0, n, before;
  for (int i = tid; i < chunks; i += 256) {
    const int k = u.used_in[i];
    a += k;
    b += i < (int)blockIdx.x ? k : 0;
  }
  scan256(a, &n);
  scan256(b, &before);
  // used pages below n: whole chunks, and the part of the chunk that holds n
  int low = 0, low_used;
  for (int i = tid; i < n / kChunk; i += 256) low += u.used_in[i];
  for (int p = n / kChunk * kChunk + tid; p < n; p += 256) low += u.ref[p] > 0;
  scan256(low, &low_used);
  const int base = blockIdx.x * kChunk + tid * (kChunk / 256);
  int used[kChunk / 256], cnt = 0, all;
#pragma unroll
  for (int i = 0; i < kChunk / 256; i++) {
    used[i] = base + i < u.P && u.ref[base + i] > 0;
    cnt += used[i];
  }
  int r = before + scan256(cnt, &all);   // used pages before this one
#pragma unroll
  for (int i = 0; i < kChunk / 256; i++) {
    const int p = base + i;
    if (p >= u.P) break;
    if (used[i] && p >= n) {
      u.movers[r - low_used] = p;
      u.rank[p] = r - low_used;
    } else if (!used[i] && p < n) {
      u.holes[p - r] = p;
      u.rank[p] = p - r;
    }
    r += used[i];
  }
  if (blockIdx.x == 0 && tid == 0) {
    u.used[0] = n;
    u.used_in[chunks] = n - low_used;   // pages that move
  }
}

// Bound by memory: 178 MB read and written in 38 us, 4.7 TB/s.
__global__ __launch_bounds__(256) void compact_move_kernel(Compact u, Kv8 c, int parts) {
  const int n = u.used[0], movers = u.used_in[(u.P + kChunk - 1) / kChunk];
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x, stride = (int64_t)gridDim.x * 256;
  auto moved = [&](int p) QMM_INLINE {
    if (p < 0 || p >= u.P || u.ref[p] <= 0) return -1;
    return p < n ? p : u.holes[u.rank[p]];
  };
  for (int64_t i = t; i < u.entries; i += stride) u.table_out[i] = moved(u.table[i]);
  for (int64_t p = t; p < u.P; p += stride) {
    u.remap[p] = moved((int)p);
    const int r = u.ref[p];
    u.ref_out[p] = p >= n ? 0 : r > 0 ? r : u.ref[u.movers[u.rank[p]]];
  }
  for (int64_t i = blockIdx.x; i < (int64_t)movers * parts; i += gridDim.x)
    copy_page(c, u.holes[i / parts], c, u.movers[i / parts], (int)(i % parts), parts);
}

}  // namespace

int64_t kv8_pages_work(int64_t P) { return 4 * (3 * P + (P + kChunk - 1) / kChunk + 1); }

hipError_t launch_kv8_update(const Kv8& c, const int32_t* ref, const int32_t* table,
                             const int32_t* lens, const int32_t* parent, const int32_t* new_lens,
                             int64_t S, int64_t W, int32_t* ref_out, int32_t* table_out,
                             int32_t* shortage, int32_t* work, hipStream_t st) {
  const int P = c.pages, chunks = (P + kChunk - 1) / kChunk;
  Update u{ref, table, lens, parent, new_lens, ref_out, table_out, shortage, work, work + P,
           (int)S, (int)W, P, c.bt_log2};
  hipLaunchKernelGGL(update_begin_kernel, dim3((unsigned)chunks), dim3(256), 0, st, u);
  hipLaunchKernelGGL(update_count_kernel, dim3((unsigned)((W + 255) / 256), (unsigned)S), dim3(256),
                     0, st, u);
  hipLaunchKernelGGL(update_assign_kernel, dim3((unsigned)S, (unsigned)copy_parts(c)), dim3(256), 0,
                     st, u, c);
  return hipGetLastError();
}

hipError_t launch_kv8_compact(const Kv8& c, const int32_t* ref, const int32_t* table, int64_t S,
                              int64_t W, int32_t* ref_out, int32_t* table_out, int32_t* remap,
                              int32_t* used, int32_t* work, hipStream_t st) {
  const int P = c.pages, chunks = (P + kChunk - 1) / kChunk;
  Compact u{ref, table, ref_out, table_out, remap, used, work, work + chunks + 1,
            work + chunks + 1 + P, work + chunks + 1 + 2 * (int64_t)P, S * W, P};
  hipLaunchKernelGGL(compact_count_kernel, dim3((unsigned)chunks), dim3(256), 0, st, u);
  hipLaunchKernelGGL(compact_list_kernel, dim3((unsigned)chunks), dim3(256), 0, st, u);
  hipLaunchKernelGGL(compact_move_kernel, dim3(2048), dim3(256), 0, st, u, c, copy_parts(c));
  return hipGetLastError();
}

}  // namespace qmm
