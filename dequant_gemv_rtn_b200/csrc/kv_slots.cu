// kv_slots.cu -- page tables and slots of a decode step's new tokens, from the
// requests' lengths (qnt_kv_slots; the arithmetic is in include/qnt.h).
//
// With used = ceil(len / P) and need = ceil((len + add) / P) - used, request i
// takes the pages number end_i - need_i .. end_i - 1 from the top of the stack,
// end = the inclusive prefix sum of need; a token row t belongs to the request
// whose range of the prefix sum of add holds t.  So everything follows from
// three prefix sums over the requests, and each output element from a binary
// search in one of them.  Every CTA computes the sums for itself (4096 requests
// are 32 KB of reads, from L2) and keeps them in shared memory; then all CTAs
// share the outputs, one element per thread and step.  Nothing is exchanged
// between CTAs, so one launch does, and since no element that is read is also
// written (a page that is pushed and popped in the same call is read from its
// request's table row, not from the stack) the order of CTAs does not matter.
// Bound by latency: two dependent reads, two block scans, one search.
#include "common.cuh"
#include "kernels.h"

namespace qnt {
namespace {

constexpr int kSlThreads = 1024;
constexpr int kSlCtrl = 528;     // scan scratch in front of the sums

__device__ __forceinline__ int sat(long long v) { return v > 0x7FFFFFFF ? 0x7FFFFFFF : (int)v; }

// Inclusive prefix sums over the CTA's threads of two values, in place.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long (*part)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    part[warp][0] = a;
    part[warp][1] = b;
  }
  __syncthreads();
  if (warp == 0) {
    long long x = lane < warps ? part[lane][0] : 0, y = lane < warps ? part[lane][1] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) {
        x += u;
        y += v;
      }
    }
    if (lane < warps) {
      part[lane][0] = x;
      part[lane][1] = y;
    }
  }
  __syncthreads();
  if (warp) {
    a += part[warp - 1][0];
    b += part[warp - 1][1];
  }
  __syncthreads();
}

// The first row whose inclusive prefix sum is above v (v < end[rows - 1]).
__device__ __forceinline__ int row_of(const int* end, int rows, int v) {
  int lo = 0, hi = rows - 1;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (end[m] > v) hi = m;
    else lo = m + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kSlThreads) kv_slots_kernel(const KvSlotsArgs A) {
  extern __shared__ __align__(16) uint8_t smem[];
  long long (*const part)[2] = reinterpret_cast<long long (*)[2]>(smem);
  int& top_s = *reinterpret_cast<int*>(smem + 512);
  int* const add_end = reinterpret_cast<int*>(smem + kSlCtrl);   // inclusive sums: new tokens,
  int* const need_end = add_end + A.rows;                        // new pages,
  int* const out_end = need_end + A.rows;                        // released pages
  const int tid = threadIdx.x, threads = blockDim.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) top_s = 0;

  const int P = A.page;
  const long long room = (long long)A.width * P;
  // each thread takes a run of rows, so a thread's sum is a prefix of the next's
  const int per = (A.rows + threads - 1) / threads;
  const int r0 = min(tid * per, A.rows), r1 = min(r0 + per, A.rows);
  bool bad = false;
  long long n_sum = 0, out_sum = 0;
  for (int r = r0; r < r1; ++r) {
    const int len = A.len[r], add = A.add[r];
    const bool len_ok = len >= 0 && len <= room;
    bad |= !len_ok || add < -1;
    n_sum += add > 0 ? add : 0;
    out_sum += add < 0 && len_ok ? (len + (long long)P - 1) / P : 0;
  }
  long long n_end = n_sum, o_end = out_sum;
  block_scan2(n_end, o_end, part);
  long long need_sum = 0, unused = 0;
  {
    long long n = n_end - n_sum, o = o_end - out_sum;
    for (int r = r0; r < r1; ++r) {
      const int len = A.len[r], add = max(A.add[r], 0);
      const bool len_ok = len >= 0 && len <= room, out = A.add[r] < 0;
      const long long used = len_ok ? (len + (long long)P - 1) / P : 0;
      n += add;
      o += out ? used : 0;
      const bool fits = len_ok && len + (long long)add <= room && n <= A.tokens;
      bad |= !out && !fits;
      need_sum += fits && !out ? (len + (long long)add + P - 1) / P - used : 0;
      add_end[r] = sat(n);
      out_end[r] = sat(o);
      need_end[r] = sat(need_sum);     // of this thread's rows; the rows before are added below
    }
  }
  long long need_incl = need_sum;
  block_scan2(need_incl, unused, part);
  int count = *A.free_count;
  bad |= count < 0 || count > A.pages;
  count = min(max(count, 0), A.pages);
  const long long have_ll = (long long)count + out_end[A.rows - 1];
  const int have = sat(have_ll);
  // rows get what they need while the stack lasts; the served needs are a prefix
  bool short_of = false;
  int top = 0;
  {
    const long long before = need_incl - need_sum;
    int last = 0;
    for (int r = r0; r < r1; ++r) {
      const int mine = need_end[r] - last;
      last = need_end[r];
      const int end = sat(before + last);
      need_end[r] = end;
      if (mine > 0) {
        if (end <= have) top = end;
        else short_of = true;
      }
    }
  }
  if (top) atomicMax(&top_s, top);
  __syncthreads();
  // (more pages released than there are: what does not fit is dropped)
  const int taken = top_s, left = min(have - taken, A.pages);
  bad |= have - taken > A.pages;
  if (blockIdx.x == 0) {
    if (short_of) report(A.status, QNT_ERR_PAGES);
    if (bad) report(A.status, QNT_ERR_ARG);
    if (tid == 0) {
      *A.free_count_out = left;
      A.cu[0] = 0;
    }
  }

  // page number j of the stack, counted from the bottom, pushes included
  auto stack = [&](int j) -> int {
    if (j < count) return A.free[j];
    const int k = j - count, r = row_of(out_end, A.rows, k);
    return A.table[(size_t)r * A.width + (k - (r ? out_end[r - 1] : 0))];
  };
  const int t0 = blockIdx.x * threads + tid, step = gridDim.x * threads;
  for (int r = t0; r < A.rows; r += step) {
    const int len = A.len[r], add = A.add[r];
    const int need = need_end[r] - (r ? need_end[r - 1] : 0);
    const bool fits = len >= 0 && (long long)len + max(add, 0) <= room && add_end[r] <= A.tokens;
    const bool ok = fits && (need == 0 || need_end[r] <= have);
    A.len_out[r] = add < 0 ? 0 : ok ? len + add : len;
    A.cu[r + 1] = min(add_end[r], A.tokens);
  }
  for (int g = t0; g < taken; g += step) {             // new table entries
    const int r = row_of(need_end, A.rows, g);
    const int used = (A.len[r] + P - 1) / P;
    A.table[(size_t)r * A.width + used + (g - (r ? need_end[r - 1] : 0))] = stack(have - 1 - g);
  }
  for (long long j = (long long)count + t0; j < left; j += step) A.free[j] = stack((int)j);   // pushes that stay
  const int total = min(add_end[A.rows - 1], A.tokens);
  for (int t = t0; t < A.tokens; t += step) {
    int slot = -1;
    if (t < total) {
      const int r = row_of(add_end, A.rows, t);
      const int len = A.len[r], first = r ? add_end[r - 1] : 0;
      const int need0 = r ? need_end[r - 1] : 0, need = need_end[r] - need0;
      const bool fits = len >= 0 && (long long)len + (add_end[r] - first) <= room && add_end[r] <= A.tokens;
      if (fits && (need == 0 || need_end[r] <= have)) {
        const int p = len + (t - first), used = (len + P - 1) / P, j = p / P;
        const int page = j < used ? A.table[(size_t)r * A.width + j] : stack(have - 1 - (need0 + j - used));
        // a page outside the cache: a slot outside it, too, not one that the product wraps to
        slot = (unsigned)page < (unsigned)A.pages ? page * P + (p - j * P) : 0x7FFFFFFF;
      }
    }
    A.slots[t] = slot;
  }
}

}  // namespace

cudaError_t launch_kv_slots(const KvSlotsArgs& a, cudaStream_t s) {
  auto kfn = kv_slots_kernel;
  cudaError_t e = configure_smem(reinterpret_cast<const void*>(kfn));
  if (e != cudaSuccess) return e;
  // One element of the outputs per thread, and CTAs for the pages that released
  // requests push, whose number the host does not know (1500 rows, 75 of them with 250
  // pages: 15 us with two CTAs, 8 with 64).  Fewer threads scan few rows sooner, more
  // scan many in fewer steps (1500 rows, 65536 slots: 8.2 us with 512, 9.1 with 1024;
  // 4000 rows: 16.2 and 11.7).
  const int items = a.tokens > a.rows ? a.tokens : a.rows;
  const int threads = a.rows <= 256 ? 256 : a.rows <= 2048 ? 512 : kSlThreads;
  const int most = num_sms();                    // (more CTAs only read the rows more often)
  int want = (items + threads - 1) / threads;
  if (want < a.rows / 16) want = a.rows / 16 < 64 ? a.rows / 16 : 64;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(want < most ? want : most);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = kSlCtrl + (size_t)a.rows * 12;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kfn, a);
}

}  // namespace qnt
