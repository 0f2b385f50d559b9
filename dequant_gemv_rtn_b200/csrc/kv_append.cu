// kv_append.cu -- quantizes new keys and values into the paged 8-bit cache
// (qnt_kv_append; layout and definition in include/qnt.h).
//
// A run (the new tokens of one page) shares a scale per head, s = max |x| / top.
// The grid is (windows of token rows) x heads x {K, V}; a lane holds eight values of
// a token, a warp IT rounds of 256 / dim tokens.  Which rows form runs is only
// known from the slots, so the rows' values are requested first, by row number,
// and the slots are read beside them: two waits for memory, not four.  Rows that
// do not go on from the row before are bits of a mask; a row's run is what lies
// between two bits.  max |x| goes from the values to the run's entry in shared
// memory by atomicMax on the (non-negative) float's bits, which does not depend
// on the order.  A run that crosses the window's ends is completed by reading its
// other rows, too (up to a page at either end, from L2); every window writes the
// codes of its own rows, the one with the run's first row the scale.  (Another
// may read the page's old scale before or after that: max(new, old) is the same.)
//
// A run that goes on in a page begun before keeps the page's scale or raises it;
// raising re-rounds the codes of the tokens before it.  That is a map of 256
// bytes to 256 bytes: a warp tabulates it in 64 bits and applies it by look-up.
//
// Rounding to the nearest code of the real quotient x / s without a division:
// t = x * (1 / s) is off by at most two units in the last place, so only a t
// next to a tie can round wrongly, which a remainder then decides; what is not
// finite or too small for 1 / s goes through a 64-bit quotient.  INT8: adding
// 1.5 2^23 + 128 leaves q + 128 in the low byte, and |t - q| tells how near a tie
// is.  E4M3: ties have five significant bits from 2^-6 on, so t is near one only if
// its 20 low bits are within four of 2^19; below 2^-6, fewer than five.  (In one
// page of seven a is a multiple of 7, and then 2 % of all x / s are ties: with the
// 64-bit quotient for these, too, 8192 prompt tokens took 52 us.)
//
// Prompts are bound by instructions (11 a value, 57 % of the issue slots) and the five
// barriers of a window, not by memory: 8192 rows of 8 heads of 128 take 23.7 us for
// 50 MB (2 bytes read and 1 written per value), a third of the copy rate.  A decode
// step (64 rows: 3.0 us) is bound by latency, two waits for memory.
#include "common.cuh"
#include "kernels.h"

namespace qnt {
namespace {

constexpr int kApWarps = 8;
constexpr int kApThreads = 32 * kApWarps;
constexpr int kApHalo = 128;                 // rows kept on either side of the window: a page
constexpr int kApBad = 0x7FFFFFFF;           // a slot beyond the cache

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
  return h2f(h & 0xFFFFu);
}
// Code byte nearest to y.  E4M3: y rounded towards zero with the last bit set if
// that was inexact; any later rounding to 22 bits or fewer is then that of y.
template <int FMT>
__device__ __forceinline__ uint32_t nearest_byte(double y) {
  if (FMT == QNT_KV_INT8) return (uint32_t)((int)fmin(fmax(rint(y), -127.0), 127.0) + 128);
  float t = __double2float_rz(y);
  if ((double)t != y) t = __uint_as_float(__float_as_uint(t) | 1u);
  return e4m3x2(t, 0.0f) & 0xFFu;
}
template <int FMT>
__device__ __forceinline__ uint32_t requant_byte(uint32_t b, double s0, double s) {
  const double v = FMT == QNT_KV_INT8 ? (double)((int)b - 128) : (double)e4m3_value(b);
  return nearest_byte<FMT>(v * s0 / s);
}

template <bool BF16>
__device__ __forceinline__ float2 value_pair(uint32_t w) {
  if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return make_float2(h2f(w & 0xFFFFu), h2f(w >> 16));
}
// The eight codes of v in 64 bits (rare).
template <int FMT, bool BF16>
__device__ __noinline__ uint2 codes_exact(uint4 v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[2] = {0, 0};
#pragma unroll 1
  for (int j = 0; j < 8; ++j) {
    const float2 p = value_pair<BF16>(w[j >> 1]);
    float x = j & 1 ? p.y : p.x;
    if (!(x == x)) x = 0.0f;                                 // the cache holds no NaN
    o[j >> 2] |= (s > 0.0f ? nearest_byte<FMT>((double)x / (double)s) : FMT == QNT_KV_INT8 ? 128u : 0u) << (8 * (j & 3));
  }
  return make_uint2(o[0], o[1]);
}
// max(|a|, b), NaN if either is
__device__ __forceinline__ float max_abs_nan(float a, float b) {
  float d;
  asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %1;\n\tmax.NaN.f32 %0, t, %2;\n\t}" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// The same with t = x * inv next to a tie somewhere: the sign of a remainder,
// rounded once, decides.  INT8: x - q s against s / 2 (exact: q s has 31 bits, the
// difference cancels to 24).  E4M3: t is moved off the five-bit number m that it
// is next to, to the side that x - m s tells (away from 0 if that has t's sign; by sign
// bits, since t may have underflowed to a zero).
template <int FMT, bool BF16>
__device__ __forceinline__ uint2 codes_near(uint4 v, float s, float inv) {
  if (FMT == QNT_KV_E4M3 && s == 0.0f) return make_uint2(0, 0);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[8];
  bool nan = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 p = value_pair<BF16>(w[j >> 1]);
    const float x = j & 1 ? p.y : p.x;
    const float t = x * inv;
    nan |= !(fabsf(t) < 1e30f);
    if (FMT == QNT_KV_INT8) {
      float q = rintf(t);
      const float d = fmaf(-q, s, x), half = 0.5f * s;
      const bool odd = ((int)q & 1) != 0;
      q += (d > half || (d == half && odd) ? 1.0f : 0.0f) - (d < -half || (d == -half && odd) ? 1.0f : 0.0f);
      c[j] = (uint32_t)((int)fminf(fmaxf(q, -127.0f), 127.0f) + 128);
    } else {
      const uint32_t b = __float_as_uint(t), m = (b + 4u) & ~0x7FFFFu;
      const float r = fmaf(-__uint_as_float(m), s, x);
      const uint32_t to = r == 0.0f ? m : (r < 0.0f) == ((int)b < 0) ? m + 1u : m - 1u;
      c[j] = ((b + 4u) & 0x7FFFFu) < 9u ? to : b;
    }
  }
  if (nan) return codes_exact<FMT, BF16>(v, s);
  if (FMT == QNT_KV_INT8)
    return make_uint2(c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24), c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24));
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = e4m3x2(__uint_as_float(c[2 * j]), __uint_as_float(c[2 * j + 1]));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
// The eight codes of v; inv = 1 / s, 0 for s = 0, NaN where that is out of range.
template <int FMT, bool BF16>
__device__ __forceinline__ uint2 codes_of(uint4 v, float s, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[2];
  bool sure;
  if (FMT == QNT_KV_INT8) {
    constexpr float kMagic = 12582912.0f + 128.0f;
    uint32_t b[8];
    float off = 0.0f;                          // the largest distance from a whole number
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = value_pair<BF16>(w[j]);
      const float tx = p.x * inv, ty = p.y * inv;
      const float rx = tx + kMagic, ry = ty + kMagic;
      off = max_abs_nan(tx - (rx - kMagic), off);
      off = max_abs_nan(ty - (ry - kMagic), off);
      b[2 * j] = __float_as_uint(rx);
      b[2 * j + 1] = __float_as_uint(ry);
    }
    sure = off < 0.4999f;                      // false for NaN
#pragma unroll
    for (int j = 0; j < 2; ++j)
      o[j] = prmt(prmt(b[4 * j], b[4 * j + 1], 0x0040u), prmt(b[4 * j + 2], b[4 * j + 3], 0x0040u), 0x5410u);
  } else {
    uint32_t near = 0xFFFFFFFFu, c[4];         // the least of (20 low bits - 2^19 + 4) << 12: ties of 2^-6 and above
    float all = 0.0f, least = 1.0f;                        // smaller ones have their ties elsewhere
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = value_pair<BF16>(w[j]);
      const float tx = p.x * inv, ty = p.y * inv;
      near = min(near, min(__float_as_uint(tx) * 4096u + 0x80004000u, __float_as_uint(ty) * 4096u + 0x80004000u));
      least = fminf(least, fminf(fabsf(tx), fabsf(ty)));
      all = fmaf(tx, 0.0f, fmaf(ty, 0.0f, all));   // NaN if one is not finite
      c[j] = e4m3x2(tx, ty);
    }
    o[0] = c[0] | (c[1] << 16);
    o[1] = c[2] | (c[3] << 16);
    sure = near >= 9u * 4096u && least >= 0.015625f && all == all;
  }
  return sure ? make_uint2(o[0], o[1]) : codes_near<FMT, BF16>(v, s, inv);
}

// Larger magnitudes of two pairs (their sign bits are 0), NaN if either is.
template <bool BF16>
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  uint32_t d;
  if (BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool BF16>
__device__ __forceinline__ bool finite_pair(uint32_t m) {
  constexpr uint32_t kInf = BF16 ? 0x7F80u : 0x7C00u;
  return (m & 0xFFFFu) < kInf && (m >> 16) < kInf;
}
// Pair of the largest |x| of eight values, without those that are not finite.
template <bool BF16>
__device__ __forceinline__ uint32_t top_of(uint4 v, bool& bad) {
  uint32_t m = max_pair<BF16>(max_pair<BF16>(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                              max_pair<BF16>(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  if (!finite_pair<BF16>(m)) {
    bad = true;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    m = 0;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = w[j] & 0x7FFFu, hi = w[j] & 0x7FFF0000u;
      m = max_pair<BF16>(m, (finite_pair<BF16>(lo) ? lo : 0u) | (finite_pair<BF16>(hi) ? hi : 0u));
    }
  }
  return m;
}

template <int FMT, bool BF16, int D, int IT>
__global__ void __launch_bounds__(kApThreads, 4) kv_append_kernel(const KvAppendArgs A) {
  constexpr int LPT = D / 8;                   // lanes of a token
  constexpr int TPL = 32 / LPT;                // tokens of a round
  constexpr int RW = IT * TPL;                 // rows of a warp
  constexpr int ROWS = kApWarps * RW;          // rows of the window
  constexpr int ALL = kApHalo + ROWS + kApHalo;
  constexpr float kTop = FMT == QNT_KV_INT8 ? 127.0f : 448.0f;
  static_assert(ROWS <= kApThreads && ROWS % 32 == 0, "a thread per row, whole mask words");
  __shared__ int slot_s[ALL];
  __shared__ uint32_t brk_s[ALL / 32];         // bit: the row does not go on from the row before
  __shared__ uint32_t top_s[kApHalo + ROWS];   // max |x| of the run that begins at a row
  __shared__ uint8_t refused_s[kApHalo + ROWS];
  __shared__ short start_s[ROWS];              // where the row's run begins; -1: not written
  __shared__ float scale_s[ROWS], inv_s[ROWS];
  __shared__ int grow_row[ROWS], grow_n;
  __shared__ float grow_old[ROWS];
  __shared__ uint8_t lut_s[kApWarps][256];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y, kv = blockIdx.z;
  const int w0 = blockIdx.x * ROWS;            // first token row
  const int P = A.page, pl = 31 - __clz(P);
  uint8_t* const codes = kv ? A.codes[1] : A.codes[0];
  float* const scales = kv ? A.scales[1] : A.scales[0];
  const uint16_t* const x = static_cast<const uint16_t*>(kv ? A.x[1] : A.x[0]) + (int64_t)h * D + 8 * (lane % LPT);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  uint4 v[IT];
  const int mine = warp * RW + lane / LPT;     // this lane's first row in the window
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int row = w0 + mine + i * TPL;
    v[i] = row < A.tokens ? ldg_cg128(x + (int64_t)row * A.stride) : make_uint4(0, 0, 0, 0);
  }
  const int limit = A.pages << pl;
  for (int i = tid; i < ALL; i += kApThreads) {
    const int row = w0 - kApHalo + i;
    const int s = row >= 0 && row < A.tokens ? A.slots[row] : -1;
    slot_s[i] = s < limit ? s : kApBad;
    if (s >= limit && (h | kv) == 0) report(A.status, QNT_ERR_ARG);
    if (i < kApHalo + ROWS) {
      top_s[i] = 0;
      refused_s[i] = 0;
    }
  }
  if (tid == 0) grow_n = 0;
  __syncthreads();

  // ---- runs
  for (int i = tid; i < ALL; i += kApThreads) {
    const int s = slot_s[i], p = i ? slot_s[i - 1] : -1;
    const bool on = s >= 0 && s != kApBad && p >= 0 && p + 1 == s && (s & (P - 1)) != 0;
    const uint32_t m = __ballot_sync(0xffffffffu, !on);
    if (lane == 0) brk_s[i >> 5] = m;
  }
  __syncthreads();
  const int idx = kApHalo + tid;               // this thread's row, for tid < ROWS
  int start = -1;
  float s0 = 0.0f;
  if (tid < ROWS) {                            // whole warps
    const int s = slot_s[idx];
    const bool live = s >= 0 && s != kApBad;
    if (live) {
      int word = idx >> 5;
      uint32_t m = brk_s[word] & (0xFFFFFFFFu >> (31 - (idx & 31)));
      while (!m) m = brk_s[--word];            // a run is at most a page long
      start = 32 * word + 31 - __clz(m);
      if (slot_s[start] & (P - 1)) s0 = scales[(int64_t)(s >> pl) * A.heads + h];
    }
    // the run is refused if its page had one before it with only skipped rows in between
    const int prev = start > 0 ? slot_s[start - 1] : -1;
    const bool first = live && (idx == start || tid == 0);
    bool refuse = first && prev >= 0 && prev != kApBad && (prev >> pl) == (s >> pl);
    uint32_t look = __ballot_sync(0xffffffffu, first && (prev < 0 || prev == kApBad));
    while (look) {
      const int src = __ffs(look) - 1;
      look &= look - 1;
      const int page = __shfl_sync(0xffffffffu, s, src) >> pl;
      int found = -1;
      for (int at = w0 - kApHalo + __shfl_sync(0xffffffffu, start, src) - 2; found < 0 && at >= 0; at -= 256) {
        int near = 256;
#pragma unroll
        for (int i = 7; i >= 0; --i) {         // rows at - 255 .. at, the nearest counts
          const int r = at - 32 * i - lane;
          if (r >= 0 && (unsigned)A.slots[r] < (unsigned)limit) near = 32 * i + lane;
        }
        near = __reduce_min_sync(0xffffffffu, near);
        if (near < 256) found = A.slots[at - near];
      }
      if (lane == src && found >= 0 && (found >> pl) == page) refuse = true;
    }
    if (refuse) {
      refused_s[start] = 1;
      if ((h | kv) == 0) report(A.status, QNT_ERR_ARG);
    }
    start_s[tid] = (short)start;
  }
  __syncthreads();
  if (start >= 0 && refused_s[start]) start = start_s[tid] = -1;
  __syncthreads();

  // ---- max |x| of the runs: what a lane's rows of one run have in common is
  // reduced over the token's lanes once
  bool bad = false;
  auto flush = [&](uint32_t m, int st) {
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) m = max_pair<BF16>(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = max(m & 0xFFFFu, m >> 16);
    if (lane % LPT == 0 && st >= 0) atomicMax(top_s + st, BF16 ? m << 16 : __float_as_uint(h2f(m)));
  };
  {
    uint32_t m = 0;
    int st = start_s[mine];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int now = i ? start_s[mine + i * TPL] : st;
      if (__any_sync(0xffffffffu, now != st)) {
        flush(m, st);
        m = 0;
        st = now;
      }
      bool odd = false;
      m = max_pair<BF16>(m, top_of<BF16>(v[i], odd));
      bad |= odd && now >= 0;
    }
    flush(m, st);
  }
  // rows of a run that crosses an end of the window
  const int st_first = start_s[0], st_last = start_s[ROWS - 1];
  const int back = st_first >= 0 ? max(kApHalo - st_first, 0) : 0;
  int fwd = 0;
  if (st_last >= 0) {
    int word = (kApHalo + ROWS) >> 5;
    while (word < ALL / 32 && !brk_s[word]) ++word;
    fwd = word < ALL / 32 ? 32 * word + __ffs(brk_s[word]) - 1 - (kApHalo + ROWS) : kApHalo;
  }
#pragma unroll 4
  for (int t = warp * TPL; t < back + fwd; t += kApWarps * TPL) {
    const int k = t + lane / LPT;
    const int row = k < back ? w0 - back + k : w0 + ROWS + (k - back);
    bool odd = false;                          // reported by the row's own window
    flush(top_of<BF16>(k < back + fwd ? ldg_cg128(x + (int64_t)row * A.stride) : make_uint4(0, 0, 0, 0), odd),
          k < back + fwd ? (k < back ? st_first : st_last) : -1);
  }
  if (bad) report(A.status, QNT_ERR_NONFINITE);
  __syncthreads();

  // ---- scales
  if (start >= 0) {
    const float s = fmaxf(__uint_as_float(top_s[start]) / kTop, s0);
    scale_s[tid] = s;
    inv_s[tid] = s > 1e-30f && s < 1e30f ? 1.0f / s : s == 0.0f ? 0.0f : __int_as_float(0x7FC00000);
    if (idx == start) {
      const int slot = slot_s[idx];
      scales[(int64_t)(slot >> pl) * A.heads + h] = s;
      if ((slot & (P - 1)) && s > s0) {
        const int k = atomicAdd(&grow_n, 1);
        grow_row[k] = tid;
        grow_old[k] = s0;
      }
    }
  }
  __syncthreads();

  // ---- codes
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int row = mine + i * TPL;
    if (start_s[row] < 0) continue;
    const int slot = slot_s[kApHalo + row];
    const uint2 o = codes_of<FMT, BF16>(v[i], scale_s[row], inv_s[row]);
    uint8_t* const dst = codes + (((((int64_t)(slot >> pl)) * A.heads + h) << pl) + (slot & (P - 1))) * D + 8 * (lane % LPT);
    *reinterpret_cast<uint2*>(dst) = o;
  }
  // ---- the tokens before a run whose page's scale grew, 16 codes a lane and step
  for (int k = warp; k < grow_n; k += kApWarps) {
    const int row = grow_row[k], slot = slot_s[kApHalo + row];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = 8 * lane + i;
      lut_s[warp][b] = (uint8_t)requant_byte<FMT>(b, grow_old[k], scale_s[row]);
    }
    __syncwarp();
    uint8_t* const page = codes + (((((int64_t)(slot >> pl)) * A.heads + h) << pl)) * D;
    const int bytes = (slot & (P - 1)) * D;
#pragma unroll 4
    for (int i = 16 * lane; i < bytes; i += 512) {
      uint4* const p = reinterpret_cast<uint4*>(page + i);
      const uint4 c = *p;
      const uint32_t in[4] = {c.x, c.y, c.z, c.w};
      uint32_t out[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        out[j] = (uint32_t)lut_s[warp][in[j] & 255u] | ((uint32_t)lut_s[warp][(in[j] >> 8) & 255u] << 8) |
                 ((uint32_t)lut_s[warp][(in[j] >> 16) & 255u] << 16) | ((uint32_t)lut_s[warp][in[j] >> 24] << 24);
      *p = make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
}

template <int FMT, bool BF16, int D, int IT>
cudaError_t ap_launch(const KvAppendArgs& a, cudaStream_t s) {
  constexpr int ROWS = kApWarps * IT * (256 / D);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.tokens + ROWS - 1) / ROWS, a.heads, 2);
  cfg.blockDim = dim3(kApThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_append_kernel<FMT, BF16, D, IT>, a);
}

template <int FMT, bool BF16, int D>
cudaError_t ap_rounds(const KvAppendArgs& a, cudaStream_t s) {
  // eight rounds a warp once that fills every SM; few rows are spread wider
  const long long windows = ((long long)a.tokens + 8 * kApWarps * (256 / D) - 1) / (8 * kApWarps * (256 / D));
  return windows * a.heads * 2 >= num_sms() ? ap_launch<FMT, BF16, D, 8>(a, s) : ap_launch<FMT, BF16, D, D == 256 ? 4 : 2>(a, s);
}

template <int FMT, bool BF16>
cudaError_t ap_dim(int dim, const KvAppendArgs& a, cudaStream_t s) {
  switch (dim) {
    case 64: return ap_rounds<FMT, BF16, 64>(a, s);
    case 128: return ap_rounds<FMT, BF16, 128>(a, s);
    default: return ap_rounds<FMT, BF16, 256>(a, s);
  }
}

}  // namespace

cudaError_t launch_kv_append(const qnt_kv_desc& d, const KvAppendArgs& a, int xbf16, cudaStream_t s) {
  if (d.fmt == QNT_KV_INT8) return xbf16 ? ap_dim<QNT_KV_INT8, true>(d.dim, a, s) : ap_dim<QNT_KV_INT8, false>(d.dim, a, s);
  return xbf16 ? ap_dim<QNT_KV_E4M3, true>(d.dim, a, s) : ap_dim<QNT_KV_E4M3, false>(d.dim, a, s);
}

}  // namespace qnt
