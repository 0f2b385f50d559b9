// kv_append.cu -- quantizes new keys and values into the paged 8-bit cache
// (qnt_kv_append; layout and definition in include/qnt.h).
//
// A run (the new tokens of one page) shares a scale per head, s = max |x| / top,
// so a run is one unit of work: read it once into registers, reduce max |x|,
// write the codes.  The grid is (windows of eight token rows) x heads x {K, V},
// a warp per token row: the warp whose row begins a run takes it when it has at
// most eight tokens (a decode step's, a draft's); a longer one, of which a
// window can begin only one, is shared by the CTA's eight warps, up to 16
// tokens each.  A run that goes on in a page begun before keeps the page's
// scale or raises it; raising it re-rounds the codes of the tokens before it.
// That is a map of 256 bytes to 256 bytes, so it is tabulated in 64 bits (8
// entries a lane) and applied by the whole CTA with table look-ups.
//
// Rounding to the nearest code of the real quotient x / s without a division:
// t = x * (1 / s) is off by at most two units in the last place, so only a t
// next to a tie can round wrongly.  INT8: with q = rint(t), d = x - q s is exact
// in fp32 (q s has 31 bits, the difference cancels to at most 24), so comparing
// d with s / 2 decides.  E4M3: ties have at most five significant bits, so a t
// whose 19 low bits are within four of zero goes through a 64-bit quotient
// (exact enough: two products of 11 and 29 bits that differ, differ by 2^-33).
// Bound by memory for prompts (2 bytes read and 1 written per value), by latency
// for a decode step (slots, then x and the scale, then the codes).
#include "common.cuh"
#include "kernels.h"

namespace qnt {
namespace {

constexpr int kApWarps = 8;            // token rows of a window, warps of a CTA
constexpr int kApShort = 8;            // longest run that one warp takes

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
// y rounded towards zero, its last bit set if that was inexact: any later
// rounding to 22 bits or fewer is then that of y.
__device__ __forceinline__ float to_odd(double y) {
  const float t = __double2float_rz(y);
  return (double)t != y ? __uint_as_float(__float_as_uint(t) | 1u) : t;
}

// x / s -> code byte, x and s scaled alike by a power of two, inv = 1 / s.
__device__ __forceinline__ uint32_t int8_byte(float x, float s, float inv, float half) {
  float q = rintf(x * inv);
  const float d = fmaf(-q, s, x);
  const bool odd = ((int)q & 1) != 0;
  if (d > half || (d == half && odd)) q += 1.0f;
  else if (d < -half || (d == -half && odd)) q -= 1.0f;
  return (uint32_t)((int)fminf(fmaxf(q, -127.0f), 127.0f) + 128);
}
__device__ __forceinline__ float e4m3_quotient(float x, float s, float inv) {
  float t = x * inv;
  if (((__float_as_uint(t) + 4u) & 0x7FFFFu) < 9u && t != 0.0f) t = to_odd((double)x / (double)s);
  return t;
}

template <int FMT>
__device__ __forceinline__ uint32_t requant_byte(uint32_t b, double s0, double s) {
  if (FMT == QNT_KV_INT8) {
    const double q = rint((double)((int)b - 128) * s0 / s);
    return (uint32_t)((int)q + 128);
  }
  return e4m3x2(to_odd((double)e4m3_value(b) * s0 / s), 0.0f) & 0xFFu;
}

// A run or a warp's share of one: tokens t, t + step, ... of the rows
// [t, end), IT rounds of TPL tokens; a lane holds eight values of a token.
template <bool BF16, int D, int IT>
struct Share {
  static constexpr int LPT = D / 8;            // lanes of a token
  uint4 v[IT];
  float top;
  bool bad;
  __device__ __forceinline__ void load(const uint16_t* x, int64_t stride, int t, int end, int step, int lane) {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int tok = t + i * step + lane / LPT;
      v[i] = tok < end ? ldg_cg128(x + (int64_t)tok * stride + 8 * (lane % LPT)) : make_uint4(0, 0, 0, 0);
    }
  }
  static __device__ __forceinline__ float2 pair(uint32_t w) {
    if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return make_float2(h2f(w & 0xFFFFu), h2f(w >> 16));
  }
  // max |x| of the finite values, over the warp
  __device__ __forceinline__ void reduce() {
    top = 0.0f;
    bad = false;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 p = pair(w[j]);
        const float a = fabsf(p.x), b = fabsf(p.y);
        const bool fa = a < __int_as_float(0x7F800000), fb = b < __int_as_float(0x7F800000);
        bad |= !fa || !fb;
        top = fmaxf(top, fmaxf(fa ? a : 0.0f, fb ? b : 0.0f));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  // codes of the tokens: `out` is the run's first token's place, row0 its token row
  template <int FMT>
  __device__ __forceinline__ void store(uint8_t* out, int row0, float s, int t, int end, int step, int lane) const {
    // scales below 2^-100 are scaled up, with x, so that 1 / s and the remainders stay normal
    const float up = s < 7.888609e-31f ? 1.2089258e24f : 1.0f;
    const float su = s * up, inv = s > 0.0f ? 1.0f / su : 0.0f, half = 0.5f * su;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int tok = t + i * step + lane / LPT;
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t o[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 p = pair(w[j]);
        p.x *= up;
        p.y *= up;
        uint32_t b;
        if (FMT == QNT_KV_INT8) {
          b = s > 0.0f ? int8_byte(p.x, su, inv, half) | (int8_byte(p.y, su, inv, half) << 8) : 0x8080u;
        } else {
          // a NaN quotient (x not finite, or s = 0) becomes 0: the cache holds no NaN
          const float qx = s > 0.0f ? e4m3_quotient(p.x, su, inv) : 0.0f, qy = s > 0.0f ? e4m3_quotient(p.y, su, inv) : 0.0f;
          b = e4m3x2(qx == qx ? qx : 0.0f, qy == qy ? qy : 0.0f);
        }
        o[j >> 1] |= b << (16 * (j & 1));
      }
      if (tok < end) *reinterpret_cast<uint2*>(out + (int64_t)(tok - row0) * D + 8 * (lane % LPT)) = make_uint2(o[0], o[1]);
    }
  }
};

struct Growth { int64_t base; int bytes; };   // codes to map with a warp's table

template <int FMT, bool BF16, int D>
__global__ void __launch_bounds__(32 * kApWarps) kv_append_kernel(const KvAppendArgs A) {
  __shared__ uint8_t lut[kApWarps][256];
  __shared__ Growth grow[kApWarps];
  __shared__ int long_row, long_end;
  __shared__ float tops[kApWarps];
  constexpr int TPL = 32 / (D / 8);
  constexpr float kTop = FMT == QNT_KV_INT8 ? 127.0f : 448.0f;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y, kv = blockIdx.z;
  const int row = blockIdx.x * kApWarps + warp;
  if (tid == 0) long_row = -1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();

  const int P = A.page;
  const long long limit = (long long)A.pages * P;
  uint8_t* const codes = kv ? A.codes[1] : A.codes[0];
  float* const scales = kv ? A.scales[1] : A.scales[0];
  const uint16_t* const x = static_cast<const uint16_t*>(kv ? A.x[1] : A.x[0]) + (int64_t)h * D;
  auto slot_at = [&](int r) -> int { return r >= 0 && r < A.tokens ? A.slots[r] : -1; };
  auto place = [&](int slot) -> int64_t {          // first byte of a slot's values
    return (((int64_t)(slot / P) * A.heads + h) * P + slot % P) * D;
  };
  // the run's final scale; a larger one than the page had goes on record
  auto settle = [&](int slot, float top, float& s0) -> float {
    const float s_new = top / kTop;
    float* const sp = scales + (int64_t)(slot / P) * A.heads + h;
    s0 = slot % P ? *sp : 0.0f;
    __syncwarp();
    const float s = fmaxf(s_new, s0);
    if (lane == 0) *sp = s;
    return s;
  };
  auto tabulate = [&](int w, float s0, float s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = 8 * lane + i;
      lut[w][b] = (uint8_t)requant_byte<FMT>(b, s0, s);
    }
  };

  // does this warp's row begin a run, and where does the run end?
  const int slot = slot_at(row);
  int prev = slot_at(row - 1);
  const bool next_to = prev >= 0;
  bool head = slot >= 0 && slot < limit;
  // a page's token rows with only skipped rows in between are found out, too
  for (int at = row - 2; head && prev < 0 && at >= 0; at -= 256) {
    int found = -1;
#pragma unroll
    for (int i = 7; i >= 0; --i) {                           // rows at - 255 .. at, the nearest counts
      const int v = slot_at(at - 32 * i - lane);
      if (v >= 0) found = 32 * i + lane;
    }
    const int nearest = __reduce_min_sync(0xffffffffu, found < 0 ? 256 : found);
    if (nearest < 256) prev = slot_at(at - nearest);
  }
  if (slot >= limit && lane == 0 && h == 0) report(A.status, QNT_ERR_ARG);
  if (head && prev >= 0 && prev / P == slot / P) {           // the row before is of the same page:
    head = false;                                            // the run goes on from there,
    if (!(next_to && prev + 1 == slot) && lane == 0 && h == 0) report(A.status, QNT_ERR_ARG);   // or this is a second one
  }
  int end = row;
  if (head) {
    const int most = P - slot % P;                           // to the end of the page
    end = row + 1;
    for (int k = 1; k < most; k += 32) {
      const bool on = k + lane < most && slot_at(row + k + lane) == slot + k + lane;
      const uint32_t m = __ballot_sync(0xffffffffu, on);
      end += __ffs(~m) ? __ffs(~m) - 1 : 32;
      if (~m) break;
    }
    if (end - row > kApShort && lane == 0) {
      long_row = row;
      long_end = end;
    }
  }
  if (lane == 0) grow[warp].bytes = 0;
  if (head && end - row <= kApShort) {
    Share<BF16, D, (kApShort + TPL - 1) / TPL> sh;
    sh.load(x, A.stride, row, end, TPL, lane);
    sh.reduce();
    if (sh.bad) report(A.status, QNT_ERR_NONFINITE);
    float s0;
    const float s = settle(slot, sh.top, s0);
    sh.template store<FMT>(codes + place(slot), row, s, row, end, TPL, lane);
    if (slot % P && s > s0) {
      tabulate(warp, s0, s);
      if (lane == 0) grow[warp] = {place(slot - slot % P), (slot % P) * D};
    }
  }
  __syncthreads();
  if (long_row >= 0) {
    // the CTA's warps take TPL tokens each, in turn
    constexpr int IT = 128 / (kApWarps * TPL);
    const int r0 = long_row, e0 = long_end, first = A.slots[r0];
    const int t = r0 + warp * TPL;
    Share<BF16, D, IT> sh;
    sh.load(x, A.stride, t, e0, kApWarps * TPL, lane);
    sh.reduce();
    if (sh.bad) report(A.status, QNT_ERR_NONFINITE);
    if (lane == 0) tops[warp] = sh.top;
    float* const sp = scales + (int64_t)(first / P) * A.heads + h;
    const float s0 = first % P ? *sp : 0.0f;
    __syncthreads();                                         // every warp has read the old scale
    float top = 0.0f;
#pragma unroll
    for (int w = 0; w < kApWarps; ++w) top = fmaxf(top, tops[w]);
    const float s = fmaxf(top / kTop, s0);
    if (tid == 0) *sp = s;
    sh.template store<FMT>(codes + place(first), r0, s, t, e0, kApWarps * TPL, lane);
    const int owner = long_row % kApWarps;
    if (first % P && s > s0 && warp == owner) {
      tabulate(owner, s0, s);
      if (lane == 0) grow[owner] = {place(first - first % P), (first % P) * D};
    }
    __syncthreads();
  }
  // the tokens before a run whose page's scale grew, 16 codes a thread and step
  for (int w = 0; w < kApWarps; ++w) {
    const Growth g = grow[w];
    for (int i = tid * 16; i < g.bytes; i += 32 * kApWarps * 16) {
      uint4* const p = reinterpret_cast<uint4*>(codes + g.base + i);
      const uint4 v = *p;
      uint32_t in[4] = {v.x, v.y, v.z, v.w}, out[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        out[j] = (uint32_t)lut[w][in[j] & 255u] | ((uint32_t)lut[w][(in[j] >> 8) & 255u] << 8) |
                 ((uint32_t)lut[w][(in[j] >> 16) & 255u] << 16) | ((uint32_t)lut[w][in[j] >> 24] << 24);
      *p = make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
}

template <int FMT, bool BF16, int D>
cudaError_t ap_launch(const KvAppendArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.tokens + kApWarps - 1) / kApWarps, a.heads, 2);
  cfg.blockDim = dim3(32 * kApWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_append_kernel<FMT, BF16, D>, a);
}

template <int FMT, bool BF16>
cudaError_t ap_dim(int dim, const KvAppendArgs& a, cudaStream_t s) {
  switch (dim) {
    case 64: return ap_launch<FMT, BF16, 64>(a, s);
    case 128: return ap_launch<FMT, BF16, 128>(a, s);
    default: return ap_launch<FMT, BF16, 256>(a, s);
  }
}

}  // namespace

cudaError_t launch_kv_append(const qnt_kv_desc& d, const KvAppendArgs& a, int xbf16, cudaStream_t s) {
  if (d.fmt == QNT_KV_INT8) return xbf16 ? ap_dim<QNT_KV_INT8, true>(d.dim, a, s) : ap_dim<QNT_KV_INT8, false>(d.dim, a, s);
  return xbf16 ? ap_dim<QNT_KV_E4M3, true>(d.dim, a, s) : ap_dim<QNT_KV_E4M3, false>(d.dim, a, s);
}

}  // namespace qnt
