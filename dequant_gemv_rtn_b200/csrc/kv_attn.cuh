// kv_attn.cuh -- what the two attention kernels share (kv_attn.cu: few query rows
// of a key/value head; kv_attn_tc.cu: many).
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace qnt {

constexpr size_t kKaCounters = 16384;             // workspace: counters in front of the partial results
constexpr float kKaFloor = -3e38f;                // reference of the softmax before the first token, below any logit
constexpr float kKaSlack = 8.0f;                  // log2 of the largest weight: the reference moves when one passes it

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// Two E4M3 bytes (the low / high half of w) as an fp16 pair, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(w));
  return d;
}
__device__ __forceinline__ uint32_t e4m3x2_f16_hi(uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(d) : "r"(w));
  return d;
}
// A bf16 row whose largest magnitude is `top` times up = 2^k has it in
// [2^14, 2^15), an fp16 number; down = 2^-k.
__device__ __forceinline__ void f16_range(float top, float& up, float& down) {
  const int e = (int)((__float_as_uint(top) >> 23) & 255u);
  const int k = e == 0 || e == 255 ? 0 : min(max(14 - (e - 127), -126), 126);
  up = __uint_as_float((uint32_t)(127 + k) << 23);
  down = __uint_as_float((uint32_t)(127 - k) << 23);
}
// Four values of an output row in its type.
template <bool BF16>
__device__ __forceinline__ uint2 pack_out(float4 v) {
  if (!BF16) return make_uint2(pack_f16(v.x, v.y), pack_f16(v.z, v.w));
  const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), z = __floats2bfloat162_rn(v.z, v.w);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&z));
}
// 1 / sum of the weights; 0 for a row that sees nothing.
__device__ __forceinline__ float inv_sum(float sum) { return sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum; }

// n / d: 64-bit divisions take ten times as long and are rarely needed.
__device__ __forceinline__ long long div_units(long long n, long long d) {
  return ((n | d) >> 32) == 0 ? (long long)((uint32_t)n / (uint32_t)d) : n / d;
}
// `total` units cut into parts for `ctas` CTAs, the first ones a unit longer.
struct KaParts {
  long long each, longer;       // units of a part; CTAs with one more
  __device__ __forceinline__ KaParts(long long total, long long ctas) {
    each = ctas ? div_units(total, ctas) : 0;
    longer = total - each * ctas;
  }
  __device__ __forceinline__ long long begin(long long c) const { return c * each + min(c, longer); }
  __device__ __forceinline__ int cta_of(long long u) const {   // whose part holds unit u
    const long long split = longer * (each + 1);
    return (int)(u < split ? div_units(u, each + 1) : longer + div_units(u - split, each));
  }
};
// Query row -> token and back: row / group, group = A.group.
__device__ __forceinline__ int token_of(const KvAttnArgs& A, int row) {
  return A.group == 1 ? row : (int)(__umulhi((uint32_t)row, A.group_mul) >> A.group_shift);
}

// The wide kernel (kv_attn_tc.cu): requests of more than `narrow` query rows a head.
size_t kv_attn_tc_part_bytes(int dim);            // a partial result
cudaError_t launch_kv_attn_tc(const qnt_kv_desc& d, KvAttnArgs a, int xbf16, cudaStream_t s);

}  // namespace qnt
