// kv_attn.cu -- attention of a decode step's new tokens over the paged 8-bit
// key/value cache (qnt_kv_attn; layout and definition in include/qnt.h).
//
// y = sum_j p_j v_j / sum_j p_j, p_j = 2^(x_j - m), x_j = log2(e) scale q.k_j, in
// one pass over the cache with a running reference m (flash decoding).  The
// cache bytes are read once and bound the kernel: 2 dim bytes per token and
// key/value head against 4 dim flops per query row, so up to 8 or 16 query rows
// (the query heads of a key/value head x the new tokens) share every byte.
//
//  * Tensor cores, transposed: S^T = K Q^T with 16 tokens as the rows of an
//    m16n8k16 MMA and 8 query rows as its columns, O^T = V^T P^T with 16 values
//    of dim as the rows.  The 8-bit operand is always A: a decoded register
//    serves every group of 8 query rows, and with 8 rows nothing is padding.
//    K's and Q's order along dim within an MMA is free as long as it is the
//    same, so lane (g, r) of a quad row takes 16 consecutive bytes of tokens g
//    and g + 8 (one 16-byte load each, four MMAs), and V's 16 rows are the
//    dim / 8 consecutive bytes that lane group g holds of four tokens.  Nothing
//    passes through shared memory; P^T is S^T packed to fp16 and transposed 8 x 8
//    by movmatrix.
//  * Decoding: an INT8 byte is q + 128, and a zero-extended byte is the fp16
//    subnormal (q + 128) 2^-24: one byte permute per two codes.  The 128 comes off
//    as the MMA's initial value (-128 sum of q) for S and as 128 sum of p for O,
//    whose sums are another MMA with an operand of ones.  E4M3 goes through the
//    hardware conversion.  Both are exact.  The scale of K multiplies S; the
//    products with V are summed page by page and multiplied into O in fp32, so a
//    page's scale, however small or large, costs no precision.
//  * p is rounded to fp16 for the second product (relative error 2^-11, which
//    averages out over tokens; the sum uses the rounded values).  m follows the
//    maximum only when a logit passes it by 8, decided by one vote.  Every p carries
//    2^7, what that leaves of fp16's range (it cancels with the sum): full precision
//    down to 2^-21 of the reference, below that an absolute error of 2^-32 of it.
//  * Work: units of 16 or 32 tokens a warp of one (request, key/value head, group of
//    query rows), in one row of all units of the call, cut into equal parts,
//    one per CTA.  So requests of very unlike length keep every SM busy, and
//    which part is whose follows from d_cu and d_len on the device.  A CTA's
//    warps take the tokens of its part in turn and are merged in shared memory; a
//    (request, head) that spans several CTAs is merged by the one that arrives
//    last (one counter), in CTA order, so the result does not depend on timing.
//
// Measured (B200): 64 requests of 8192 tokens on 8 heads of 128 (64 query heads),
// E4M3: 178 us, 6.06 TB/s; lengths from 1 to 16384: 190 to 196 us, 5.6 TB/s; one request
// of 131072, INT8: 53 us, 5.1 TB/s.  One of 700 tokens on 32 heads: 8.4 us, of which 1.4
// is the schedule, 3 until the first bytes are there, 1 the tokens, 2.5 publishing
// and merging six parts a head.
#include <climits>
#include "kv_attn.cuh"

namespace qnt {
namespace {

constexpr int kKaBatch = 10;                      // parts of a split job that a thread reads at once
constexpr int kKaMaxPerSm = 4;                    // CTAs per SM of any variant
// A weight at the reference is held as 2^kKaBias; with the slack of the reference 2^15 in all.
constexpr float kKaBias = 7.0f;
static_assert(kKaBias + kKaSlack <= 15.0f, "weights in fp16");
// INT8 logits come in units of 2^-24.  The row's factor takes 2^16 of that and K's scale 2^8,
// so that neither overflows where bf16 queries or keys do not.
constexpr float kKaRowUp = 65536.0f, kKaScaleUp = 256.0f;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// Four consecutive codes of one token: (0, 1) and (2, 3).
template <int FMT>
__device__ __forceinline__ void decode_k(uint32_t w, uint32_t& a, uint32_t& b) {
  if (FMT == QNT_KV_INT8) {
    a = prmt(w, 0u, 0x4140u);
    b = prmt(w, 0u, 0x4342u);
  } else {
    a = e4m3x2_f16(w);
    b = e4m3x2_f16_hi(w);
  }
}
// Four consecutive codes of tokens s and t: (s0, t0), (s1, t1), (s2, t2), (s3, t3).
template <int FMT>
__device__ __forceinline__ void decode_v(uint32_t s, uint32_t t, uint32_t (&o)[4]) {
  if (FMT == QNT_KV_INT8) {
    const uint32_t x = prmt(s, t, 0x5410u), y = prmt(s, t, 0x7632u);
    o[0] = x & 0x00FF00FFu;
    o[1] = prmt(x, 0u, 0x4341u);
    o[2] = y & 0x00FF00FFu;
    o[3] = prmt(y, 0u, 0x4341u);
  } else {
    const uint32_t x = prmt(s, t, 0x5140u), y = prmt(s, t, 0x7362u);
    o[0] = e4m3x2_f16(x);
    o[1] = e4m3x2_f16_hi(x);
    o[2] = e4m3x2_f16(y);
    o[3] = e4m3x2_f16_hi(y);
  }
}

// What a request asks of the kernel.
struct KaRow {
  int first, n, len;           // first token row, new tokens, cached tokens
  int seen, begin;             // first token that a row sees, first token of the work
  int tiles;                   // groups of query rows
  int units;                   // units of one (head, group)
  long long all;
};
template <int ROWS, int UNIT>
__device__ __forceinline__ KaRow ka_row(const KvAttnArgs& A, int b) {
  KaRow w;
  w.first = min(max(A.cu[b], 0), A.tokens);
  w.n = min(max(A.cu[b + 1], w.first), A.tokens) - w.first;
  w.len = min(max(A.len[b], 0), A.width << A.page_log2);
  w.seen = A.window ? max(w.len - w.n + 1 - A.window, 0) : 0;
  w.begin = w.seen & ~15;      // no page before the window is looked up
  w.tiles = (int)(((long long)w.n * A.group + ROWS - 1) / ROWS);
  w.units = max(1, (w.len - w.begin + UNIT - 1) / UNIT);
  w.all = (long long)w.n * A.group > A.narrow ? 0 : (long long)w.tiles * w.units * A.heads;
  return w;
}

template <int FMT, bool BF16, int D, int NR, int W, int PER_SM>
__global__ void __launch_bounds__(32 * W, PER_SM) kv_attn_kernel(const KvAttnArgs A) {
  constexpr int kKaWarps = W, kKaThreads = 32 * W;
  constexpr int ROWS = 8 * NR;                              // query rows of a CTA
  constexpr int TT = D == 256 ? 16 : 32;                    // tokens of a warp's step
  constexpr int NB = TT / 16;
  constexpr int UNIT = kKaWarps * TT;
  constexpr int C = D / 64;                                 // 16-byte pieces of a K token that a lane holds
  constexpr int VB = D / 8, VW = VB / 4;                    // bytes / words of a V token that a lane holds
  constexpr int MT = D / 16;                                // m-tiles of O^T
  constexpr int LD = D + 4;
  extern __shared__ __align__(16) float sm[];
  float* const o_s = sm + 64;                               // [kKaWarps][ROWS][LD]
  float* const m_s = o_s + kKaWarps * ROWS * LD;            // [kKaWarps][ROWS]
  float* const l_s = m_s + kKaWarps * ROWS;
  long long* const part = reinterpret_cast<long long*>(sm); // a sum per warp, in the first 64 words
  long long& start_off = part[16];
  int& start_row = reinterpret_cast<int*>(sm)[34];
  int& last_s = reinterpret_cast<int*>(sm)[35];
  static_assert(W <= 16, "scan scratch");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, r = lane & 3;
  const int pl = A.page_log2, P = 1 << pl;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- the call's units, and this CTA's part [lo, hi) of them
  const int per = (A.rows + kKaThreads - 1) / kKaThreads;
  const int b0 = min(tid * per, A.rows), b1 = min(b0 + per, A.rows);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    mine += ka_row<ROWS, UNIT>(A, b).all;
    if (blockIdx.x == 0 && (A.len[b] < 0 || A.len[b] > A.width << pl)) report(A.status, QNT_ERR_ARG);
  }
  long long end = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end += v;
  }
  if (lane == 31) part[warp] = end;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kKaWarps; ++w) {
    if (w < warp) end += part[w];
    total += part[w];
  }
  if (total == 0) return;
  const long long ctas = min((long long)gridDim.x, total);
  if (blockIdx.x >= ctas) return;
  const KaParts parts(total, ctas);
  const long long lo = parts.begin(blockIdx.x), hi = parts.begin(blockIdx.x + 1);
  if (lo >= end - mine && lo < end) {
    long long at = end - mine;
    int b = b0;
    for (;; ++b) {
      const long long all = ka_row<ROWS, UNIT>(A, b).all;
      if (lo < at + all) break;
      at += all;
    }
    start_row = b;
    start_off = lo - at;
  }
  __syncthreads();

  uint32_t* const counters = static_cast<uint32_t*>(A.work);
  float* const partials = reinterpret_cast<float*>(static_cast<uint8_t*>(A.work) + kKaCounters);
  constexpr int PART = ROWS * (D + 2);                      // floats: O, m, l
  int b = start_row;
  KaRow w = ka_row<ROWS, UNIT>(A, b);
  long long off = start_off;                                // place in the request's units
  for (long long pos = lo; pos < hi;) {
    while (off >= w.all) {
      off -= w.all;
      w = ka_row<ROWS, UNIT>(A, ++b);
    }
    const int job = (int)div_units(off, w.units), u0 = (int)(off - (long long)job * w.units);
    const int u1 = (int)min((long long)w.units, u0 + (hi - pos));
    const int h = job / w.tiles, row0 = (job - h * w.tiles) * ROWS;
    const int rows = min(ROWS, w.n * A.group - row0);       // query rows of this job
    const int base = w.len - w.n;                           // position of the first new token
    const int t_first = token_of(A, row0), t_last = token_of(A, row0 + rows - 1);
    const int lo_tok = w.begin + u0 * UNIT;
    const int hi_tok = min(min(w.begin + u1 * UNIT, w.len), base + t_last + 1);   // behind the last that a row sees
    const int32_t* const table = A.table + (size_t)b * A.width;

    // ---- tokens, TT at a time
    int page[NB];
    auto load_pages = [&](int tk) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int tok = tk + 16 * nb;
        page[nb] = tok < hi_tok ? table[tok >> pl] : 0;
        if ((unsigned)page[nb] >= (unsigned)A.pages) {
          page[nb] = 0;
          if (lane == 0) report(A.status, QNT_ERR_ARG);
        }
      }
    };
    uint4 kreg[NB][2][C];
    float ks[NB];
    auto load_k = [&](int tk) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int tok = tk + 16 * nb;
        const int64_t ph = (int64_t)page[nb] * A.heads + h;
        const uint8_t* const p = A.kcodes + ((ph << pl) + (tok & (P - 1)) + g) * D + 16 * r;
        const bool on = tok < hi_tok;
        ks[nb] = on ? A.kscales[ph] : 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          kreg[nb][0][c] = on ? ldg_cg128(p + 64 * c) : make_uint4(0, 0, 0, 0);
          kreg[nb][1][c] = on ? ldg_cg128(p + 8 * D + 64 * c) : make_uint4(0, 0, 0, 0);
        }
      }
    };
    uint32_t vreg[NB][4][VW];
    float vs[NB];
    auto load_v = [&](int tk) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int tok = tk + 16 * nb;
        const int64_t ph = (int64_t)page[nb] * A.heads + h;
        const uint8_t* const p = A.vcodes + ((ph << pl) + (tok & (P - 1)) + 2 * r) * D + VB * g;
        const bool on = tok < hi_tok;
        vs[nb] = on ? A.vscales[ph] : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {                        // tokens 2r, 2r + 1, 2r + 8, 2r + 9
          const uint8_t* const s = p + ((i & 1) + 8 * (i >> 1)) * D;
          if constexpr (VB == 8) {
            const uint2 v = on ? ldg_cg64(s) : make_uint2(0, 0);
            vreg[nb][i][0] = v.x;
            vreg[nb][i][1] = v.y;
          } else {
#pragma unroll
            for (int k = 0; k < VW / 4; ++k) {
              const uint4 v = on ? ldg_cg128(s + 16 * k) : make_uint4(0, 0, 0, 0);
              vreg[nb][i][4 * k] = v.x;
              vreg[nb][i][4 * k + 1] = v.y;
              vreg[nb][i][4 * k + 2] = v.z;
              vreg[nb][i][4 * k + 3] = v.w;
            }
          }
        }
      }
    };

    // ---- the query rows as the MMAs' B operand, in fp16
    uint32_t q[NR][C][8];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      const int row = 8 * nr + g;
      const bool live = row < rows;
      const int t = token_of(A, row0 + row), hq = h * A.group + row0 + row - t * A.group;
      const uint16_t* const src = static_cast<const uint16_t*>(A.q) + (int64_t)(w.first + t) * A.q_stride + (int64_t)hq * D + 16 * r;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint4 x = live ? ldg_cg128(src + 64 * c) : make_uint4(0, 0, 0, 0);
        const uint4 z = live ? ldg_cg128(src + 64 * c + 8) : make_uint4(0, 0, 0, 0);
        q[nr][c][0] = x.x; q[nr][c][1] = x.y; q[nr][c][2] = x.z; q[nr][c][3] = x.w;
        q[nr][c][4] = z.x; q[nr][c][5] = z.y; q[nr][c][6] = z.z; q[nr][c][7] = z.w;
      }
    }
    // the first step's codes are requested before the queries have to be there
    int tk = lo_tok + warp * TT;
    load_pages(tk);
    load_k(tk);
    load_v(tk);
    load_pages(tk + UNIT);
    float c0[NR][2], init[NR][2];                           // rows 2r, 2r + 1: factor of the logits, -128 sum of q
    int sees[NR][2];                                        // last visible token
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      float factor = A.scale_log2;
      if (BF16) {
        // a power of two brings the row's largest |q| into [2^14, 2^15)
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(q[nr][c][i] << 16)), fabsf(__uint_as_float(q[nr][c][i] & 0xFFFF0000u))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float up, down;
        f16_range(top, up, down);
        factor *= top > 0.0f ? down : 0.0f;                 // (a query of zero may meet a scale of any size)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            q[nr][c][i] = pack_f16(__uint_as_float(q[nr][c][i] << 16) * up, __uint_as_float(q[nr][c][i] & 0xFFFF0000u) * up);
      }
      float sum = 0.0f;
      if (FMT == QNT_KV_INT8) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) sum += h2f(q[nr][c][i] & 0xFFFFu) + h2f(q[nr][c][i] >> 16);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        factor *= kKaRowUp;                                 // codes are q 2^-24
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {                          // row n's values are in the lanes with g = n
        c0[nr][i] = __shfl_sync(0xffffffffu, factor, (2 * r + i) * 4);
        init[nr][i] = FMT == QNT_KV_INT8 ? -128.0f / 16777216.0f * __shfl_sync(0xffffffffu, sum, (2 * r + i) * 4) : 0.0f;
        sees[nr][i] = base + token_of(A, row0 + 8 * nr + 2 * r + i);
      }
    }

    float o[NR][MT][4], l[NR][4], m[NR][2], corr[NR][2];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nr][i][k] = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) l[nr][k] = 0.0f;
      m[nr][0] = m[nr][1] = kKaFloor;
      corr[nr][0] = corr[nr][1] = 0.0f;
    }

    for (; tk < hi_tok; tk += UNIT) {
      // S^T = K Q^T
      float s[NB][NR][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          s[nb][nr][0] = s[nb][nr][2] = init[nr][0];
          s[nb][nr][1] = s[nb][nr][3] = init[nr][1];
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint32_t x[4] = {kreg[nb][0][c].x, kreg[nb][0][c].y, kreg[nb][0][c].z, kreg[nb][0][c].w};
          const uint32_t z[4] = {kreg[nb][1][c].x, kreg[nb][1][c].y, kreg[nb][1][c].z, kreg[nb][1][c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t a0, a1, a2, a3;
            decode_k<FMT>(x[i], a0, a2);
            decode_k<FMT>(z[i], a1, a3);
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) mma16816(s[nb][nr], a0, a1, a2, a3, q[nr][c][2 * i], q[nr][c][2 * i + 1]);
          }
        }
      }
      float ks_now[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) ks_now[nb] = FMT == QNT_KV_INT8 ? ks[nb] * kKaScaleUp : ks[nb];
      load_k(tk + UNIT);                                     // with the pages read a step ahead
      // base-2 logits, relative to the reference
      float over = 0.0f;
      const bool edge = tk + TT - 1 > base + t_first || (A.window && tk <= base + t_last - A.window);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[nb][nr][k] *= c0[nr][k & 1] * ks_now[nb];
      if (edge) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j = tk + 16 * nb + g + 8 * (k >> 1), p = sees[nr][k & 1];
              if (j > p || j >= w.len || (A.window && j <= p - A.window)) s[nb][nr][k] = -INFINITY;
            }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int k = 0; k < 4; ++k) over = fmaxf(over, s[nb][nr][k] - m[nr][k & 1]);
      if (__any_sync(0xffffffffu, over > kKaSlack + kKaBias)) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) top = fmaxf(top, fmaxf(s[nb][nr][i], s[nb][nr][i + 2]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            top = fmaxf(m[nr][i], top - kKaBias);            // m: the reference, less the bias
            const float alpha = exp2_approx(m[nr][i] - top);
            m[nr][i] = top;
            corr[nr][i] *= alpha;
            l[nr][i] *= alpha;
            l[nr][i + 2] *= alpha;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              o[nr][t][i] *= alpha;
              o[nr][t][i + 2] *= alpha;
            }
          }
      }
      // P^T as the B operand of O^T = V^T P^T
      uint32_t p[NB][NR][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) e[k] = exp2_approx(s[nb][nr][k] - m[nr][k & 1]);
          p[nb][nr][0] = transpose8x8(pack_f16(e[0], e[1]));
          p[nb][nr][1] = transpose8x8(pack_f16(e[2], e[3]));
        }
      if (FMT == QNT_KV_E4M3 && (tk + TT > w.len || tk < w.seen)) {   // bytes that no row sees may be NaN
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = tk + 16 * nb + 2 * r + (i & 1) + 8 * (i >> 1);
            if (j >= w.len || j < w.seen)
#pragma unroll
              for (int k = 0; k < VW; ++k) vreg[nb][i][k] = 0;
          }
      }
      const uint32_t one = 0x3C003C00u;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float f = FMT == QNT_KV_INT8 ? vs[nb] * 16777216.0f : vs[nb];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma16816(sum, one, one, one, one, p[nb][nr][0], p[nb][nr][1]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            l[nr][i] += sum[i];
            if (FMT == QNT_KV_INT8) corr[nr][i] += 128.0f * vs[nb] * sum[i];
          }
        }
#pragma unroll
        for (int k = 0; k < VW; ++k) {
          uint32_t a[4], c[4];
          decode_v<FMT>(vreg[nb][0][k], vreg[nb][1][k], a);
          decode_v<FMT>(vreg[nb][2][k], vreg[nb][3][k], c);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
              float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              mma16816(acc, a[2 * i], a[2 * i + 1], c[2 * i], c[2 * i + 1], p[nb][nr][0], p[nb][nr][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[nr][2 * k + i][e] = fmaf(acc[e], f, o[nr][2 * k + i][e]);
            }
        }
      }
      load_v(tk + UNIT);
      load_pages(tk + 2 * UNIT);
    }

    // ---- merge the warps
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 8 * nr + 2 * r + i;
        if (g == 0) {
          m_s[warp * ROWS + row] = m[nr][i];
          l_s[warp * ROWS + row] = l[nr][i];
        }
        float* const dst = o_s + (warp * ROWS + row) * LD + VB * g;
#pragma unroll
        for (int t = 0; t < MT; t += 2)
          *reinterpret_cast<float4*>(dst + 2 * t) = make_float4(o[nr][t][i] - corr[nr][i], o[nr][t][i + 2] - corr[nr][i],
                                                                o[nr][t + 1][i] - corr[nr][i], o[nr][t + 1][i + 2] - corr[nr][i]);
      }
    __syncthreads();
    auto put = [&](int row, int d, float4 v, float sum) {    // the row's output, four values from d
      const float f = inv_sum(sum);
      const int t = token_of(A, row0 + row), hq = h * A.group + row0 + row - t * A.group;
      const uint2 out = pack_out<BF16>(make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.y) + (int64_t)(w.first + t) * A.y_stride + (int64_t)hq * D + d) = out;
    };
    const bool whole = u0 == 0 && u1 == w.units;
    float* const mypart = partials + (size_t)(2 * blockIdx.x + (u0 == 0 ? 1 : 0)) * PART;
    for (int i = tid; i < rows * (D / 4); i += kKaThreads) {
      const int row = i / (D / 4), d = 4 * (i % (D / 4));
      float top = m_s[row];
#pragma unroll
      for (int k = 1; k < kKaWarps; ++k) top = fmaxf(top, m_s[k * ROWS + row]);
      float sum = 0.0f;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kKaWarps; ++k) {
        const float f = exp2_approx(m_s[k * ROWS + row] - top);
        const float4 x = *reinterpret_cast<const float4*>(o_s + (k * ROWS + row) * LD + d);
        sum = fmaf(f, l_s[k * ROWS + row], sum);
        v.x = fmaf(f, x.x, v.x);
        v.y = fmaf(f, x.y, v.y);
        v.z = fmaf(f, x.z, v.z);
        v.w = fmaf(f, x.w, v.w);
      }
      if (whole) {
        put(row, d, v, sum);
      } else {
        __stcg(reinterpret_cast<float4*>(mypart + row * D + d), v);
        if (d == 0) {
          __stcg(mypart + ROWS * D + row, top);
          __stcg(mypart + ROWS * D + ROWS + row, sum);
        }
      }
    }
    if (!whole) {
      // the CTAs first .. last share the job; the one that arrives last merges
      const long long u_first = pos - u0, u_last = u_first + w.units - 1;
      const int first = parts.cta_of(u_first), last = parts.cta_of(u_last);
      __syncthreads();
      if (tid == 0) {
        // releases what the CTA wrote, acquires what the others did
        uint32_t before;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(counters + first) : "memory");
        last_s = before == (uint32_t)(last - first);
        if (last_s) counters[first] = 0;                     // ready for the next call
      }
      __syncthreads();
      if (last_s) {
        auto at = [&](int c) { return partials + (size_t)(2 * c + (c == first ? 1 : 0)) * PART; };
        for (int i = tid; i < rows * (D / 4); i += kKaThreads) {
          const int row = i / (D / 4), d = 4 * (i % (D / 4));
          float top = kKaFloor, sum = 0.0f;
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int c = first; c <= last; c += kKaBatch) {     // a batch of parts is requested at once
            float pm[kKaBatch], pl_[kKaBatch];
            float4 po[kKaBatch];
#pragma unroll
            for (int k = 0; k < kKaBatch; ++k) {
              const float* const src = at(min(c + k, last));
              pm[k] = __ldcg(src + ROWS * D + row);
              pl_[k] = __ldcg(src + ROWS * D + ROWS + row);
              po[k] = __ldcg(reinterpret_cast<const float4*>(src + row * D + d));
            }
            float most = top;
#pragma unroll
            for (int k = 0; k < kKaBatch; ++k) most = fmaxf(most, pm[k]);
            const float by = exp2_approx(top - most);
            top = most;
            sum *= by;
            v = make_float4(v.x * by, v.y * by, v.z * by, v.w * by);
#pragma unroll
            for (int k = 0; k < kKaBatch; ++k) {
              const float f = c + k <= last ? exp2_approx(pm[k] - top) : 0.0f;
              sum = fmaf(f, pl_[k], sum);
              v = make_float4(fmaf(f, po[k].x, v.x), fmaf(f, po[k].y, v.y), fmaf(f, po[k].z, v.z), fmaf(f, po[k].w, v.w));
            }
          }
          put(row, d, v, sum);
        }
      }
    }
    __syncthreads();                                         // shared memory is free for the next job
    pos += u1 - u0;
    off += u1 - u0;
  }
}

template <int FMT, bool BF16, int D, int NR, int W, int PER_SM>
cudaError_t ka_launch_w(const KvAttnArgs& a, cudaStream_t s) {
  auto kfn = kv_attn_kernel<FMT, BF16, D, NR, W, PER_SM>;
  cudaError_t e = configure_smem(reinterpret_cast<const void*>(kfn));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms() * PER_SM);
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = 256 + (size_t)W * 8 * NR * (D + 4 + 2) * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kfn, a);
}
template <int FMT, bool BF16, int D, int NR>
cudaError_t ka_launch(const KvAttnArgs& a, long long rows, cudaStream_t s) {
  // 16 query rows of 128: two CTAs leave registers for steps of 32 tokens a warp, whose
  // loads are what keeps memory busy (64 rows of 16 query heads a head to 16384 tokens:
  // 252 us; three CTAs and steps of 16: 274; two and 16: 296).  24 rows a pass in two
  // CTAs' registers were slower than 16 in two passes (28 drafted rows, 8 heads: 76, 65).
  constexpr int PER_SM = D == 64 && NR == 1 ? 4 : D == 256 || (D == 128 && NR > 1) ? 2 : 3;
  static_assert(PER_SM <= kKaMaxPerSm, "workspace");
  // A few long jobs are cut into many parts each; one large CTA per SM then leaves a
  // third of the parts to merge (one row of 131072 tokens on 8 heads: 60 -> 53 us),
  // while with many jobs small CTAs overlap one's start and end with another's
  // tokens (64 rows on 8 heads: 193 us, large CTAs 224; 32 jobs: 8.9, 9.4).
  const long long tiles = (rows + 8 * NR - 1) / (8 * NR);
  if ((long long)a.rows * a.heads * tiles < 32) return ka_launch_w<FMT, BF16, D, NR, 4 * PER_SM, 1>(a, s);
  return ka_launch_w<FMT, BF16, D, NR, 4, PER_SM>(a, s);
}

template <int FMT, bool BF16>
cudaError_t ka_dim(int dim, const KvAttnArgs& a, long long rows, cudaStream_t s) {
  // up to 16 query rows share a pass where their accumulators fit in registers
  switch (dim) {
    case 64: return rows <= 8 ? ka_launch<FMT, BF16, 64, 1>(a, rows, s) : ka_launch<FMT, BF16, 64, 2>(a, rows, s);
    case 128: return rows <= 8 ? ka_launch<FMT, BF16, 128, 1>(a, rows, s) : ka_launch<FMT, BF16, 128, 2>(a, rows, s);
    default: return ka_launch<FMT, BF16, 256, 1>(a, rows, s);
  }
}

// Most query rows of a key/value head that this file's kernel takes; requests with
// more go to kv_attn_tc.cu's.  16 rows a pass cost a pass over the tokens each, the
// tcgen05 kernel costs the same up to 256 rows, but its few large jobs take longer to
// start and to merge.  So the border goes by the number of jobs (us here / there, 6500
// tokens, 8 heads): 2 requests of 48 rows 29 / 42, 96 rows 40 / 52, 128 rows 50 / 53;
// 16 requests of 48 rows 141 / 145, 64 rows 182 / 147, 96 rows 267 / 152; 16 requests
// of 35 rows on 4 heads, 3000 tokens, 58 / 60.  Those are all at dim 128; between 16
// and 128 jobs nothing was measured, and at dim 256, whose passes are of 8 rows, 16
// requests of 24 rows take 224 / 213, so the border is too high there.
constexpr int kKaNarrow = 32, kKaNarrowFewJobs = 96;
int ka_narrow(const KvAttnArgs& a) { return a.rows * a.heads >= 128 ? kKaNarrow : kKaNarrowFewJobs; }

}  // namespace

size_t kv_attn_work_bytes(const qnt_kv_desc& d, int heads, int max_new) {
  const size_t rows = d.dim == 256 ? 8 : 16;
  size_t parts = (size_t)num_sms() * kKaMaxPerSm * 2 * rows * (d.dim + 2) * 4;
  if ((long long)max_new * (heads / d.heads) > kKaNarrow) {
    const size_t wide = (size_t)num_sms() * 2 * kv_attn_tc_part_bytes(d.dim);
    if (wide > parts) parts = wide;
  }
  return kKaCounters + parts;
}

cudaError_t launch_kv_attn(const qnt_kv_desc& d, KvAttnArgs a, int max_new, int xbf16, cudaStream_t s) {
  long long rows = (long long)max_new * a.group;
  a.narrow = INT_MAX;
  // row / group by a product: mul = ceil(2^(32 + shift) / group), 2^shift < group <= 2^(shift + 1)
  for (a.group_shift = 0; (2 << a.group_shift) < a.group; ++a.group_shift) {}
  a.group_mul = a.group > 1 ? (uint32_t)((((uint64_t)1 << (32 + a.group_shift)) + a.group - 1) / a.group) : 0;
  if (rows > ka_narrow(a)) {
    a.narrow = ka_narrow(a);
    rows = a.narrow;
    const cudaError_t e = launch_kv_attn_tc(d, a, xbf16, s);
    if (e != cudaSuccess) return e;
  }
  if (d.fmt == QNT_KV_INT8)
    return xbf16 ? ka_dim<QNT_KV_INT8, true>(d.dim, a, rows, s) : ka_dim<QNT_KV_INT8, false>(d.dim, a, rows, s);
  return xbf16 ? ka_dim<QNT_KV_E4M3, true>(d.dim, a, rows, s) : ka_dim<QNT_KV_E4M3, false>(d.dim, a, rows, s);
}

}  // namespace qnt
