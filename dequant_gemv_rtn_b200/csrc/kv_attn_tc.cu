// kv_attn_tc.cu -- attention of many query rows over the paged 8-bit key/value
// cache on the 5th-generation tensor cores (qnt_kv_attn; definition in
// include/qnt.h): requests whose new tokens x query heads of a key/value head are
// many rows, that is prompt chunks and long drafts on shared heads.
//
// With 128 rows every cached byte meets 256 flops and more, so the tensor cores,
// the exponentials (128 x 128 of them a tile at 16 a cycle take as long as the
// tile's two products) and the issue slots bound the kernel, not memory.
//
//  * A CTA takes up to two tiles of 128 query rows ("streams"; one at dim 256) of
//    one key/value head through 128 cached tokens at a time.  Both streams use the
//    same decoded tokens, and while one's softmax runs the other's products do.
//  * Four warps decode: codes from global memory to registers a tile ahead, to
//    fp16 (exact: INT8 by a byte permute into 0x64xx minus 1152, E4M3 by the
//    conversion instruction), to shared memory in the 128-byte-swizzled layout.
//    K is the K-major operand B of S = Q K^T; V, stored alike (64 values of a
//    token a line), is the MN-major operand B of O += P V.  No transposition.
//  * S of a stream goes to 128 columns of tensor memory; P overwrites S there and is
//    the A operand of O += P V; O stays in tensor memory.  A thread of the stream's
//    first softmax warp issues its MMAs, which has nothing else to do by then.
//  * Four warps per stream do the softmax, a thread a row, 32 columns at a time in
//    two loops (the maximum; the weights), packed fp32 arithmetic taking two logits
//    at once.  Only if one passes the reference by 8 is the reference moved and O
//    rescaled before its next product.  Logits beyond 2^20 take a loop more (with the
//    choice inside the loop of the weights every call was 6 % slower).
//  * Scales: K's multiplies the row's factor, per 16 tokens (a page or a part of
//    one).  V's goes into the exponent: the weight that meets V's codes is
//    2^(x - m + log2(vs) - u), and a page's share of the sum is taken back by
//    2^(u - log2 vs) once per 16 tokens.  u is the largest V scale of the tile, within
//    a factor of two: beyond that u moves and O is rescaled, as for the maximum.
//    With the 2^6 that every weight carries (what the slack of the reference and of u
//    leaves of fp16's range; it cancels with the sum) a weight has fp16's 11 bits down
//    to 2^-20 of the reference and u, and below that an absolute error of 2^-31 of
//    them, 2^-30 of the tile's largest scale.
//    Two limits keep both factors in fp32's range, since scales may differ by 2^270:
//    a page's values do not count below 2^-40 of u (2^(u - log2 vs) would overflow, and
//    its weights vanish from the sum), and u does not fall below 2^-64 of the highest
//    it had (O, whose weights of then may be all that counts, would overflow) nor below
//    2^-100 (2^u, and that over the sum of weights, would be 0).
//  * Work is cut into equal parts of tiles of all requests, one per CTA, as in
//    kv_attn.cu, here with each row tile's own causal range.
//
// Measured on two chunks of 1024 tokens, the cache 5000 and 8000 long (32 / 8 heads,
// dim 128, INT8): 301 us, 668 TFLOP/s (the mma.sync kernel: 1268 us); 297 without the
// limits on the unit and the way of large logits.  Then a tile took 5100 cycles, of
// which a stream's maximum 800, its weights 2200 (the other stream's turn meanwhile is
// over or not begun) and its two products 1500.  Slower were, in
// us: the loops over a tile's columns unrolled, with the row in registers (437 to
// 570: instruction fetch), one pass with the weights corrected where the maximum
// moved (359), no turns (371 against 343 then), two threads a row (400 and, with
// the registers that leaves, 595), decoding in the softmax warps (743: the streams
// wait for each other), a warp of its own for the MMAs (404).  A split job costs its
// last CTA about 2 us a part (160 rows); two chunks of 40 tokens take 64 us.
//
// Every wait is bounded (2 s); on expiry the kernel reports QNT_ERR_TIMEOUT, every
// role runs through without waiting, and tensor memory is freed after the last MMA.
#include <climits>
#include "kv_attn.cuh"
#include "tc.cuh"

namespace qnt {
namespace {

constexpr int kKtRows = 128;                 // query rows of a stream, tensor-memory lanes
constexpr int kKtTok = 128;                  // cached tokens of a tile
constexpr int kKtGroups = kKtTok / 16;       // runs of 16 tokens: one page each
constexpr int kKtCtrl = 5120;                // barriers, scales, the warps' jobs
constexpr int kKtScaleRing = 4;
constexpr int kKtSlots = 2048;               // where the warps' jobs begin
// A weight at the reference is held as 2^kKtBias; a new reference is at most kKaSlack
// behind the maximum, and the unit at most kKtNear behind a tile's: 2^15 in all, which fp16 takes.
constexpr float kKtBias = 6.0f, kKtNear = 1.0f;
static_assert(kKtBias + kKaSlack + kKtNear <= 15.0f, "weights in fp16");
// log2 of V scales: below the unit by more than kKtNone a page's values do not count;
// the unit stays within kKtFall of the highest it had, and above kKtLowest.
constexpr float kKtNone = 40.0f, kKtFall = 64.0f, kKtLowest = -100.0f;
constexpr uint32_t kKtCols = 512;
constexpr unsigned long long kKtTimeoutNs = 2000000000ull;

template <int D> struct Kt {
  static constexpr int NS = D == 256 ? 1 : 2;             // streams
  static constexpr int ST = D == 256 ? 1 : 2;             // stages of K and of V
  static constexpr int SoftWarps = 4 * NS;               // a thread a row
  static constexpr int Warps = SoftWarps + 4;            // then the decode warps
  static constexpr int Threads = 32 * Warps;
  static constexpr int Tile = 128 * D * 2;                // bytes of an fp16 operand tile
  static constexpr int Smem = kKtCtrl + Tile * (NS + 2 * ST);
  // tensor memory: S (and P) of stream s at 128 s, O behind
  static constexpr int ColO = 128 * NS;
  static_assert(ColO + NS * D <= (int)kKtCols, "tensor memory");
};

struct KtRow { int first, n, len, rows, tiles; long long all, per_head; };
struct KtTile { int t_first, t_last, seen, begin, end, units; };   // seen: the first token that a row sees

// Tokens that the rows [row0, row0 + cap) of a request see.
__device__ __forceinline__ KtTile kt_tile(const KvAttnArgs& A, const KtRow& w, int row0, int cap) {
  KtTile t;
  t.t_first = token_of(A, row0);
  t.t_last = token_of(A, min(w.rows, row0 + cap) - 1);
  const int base = w.len - w.n;
  t.seen = A.window ? max(base + t.t_first + 1 - A.window, 0) : 0;
  t.begin = t.seen & ~15;
  t.end = min(w.len, base + t.t_last + 1);
  t.units = max(1, (t.end - t.begin + kKtTok - 1) / kKtTok);
  return t;
}
template <int CAP>
__device__ __forceinline__ KtRow kt_row(const KvAttnArgs& A, int b) {
  KtRow w;
  w.first = min(max(A.cu[b], 0), A.tokens);
  w.n = min(max(A.cu[b + 1], w.first), A.tokens) - w.first;
  w.len = min(max(A.len[b], 0), A.width << A.page_log2);
  const long long rows = (long long)w.n * A.group;
  w.rows = rows > A.narrow ? (int)min(rows, (long long)0x7FFFFFFF) : 0;
  w.tiles = (w.rows + CAP - 1) / CAP;
  w.per_head = 0;
  for (int j = 0; j < w.tiles; ++j) w.per_head += kt_tile(A, w, j * CAP, CAP).units;
  w.all = w.per_head * A.heads;
  return w;
}

// One job of a CTA: a group of query rows and the tiles [u0, u1) of its tokens.
struct KtJob {
  int h, row0, rows, base, u0, u1;
  KtTile t;
  long long u_first;        // the job's first unit among all
};
// Walks a CTA's part of the units; every role walks it alike.
template <int CAP>
struct KtWalk {
  int b;
  long long pos, hi, off;
  KtRow w;
  __device__ __forceinline__ bool next(const KvAttnArgs& A, KtJob& j) {
    if (pos >= hi) return false;
    while (off >= w.all) {
      off -= w.all;
      w = kt_row<CAP>(A, ++b);
    }
    j.h = (int)div_units(off, w.per_head);
    int u = (int)(off - j.h * w.per_head), k = 0;
    for (;; ++k) {
      j.t = kt_tile(A, w, k * CAP, CAP);
      if (u < j.t.units) break;
      u -= j.t.units;
    }
    j.row0 = k * CAP;
    j.rows = min(CAP, w.rows - j.row0);
    j.base = w.len - w.n;
    j.u0 = u;
    j.u1 = (int)min((long long)j.t.units, u + (hi - pos));
    j.u_first = pos - u;
    pos += j.u1 - j.u0;
    off += j.u1 - j.u0;
    return true;
  }
};

// A warp's walk, in shared memory: the roles have no registers to spare for it.
template <int CAP>
struct KtSlot { KtWalk<CAP> walk; KtJob job; int more; };

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_addr(bar)) : "memory");
}
// D[128 x N] (+)= A[128 x 16] (shared memory) * B[16 x N] (shared memory)
__device__ __forceinline__ void tc_mma_smem_a(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%5, %5, %5, %5}, p;\n\t}"
      :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(0u) : "memory");
}
// MN-major operand with 128-byte swizzle: lines of 64 values of one k, eight k
// 1024 bytes apart, blocks of 64 values `block` bytes apart.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr, uint32_t block) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((block >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// Packed fp32 pairs (one rounding each).
__device__ __forceinline__ uint64_t pair_u32(uint32_t a, uint32_t b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint64_t pair_f32(float a, float b) { return pair_u32(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ void unpair_f32(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// One lane of the (converged) warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// A logit's factor; never 0, since it meets -infinity.
constexpr float kKtLeast = 1e-37f;
__device__ __forceinline__ float factor(float row, float scale) { return fmaxf(row * scale, kKtLeast); }

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* d) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]), "=r"(d[4]), "=r"(d[5]), "=r"(d[6]), "=r"(d[7]),
        "=r"(d[8]), "=r"(d[9]), "=r"(d[10]), "=r"(d[11]), "=r"(d[12]), "=r"(d[13]), "=r"(d[14]), "=r"(d[15]),
        "=r"(d[16]), "=r"(d[17]), "=r"(d[18]), "=r"(d[19]), "=r"(d[20]), "=r"(d[21]), "=r"(d[22]), "=r"(d[23]),
        "=r"(d[24]), "=r"(d[25]), "=r"(d[26]), "=r"(d[27]), "=r"(d[28]), "=r"(d[29]), "=r"(d[30]), "=r"(d[31])
      : "r"(taddr) : "memory");
}
// The loads into d have arrived (d: what the wait orders).
__device__ __forceinline__ void tmem_wait_ld32(uint32_t* d) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3]), "+r"(d[4]), "+r"(d[5]), "+r"(d[6]), "+r"(d[7]),
                 "+r"(d[8]), "+r"(d[9]), "+r"(d[10]), "+r"(d[11]), "+r"(d[12]), "+r"(d[13]), "+r"(d[14]), "+r"(d[15]),
                 "+r"(d[16]), "+r"(d[17]), "+r"(d[18]), "+r"(d[19]), "+r"(d[20]), "+r"(d[21]), "+r"(d[22]), "+r"(d[23]),
                 "+r"(d[24]), "+r"(d[25]), "+r"(d[26]), "+r"(d[27]), "+r"(d[28]), "+r"(d[29]), "+r"(d[30]), "+r"(d[31])
               :: "memory");
}

// Sixteen codes of one token -> 32 bytes of fp16, in order.
template <int FMT>
__device__ __forceinline__ void decode16(uint4 c, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (FMT == QNT_KV_INT8) {                 // 0x6400 + byte = 1024 + byte; byte - 128 = that - 1152
      o[2 * j] = hsub2(prmt(w[j], 0x64646464u, 0x4140u), 0x64806480u);
      o[2 * j + 1] = hsub2(prmt(w[j], 0x64646464u, 0x4342u), 0x64806480u);
    } else {
      o[2 * j] = e4m3x2_f16(w[j]);
      o[2 * j + 1] = e4m3x2_f16_hi(w[j]);
    }
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Byte of 16-byte piece p (of a row of D fp16 values) of row r in an operand tile:
// blocks of 64 values, 128-byte rows, pieces swizzled by the row.
__device__ __forceinline__ uint32_t tile_at(int r, int p) {
  return (uint32_t)((p >> 3) * (128 * 128) + r * 128 + (((p & 7) ^ (r & 7)) << 4));
}

template <int FMT, bool BF16, int D>
__global__ void __launch_bounds__(Kt<D>::Threads, 1) kv_attn_tc_kernel(const KvAttnArgs A) {
  using T = Kt<D>;
  constexpr int NS = T::NS, ST = T::ST, CAP = kKtRows * NS;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* const k_full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* const k_empty = k_full + 2;
  uint64_t* const v_full = k_full + 4;
  uint64_t* const v_empty = k_full + 6;
  uint64_t* const s_full = k_full + 8;      // S of the stream is in tensor memory
  uint64_t* const p_full = k_full + 10;     // P is, and S and O are read
  uint64_t* const o_full = k_full + 12;     // the job's last product is complete
  uint64_t* const q_full = k_full + 14;     // Q is in shared memory, O of the job before is read
  uint64_t* const drained = k_full + 16;
  uint32_t* const tbase_p = reinterpret_cast<uint32_t*>(smem + 160);
  volatile int* const abort_s = reinterpret_cast<volatile int*>(smem + 164);
  int* const last_s = reinterpret_cast<int*>(smem + 168);
  int* const start_b = reinterpret_cast<int*>(smem + 172);
  long long* const start_off = reinterpret_cast<long long*>(smem + 176);
  long long* const part = reinterpret_cast<long long*>(smem + 192);                // a sum per warp
  float4* const scales_s = reinterpret_cast<float4*>(smem + 512);                  // [ring][group]: K's, log2 of V's
  const uint32_t q_s = smem_addr(smem + kKtCtrl), k_s = q_s + NS * T::Tile, v_s = k_s + ST * T::Tile;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);     // (so that the compiler knows it as uniform)

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init_nofence(k_full + i, 4);
      mbar_init_nofence(k_empty + i, NS);
      mbar_init_nofence(v_full + i, 4);
      mbar_init_nofence(v_empty + i, NS);
      mbar_init_nofence(s_full + i, 2);
      mbar_init_nofence(p_full + i, 4);
      mbar_init_nofence(o_full + i, 1);
      mbar_init_nofence(q_full + i, 4);
    }
    mbar_init_nofence(drained, NS);
    mbar_init_fence();
    *abort_s = 0;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_addr(tbase_p)), "r"(kKtCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }

  // ---- the call's units and this CTA's part of them
  const int per = (A.rows + T::Threads - 1) / T::Threads;
  const int b0 = min(tid * per, A.rows), b1 = min(b0 + per, A.rows);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += kt_row<CAP>(A, b).all;
  long long end = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end += v;
  }
  if (lane == 31) part[warp] = end;
  __syncthreads();
  tc_fence_after();
  long long total = 0;
  for (int w = 0; w < T::Threads / 32; ++w) {
    if (w < warp) end += part[w];
    total += part[w];
  }
  const long long ctas = min((long long)gridDim.x, total);
  const bool busy = blockIdx.x < ctas;
  const KaParts parts(total, ctas);
  const long long lo = busy ? parts.begin(blockIdx.x) : 0, hi = busy ? parts.begin(blockIdx.x + 1) : 0;
  if (busy && lo >= end - mine && lo < end) {
    long long at = end - mine;
    int b = b0;
    for (;; ++b) {
      const long long all = kt_row<CAP>(A, b).all;
      if (lo < at + all) break;
      at += all;
    }
    *start_b = b;
    *start_off = lo - at;
  }
  __syncthreads();
  static_assert(kKtSlots + sizeof(KtSlot<CAP>) * (T::Threads / 32) <= (size_t)kKtCtrl, "control area");
  KtSlot<CAP>& slot = reinterpret_cast<KtSlot<CAP>*>(smem + kKtSlots)[warp];
  const KtJob& job = slot.job;
  if (lane == 0) {
    slot.walk.pos = lo;
    slot.walk.hi = hi;
    if (busy) {
      slot.walk.b = *start_b;
      slot.walk.w = kt_row<CAP>(A, *start_b);
      slot.walk.off = *start_off;
    }
  }
  auto next_job = [&]() {
    __syncwarp();
    if (lane == 0) slot.more = slot.walk.next(A, slot.job);
    __syncwarp();
    return slot.more != 0;
  };
  const uint32_t tbase = __shfl_sync(0xffffffffu, *tbase_p, 0);
  const int pl = A.page_log2, P = 1 << pl;

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (gt_wait(bar, parity & 1u, abort_s, A.timeout_ns, 0)) return true;
    if (!*abort_s) {
      *abort_s = 1;
      report(A.status, QNT_ERR_TIMEOUT);
    }
    return false;
  };

  if (warp < T::SoftWarps) {
    // ---------------------------------------------------------------- softmax, MMAs
    const int s = warp >> 2, r = 32 * (warp & 3) + lane;      // stream, row
    const bool issuing = (warp & 3) == 0;                     // one lane of the warp issues the stream's MMAs
    const uint32_t id_s = f16_idesc(kKtTok, 0), id_o = f16_idesc(D, 0) | (1u << 16);   // bit 16: B is MN-major
    const uint64_t q_desc = sw128_desc(q_s + (uint32_t)(s * T::Tile));
    const uint32_t col_s = tbase + 128u * (uint32_t)s, col_o = tbase + (uint32_t)(T::ColO + D * s);
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = col_s + lanes, to = col_o + lanes;
    uint32_t tiles = 0, jobs = 0, it = 0;                     // of this stream; of the CTA
    bool alone = false;                                       // the other stream has no rows
    auto free_stage = [&](uint64_t* bar) {                    // once the MMAs issued so far are complete
      tc_commit(bar);
      if (NS == 2 && alone) tc_commit(bar);
    };
    auto qk = [&](uint32_t t) {                               // S = Q K^T of the CTA's tile t
      const uint32_t stage = t % ST;
      if (!wait(k_full + stage, t / ST)) return false;
      tc_fence_after();
      const uint64_t k_desc = sw128_desc(k_s + stage * T::Tile);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t at = (uint32_t)((kk >> 2) * (128 * 128) + 32 * (kk & 3)) >> 4;
        tc_mma_smem_a(col_s, q_desc + at, k_desc + at, id_s, kk > 0);
      }
      tc_commit(s_full + s);
      mbar_arrive(s_full + s);                                // hands on what the decode warps wrote (scales)
      free_stage(k_empty + stage);
      return true;
    };
    auto pv = [&](uint32_t t, bool first) {                   // O (+)= P V
      const uint32_t stage = t % ST;
      if (!wait(v_full + stage, t / ST)) return false;
      tc_fence_after();
      const uint64_t v_desc = sw128_mn_desc(v_s + stage * T::Tile, 128 * 128);
#pragma unroll
      for (int kk = 0; kk < kKtTok / 16; ++kk)
        tc_mma_tmem_a(col_o, col_s + 8u * (uint32_t)kk, v_desc + 128u * (uint32_t)kk, id_o, !first || kk > 0);
      free_stage(v_empty + stage);
      return true;
    };
    auto soft_sync = [&]() {                                  // all softmax warps, each of them whole
      __syncwarp();
      asm volatile("bar.sync 1, %0;" :: "r"(32 * T::SoftWarps) : "memory");
    };
    while (next_job()) {
      const int ntiles = job.u1 - job.u0;
      const int row = job.row0 + kKtRows * s + r;             // query row of the request's head
      const bool live = kKtRows * s + r < job.rows;
      const bool on = kKtRows * s < job.rows;                 // the stream has rows
      alone = job.rows <= kKtRows;
      const int t = token_of(A, row), hq = job.h * A.group + row - t * A.group;
      float m = kKaFloor, l = 0.0f, unit = 0.0f, highest = 0.0f;
      bool has_unit = false, far = false, ok = true;
      if (on) {
        // Q in fp16, bf16 rows scaled by a power of two; a negative factor goes into Q
        const uint16_t* const src = static_cast<const uint16_t*>(A.q) + (int64_t)(slot.walk.w.first + t) * A.q_stride + (int64_t)hq * D;
        float up = 1.0f, down = 1.0f;
        uint4 v[D / 8];                                       // the whole row at once: one wait for memory
#pragma unroll
        for (int p = 0; p < D / 8; ++p) v[p] = live ? ldg_cg128(src + 8 * p) : make_uint4(0, 0, 0, 0);
        if (BF16) {
          float top = 0.0f;
#pragma unroll
          for (int p = 0; p < D / 8; ++p) {
            const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
          }
          f16_range(top, up, down);
        }
        const uint32_t flip = A.scale_log2 < 0.0f ? 0x80008000u : 0u;
#pragma unroll
        for (int p = 0; p < D / 8; ++p) {
          uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (BF16) w[i] = pack_f16(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
            w[i] ^= flip;
          }
          sts128(q_s + (uint32_t)(s * T::Tile) + tile_at(r, p), make_uint4(w[0], w[1], w[2], w[3]));
        }
        const float c0 = fabsf(A.scale_log2) * down;
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full + s);
        if (issuing && elect_one()) ok = wait(q_full + s, jobs) && qk(it);
        __syncwarp();
        const int sees = live ? job.base + t : -1;
        // a tile has something to hide if it ends behind all_see or begins at or before hidden
        const int all_see = job.base + token_of(A, job.row0 + kKtRows * s);
        const int hidden = A.window ? job.base + token_of(A, job.row0 + min(job.rows, kKtRows * (s + 1)) - 1) - A.window : INT_MIN;
        int tok0 = job.t.begin + job.u0 * kKtTok;

        // two streams compute their weights in turn: while one does, the other's products
        // run (both at once finish at once, and then both wait for their products)
        const bool turns = !alone;
        auto turn_wait = [&]() {
          if (turns) asm volatile("bar.sync %0, 256;" :: "r"(2 + s) : "memory");
        };
        auto turn_pass = [&](int i) {
          if (turns && (s == 0 || i + 1 < ntiles)) asm volatile("bar.arrive %0, 256;" :: "r"(3 - s) : "memory");
        };
        if (turns && s == 1) asm volatile("bar.arrive 2, 256;" ::: "memory");
        for (int i = 0; i < ntiles; ++i, ++tiles, ++it, tok0 += kKtTok) {
          ok = __all_sync(0xffffffffu, ok && wait(s_full + s, tiles));
          if (!ok) {
            turn_wait();
            turn_pass(i);
            continue;
          }
          tc_fence_after();
          const float4* const sc = scales_s + (it % kKtScaleRing) * (kKtGroups + 1);
          const bool edge = tok0 + kKtTok - 1 > all_see || tok0 <= hidden;
          uint32_t x[2][32];
          tmem_ld32(ts, x[0]);
          // the unit of the tile's weights, from its largest V scale
          float grow = 1.0f;
          const float lv = sc[kKtGroups].y;
          if (lv > -INFINITY) {
            if (!has_unit) {
              unit = highest = fmaxf(lv, kKtLowest);
              has_unit = true;
            } else if (fabsf(lv - unit) > kKtNear) {
              highest = fmaxf(highest, lv);
              const float next = fmaxf(fmaxf(lv, kKtLowest), highest - kKtFall);
              grow = exp2_approx(unit - next);
              unit = next;
            }
          }
          auto hide = [&](uint32_t (&v)[32], int q) {          // what the row does not see becomes -infinity
            const int hi_k = sees - tok0 - 32 * q, lo_k = A.window ? hi_k - A.window : INT_MIN;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (k > hi_k || k <= lo_k) v[k] = 0xFF800000u;
          };
          // the tile's maximum, 32 columns at a time, before the stream's turn
          float top = -INFINITY;
#pragma unroll 1
          for (int q2 = 0; q2 < kKtTok / 32; q2 += 2) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int q = q2 + b;
              uint32_t(&v)[32] = x[b];
              tmem_wait_ld32(v);
              if (q + 1 < kKtTok / 32) tmem_ld32(ts + 32u * (uint32_t)(q + 1), x[b ^ 1]);
              if (edge) hide(v, q);
              float most[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                most[k] = __uint_as_float(v[8 * k]);
#pragma unroll
                for (int j = 1; j < 8; ++j) most[k] = fmaxf(most[k], __uint_as_float(v[8 * k + j]));
              }
              top = fmaxf(top, fmaxf(fmaxf(most[0], most[1]) * factor(c0, sc[2 * q].x), fmaxf(most[2], most[3]) * factor(c0, sc[2 * q + 1].x)));
            }
          }
          tmem_ld32(ts, x[0]);
          float alpha = 1.0f;
          if (__any_sync(0xffffffffu, top > m + (kKaSlack + kKtBias))) {
            const float next = fmaxf(m, top - kKtBias);       // m: the reference, less the bias
            alpha = exp2_approx(m - next);
            m = next;
            far = __any_sync(0xffffffffu, fabsf(m) > 1048576.0f && fabsf(m) < -kKaFloor);   // neither unset nor infinite
          }
          // Beyond 2^20 a logit's product with its factor is rounded as the maximum's was before
          // the reference is taken off (an exact product and a rounded one may differ by any
          // number there).  S becomes that difference, apart from the loop below.
          float row_c = c0, least_c = kKtLeast, at = m;
          if (far) {
#pragma unroll 1
            for (int q = 0; q < kKtTok / 32; ++q) {
              if (q) tmem_ld32(ts + 32u * (uint32_t)q, x[0]);
              tmem_wait_ld32(x[0]);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                x[0][k] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(x[0][k]), factor(c0, sc[2 * q + k / 16].x)), m));
              tmem_st16(ts + 32u * (uint32_t)q, *reinterpret_cast<uint32_t(*)[16]>(x[0]));
              tmem_st16(ts + 32u * (uint32_t)q + 16u, *reinterpret_cast<uint32_t(*)[16]>(x[0] + 16));
            }
            tmem_wait_st();
            tmem_ld32(ts, x[0]);
            row_c = at = 0.0f;
            least_c = 1.0f;
          }
          // the weights; P's columns 16 q .. 16 q + 15 lie in S's that are read already
          turn_wait();
          float sum = 0.0f;
#pragma unroll 1
          for (int q2 = 0; q2 < kKtTok / 32; q2 += 2) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int q = q2 + b;
              uint32_t(&v)[32] = x[b];
              tmem_wait_ld32(v);
              if (q + 1 < kKtTok / 32) tmem_ld32(ts + 32u * (uint32_t)(q + 1), x[b ^ 1]);
              if (edge) hide(v, q);
              uint32_t p[16];
#pragma unroll
              for (int h2 = 0; h2 < 2; ++h2) {
                const float2 f = *reinterpret_cast<const float2*>(sc + 2 * q + h2);
                const float c = fmaxf(row_c * f.x, least_c);  // factor(c0, f.x)
                const bool none = f.y < unit - kKtNone;       // V's scale is 0, or nearly: the weights count, the values do not
                const float ref = none ? at : at - (f.y - unit);
                const uint64_t c2 = pair_f32(c, c), ref2 = pair_f32(-ref, -ref);
                float e[16];
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                  unpair_f32(fma_f32x2(pair_u32(v[16 * h2 + k], v[16 * h2 + k + 1]), c2, ref2), e[k], e[k + 1]);
                  e[k] = exp2_approx(e[k]);
                  e[k + 1] = exp2_approx(e[k + 1]);
                }
                uint64_t part0 = pair_f32(e[0], e[1]), part1 = pair_f32(e[2], e[3]);
#pragma unroll
                for (int k = 4; k < 16; k += 4) {
                  part0 = add_f32x2(part0, pair_f32(e[k], e[k + 1]));
                  part1 = add_f32x2(part1, pair_f32(e[k + 2], e[k + 3]));
                }
                float s0, s1;
                unpair_f32(add_f32x2(part0, part1), s0, s1);
                sum = fmaf(s0 + s1, none ? 1.0f : exp2_approx(unit - f.y), sum);
#pragma unroll
                for (int k = 0; k < 16; k += 2) p[8 * h2 + k / 2] = none ? 0u : pack_f16(e[k], e[k + 1]);
              }
              tmem_st16(ts + 16u * (uint32_t)q, p);
            }
          }
          turn_pass(i);
          l = fmaf(l, alpha, sum);
          const float by = alpha * grow;
          if (i > 0 && __any_sync(0xffffffffu, by != 1.0f)) {  // O, whose products are complete
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(to + (uint32_t)c, o);
              tmem_wait_ld32(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * by);
              tmem_st16(to + (uint32_t)c, *reinterpret_cast<uint32_t(*)[16]>(o));
              tmem_st16(to + (uint32_t)c + 16u, *reinterpret_cast<uint32_t(*)[16]>(o + 16));
            }
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + s);
          if (issuing && elect_one()) {
            ok = wait(p_full + s, tiles) && pv(it, i == 0);
            if (i + 1 == ntiles) tc_commit(o_full + s);
            else ok = ok && qk(it + 1);
          }
          __syncwarp();
        }
        ok = __all_sync(0xffffffffu, ok && wait(o_full + s, jobs));
        ++jobs;
        tc_fence_after();
      } else {
        it += ntiles;
      }
      // ---- the row's result, or the CTA's part of it
      const bool whole = job.u0 == 0 && job.u1 == job.t.units;
      constexpr int PART = CAP * (D + 2);
      float* const partials = reinterpret_cast<float*>(static_cast<uint8_t*>(A.work) + kKaCounters);
      uint16_t* const y = static_cast<uint16_t*>(A.y);
      auto out_at = [&](int rr) {                             // place of the job's row rr in y
        const int q = job.row0 + rr, tt = token_of(A, q);
        return y + (int64_t)(slot.walk.w.first + tt) * A.y_stride + (int64_t)(job.h * A.group + q - tt * A.group) * D;
      };
      if (on && ok) {
        const float f = whole ? exp2_approx(unit) * inv_sum(l) : exp2_approx(unit);
        float* const mypart = partials + (size_t)(2 * blockIdx.x + (job.u0 == 0 ? 1 : 0)) * PART;
        const int rr = kKtRows * s + r;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(to + (uint32_t)c, o);
          tmem_wait_ld32(o);
          if (live) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(o[k + e]) * f;
              const float4 a = make_float4(v[0], v[1], v[2], v[3]), z = make_float4(v[4], v[5], v[6], v[7]);
              if (whole) {
                const uint2 x = pack_out<BF16>(a), w = pack_out<BF16>(z);
                *reinterpret_cast<uint4*>(out_at(rr) + c + k) = make_uint4(x.x, x.y, w.x, w.y);
              } else {
                __stcg(reinterpret_cast<float4*>(mypart + rr * D + c + k), a);
                __stcg(reinterpret_cast<float4*>(mypart + rr * D + c + k + 4), z);
              }
            }
          }
          __syncwarp();                                       // the next load needs the whole warp
        }
        if (!whole && live) {
          __stcg(mypart + CAP * D + rr, m);
          __stcg(mypart + CAP * D + CAP + rr, l);
        }
        tc_fence_before();
      }
      if (!whole) {
        // the CTAs first .. last share the job; the one that arrives last merges
        uint32_t* const counters = static_cast<uint32_t*>(A.work);
        const int first = parts.cta_of(job.u_first), last = parts.cta_of(job.u_first + job.t.units - 1);
        __threadfence();
        soft_sync();
        if (tid == 0) {
          const uint32_t before = atomicAdd(counters + first, 1u);
          *last_s = before == (uint32_t)(last - first);
          if (*last_s) counters[first] = 0;                   // ready for the next call
          __threadfence();
        }
        soft_sync();
        if (*last_s) {
          auto at = [&](int c) { return partials + (size_t)(2 * c + (c == first ? 1 : 0)) * PART; };
          constexpr int TH = 32 * T::SoftWarps;                 // a thread per row
          constexpr int FIT = T::Tile * NS / (4 * CAP);         // parts whose factors fit in Q's place
          float* const f_s = reinterpret_cast<float*>(smem + kKtCtrl);   // [part][row]
          const int n = last - first + 1;
          float top = kKaFloor, sum = 0.0f;                     // of row tid
          auto batch = [&](int c0, int most, bool keep) {       // 16 parts' references and sums, in flight together
            float pm[16], ps[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float* const src = at(first + min(c0 + k, most - 1)) + CAP * D + tid;
              pm[k] = __ldcg(src);
              ps[k] = __ldcg(src + CAP);
            }
            float next = top;
#pragma unroll
            for (int k = 0; k < 16; ++k) next = fmaxf(next, pm[k]);
            sum *= exp2_approx(top - next);
            top = next;
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (c0 + k < most) {
                sum = fmaf(exp2_approx(pm[k] - top), ps[k], sum);
                if (keep) f_s[(c0 + k) * CAP + tid] = pm[k];
              }
          };
          const bool mine_row = tid < job.rows;
          if (mine_row)
            for (int c = 0; c < n; c += 16) batch(c, n, c + 16 <= FIT);
          const float inv = inv_sum(sum);
          constexpr int U = 8;                                  // pieces of four values that a thread has in flight
          for (int c0 = 0; c0 < n; c0 += FIT) {                 // (one round, unless there are more parts)
            const int cn = min(FIT, n - c0);
            if (c0) soft_sync();
            if (mine_row)
              for (int c = 0; c < cn; ++c) {
                const float pm = c0 ? __ldcg(at(first + c0 + c) + CAP * D + tid) : f_s[c * CAP + tid];
                f_s[c * CAP + tid] = exp2_approx(pm - top) * inv;
              }
            soft_sync();
            for (int x0 = tid; x0 < job.rows * (D / 4); x0 += U * TH) {
              float4 v[U];
#pragma unroll
              for (int u = 0; u < U; ++u) {
                v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                const int x = x0 + u * TH;
                if (c0 && x < job.rows * (D / 4)) v[u] = *reinterpret_cast<const float4*>(at(first) + 4 * x);
              }
#pragma unroll 2
              for (int c = 0; c < cn; ++c) {
                const float* const src = at(first + c0 + c);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                  const int x = min(x0 + u * TH, job.rows * (D / 4) - 1);
                  const float f = f_s[c * CAP + x / (D / 4)];
                  const float4 o = __ldcg(reinterpret_cast<const float4*>(src + 4 * x));
                  v[u] = make_float4(fmaf(f, o.x, v[u].x), fmaf(f, o.y, v[u].y), fmaf(f, o.z, v[u].z), fmaf(f, o.w, v[u].w));
                }
              }
#pragma unroll
              for (int u = 0; u < U; ++u) {
                const int x = x0 + u * TH, rr = x / (D / 4), d = 4 * (x % (D / 4));
                if (x >= job.rows * (D / 4)) break;
                if (c0 + cn < n) *reinterpret_cast<float4*>(at(first) + 4 * x) = v[u];   // goes on in the next round
                else *reinterpret_cast<uint2*>(out_at(rr) + d) = pack_out<BF16>(v[u]);
              }
            }
          }
          soft_sync();   // last_s is read
        }
      } else if (NS == 2 && alone) {
        // the stream without rows skipped the job's tiles: it may go on when the other has
        // taken them, since a wait by parity tells a stage's use only from the one before
        soft_sync();
      }
    }
    if (issuing && elect_one()) tc_commit(drained);           // arrives once every MMA issued has completed
  } else {
    // ---------------------------------------------------------------- decode
    const int dw = warp - T::SoftWarps;
    constexpr int CPT = D / 16, NCH = CPT;                    // 16-byte pieces of a token, of a thread
    // a thread's pieces are TPI tokens apart.  Lane -> piece and token so that eight
    // lanes' 16-byte stores meet eight banks: four even (odd) pieces of a token and of
    // the next, which the swizzle sets apart
    constexpr int TPI = 128 / CPT, CB = D == 64 ? 0 : D == 128 ? 1 : 2;   // CB: log2(CPT) - 2
    const int my_c = (lane & 3) | (((lane >> 3) & ((1 << CB) - 1)) << 2);
    const int my_tok = dw * (32 / CPT) + (((lane >> 2) & 1) | ((lane >> (3 + CB)) << 1));
    uint4 kreg[NCH], vreg[NCH];
    int page[NCH];
    float2 sc = make_float2(0.0f, 0.0f);                      // first warp: scales of the tile's runs of 16 tokens
    uint32_t it = 0;
    bool ok = true;
    auto load_pages = [&](const int32_t* table, int h, int tok0, int seen, int end) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int tok = tok0 + my_tok + TPI * i;
        page[i] = tok < end && tok >= seen ? table[tok >> pl] : -1;   // what no row sees may be NaN: not read
      }
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (tok0 + my_tok + TPI * i < end && tok0 + my_tok + TPI * i >= seen && (unsigned)page[i] >= (unsigned)A.pages) page[i] = 0;
      if (dw == 0) {
        const int tok = tok0 + 16 * lane;
        sc = make_float2(0.0f, 0.0f);
        if (lane < kKtGroups && tok < end) {
          int p = table[tok >> pl];
          if ((unsigned)p >= (unsigned)A.pages) {
            p = 0;
            report(A.status, QNT_ERR_ARG);
          }
          const int64_t ph = (int64_t)p * A.heads + h;
          sc = make_float2(A.kscales[ph], A.vscales[ph]);
        }
      }
    };
    auto load = [&](const uint8_t* codes, int h, int tok0, uint4 (&reg)[NCH]) {
      const uint8_t* const head = codes + ((int64_t)h << pl) * D + 16 * my_c;
      const int64_t step = ((int64_t)A.heads << pl) * D;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int tok = tok0 + my_tok + TPI * i;
        reg[i] = page[i] >= 0 ? ldg_cg128(head + page[i] * step + (tok & (P - 1)) * D) : make_uint4(0, 0, 0, 0);
      }
    };
    auto store = [&](uint32_t tile, const uint4 (&reg)[NCH]) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        uint4 lo4, hi4;
        decode16<FMT>(reg[i], lo4, hi4);
        sts128(tile + tile_at(my_tok + TPI * i, 2 * my_c), lo4);
        sts128(tile + tile_at(my_tok + TPI * i, 2 * my_c + 1), hi4);
      }
    };
    while (next_job()) {
      const int ntiles = job.u1 - job.u0;
      const int32_t* const table = A.table + (size_t)slot.walk.b * A.width;
      int tok0 = job.t.begin + job.u0 * kKtTok;
      const int end_tok = job.t.end, seen_tok = job.t.seen, h = job.h;
      load_pages(table, h, tok0, seen_tok, end_tok);
      load(A.kcodes, h, tok0, kreg);
      load(A.vcodes, h, tok0, vreg);
      for (int i = 0; i < ntiles; ++i, ++it, tok0 += kKtTok) {
        const uint32_t stage = it % ST, use = it / ST;
        if (use) ok = ok && wait(k_empty + stage, use - 1);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          if (dw == 0) {                                      // K's scale and log2 of V's; behind the runs' the largest of these
            float lv = sc.y > 0.0f ? log2f(sc.y) : -INFINITY, most = lv;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            if (lane == kKtGroups) lv = most;
            if (lane <= kKtGroups) scales_s[(it % kKtScaleRing) * (kKtGroups + 1) + lane] = make_float4(sc.x, lv, 0.0f, 0.0f);
          }
          store(k_s + stage * T::Tile, kreg);
          fence_proxy_async();
          __syncwarp();
#ifdef QNT_TEST_FAULTS
          // fault 1 (test builds): in CTA 0 a decode warp never reports the first tile of K
          const bool skip = A.fault == 1 && blockIdx.x == 0 && it == 0 && dw == 1;
#else
          constexpr bool skip = false;
#endif
          if (lane == 0 && !skip) mbar_arrive(k_full + stage);
          if (i + 1 < ntiles) {
            load_pages(table, h, tok0 + kKtTok, seen_tok, end_tok);
            load(A.kcodes, h, tok0 + kKtTok, kreg);
          }
        }
        if (use) ok = ok && wait(v_empty + stage, use - 1);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          store(v_s + stage * T::Tile, vreg);
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(v_full + stage);
          if (i + 1 < ntiles) load(A.vcodes, h, tok0 + kKtTok, vreg);
        }
      }
    }
  }
  // teardown: every MMA issued has completed before tensor memory is freed
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) gt_wait(drained, 0, nullptr, kKtTimeoutNs, 64);
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tbase), "r"(kKtCols) : "memory");
  }
}

#ifdef QNT_TEST_FAULTS
static thread_local int t_kt_fault = 0;
static thread_local unsigned long long t_kt_timeout_ns = kKtTimeoutNs;
#define QNT_KT_FAULT t_kt_fault
#define QNT_KT_TIMEOUT t_kt_timeout_ns
#else
#define QNT_KT_FAULT 0
#define QNT_KT_TIMEOUT kKtTimeoutNs
#endif

template <int FMT, bool BF16, int D>
cudaError_t kt_launch(const KvAttnArgs& a, cudaStream_t s) {
  auto kfn = kv_attn_tc_kernel<FMT, BF16, D>;
  cudaError_t e = configure_smem(reinterpret_cast<const void*>(kfn));
  if (e != cudaSuccess) return e;
  // one CTA per SM: more than half of its shared memory, since each takes all of tensor memory
  constexpr int smem = Kt<D>::Smem > 120 * 1024 ? Kt<D>::Smem : 120 * 1024;
  static_assert(smem <= kMaxDynSmem, "shared memory");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms());
  cfg.blockDim = dim3(Kt<D>::Threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kfn, a);
}

template <int FMT, bool BF16>
cudaError_t kt_dim(int dim, const KvAttnArgs& a, cudaStream_t s) {
  switch (dim) {
    case 64: return kt_launch<FMT, BF16, 64>(a, s);
    case 128: return kt_launch<FMT, BF16, 128>(a, s);
    default: return kt_launch<FMT, BF16, 256>(a, s);
  }
}

}  // namespace

size_t kv_attn_tc_part_bytes(int dim) { return (size_t)kKtRows * (dim == 256 ? 1 : 2) * (dim + 2) * 4; }

#ifdef QNT_TEST_FAULTS
void set_test_attn_fault(int fault, unsigned long long timeout_ns) {
  t_kt_fault = fault;
  t_kt_timeout_ns = timeout_ns;
}
#endif

cudaError_t launch_kv_attn_tc(const qnt_kv_desc& d, KvAttnArgs a, int xbf16, cudaStream_t s) {
  a.timeout_ns = QNT_KT_TIMEOUT;
  a.fault = QNT_KT_FAULT;
  if (d.fmt == QNT_KV_INT8) return xbf16 ? kt_dim<QNT_KV_INT8, true>(d.dim, a, s) : kt_dim<QNT_KV_INT8, false>(d.dim, a, s);
  return xbf16 ? kt_dim<QNT_KV_E4M3, true>(d.dim, a, s) : kt_dim<QNT_KV_E4M3, false>(d.dim, a, s);
}

}  // namespace qnt
