// kernels.h -- host-side entry points of the libqnt kernels (internal; the C
// ABI in qnt_abi.cu validates arguments and dispatches to these).
#pragma once
#include <cuda_runtime.h>
#include "qnt.h"

namespace qnt {

// Streaming multiprocessors of the current device (cached per device).
int num_sms();
// Dynamic shared memory that one CTA may request on sm_100.
constexpr int kMaxDynSmem = 227 * 1024;
// Raise a kernel's dynamic shared-memory limit once per process and device;
// later launches make no attribute calls, so they are safe inside stream capture.
cudaError_t configure_smem(const void* fn);

// RTN quantization (quantize.cu).
cudaError_t launch_quantize(const qnt_desc& d, const float* W, void* codes, void* meta, long z0, int* st,
                            cudaStream_t s);

// Y[m] = W x[m] for m < M on CUDA cores, any format (gemv.cu).
cudaError_t launch_gemv_simt(const qnt_desc& d, const void* codes, const void* meta, long z0, const void* X,
                             void* Y, int M, int xbf16, int* st, cudaStream_t s);

// y = W x for one activation vector, 4-bit formats, on the tensor cores with
// mma.sync straight from the packed codes (gemv1.cu).  *handled = false when it
// does not apply (the activation vector and a weight ring do not fit in shared
// memory).
cudaError_t launch_gemv4_one(const qnt_desc& d, const void* codes, const void* meta, long z0, const void* X, void* Y,
                             int xbf16, int* st, cudaStream_t s, bool* handled);

// Two to eight vectors of the 4-bit formats, group 128, K a multiple of 1024:
// the batch-1 kernel with the vectors sharing every MMA (gemv1.cu).
// *handled = false when the case is not covered or does not fit.
cudaError_t launch_gemv1_multi(const qnt_desc& d, const void* codes, const void* meta, const void* X, void* Y, int M,
                              int xbf16, int* st, cudaStream_t s, bool* handled);

// A sequence of batch-1 GEMVs (4-bit formats) in one cooperative launch
// (gemv1.cu); clears the workspace first.  *handled = false when the
// activation vector and a weight ring do not fit in shared memory.
cudaError_t launch_gemv_seq(const qnt_seq_step* steps, int n, int xbf16, void* work, int* st, cudaStream_t s,
                            bool* handled);

// qnt_gemv_seq with the completion counters in a library-owned device array
// (gemv1.cu); n <= QNT_SEQ_NOALLOC_MAX_STEPS.
cudaError_t launch_gemv_seq_noalloc(const qnt_seq_step* steps, int n, int xbf16, int* st, cudaStream_t s,
                                    bool* handled);

#ifdef QNT_TEST_FAULTS
// Test builds only (gemv1.cu): inject `fault` into this thread's next batch-1 /
// sequence launches and use `timeout_ns` as their wait limit.
void set_test_fault(int fault, unsigned long long timeout_ns);
// Test builds only (gemm_tc.cu): the same for this thread's next tcgen05 GEMM launches.
void set_test_gemm_fault(int fault, unsigned long long timeout_ns);
// Test builds only (kv_attn_tc.cu): the same for this thread's next tcgen05 attention launches.
void set_test_attn_fault(int fault, unsigned long long timeout_ns);
#endif

// An empty kernel: the next kernel in the stream cannot overlap the ones before it.
cudaError_t launch_stream_fence(cudaStream_t s);

// Y[m] = W x[m] for 1 <= M <= 128 on the tensor cores in one pass over the
// weights (gemm_tc.cu, 4-bit formats).  *handled = false when it does not apply.
cudaError_t launch_gemm_tc(const qnt_desc& d, const void* codes, const void* meta, long z0, const void* X, void* Y,
                           int M, int xbf16, int* st, cudaStream_t s, bool* handled);

// Page tables and slots (kv_slots.cu).
struct KvSlotsArgs {
  const int32_t *len, *add;
  int32_t *table, *free;
  const int32_t* free_count;
  int32_t *len_out, *cu, *slots, *free_count_out;
  int rows, width, tokens, page, pages;
  int* status;
};
cudaError_t launch_kv_slots(const KvSlotsArgs& a, cudaStream_t s);

// Quantizing write into the key/value cache (kv_append.cu); index 0: K, 1: V.
struct KvAppendArgs {
  uint8_t* codes[2];
  float* scales[2];
  const void* x[2];
  int64_t stride;
  const int32_t* slots;
  int tokens, page, pages, heads;
  int* status;
};
cudaError_t launch_kv_append(const qnt_kv_desc& d, const KvAppendArgs& a, int xbf16, cudaStream_t s);

// Attention over the key/value cache (kv_attn.cu, kv_attn_tc.cu).
struct KvAttnArgs {
  const uint8_t *kcodes, *vcodes;
  const float *kscales, *vscales;
  const void* q;
  void* y;
  int64_t q_stride, y_stride;
  const int32_t *cu, *len, *table;
  void* work;
  int* status;
  int rows, width, tokens;
  int heads, group;      // key/value heads, query heads of each
  int page_log2, pages, window;
  float scale_log2;      // scale * log2(e)
  uint32_t group_mul, group_shift;   // row / group = (row * group_mul >> 32) >> group_shift, for 2 <= group, row < 2^31
  int narrow;            // most query rows of a key/value head that the narrow kernel takes
  unsigned long long timeout_ns;   // limit of every wait (kv_attn_tc.cu)
  int fault;             // test builds only: an injected fault (0: none)
};
size_t kv_attn_work_bytes(const qnt_kv_desc& d, int heads, int max_new);
cudaError_t launch_kv_attn(const qnt_kv_desc& d, KvAttnArgs a, int max_new, int xbf16, cudaStream_t s);

}  // namespace qnt
