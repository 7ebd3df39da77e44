// Internal interface between the training attention's C-ABI layer (arl2_attn.cu) and its
// kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "arl2_attn.cuh"

namespace arl2 {

struct AttnOut {          // an output tensor [B, T, heads, d], strides in elements
  uint16_t* ptr;
  long long sb, st, sh;
};

// fp16 holds normal values from 2^-14 to 2^16 only, and P (about 1 / Tk) and dS (P times a gradient)
// leave that range where the gradients themselves do not. So the backward pass carries 2^14 P, and 2^e dS
// with e from a bound (Cauchy-Schwarz) of |dP - delta| <= 2 |do_i| |v_j|: e follows the row in dq, where a
// row's sum is over keys, and the rows that see a key tile in dk. Both are undone in fp32, by powers of
// two. The largest |do|^2 of a query tile and |v|^2 of a key head are found by prep as words of
// (call << 9) + exponent field, so that what an earlier call left is below any of this call's.
struct GradRange {
  unsigned long long* call;   // counts the calls; the main kernel of a call adds 1
  unsigned long long* g;      // [B][Hkv][query tiles]: over the query heads of the group
  unsigned long long* v;      // [B][Hkv]
};
// Rows of statistics: -lse in log2 units (fp16: + 14), -delta; fp16: the exponent field of |do|^2.
__host__ __device__ constexpr int attn_stat_rows(bool half) { return half ? 3 : 2; }

struct AttnArgs {
  AttnMask mask;
  int B, H, Hkv;
  float scale;            // of the scores
  AttnOut o;              // forward: o; backward: dq
  AttnOut dk, dv;         // backward
  float* lse;             // forward: [B, H, Tq] out
  const float* stats;     // backward: [B H][kStatRows][Tq rounded up to 128], see attn_stat_rows
  GradRange range;        // backward, fp16
  float* records;         // partial records, two per CTA
  float* dq_records;      // the dq kernel's
  void* splits;           // the CTAs' splits, written by a launch of its own, or null: each computes its own
  unsigned int* tickets;  // backward: ranges handed out, [dk and dv, dq]
  unsigned int* err;
  unsigned long long timeout_ns;
};

// Row statistics of the backward pass from o, do and lse (see arl2_attn_bwd.cu).
struct AttnPrepArgs {
  const uint16_t* o;
  const uint16_t* g;      // do
  long long o_sb, o_st, o_sh, g_sb, g_st, g_sh;
  const float* lse;       // [B, H, Tq]
  float* stats;
  const int* q_len;
  unsigned int* tickets;  // zeroed
  int B, H, Tq, d;
  // fp16: v and where its range and that of do go.
  const uint16_t* v;
  long long v_sb, v_st, v_sh;
  const int* k_len;
  GradRange range;
  int Hkv, Tk;
};

// Forward, and dk with dv.
__host__ __device__ constexpr size_t attn_record_floats(int d) { return 2ull * 128 * d + 4 * 128; }
__host__ __device__ constexpr size_t attn_dq_record_floats(int d) { return 128ull * d; }
cudaError_t attn_fwd_setup();
cudaError_t attn_bwd_setup();
// Of the backward kernel's CTAs, those that compute dk and dv; the others compute dq. Both have the
// same tile pairs to do, of 4 and 3 products: 2590 and 2230 cycles each as measured at d = 128.
// An even number, for whole pairs of SMs.
inline int attn_dkv_ctas(int ctas) { return ctas < 4 ? 1 : (ctas * 259 / (259 + 223) + 1) / 2 * 2; }
// Within a call the backward kernel (behind prep) and the combining launches are programmatic dependents
// of the launch before; a call's first launch, and what follows a split launch, are not. combine: a
// tile may be shared between CTAs, so its records have to be added up.
cudaError_t launch_attn_fwd(int d, bool half, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            const AttnArgs& a, int ctas, bool combine, cudaStream_t st);
cudaError_t launch_attn_bwd(int d, bool half, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            const CUtensorMap& g, const AttnPrepArgs& prep, const AttnArgs& a, int ctas, bool combine,
                            cudaStream_t st);
// Launch a kernel, behind the preceding one in the stream if `dependent`.
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, bool dependent,
                           const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace arl2
