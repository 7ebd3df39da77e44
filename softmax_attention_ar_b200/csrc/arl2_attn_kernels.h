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

struct AttnArgs {
  AttnMask mask;
  int B, H, Hkv;
  float scale;            // of the scores
  AttnOut o;              // forward: o; backward: dq
  AttnOut dk, dv;         // backward
  float* lse;             // forward: [B, H, Tq] out
  const float* stats;     // backward: [B H][2][Tq rounded up to 128]: lse in log2 units, then delta
  float* records;         // partial records, two per CTA
  unsigned int* counters; // arrivals per tile, all 0 between calls
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
  int B, H, Tq, d;
};

__host__ __device__ constexpr size_t attn_record_floats(int d) { return 2ull * 128 * d + 4 * 128; }   // the largest of the three kernels'
cudaError_t attn_fwd_setup();
cudaError_t attn_bwd_setup();
cudaError_t launch_attn_fwd(int d, bool half, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            const AttnArgs& a, int ctas, cudaStream_t st);
cudaError_t launch_attn_prep(bool half, const AttnPrepArgs& a, cudaStream_t st);
cudaError_t launch_attn_dkv(int d, bool half, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            const CUtensorMap& g, const AttnArgs& a, int ctas, cudaStream_t st);
cudaError_t launch_attn_dq(int d, bool half, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                           const CUtensorMap& g, const AttnArgs& a, int ctas, cudaStream_t st);

}  // namespace arl2
