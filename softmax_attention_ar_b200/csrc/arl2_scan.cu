// Gated linear recurrence over a sequence, and its backward pass (arl2_scan_* in arl2.h):
//     h_t   = a_t h_{t-1} + x_t                                     h_{-1} = h0 (or 0)
//     lam_t = dh_t + a_{t+1} lam_{t+1},  lam_{T-1} = dh_{T-1} + dfinal
//     dx_t = lam_t,  da_t = lam_t h_{t-1},  dh0 = a_0 lam_0
// per channel, with a gate per channel and token, or one per head and token (da is then the
// sum over the head's channels). Both directions are the same scan: (A, X) pairs compose as
// (A2, X2) after (A1, X1) = (A1 A2, A2 X1 + X2).
//
// The work is a few operations per element read, so memory traffic bounds it: every element
// is read once and written once. The sequence is cut three ways, so that few channels still
// fill the GPU: a thread holds kTok tokens of V channels in registers, the W warps of a CTA
// follow one another in time, and the N CTAs of a cluster follow one another again. One such
// super-chunk of N W kTok tokens is scanned at a time:
//   1. each thread loads its tokens and composes them to one (A, X) per channel;
//   2. warps combine through shared memory, CTAs through distributed shared memory and one
//      cluster barrier (two slots by turns, so one barrier per super-chunk is enough);
//   3. each thread scans its registers again from the state that reaches it, and writes.
// Every thread carries the running state of its channels to the next super-chunk itself. The
// order of all products and sums is fixed, so results do not depend on timing. All of it is
// fp32; only the stored h, dx and da are rounded, once, to their types.
#include <algorithm>
#include <climits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/arl2.h"
#include "arl2_device.cuh"
#include "arl2_kernels.h"

namespace arl2 {
namespace {

constexpr int kMaxWarps = 8;
constexpr int kMaxCluster = 16;

struct ScanParams {
  const void* in;      // x, or dh
  const void* a;
  const void* hprev;   // backward: the forward's h
  void* out;           // h, or dx
  void* da;            // backward
  const float* init;   // h0, or dfinal (may be null)
  float* last;         // final, or dh0 (may be null)
  const float* h0;     // backward: h_{-1} (may be null)
  const int* lens;     // may be null
  long long in_b, in_t, a_b, a_t, a_h, h_b, h_t, out_b, out_t, da_b, da_t, da_h;   // strides, elements
  int T, C, d;         // d: channels per gate (heads), or 1
  int groups;          // channel groups (CTAs per cluster position and batch)
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// V values of type T as one aligned access.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
};

// Forward (kBack = false): position p is token p. Backward: position p is token T - 1 - p.
template <typename X, typename G, int V, int kTok, bool kHead, bool kBack>
__global__ void __launch_bounds__(32 * kMaxWarps)
    arl2_scan_kernel(const __grid_constant__ ScanParams a) {
  constexpr int GV = kHead ? 1 : V;   // gates per token a thread holds
  __shared__ float s_warp[2][kMaxWarps][2][32 * V];         // [slot][warp][A | X][channel]
  __shared__ float s_cta[2][kMaxCluster][2][32 * V];        // [slot][rank][A | X][channel], written by the peers
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
  uint32_t N;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(N));
  const int rank = static_cast<int>(cluster_rank());
  const int unit = blockIdx.x / N;
  const int b = unit / a.groups;
  const int c = (unit % a.groups) * 32 * V + lane * V;
  const bool in_c = c < a.C;          // V divides C, or V = 1
  const int head = kHead ? c / a.d : 0;
  const int T = a.T;
  const int len = a.lens ? min(max(a.lens[b], 0), T) : T;
  const X* in = static_cast<const X*>(a.in) + b * a.in_b + c;
  const G* ga = static_cast<const G*>(a.a) + b * a.a_b + (kHead ? head * a.a_h : static_cast<long long>(c));
  const X* hp = static_cast<const X*>(a.hprev) + (kBack ? b * a.h_b + c : 0);
  X* out = static_cast<X*>(a.out) + b * a.out_b + c;
  G* da = static_cast<G*>(a.da) + (kBack ? b * a.da_b + (kHead ? head * a.da_h : static_cast<long long>(c)) : 0);

  float state[V];
#pragma unroll
  for (int v = 0; v < V; ++v)
    state[v] = a.init && in_c ? a.init[static_cast<long long>(b) * a.C + c + v] : 0.f;

  // A peer's shared memory may be written only once that CTA runs: arrive here, wait before
  // the first write.
  if (N > 1) cluster_arrive();
  const int chunk = W * kTok;
  const long long super = static_cast<long long>(N) * chunk;
  int slot = 0;
  for (long long s0 = 0; s0 < T; s0 += super, slot ^= 1) {
    const long long p0 = s0 + static_cast<long long>(rank) * chunk + warp * kTok;
    // 1. Load. Behind the length: gate 1 and input 0, so the state passes unchanged.
    Pack<X, V> xs[kTok], hs[kBack ? kTok : 1];
    Pack<G, GV> gs[kTok];
    bool ok[kTok];
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      const long long t = kBack ? T - 1 - (p0 + i) : p0 + i;
      ok[i] = in_c && t >= 0 && t < len;
      const long long tg = kBack ? t + 1 : t;
#pragma unroll
      for (int v = 0; v < V; ++v) xs[i].v[v] = from_f<X>(0.f);
#pragma unroll
      for (int v = 0; v < GV; ++v) gs[i].v[v] = from_f<G>(1.f);
      if (ok[i]) {
        xs[i] = *reinterpret_cast<const Pack<X, V>*>(in + t * a.in_t);
        if (tg < len) gs[i] = *reinterpret_cast<const Pack<G, GV>*>(ga + tg * a.a_t);
      }
      if (kBack) {
#pragma unroll
        for (int v = 0; v < V; ++v) hs[i].v[v] = from_f<X>(0.f);
        if (ok[i] && t > 0) hs[i] = *reinterpret_cast<const Pack<X, V>*>(hp + (t - 1) * a.h_t);
      }
    }
    float A[GV], S[V];
#pragma unroll
    for (int v = 0; v < GV; ++v) A[v] = 1.f;
#pragma unroll
    for (int v = 0; v < V; ++v) S[v] = 0.f;
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) S[v] = fmaf(to_f(gs[i].v[kHead ? 0 : v]), S[v], to_f(xs[i].v[v]));
#pragma unroll
      for (int v = 0; v < GV; ++v) A[v] *= to_f(gs[i].v[v]);
    }
    // 2. Combine: state becomes the state before this thread's first token, next the state
    // after the super-chunk.
    float next[V];
#pragma unroll
    for (int v = 0; v < V; ++v) next[v] = fmaf(A[kHead ? 0 : v], state[v], S[v]);
    if (W > 1 || N > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s_warp[slot][warp][0][lane * V + v] = A[kHead ? 0 : v];
        s_warp[slot][warp][1][lane * V + v] = S[v];
      }
      __syncthreads();
      if (N > 1) {
        if (s0 == 0) cluster_wait();
        if (warp == 0) {   // the CTA's (A, X) to the same place in every CTA of the cluster
          float ca[V], cx[V];
#pragma unroll
          for (int v = 0; v < V; ++v) {
            ca[v] = A[kHead ? 0 : v];
            cx[v] = S[v];
            for (int w = 1; w < W; ++w) {
              const float wa = s_warp[slot][w][0][lane * V + v];
              cx[v] = fmaf(wa, cx[v], s_warp[slot][w][1][lane * V + v]);
              ca[v] *= wa;
            }
          }
          const uint32_t mine = smem_u32(&s_cta[slot][rank][0][lane * V]);
          for (uint32_t r = 0; r < N; ++r) {
            const uint32_t dst = peer_smem(mine, r);
#pragma unroll
            for (int v = 0; v < V; ++v) {
              st_cluster_f32(dst + 4 * v, ca[v]);
              st_cluster_f32(dst + 4 * (32 * V + v), cx[v]);
            }
          }
        }
        cluster_sync();
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float s = state[v];
          for (int r = 0; r < static_cast<int>(N); ++r) {
            if (r == rank) state[v] = s;
            s = fmaf(s_cta[slot][r][0][lane * V + v], s, s_cta[slot][r][1][lane * V + v]);
          }
          next[v] = s;
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float s = state[v];
        for (int w = 0; w < W; ++w) {
          if (w == warp) state[v] = s;
          s = fmaf(s_warp[slot][w][0][lane * V + v], s, s_warp[slot][w][1][lane * V + v]);
        }
        if (N == 1) next[v] = s;
      }
    }
    // 3. Scan again from the state that reaches this thread, and write.
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      const long long t = kBack ? T - 1 - (p0 + i) : p0 + i;
      const bool inside = in_c && t >= 0 && t < T;
      Pack<X, V> o;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        state[v] = fmaf(to_f(gs[i].v[kHead ? 0 : v]), state[v], to_f(xs[i].v[v]));
        o.v[v] = from_f<X>(ok[i] ? state[v] : 0.f);
      }
      if (inside) *reinterpret_cast<Pack<X, V>*>(out + t * a.out_t) = o;
      if (kBack) {
        float prev[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          prev[v] = to_f(hs[i].v[v]);
          if (t == 0 && in_c && a.h0) prev[v] = a.h0[static_cast<long long>(b) * a.C + c + v];
        }
        if (kHead) {
          float sum = 0.f;
#pragma unroll
          for (int v = 0; v < V; ++v) sum += ok[i] ? state[v] * prev[v] : 0.f;
          for (int m = a.d / V / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
          if (inside && c % a.d == 0) da[t * a.da_t] = from_f<G>(sum);
        } else {
          Pack<G, GV> g;
#pragma unroll
          for (int v = 0; v < GV; ++v) g.v[v] = from_f<G>(ok[i] ? state[v] * prev[v] : 0.f);
          if (inside) *reinterpret_cast<Pack<G, GV>*>(da + t * a.da_t) = g;
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) state[v] = next[v];
  }
  if (a.last && in_c && rank == 0 && warp == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float g = kBack && len > 0 ? to_f(ga[kHead ? 0 : v]) : 1.f;   // dh0 = a_0 lam_0
      a.last[static_cast<long long>(b) * a.C + c + v] = g * state[v];
    }
  }
}

template <typename X, typename G, int V, bool kHead, bool kBack>
cudaError_t launch(const ScanParams& p, int B, int sms, cudaStream_t st) {
  // 16 tokens per thread, or 8 where a thread's registers hold twice the bytes.
  constexpr int kTok = sizeof(X) == 4 && V > 1 ? 8 : 16;
  ScanParams a = p;
  const int per = 32 * V;
  a.groups = (a.C + per - 1) / per;
  const int W = std::max(1, std::min(kMaxWarps, (a.T + kTok - 1) / kTok));
  // Enough CTAs along the sequence to give every SM two, while each still has tokens.
  const long long units = static_cast<long long>(B) * a.groups;
  int N = 1;
  while (N < kMaxCluster && units * N < 2ll * sms && static_cast<long long>(N) * W * kTok < a.T) N *= 2;
  if (units * N > INT_MAX) return cudaErrorInvalidConfiguration;
  auto* kern = &arl2_scan_kernel<X, G, V, kTok, kHead, kBack>;
  if (N > 8) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(units * N));
  cfg.blockDim = dim3(32 * W);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = N;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename X, typename G, bool kBack>
cudaError_t by_width(const ScanParams& p, int B, int sms, bool head, bool wide, cudaStream_t st) {
  if (head) return launch<X, float, 4, true, kBack>(p, B, sms, st);
  return wide ? launch<X, G, 4, false, kBack>(p, B, sms, st) : launch<X, G, 1, false, kBack>(p, B, sms, st);
}

template <bool kBack>
cudaError_t by_type(const ScanParams& p, int B, int sms, arl2_dtype x, arl2_dtype g, bool head, bool wide,
                    cudaStream_t st) {
  const bool gf = g == ARL2_FP32;
  if (x == ARL2_FP32) return by_width<float, float, kBack>(p, B, sms, head, wide, st);
  if (x == ARL2_BF16)
    return gf ? by_width<__nv_bfloat16, float, kBack>(p, B, sms, head, wide, st)
              : by_width<__nv_bfloat16, __nv_bfloat16, kBack>(p, B, sms, head, wide, st);
  return gf ? by_width<__half, float, kBack>(p, B, sms, head, wide, st)
            : by_width<__half, __half, kBack>(p, B, sms, head, wide, st);
}

size_t elem(arl2_dtype t) { return t == ARL2_FP32 ? 4 : 2; }
bool dtype_ok(int t) { return t == ARL2_BF16 || t == ARL2_FP16 || t == ARL2_FP32; }
bool at(const void* p, size_t align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0; }

// Strides of dimensions of size 1 do not matter; they are taken as 0.
struct Strides {
  long long b, t, h;
};
Strides strides_of(const int64_t* s, const arl2_scan_shape& shape, bool gates = false) {
  return {shape.B > 1 ? s[0] : 0, shape.T > 1 ? s[1] : 0, gates && shape.heads > 1 ? s[2] : 0};
}

// A [B, T, C] tensor, unit channel stride: whether its strides are in range, and whether groups
// of 4 channels of it can be accessed at once. An output's elements must not share memory.
bool strides_ok(const Strides& x, int B, int T, int C, bool output) {
  const long long sb = x.b, st = x.t;
  if (sb < 0 || st < 0 || x.h < 0) return false;
  if (!output) return true;
  if (T > 1 && st < C) return false;
  if (B > 1 && sb < (T > 1 ? (T - 1) * st : 0) + C && !(sb >= C && T > 1 && st >= (B - 1) * sb + C)) return false;
  return true;
}
bool wide_ok(const void* p, size_t e, const Strides& x) { return at(p, 4 * e) && x.b % 4 == 0 && x.t % 4 == 0; }

arl2_status check(const arl2_scan_shape& s, bool* head) {
  if (s.B < 1 || s.T < 1 || s.C < 1 || s.heads < 0) return ARL2_ERR_INVALID_ARG;
  if (!dtype_ok(s.dtype) || !dtype_ok(s.gate_dtype)) return ARL2_ERR_INVALID_ARG;
  *head = s.heads > 0;
  if (*head) {
    if (s.C % s.heads) return ARL2_ERR_INVALID_ARG;
    const int d = s.C / s.heads;
    if (d != 32 && d != 64 && d != 128) return ARL2_ERR_UNSUPPORTED;
    if (s.gate_dtype != ARL2_FP32) return ARL2_ERR_UNSUPPORTED;
  } else if (s.gate_dtype != s.dtype && s.gate_dtype != ARL2_FP32) {
    return ARL2_ERR_UNSUPPORTED;
  }
  return ARL2_OK;
}

}  // namespace
}  // namespace arl2

extern "C" arl2_status arl2_scan_forward(const arl2_scan_fwd* f, arl2_stream stream) {
  using namespace arl2;
  if (!f) return ARL2_ERR_INVALID_ARG;
  const arl2_scan_shape& s = f->shape;
  bool head = false;
  const arl2_status cs = check(s, &head);
  if (cs != ARL2_OK) return cs;
  const size_t e = elem(s.dtype), ge = elem(s.gate_dtype);
  if (!f->x || !f->a || !f->h || !at(f->x, e) || !at(f->h, e) || !at(f->a, ge) || !at(f->h0, 4) ||
      !at(f->final_state, 4) || !at(s.lens, 4))
    return ARL2_ERR_INVALID_ARG;
  const Strides xs = strides_of(f->x_stride, s), hs = strides_of(f->h_stride, s),
                as = strides_of(f->a_stride, s, true);
  if (!strides_ok(xs, s.B, s.T, s.C, false) || !strides_ok(as, s.B, s.T, s.C, false) ||
      !strides_ok(hs, s.B, s.T, s.C, true))
    return ARL2_ERR_INVALID_ARG;
  bool wide = s.C % 4 == 0 && wide_ok(f->x, e, xs) && wide_ok(f->h, e, hs);
  if (head && !wide) return ARL2_ERR_INVALID_ARG;
  if (!head) wide = wide && wide_ok(f->a, ge, as);
  int dev = 0, sms = 0;
  const arl2_status ds = static_cast<arl2_status>(prepare_device(&dev, &sms));
  if (ds != ARL2_OK) return ds;
  ScanParams p{};
  p.in = f->x;
  p.a = f->a;
  p.out = f->h;
  p.init = f->h0;
  p.last = f->final_state;
  p.lens = s.lens;
  p.in_b = xs.b, p.in_t = xs.t;
  p.a_b = as.b, p.a_t = as.t, p.a_h = as.h;
  p.out_b = hs.b, p.out_t = hs.t;
  p.T = s.T, p.C = s.C, p.d = head ? s.C / s.heads : 1;
  return by_type<false>(p, s.B, sms, static_cast<arl2_dtype>(s.dtype), static_cast<arl2_dtype>(s.gate_dtype), head,
                        wide, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ARL2_OK
             : ARL2_ERR_CUDA;
}

extern "C" arl2_status arl2_scan_backward(const arl2_scan_bwd* f, arl2_stream stream) {
  using namespace arl2;
  if (!f) return ARL2_ERR_INVALID_ARG;
  const arl2_scan_shape& s = f->shape;
  bool head = false;
  const arl2_status cs = check(s, &head);
  if (cs != ARL2_OK) return cs;
  const size_t e = elem(s.dtype), ge = elem(s.gate_dtype);
  if (!f->dh || !f->a || !f->h || !f->dx || !f->da || !at(f->dh, e) || !at(f->h, e) || !at(f->dx, e) ||
      !at(f->a, ge) || !at(f->da, ge) || !at(f->h0, 4) || !at(f->dfinal, 4) || !at(f->dh0, 4) || !at(s.lens, 4))
    return ARL2_ERR_INVALID_ARG;
  const Strides gs = strides_of(f->dh_stride, s), hs = strides_of(f->h_stride, s),
                as = strides_of(f->a_stride, s, true), xs = strides_of(f->dx_stride, s);
  if (!strides_ok(gs, s.B, s.T, s.C, false) || !strides_ok(hs, s.B, s.T, s.C, false) ||
      !strides_ok(as, s.B, s.T, s.C, false) || !strides_ok(xs, s.B, s.T, s.C, true))
    return ARL2_ERR_INVALID_ARG;
  bool wide = s.C % 4 == 0 && wide_ok(f->dh, e, gs) && wide_ok(f->h, e, hs) && wide_ok(f->dx, e, xs);
  if (head && !wide) return ARL2_ERR_INVALID_ARG;
  if (!head) wide = wide && wide_ok(f->a, ge, as) && at(f->da, 4 * ge);
  int dev = 0, sms = 0;
  const arl2_status ds = static_cast<arl2_status>(prepare_device(&dev, &sms));
  if (ds != ARL2_OK) return ds;
  ScanParams p{};
  p.in = f->dh;
  p.a = f->a;
  p.hprev = f->h;
  p.out = f->dx;
  p.da = f->da;
  p.init = f->dfinal;
  p.last = f->dh0;
  p.h0 = f->h0;
  p.lens = s.lens;
  p.in_b = gs.b, p.in_t = gs.t;
  p.a_b = as.b, p.a_t = as.t, p.a_h = as.h;
  p.h_b = hs.b, p.h_t = hs.t;
  p.out_b = xs.b, p.out_t = xs.t;
  // da is contiguous: [B, T, C], or [B, heads, T].
  if (head) {
    p.da_b = static_cast<long long>(s.heads) * s.T, p.da_t = 1, p.da_h = s.T;
  } else {
    p.da_b = static_cast<long long>(s.T) * s.C, p.da_t = s.C;
  }
  p.T = s.T, p.C = s.C, p.d = head ? s.C / s.heads : 1;
  return by_type<true>(p, s.B, sms, static_cast<arl2_dtype>(s.dtype), static_cast<arl2_dtype>(s.gate_dtype), head,
                       wide, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ARL2_OK
             : ARL2_ERR_CUDA;
}
