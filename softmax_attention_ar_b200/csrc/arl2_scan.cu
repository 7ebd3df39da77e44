// Gated linear recurrence over a sequence, and its backward pass (arl2_scan_* in arl2.h):
//     h_t   = a_t h_{t-1} + x_t                                     h_{-1} = h0 (or 0)
//     lam_t = dh_t + a_{t+1} lam_{t+1},  lam_{T-1} = dh_{T-1} + dfinal
//     dx_t = lam_t,  da_t = lam_t h_{t-1},  dh0 = a_0 lam_0
// per channel, with a gate per channel and token, or one per head and token (da is then the
// sum over the head's channels). Both directions are the same scan: (A, X) pairs compose as
// (A2, X2) after (A1, X1) = (A1 A2, A2 X1 + X2).
//
// The work is a few operations per element read, so memory traffic bounds it. A warp owns a
// slice of consecutive tokens of 32 V channels and streams it; the kWarps slices of a CTA
// follow one another and form a chunk. Two launches:
//   - arl2_scan_pairs_kernel reads x (dh) and a, and writes the (A, X) of every slice and of
//     every chunk to the workspace;
//   - arl2_scan_apply_kernel composes the pairs before each slice onto the initial state,
//     then streams the slice again from that state and writes the results.
// The second reading is what this costs over a single pass; it comes from L2 where x and a
// fit there. A single-pass form (the cluster's CTAs following one another in time, pairs
// exchanged through distributed shared memory, data kept in a ring) reads everything once but
// moves in lock step with a barrier per 1024 tokens: it measured 115 us on 32760 tokens of
// 1536 bf16 channels, this form 73 us. A sequence that one chunk holds takes one launch, without workspace.
// The order of all products and sums is fixed, so results do not depend on timing. All of it is
// fp32; only the stored h, dx and da are rounded, once, to their types.
#include <algorithm>
#include <atomic>
#include <climits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/arl2.h"
#include "arl2_device.cuh"
#include "arl2_kernels.h"

namespace arl2 {
namespace {

constexpr int kWarps = 8;    // slices per chunk, warps per CTA
constexpr int kBatch = 4;    // tokens a warp copies and works on at once; slices are multiples of it
constexpr int kStages = 4;   // batches in flight per warp

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
  float2* slices;      // [B][chunks * kWarps][groups * 32 V] (A, X) of each slice
  float2* chunks;      // [B][chunks][groups * 32 V] of each chunk
  long long in_b, in_t, a_b, a_t, a_h, h_b, h_t, out_b, out_t, da_b, da_t, da_h;   // strides, elements
  int T, C, d;         // d: channels per gate (heads), or 1
  int groups;          // channel groups of 32 V
  int slice, nchunks;  // tokens per slice; chunks per sequence
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

// Copy one Pack from global to shared memory, or zeros where !ok (src is then not read, but is
// inside the tensor). cp.async takes 4, 8 or 16 bytes; a 2-byte element goes through a register.
template <typename P>
__device__ __forceinline__ void copy_async(P* dst, const P* src, bool ok) {
  if constexpr (sizeof(P) >= 4) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(src)), "n"(sizeof(P)), "r"(ok ? static_cast<uint32_t>(sizeof(P)) : 0u)
                 : "memory");
  } else {
    P v = *src;
    if (!ok) memset(&v, 0, sizeof v);
    *dst = v;
  }
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Bytes of the copy ring per warp: kStages batches of x (dh), the gates, and with kPrev of h.
template <typename X, typename G, int V, bool kHead, bool kPrev>
__host__ __device__ constexpr uint32_t ring_bytes() {
  return kStages * kBatch * (32u * V * sizeof(X) * (kPrev ? 2 : 1) + (kHead ? 4u * 4u : 32u * V * sizeof(G)));
}

struct True {
  static constexpr bool value = true;
};
struct False {
  static constexpr bool value = false;
};

// Where a warp works, and its stream of batches: token q of the scan is token q of the sequence
// forward and token len - 1 - q backward. kPrev: h_{t-1} comes along (the backward apply).
template <typename X, typename G, int V, bool kHead, bool kBack, bool kPrev>
struct Place {
  static constexpr int GV = kHead ? 1 : V;   // gates per token a thread holds
  using PX = Pack<X, V>;
  using PG = Pack<G, GV>;
  int lane, warp, b, group, chunk, c, len;
  bool in_c;
  int q0, end;         // this warp's slice: q0 <= q < end (empty behind the length)
  const X* in;
  const G* ga;
  const X* hp;
  PX* ring_x;          // [kStages][kBatch][32], this lane's entry of the first row
  PX* ring_h;
  PG* ring_g;          // the same; per head [kStages][4][kBatch], this lane's head of the first stage
  G* copy_g;           // per head: where this lane copies a gate to (null: it copies none)
  const G* from_g;     // and from, at token 0
  // Chunks slowest, so that the CTAs in flight work on neighbouring tokens; the apply kernel
  // takes them in reverse and begins with what the pairs kernel read last.
  __device__ Place(const ScanParams& a, bool reverse, uint8_t* smem) {
    lane = threadIdx.x & 31;
    warp = threadIdx.x >> 5;
    int u = blockIdx.x;
    group = u % a.groups;
    u /= a.groups;
    const int nb = gridDim.x / (a.groups * a.nchunks);
    b = u % nb;
    chunk = reverse ? a.nchunks - 1 - u / nb : u / nb;
    c = group * 32 * V + lane * V;
    in_c = c < a.C;                      // V divides C, or V = 1
    const int cl = in_c ? c : 0;         // lanes behind the last channel stay inside the tensor
    len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    q0 = (chunk * (blockDim.x >> 5) + warp) * a.slice;
    end = min(q0 + a.slice, len);
    in = static_cast<const X*>(a.in) + b * a.in_b + cl;
    ga = static_cast<const G*>(a.a) + b * a.a_b + (kHead ? (cl / a.d) * a.a_h : static_cast<long long>(cl));
    hp = kPrev ? static_cast<const X*>(a.hprev) + b * a.h_b + cl : nullptr;
    uint8_t* ring = smem + warp * ring_bytes<X, G, V, kHead, kPrev>();
    ring_x = reinterpret_cast<PX*>(ring) + lane;
    ring += kStages * kBatch * 32 * sizeof(PX);
    ring_h = reinterpret_cast<PX*>(ring) + lane;
    if (kPrev) ring += kStages * kBatch * 32 * sizeof(PX);
    copy_g = nullptr;
    from_g = nullptr;
    if constexpr (kHead) {   // lane l copies the gate of token l % kBatch and head l / kBatch of the group's
      const int h0 = group * 32 * V / a.d, h = lane / kBatch;
      ring_g = reinterpret_cast<PG*>(ring) + (c / a.d - h0) * kBatch;
      if (h < 32 * V / a.d && h0 + h < a.C / a.d) {
        copy_g = reinterpret_cast<G*>(ring) + lane;
        from_g = static_cast<const G*>(a.a) + b * a.a_b + (h0 + h) * a.a_h;
      }
    } else {
      ring_g = reinterpret_cast<PG*>(ring) + lane;
    }
  }
  __device__ int token(int q) const { return kBack ? len - 1 - q : q; }
  // Start copying tokens q .. q + kBatch - 1 to a stage: one group, empty behind the slice.
  __device__ void copy(const ScanParams& a, int q, int stage) const {
    if (q < end) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const bool ok = in_c && q + i < len;
        const int t = ok ? token(q + i) : 0, tg = kBack ? min(t + 1, len - 1) : t;
        copy_async(ring_x + (stage * kBatch + i) * 32, reinterpret_cast<const PX*>(in + t * a.in_t), ok);
        if constexpr (!kHead)
          copy_async(ring_g + (stage * kBatch + i) * 32, reinterpret_cast<const PG*>(ga + tg * a.a_t), ok);
        if constexpr (kPrev)
          copy_async(ring_h + (stage * kBatch + i) * 32, reinterpret_cast<const PX*>(hp + max(t - 1, 0) * a.h_t),
                     ok && t > 0);
      }
      if constexpr (kHead) {
        const int i = lane % kBatch;
        const int t = min(token(q + i) + (kBack ? 1 : 0), len - 1);
        if (copy_g)
          copy_async(reinterpret_cast<Pack<G, 1>*>(copy_g + stage * kBatch * 4),
                     reinterpret_cast<const Pack<G, 1>*>(from_g + max(t, 0) * a.a_t), q + i < len);
      }
    }
    copy_commit();
  }
  __device__ void start(const ScanParams& a) const {
#pragma unroll
    for (int k = 0; k < kStages; ++k) copy(a, q0 + k * kBatch, k);
  }
  // After start(): call work(exact, q, stage) for each batch of the slice in order. exact is
  // False where a token of the batch lies behind the length or, backward, is the last one:
  // there the gate is not what the ring holds but 1, so that a state passes unchanged (the
  // value is 0) and dfinal reaches the last token undamped.
  template <typename Work>
  __device__ void stream(const ScanParams& a, Work&& work) const {
    int stage = 0;
    for (int q = q0; q < end; q += kBatch) {
      copy_wait<kStages - 1>();
      if (kHead) __syncwarp();   // gates are copied by other lanes than those that read them
      if (q + kBatch > len || (kBack && q == 0))
        work(False{}, q, stage);
      else
        work(True{}, q, stage);
      if (kHead) __syncwarp();
      copy(a, q + kStages * kBatch, stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
  }
  __device__ PX value(int stage, int i) const { return ring_x[(stage * kBatch + i) * 32]; }
  __device__ PX prev(int stage, int i) const { return ring_h[(stage * kBatch + i) * 32]; }
  template <bool kExact>
  __device__ void gates(int q, int stage, int i, float (&g)[GV]) const {
    const PG p = kHead ? ring_g[stage * kBatch * 4 + i] : ring_g[(stage * kBatch + i) * 32];
    const bool ok = kExact || (q + i < len && (!kBack || q + i > 0));
#pragma unroll
    for (int v = 0; v < GV; ++v) g[v] = ok ? to_f(p.v[v]) : 1.f;
  }
  // The (A, X) of this warp's slice (after start()).
  __device__ void pairs(const ScanParams& a, float (&A)[V], float (&S)[V]) const {
    float Ag[GV];
#pragma unroll
    for (int v = 0; v < GV; ++v) Ag[v] = 1.f;
#pragma unroll
    for (int v = 0; v < V; ++v) S[v] = 0.f;
    stream(a, [&](auto exact, int q, int stage) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        float g[GV];
        gates<decltype(exact)::value>(q, stage, i, g);
        const PX x = value(stage, i);
#pragma unroll
        for (int v = 0; v < V; ++v) S[v] = fmaf(g[kHead ? 0 : v], S[v], to_f(x.v[v]));
#pragma unroll
        for (int v = 0; v < GV; ++v) Ag[v] *= g[v];
      }
    });
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = Ag[kHead ? 0 : v];
  }
};

template <typename X, typename G, int V, bool kHead, bool kBack>
__global__ void __launch_bounds__(32 * kWarps, V == 4 && !(kHead && kBack) ? 2 : 1)
    arl2_scan_pairs_kernel(const __grid_constant__ ScanParams a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 s_pair[kWarps][32 * V];
  griddep_launch_dependents();
  const Place<X, G, V, kHead, kBack, false> p(a, false, ring);
  float A[V], S[V];
  p.start(a);
  p.pairs(a, A, S);
  const long long width = static_cast<long long>(a.groups) * 32 * V;
  const int c = p.group * 32 * V + p.lane * V;
  float2* dst = a.slices + ((static_cast<long long>(p.b) * a.nchunks + p.chunk) * kWarps + p.warp) * width + c;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    dst[v] = make_float2(A[v], S[v]);
    s_pair[p.warp][p.lane * V + v] = make_float2(A[v], S[v]);
  }
  __syncthreads();
  for (int k = threadIdx.x; k < 32 * V; k += blockDim.x) {
    float2 r = s_pair[0][k];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float2 n = s_pair[w][k];
      r = make_float2(r.x * n.x, fmaf(n.x, r.y, n.y));
    }
    a.chunks[(static_cast<long long>(p.b) * a.nchunks + p.chunk) * width + p.group * 32 * V + k] = r;
  }
}

// Sums of kBatch values over the lanes of a head (d / 4 of them: 8, 16 or 32), by halving the
// values held: each exchange sends the half that the partner keeps. Lane l of a head ends with
// the sum of value (l / same) % kBatch, which `same` = lanes / kBatch neighbouring lanes hold.
__device__ __forceinline__ float head_sums(float (&r)[kBatch], int lanes, int lane, int* index) {
  int m = lanes >> 1;
#pragma unroll
  for (int n = kBatch / 2; n >= 1; n >>= 1, m >>= 1) {
    const bool upper = (lane & m) != 0;   // keeps the upper half of the values
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = upper ? r[i] : r[i + n], keep = upper ? r[i + n] : r[i];
      r[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
    }
  }
  for (; m > 0; m >>= 1) r[0] += __shfl_xor_sync(0xffffffffu, r[0], m);
  *index = lane / (lanes / kBatch) % kBatch;
  return r[0];
}

template <typename X, typename G, int V, bool kHead, bool kBack>
__global__ void __launch_bounds__(32 * kWarps, V == 4 && !(kHead && kBack) ? 2 : 1)
    arl2_scan_apply_kernel(const __grid_constant__ ScanParams a) {
  using P = Place<X, G, V, kHead, kBack, kBack>;
  using PX = typename P::PX;
  using PG = typename P::PG;
  constexpr int GV = P::GV;
  __shared__ float2 s_pair[kWarps][32 * V];    // each warp's share of the earlier chunks
  __shared__ float2 s_slice[kWarps][32 * V];   // the chunk's slices
  extern __shared__ __align__(16) uint8_t ring[];
  const P p(a, true, ring);
  const int lane = p.lane, warp = p.warp, len = p.len, W = blockDim.x >> 5;
  p.start(a);   // in flight while the state it starts from is composed
  float state[V];
#pragma unroll
  for (int v = 0; v < V; ++v) state[v] = a.init && p.in_c ? a.init[static_cast<long long>(p.b) * a.C + p.c + v] : 0.f;

  // The state this warp's slice starts from: every warp brings its slice's pair and composes its
  // share of the earlier chunks; all meet in shared memory.
  float A[V], S[V];
  if (a.nchunks == 1) {
    if (W > 1) {
      p.pairs(a, A, S);
      p.start(a);
#pragma unroll
      for (int v = 0; v < V; ++v) s_slice[warp][lane * V + v] = make_float2(A[v], S[v]);
    }
  } else {
    griddep_wait();   // the pairs kernel's results
    const long long width = static_cast<long long>(a.groups) * 32 * V;
    const float2* mine =
        a.slices + ((static_cast<long long>(p.b) * a.nchunks + p.chunk) * kWarps + warp) * width + p.group * 32 * V;
    Pack<float2, V> own;
#pragma unroll
    for (int v = 0; v < V; ++v) own.v[v] = mine[lane * V + v];
    const int share = (p.chunk + kWarps - 1) / kWarps;
    const int k0 = min(warp * share, p.chunk), k1 = min(k0 + share, p.chunk);
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f, S[v] = 0.f;
    const float2* src =
        a.chunks + (static_cast<long long>(p.b) * a.nchunks + k0) * width + p.group * 32 * V + lane * V;
    for (int k = k0; k < k1; k += 4) {
      Pack<float2, V> n[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) n[i].v[v] = src[min(k - k0 + i, k1 - 1 - k0) * width + v];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k + i < k1) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            S[v] = fmaf(n[i].v[v].x, S[v], n[i].v[v].y);
            A[v] *= n[i].v[v].x;
          }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s_pair[warp][lane * V + v] = make_float2(A[v], S[v]);
      s_slice[warp][lane * V + v] = own.v[v];
    }
  }
  if (W > 1) {
    __syncthreads();
    if (a.nchunks > 1) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float2 n = s_pair[w][lane * V + v];
          state[v] = fmaf(n.x, state[v], n.y);
        }
    }
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w)
      if (w < warp) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float2 n = s_slice[w][lane * V + v];
          state[v] = fmaf(n.x, state[v], n.y);
        }
      }
  }

  X* out = static_cast<X*>(a.out) + p.b * a.out_b + p.c;
  G* da = kBack ? static_cast<G*>(a.da) + p.b * a.da_b + (kHead ? 0 : static_cast<long long>(p.c)) : nullptr;
  const int head = kHead ? p.c / a.d : 0;
  float first[kBack ? V : 1];   // backward: h_{-1}
  if constexpr (kBack) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      first[v] = a.h0 && p.in_c ? a.h0[static_cast<long long>(p.b) * a.C + p.c + v] : 0.f;
  }
  p.stream(a, [&](auto exact, int q, int stage) {
    [[maybe_unused]] float sums[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const bool ok = (decltype(exact)::value || q + i < len) && p.in_c;
      const int t = p.token(q + i);
      float g[GV];
      p.template gates<decltype(exact)::value>(q, stage, i, g);
      const PX x = p.value(stage, i);
      PX o;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        state[v] = fmaf(g[kHead ? 0 : v], state[v], to_f(x.v[v]));
        o.v[v] = from_f<X>(state[v]);
      }
      if (ok) *reinterpret_cast<PX*>(out + t * a.out_t) = o;
      if constexpr (kBack) {
        const PX h = p.prev(stage, i);
        float prod[V];
#pragma unroll
        for (int v = 0; v < V; ++v) prod[v] = state[v] * (t > 0 ? to_f(h.v[v]) : first[v]);
        if constexpr (kHead) {
          float sum = prod[0];
#pragma unroll
          for (int v = 1; v < V; ++v) sum += prod[v];
          sums[i] = sum;
        } else {
          PG o2;
#pragma unroll
          for (int v = 0; v < GV; ++v) o2.v[v] = from_f<G>(prod[v]);
          if (ok) *reinterpret_cast<PG*>(da + t * a.da_t) = o2;
        }
      }
    }
    if constexpr (kBack && kHead) {
      const int lanes = a.d / V;
      int i = 0;
      const float sum = head_sums(sums, lanes, lane, &i);
      const bool writer = p.in_c && lane % (lanes / kBatch) == 0;   // one of the lanes that hold it
      if (writer && q + i < len) da[head * a.da_h + p.token(q + i) * a.da_t] = from_f<G>(sum);
    }
  });

  // The warp whose slice holds the last token (the first slice, of an empty sequence) has the
  // final state.
  if (a.last && p.in_c && (len > 0 ? p.q0 < len && p.q0 + a.slice >= len : p.q0 == 0)) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float g = kBack && len > 0 ? to_f(p.ga[kHead ? 0 : v]) : 1.f;   // dh0 = a_0 lam_0
      a.last[static_cast<long long>(p.b) * a.C + p.c + v] = g * state[v];
    }
  }
  // Behind the length: zeros (each warp in its own slice's place).
  for (int t = max(p.q0, len); t < min(p.q0 + a.slice, a.T); ++t) {
    PX z;
#pragma unroll
    for (int v = 0; v < V; ++v) z.v[v] = from_f<X>(0.f);
    if (p.in_c) *reinterpret_cast<PX*>(out + t * a.out_t) = z;
    if constexpr (kBack && kHead) {
      if (p.in_c && p.c % a.d == 0) da[head * a.da_h + t * a.da_t] = from_f<G>(0.f);
    } else if constexpr (kBack) {
      PG gz;
#pragma unroll
      for (int v = 0; v < GV; ++v) gz.v[v] = from_f<G>(0.f);
      if (p.in_c) *reinterpret_cast<PG*>(da + t * a.da_t) = gz;
    }
  }
}

// How a call is cut. Slices are as long as they can be while there are four CTAs for every SM
// of a B200 (kFill), since shorter ones mean more pairs to write and compose: between 8 and 64
// tokens, longer only where a sequence would have more than 256 chunks (each CTA composes all
// the chunks before its own). A sequence of at most kWarps 64-token slices is one chunk, cut into no
// more warps than it has batches.
struct ScanPlan {
  int groups, slice, nchunks, warps;
  size_t slice_pairs, chunk_pairs;   // workspace, in (A, X) pairs
};
constexpr int kFill = 4 * 148;
ScanPlan plan_scan(int B, int T, int C, int V) {
  ScanPlan p{};
  p.groups = (C + 32 * V - 1) / (32 * V);
  const long long units = static_cast<long long>(B) * p.groups;
  auto chunks = [&](long long slice) { return (T + kWarps * slice - 1) / (kWarps * slice); };
  long long slice = 64;
  while (slice > 8 && chunks(slice) > 1 && units * chunks(slice) < kFill) slice /= 2;
  while (chunks(slice) > 256) slice *= 2;
  p.nchunks = static_cast<int>(chunks(slice));
  p.warps = kWarps;
  if (p.nchunks == 1) {
    p.warps = std::max(1, std::min(kWarps, T / kBatch));
    slice = ((T + p.warps - 1) / p.warps + kBatch - 1) / kBatch * kBatch;
  } else {
    const size_t width = static_cast<size_t>(p.groups) * 32 * V;
    p.chunk_pairs = static_cast<size_t>(B) * p.nchunks * width;
    p.slice_pairs = p.chunk_pairs * kWarps;
  }
  p.slice = static_cast<int>(slice);
  return p;
}

template <typename X, typename G, int V, bool kHead, bool kBack>
cudaError_t launch(const ScanParams& p, int B, int dev, void* workspace, cudaStream_t st) {
  const ScanPlan plan = plan_scan(B, p.T, p.C, V);
  ScanParams a = p;
  a.groups = plan.groups;
  a.slice = plan.slice;
  a.nchunks = plan.nchunks;
  a.slices = static_cast<float2*>(workspace);
  a.chunks = a.slices + plan.slice_pairs;
  const long long ctas = static_cast<long long>(B) * plan.groups * plan.nchunks;
  if (ctas > INT_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(32 * plan.warps);
  cfg.stream = st;
  auto* pairs = &arl2_scan_pairs_kernel<X, G, V, kHead, kBack>;
  auto* apply = &arl2_scan_apply_kernel<X, G, V, kHead, kBack>;
  constexpr uint32_t kPairsRing = kWarps * ring_bytes<X, G, V, kHead, false>();
  constexpr uint32_t kApplyRing = kWarps * ring_bytes<X, G, V, kHead, kBack>();
  cudaError_t e = cudaSuccess;
  static std::atomic<unsigned long long> allowed{0};   // devices that were told, by bit
  if (!(allowed.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(pairs, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kPairsRing));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(apply, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kApplyRing));
    if (e != cudaSuccess) return e;
    allowed.fetch_or(1ull << dev, std::memory_order_release);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 0;
  if (plan.nchunks > 1) {
    cfg.dynamicSmemBytes = kPairsRing;
    e = cudaLaunchKernelEx(&cfg, pairs, a);
    if (e != cudaSuccess) return e;
    cfg.numAttrs = 1;
  }
  cfg.dynamicSmemBytes = kApplyRing / kWarps * plan.warps;
  return cudaLaunchKernelEx(&cfg, apply, a);
}

template <typename X, typename G, bool kBack>
cudaError_t by_width(const ScanParams& p, int B, int dev, void* ws, bool head, bool wide, cudaStream_t st) {
  if (head) return launch<X, float, 4, true, kBack>(p, B, dev, ws, st);
  return wide ? launch<X, G, 4, false, kBack>(p, B, dev, ws, st) : launch<X, G, 1, false, kBack>(p, B, dev, ws, st);
}

template <bool kBack>
cudaError_t by_type(const ScanParams& p, int B, int dev, void* ws, arl2_dtype x, arl2_dtype g, bool head, bool wide,
                    cudaStream_t st) {
  const bool gf = g == ARL2_FP32;
  if (x == ARL2_FP32) return by_width<float, float, kBack>(p, B, dev, ws, head, wide, st);
  if (x == ARL2_BF16)
    return gf ? by_width<__nv_bfloat16, float, kBack>(p, B, dev, ws, head, wide, st)
              : by_width<__nv_bfloat16, __nv_bfloat16, kBack>(p, B, dev, ws, head, wide, st);
  return gf ? by_width<__half, float, kBack>(p, B, dev, ws, head, wide, st)
            : by_width<__half, __half, kBack>(p, B, dev, ws, head, wide, st);
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
  if (s.T > 1 << 30) return ARL2_ERR_UNSUPPORTED;
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

// The current device, checked on its first call.
arl2_status current_device(int* dev) {
  static std::atomic<unsigned long long> known{0};
  if (cudaGetDevice(dev) != cudaSuccess) return ARL2_ERR_CUDA;
  if (*dev < 0 || *dev > 63) return ARL2_ERR_UNSUPPORTED;
  if (known.load(std::memory_order_acquire) >> *dev & 1) return ARL2_OK;
  int sms = 0;
  const arl2_status s = static_cast<arl2_status>(prepare_device(dev, &sms));
  if (s == ARL2_OK) known.fetch_or(1ull << *dev, std::memory_order_release);
  return s;
}

size_t workspace_bytes(const arl2_scan_shape& s) {
  // Whether groups of 4 channels can be accessed at once is known only with the pointers.
  size_t pairs = 0;
  for (int V : {1, 4}) {
    const ScanPlan p = plan_scan(s.B, s.T, s.C, V);
    pairs = std::max(pairs, p.slice_pairs + p.chunk_pairs);
  }
  return pairs * sizeof(float2);
}
bool needs_workspace(const arl2_scan_shape& s) { return workspace_bytes(s) > 0; }

}  // namespace
}  // namespace arl2

extern "C" size_t arl2_scan_workspace_bytes(const arl2_scan_shape* s) {
  bool head = false;
  return s && arl2::check(*s, &head) == ARL2_OK ? arl2::workspace_bytes(*s) : 0;
}

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
  if (needs_workspace(s) && !(f->workspace && at(f->workspace, 16))) return ARL2_ERR_INVALID_ARG;
  int dev = 0;
  const arl2_status ds = current_device(&dev);
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
  return by_type<false>(p, s.B, dev, f->workspace, static_cast<arl2_dtype>(s.dtype), static_cast<arl2_dtype>(s.gate_dtype), head,
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
  if (needs_workspace(s) && !(f->workspace && at(f->workspace, 16))) return ARL2_ERR_INVALID_ARG;
  int dev = 0;
  const arl2_status ds = current_device(&dev);
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
  return by_type<true>(p, s.B, dev, f->workspace, static_cast<arl2_dtype>(s.dtype), static_cast<arl2_dtype>(s.gate_dtype), head,
                       wide, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ARL2_OK
             : ARL2_ERR_CUDA;
}
