// Gated linear recurrence over a sequence, and its backward pass (arl2_scan_* in arl2.h):
//     h_t   = a_t h_{t-1} + x_t                                     h_{-1} = h0 (or 0)
//     lam_t = dh_t + a_{t+1} lam_{t+1},  lam_{T-1} = dh_{T-1} + dfinal
//     dx_t = lam_t,  da_t = lam_t h_{t-1},  dh0 = a_0 lam_0
// per channel, with a gate per channel and token, or one per head and token (da is then the
// sum over the head's channels). Both directions are the same scan: (A, X) pairs compose as
// (A2, X2) after (A1, X1) = (A1 A2, A2 X1 + X2).
//
// The work is a few operations per element read, so memory traffic bounds it, provided that few
// instructions are spent per byte: a lane takes V channels, 16 bytes, at once. `lanes` lanes hold
// a row of a channel group; they own a slice of consecutive tokens and stream it through a ring
// in shared memory (cp.async, each lane copying what it reads itself, so no barrier is needed).
// The slices of a CTA follow one another in time and form a chunk. Two launches:
//   - arl2_scan_pairs_kernel reads x (dh) and a, and writes the (A, X) of every slice and of
//     every chunk to the workspace;
//   - arl2_scan_apply_kernel composes the pairs before each slice onto the initial state,
//     then streams the slice again from that state and writes the results.
// The second reading is what this costs over a single pass: 100 + 100 read and 100 written MB take
// 58 us on 32760 tokens of 1536 bf16 channels (5.2 TB/s; without the stores 43 us). Part of it comes
// from L2: the first launch goes through each slice from its end to its start, so that the second
// begins with what was read last, and results are stored evict-first. Cutting long sequences into
// segments that fit L2, one launch each, lost more to the launches (81 us). A single-pass form (a
// cluster's CTAs following one another in time, pairs exchanged through distributed shared memory)
// moved in lock step with a barrier per 1024 tokens (115 us). A sequence that one chunk holds takes
// one launch, without workspace.
// The order of all products and sums is fixed, so results do not depend on timing. All of it is
// fp32; only the stored h, dx and da are rounded, once, to their types.
#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/arl2.h"
#include "arl2_device.cuh"
#include "arl2_kernels.h"

namespace arl2 {
namespace {

constexpr int kWarps = 8;       // warps per CTA
constexpr int kMinLanes = 8;    // lanes of a row, at least
constexpr int kBatchMax = 8;    // slices are multiples of it

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
  float2* slices;      // [B][chunks * parts][width] (A, X) of each slice
  float2* chunks;      // [B][chunks][width] of each chunk
  long long in_b, in_t, a_b, a_t, a_h, h_b, h_t, out_b, out_t, da_b, da_t, da_h;   // strides, elements
  int T, C, d;         // d: channels per gate (heads), or 1
  int lanes;           // lanes per row: 8, 16 or 32
  int groups;          // channel groups of lanes * V; width = groups * lanes * V
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

// Two 16-bit values, and two fp32 ones rounded to them.
template <typename T>
__device__ __forceinline__ float2 widen_pair(uint32_t w) {
  if constexpr (std::is_same_v<T, __half>)
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t round_pair(float lo, float hi) {
  if constexpr (std::is_same_v<T, __half>) {
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    return pack_bf16x2(lo, hi);
  }
}

// V values of type T, accessed 16 bytes at a time.
template <typename T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Pack {
  T v[V];
  __device__ __forceinline__ void widen(float (&f)[V]) const {
    if constexpr (sizeof(T) == 2 && V > 1) {   // by pairs: one instruction a value
      const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 x = widen_pair<T>(w[i / 2]);
        f[i] = x.x;
        f[i + 1] = x.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = to_f(v[i]);
    }
  }
  __device__ __forceinline__ void round(const float (&f)[V]) {
    if constexpr (sizeof(T) == 2 && V > 1) {
      uint32_t* w = reinterpret_cast<uint32_t*>(v);
#pragma unroll
      for (int i = 0; i < V; i += 2) w[i / 2] = round_pair<T>(f[i], f[i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = from_f<T>(f[i]);
    }
  }
};

// A load of one element that stays where it is written: the compiler would otherwise move each next
// to its use, to save registers, and the loads of a batch would wait for one another.
template <typename P>
__device__ __forceinline__ P load_now(const void* src) {
  P r;
  if constexpr (sizeof(P) == 4) {
    asm volatile("ld.global.u32 %0, [%1];" : "=r"(*reinterpret_cast<uint32_t*>(&r)) : "l"(src));
  } else {
    static_assert(sizeof(P) == 2);
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(*reinterpret_cast<uint16_t*>(&r)) : "l"(src));
  }
  return r;
}

// s = g s + x with the paired fp32 operations; one gate (GV = 1) or one per value.
template <int V, int GV>
__device__ __forceinline__ void advance(float (&s)[V], const float (&g)[GV], const float (&x)[V]) {
  if constexpr (V == 1) {
    s[0] = fmaf(g[0], s[0], x[0]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 r = __ffma2_rn(make_float2(g[GV == 1 ? 0 : i], g[GV == 1 ? 0 : i + 1]), make_float2(s[i], s[i + 1]),
                                  make_float2(x[i], x[i + 1]));
      s[i] = r.x;
      s[i + 1] = r.y;
    }
  }
}
// s += g x.
template <int V, int GV>
__device__ __forceinline__ void accumulate(float (&s)[V], const float (&g)[GV], const float (&x)[V]) {
  if constexpr (V == 1) {
    s[0] = fmaf(g[0], x[0], s[0]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 r = __ffma2_rn(make_float2(g[GV == 1 ? 0 : i], g[GV == 1 ? 0 : i + 1]), make_float2(x[i], x[i + 1]),
                                  make_float2(s[i], s[i + 1]));
      s[i] = r.x;
      s[i + 1] = r.y;
    }
  }
}
template <int GV>
__device__ __forceinline__ void scale_by(float (&a)[GV], const float (&g)[GV]) {
#pragma unroll
  for (int i = 0; i < GV; ++i) a[i] *= g[i];
}
// Products of gates above 1 over many tokens may pass fp32's range where the state they meet does not:
// a state of 0 stays 0, and a gate of 0 makes the product 0, where inf * 0 would be a NaN. Of the gates
// themselves, only a NaN does that.
__device__ __forceinline__ float past(float2 pair, float s) {   // a state moved past a pair
  return s == 0.f && pair.x == pair.x ? pair.y : fmaf(pair.x, s, pair.y);
}
__device__ __forceinline__ float gate_product(float x, float y) {
  return (x == 0.f && y == y) || (y == 0.f && x == x) ? 0.f : x * y;
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// A store of data that this call does not read again: evict-first in L2.
template <typename P>
__device__ __forceinline__ void store_streaming(void* dst, const P& v) {
  if constexpr (sizeof(P) >= 16) {
#pragma unroll
    for (size_t i = 0; i < sizeof(P) / 16; ++i)
      __stcs(static_cast<uint4*>(dst) + i, reinterpret_cast<const uint4*>(&v)[i]);
  } else if constexpr (sizeof(P) == 4) {
    __stcs(static_cast<uint32_t*>(dst), *reinterpret_cast<const uint32_t*>(&v));
  } else {
    __stcs(static_cast<unsigned short*>(dst), *reinterpret_cast<const unsigned short*>(&v));
  }
}

// 4 bytes, 16 or 32 from global to shared memory in the background; zeros where !ok, and then src,
// though inside the tensor, is not read.
template <typename P>
__device__ __forceinline__ void copy_async(P* dst, const P* src, bool ok) {
  if constexpr (sizeof(P) == 4) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(ok ? 4u : 0u)
                 : "memory");
  } else {
    static_assert(sizeof(P) % 16 == 0);
#pragma unroll
    for (uint32_t i = 0; i < sizeof(P) / 16; ++i)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst) + 16u * i),
                   "l"(reinterpret_cast<uint64_t>(src) + 16 * i), "r"(ok ? 16u : 0u)
                   : "memory");
  }
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

struct True {
  static constexpr bool value = true;
};
struct False {
  static constexpr bool value = false;
};

// The copy ring of a warp: kStages batches of kB tokens of x (dh), of the gates and, with kPrev, of
// h, at most 9.75 KiB in all, so that two CTAs (their pairs included) fit an SM. Single elements
// (V = 1) are loaded straight, 8 tokens at once: 16-bit ones are too small for cp.async, and 32-bit
// ones cost less instructions this way (3 x 1561 tokens of 517 fp32 channels: 16 us, 29 us by ring).
template <typename X, typename G, int V, bool kHead, bool kPrev>
struct Ring {
  static constexpr bool kUsed = V > 1;
  static constexpr uint32_t kRowX = 32 * V * sizeof(X);
  static constexpr uint32_t kRow = kRowX * (kPrev ? 2 : 1) + (kHead ? 32 : 32 * V * sizeof(G));
  static constexpr int kB = V == 1 ? 8 : !kHead && kRow > 1024 ? 2 : 4;   // tokens worked on at once
  static constexpr uint32_t kBatchG = kHead ? 32 * 4 : kB * 32 * V * sizeof(G);
  static constexpr uint32_t kBatchBytes = kB * kRowX * (kPrev ? 2 : 1) + kBatchG;
  static constexpr int kMost = 9984 / kBatchBytes;
  static constexpr int kStages = kMost < 2 ? 2 : kMost > 8 ? 8 : kMost;
  static constexpr uint32_t kBytes = kUsed ? kStages * kBatchBytes : 0;   // per warp
};

// kB tokens of a lane's channels: values, gates, and (kPrev) the states before them.
template <typename PX, typename PG, int kB, bool kPrev>
struct Batch {
  PX x[kB], h[kPrev ? kB : 1];
  PG g[kB];
};

// Where a thread works: token q of the scan is token q of the sequence forward and token
// len - 1 - q backward.
template <typename X, typename G, int V, bool kHead, bool kBack, bool kPrev>
struct Place {
  static constexpr int GV = kHead ? 1 : V;   // gates per token a thread holds
  using R = Ring<X, G, V, kHead, kPrev>;
  static constexpr int kB = R::kB;
  using B = Batch<Pack<X, V>, Pack<G, GV>, kB, kPrev>;
  using PX = Pack<X, V>;
  using PG = Pack<G, GV>;
  int row_lane, part, parts, b, group, chunk, k, c, len;
  bool in_c;
  int q0, batches;     // this slice's first token; batches with a token inside, over the warp
  const X* in;
  const G* ga;
  const X* hp;
  uint8_t* ring;       // this warp's
  const G* head_ga;    // per head: the gates this lane copies (null: none)
  // Chunks slowest, so that the CTAs in flight work on neighbouring tokens.
  __device__ Place(const ScanParams& a, uint8_t* smem) {
    row_lane = threadIdx.x & (a.lanes - 1);
    part = threadIdx.x / a.lanes;
    parts = blockDim.x / a.lanes;
    int u = blockIdx.x;
    group = u % a.groups;
    u /= a.groups;
    const int nb = gridDim.x / (a.groups * a.nchunks);
    b = u % nb;
    chunk = u / nb;
    k = row_lane * V;                    // channel within the group
    c = group * a.lanes * V + k;
    in_c = c < a.C;                      // V divides C, or V = 1
    const int cl = in_c ? c : 0;         // lanes behind the last channel stay inside the tensor
    len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    q0 = (chunk * parts + part) * a.slice;
    batches = __reduce_max_sync(0xffffffffu, max(0, (min(q0 + a.slice, len) - q0 + kB - 1) / kB));
    in = static_cast<const X*>(a.in) + b * a.in_b + cl;
    ga = static_cast<const G*>(a.a) + b * a.a_b + (kHead ? (cl / a.d) * a.a_h : static_cast<long long>(cl));
    hp = kPrev ? static_cast<const X*>(a.hprev) + b * a.h_b + cl : nullptr;
    ring = smem + (threadIdx.x >> 5) * R::kBytes;
    head_ga = nullptr;
    if constexpr (kHead) {   // lane l of a row copies the gate of token l % kB and head l / kB of the group's
      const int head = group * a.lanes * V / a.d + row_lane / kB;
      if (row_lane / kB < a.lanes * V / a.d && head < a.C / a.d)
        head_ga = static_cast<const G*>(a.a) + b * a.a_b + head * a.a_h;
    }
  }
  __device__ int token(int q) const { return kBack ? len - 1 - q : q; }
  __device__ PX* ring_x(int stage, int i) const {
    return reinterpret_cast<PX*>(ring + stage * R::kBatchBytes + i * R::kRowX) + (threadIdx.x & 31);
  }
  __device__ PX* ring_h(int stage, int i) const {
    return reinterpret_cast<PX*>(ring + stage * R::kBatchBytes + (kB + i) * R::kRowX) + (threadIdx.x & 31);
  }
  __device__ uint8_t* ring_g(int stage) const {
    return ring + stage * R::kBatchBytes + kB * R::kRowX * (kPrev ? 2 : 1);
  }
  // The slice's batches are worked on in order (kReverse: from the last to the first). Start copying
  // the j-th of them to its stage: one group, empty behind the last.
  template <bool kReverse>
  __device__ __forceinline__ void copy(const ScanParams& a, int j) const {
    if constexpr (R::kUsed) {
      const int q = q0 + (kReverse ? batches - 1 - j : j) * kB, stage = j % R::kStages;
      if (j >= batches || q >= len) {
        // nothing
      } else if ((!kBack || q > 0) && q + kB + (kBack ? 1 : 0) <= len) {   // all inside: no clamping
        const int t0 = token(q);
        const X* px = in + t0 * a.in_t;
        const G* pg = ga + (kBack ? t0 + 1 : t0) * a.a_t;
        const X* ph = kPrev ? hp + (t0 - 1) * a.h_t : nullptr;
#pragma unroll
        for (int i = 0; i < kB; ++i) {
          copy_async(ring_x(stage, i), reinterpret_cast<const PX*>(px), true);
          px = kBack ? px - a.in_t : px + a.in_t;
          if constexpr (!kHead) {
            copy_async(reinterpret_cast<PG*>(ring_g(stage)) + i * 32 + (threadIdx.x & 31),
                       reinterpret_cast<const PG*>(pg), true);
            pg = kBack ? pg - a.a_t : pg + a.a_t;
          }
          if constexpr (kPrev) {
            copy_async(ring_h(stage, i), reinterpret_cast<const PX*>(ph), true);
            ph -= a.h_t;
          }
        }
        if constexpr (kHead) {
          if (head_ga)
            copy_async(reinterpret_cast<G*>(ring_g(stage)) + (threadIdx.x & 31),
                       head_ga + (token(q + row_lane % kB) + (kBack ? 1 : 0)) * a.a_t, true);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kB; ++i) {
          const bool ok = q + i < len && in_c;
          const int t = max(token(q + i), 0), tl = min(t, len - 1);
          copy_async(ring_x(stage, i), reinterpret_cast<const PX*>(in + tl * a.in_t), ok);
          if constexpr (!kHead)
            copy_async(reinterpret_cast<PG*>(ring_g(stage)) + i * 32 + (threadIdx.x & 31),
                       reinterpret_cast<const PG*>(ga + (kBack ? min(tl + 1, len - 1) : tl) * a.a_t), ok);
          if constexpr (kPrev)
            copy_async(ring_h(stage, i), reinterpret_cast<const PX*>(hp + max(tl - 1, 0) * a.h_t), ok && t > 0);
        }
        if constexpr (kHead) {
          const int qi = q + row_lane % kB, t = min(max(token(qi), 0) + (kBack ? 1 : 0), len - 1);
          if (head_ga)
            copy_async(reinterpret_cast<G*>(ring_g(stage)) + (threadIdx.x & 31), head_ga + t * a.a_t, qi < len);
        }
      }
      copy_commit();
    }
  }
  template <bool kReverse>
  __device__ __forceinline__ void start(const ScanParams& a) const {
#pragma unroll
    for (int j = 0; j < R::kStages; ++j) copy<kReverse>(a, j);
  }
  // After start(): work(inner, q, batch) for each batch of the slice, by whole warps.
  // inner is True where all of the batch, and of its neighbours, is inside the sequence.
  // Elsewhere what lies behind the length has value 0 and gate 1, so that a state passes
  // unchanged; backward, the last token's gate is 1 too (dfinal reaches it undamped).
  template <bool kReverse, typename Work>
  __device__ __forceinline__ void stream(const ScanParams& a, Work&& work) const {
    for (int j = 0; j < batches; ++j) {
      const int q = q0 + (kReverse ? batches - 1 - j : j) * kB;
      const bool inner = __all_sync(0xffffffffu, (!kBack || q > 0) && q + kB + (kBack ? 1 : 0) <= len);
      B r;
      if constexpr (R::kUsed) {
        const int stage = j % R::kStages;
        copy_wait<R::kStages - 1>();
        if (kHead) __syncwarp();   // gates are copied by other lanes than those that read them
#pragma unroll
        for (int i = 0; i < kB; ++i) {
          r.x[i] = *ring_x(stage, i);
          if constexpr (kPrev) r.h[i] = *ring_h(stage, i);
          if constexpr (kHead)   // this row's lanes, its head, its token
            r.g[i].v[0] = reinterpret_cast<const float*>(ring_g(stage))[(threadIdx.x & 31 & ~(a.lanes - 1)) +
                                                                        row_lane * V / a.d * kB + i];
          else
            r.g[i] = reinterpret_cast<const PG*>(ring_g(stage))[i * 32 + (threadIdx.x & 31)];
        }
      } else {
#pragma unroll
        for (int i = 0; i < kB; ++i) {
          const int t = max(token(q + i), 0), tl = min(t, len - 1);
          r.x[i] = load_now<PX>(in + tl * a.in_t);
          r.g[i] = load_now<PG>(ga + (kBack ? min(tl + 1, len - 1) : tl) * a.a_t);
          if constexpr (kPrev) r.h[i] = load_now<PX>(hp + max(tl - 1, 0) * a.h_t);
        }
      }
      if (inner) {
        work(True{}, q, r);
      } else {
#pragma unroll
        for (int i = 0; i < kB; ++i) {
          const bool ok = q + i < len, gok = ok && (!kBack || q + i > 0);
#pragma unroll
          for (int v = 0; v < V; ++v) r.x[i].v[v] = ok ? r.x[i].v[v] : from_f<X>(0.f);
#pragma unroll
          for (int v = 0; v < GV; ++v) r.g[i].v[v] = gok ? r.g[i].v[v] : from_f<G>(1.f);
        }
        work(False{}, q, r);
      }
      if (kHead) __syncwarp();
      copy<kReverse>(a, j + R::kStages);
    }
  }
  // The (A, X) of this slice, after start<true>(): from the end, X = sum of x times the gates behind.
  // Where their product passed fp32's range (rare), X was made of it too: then once more in the order
  // of the recurrence, in which X stays a state.
  __device__ __forceinline__ void pairs(const ScanParams& a, float2 (&pair)[V]) const {
    float A[GV], S[V];
#pragma unroll
    for (int v = 0; v < GV; ++v) A[v] = 1.f;
#pragma unroll
    for (int v = 0; v < V; ++v) S[v] = 0.f;
    stream<true>(a, [&](auto, int, const B& r) {
#pragma unroll
      for (int i = kB - 1; i >= 0; --i) {
        float xf[V], gf[GV];
        r.x[i].widen(xf);
        r.g[i].widen(gf);
        accumulate(S, A, xf);
        scale_by(A, gf);
      }
    });
    bool in_range = true;
#pragma unroll
    for (int v = 0; v < GV; ++v) in_range = in_range && finite(A[v]);
#pragma unroll
    for (int v = 0; v < V; ++v) in_range = in_range && finite(S[v]);
    if (__any_sync(0xffffffffu, !in_range && in_c)) {
#pragma unroll
      for (int v = 0; v < GV; ++v) A[v] = 1.f;
#pragma unroll
      for (int v = 0; v < V; ++v) S[v] = 0.f;
      start<false>(a);
      stream<false>(a, [&](auto, int, const B& r) {
#pragma unroll
        for (int i = 0; i < kB; ++i) {
          float xf[V], gf[GV];
          r.x[i].widen(xf);
          r.g[i].widen(gf);
          advance(S, gf, xf);
#pragma unroll
          for (int v = 0; v < GV; ++v) A[v] = gate_product(A[v], gf[v]);
        }
      });
    }
#pragma unroll
    for (int v = 0; v < V; ++v) pair[v] = make_float2(A[kHead ? 0 : v], S[v]);
  }
};

// A row of pairs, V of them per lane.
template <int V>
__device__ __forceinline__ void load_pairs(const float2* src, float2 (&r)[V]) {
  if constexpr (V == 1) {
    r[0] = src[0];
  } else {
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      const float4 p = *reinterpret_cast<const float4*>(src + v);
      r[v] = make_float2(p.x, p.y);
      r[v + 1] = make_float2(p.z, p.w);
    }
  }
}
template <int V>
__device__ __forceinline__ void store_pairs(float2* dst, const float2 (&r)[V]) {
  if constexpr (V == 1) {
    dst[0] = r[0];
  } else {
#pragma unroll
    for (int v = 0; v < V; v += 2)
      *reinterpret_cast<float4*>(dst + v) = make_float4(r[v].x, r[v].y, r[v + 1].x, r[v + 1].y);
  }
}

template <typename X, typename G, int V, bool kHead, bool kBack>
__global__ void __launch_bounds__(32 * kWarps, 2)
    arl2_scan_pairs_kernel(const __grid_constant__ ScanParams a) {
  __shared__ __align__(16) float2 s_pair[kWarps * 32 * V];   // [parts][lanes V]
  extern __shared__ __align__(16) uint8_t ring[];
  griddep_launch_dependents();
  const Place<X, G, V, kHead, kBack, false> p(a, ring);
  float2 r[V];
  p.template start<true>(a);
  p.pairs(a, r);
  const int wide = a.lanes * V;
  const long long width = static_cast<long long>(a.groups) * wide;
  const long long row = static_cast<long long>(p.b) * a.nchunks + p.chunk;
  store_pairs(a.slices + (row * p.parts + p.part) * width + p.group * wide + p.k, r);
  store_pairs(s_pair + p.part * wide + p.k, r);
  __syncthreads();
  for (int k = threadIdx.x; k < wide; k += blockDim.x) {
    float2 n = s_pair[k];
#pragma unroll 4
    for (int w = 1; w < p.parts; ++w) {
      const float2 m = s_pair[w * wide + k];
      n = make_float2(gate_product(n.x, m.x), past(m, n.y));
    }
    a.chunks[row * width + p.group * wide + k] = n;
  }
}

// Sums of kB values over the lanes of a head (d / V of them, a power of two >= kB), by halving
// the values held: each exchange sends the half that the partner keeps. Lane l of a head ends
// with the sum of value l / same % kB, which `same` = lanes / kB neighbouring lanes hold.
template <int kB>
__device__ __forceinline__ float head_sums(float (&r)[kB], int lanes, int lane, int* index) {
  int m = lanes >> 1;
#pragma unroll
  for (int n = kB / 2; n >= 1; n >>= 1, m >>= 1) {
    const bool upper = (lane & m) != 0;   // keeps the upper half of the values
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = upper ? r[i] : r[i + n], keep = upper ? r[i + n] : r[i];
      r[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
    }
  }
  for (; m > 0; m >>= 1) r[0] += __shfl_xor_sync(0xffffffffu, r[0], m);
  *index = lane / (lanes / kB) % kB;
  return r[0];
}

template <typename X, typename G, int V, bool kHead, bool kBack>
__global__ void __launch_bounds__(32 * kWarps, 2)
    arl2_scan_apply_kernel(const __grid_constant__ ScanParams a) {
  using P = Place<X, G, V, kHead, kBack, kBack>;
  using PX = typename P::PX;
  using PG = typename P::PG;
  constexpr int GV = P::GV, kB = P::kB;
  __shared__ __align__(16) float2 s_pair[kWarps * 32 * V];    // each part's share of the earlier chunks
  __shared__ __align__(16) float2 s_slice[kWarps * 32 * V];   // the chunk's slices
  extern __shared__ __align__(16) uint8_t ring[];
  const P p(a, ring);
  const bool single = a.nchunks == 1 && p.parts > 1;   // the slices' pairs are made here
  if (single)
    p.template start<true>(a);
  else
    p.template start<false>(a);   // in flight while the state it starts from is composed
  const int len = p.len, wide = a.lanes * V;
  float state[V];
#pragma unroll
  for (int v = 0; v < V; ++v) state[v] = a.init && p.in_c ? a.init[static_cast<long long>(p.b) * a.C + p.c + v] : 0.f;

  // The state this slice starts from: every part brings its slice's pair and composes its share
  // of the earlier chunks; all meet in shared memory.
  if (single) {
    float2 own[V];
    p.pairs(a, own);
    p.template start<false>(a);
    store_pairs(s_slice + p.part * wide + p.k, own);
  } else if (a.nchunks > 1) {
    griddep_wait();   // the pairs kernel's results
    const long long width = static_cast<long long>(a.groups) * wide;
    const long long row = static_cast<long long>(p.b) * a.nchunks;
    float2 own[V], sum[V];
    load_pairs(a.slices + ((row + p.chunk) * p.parts + p.part) * width + p.group * wide + p.k, own);
    const int share = (p.chunk + p.parts - 1) / p.parts;
    const int k0 = min(p.part * share, p.chunk), k1 = min(k0 + share, p.chunk);
#pragma unroll
    for (int v = 0; v < V; ++v) sum[v] = make_float2(1.f, 0.f);
    const float2* src = a.chunks + (row + k0) * width + p.group * wide + p.k;
#pragma unroll 2
    for (int i = k0; i < k1; ++i, src += width) {
      float2 n[V];
      load_pairs(src, n);
#pragma unroll
      for (int v = 0; v < V; ++v) sum[v] = make_float2(gate_product(sum[v].x, n[v].x), past(n[v], sum[v].y));
    }
    store_pairs(s_pair + p.part * wide + p.k, sum);
    store_pairs(s_slice + p.part * wide + p.k, own);
  }
  if (p.parts > 1) {
    __syncthreads();
    if (a.nchunks > 1) {
#pragma unroll 2
      for (int w = 0; w < p.parts; ++w) {
        float2 n[V];
        load_pairs(s_pair + w * wide + p.k, n);
#pragma unroll
        for (int v = 0; v < V; ++v) state[v] = past(n[v], state[v]);
      }
    }
#pragma unroll 2
    for (int w = 0; w < p.part; ++w) {
      float2 n[V];
      load_pairs(s_slice + w * wide + p.k, n);
#pragma unroll
      for (int v = 0; v < V; ++v) state[v] = past(n[v], state[v]);
    }
  }

  X* out = static_cast<X*>(a.out) + p.b * a.out_b + p.c;
  G* da = kBack ? static_cast<G*>(a.da) + p.b * a.da_b + (kHead ? (p.c / a.d) * a.da_h : static_cast<long long>(p.c))
                : nullptr;
  p.template stream<false>(a, [&](auto inner, int q, const typename P::B& r) {
    constexpr bool kInner = decltype(inner)::value;
    const int t0 = p.token(q);
    X* po = out + t0 * a.out_t;
    [[maybe_unused]] G* pa = kBack && !kHead ? da + t0 * a.da_t : nullptr;
    [[maybe_unused]] float sums[kB];
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      const bool ok = (kInner || q + i < len) && p.in_c;
      float xf[V], gf[GV];
      r.x[i].widen(xf);
      r.g[i].widen(gf);
      advance(state, gf, xf);
      PX o;
      o.round(state);
      if (ok) store_streaming(po, o);
      po = kBack ? po - a.out_t : po + a.out_t;
      if constexpr (kBack) {
        float hf[V];
        r.h[i].widen(hf);
        if constexpr (!kInner) {
          if (p.token(q + i) <= 0) {   // h_{-1}
#pragma unroll
            for (int v = 0; v < V; ++v)
              hf[v] = a.h0 && p.in_c ? a.h0[static_cast<long long>(p.b) * a.C + p.c + v] : 0.f;
          }
        }
        if constexpr (kHead) {
          float2 s = make_float2(0.f, 0.f);
#pragma unroll
          for (int v = 0; v < V; v += 2)
            s = __ffma2_rn(make_float2(state[v], state[v + 1]), make_float2(hf[v], hf[v + 1]), s);
          sums[i] = s.x + s.y;
        } else {
          PG o2;
#pragma unroll
          for (int v = 0; v < GV; ++v) hf[v] *= state[v];
          o2.round(hf);
          if (ok) store_streaming(pa, o2);
          pa -= a.da_t;
        }
      }
    }
    if constexpr (kBack && kHead) {
      const int lanes = a.d / V;
      int i = 0;
      const float sum = head_sums(sums, lanes, threadIdx.x & 31, &i);
      const bool writer = p.in_c && p.row_lane % (lanes / kB) == 0;   // one of the lanes that hold it
      if (writer && (kInner || q + i < len)) da[p.token(q + i) * a.da_t] = from_f<G>(sum);
    }
  });

  // The part whose slice holds the last token (the first slice, of an empty sequence) has the
  // final state.
  if (a.last && p.in_c && (len > 0 ? p.q0 < len && p.q0 + a.slice >= len : p.q0 == 0)) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float g = kBack && len > 0 ? to_f(p.ga[kHead ? 0 : v]) : 1.f;   // dh0 = a_0 lam_0
      a.last[static_cast<long long>(p.b) * a.C + p.c + v] = g * state[v];
    }
  }
  // Behind the length: zeros (each part in its own slice's place).
  for (int t = max(p.q0, len); t < min(p.q0 + a.slice, a.T); ++t) {
    PX z;
#pragma unroll
    for (int v = 0; v < V; ++v) z.v[v] = from_f<X>(0.f);
    if (p.in_c) *reinterpret_cast<PX*>(out + t * a.out_t) = z;
    if constexpr (kBack && kHead) {
      if (p.in_c && p.c % a.d == 0) da[t * a.da_t] = from_f<G>(0.f);
    } else if constexpr (kBack) {
      PG gz;
#pragma unroll
      for (int v = 0; v < GV; ++v) gz.v[v] = from_f<G>(0.f);
      if (p.in_c) *reinterpret_cast<PG*>(da + t * a.da_t) = gz;
    }
  }
}

// How a call is cut. The CTAs are to fill the GPU once, two for each SM of a B200: more would mean
// more pairs to write and to compose (each CTA composes all the chunks before its own), fewer leave
// SMs idle (32760 tokens of 1536 channels: 62 us with two, 72 with three, 79 with four). Without the
// ring, twice as many: their loads are hidden by other warps alone. So chunks are as many as that
// allows, at most 256 a sequence, in slices of 8 tokens or more. A sequence of at most one chunk of
// 64-token slices is one chunk, cut into no more parts than it has batches.
struct ScanPlan {
  int lanes, groups, slice, nchunks, warps;
  size_t slice_pairs, chunk_pairs;   // workspace, in (A, X) pairs
  size_t init_floats;                // behind them, room for a copy of h0
};
ScanPlan plan_scan(int B, int T, int C, int V) {
  ScanPlan p{};
  p.lanes = 32;
  while (p.lanes > kMinLanes && (p.lanes / 2) * V >= C) p.lanes /= 2;
  p.groups = (C + p.lanes * V - 1) / (p.lanes * V);
  const int per_warp = 32 / p.lanes, parts = kWarps * per_warp;
  const long long units = static_cast<long long>(B) * p.groups;
  auto chunks = [&](long long slice) { return (T + parts * slice - 1) / (parts * slice); };
  long long slice = 64;
  if (chunks(slice) > 1) {
    const long long fill = (V > 1 ? 2 : 4) * 148;
    const long long want = std::min<long long>(256, std::max<long long>(1, fill / units));
    slice = (T + parts * want - 1) / (parts * want);
    slice = std::max<long long>(kBatchMax, (slice + kBatchMax - 1) / kBatchMax * kBatchMax);
  }
  p.nchunks = static_cast<int>(chunks(slice));
  p.warps = kWarps;
  if (p.nchunks == 1) {
    p.warps = std::max(1, std::min(kWarps, T / (kBatchMax * per_warp)));
    const int n = p.warps * per_warp;
    slice = ((T + n - 1) / n + kBatchMax - 1) / kBatchMax * kBatchMax;
  } else {
    const size_t width = static_cast<size_t>(p.groups) * p.lanes * V;
    p.chunk_pairs = static_cast<size_t>(B) * p.nchunks * width;
    p.slice_pairs = p.chunk_pairs * parts;
    p.init_floats = static_cast<size_t>(B) * C;
  }
  p.slice = static_cast<int>(slice);
  return p;
}

template <typename X, typename G, int V, bool kHead, bool kBack>
cudaError_t launch(const ScanParams& p, int B, int dev, void* workspace, cudaStream_t st) {
  const ScanPlan plan = plan_scan(B, p.T, p.C, V);
  ScanParams a = p;
  a.lanes = plan.lanes;
  a.groups = plan.groups;
  a.slice = plan.slice;
  a.nchunks = plan.nchunks;
  a.slices = static_cast<float2*>(workspace);
  a.chunks = a.slices + plan.slice_pairs;
  if (a.init && a.init == a.last && plan.nchunks > 1) {
    // The final state goes where the initial one stands, which CTAs that start late still have to read.
    void* copy = a.chunks + plan.chunk_pairs;
    const cudaError_t e =
        cudaMemcpyAsync(copy, a.init, plan.init_floats * sizeof(float), cudaMemcpyDeviceToDevice, st);
    if (e != cudaSuccess) return e;
    a.init = static_cast<const float*>(copy);
  }
  const long long ctas = static_cast<long long>(B) * plan.groups * plan.nchunks;
  if (ctas > INT_MAX) return cudaErrorInvalidConfiguration;
  auto* pairs = &arl2_scan_pairs_kernel<X, G, V, kHead, kBack>;
  auto* apply = &arl2_scan_apply_kernel<X, G, V, kHead, kBack>;
  constexpr uint32_t kPairsRing = Ring<X, G, V, kHead, false>::kBytes, kApplyRing = Ring<X, G, V, kHead, kBack>::kBytes;
  static std::atomic<unsigned long long> allowed{0};   // devices that were told of the rings, by bit
  if (!(allowed.load(std::memory_order_acquire) >> dev & 1)) {
    cudaError_t e = cudaFuncSetAttribute(pairs, cudaFuncAttributeMaxDynamicSharedMemorySize, kWarps * kPairsRing);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(apply, cudaFuncAttributeMaxDynamicSharedMemorySize, kWarps * kApplyRing);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(1ull << dev, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(32 * plan.warps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 0;
  if (plan.nchunks > 1) {
    cfg.dynamicSmemBytes = kWarps * kPairsRing;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, pairs, a);
    if (e != cudaSuccess) return e;
    cfg.numAttrs = 1;
  }
  cfg.dynamicSmemBytes = plan.warps * kApplyRing;
  return cudaLaunchKernelEx(&cfg, apply, a);
}

template <typename X, typename G, bool kBack>
cudaError_t by_width(const ScanParams& p, int B, int dev, void* ws, bool head, bool wide, cudaStream_t st) {
  constexpr int V = 16 / sizeof(X);
  if (head) return launch<X, float, V, true, kBack>(p, B, dev, ws, st);
  return wide ? launch<X, G, V, false, kBack>(p, B, dev, ws, st) : launch<X, G, 1, false, kBack>(p, B, dev, ws, st);
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

// A [B, T, C] tensor, unit channel stride: whether its strides are in range, and whether 16 bytes
// of it can be accessed at once. An output's elements must not share memory.
bool strides_ok(const Strides& x, int B, int T, int C, bool output) {
  const long long sb = x.b, st = x.t;
  if (sb < 0 || st < 0 || x.h < 0) return false;
  if (!output) return true;
  if (T > 1 && st < C) return false;
  if (B > 1 && sb < (T > 1 ? (T - 1) * st : 0) + C && !(sb >= C && T > 1 && st >= (B - 1) * sb + C)) return false;
  return true;
}
bool wide_ok(const void* p, size_t e, const Strides& x) {
  const long long v = 16 / e;
  return at(p, 16) && x.b % v == 0 && x.t % v == 0;
}

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
  // Whether 16 bytes can be accessed at once is known only with the pointers.
  size_t bytes = 0;
  for (int V : {1, static_cast<int>(16 / elem(s.dtype))}) {
    const ScanPlan p = plan_scan(s.B, s.T, s.C, V);
    bytes = std::max(bytes, (p.slice_pairs + p.chunk_pairs) * sizeof(float2) + p.init_floats * sizeof(float));
  }
  return bytes;
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
  bool wide = s.C % (16 / e) == 0 && wide_ok(f->x, e, xs) && wide_ok(f->h, e, hs);
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
  return by_type<false>(p, s.B, dev, f->workspace, static_cast<arl2_dtype>(s.dtype),
                        static_cast<arl2_dtype>(s.gate_dtype), head, wide, static_cast<cudaStream_t>(stream)) == cudaSuccess
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
  bool wide = s.C % (16 / e) == 0 && wide_ok(f->dh, e, gs) && wide_ok(f->h, e, hs) && wide_ok(f->dx, e, xs);
  if (head && !wide) return ARL2_ERR_INVALID_ARG;
  if (!head) wide = wide && wide_ok(f->a, ge, as) && at(f->da, 16);
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
  return by_type<true>(p, s.B, dev, f->workspace, static_cast<arl2_dtype>(s.dtype),
                       static_cast<arl2_dtype>(s.gate_dtype), head, wide, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ARL2_OK
             : ARL2_ERR_CUDA;
}
