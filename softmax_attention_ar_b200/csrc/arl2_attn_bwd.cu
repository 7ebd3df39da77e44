// Backward pass of softmax attention with the probabilities recomputed (arl2_attn_backward):
//     P = exp(scale q k^T - lse),   delta_i = sum_c do_ic o_ic,   dP = do v^T,   dS = P (dP - delta)
//     dv = P^T do,   dk = scale dS^T q,   dq = scale dS k
// over the visible pairs (arl2_attn.cuh). lse comes from the forward call, so P needs no second
// pass over the keys.
//
// The tensor cores bound it. Launches, the second and the third each a programmatic dependent of the
// one before (behind a split launch, arl2_attn.cuh, prep is an ordinary one):
//   - arl2_attn_prep_kernel: -delta, and -lse in log2 units (-inf where a row sees nothing or lies
//     behind its length: P is then 0), padded to whole 128-row tiles;
//   - arl2_attn_bwd_kernel, some of whose CTAs compute dk and dv (dkv_cta): a tile is 128 keys of
//     one key head and runs over the query tiles of every query head that shares the head, so the
//     heads' sum stays in the accumulators; and the others dq (dq_cta): a tile is 128 query rows of
//     one head and runs over the key tiles;
//   - arl2_attn_bwd_combine_kernel: adds up the records of tiles shared between CTAs.
// S and dP are computed in both, 7 products a tile pair instead of the 5 of a single pass. In
// return no dq leaves the SM before it is complete: a single pass would add 64 KiB of fp32 per
// tile pair to memory, with atomics whose order changes the result or an ordering that stalls,
// and dS would pass through shared memory. Here P and dS go back to TMEM, in place over the
// scores they came from, and feed the next product as its A operand; shared memory holds only
// what TMA brought.
//
// Roles (384 threads, one CTA per SM): warp 0 copies, warp 1 issues every MMA, warps 4-11 turn
// scores into P and dS: thread = TMEM lane = row of the tile, warps 4-7 columns 0-63, 8-11 columns
// 64-127, each in two packed halves (32 columns in place of 64 fp32 ones, at columns 0 and 64).
// P and dS are rounded to 16 bits for the tensor cores, in fp16 times powers of two that keep them in
// its range (GradRange); sums, statistics and gradients are fp32.
#include <algorithm>

#include "arl2_attn_kernels.h"

namespace arl2 {
namespace {

constexpr int kBwdThreads = 384;
constexpr uint32_t kBCtl = 512;   // barriers, split, flags
// Exponentials on the FMA pipe: pairs 2, 5, 7 of 8. One 480p frame 78.8 us, 79.6 with none there; eight
// frames 1714 and 1739.
constexpr uint32_t kBwdFmaPairs = 0xA4u;
struct Ctl {                      // after the barriers, at ctl + 320
  Split split;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Ctl) <= 192, "control block");
template <int D>
constexpr uint32_t bwd_smem() {
  return 7 * TileOf<D>::kBytes + 2 * 1024 + kBCtl;
}
static_assert(bwd_smem<128>() <= 232448, "shared memory per CTA");

template <bool kHalf>
__device__ __forceinline__ void store32(uint16_t* dst, const float (&x)[32]) {
#pragma unroll
  for (int c = 0; c < 32; c += 8)
    *reinterpret_cast<uint4*>(dst + c) =
        make_uint4(pack2<kHalf>(x[c], x[c + 1]), pack2<kHalf>(x[c + 2], x[c + 3]), pack2<kHalf>(x[c + 4], x[c + 5]),
                   pack2<kHalf>(x[c + 6], x[c + 7]));
}

// fp16's powers of two (GradRange).
constexpr int kPShift = 14;   // P <= 1 becomes at most 2^14: a factor of 4 below the type's end
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int range_field(const unsigned long long* w) { return static_cast<int>(__ldcg(w) & 0x1ff); }
// The e of 2^e dS <= 2^14 from the exponent fields of |do|^2 < 2^(x + 1) and |v|^2 < 2^(y + 1): |do| |v| is
// below 2^ceil((x + y + 2) / 2), |dP - delta| below twice that. x and y of finite fp16 rows are in
// [-48, 39] (or the field is that of 0).
__device__ __forceinline__ int ds_exponent(int g_field, int v_field) {
  const int x = min(max(g_field - 127, -48), 40), y = min(max(v_field - 127, -48), 40);
  return 13 - ((x + y + 3) >> 1);
}
// That of a key tile (one warp): over the query tiles that see it.
__device__ __forceinline__ int dk_exponent(const AttnArgs& a, int b, int h, int tile, int ql) {
  const size_t bh = static_cast<size_t>(b) * a.Hkv + h;
  const unsigned long long* g = a.range.g + bh * RowTiles<kRows>::count(a.mask);
  int x = 0;
  for (int i = KeyTiles::first_tile(a.mask, tile) + (threadIdx.x & 31); i * kRows < ql; i += 32)
    x = max(x, range_field(g + i));
  return ds_exponent(__reduce_max_sync(0xffffffffu, x), range_field(a.range.v + bh));
}

// Write kCols accumulator columns of this thread's row: to the output, times scale (fp16: and unscale,
// for which the product of both might leave fp32's range), when the segment is the whole tile, otherwise
// to this group's place in a record, [kCols / 4][128] float4.
template <int kCols, bool kHalf>
__device__ __forceinline__ void write_rows(const Seg& sg, uint32_t acc, int r, bool inside, bool zero, uint16_t* dst,
                                           float scale, float unscale, float* rec, uint32_t empty_bar) {
#pragma unroll 1
  for (int k = 0; k < kCols; k += 32) {
    uint32_t x[32];
    tmem_ld32_wait(acc + k, x);
    if (sg.whole) {
      float y[32];
#pragma unroll
      for (int e = 0; e < 32; ++e)
        y[e] = zero ? 0.f : (kHalf ? __uint_as_float(x[e]) * unscale : __uint_as_float(x[e])) * scale;
      if (inside) store32<kHalf>(dst + k, y);
    } else {
      float4* ro = reinterpret_cast<float4*>(rec);
#pragma unroll
      for (int e = 0; e < 32; e += 4)
        ro[(k + e) / 4 * kRows + r] = make_float4(__uint_as_float(x[e]), __uint_as_float(x[e + 1]),
                                                 __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
    }
  }
  tc_fence_before();
  warp_arrive(empty_bar);
}
// Sum of the records' 32 columns from quad q0 on, row r, over the CTAs c0..c1 in order.
template <typename Rec>
__device__ __forceinline__ void add_records(Rec&& record, int c0, int c1, int q0, int r, float (&y)[32]) {
#pragma unroll
  for (int e = 0; e < 32; ++e) y[e] = 0.f;
#pragma unroll 4
  for (int j = c0; j <= c1; ++j) {
    const float4* x = reinterpret_cast<const float4*>(record(j)) + q0 * kRows + r;
    float4 v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __ldcg(x + e * kRows);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[4 * e] += v[e].x;
      y[4 * e + 1] += v[e].y;
      y[4 * e + 2] += v[e].z;
      y[4 * e + 3] += v[e].w;
    }
  }
}

// ------------------------------------------------------------------ prep
__device__ __forceinline__ float row_sum(float s, int lanes, unsigned mask) {
  for (int m = lanes / 2; m > 0; m >>= 1) s += __shfl_xor_sync(mask, s, m);
  return s;
}
// fp16: the sum of the squares of 8 values, and by all 256 threads: a word of GradRange raised to the
// largest exponent field among them. With 18720 rows each of do and v the launch takes 10.8 us, 6.5 without
// the ranges; with an atomic per row instead of one per block it took 24.
__device__ __forceinline__ float sum_squares(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float n = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    n = fmaf(x.x, x.x, n);
    n = fmaf(x.y, x.y, n);
  }
  return n;
}
struct RangeWord {
  unsigned long long* word;
  unsigned long long call, now;
  __device__ void start(unsigned long long* w, const unsigned long long* c) {
    word = w;
    if (threadIdx.x == 0) call = __ldcg(c), now = __ldcg(w);
  }
  __device__ void raise(int field) const {
    __shared__ int top[8];
    field = __reduce_max_sync(0xffffffffu, field);
    if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = field;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int i = 1; i < 8; ++i) field = max(field, top[i]);
    const unsigned long long w = (call << 9) + field;
    if (now < w) atomicMax(word, w);
  }
};
constexpr int kPrepVRows = 4;

template <bool kHalf>
__global__ void __launch_bounds__(256) arl2_attn_prep_kernel(const __grid_constant__ AttnPrepArgs a, int v_blocks) {
  griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x < 2) a.tickets[threadIdx.x] = 0;
  const int lanes = a.d / 8;                        // lanes per row, 16 bytes each
  const int Tpad = (a.Tq + kRows - 1) / kRows * kRows;
  const int part = threadIdx.x % lanes, lane = threadIdx.x & 31;
  const unsigned mask = ((1u << lanes) - 1) << (lane / lanes * lanes);   // the row's lanes
  int b, t, h;
  RangeWord word{};
  if constexpr (kHalf) {
    const int block = static_cast<int>(blockIdx.x);
    if (block < v_blocks) {   // v: kPrepVRows rows of a thread's place each, of one head
      const int step = 256 / lanes, chunks = (a.Tk + kPrepVRows * step - 1) / (kPrepVRows * step);
      h = block / chunks % a.Hkv;
      b = block / chunks / a.Hkv;
      t = block % chunks * kPrepVRows * step + threadIdx.x / lanes;
      word.start(a.range.v + static_cast<size_t>(b) * a.Hkv + h, a.range.call);
      const int kl = a.k_len ? min(max(a.k_len[b], 0), a.Tk) : a.Tk;
      const uint16_t* src = a.v + b * a.v_sb + h * a.v_sh + part * 8;
      float n = 0.f;
#pragma unroll
      for (int i = 0; i < kPrepVRows; ++i) {
        const int ti = t + i * step;
        const float ni = ti < kl ? sum_squares(*reinterpret_cast<const uint4*>(src + ti * a.v_st)) : 0.f;
        n = fmax_nan(n, row_sum(ni, lanes, mask));
      }
      word.raise((__float_as_int(n) >> 23) & 0xff);
      return;
    }
    // The others: a block's 256 / lanes rows (which divide 128) share a tile of 128 rows and a head.
    const int in_tile = lanes / 2, bth = (block - v_blocks) / in_tile, bt = bth / a.H;
    h = bth % a.H;
    b = bt / (Tpad / kRows);
    t = bt % (Tpad / kRows) * kRows + (block - v_blocks) % in_tile * (256 / lanes) + threadIdx.x / lanes;
    word.start(a.range.g + (static_cast<size_t>(b) * a.Hkv + h / (a.H / a.Hkv)) * (Tpad / kRows) + t / kRows,
               a.range.call);
  } else {
    const long long row = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / lanes, bt = row / a.H;
    if (row >= static_cast<long long>(a.B) * Tpad * a.H) return;   // whole rows leave together
    h = static_cast<int>(row % a.H);   // fastest
    t = static_cast<int>(bt % Tpad), b = static_cast<int>(bt / Tpad);
  }
  const int ql = a.q_len ? min(max(a.q_len[b], 0), a.Tq) : a.Tq;
  float s = 0.f, l = -INFINITY;   // both negated: the consumers add them
  [[maybe_unused]] float n = 0.f;
  if (t < ql) {
    const uint4 ov = *reinterpret_cast<const uint4*>(a.o + b * a.o_sb + t * a.o_st + h * a.o_sh + part * 8);
    const uint4 gv = *reinterpret_cast<const uint4*>(a.g + b * a.g_sb + t * a.g_st + h * a.g_sh + part * 8);
    const uint32_t ow[4] = {ov.x, ov.y, ov.z, ov.w}, gw[4] = {gv.x, gv.y, gv.z, gv.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 x, y;
      if constexpr (kHalf) {
        x = __half22float2(*reinterpret_cast<const __half2*>(&ow[i]));
        y = __half22float2(*reinterpret_cast<const __half2*>(&gw[i]));
      } else {
        x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&ow[i]));
        y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&gw[i]));
      }
      s = fmaf(x.x, y.x, s);
      s = fmaf(x.y, y.y, s);
    }
    const float lse = a.lse[(static_cast<size_t>(b) * a.H + h) * a.Tq + t];
    l = lse == -INFINITY ? -INFINITY : fmaf(lse, -1.4426950408889634f, kHalf ? kPShift : 0);
    if constexpr (kHalf) n = sum_squares(gv);
  }
  s = row_sum(s, lanes, mask);
  const int field = kHalf ? (__float_as_int(row_sum(n, lanes, mask)) >> 23) & 0xff : 0;
  if (part == 0) {
    float* out = a.stats + (static_cast<size_t>(b) * a.H + h) * attn_stat_rows(kHalf) * Tpad + t;
    out[0] = l;
    out[Tpad] = -s;
    if constexpr (kHalf) out[2 * Tpad] = static_cast<float>(field);
  }
  if constexpr (kHalf) word.raise(field);
}

// ------------------------------------------------------------------ dk, dv
enum : int {
  kKKVFull = 0,
  kKKVEmpty,
  kKQFull,                // + stage (3)
  kKQEmpty = kKQFull + 3,
  kKGFull = kKQEmpty + 3,   // + stage (2): do
  kKGEmpty = kKGFull + 2,
  kKTFull = kKGEmpty + 2,   // + stage (2): statistics
  kKTEmpty = kKTFull + 2,   // 8 warps
  kKSFull = kKTEmpty + 2,
  kKPReady,               // 8 warps
  kKDFull,
  kKDReady,               // 8 warps
  kKAccFull,
  kKAccEmpty,             // 8 warps
  kKSide,
  kKFinal,                // the MMA warp's commit and 8 warps
  kKBars
};
static_assert(kKBars * 8 <= 320, "control block");

template <int D, bool kHalf>
__device__ __forceinline__ void dkv_cta(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                        const CUtensorMap& tm_g, const AttnArgs& a, uint8_t* attn_smem, int cta,
                                        int nctas) {
  using TO = TileOf<D>;
  const uint32_t base = smem_u32(attn_smem);
  const uint32_t k_tile = base, v_tile = base + TO::kBytes, q_ring = base + 2 * TO::kBytes,
                 g_ring = base + 5 * TO::kBytes, t_ring = base + 7 * TO::kBytes, ctl = t_ring + 2048;
  uint8_t* gctl = attn_smem + 7 * TO::kBytes + 2048;
  auto bar = [&](int i) { return ctl + 8u * i; };
  Ctl* shared = reinterpret_cast<Ctl*>(gctl + 320);
  const int warp = threadIdx.x >> 5;
  const Guard g{&shared->abort, a.err, a.timeout_ns};
  const int group = a.H / a.Hkv;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kKBars; ++i) {
      const bool by8 = i == kKTEmpty || i == kKTEmpty + 1 || i == kKPReady || i == kKDReady || i == kKAccEmpty;
      mbar_init(bar(i), by8 ? 8 : i == kKFinal ? 9 : 1);
    }
    shared->abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    if (elect_one()) {
      prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
      prefetch_tmap(&tm_g);
    }
    __syncwarp();
    get_split<KeyTiles>(a.mask, a.B, a.Hkv, group, cta, nctas, static_cast<const Split*>(a.splits), &shared->split);
  }
  if (warp == 1) tmem_alloc(smem_u32(&shared->tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = shared->tmem;
  const uint32_t c_s = tmem, c_dp = tmem + 128, c_dv = tmem + 256, c_dk = tmem + 384;

  // Registers move from the copy and MMA warps to the others: 128 threads x 88 + 256 x 200 = 62464
  // of the block's 384 x 168.
  if (warp == 0) {
    regs_dec<88>();
    const Split& sp = shared->split;
    Walk<KeyTiles> walk(a.mask, sp, a.Hkv, group);
    Seg sg;
    const bool lead = elect_one();
    const int Tpad = (a.mask.Tq + kRows - 1) / kRows * kRows;
    uint32_t ns = 0, nq = 0, ng = 0, nt = 0, side_phase = 0;   // copies made
    bool ok = true;
    while (ok && walk.next(sg)) {
      if (sg.units == 0) continue;
      if (ns > 0 && !mbar_wait_warp(bar(kKKVEmpty), (ns - 1) & 1, g)) break;
      if (lead) {
        mbar_expect_tx(bar(kKKVFull), 2 * TO::kBytes);
        load_tile<D>(k_tile, &tm_k, bar(kKKVFull), sg.h, sg.tile * kRows, sg.b);
        load_tile<D>(v_tile, &tm_v, bar(kKKVFull), sg.h, sg.tile * kRows, sg.b);
      }
      ++ns;
      const int per_head = sg.units / group, first = KeyTiles::first_tile(a.mask, sg.tile);
      int hd = sg.h * group + sg.kb / per_head, i = first + sg.kb % per_head;
      for (int u = sg.kb; u < sg.ke; ++u) {
        const int r0 = sg.ql < a.mask.Tq ? sg.ql - i * kRows : kRows;   // rows behind the length read as zero
        ok = nq < 3 || mbar_wait_warp(bar(kKQEmpty + nq % 3), (nq / 3 - 1) & 1, g);
        if (!ok) break;
        ok = load_clean<D>(q_ring + nq % 3 * TO::kBytes, &tm_q, bar(kKQFull + nq % 3), bar(kKSide), side_phase, hd,
                           i * kRows, sg.b, r0, lead, g);
        ++nq;
        if (!ok) break;
        ok = nt < 2 || mbar_wait_warp(bar(kKTEmpty + nt % 2), (nt / 2 - 1) & 1, g);
        if (!ok) break;
        if (lead) {
          const float* st =
              a.stats + (static_cast<size_t>(sg.b) * a.H + hd) * attn_stat_rows(kHalf) * Tpad + i * kRows;
          mbar_expect_tx(bar(kKTFull + nt % 2), 1024);
          bulk_load(t_ring + nt % 2 * 1024, st, 512, bar(kKTFull + nt % 2));
          bulk_load(t_ring + nt % 2 * 1024 + 512, st + Tpad, 512, bar(kKTFull + nt % 2));
        }
        ++nt;
        ok = ng < 2 || mbar_wait_warp(bar(kKGEmpty + ng % 2), (ng / 2 - 1) & 1, g);
        if (!ok) break;
        ok = load_clean<D>(g_ring + ng % 2 * TO::kBytes, &tm_g, bar(kKGFull + ng % 2), bar(kKSide), side_phase, hd,
                           i * kRows, sg.b, r0, lead, g);
        ++ng;
        if (!ok) break;
        if (++i == first + per_head) {
          i = first;
          ++hd;
        }
      }
    }
    __syncwarp();
    // Every copy issued lands before the CTA may exit.
    if (ns > 0) mbar_wait_drain(bar(kKKVFull), (ns - 1) & 1);
    for (uint32_t s = 0; s < 3; ++s)
      if (nq > s) mbar_wait_drain(bar(kKQFull + s), ((nq - s + 2) / 3 - 1) & 1);
    for (uint32_t s = 0; s < 2; ++s) {
      if (ng > s) mbar_wait_drain(bar(kKGFull + s), ((ng - s + 1) / 2 - 1) & 1);
      if (nt > s) mbar_wait_drain(bar(kKTFull + s), ((nt - s + 1) / 2 - 1) & 1);
    }
  } else if (warp == 1) {
    regs_dec<88>();
    const Split& sp = shared->split;
    Walk<KeyTiles> walk(a.mask, sp, a.Hkv, group);
    Seg sg;
    const bool lead = elect_one();
    constexpr uint32_t id_s = attn_idesc<kHalf>(128, false, false), id_d = attn_idesc<kHalf>(D, false, true);
    uint32_t ns = 0, n = 0;   // segments and units begun
    bool ok = true;
    auto q_full = [&](uint32_t i) { return mbar_wait_warp(bar(kKQFull + i % 3), (i / 3) & 1, g); };
    auto g_full = [&](uint32_t i) { return mbar_wait_warp(bar(kKGFull + i % 2), (i / 2) & 1, g); };
    auto q_at = [&](uint32_t i) { return q_ring + i % 3 * TO::kBytes; };
    auto g_at = [&](uint32_t i) { return g_ring + i % 2 * TO::kBytes; };
    while (ok && walk.next(sg)) {
      if (sg.units == 0) continue;
      ok = mbar_wait_warp(bar(kKKVFull), ns & 1, g) && q_full(n);
      if (!ok) break;
      tc_fence_after();
      if (lead) {
        mma_over_d<D>(c_s, k_tile, q_at(n), id_s);
        mma_commit(bar(kKSFull));
      }
      __syncwarp();
      ok = g_full(n);
      if (!ok) break;
      tc_fence_after();
      if (lead) {
        mma_over_d<D>(c_dp, v_tile, g_at(n), id_s);
        mma_commit(bar(kKDFull));
      }
      __syncwarp();
      for (int u = sg.kb; u < sg.ke; ++u, ++n) {
        const bool more = u + 1 < sg.ke;
        const uint32_t acc = u > sg.kb;
        // Everything but P first: what is left after P's arrival is on the critical path.
        if (!acc && ns > 0) ok = mbar_wait_warp(bar(kKAccEmpty), (ns - 1) & 1, g);
        ok = ok && (!more || q_full(n + 1)) && mbar_wait_warp(bar(kKPReady), n & 1, g);
        if (!ok) break;
        tc_fence_after();
        if (lead) {
          mma_over_rows(c_dv, c_s, g_at(n), id_d, acc);
          if (more) {
            mma_over_d<D>(c_s, k_tile, q_at(n + 1), id_s);
            mma_commit(bar(kKSFull));
          }
          mma_commit(bar(kKGEmpty + n % 2));
        }
        __syncwarp();
        ok = (!more || g_full(n + 1)) && mbar_wait_warp(bar(kKDReady), n & 1, g);
        if (!ok) break;
        tc_fence_after();
        if (lead) {
          mma_over_rows(c_dk, c_dp, q_at(n), id_d, acc);
          if (more) {
            mma_over_d<D>(c_dp, v_tile, g_at(n + 1), id_s);
            mma_commit(bar(kKDFull));
          }
          mma_commit(bar(kKQEmpty + n % 3));
        }
        __syncwarp();
      }
      if (!ok) break;
      if (lead) {
        mma_commit(bar(kKAccFull));
        mma_commit(bar(kKKVEmpty));
      }
      __syncwarp();
      ++ns;
    }
    __syncwarp();
    if (lead) mma_commit(bar(kKFinal));
    __syncwarp();
  } else if (warp < 4) {
    regs_dec<88>();
  } else {
    regs_inc<200>();
    const Split& sp = shared->split;
    Walk<KeyTiles> walk(a.mask, sp, a.Hkv, group);
    Seg sg;
    const int wg = (warp >> 2) - 1;                            // columns 64 wg ..; dv (0) or dk (1) at the end
    const int r = (warp & 3) * 32 + (threadIdx.x & 31);        // key row == TMEM lane
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) * 32 << 16;
    const uint32_t s_col = c_s + lanes + 64u * wg, dp_col = c_dp + lanes + 64u * wg;
    const float2 sc = make_float2(a.scale * 1.4426950408889634f, a.scale * 1.4426950408889634f);
    uint32_t n = 0, ns = 0;
    bool ok = true;
    while (ok && walk.next(sg)) {
      const int j = sg.tile * kRows + r;
      const AttnOut& out = wg ? a.dk : a.dv;
      uint16_t* dst = out.ptr + sg.b * out.sb + j * out.st + sg.h * out.sh;
      const bool inside = j < a.mask.Tk;
      if (sg.units == 0) {
        float z[32] = {};
        for (int k = 0; k < D; k += 32)
          if (inside) store32<kHalf>(dst + k, z);
        continue;
      }
      const int per_head = sg.units / group, first = KeyTiles::first_tile(a.mask, sg.tile);
      const int row0 = first_row(a.mask, j);   // the first query row that sees this key
      const int e = kHalf ? dk_exponent(a, sg.b, sg.h, sg.tile, sg.ql) : 0;
      [[maybe_unused]] const float2 to_ds = make_float2(pow2(e - kPShift), pow2(e - kPShift));
      int i = first + sg.kb % per_head;
      for (int u = sg.kb; u < sg.ke; ++u, ++n) {
        ok = mbar_wait_warp(bar(kKTFull + n % 2), (n / 2) & 1, g);
        if (!ok) break;
        // The statistics come to registers while the scores are not there yet: shared memory is busy
        // with the MMAs' operands, and a load behind them is slow.
        const float4* st = reinterpret_cast<const float4*>(attn_smem + 7 * TO::kBytes + n % 2 * 1024) + 16 * wg;
        float4 lse[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) lse[k] = st[k];
        ok = mbar_wait_warp(bar(kKSFull), n & 1, g);
        if (!ok) break;
        tc_fence_after();
        // Of this thread's columns, those below `hidden` do not see the key. Those from `rows` on are behind
        // the length: q reads as 0 there, and 0 times an infinite key is no score.
        const int hidden = row0 - (i * kRows + 64 * wg), rows = sg.ql - (i * kRows + 64 * wg);
        float2 p[32];
        {
          uint32_t s[2][32];
          tmem_ld32x2_wait(s_col, s[0], s_col + 32, s[1]);
#pragma unroll
          for (int k = 0; k < 64; k += 4) {
            const float4 l = lse[k / 4];
            const uint32_t* x = &s[k >> 5][k & 31];
            const float2 x0 = make_float2(__uint_as_float(x[0]), __uint_as_float(x[1]));
            const float2 x1 = make_float2(__uint_as_float(x[2]), __uint_as_float(x[3]));
            p[k / 2] = exp2_pair(__ffma2_rn(x0, sc, make_float2(l.x, l.y)), fma_pair(kBwdFmaPairs, k / 2));
            p[k / 2 + 1] = exp2_pair(__ffma2_rn(x1, sc, make_float2(l.z, l.w)), fma_pair(kBwdFmaPairs, k / 2 + 1));
          }
        }
        if (__any_sync(0xffffffffu, hidden > 0 || rows < 64)) {
#pragma unroll
          for (int k = 0; k < 64; k += 2) {
            if (k < hidden || k >= rows) p[k / 2].x = 0.f;
            if (k + 1 < hidden || k + 1 >= rows) p[k / 2].y = 0.f;
          }
        }
        {
          uint32_t w[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) w[k] = pack2<kHalf>(p[k].x, p[k].y);
          tmem_st32(s_col, w);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(bar(kKPReady));
        if constexpr (kHalf) {   // from 2^14 P to 2^e P, while dP is under way
#pragma unroll
          for (int k = 0; k < 32; ++k) p[k] = __fmul2_rn(p[k], to_ds);
        }
        ok = mbar_wait_warp(bar(kKDFull), n & 1, g);
        if (!ok) break;
        tc_fence_after();
        {
          uint32_t d[2][32], w[32];
          tmem_ld32x2_wait(dp_col, d[0], dp_col + 32, d[1]);
#pragma unroll
          for (int k = 0; k < 64; k += 4) {
            const float4 dl = st[32 + k / 4];
            const uint32_t* x = &d[k >> 5][k & 31];
            const float2 d0 = __fmul2_rn(
                p[k / 2], __fadd2_rn(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), make_float2(dl.x, dl.y)));
            const float2 d1 = __fmul2_rn(
                p[k / 2 + 1],
                __fadd2_rn(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])), make_float2(dl.z, dl.w)));
            w[k / 2] = pack2<kHalf>(d0.x, d0.y);
            w[k / 2 + 1] = pack2<kHalf>(d1.x, d1.y);
          }
          tmem_st32(dp_col, w);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(bar(kKDReady));
        warp_arrive(bar(kKTEmpty + n % 2));
        if (++i == first + per_head) i = first;
      }
      if (ok) ok = mbar_wait_warp(bar(kKAccFull), ns & 1, g);
      if (!ok) break;
      ++ns;
      tc_fence_after();
      float* rec = a.records + record_slot(sp, cta, sg.first) * attn_record_floats(D) + wg * D * kRows;
      write_rows<D, kHalf>(sg, (wg ? c_dk : c_dv) + lanes, r, inside, j >= sg.kl, dst, wg ? a.scale : 1.f,
                           pow2(wg ? -e : -kPShift), rec, bar(kKAccEmpty));
    }
    __syncwarp();
    tc_fence_before();
    warp_arrive(bar(kKFinal));
  }
  __syncwarp();
  if (warp == 1) {
    // Every MMA is done and every other warp finished with TMEM.
    mbar_wait_drain(bar(kKFinal), 0);
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ dq
enum : int {
  kQQFull = 0,            // q and do of a segment
  kQQEmpty,
  kQKFull,                // + stage (3)
  kQKEmpty = kQKFull + 3,
  kQVFull = kQKEmpty + 3,   // + stage (2)
  kQVEmpty = kQVFull + 2,
  kQSFull = kQVEmpty + 2,   // + buffer (2)
  kQDFull = kQSFull + 2,
  kQDReady,               // 8 warps
  kQAccFull,
  kQAccEmpty,             // 8 warps
  kQSide,
  kQFinal,                // the MMA warp's commit and 8 warps
  kQBars
};
static_assert(kQBars * 8 <= 320, "control block");
using QTiles = RowTiles<kRows>;

template <int D, bool kHalf>
__device__ __forceinline__ void dq_cta(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                       const CUtensorMap& tm_g, const AttnArgs& a, uint8_t* attn_smem, int cta,
                                       int nctas) {
  using TO = TileOf<D>;
  const uint32_t base = smem_u32(attn_smem);
  const uint32_t q_tile = base, g_tile = base + TO::kBytes, k_ring = base + 2 * TO::kBytes,
                 v_ring = base + 5 * TO::kBytes, ctl = base + 7 * TO::kBytes;
  uint8_t* gctl = attn_smem + 7 * TO::kBytes;
  auto bar = [&](int i) { return ctl + 8u * i; };
  Ctl* shared = reinterpret_cast<Ctl*>(gctl + 320);
  const int warp = threadIdx.x >> 5;
  const Guard g{&shared->abort, a.err, a.timeout_ns};
  const int group = a.H / a.Hkv;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kQBars; ++i)
      mbar_init(bar(i), i == kQDReady || i == kQAccEmpty ? 8 : i == kQFinal ? 9 : 1);
    shared->abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    if (elect_one()) {
      prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
      prefetch_tmap(&tm_g);
    }
    __syncwarp();
    // The dq kernel's splits stand behind those of the gridDim.x - nctas others.
    const Split* made = static_cast<const Split*>(a.splits);
    get_split<QTiles>(a.mask, a.B, a.H, 1, cta, nctas, made ? made + (gridDim.x - nctas) : nullptr, &shared->split);
  }
  if (warp == 1) tmem_alloc(smem_u32(&shared->tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = shared->tmem;
  const uint32_t c_dp = tmem + 256, c_dq = tmem + 384;   // S buffers at 0 and 128

  if (warp == 0) {
    const Split& sp = shared->split;
    Walk<QTiles> walk(a.mask, sp, a.H, 1);
    Seg sg;
    const bool lead = elect_one();
    uint32_t ns = 0, nk = 0, nv = 0, side_phase = 0;   // copies made
    bool ok = true;
    while (ok && walk.next(sg)) {
      if (sg.units == 0) continue;
      if (ns > 0 && !mbar_wait_warp(bar(kQQEmpty), (ns - 1) & 1, g)) break;
      if (lead) {
        mbar_expect_tx(bar(kQQFull), 2 * TO::kBytes);
        load_tile<D>(q_tile, &tm_q, bar(kQQFull), sg.h, sg.tile * kRows, sg.b);
        load_tile<D>(g_tile, &tm_g, bar(kQQFull), sg.h, sg.tile * kRows, sg.b);
      }
      ++ns;
      for (int t = sg.kb; t < sg.ke; ++t) {
        ok = nk < 3 || mbar_wait_warp(bar(kQKEmpty + nk % 3), (nk / 3 - 1) & 1, g);
        if (!ok) break;
        const int r0 = sg.kl < a.mask.Tk ? sg.kl - t * kRows : kRows;   // keys behind the length read as zero
        ok = load_clean<D>(k_ring + nk % 3 * TO::kBytes, &tm_k, bar(kQKFull + nk % 3), bar(kQSide), side_phase,
                           sg.h / group, t * kRows, sg.b, r0, lead, g);
        ++nk;
        if (!ok) break;
        ok = nv < 2 || mbar_wait_warp(bar(kQVEmpty + nv % 2), (nv / 2 - 1) & 1, g);
        if (!ok) break;
        if (lead) {
          mbar_expect_tx(bar(kQVFull + nv % 2), TO::kBytes);
          load_tile<D>(v_ring + nv % 2 * TO::kBytes, &tm_v, bar(kQVFull + nv % 2), sg.h / group, t * kRows, sg.b);
        }
        ++nv;
      }
    }
    __syncwarp();
    // Every copy issued lands before the CTA may exit.
    if (ns > 0) mbar_wait_drain(bar(kQQFull), (ns - 1) & 1);
    for (uint32_t s = 0; s < 3; ++s)
      if (nk > s) mbar_wait_drain(bar(kQKFull + s), ((nk - s + 2) / 3 - 1) & 1);
    for (uint32_t s = 0; s < 2; ++s)
      if (nv > s) mbar_wait_drain(bar(kQVFull + s), ((nv - s + 1) / 2 - 1) & 1);
  } else if (warp == 1) {
    const Split& sp = shared->split;
    Walk<QTiles> walk(a.mask, sp, a.H, 1);
    Seg sg;
    const bool lead = elect_one();
    constexpr uint32_t id_s = attn_idesc<kHalf>(128, false, false), id_d = attn_idesc<kHalf>(D, false, true);
    uint32_t ns = 0, n = 0;   // segments and units begun
    bool ok = true;
    auto k_full = [&](uint32_t i) { return mbar_wait_warp(bar(kQKFull + i % 3), (i / 3) & 1, g); };
    auto v_full = [&](uint32_t i) { return mbar_wait_warp(bar(kQVFull + i % 2), (i / 2) & 1, g); };
    auto k_at = [&](uint32_t i) { return k_ring + i % 3 * TO::kBytes; };
    auto scores = [&](uint32_t i) {   // unit i's S
      if (!k_full(i)) return false;
      tc_fence_after();
      if (lead) {
        mma_over_d<D>(tmem + 128u * (i & 1), q_tile, k_at(i), id_s);
        mma_commit(bar(kQSFull + (i & 1)));
      }
      __syncwarp();
      return true;
    };
    auto grads = [&](uint32_t i) {   // unit i's dP
      if (!v_full(i)) return false;
      tc_fence_after();
      if (lead) {
        mma_over_d<D>(c_dp, g_tile, v_ring + i % 2 * TO::kBytes, id_s);
        mma_commit(bar(kQDFull));
        mma_commit(bar(kQVEmpty + i % 2));
      }
      __syncwarp();
      return true;
    };
    while (ok && walk.next(sg)) {
      if (sg.units == 0) continue;
      const int cnt = sg.ke - sg.kb;
      ok = mbar_wait_warp(bar(kQQFull), ns & 1, g) && scores(n) && grads(n) && (cnt < 2 || scores(n + 1));
      if (!ok) break;
      for (int u = 0; u < cnt; ++u, ++n) {
        // Everything but dS first: what is left after its arrival is on the critical path.
        const bool more = u + 1 < cnt, more2 = u + 2 < cnt;
        if (u == 0 && ns > 0) ok = mbar_wait_warp(bar(kQAccEmpty), (ns - 1) & 1, g);
        ok = ok && (!more || v_full(n + 1)) && mbar_wait_warp(bar(kQDReady), n & 1, g);
        if (!ok) break;
        tc_fence_after();
        if (lead) {
          if (more) {   // first: the next softmax waits for it
            mma_over_d<D>(c_dp, g_tile, v_ring + (n + 1) % 2 * TO::kBytes, id_s);
            mma_commit(bar(kQDFull));
            mma_commit(bar(kQVEmpty + (n + 1) % 2));
          }
          mma_over_rows(c_dq, tmem + 128u * (n & 1), k_at(n), id_d, u > 0);
          mma_commit(bar(kQKEmpty + n % 3));
        }
        __syncwarp();
        ok = !more2 || scores(n + 2);
        if (!ok) break;
      }
      if (!ok) break;
      if (lead) {
        mma_commit(bar(kQAccFull));
        mma_commit(bar(kQQEmpty));
      }
      __syncwarp();
      ++ns;
    }
    __syncwarp();
    if (lead) mma_commit(bar(kQFinal));
    __syncwarp();
  } else if (warp >= 4) {
    const Split& sp = shared->split;
    Walk<QTiles> walk(a.mask, sp, a.H, 1);
    Seg sg;
    constexpr int kCols = D > 32 ? D / 2 : 32;                 // output columns of a group; d = 32: of the first
    const int wg = (warp >> 2) - 1;                            // score columns 64 wg ..
    const int r = (warp & 3) * 32 + (threadIdx.x & 31);        // query row == TMEM lane
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) * 32 << 16;
    const float2 sc = make_float2(a.scale * 1.4426950408889634f, a.scale * 1.4426950408889634f);
    const int Tpad = (a.mask.Tq + kRows - 1) / kRows * kRows;
    const bool writes = D > 32 || wg == 0;
    uint32_t n = 0, ns = 0;
    bool ok = true;
    while (ok && walk.next(sg)) {
      const int row = sg.tile * kRows + r;
      uint16_t* dst = a.o.ptr + sg.b * a.o.sb + row * a.o.st + sg.h * a.o.sh + kCols * wg;
      const bool inside = row < a.mask.Tq;
      if (sg.units == 0) {
        float z[32] = {};
        for (int k = 0; k < kCols; k += 32)
          if (inside && writes) store32<kHalf>(dst + k, z);
        continue;
      }
      const float* st = a.stats + (static_cast<size_t>(sg.b) * a.H + sg.h) * attn_stat_rows(kHalf) * Tpad + row;
      int e = 0;
      float bias = st[0];
      if constexpr (kHalf) {   // 2^e P straight away
        e = ds_exponent(static_cast<int>(st[2 * Tpad]),
                        range_field(a.range.v + static_cast<size_t>(sg.b) * a.Hkv + sg.h / group));
        bias += e - kPShift;
      }
      const float2 neg_lse = make_float2(bias, bias), neg_delta = make_float2(st[Tpad], st[Tpad]);
      // Rows behind the length are not written; they count as seeing all, so that they do not make
      // every tile a masked one.
      const int limit = row < sg.ql ? key_limit(a.mask, row, sg.kl) : sg.kl;
      for (int t = sg.kb; t < sg.ke; ++t, ++n) {
        ok = mbar_wait_warp(bar(kQSFull + (n & 1)), (n / 2) & 1, g);
        if (!ok) break;
        tc_fence_after();
        const uint32_t s_col = tmem + lanes + 128u * (n & 1) + 64u * wg, dp_col = c_dp + lanes + 64u * wg;
        const int seen = limit - (t * kRows + 64 * wg);   // this thread's columns that the row sees
        float2 p[32];
        {
          uint32_t s[2][32];
          tmem_ld32x2_wait(s_col, s[0], s_col + 32, s[1]);
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const uint32_t* x = &s[k >> 4][2 * (k & 15)];
            p[k] = exp2_pair(__ffma2_rn(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), sc, neg_lse),
                             fma_pair(kBwdFmaPairs, k));
          }
        }
        ok = mbar_wait_warp(bar(kQDFull), n & 1, g);
        if (!ok) break;
        tc_fence_after();
        uint32_t d[2][32], w[32];
        tmem_ld32x2_wait(dp_col, d[0], dp_col + 32, d[1]);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const uint32_t* x = &d[k >> 4][2 * (k & 15)];
          p[k] = __fmul2_rn(p[k], __fadd2_rn(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), neg_delta));
        }
        if (__any_sync(0xffffffffu, seen < 64)) {
#pragma unroll
          for (int k = 0; k < 64; k += 2) {
            if (k >= seen) p[k / 2].x = 0.f;
            if (k + 1 >= seen) p[k / 2].y = 0.f;
          }
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) w[k] = pack2<kHalf>(p[k].x, p[k].y);
        tmem_st32(s_col, w);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(bar(kQDReady));
      }
      if (ok) ok = mbar_wait_warp(bar(kQAccFull), ns & 1, g);
      if (!ok) break;
      ++ns;
      tc_fence_after();
      float* rec = a.dq_records + record_slot(sp, cta, sg.first) * attn_dq_record_floats(D) + wg * kCols * kRows;
      if (writes)
        write_rows<kCols, kHalf>(sg, c_dq + lanes + kCols * wg, r, inside, row >= sg.ql, dst, a.scale, pow2(-e), rec,
                                 bar(kQAccEmpty));
      else
        warp_arrive(bar(kQAccEmpty));
    }
    __syncwarp();
    tc_fence_before();
    warp_arrive(bar(kQFinal));
  }
  __syncwarp();
  if (warp == 1) {
    // Every MMA is done and every other warp finished with TMEM.
    mbar_wait_drain(bar(kQFinal), 0);
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ one launch of both
// n_dkv CTAs compute dk and dv, the others dq: one start-up, one end and half as many shared tiles
// as two launches that each use every SM. Where the two SMs of a pair (2 i, 2 i + 1) run different
// kinds, both run up to 1.4 times as long (measured; the cause is not known). So a CTA asks for its work by the SM it finds itself
// on, and gets the next range of that kind, or of the other one once it has run out. Which CTA
// computes a range changes nothing in the result.
template <int D, bool kHalf>
__global__ void __launch_bounds__(kBwdThreads, 1)
    arl2_attn_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_g,
                         const __grid_constant__ AttnArgs a, int n_dkv) {
  extern __shared__ __align__(1024) uint8_t attn_smem[];
  griddep_launch_dependents();   // the combining launch waits for this grid's end before it reads
  const int n_dq = static_cast<int>(gridDim.x) - n_dkv;
  int* ticket = reinterpret_cast<int*>(attn_smem);
  if (threadIdx.x == 0) {
    griddep_wait();   // for all threads: the launch before this one zeroed the tickets and made the statistics
    uint32_t sm;
    asm volatile("mov.u32 %0, %%smid;" : "=r"(sm));
    int kind = static_cast<int>(sm & ~1u) < n_dkv ? 0 : 1;
    int c = static_cast<int>(atomicAdd(a.tickets + kind, 1u));
    if (c >= (kind ? n_dq : n_dkv)) {
      kind ^= 1;
      c = static_cast<int>(atomicAdd(a.tickets + kind, 1u));
    }
    // The one CTA with dk's first range counts the call: the next prep, which is the next to read it,
    // starts after this grid.
    if (kHalf && kind == 0 && c == 0) ++*a.range.call;
    ticket[0] = kind;
    ticket[1] = c;
  }
  __syncthreads();
  const int kind = ticket[0], c = ticket[1];
  __syncthreads();   // read before the CTA lays out its shared memory
  if (kind == 0)
    dkv_cta<D, kHalf>(tm_q, tm_k, tm_v, tm_g, a, attn_smem, c, n_dkv);
  else
    dq_cta<D, kHalf>(tm_q, tm_k, tm_v, tm_g, a, attn_smem, c, n_dq);
}

// ------------------------------------------------------------------ records
// Adds up the records of the tiles shared between CTAs, as the forward's (arl2_attn_fwd.cu): block
// (c, y) takes 32 columns of the tile at the start of CTA c's range; y < D / 32: of dv, then of
// dk, then, in the dq kernel's split, of dq.
template <int D, bool kHalf>
__global__ void __launch_bounds__(kRows, 4)
    arl2_attn_bwd_combine_kernel(const __grid_constant__ AttnArgs a, int n_dkv, int n_dq) {
  __shared__ Split split;
  constexpr int kParts = D / 32;
  const int c = static_cast<int>(blockIdx.x) + 1, r = threadIdx.x, what = blockIdx.y / kParts;
  const int k0 = 32 * (blockIdx.y % kParts), group = a.H / a.Hkv;
  if (threadIdx.x < 32) {
    const Split* made = static_cast<const Split*>(a.splits);
    if (what < 2)
      get_split<KeyTiles>(a.mask, a.B, a.Hkv, group, c, n_dkv, made, &split);
    else
      get_split<QTiles>(a.mask, a.B, a.H, 1, c, n_dq, made ? made + n_dkv : nullptr, &split);
  }
  __syncthreads();
  const Split sp = split;
  griddep_wait();   // the records; every block, so that this grid ends after the one before it
  const long long first = sp.u0 - sp.off;
  if (sp.whole || c >= sp.ctas || sp.off == 0 || unit_owner(sp, first) != c - 1) return;
  const int ql = q_length(a.mask, sp.b), kl = k_length(a.mask, sp.b);
  const int units =
      what < 2 ? KeyTiles::units(a.mask, sp.tile, ql, kl, group) : QTiles::units(a.mask, sp.tile, ql, kl, 1);
  const int c1 = unit_owner(sp, first + max(1, units) - 1);
  const int row = sp.tile * kRows + r;
  float y[32];
  if (what < 2)
    add_records([&](int j) { return a.records + record_slot(sp, j, first) * attn_record_floats(D) + what * D * kRows; },
                c - 1, c1, k0 / 4, r, y);
  else
    add_records([&](int j) { return a.dq_records + record_slot(sp, j, first) * attn_dq_record_floats(D); }, c - 1, c1,
                k0 / 4, r, y);
  const bool zero = row >= (what < 2 ? kl : ql);
  const float scale = what == 0 ? 1.f : a.scale;
  if constexpr (kHalf) {
    int e = kPShift;   // as the kernel that wrote the records
    if (what == 1) {
      e = dk_exponent(a, sp.b, sp.h, sp.tile, ql);
    } else if (what == 2) {
      const int Tpad = RowTiles<kRows>::count(a.mask) * kRows;
      e = ds_exponent(
          static_cast<int>(a.stats[((static_cast<size_t>(sp.b) * a.H + sp.h) * attn_stat_rows(kHalf) + 2) * Tpad + row]),
          range_field(a.range.v + static_cast<size_t>(sp.b) * a.Hkv + sp.h / group));
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) y[k] *= pow2(-e);
  }
#pragma unroll
  for (int k = 0; k < 32; ++k) y[k] = zero ? 0.f : y[k] * scale;
  const AttnOut& out = what == 0 ? a.dv : what == 1 ? a.dk : a.o;
  if (row < (what < 2 ? a.mask.Tk : a.mask.Tq))
    store32<kHalf>(out.ptr + sp.b * out.sb + row * out.st + sp.h * out.sh + k0, y);
}

// Block c writes the split of CTA c of those that compute dk and dv, and behind them dq.
__global__ void __launch_bounds__(32) arl2_attn_bwd_split_kernel(const __grid_constant__ AttnArgs a, int n_dkv) {
  const int i = static_cast<int>(blockIdx.x);
  Split* out = static_cast<Split*>(a.splits) + i;
  if (i < n_dkv)
    make_split<KeyTiles, true>(a.mask, a.B, a.Hkv, a.H / a.Hkv, i, n_dkv, out);
  else
    make_split<QTiles, true>(a.mask, a.B, a.H, 1, i - n_dkv, static_cast<int>(gridDim.x) - n_dkv, out);
}

// Also loads the kernels, so that a first call inside a stream capture finds them there.
template <int D, bool kHalf>
cudaError_t setup() {
  cudaFuncAttributes attr;
  cudaError_t e = cudaFuncGetAttributes(&attr, arl2_attn_prep_kernel<kHalf>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, arl2_attn_bwd_combine_kernel<D, kHalf>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, arl2_attn_bwd_split_kernel);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(arl2_attn_bwd_kernel<D, kHalf>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(bwd_smem<D>()));
}
template <int D, bool kHalf>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& g,
                   const AttnPrepArgs& prep, const AttnArgs& a, int ctas, bool combine, cudaStream_t st) {
  const long long rows = static_cast<long long>(a.B) * ((a.mask.Tq + kRows - 1) / kRows * kRows) * a.H;
  const int v_rows = kPrepVRows * 256 / (D / 8);   // of a block
  const long long v_blocks = kHalf ? static_cast<long long>(a.B) * a.Hkv * ((a.mask.Tk + v_rows - 1) / v_rows) : 0;
  const unsigned blocks = static_cast<unsigned>((rows * (D / 8) + 255) / 256 + v_blocks);
  const int n_dkv = attn_dkv_ctas(ctas), n_dq = ctas - n_dkv;
  cudaError_t e = cudaSuccess;
  if (a.splits) e = launch_chained(arl2_attn_bwd_split_kernel, dim3(ctas), 32, 0, st, false, a, n_dkv);
  if (e == cudaSuccess) e = launch_chained(arl2_attn_prep_kernel<kHalf>, dim3(blocks), 256, 0, st, false, prep,
                                            static_cast<int>(v_blocks));
  if (e == cudaSuccess)
    e = launch_chained(arl2_attn_bwd_kernel<D, kHalf>, dim3(ctas), kBwdThreads, bwd_smem<D>(), st, true, q, k, v, g, a,
                       n_dkv);
  if (e != cudaSuccess || !combine) return e;
  return launch_chained(arl2_attn_bwd_combine_kernel<D, kHalf>, dim3(std::max(n_dkv, n_dq), 3 * (D / 32)), kRows, 0, st,
                        true, a, n_dkv, n_dq);
}

}  // namespace

cudaError_t attn_bwd_setup() {
  cudaError_t e = setup<32, false>();
  if (e == cudaSuccess) e = setup<64, false>();
  if (e == cudaSuccess) e = setup<128, false>();
  if (e == cudaSuccess) e = setup<32, true>();
  if (e == cudaSuccess) e = setup<64, true>();
  if (e == cudaSuccess) e = setup<128, true>();
  return e;
}

cudaError_t launch_attn_bwd(int d, bool half, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            const CUtensorMap& g, const AttnPrepArgs& prep, const AttnArgs& a, int ctas, bool combine,
                            cudaStream_t st) {
  if (half)
    return d == 32   ? launch<32, true>(q, k, v, g, prep, a, ctas, combine, st)
           : d == 64 ? launch<64, true>(q, k, v, g, prep, a, ctas, combine, st)
                     : launch<128, true>(q, k, v, g, prep, a, ctas, combine, st);
  return d == 32   ? launch<32, false>(q, k, v, g, prep, a, ctas, combine, st)
         : d == 64 ? launch<64, false>(q, k, v, g, prep, a, ctas, combine, st)
                   : launch<128, false>(q, k, v, g, prep, a, ctas, combine, st);
}

}  // namespace arl2
