// Softmax attention that keeps its row statistics, for training (arl2_attn_forward):
//     o = softmax(scale q k^T + mask) v,    lse_i = log sum_j exp(scale q_i.k_j)
// over the visible keys (arl2_attn.cuh). The 4 d flops per visible pair on the tensor cores
// bound it; the exponentials come next (16 a clock and SM on the MUFU unit: 1024 clocks for a
// 128 x 128 tile whose two products take 1024 clocks on the tensor pipe at d = 128). All of them go
// there: with 3 of 8 as polynomials on the FMA pipe, which the rest of the softmax loads, one 480p frame
// took 36.6 us (35.0 without) and eight frames 486 (478).
//
// A tile is two 128-row query tiles of one head (256 rows), which share every K and V tile
// that is loaded. While the softmax of one works on its scores, the tensor pipe does the
// products of the other. Online softmax: scores in log2 units, the running maximum m raised
// only when a key tile exceeds it by more than 8, so that the output accumulator is rescaled
// rarely; m, the sum l and the accumulator are fp32, only the probabilities (below 2^8) are
// rounded to 16 bits for the second product.
//
// A narrow tile, with rows in its first query tile only (few queries, a ragged end), would leave
// half of the softmax idle and the copies waiting for a chain of score, softmax and product: there
// the two groups take the key tiles by turns, and the first adds both accumulators up at the end.
//
// Roles (384 threads, one CTA per SM): warp 0 copies (Q per segment; K and V tiles through a
// ring of 5), warp 1 issues every MMA, warps 4-7 and 8-11 are the softmax of query tile 0 and 1,
// thread = row = TMEM lane. TMEM: S0, S1 (columns 0, 128; the packed P overwrites the first 64
// of its S), O0, O1 (256, 384). One issuing thread keeps the MMAs that touch the same columns
// in order; the rest is ordered by barriers:
//   - S full (commit) -> softmax; P ready (4 warps, by halves of the keys, so that the first half's
//     product runs while the second is made) -> P V MMA; the commit of S(t + 1) also says
//     that P V (t) is done, so the softmax may rescale O before it hands over P (t + 1);
//   - O full -> epilogue, O empty -> the next segment's first P V.
#include <algorithm>

#include "arl2_attn_kernels.h"

namespace arl2 {
namespace {

constexpr int kFwdRows = 256;
constexpr int kFwdThreads = 384;
constexpr int kRing = 5;
using FwdTiles = RowTiles<kFwdRows>;
enum : int {
  kFQFull = 0,
  kFQEmpty = 1,
  kFFull = 2,              // + stage
  kFEmpty = kFFull + kRing,
  kFSFull = kFEmpty + kRing,   // + query tile (2)
  kFPReady = kFSFull + 2,      // + 2 query tile + half (4)
  kFOFull = kFPReady + 4,
  kFOEmpty = kFOFull + 2,
  kFSide = kFOEmpty + 2,
  kFPairFull = kFSide + 1,   // narrow tiles: group 1's m and l are there (4 warps)
  kFPairEmpty,               // and were read (4 warps)
  kFFinal,
  kFBars = kFFinal + 1
};
constexpr uint32_t kFCtl = 512 + 1024;   // barriers, split, flags; m and l of narrow tiles [2][128]
static_assert(kFBars * 8 <= 256 && sizeof(Split) + 32 <= 256, "control block");
template <int D>
constexpr uint32_t fwd_smem() {
  return (2 + kRing) * TileOf<D>::kBytes + kFCtl;
}
static_assert(fwd_smem<128>() <= 232448, "shared memory per CTA");
constexpr float kRaise = 8.0f;    // log2 units

// Per record: [2 query tiles][d / 4 quads][128 rows] float4 of O, then [2][2][128] m and l.
template <int D>
__device__ __forceinline__ float* fwd_record(const AttnArgs& a, int slot) {
  return a.records + static_cast<size_t>(slot) * attn_record_floats(D);
}

template <int D, bool kHalf>
__device__ __forceinline__ void store_row(const AttnArgs& a, int b, int h, int row, const float (&x)[32], int c0) {
  uint16_t* dst = a.o.ptr + b * a.o.sb + row * a.o.st + h * a.o.sh + c0;
#pragma unroll
  for (int c = 0; c < 32; c += 8) {
    uint4 v = make_uint4(pack2<kHalf>(x[c], x[c + 1]), pack2<kHalf>(x[c + 2], x[c + 3]),
                         pack2<kHalf>(x[c + 4], x[c + 5]), pack2<kHalf>(x[c + 6], x[c + 7]));
    *reinterpret_cast<uint4*>(dst + c) = v;
  }
}

template <int D, bool kHalf>
__global__ void __launch_bounds__(kFwdThreads, 1)
    arl2_attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ AttnArgs a) {
  using TO = TileOf<D>;
  extern __shared__ __align__(1024) uint8_t attn_smem[];
  const uint32_t base = smem_u32(attn_smem);
  const uint32_t ctl = base + (2 + kRing) * TO::kBytes;
  uint8_t* gctl = attn_smem + (2 + kRing) * TO::kBytes;
  auto bar = [&](int i) { return ctl + 8u * i; };
  Split* split = reinterpret_cast<Split*>(gctl + 256);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gctl + 256 + sizeof(Split));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;
  const Guard g{abort_flag, a.err, a.timeout_ns};

  griddep_launch_dependents();   // the combining launch waits for this grid's end before it reads
  if (threadIdx.x == 0) {
    for (int i = 0; i < kFBars; ++i) {
      const bool by4 = (i >= kFPReady && i < kFPReady + 4) || (i >= kFOEmpty && i < kFOEmpty + 2) ||
                       i == kFPairFull || i == kFPairEmpty;
      mbar_init(bar(i), i == kFFinal ? 9 : by4 ? 4 : 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    if (elect_one()) {
      prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
    }
    __syncwarp();
    get_split<FwdTiles>(a.mask, a.B, a.H, 1, blockIdx.x, gridDim.x, static_cast<const Split*>(a.splits), split);
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Registers move from the copy and MMA warps to the softmax, which holds a row of 128 scores:
  // 128 threads x 72 + 256 x 216 = 64512, the block's 384 x 168.
  const int group = a.H / a.Hkv;
  const uint32_t q_tile = base, ring0 = base + 2 * TO::kBytes;

  if (warp == 0) {
    regs_dec<72>();
    const Split& sp = *split;
    Walk<FwdTiles> walk(a.mask, sp, a.H, 1);
    Seg sg;
    const bool lead = elect_one();
    uint32_t ns = 0, r = 0, side_phase = 0;
    bool ok = true;
    while (ok && walk.next(sg)) {
      if (sg.units == 0) continue;
      if (ns > 0 && !mbar_wait_warp(bar(kFQEmpty), (ns - 1) & 1, g)) break;
      const int tiles = sg.tile * kFwdRows + kRows < sg.ql ? 2 : 1;
      if (lead) {
        mbar_expect_tx(bar(kFQFull), tiles * TO::kBytes);
        for (int i = 0; i < tiles; ++i)
          load_tile<D>(q_tile + i * TO::kBytes, &tm_q, bar(kFQFull), sg.h, sg.tile * kFwdRows + i * kRows, sg.b);
      }
      ++ns;
      const int n = sg.ke - sg.kb;
      for (int k = 0; k < 2 * n; ++k, ++r) {
        // K and V by turns; in a narrow tile the keys run one tile ahead.
        const int kv = tiles == 2 ? k & 1 : k < 2 ? n == 1 && k == 1 : k == 2 * n - 1 || !(k & 1);
        const int t =
            sg.kb + (tiles == 2 ? k >> 1 : kv ? (k == 2 * n - 1 ? n - 1 : k / 2 - 1) : k < 2 ? k : (k + 1) / 2);
        const uint32_t st = r % kRing;
        ok = r < kRing || mbar_wait_warp(bar(kFEmpty + st), (r / kRing - 1) & 1, g);
        if (!ok) break;
        // Values behind the length must not reach P V; keys there are masked in the scores.
        const int r0 = kv && sg.kl < a.mask.Tk ? sg.kl - t * kRows : kRows;
        ok = load_clean<D>(ring0 + st * TO::kBytes, kv ? &tm_v : &tm_k, bar(kFFull + st), bar(kFSide), side_phase,
                           sg.h / group, t * kRows, sg.b, r0, lead, g);
        if (!ok) {
          ++r;
          break;
        }
      }
    }
    __syncwarp();
    // Every copy issued lands before the CTA may exit.
    if (ns > 0) mbar_wait_drain(bar(kFQFull), (ns - 1) & 1);
    for (uint32_t st = 0; st < kRing; ++st) {
      const uint32_t uses = r > st ? (r - st + kRing - 1) / kRing : 0;
      if (uses) mbar_wait_drain(bar(kFFull + st), (uses - 1) & 1);
    }
  } else if (warp == 1) {
    regs_dec<72>();
    const Split& sp = *split;
    Walk<FwdTiles> walk(a.mask, sp, a.H, 1);
    Seg sg;
    const bool lead = elect_one();
    constexpr uint32_t id_s = attn_idesc<kHalf>(128, false, false), id_o = attn_idesc<kHalf>(D, false, true);
    uint32_t ns = 0, r = 0, np[2] = {0, 0}, nseg[2] = {0, 0};
    bool ok = true;
    auto full = [&](uint32_t i) { return mbar_wait_warp(bar(kFFull + i % kRing), (i / kRing) & 1, g); };
    auto slot = [&](uint32_t i) { return ring0 + (i % kRing) * TO::kBytes; };
    while (ok && walk.next(sg)) {
      if (sg.units == 0) continue;
      const int tiles = sg.tile * kFwdRows + kRows < sg.ql ? 2 : 1;
      const int n = sg.ke - sg.kb;
      ok = mbar_wait_warp(bar(kFQFull), ns & 1, g) && full(r);
      if (!ok) break;
      tc_fence_after();
      if (tiles == 1) {
        // Narrow: the two groups take the key tiles by turns, each with an S and an O of its own.
        // Ring order K0 K1 V0 K2 V1 .. (as the copying warp's).
        auto at_k = [&](int t) { return r + (t < 2 ? t : 2 * t - 1); };
        auto at_v = [&](int t) { return r + (t < n - 1 ? 2 * t + 2 : 2 * n - 1); };
        auto scores = [&](int t) {
          const uint32_t p = at_k(t);
          if (!full(p)) return false;
          tc_fence_after();
          if (lead) {
            mma_over_d<D>(tmem + 128u * (t & 1), q_tile, slot(p), id_s);
            mma_commit(bar(kFSFull + (t & 1)));
            mma_commit(bar(kFEmpty + p % kRing));
          }
          __syncwarp();
          return true;
        };
        ok = scores(0) && (n < 2 || scores(1));
        for (int t = 0; ok && t < n; ++t) {
          const int i = t & 1;
          const uint32_t p = at_v(t);
          ok = full(p);
          if (ok && t < 2 && nseg[i] > 0) ok = mbar_wait_warp(bar(kFOEmpty + i), (nseg[i] - 1) & 1, g);
          ok = ok && mbar_wait_warp(bar(kFPReady + 2 * i), np[i] & 1, g);
          if (!ok) break;
          tc_fence_after();
          if (lead) mma_over_half_rows<0>(tmem + 256u + 128u * i, tmem + 128u * i, slot(p), id_o, t > 1);
          __syncwarp();
          ok = mbar_wait_warp(bar(kFPReady + 2 * i + 1), np[i] & 1, g);
          if (!ok) break;
          ++np[i];
          tc_fence_after();
          if (lead) {
            mma_over_half_rows<1>(tmem + 256u + 128u * i, tmem + 128u * i, slot(p), id_o, 1u);
            mma_commit(bar(kFEmpty + p % kRing));
          }
          __syncwarp();
          ok = t + 2 >= n || scores(t + 2);
        }
        r += 2 * n;
        if (!ok) break;
        if (lead) {
          mma_commit(bar(kFOFull));
          mma_commit(bar(kFQEmpty));
        }
        __syncwarp();
        ++ns;
        ++nseg[0];
        ++nseg[1];
        continue;
      }
      if (lead) {
        for (int i = 0; i < tiles; ++i) {
          mma_over_d<D>(tmem + 128u * i, q_tile + i * TO::kBytes, slot(r), id_s);
          mma_commit(bar(kFSFull + i));
        }
        mma_commit(bar(kFEmpty + r % kRing));
      }
      __syncwarp();
      for (int t = 0; ok && t < n; ++t, r += 2) {
        const bool more = t + 1 < n;
        // Everything but P first: what is left after P's arrival is on the critical path.
        ok = full(r + 1) && (!more || full(r + 2));
        for (int i = 0; ok && i < tiles; ++i) {
          if (t == 0 && nseg[i] > 0) ok = mbar_wait_warp(bar(kFOEmpty + i), (nseg[i] - 1) & 1, g);
          ok = ok && mbar_wait_warp(bar(kFPReady + 2 * i), np[i] & 1, g);
          if (!ok) break;
          tc_fence_after();
          if (lead)
            mma_over_half_rows<0>(tmem + 256u + 128u * i, tmem + 128u * i, slot(r + 1), id_o, t > 0);
          __syncwarp();
          ok = mbar_wait_warp(bar(kFPReady + 2 * i + 1), np[i] & 1, g);
          if (!ok) break;
          ++np[i];
          tc_fence_after();
          if (lead) {
            mma_over_half_rows<1>(tmem + 256u + 128u * i, tmem + 128u * i, slot(r + 1), id_o, 1u);
            if (more) {
              mma_over_d<D>(tmem + 128u * i, q_tile + i * TO::kBytes, slot(r + 2), id_s);
              mma_commit(bar(kFSFull + i));
            } else {
              mma_commit(bar(kFOFull + i));
            }
            if (i + 1 == tiles) {
              mma_commit(bar(kFEmpty + (r + 1) % kRing));
              if (more) mma_commit(bar(kFEmpty + (r + 2) % kRing));
            }
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      if (lead) mma_commit(bar(kFQEmpty));
      __syncwarp();
      ++ns;
      for (int i = 0; i < tiles; ++i) ++nseg[i];
    }
    __syncwarp();
    if (lead) mma_commit(bar(kFFinal));
    __syncwarp();
  } else if (warp < 4) {
    regs_dec<72>();
  } else {
    regs_inc<216>();
    const Split& sp = *split;
    Walk<FwdTiles> walk(a.mask, sp, a.H, 1);
    Seg sg;
    const int i = (warp >> 2) - 1;                              // query tile
    const int r = (warp & 3) * 32 + (threadIdx.x & 31);         // its row == TMEM lane
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) * 32 << 16;
    const uint32_t s_col = tmem + lanes + 128u * i, o_col = tmem + lanes + 256u + 128u * i;
    const float to_log2 = a.scale * 1.4426950408889634f;
    uint32_t nt = 0, nseg = 0, npair = 0;
    float* pair = reinterpret_cast<float*>(gctl + 512);
    const int c = static_cast<int>(blockIdx.x);
    bool ok = true;
    while (ok && walk.next(sg)) {
      const bool narrow = sg.units > 0 && sg.tile * kFwdRows + kRows >= sg.ql;   // one query tile
      float* lse = a.lse + (static_cast<size_t>(sg.b) * a.H + sg.h) * a.mask.Tq;
      int row = sg.tile * kFwdRows + i * kRows + r;
      if (sg.units == 0 || sg.tile * kFwdRows + i * kRows >= sg.ql) {
        // Nothing to see, or rows behind the length: zeros, once per tile.
        if (sg.kb == 0 && row < a.mask.Tq) {
          float z[32] = {};
#pragma unroll
          for (int k = 0; k < D; k += 32) store_row<D, kHalf>(a, sg.b, sg.h, row, z, k);
          lse[row] = -INFINITY;
        }
        if (!narrow) continue;
        row -= i * kRows;   // group 1 helps with the first query tile
      }
      const bool in_q = row < sg.ql;
      // Rows behind the length are not written; they count as seeing all, so that they do not make
      // every tile a masked one.
      const int limit = in_q ? key_limit(a.mask, row, sg.kl) : sg.kl;
      // A warp without a row inside the length leaves its P and O as they are: an MMA's rows do not
      // mix, and these are not written.
      const bool idle = row - (r & 31) >= sg.ql;
      float m = -INFINITY, l = 0.f;
      const int step = narrow ? 2 : 1, t0 = sg.kb + (narrow ? i : 0);
      for (int t = t0; t < sg.ke; t += step) {
        ok = mbar_wait_warp(bar(kFSFull + i), nt & 1, g);
        if (!ok) break;
        ++nt;
        tc_fence_after();
        if (idle) {
          warp_arrive(bar(kFPReady + 2 * i));
          warp_arrive(bar(kFPReady + 2 * i + 1));
          continue;
        }
        uint32_t s[4][32];
        tmem_ld32x2_wait(s_col, s[0], s_col + 32, s[1]);
        tmem_ld32x2_wait(s_col + 64, s[2], s_col + 96, s[3]);
        const int seen = limit - t * kRows;   // columns of this tile that the row sees
        const bool masked = __any_sync(0xffffffffu, seen < kRows);
        if (masked) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (32 * q + k >= seen) s[q][k] = 0xff800000u;   // -inf
        }
        float top[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          top[q] = __uint_as_float(s[q][0]);
#pragma unroll
          for (int k = 1; k < 31; k += 2)
            top[q] = fmax3_nan(top[q], __uint_as_float(s[q][k]), __uint_as_float(s[q][k + 1]));
        }
        top[0] = fmax3_nan(top[0], __uint_as_float(s[0][31]), __uint_as_float(s[1][31]));
        top[1] = fmax3_nan(top[1], __uint_as_float(s[2][31]), __uint_as_float(s[3][31]));
        const float tile_top = fmax3_nan(fmax3_nan(top[0], top[1], top[2]), top[3], top[3]) * to_log2;
        const bool raise = tile_top > m + kRaise || (m == -INFINITY && tile_top > m);
        if (__any_sync(0xffffffffu, raise)) {
          const float m_new = raise ? tile_top : m;
          const float f = raise && m != -INFINITY ? ex2_approx(m - m_new) : 1.f;
          l *= f;
          m = m_new;
          if (t > t0) {
#pragma unroll 1
            for (int k = 0; k < D; k += 32) {
              uint32_t x[32];
              tmem_ld32_wait(o_col + k, x);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
              tmem_st32(o_col + k, x);
            }
          }
        }
        const float shift = m == -INFINITY ? 0.f : m;
        const float2 sc = make_float2(to_log2, to_log2), sh = make_float2(-shift, -shift);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float2 e[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 x =
                __ffma2_rn(make_float2(__uint_as_float(s[q][2 * k]), __uint_as_float(s[q][2 * k + 1])), sc, sh);
            e[k] = make_float2(ex2_approx(x.x), ex2_approx(x.y));
          }
          uint32_t p[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            sum[k & 1] = __fadd2_rn(sum[k & 1], e[k]);
            p[k] = pack2<kHalf>(e[k].x, e[k].y);
          }
          tmem_st16(s_col + 16 * q, p);
          if (q & 1) {   // half of the keys: their product may start
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(bar(kFPReady + 2 * i + (q >> 1)));
          }
        }
        sum[0] = __fadd2_rn(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
        if (!(tile_top < INFINITY)) l = NAN;   // a NaN or +inf among the scores: the row has no softmax
      }
      if (!ok) break;
      if (narrow && i == 1) {   // m and l to group 0, which finishes the rows
        if (npair > 0) ok = mbar_wait_warp(bar(kFPairEmpty), (npair - 1) & 1, g);
        if (!ok) break;
        ++npair;
        pair[r] = m;
        pair[kRows + r] = l;
        warp_arrive(bar(kFPairFull));
        continue;
      }
      ok = mbar_wait_warp(bar(kFOFull + i), nseg & 1, g);
      if (!ok) break;
      ++nseg;
      // Narrow: O = keep O0 + add O1.
      float keep = 1.f, add = 0.f;
      if (narrow) {
        ok = mbar_wait_warp(bar(kFPairFull), npair & 1, g);
        if (!ok) break;
        ++npair;
        const float m1 = pair[r], l1 = pair[kRows + r], top = fmaxf(m, m1);
        warp_arrive(bar(kFPairEmpty));
        keep = m == -INFINITY ? 0.f : exp2f(m - top);
        add = m1 == -INFINITY ? 0.f : exp2f(m1 - top);
        l = l * keep + (l1 != l1 ? l1 : l1 * add);
        m = top;
      }
      const bool two = narrow && sg.ke - sg.kb > 1;
      tc_fence_after();
      auto load_o = [&](int k, uint32_t (&x)[32]) {
        if (!two) {
          tmem_ld32_wait(o_col + k, x);
        } else {
          uint32_t z[32];
          tmem_ld32x2_wait(o_col + k, x, o_col + 128 + k, z);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            x[e] = __float_as_uint(__uint_as_float(x[e]) * keep + (add == 0.f ? 0.f : __uint_as_float(z[e]) * add));
        }
      };
      auto release_o = [&] {
        tc_fence_before();
        warp_arrive(bar(kFOEmpty + i));
        if (narrow) warp_arrive(bar(kFOEmpty + 1));
      };
      if (sg.whole) {
        const float f = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
          uint32_t x[32];
          float y[32];
          load_o(k, x);
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = in_q && limit > 0 ? __uint_as_float(x[e]) * f : 0.f;
          if (row < a.mask.Tq) store_row<D, kHalf>(a, sg.b, sg.h, row, y, k);
        }
        release_o();
        if (row < a.mask.Tq) lse[row] = in_q && limit > 0 ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
        continue;
      }
      // A part of the tile: its record.
      float* rec = fwd_record<D>(a, record_slot(sp, c, sg.first));
      float4* ro = reinterpret_cast<float4*>(rec) + i * (D / 4) * kRows;
      float* rml = rec + 2 * kRows * D + i * 2 * kRows;
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        uint32_t x[32];
        load_o(k, x);
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          ro[(k + e) / 4 * kRows + r] = make_float4(__uint_as_float(x[e]), __uint_as_float(x[e + 1]),
                                                   __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
      }
      release_o();
      rml[r] = m;
      rml[kRows + r] = l;
    }
    __syncwarp();
    tc_fence_before();
    warp_arrive(bar(kFFinal));
  }
  __syncwarp();
  if (warp == 1) {
    // Every MMA is done and every softmax warp finished with TMEM.
    mbar_wait_drain(bar(kFFinal), 0);
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds up the records of the tiles shared between CTAs, in the order of the CTAs. Block (c, y)
// takes the tile at the start of CTA c's range, if it is the second to hold a part of it; y is
// one of its two query tiles and 32 of its columns. Thread = row.
template <int D, bool kHalf>
__global__ void __launch_bounds__(kRows, 4) arl2_attn_fwd_combine_kernel(const __grid_constant__ AttnArgs a) {
  __shared__ Split split;
  const int c = static_cast<int>(blockIdx.x) + 1, r = threadIdx.x;
  if (threadIdx.x < 32)
    get_split<FwdTiles>(a.mask, a.B, a.H, 1, c, gridDim.x + 1, static_cast<const Split*>(a.splits), &split);
  __syncthreads();
  const Split sp = split;
  griddep_wait();   // the records; every block, so that this grid ends after the one before it
  const long long first = sp.u0 - sp.off;
  if (sp.whole || c >= sp.ctas || sp.off == 0 || unit_owner(sp, first) != c - 1) return;
  const int i = blockIdx.y & 1, k0 = 32 * (blockIdx.y >> 1);
  const int ql = q_length(a.mask, sp.b), kl = k_length(a.mask, sp.b);
  const int row = sp.tile * kFwdRows + i * kRows + r;
  if (sp.tile * kFwdRows + i * kRows >= ql) return;   // written by the forward kernel
  const int units = max(1, FwdTiles::units(a.mask, sp.tile, ql, kl, 1));
  const int c1 = unit_owner(sp, first + units - 1);
  const bool sees = row < ql && key_limit(a.mask, row, kl) > 0;
  float m = -INFINITY, l = 0.f, y[32] = {};
#pragma unroll 2
  for (int j = c - 1; j <= c1; ++j) {
    const float* rec = fwd_record<D>(a, record_slot(sp, j, first));
    const float4* o = reinterpret_cast<const float4*>(rec) + (i * (D / 4) + k0 / 4) * kRows + r;
    const float* ml = rec + 2 * kRows * D + i * 2 * kRows + r;
    float4 x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __ldcg(o + e * kRows);
    const float mj = __ldcg(ml), lj = __ldcg(ml + kRows), top = fmaxf(m, mj);
    const float keep = m == -INFINITY ? 0.f : exp2f(m - top), w = mj == -INFINITY ? 0.f : exp2f(mj - top);
    m = top;
    l = l * keep + (lj != lj ? lj : lj * w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[4 * e] = fmaf(x[e].x, w, y[4 * e] * keep);
      y[4 * e + 1] = fmaf(x[e].y, w, y[4 * e + 1] * keep);
      y[4 * e + 2] = fmaf(x[e].z, w, y[4 * e + 2] * keep);
      y[4 * e + 3] = fmaf(x[e].w, w, y[4 * e + 3] * keep);
    }
  }
  if (row >= a.mask.Tq) return;
  const float f = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < 32; ++e) y[e] = sees ? y[e] * f : 0.f;
  store_row<D, kHalf>(a, sp.b, sp.h, row, y, k0);
  if (k0 == 0)
    a.lse[(static_cast<size_t>(sp.b) * a.H + sp.h) * a.mask.Tq + row] =
        sees ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// Block c writes the split of CTA c.
__global__ void __launch_bounds__(32) arl2_attn_fwd_split_kernel(const __grid_constant__ AttnArgs a) {
  make_split<FwdTiles, true>(a.mask, a.B, a.H, 1, blockIdx.x, gridDim.x, static_cast<Split*>(a.splits) + blockIdx.x);
}

// Also loads the kernels, so that a first call inside a stream capture finds them there.
template <int D, bool kHalf>
cudaError_t setup() {
  cudaFuncAttributes attr;
  cudaError_t e = cudaFuncGetAttributes(&attr, arl2_attn_fwd_combine_kernel<D, kHalf>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, arl2_attn_fwd_split_kernel);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(arl2_attn_fwd_kernel<D, kHalf>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(fwd_smem<D>()));
}
template <int D, bool kHalf>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const AttnArgs& a, int ctas,
                   bool combine, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (a.splits) e = launch_chained(arl2_attn_fwd_split_kernel, dim3(ctas), 32, 0, st, false, a);
  if (e == cudaSuccess)
    e = launch_chained(arl2_attn_fwd_kernel<D, kHalf>, dim3(ctas), kFwdThreads, fwd_smem<D>(), st, false, q, k, v, a);
  if (e != cudaSuccess || !combine || ctas < 2) return e;
  return launch_chained(arl2_attn_fwd_combine_kernel<D, kHalf>, dim3(ctas - 1, 2 * (D / 32)), kRows, 0, st, true, a);
}

}  // namespace

cudaError_t attn_fwd_setup() {
  cudaError_t e = setup<32, false>();
  if (e == cudaSuccess) e = setup<64, false>();
  if (e == cudaSuccess) e = setup<128, false>();
  if (e == cudaSuccess) e = setup<32, true>();
  if (e == cudaSuccess) e = setup<64, true>();
  if (e == cudaSuccess) e = setup<128, true>();
  return e;
}

cudaError_t launch_attn_fwd(int d, bool half, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            const AttnArgs& a, int ctas, bool combine, cudaStream_t st) {
  if (half)
    return d == 32 ? launch<32, true>(q, k, v, a, ctas, combine, st)
                   : d == 64 ? launch<64, true>(q, k, v, a, ctas, combine, st)
                            : launch<128, true>(q, k, v, a, ctas, combine, st);
  return d == 32 ? launch<32, false>(q, k, v, a, ctas, combine, st)
                 : d == 64 ? launch<64, false>(q, k, v, a, ctas, combine, st)
                           : launch<128, false>(q, k, v, a, ctas, combine, st);
}

}  // namespace arl2
