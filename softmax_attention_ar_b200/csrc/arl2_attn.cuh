// Shared parts of the training attention kernels (arl2_attn_fwd.cu, arl2_attn_bwd.cu): the
// mask, the split of the work over the CTAs, tile copies and MMA blocks.
//
// Mask. Key j is visible to query i of batch b if i < q_len[b], j < k_len[b] and, with
// frame_len F > 0, j < (floor((i + q_start) / F) + 1) F. The visible keys of a row are thus a
// prefix: row i sees the keys below limit(i), which never falls as i grows. A key's visible
// rows are a suffix of the rows inside q_len, from first_row(j) on.
//
// Split. A tile (of query rows, or of keys in the dk/dv kernel) has as many units as it has
// visible (query tile, key tile) pairs, at least one (an empty tile still writes its zeros).
// The units of all tiles, in order, are cut into equal contiguous ranges, one per CTA, so that
// every SM gets the same work whatever the lengths and masks are. A tile whose units fall to
// several CTAs is a sum of partial records in the workspace: a launch that follows adds them in
// the order of the CTAs, so the result does not depend on timing. No CTA waits for another. Where
// whole tiles, one per CTA, take hardly longer than equal ranges would, nothing is cut.
#pragma once

#include <cuda_fp16.h>

#include "arl2_device.cuh"

namespace arl2 {

struct AttnMask {
  const int* q_len;   // [B] or null
  const int* k_len;   // [B] or null
  int Tq, Tk;
  int F;              // frame_len, 0: none
  int q_start;
};

namespace {

__device__ __forceinline__ int q_length(const AttnMask& m, int b) {
  return m.q_len ? min(max(m.q_len[b], 0), m.Tq) : m.Tq;
}
__device__ __forceinline__ int k_length(const AttnMask& m, int b) {
  return m.k_len ? min(max(m.k_len[b], 0), m.Tk) : m.Tk;
}
__device__ __forceinline__ int floor_div(int x, int y) {
  const int q = x / y;
  return q * y > x ? q - 1 : q;
}
// Keys visible to row i (kl: the batch's key length).
__device__ __forceinline__ int key_limit(const AttnMask& m, int i, int kl) {
  if (m.F == 0) return kl;
  const long long lim = (static_cast<long long>(floor_div(i + m.q_start, m.F)) + 1) * m.F;
  return static_cast<int>(lim < 0 ? 0 : lim < kl ? lim : kl);
}
// First row that sees key j (may be negative or past the last row).
__device__ __forceinline__ int first_row(const AttnMask& m, int j) {
  return m.F == 0 ? -(1 << 30) : j / m.F * m.F - m.q_start;
}

// Units of a tile. Rows: tile i is query rows [i kRowsPerTile, ...), its units the key tiles that
// its last row sees. Keys: tile j is keys [128 j, ...), its units the (query head of the group,
// query tile) pairs that see its first key.
template <int kRowsPerTile>
struct RowTiles {
  // What cutting tiles costs, in units per CTA: records to write, the pipeline to fill again, and
  // the launch that adds. Forward, one 480p frame of 12 heads: 84 tiles of 13 units take 33 us
  // whole and 39 us cut into 148 ranges of 7.4 units. Backward, it hardly matters.
  static constexpr int kCutCost = kRowsPerTile == kRows ? 2 : 8;
  static __device__ int count(const AttnMask& m) { return (m.Tq + kRowsPerTile - 1) / kRowsPerTile; }
  static __device__ int valid(const AttnMask& m, int ql, int) { return (ql + kRowsPerTile - 1) / kRowsPerTile; }
  static __device__ int units(const AttnMask& m, int i, int ql, int kl, int) {
    if (i * kRowsPerTile >= ql) return 0;
    return (key_limit(m, min(ql, (i + 1) * kRowsPerTile) - 1, kl) + kRows - 1) / kRows;
  }
};
struct KeyTiles {
  static constexpr int kCutCost = 2;
  static __device__ int count(const AttnMask& m) { return (m.Tk + kRows - 1) / kRows; }
  static __device__ int valid(const AttnMask& m, int, int kl) { return (kl + kRows - 1) / kRows; }
  static __device__ int first_tile(const AttnMask& m, int j) { return max(0, first_row(m, j * kRows)) / kRows; }
  static __device__ int units(const AttnMask& m, int j, int ql, int kl, int group) {
    if (j * kRows >= kl) return 0;
    return max(0, (ql + kRows - 1) / kRows - first_tile(m, j)) * group;
  }
};

// x / y for x, y > 0 (x >= 0): a 64-bit division takes several times as long.
__device__ __forceinline__ long long quick_div(long long x, long long y) {
  return (x | y) >> 32 == 0 ? static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y)) : x / y;
}

// Where a CTA's range starts; computed by one warp, read by every role.
struct alignas(16) Split {
  long long u0, u1, total;
  int ctas;                  // CTAs that have a range
  int b, h, tile, off;       // of unit u0
  int whole;                 // nothing is cut: CTA c has tile c, and its first unit is u0 = 0
};

// Sum over a batch's tiles of the units of one head (at least one each), and the most that a tile
// has, by one warp.
template <typename Tiles>
__device__ long long head_units(const AttnMask& m, int b, int group, int* most) {
  const int ql = q_length(m, b), kl = k_length(m, b), n = Tiles::count(m);
  if (m.F == 0) {   // every valid tile has the same
    const int v = Tiles::valid(m, ql, kl), u = max(1, Tiles::units(m, 0, ql, kl, group));
    *most = max(*most, u);
    return static_cast<long long>(v) * u + (n - v);
  }
  long long s = 0;
  int top = 1;
  for (int i = threadIdx.x & 31; i < n; i += 32) {
    const int u = max(1, Tiles::units(m, i, ql, kl, group));
    s += u;
    top = max(top, u);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  *most = max(*most, __reduce_max_sync(0xffffffffu, top));
  return s;
}

// The same sum of batch b, by one thread.
template <typename Tiles>
__device__ long long thread_units(const AttnMask& m, int b, int group, int* most) {
  const int ql = q_length(m, b), kl = k_length(m, b), n = Tiles::count(m);
  if (m.F == 0) {
    const int v = Tiles::valid(m, ql, kl), u = max(1, Tiles::units(m, 0, ql, kl, group));
    *most = max(*most, u);
    return static_cast<long long>(v) * u + (n - v);
  }
  long long s = 0;
  for (int i = 0; i < n; ++i) {
    const int u = max(1, Tiles::units(m, i, ql, kl, group));
    s += u;
    *most = max(*most, u);
  }
  return s;
}

// By one warp, a lane for each batch: the units of all batches and the most that a tile has; and the
// batch that holds unit *r, which becomes the unit's place in it, with the units of one head.
template <typename Tiles>
__device__ long long lane_units(const AttnMask& m, int B, int heads, int group, int* most) {
  long long total = 0;
  int top = 1;
  for (int b = threadIdx.x & 31; b < B; b += 32) total += thread_units<Tiles>(m, b, group, &top) * heads;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  *most = __reduce_max_sync(0xffffffffu, top);
  return total;
}
template <typename Tiles>
__device__ int lane_batch(const AttnMask& m, int B, int heads, int group, long long* r,
                                       long long* per_head) {
  const int lane = threadIdx.x & 31;
  int top = 1;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const long long mine = b0 + lane < B ? thread_units<Tiles>(m, b0 + lane, group, &top) : 0, w = mine * heads;
    long long inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const long long sum = __shfl_sync(0xffffffffu, inc, 31);
    if (*r < sum) {
      const int l = __ffs(__ballot_sync(0xffffffffu, *r < inc)) - 1;
      *per_head = __shfl_sync(0xffffffffu, mine, l);
      *r -= __shfl_sync(0xffffffffu, inc - w, l);
      return b0 + l;
    }
    *r -= sum;
  }
  return B;   // not reached: r is below the sum of all
}

// With lengths, going through the batches one by one takes a CTA 0.3 us each. More batches than this
// are gone through by lanes in a launch of its own, which writes every CTA's split to memory: 64
// batches of 128 tokens and 12 heads 89 -> 49 us (37 without lengths). Where the kernels did that
// themselves, the code alone made every small call 2 us longer.
constexpr int kSplitBatches = 4;

// Whether nothing is cut, and the number of CTAs that get a range otherwise. Few units per CTA cost
// more in adding up records than they save: at least kMinUnits each, unless the tiles alone are more.
constexpr int kMinUnits = 4;
__host__ __device__ inline bool split_whole(long long tiles, long long total, long long most, long long grid,
                                            int cut_cost) {
  return tiles <= grid && most * grid <= total + cut_cost * grid;
}
__host__ __device__ inline long long split_ctas(long long tiles, long long total, long long grid) {
  long long n = total / kMinUnits;
  n = n > tiles ? n : tiles;
  n = n < total ? n : total;
  n = n < grid ? n : grid;
  return n > 1 ? n : 1;
}

// kLanes: for many batches with lengths.
template <typename Tiles, bool kLanes = false>
__device__ void make_split(const AttnMask& m, int B, int heads, int group, int c, int grid, Split* out) {
  const int lane = threadIdx.x & 31;
  const bool ragged = m.q_len || m.k_len;
  const int n = Tiles::count(m);
  // A lane sums up a batch of its own, unless the tiles are more.
  const bool by_lane =
      kLanes && ragged && (m.F == 0 || static_cast<long long>((B + 31) / 32) * n <= 8ll * B);
  long long total = 0, per_head = 0;
  int most = 1;
  if (!ragged) {
    per_head = head_units<Tiles>(m, 0, group, &most);
    total = per_head * heads * B;
  } else if (by_lane) {
    total = lane_units<Tiles>(m, B, heads, group, &most);
  } else {
    for (int b = 0; b < B; ++b) total += head_units<Tiles>(m, b, group, &most) * heads;
  }
  const long long tiles = static_cast<long long>(n) * heads * B;
  Split s{};
  s.total = total;
  if (split_whole(tiles, total, most, grid, Tiles::kCutCost)) {
    s.whole = 1;
    s.ctas = static_cast<int>(tiles);
    if (c < s.ctas) {
      s.b = c / (heads * n);
      s.h = c / n % heads;
      s.tile = c % n;
      s.u1 = max(1, Tiles::units(m, s.tile, q_length(m, s.b), k_length(m, s.b), group));
    }
    if (lane == 0) *out = s;
    return;
  }
  const long long ctas = split_ctas(tiles, total, grid);
  s.ctas = static_cast<int>(ctas);
  if (c < ctas) {
    s.u0 = quick_div(c * total, ctas);
    s.u1 = quick_div((c + 1) * total, ctas);
    long long r = s.u0;
    if (!ragged) {
      const long long per_batch = per_head * heads;
      s.b = static_cast<int>(quick_div(r, per_batch));
      r -= s.b * per_batch;
    } else if (by_lane) {
      s.b = lane_batch<Tiles>(m, B, heads, group, &r, &per_head);
    } else {
      for (; s.b < B; ++s.b) {
        per_head = head_units<Tiles>(m, s.b, group, &most);
        if (r < per_head * heads) break;
        r -= per_head * heads;
      }
    }
    s.h = static_cast<int>(quick_div(r, per_head));
    r -= s.h * per_head;
    const int ql = q_length(m, s.b), kl = k_length(m, s.b);
    if (m.F == 0) {
      const int v = Tiles::valid(m, ql, kl), w = max(1, Tiles::units(m, 0, ql, kl, group));
      if (r < static_cast<long long>(v) * w) {
        s.tile = static_cast<int>(quick_div(r, w));
        s.off = static_cast<int>(r - static_cast<long long>(s.tile) * w);
      } else {
        s.tile = v + static_cast<int>(r - static_cast<long long>(v) * w);
      }
    } else {
      for (int i0 = 0; i0 < n; i0 += 32) {
        const int w = i0 + lane < n ? max(1, Tiles::units(m, i0 + lane, ql, kl, group)) : 0;
        int inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        const int sum = __shfl_sync(0xffffffffu, inc, 31);
        if (r < sum) {
          const unsigned found = __ballot_sync(0xffffffffu, r < inc);
          const int l = __ffs(found) - 1;
          s.tile = i0 + l;
          s.off = static_cast<int>(r) - (__shfl_sync(0xffffffffu, inc, l) - __shfl_sync(0xffffffffu, w, l));
          break;
        }
        r -= sum;
      }
    }
  }
  if (lane == 0) *out = s;
}
// The split of CTA c: from `made` (see kSplitBatches) or computed here.
template <typename Tiles>
__device__ __forceinline__ void get_split(const AttnMask& m, int B, int heads, int group, int c, int grid,
                                          const Split* made, Split* out) {
  if (made) {
    const int lane = threadIdx.x & 31;
    const uint4* src = reinterpret_cast<const uint4*>(made + min(c, grid - 1));
    if (lane < static_cast<int>(sizeof(Split) / 16)) reinterpret_cast<uint4*>(out)[lane] = __ldcg(src + lane);
  } else {
    make_split<Tiles>(m, B, heads, group, c, grid, out);
  }
}

// One segment: units [kb, ke) of a tile.
struct Seg {
  int b, h, tile, kb, ke;
  int units;         // the tile's units (0: nothing is visible, one unit stands for writing zeros)
  int ql, kl;
  long long first;   // global index of the tile's first unit
  bool whole;
};
template <typename Tiles>
struct Walk {
  const AttnMask& m;
  int heads, group, ntiles;
  long long u, u1;
  int b, h, tile, off;
  __device__ Walk(const AttnMask& mask, const Split& s, int heads_, int group_)
      : m(mask), heads(heads_), group(group_), ntiles(Tiles::count(mask)), u(s.u0), u1(s.u1), b(s.b), h(s.h),
        tile(s.tile), off(s.off) {}
  __device__ bool next(Seg& g) {
    if (u >= u1) return false;
    g.b = b;
    g.h = h;
    g.tile = tile;
    g.ql = q_length(m, b);
    g.kl = k_length(m, b);
    g.units = Tiles::units(m, tile, g.ql, g.kl, group);
    const int w = max(1, g.units);
    g.kb = off;
    g.ke = static_cast<int>(min(static_cast<long long>(w), off + (u1 - u)));
    g.first = u - off;
    g.whole = g.kb == 0 && g.ke == w;
    u += g.ke - g.kb;
    off = 0;
    if (++tile == ntiles) {
      tile = 0;
      if (++h == heads) {
        h = 0;
        ++b;
      }
    }
    return true;
  }
};
// The CTA that holds unit u, and the record slot of a CTA's segment of the tile whose first unit
// is `first`: a CTA has at most two segments of tiles it shares, the first and the last of its
// range.
__device__ __forceinline__ int unit_owner(const Split& s, long long u) {
  return static_cast<int>(quick_div((u + 1) * s.ctas - 1, s.total));
}
__device__ __forceinline__ int record_slot(const Split& s, int c, long long first) {
  return 2 * c + (quick_div(c * s.total, s.ctas) >= first ? 0 : 1);
}

// ------------------------------------------------------------------ element types
template <bool kHalf>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kHalf) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    return pack_bf16x2(lo, hi);
  }
}
// Maxima that keep a NaN.
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// 2^x for a pair on the FMA pipe with paired fp32 operations, max relative error 2.7e-6 for x in
// [-125, 64]. Method as exp2_poly in arl2_device.cuh: x = n + f with n = round(x), then a degree-4
// polynomial for 2^f with equioscillating relative error (fit_exp2_poly.py). Here it is multiplied by
// 2^n, made from n's bits, in place of adding n to the exponent field: that keeps a NaN, and at the
// lower end (n = -127, where the bits give 0) the result is exactly 0, as for -inf on the MUFU unit.
__device__ __forceinline__ float2 exp2_poly4(float2 x) {
  x.x = fmax_nan(x.x, -127.f);
  x.y = fmax_nan(x.y, -127.f);
  const float2 t = __fadd2_rn(x, make_float2(12582912.f, 12582912.f));
  const float2 n = __fadd2_rn(t, make_float2(-12582912.f, -12582912.f));
  const float2 f = __ffma2_rn(n, make_float2(-1.f, -1.f), x);
  float2 p = __ffma2_rn(make_float2(0.0095701022f, 0.0095701022f), f, make_float2(0.0559178591f, 0.0559178591f));
  p = __ffma2_rn(p, f, make_float2(0.2402474433f, 0.2402474433f));
  p = __ffma2_rn(p, f, make_float2(0.6931217909f, 0.6931217909f));
  p = __ffma2_rn(p, f, make_float2(0.9999992847f, 0.9999992847f));
  return __fmul2_rn(p, make_float2(__int_as_float((__float_as_int(t.x) << 23) + 0x3f800000),
                                   __int_as_float((__float_as_int(t.y) << 23) + 0x3f800000)));
}
// Column pairs, of every 8, that take it in the backward pass; the others go to the MUFU unit.
__host__ __device__ constexpr bool fma_pair(uint32_t pairs, int j) { return (pairs >> (j & 7)) & 1u; }
__device__ __forceinline__ float2 exp2_pair(float2 x, bool on_fma) {
  return on_fma ? exp2_poly4(x) : make_float2(ex2_approx(x.x), ex2_approx(x.y));
}
// kind::f16 instruction descriptor for fp16 or bf16 operands (both of one type).
template <bool kHalf>
__host__ __device__ constexpr uint32_t attn_idesc(int N, bool a_mn, bool b_mn) {
  return kHalf ? idesc_bf16(128, N, a_mn, b_mn) & ~((7u << 7) | (7u << 10)) : idesc_bf16(128, N, a_mn, b_mn);
}

// ------------------------------------------------------------------ tiles
template <int D>
struct TileOf {
  static constexpr int kPanels = D > 64 ? 2 : 1;
  static constexpr uint32_t kBytes = kPanels * kPanelBytes;
  static constexpr int kSteps = D / 16;   // K-steps of a contraction over the head dim
};
// Copy 128 rows of one head to a swizzled tile (the caller has announced kBytes to the barrier).
// Rows behind the tensor's end and columns behind d read as zero.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int head, int row, int b) {
#pragma unroll
  for (int p = 0; p < TileOf<D>::kPanels; ++p) tma_load_4d(dst + p * kPanelBytes, map, bar, 64 * p, head, row, b);
}
// Zero rows [r0, 128) of a tile, by one warp: what stands behind a length must not reach a
// contraction over rows (0 times a NaN is a NaN).
template <int D>
__device__ __forceinline__ void zero_rows(uint32_t tile, int r0) {
  const int n = (kRows - r0) * 8;
#pragma unroll
  for (int p = 0; p < TileOf<D>::kPanels; ++p)
    for (int i = threadIdx.x & 31; i < n; i += 32) st_shared_v4(tile + p * kPanelBytes + r0 * 128 + i * 16, 0, 0, 0, 0);
}
// A tile whose rows from r0 on (r0 < 128: some) are to read as zero: copied on the side barrier,
// patched, then handed over on `full` as a plain arrival. Otherwise copied straight to `full`.
template <int D>
__device__ __forceinline__ bool load_clean(uint32_t dst, const CUtensorMap* map, uint32_t full, uint32_t side,
                                           uint32_t& side_phase, int head, int row, int b, int r0, bool lead,
                                           const Guard& g) {
  if (r0 >= kRows) {
    if (lead) {
      mbar_expect_tx(full, TileOf<D>::kBytes);
      load_tile<D>(dst, map, full, head, row, b);
    }
    return true;
  }
  if (lead) {
    mbar_expect_tx(side, TileOf<D>::kBytes);
    load_tile<D>(dst, map, side, head, row, b);
  }
  __syncwarp();
  // The copy lands by itself: the wait must not end before it, whatever other roles do.
  if (!mbar_wait_drain(side, side_phase & 1)) {
    raise_timeout(g);
    return false;
  }
  ++side_phase;
  zero_rows<D>(dst, r0);
  fence_proxy_async_smem();
  __syncwarp();
  if (lead) mbar_arrive(full);
  return true;
}

// ------------------------------------------------------------------ MMA blocks (issuing lane)
// D[tmem] = A B^T over the head dim, both operands K-major tiles.
template <int D>
__device__ __forceinline__ void mma_over_d(uint32_t d_tmem, uint32_t a_tile, uint32_t b_tile, uint32_t idesc) {
  if constexpr (D == 128) {
    mma8_ss<false, false>(d_tmem, desc_kmajor(a_tile, 0), desc_kmajor(b_tile, 0), idesc, 0u);
  } else {
    const uint64_t a0 = desc_kmajor(a_tile, 0), b0 = desc_kmajor(b_tile, 0);
#pragma unroll
    for (int s = 0; s < TileOf<D>::kSteps; ++s)
      mma_bf16(d_tmem, a0 + kmajor_step16(s), b0 + kmajor_step16(s), idesc, s > 0);
  }
}
// D[tmem] (+)= P B over 128 rows: P packed in TMEM in two parts (columns a + 8 s, and from a + 64 on
// for the second four steps), B a tile of 128 rows (MN-major).
__device__ __forceinline__ void mma_over_rows(uint32_t d_tmem, uint32_t a, uint32_t b_tile, uint32_t idesc,
                                              uint32_t acc) {
  constexpr uint32_t col[8] = {0, 8, 16, 24, 64, 72, 80, 88};
  mma8_ts(d_tmem, a, col, desc_mnmajor(b_tile, 0), idesc, acc);
}
// Steps [4 kHalf, 4 kHalf + 4) of it, P in one part (columns a + 8 s).
template <int kHalf>
__device__ __forceinline__ void mma_over_half_rows(uint32_t d_tmem, uint32_t a, uint32_t b_tile, uint32_t idesc,
                                                   uint32_t acc) {
  const uint64_t b0 = desc_mnmajor(b_tile, 0);
#pragma unroll
  for (int s = 4 * kHalf; s < 4 * kHalf + 4; ++s)
    mma_bf16_ts(d_tmem, a + 8 * s, b0 + mnmajor_step16(s), idesc, s > 0 ? 1u : acc);
}

// Registers per thread of the calling warpgroup (all four of its warps): give some back, or take
// them. The sum over the block must not exceed what it was launched with.
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

}  // namespace
}  // namespace arl2
