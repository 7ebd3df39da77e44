// C-ABI layer of the training attention (arl2_attn_* in arl2.h): the context with its scratch,
// argument checks, tensor maps and launches. The kernels are in arl2_attn_fwd.cu and
// arl2_attn_bwd.cu.
#include <algorithm>
#include <cmath>
#include <mutex>
#include <new>

#include "../../include/arl2.h"
#include "arl2_attn_kernels.h"

struct arl2_attn {
  int B = 0, H = 0, Hkv = 0, max_Tq = 0, max_Tk = 0, d = 0;
  bool half = false;
  int device = 0, sms = 0;
  float* records = nullptr;        // partial records of shared tiles, two per CTA
  float* dq_records = nullptr;     // the dq kernel's
  float* stats = nullptr;          // backward: row statistics
  unsigned long long* range = nullptr;   // backward, fp16: the words of arl2::GradRange, call first
  void* splits = nullptr;          // the CTAs' splits, where a launch of its own makes them
  unsigned int* err = nullptr;     // the error word, then the backward kernel's two tickets
  unsigned long long timeout_ns = 1000000000ull;
  size_t bytes = 0;
};

namespace {

constexpr int kMaxLen = 1 << 28;

std::mutex g_attn_mu;
bool g_attn_ready[64] = {};

arl2_status attn_prepare(int* dev, int* sms) {
  const arl2_status s = static_cast<arl2_status>(arl2::prepare_device(dev, sms));
  if (s != ARL2_OK) return s;
  std::lock_guard<std::mutex> lk(g_attn_mu);
  if (*dev < 0 || *dev >= 64) return ARL2_ERR_UNSUPPORTED;
  if (g_attn_ready[*dev]) return ARL2_OK;
  if (arl2::attn_fwd_setup() != cudaSuccess || arl2::attn_bwd_setup() != cudaSuccess) return ARL2_ERR_CUDA;
  g_attn_ready[*dev] = true;
  return ARL2_OK;
}

long long tiles(long long n, int rows) { return (n + rows - 1) / rows; }

bool at(const void* p, uintptr_t align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0; }

// A tensor [B, T, heads, d]: 16-byte aligned, strides positive multiples of 8 elements (those of
// dimensions of size 1 do not matter). An output's elements must not share memory: sorted by
// stride, each dimension steps over all of the one inside it.
bool tensor_ok(const arl2_tensor* t, int B, int T, int heads, int d, bool output) {
  if (!t || !t->ptr || !at(t->ptr, 16)) return false;
  struct Dim {
    long long n, s;
  } dims[3] = {{B, t->stride[0]}, {T, t->stride[1]}, {heads, t->stride[2]}};
  for (const Dim& x : dims)
    if (x.n > 1 && (x.s <= 0 || x.s % 8 != 0 || x.s >= (1ll << 38))) return false;
  if (!output) return true;
  std::sort(dims, dims + 3, [](const Dim& x, const Dim& y) { return x.s < y.s; });
  long long span = d;
  for (const Dim& x : dims) {
    if (x.n == 1) continue;
    if (x.s < span) return false;
    span = x.s * (x.n - 1) + span;
  }
  return true;
}

arl2_status check_call(const arl2_attn* c, const arl2_attn_shape* s) {
  if (!c || !s) return ARL2_ERR_INVALID_ARG;
  if (s->Tq < 1 || s->Tk < 1 || s->Tq > c->max_Tq || s->Tk > c->max_Tk) return ARL2_ERR_INVALID_ARG;
  if (s->frame_len < 0 || s->frame_len > kMaxLen || s->q_start < -kMaxLen || s->q_start > kMaxLen)
    return ARL2_ERR_INVALID_ARG;
  if (!(s->scale >= 0.f) || std::isinf(s->scale)) return ARL2_ERR_INVALID_ARG;
  if (!at(s->q_len, 4) || !at(s->k_len, 4)) return ARL2_ERR_INVALID_ARG;
  return ARL2_OK;
}

arl2_status on_device(const arl2_attn* c) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return ARL2_ERR_CUDA;
  return dev == c->device ? ARL2_OK : ARL2_ERR_INVALID_ARG;
}

bool tensor_map(CUtensorMap* m, const arl2_tensor* t, int B, int T, int heads, int d) {
  return arl2::encode_strided_map(m, t->ptr, B, T, heads, d, B > 1 ? t->stride[0] : d, T > 1 ? t->stride[1] : d,
                                  heads > 1 ? t->stride[2] : d);
}

// Whether the split may give parts of a tile to several CTAs. Without lengths and frames every tile
// has the same units, and the ranges' starts tell; otherwise only the device knows.
bool cuts_tiles(long long ntiles, long long units, int grid, int cut_cost) {
  const long long total = ntiles * units, ctas = arl2::split_ctas(ntiles, total, grid);
  if (arl2::split_whole(ntiles, total, units, grid, cut_cost)) return false;
  for (long long i = 1; i < ctas; ++i)
    if (i * total / ctas % units != 0) return true;
  return false;
}
bool shares_tiles(const arl2_attn* c, const arl2_attn_shape* s, bool forward) {
  if (s->q_len || s->k_len || s->frame_len) return true;
  const long long qt = tiles(s->Tq, 128), kt = tiles(s->Tk, 128), bh = static_cast<long long>(c->B) * c->H;
  if (forward) return cuts_tiles(bh * tiles(s->Tq, 256), kt, c->sms, arl2::RowTiles<256>::kCutCost);
  const int n_dkv = arl2::attn_dkv_ctas(c->sms);
  return cuts_tiles(bh * qt, kt, c->sms - n_dkv, arl2::RowTiles<128>::kCutCost) ||
         cuts_tiles(static_cast<long long>(c->B) * c->Hkv * kt, qt * (c->H / c->Hkv), n_dkv,
                    arl2::KeyTiles::kCutCost);
}

arl2::AttnOut out_of(const arl2_tensor* t) {
  return {static_cast<uint16_t*>(t->ptr), t->stride[0], t->stride[1], t->stride[2]};
}

arl2::GradRange range_of(const arl2_attn* c) {
  if (!c->range) return {};
  return {c->range, c->range + 1, c->range + 1 + static_cast<size_t>(c->B) * c->Hkv * tiles(c->max_Tq, 128)};
}

arl2::AttnArgs args_of(const arl2_attn* c, const arl2_attn_shape* s) {
  arl2::AttnArgs a{};
  a.mask = {s->q_len, s->k_len, s->Tq, s->Tk, s->frame_len, s->q_start};
  a.B = c->B;
  a.H = c->H;
  a.Hkv = c->Hkv;
  a.scale = s->scale > 0.f ? s->scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(c->d)));
  a.stats = c->stats;
  a.range = range_of(c);
  a.records = c->records;
  a.dq_records = c->dq_records;
  a.splits = (s->q_len || s->k_len) && c->B > arl2::kSplitBatches ? c->splits : nullptr;
  a.err = c->err;
  a.tickets = c->err + 1;
  a.timeout_ns = c->timeout_ns;
  return a;
}

template <typename T>
bool alloc(T** p, size_t n, size_t* total) {
  if (cudaMalloc(reinterpret_cast<void**>(p), n * sizeof(T)) != cudaSuccess) {
    *p = nullptr;
    cudaGetLastError();
    return false;
  }
  *total += n * sizeof(T);
  return true;
}

}  // namespace

extern "C" {

arl2_status arl2_attn_create(int B, int H, int H_kv, int max_Tq, int max_Tk, int d, arl2_dtype dtype,
                             arl2_attn** out) {
  if (!out) return ARL2_ERR_INVALID_ARG;
  *out = nullptr;
  if (B < 1 || H < 1 || H_kv < 1 || H % H_kv != 0 || max_Tq < 1 || max_Tk < 1 || d < 1) return ARL2_ERR_INVALID_ARG;
  if (dtype != ARL2_BF16 && dtype != ARL2_FP16) return ARL2_ERR_UNSUPPORTED;
  if ((d != 32 && d != 64 && d != 128) || static_cast<long long>(B) * H > 65535 || max_Tq > kMaxLen || max_Tk > kMaxLen)
    return ARL2_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  const arl2_status st = attn_prepare(&dev, &sms);
  if (st != ARL2_OK) return st;
  arl2_attn* c = new (std::nothrow) arl2_attn();
  if (!c) return ARL2_ERR_OOM;
  c->B = B, c->H = H, c->Hkv = H_kv, c->max_Tq = max_Tq, c->max_Tk = max_Tk, c->d = d;
  c->half = dtype == ARL2_FP16;
  c->device = dev, c->sms = sms;
  const size_t bh = static_cast<size_t>(B) * H;
  const size_t words = c->half ? 1 + static_cast<size_t>(B) * H_kv * (tiles(max_Tq, 128) + 1) : 0;
  const bool ok = alloc(&c->records, 2 * static_cast<size_t>(sms) * arl2::attn_record_floats(d), &c->bytes) &&
                  alloc(&c->dq_records, 2 * static_cast<size_t>(sms) * arl2::attn_dq_record_floats(d), &c->bytes) &&
                  alloc(reinterpret_cast<arl2::Split**>(&c->splits), sms, &c->bytes) &&
                  alloc(&c->stats, bh * arl2::attn_stat_rows(c->half) * tiles(max_Tq, 128) * 128, &c->bytes) &&
                  alloc(&c->err, 3, &c->bytes) && cudaMemset(c->err, 0, sizeof(unsigned int)) == cudaSuccess &&
                  (!words || (alloc(&c->range, words, &c->bytes) &&
                              cudaMemset(c->range, 0, words * sizeof(*c->range)) == cudaSuccess)) &&
                  cudaDeviceSynchronize() == cudaSuccess;
  if (!ok) {
    arl2_attn_destroy(c);
    return ARL2_ERR_OOM;
  }
  *out = c;
  return ARL2_OK;
}

arl2_status arl2_attn_forward(arl2_attn* c, const arl2_attn_fwd* f, arl2_stream stream) {
  if (!f) return ARL2_ERR_INVALID_ARG;
  const arl2_attn_shape* s = &f->shape;
  arl2_status st = check_call(c, s);
  if (st != ARL2_OK) return st;
  if (!tensor_ok(&f->q, c->B, s->Tq, c->H, c->d, false) || !tensor_ok(&f->k, c->B, s->Tk, c->Hkv, c->d, false) ||
      !tensor_ok(&f->v, c->B, s->Tk, c->Hkv, c->d, false) || !tensor_ok(&f->o, c->B, s->Tq, c->H, c->d, true) ||
      !f->lse || !at(f->lse, 4))
    return ARL2_ERR_INVALID_ARG;
  st = on_device(c);
  if (st != ARL2_OK) return st;
  CUtensorMap q, k, v;
  if (!tensor_map(&q, &f->q, c->B, s->Tq, c->H, c->d) || !tensor_map(&k, &f->k, c->B, s->Tk, c->Hkv, c->d) ||
      !tensor_map(&v, &f->v, c->B, s->Tk, c->Hkv, c->d))
    return ARL2_ERR_CUDA;
  arl2::AttnArgs a = args_of(c, s);
  a.o = out_of(&f->o);
  a.lse = f->lse;
  return arl2::launch_attn_fwd(c->d, c->half, q, k, v, a, c->sms, shares_tiles(c, s, true),
                               static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ARL2_OK
             : ARL2_ERR_CUDA;
}

arl2_status arl2_attn_backward(arl2_attn* c, const arl2_attn_bwd* f, arl2_stream stream) {
  if (!f) return ARL2_ERR_INVALID_ARG;
  const arl2_attn_shape* s = &f->shape;
  arl2_status st = check_call(c, s);
  if (st != ARL2_OK) return st;
  if (!tensor_ok(&f->q, c->B, s->Tq, c->H, c->d, false) || !tensor_ok(&f->k, c->B, s->Tk, c->Hkv, c->d, false) ||
      !tensor_ok(&f->v, c->B, s->Tk, c->Hkv, c->d, false) || !tensor_ok(&f->o, c->B, s->Tq, c->H, c->d, false) ||
      !tensor_ok(&f->d_o, c->B, s->Tq, c->H, c->d, false) || !tensor_ok(&f->dq, c->B, s->Tq, c->H, c->d, true) ||
      !tensor_ok(&f->dk, c->B, s->Tk, c->Hkv, c->d, true) || !tensor_ok(&f->dv, c->B, s->Tk, c->Hkv, c->d, true) ||
      !f->lse || !at(f->lse, 4))
    return ARL2_ERR_INVALID_ARG;
  st = on_device(c);
  if (st != ARL2_OK) return st;
  CUtensorMap q, k, v, g;
  if (!tensor_map(&q, &f->q, c->B, s->Tq, c->H, c->d) || !tensor_map(&k, &f->k, c->B, s->Tk, c->Hkv, c->d) ||
      !tensor_map(&v, &f->v, c->B, s->Tk, c->Hkv, c->d) || !tensor_map(&g, &f->d_o, c->B, s->Tq, c->H, c->d))
    return ARL2_ERR_CUDA;
  arl2::AttnPrepArgs p{};
  p.o = static_cast<const uint16_t*>(f->o.ptr);
  p.g = static_cast<const uint16_t*>(f->d_o.ptr);
  p.o_sb = f->o.stride[0], p.o_st = f->o.stride[1], p.o_sh = f->o.stride[2];
  p.g_sb = f->d_o.stride[0], p.g_st = f->d_o.stride[1], p.g_sh = f->d_o.stride[2];
  p.lse = f->lse;
  p.stats = c->stats;
  p.q_len = s->q_len;
  p.tickets = c->err + 1;
  p.B = c->B, p.H = c->H, p.Tq = s->Tq, p.d = c->d;
  p.v = static_cast<const uint16_t*>(f->v.ptr);
  p.v_sb = f->v.stride[0], p.v_st = f->v.stride[1], p.v_sh = f->v.stride[2];
  p.k_len = s->k_len;
  p.range = range_of(c);
  p.Hkv = c->Hkv, p.Tk = s->Tk;
  arl2::AttnArgs a = args_of(c, s);
  a.o = out_of(&f->dq);
  a.dk = out_of(&f->dk);
  a.dv = out_of(&f->dv);
  return arl2::launch_attn_bwd(c->d, c->half, q, k, v, g, p, a, c->sms, shares_tiles(c, s, false),
                               static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ARL2_OK
             : ARL2_ERR_CUDA;
}

arl2_status arl2_attn_get_status(arl2_attn* c) {
  if (!c) return ARL2_ERR_INVALID_ARG;
  if (cudaDeviceSynchronize() != cudaSuccess) return ARL2_ERR_CUDA;
  unsigned int h = 0;
  if (cudaMemcpy(&h, c->err, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess) return ARL2_ERR_CUDA;
  if (h == 0) return ARL2_OK;
  if (cudaMemset(c->err, 0, sizeof(h)) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return ARL2_ERR_CUDA;
  return ARL2_ERR_TIMEOUT;
}

size_t arl2_attn_memory_bytes(const arl2_attn* c) { return c ? c->bytes : 0; }

void arl2_attn_destroy(arl2_attn* c) {
  if (!c) return;
  cudaFree(c->records);
  cudaFree(c->dq_records);
  cudaFree(c->stats);
  cudaFree(c->range);
  cudaFree(c->splits);
  cudaFree(c->err);
  delete c;
}

}  // extern "C"
