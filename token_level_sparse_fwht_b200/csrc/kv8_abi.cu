// C ABI of the 8-bit cache entry points: host-side argument checks, then dispatch.
// Every check runs before any launch; a rejected call launches nothing.
#include <cmath>

#include "kv8_internal.cuh"

namespace adamas {

int device_sms() {
  const int sms = current_device_sms(nullptr);
  return sms > 0 ? sms : 148;
}

cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done,
                       bool nonportable_cluster) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // setting it twice is harmless, so a plain flag per device (the first 64) will do
  const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && nonportable_cluster)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace adamas

using namespace adamas;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool pow2(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }
// The launchers answer cudaErrorNotSupported for sizes that no grid holds.
adamas_status from_cuda(cudaError_t e) {
  return e == cudaSuccess             ? ADAMAS_OK
         : e == cudaErrorNotSupported ? ADAMAS_ERR_UNSUPPORTED
                                      : ADAMAS_ERR_CUDA;
}
bool good_dtype(adamas_dtype dt) { return dt == ADAMAS_F32 || dt == ADAMAS_BF16; }

constexpr int64_t kMaxLen = int64_t(1) << 30;   // positions of a sequence (int32 arithmetic)

// Position layout shared by caches and by plain row buffers.
adamas_status check_layout(int B, int Hkv, int64_t Lmax, int page_size, int64_t num_pages,
                           const int32_t* table, int max_blocks, Kv8& c) {
  if (B <= 0 || Hkv <= 0 || Lmax <= 0) return ADAMAS_ERR_INVALID_ARG;
  if (int64_t(B) * Hkv > (1 << 24) || Lmax > kMaxLen) return ADAMAS_ERR_UNSUPPORTED;
  c.B = B;
  c.Hkv = Hkv;
  c.Lmax = Lmax;
  if (page_size == 0) {
    if (table != nullptr) return ADAMAS_ERR_INVALID_ARG;
    return int64_t(B) * Hkv * Lmax <= INT32_MAX ? ADAMAS_OK : ADAMAS_ERR_UNSUPPORTED;
  }
  if (page_size < 0 || page_size > (1 << 20) || !pow2(page_size)) return ADAMAS_ERR_INVALID_ARG;
  if (num_pages < 1 || num_pages > INT32_MAX || max_blocks < 1 || table == nullptr ||
      !aligned(table, 4) || int64_t(max_blocks) * page_size < Lmax)
    return ADAMAS_ERR_INVALID_ARG;
  if (num_pages > INT32_MAX / Hkv || num_pages * Hkv > INT32_MAX / page_size)
    return ADAMAS_ERR_UNSUPPORTED;   // kernels index rows with 32 bits
  c.table = table;
  c.num_pages = num_pages;
  c.max_blocks = max_blocks;
  while ((1 << c.page_shift) < page_size) ++c.page_shift;
  return ADAMAS_OK;
}

adamas_status check_cache(const adamas_kv8_cache* p, Kv8& c) {
  c = Kv8{};
  if (!p || !p->k || !p->v || !p->k_scale || !p->v_scale || p->reserved != 0)
    return ADAMAS_ERR_INVALID_ARG;
  if (p->format != ADAMAS_KV8_E4M3 && p->format != ADAMAS_KV8_INT8) return ADAMAS_ERR_INVALID_ARG;
  if (p->block_size < 1 || p->block_size > 256 || !pow2(p->block_size))
    return ADAMAS_ERR_INVALID_ARG;
  if (p->B <= 0 || p->Hkv <= 0 || p->Lmax <= 0) return ADAMAS_ERR_INVALID_ARG;
  if (p->d != kD) return ADAMAS_ERR_UNSUPPORTED;
  if (!aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->k_scale, 4) ||
      !aligned(p->v_scale, 4) || !aligned(p->codes, 16))
    return ADAMAS_ERR_INVALID_ARG;
  const adamas_status s = check_layout(p->B, p->Hkv, p->Lmax, p->page_size, p->num_pages,
                                       p->block_table, p->max_blocks_per_seq, c);
  if (s != ADAMAS_OK) return s;
  if (p->page_size == 0 ? p->Lmax % p->block_size != 0 : p->page_size < p->block_size)
    return ADAMAS_ERR_INVALID_ARG;
  c.k = p->k;
  c.v = p->v;
  c.ks = p->k_scale;
  c.vs = p->v_scale;
  c.codes = p->codes;
  while ((1 << c.bshift) < p->block_size) ++c.bshift;
  return ADAMAS_OK;
}

struct Range {
  const void* p;
  size_t bytes;
};
bool overlap(const Range& x, const Range& y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return x.p && y.p && a < b + y.bytes && b < a + x.bytes;
}
// Rows of a layout's buffer.
size_t buffer_rows(const Kv8& c) {
  return c.table ? size_t(c.num_pages) * size_t(c.Hkv) << c.page_shift
                 : size_t(c.B) * size_t(c.Hkv) * size_t(c.Lmax);
}
bool caches_overlap(const Kv8& a, const Kv8& b) {
  const auto ranges = [](const Kv8& c, Range (&r)[5]) {
    const size_t n = buffer_rows(c), blocks = n >> c.bshift;
    r[0] = {c.k, n * kD};
    r[1] = {c.v, n * kD};
    r[2] = {c.ks, blocks * 4};
    r[3] = {c.vs, blocks * 4};
    r[4] = {c.codes, n * kCodeBytes};
  };
  Range ra[5], rb[5];
  ranges(a, ra);
  ranges(b, rb);
  for (const Range& x : ra)
    for (const Range& y : rb)
      if (overlap(x, y)) return true;
  return false;
}

bool good_ws(const void* ws, size_t bytes, size_t need) {
  return ws != nullptr && aligned(ws, 256) && bytes >= need;
}
uint32_t* err_word(void* ws) {
  return reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + decode_workspace_error_offset());
}

adamas_status check_heads(int Hq, int Hkv) {
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv) return ADAMAS_ERR_INVALID_ARG;
  return Hq / Hkv <= 8 ? ADAMAS_OK : ADAMAS_ERR_UNSUPPORTED;
}

adamas_status check_weights(const float* in, const float* out) {
  if (!out) return in ? ADAMAS_ERR_INVALID_ARG : ADAMAS_OK;
  return in && aligned(in, 4) && aligned(out, 4) ? ADAMAS_OK : ADAMAS_ERR_INVALID_ARG;
}

// A call's 128-key steps are counted in 32 bits.
bool few_steps(int64_t units, int64_t n) { return units * ((n + 127) / 128) <= INT32_MAX / 2; }

// Workspace sizes also answer for arguments that no call accepts: 0.
adamas_status check_attention_sizes(int B, int Hq, int Hkv, int d, int64_t n) {
  if (B <= 0 || n <= 0) return ADAMAS_ERR_INVALID_ARG;
  const adamas_status s = check_heads(Hq, Hkv);
  if (s != ADAMAS_OK) return s;
  if (d != kD || int64_t(B) * Hkv > (1 << 24) || n > kMaxLen || !few_steps(int64_t(B) * Hq, n))
    return ADAMAS_ERR_UNSUPPORTED;
  return ADAMAS_OK;
}

adamas_status attention_common(const void* q, adamas_dtype dt, const adamas_kv8_cache* cache,
                               int Hq, const int32_t* seq_lens, const int32_t* idx, int k,
                               bool shared, void* ws, size_t ws_bytes, const float* w_in,
                               float* w_out, float* out, cudaStream_t stream) {
  if (!q || !out || !good_dtype(dt)) return ADAMAS_ERR_INVALID_ARG;
  Kv8 c;
  adamas_status s = check_cache(cache, c);
  if (s != ADAMAS_OK) return s;
  s = check_heads(Hq, c.Hkv);
  if (s != ADAMAS_OK) return s;
  if (!few_steps(int64_t(c.B) * Hq, idx ? k : c.Lmax)) return ADAMAS_ERR_UNSUPPORTED;
  s = check_weights(w_in, w_out);
  if (s != ADAMAS_OK) return s;
  const size_t w_bytes = size_t(c.B) * size_t(c.Hkv) * size_t(c.Lmax) * 4;
  if (w_in != w_out && overlap({w_in, w_bytes}, {w_out, w_bytes})) return ADAMAS_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(seq_lens, 4) || !aligned(idx, 4))
    return ADAMAS_ERR_INVALID_ARG;
  if (!good_ws(ws, ws_bytes,
               kv8_attention_workspace(c.B, Hq, c.Hkv, c.Lmax, k, shared, w_out != nullptr)))
    return ADAMAS_ERR_INVALID_ARG;
  return from_cuda(launch_kv8_attention(c, cache->format, q, dt, Hq, seq_lens, idx, k, shared, ws,
                                        w_in, w_out, out, stream));
}

}  // namespace

extern "C" {

adamas_status adamas_kv8_append(const adamas_kv8_cache* cache, const void* k_new,
                                const void* v_new, adamas_dtype dt, int64_t n_new,
                                int64_t stride_b, int64_t stride_h, int64_t stride_n,
                                const int32_t* starts, const int32_t* counts, float t,
                                float ratio, void* workspace, size_t ws_bytes,
                                cudaStream_t stream) {
  if (!k_new || !v_new || !starts || !good_dtype(dt)) return ADAMAS_ERR_INVALID_ARG;
  Kv8 c;
  const adamas_status s = check_cache(cache, c);
  if (s != ADAMAS_OK) return s;
  if (n_new <= 0 || n_new > c.Lmax) return ADAMAS_ERR_INVALID_ARG;
  const int64_t unit = dt == ADAMAS_F32 ? 4 : 8;   // elements in 16 bytes
  for (const int64_t st : {stride_b, stride_h, stride_n})
    if (st < 0 || st % unit || st > (int64_t(1) << 40)) return ADAMAS_ERR_INVALID_ARG;
  if (c.codes != nullptr) {
    if (ratio == 0.0f ? !(std::isfinite(t) && t >= 0.0f) : !(ratio > 0.0f && ratio <= 1.0f))
      return ADAMAS_ERR_INVALID_ARG;
  }
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(starts, 4) || !aligned(counts, 4) ||
      !good_ws(workspace, ws_bytes, 256))
    return ADAMAS_ERR_INVALID_ARG;
  return from_cuda(launch_kv8_append(c, cache->format, k_new, v_new, dt, n_new, stride_b, stride_h,
                                     stride_n, starts, counts, t, ratio, err_word(workspace),
                                     stream));
}

adamas_status adamas_kv8_read(const adamas_kv8_cache* cache, const int32_t* starts, int64_t n,
                              adamas_dtype out_dt, void* k_out, void* v_out, void* workspace,
                              size_t ws_bytes, cudaStream_t stream) {
  if (!starts || !k_out || !v_out || !good_dtype(out_dt)) return ADAMAS_ERR_INVALID_ARG;
  Kv8 c;
  const adamas_status s = check_cache(cache, c);
  if (s != ADAMAS_OK) return s;
  if (n <= 0 || n > kMaxLen) return ADAMAS_ERR_INVALID_ARG;
  if (!aligned(starts, 4) || !aligned(k_out, 16) || !aligned(v_out, 16) ||
      !good_ws(workspace, ws_bytes, 256))
    return ADAMAS_ERR_INVALID_ARG;
  return from_cuda(launch_kv8_read(c, cache->format, starts, n, out_dt, k_out, v_out,
                                   err_word(workspace), stream));
}

size_t adamas_kv8_attention_workspace_bytes(int B, int Hq, int Hkv, int d, int64_t Lmax,
                                            int weights) {
  if (check_attention_sizes(B, Hq, Hkv, d, Lmax) != ADAMAS_OK || (weights != 0 && weights != 1))
    return 0;
  return kv8_attention_workspace(B, Hq, Hkv, Lmax, 0, false, weights != 0);
}

adamas_status adamas_kv8_attention(const void* q, adamas_dtype dt, const adamas_kv8_cache* cache,
                                   int Hq, const int32_t* seq_lens, void* workspace,
                                   size_t ws_bytes, const float* weights_in, float* weights_out,
                                   float* out, cudaStream_t stream) {
  return attention_common(q, dt, cache, Hq, seq_lens, nullptr, 0, false, workspace, ws_bytes,
                          weights_in, weights_out, out, stream);
}

size_t adamas_kv8_sparse_attention_workspace_bytes(int B, int Hq, int Hkv, int d, int k,
                                                   int shared, int weights) {
  if (check_attention_sizes(B, Hq, Hkv, d, k) != ADAMAS_OK || (shared != 0 && shared != 1) ||
      (weights != 0 && weights != 1))
    return 0;
  return kv8_attention_workspace(B, Hq, Hkv, 1, k, shared != 0, weights != 0);
}

adamas_status adamas_kv8_sparse_attention(const void* q, adamas_dtype dt,
                                          const adamas_kv8_cache* cache, int Hq,
                                          const int32_t* idx, int k, int shared,
                                          void* workspace, size_t ws_bytes,
                                          const float* weights_in, float* weights_out,
                                          float* out, cudaStream_t stream) {
  if (!idx || k <= 0 || int64_t(k) > kMaxLen || (shared != 0 && shared != 1))
    return ADAMAS_ERR_INVALID_ARG;
  return attention_common(q, dt, cache, Hq, nullptr, idx, k, shared != 0, workspace, ws_bytes,
                          weights_in, weights_out, out, stream);
}

adamas_status adamas_evict_select(const float* weights, int B, int Hkv, int64_t Lmax,
                                  const int32_t* seq_lens, int budget, int sink, int recent,
                                  int32_t* keep, float* weights_out, int64_t Lmax_out,
                                  void* workspace, size_t ws_bytes, cudaStream_t stream) {
  if (!weights || !seq_lens || !keep || B <= 0 || Hkv <= 0 || Lmax <= 0)
    return ADAMAS_ERR_INVALID_ARG;
  // weights are indexed with 64 bits: no limit on B * Hkv * Lmax
  if (int64_t(B) * Hkv > (1 << 24) || Lmax > kMaxLen) return ADAMAS_ERR_UNSUPPORTED;
  if (budget <= 0 || sink < 0 || recent < 0 || int64_t(sink) + recent > budget ||
      int64_t(budget) > kMaxLen)
    return ADAMAS_ERR_INVALID_ARG;
  if (weights_out && (Lmax_out < budget || Lmax_out > kMaxLen || !aligned(weights_out, 4) ||
                      (weights_out == weights && Lmax_out != Lmax)))
    return ADAMAS_ERR_INVALID_ARG;
  const size_t units = size_t(B) * size_t(Hkv);
  if (weights_out != weights && overlap({weights, units * size_t(Lmax) * 4},
                                        {weights_out, units * size_t(Lmax_out) * 4}))
    return ADAMAS_ERR_INVALID_ARG;
  if (!aligned(weights, 4) || !aligned(seq_lens, 4) || !aligned(keep, 4) ||
      !good_ws(workspace, ws_bytes, 256))
    return ADAMAS_ERR_INVALID_ARG;
  if (!evict_fits(Lmax)) return ADAMAS_ERR_UNSUPPORTED;
  return from_cuda(launch_evict_select(weights, B, Hkv, Lmax, seq_lens, budget, sink, recent, keep,
                                       weights_out, Lmax_out, err_word(workspace), stream));
}

adamas_status adamas_compact_rows(const void* src, void* dst, int row_bytes, int B, int Hkv,
                                  int64_t Lmax, int page_size, int64_t num_pages,
                                  const int32_t* block_table, int max_blocks_per_seq,
                                  const int32_t* keep, int n_keep, const int32_t* seq_lens,
                                  void* workspace, size_t ws_bytes, cudaStream_t stream) {
  if (!src || !dst || !keep || !seq_lens) return ADAMAS_ERR_INVALID_ARG;
  if (row_bytes != 32 && row_bytes != 256 && row_bytes != 512) return ADAMAS_ERR_INVALID_ARG;
  Kv8 c{};
  const adamas_status s = check_layout(B, Hkv, Lmax, page_size, num_pages, block_table,
                                       max_blocks_per_seq, c);
  if (s != ADAMAS_OK) return s;
  if (n_keep <= 0 || n_keep > Lmax) return ADAMAS_ERR_INVALID_ARG;
  const size_t bytes = buffer_rows(c) * size_t(row_bytes);
  if (src != dst && overlap({src, bytes}, {dst, bytes})) return ADAMAS_ERR_INVALID_ARG;
  if (!aligned(src, 16) || !aligned(dst, 16) || !aligned(keep, 4) || !aligned(seq_lens, 4) ||
      !good_ws(workspace, ws_bytes, 256))
    return ADAMAS_ERR_INVALID_ARG;
  return from_cuda(launch_compact_rows(c, src, dst, row_bytes, keep, n_keep, seq_lens,
                                       err_word(workspace), stream));
}

adamas_status adamas_kv8_evict(const adamas_kv8_cache* src, const adamas_kv8_cache* dst,
                               const float* weights_in, float* weights_out,
                               const int32_t* seq_lens, int32_t* lens_out, int budget, int sink,
                               int recent, int32_t* keep, void* workspace, size_t ws_bytes,
                               cudaStream_t stream) {
  Kv8 a, b;
  adamas_status s = check_cache(src, a);
  if (s != ADAMAS_OK) return s;
  s = check_cache(dst, b);
  if (s != ADAMAS_OK) return s;
  if (!weights_out || !lens_out || !aligned(lens_out, 4)) return ADAMAS_ERR_INVALID_ARG;
  const size_t len_bytes = size_t(a.B) * 4;
  if (lens_out != seq_lens && overlap({seq_lens, len_bytes}, {lens_out, len_bytes}))
    return ADAMAS_ERR_INVALID_ARG;
  if (src->format != dst->format || a.B != b.B || a.Hkv != b.Hkv || b.Lmax < budget)
    return ADAMAS_ERR_INVALID_ARG;
  if (b.codes && !a.codes) return ADAMAS_ERR_INVALID_ARG;
  // in place: the same buffers in the same layout; else nothing in common
  const bool k = a.k == b.k, v = a.v == b.v, ks = a.ks == b.ks, vs = a.vs == b.vs;
  if (k != v || k != ks || k != vs || (b.codes && (a.codes == b.codes) != k))
    return ADAMAS_ERR_INVALID_ARG;
  if (!k && caches_overlap(a, b)) return ADAMAS_ERR_INVALID_ARG;
  if (k && (a.Lmax != b.Lmax || a.table != b.table || a.num_pages != b.num_pages ||
            a.page_shift != b.page_shift || a.max_blocks != b.max_blocks || a.bshift != b.bshift ||
            a.codes != b.codes))
    return ADAMAS_ERR_INVALID_ARG;
  s = adamas_evict_select(weights_in, a.B, a.Hkv, a.Lmax, seq_lens, budget, sink, recent, keep,
                          weights_out, b.Lmax, workspace, ws_bytes, stream);
  if (s != ADAMAS_OK) return s;
  return from_cuda(launch_kv8_compact(a, b, src->format, keep, budget, seq_lens, lens_out,
                                      err_word(workspace), stream));
}

}  // extern "C"
