// Shared pieces of the 8-bit cache kernels (sm_100a): formats, scales, layouts.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "adamas_internal.cuh"

namespace adamas {

constexpr int kFmtE4m3 = ADAMAS_KV8_E4M3;
constexpr int kFmtInt8 = ADAMAS_KV8_INT8;

// An 8-bit cache as the kernels see it.  Row indexes count d-byte rows of the whole
// buffer; since blocks neither straddle pages nor (contiguous, Lmax a multiple of the
// block) units, row >> bshift indexes the scales in both layouts.
struct Kv8 {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  uint8_t* codes;
  const int32_t* table;   // nullptr: contiguous
  int64_t Lmax;
  int64_t num_pages;
  int B, Hkv;
  int bshift;             // log2 block size
  int page_shift;
  int max_blocks;
};

// Row of position pos (0 <= pos < Lmax) of (b, h), or -1 if its page id is out of range.
__device__ __forceinline__ int64_t kv8_row(const Kv8& c, int b, int h, int64_t pos) {
  if (c.table == nullptr) return (int64_t(b) * c.Hkv + h) * c.Lmax + pos;
  const int page = c.table[int64_t(b) * c.max_blocks + (pos >> c.page_shift)];
  if (page < 0 || page >= c.num_pages) return -1;
  return ((int64_t(page) * c.Hkv + h) << c.page_shift) + (pos & ((int64_t(1) << c.page_shift) - 1));
}

// The rows of one (b, kv head), for loops over its positions.  (A buffer has fewer than 2^31 rows:
// the entry points refuse others.)
struct UnitRows {
  const int32_t* table;
  int base;      // contiguous: the row of position 0
  int pages, shift, hkv, h;
  __device__ __forceinline__ UnitRows(const Kv8& c, int b, int head)
      : table(c.table == nullptr ? nullptr : c.table + int64_t(b) * c.max_blocks),
        base(c.table == nullptr ? (b * c.Hkv + head) * int(c.Lmax) : 0), pages(int(c.num_pages)),
        shift(c.page_shift), hkv(c.Hkv), h(head) {}
  // row of position pos (0 <= pos < Lmax), or -1 if its page id is out of range
  __device__ __forceinline__ int row(int pos) const {
    if (table == nullptr) return base + pos;
    const int page = __ldg(table + (pos >> shift));
    if (page < 0 || page >= pages) return -1;
    return ((page * hkv + h) << shift) + (pos & ((1 << shift) - 1));
  }
};

// A sequence length clamped into [0, top]; one out of range is recorded.
__device__ __forceinline__ int64_t checked_len(int len, int64_t top, uint32_t* err, bool report) {
  if (len < 0 || len > top) {
    if (report) atomicOr(err, kErrInput);
    return len < 0 ? 0 : top;
  }
  return len;
}

// Exponent E of the block scale 2^E for the largest magnitude a >= 0 (finite): the
// smallest E >= -126 with a <= FMAX 2^E.  FMAX = 448 = 1.75 x 2^8 (e4m3) or
// 127 = 1.984375 x 2^6 (int8), so E follows from a's exponent and one comparison of
// its mantissa: no division, no rounding.
template <int FMT>
__device__ __forceinline__ int scale_exponent(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int ex = int(bits >> 23) - 127;
  const uint32_t mant = bits & 0x7fffffu;
  const int e = FMT == kFmtE4m3 ? ex - 8 + (mant > 0x600000u) : ex - 6 + (mant > 0x7e0000u);
  return e < -126 ? -126 : e;
}
// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// |x| for the block maximum: non-finite values do not count.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.0f;
}

// Four values (already divided by the scale) to four bytes, round to nearest even.
template <int FMT>
__device__ __forceinline__ uint32_t pack8(float a, float b, float c, float d) {
  if constexpr (FMT == kFmtE4m3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return uint32_t(lo) | (uint32_t(hi) << 16);
  } else {
    // the conversion gives 0 for NaN; the clamp is on integers
    const auto q = [](float x) {
      return uint32_t(max(-127, min(127, __float2int_rn(x)))) & 0xffu;
    };
    return q(a) | (q(b) << 8) | (q(c) << 16) | (q(d) << 24);
  }
}

// Four int8 as biased bytes (v + 128).  Opaque to the compiler, which otherwise moves the operation
// up to a conditional load of w (zeros ^ constant on the other path) and so waits for every load in
// turn: adamas_kv8_read took 44 instead of 33 us for 32K rows of 8 heads.
__device__ __forceinline__ uint32_t biased(uint32_t w) {
  uint32_t x;
  asm("xor.b32 %0, %1, 0x80808080;" : "=r"(x) : "r"(w));
  return x;
}

// Bytes 2h and 2h + 1 of w as two exact fp16 values (the lower byte in the low half).
// e4m3: one conversion.  int8: the biased byte u = v + 128 under an exponent byte 0x64
// is 1024 + u; subtracting 1152 leaves v exactly.
template <int FMT>
__device__ __forceinline__ uint32_t half2_of(uint32_t w, int h) {
  uint32_t r;
  if constexpr (FMT == kFmtE4m3) {
    if (h)
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\t"
          "cvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
          : "=r"(r)
          : "r"(w));
    else
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\t"
          "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
          : "=r"(r)
          : "r"(w));
  } else {
    const uint32_t f = __byte_perm(biased(w), 0x64646464u, h ? 0x4342u : 0x4140u);
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(f), "r"(0x64806480u));
  }
  return r;
}

// Four bytes to four floats (exact).
template <int FMT>
__device__ __forceinline__ void unpack8(uint32_t w, float v[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t x = half2_of<FMT>(w, h);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
    v[2 * h] = f.x;
    v[2 * h + 1] = f.y;
  }
}

// Four finite values times inv (a power of two that brings them into the format's range) to four
// bytes, as pack8 would.  int8: adding 1.5 x 2^23 in the same fused multiply-add rounds to an integer
// (ties to even) whose low byte is the answer.
template <int FMT>
__device__ __forceinline__ uint32_t pack8_scaled(float a, float b, float c, float d, float inv) {
  if constexpr (FMT == kFmtE4m3) {
    return pack8<FMT>(a * inv, b * inv, c * inv, d * inv);
  } else {
    const float k = 12582912.0f;
    const uint32_t ab = __byte_perm(__float_as_uint(fmaf(a, inv, k)), __float_as_uint(fmaf(b, inv, k)), 0x0040);
    const uint32_t cd = __byte_perm(__float_as_uint(fmaf(c, inv, k)), __float_as_uint(fmaf(d, inv, k)), 0x0040);
    return __byte_perm(ab, cd, 0x5410);
  }
}

// Four bytes times a scale (v * s rounded once).  int8: the biased byte in the last place of 2^23
// is a float; for a power of two s its offset leaves in the same fused multiply-add, exactly
// (kPow2; s at most kLargestShifted, so that the offset times s is finite).
constexpr float kLargestShifted = 0x1p100f;
template <int FMT, bool kPow2>
__device__ __forceinline__ void scaled8(uint32_t w, float s, float v[4]) {
  if constexpr (FMT == kFmtE4m3) {
    unpack8<FMT>(w, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= s;
  } else {
    const uint32_t x = biased(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(__byte_perm(x, 0x4b000000u, 0x7440u | i));
    if constexpr (kPow2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = fmaf(v[i], s, -8388736.0f * s);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (v[i] - 8388736.0f) * s;
    }
  }
}

// Largest magnitude among four bytes' values and m (both halves), NaN left out.
template <int FMT>
__device__ __forceinline__ __half2 max_magnitude(uint32_t w, __half2 m) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t x = half2_of<FMT>(w, h);
    m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&x)));
  }
  return m;
}

// Four bytes times r (a power of two in [2^-14, 2^14], both halves of `ratio`), rounded to the
// format; the results must be in its range.  In fp16: products of the formats' values with a power of
// two are exact there (an e4m3 result below 2^-24 rounds to zero either way).  int8: adding 1536
// in the fused multiply-add rounds to an integer (ties to even) whose low byte is the answer.
template <int FMT>
__device__ __forceinline__ uint32_t rescale8(uint32_t w, __half2 ratio) {
  const uint32_t x0 = half2_of<FMT>(w, 0), x1 = half2_of<FMT>(w, 1);
  if constexpr (FMT == kFmtE4m3) {
    const __half2 y0 = __hmul2(*reinterpret_cast<const __half2*>(&x0), ratio);
    const __half2 y1 = __hmul2(*reinterpret_cast<const __half2*>(&x1), ratio);
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(*reinterpret_cast<const uint32_t*>(&y0)));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(*reinterpret_cast<const uint32_t*>(&y1)));
    return uint32_t(lo) | (uint32_t(hi) << 16);
  } else {
    const __half2 k = __float2half2_rn(1536.0f);
    const __half2 y0 = __hfma2(*reinterpret_cast<const __half2*>(&x0), ratio, k);
    const __half2 y1 = __hfma2(*reinterpret_cast<const __half2*>(&x1), ratio, k);
    return __byte_perm(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1), 0x6420);
  }
}

// Sets a kernel's dynamic shared memory limit once per device (`done`: one bit each).
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done,
                       bool nonportable_cluster);
int device_sms();

// ---------------------------------------------------------------- launchers
cudaError_t launch_kv8_append(const Kv8& c, int fmt, const void* kn, const void* vn,
                              adamas_dtype dt, int64_t n_new, int64_t sb, int64_t sh, int64_t sn,
                              const int32_t* starts, const int32_t* counts, float t, float ratio,
                              uint32_t* err, cudaStream_t stream);
cudaError_t launch_kv8_read(const Kv8& c, int fmt, const int32_t* starts, int64_t n,
                            adamas_dtype out_dt, void* ko, void* vo, uint32_t* err,
                            cudaStream_t stream);
// idx == nullptr: dense over seq_lens (nullptr: Lmax each); else k positions per list.
size_t kv8_attention_workspace(int B, int Hq, int Hkv, int64_t Lmax, int k, bool shared,
                               bool weights);
cudaError_t launch_kv8_attention(const Kv8& c, int fmt, const void* q, adamas_dtype dt, int Hq,
                                 const int32_t* seq_lens, const int32_t* idx, int k, bool shared,
                                 void* ws, const float* w_in, float* w_out, float* out,
                                 cudaStream_t stream);
bool evict_fits(int64_t Lmax);
cudaError_t launch_evict_select(const float* w, int B, int Hkv, int64_t Lmax,
                                const int32_t* seq_lens, int budget, int sink, int recent,
                                int32_t* keep, float* w_out, int64_t Lmax_out, uint32_t* err,
                                cudaStream_t stream);
cudaError_t launch_kv8_compact(const Kv8& src, const Kv8& dst, int fmt, const int32_t* keep,
                               int n_keep, const int32_t* seq_lens, int32_t* lens_out,
                               uint32_t* err, cudaStream_t stream);
cudaError_t launch_compact_rows(const Kv8& lay, const void* src, void* dst, int row_bytes,
                                const int32_t* keep, int n_keep, const int32_t* seq_lens,
                                uint32_t* err, cudaStream_t stream);

}  // namespace adamas
