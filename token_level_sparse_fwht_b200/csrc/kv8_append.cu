// 8-bit caches: append (quantise with block scales, optionally the key codes) and read.
//
// Both move bytes (256 B in, 128 B out per bf16 row and the reverse) with a handful of
// instructions per value, so HBM bounds them at length and latency at a few rows: 32K rows of 8
// kv heads take 33 us each way (201 MB, 6.1 TB/s), one row for each of 32 x 8 kv heads 4 us each.
// Key codes add the transform: chunks of up to 513 fp32 rows for 8 sequences x 4 heads take 8 us,
// 10 with a threshold per vector.
#include <type_traits>

#include "kv8_internal.cuh"

namespace adamas {

// A team of warps owns one block of one (sequence, kv head) of K or of V.  A lane takes 16
// bytes of a row per load (8 bf16 or 4 fp32 elements; 16 or 32 lanes to a row), kLoads loads
// under way at once and held in registers between the maximum and the rounding, so new rows
// are read once.  The maximum is taken on the raw bits (magnitudes of finite floats order as
// integers).  Several teams share a CTA when blocks are small; a block of fewer rows than a
// warp holds leaves lanes idle.
constexpr int kLoads = 8;
template <typename T>
struct Vec {
  static constexpr int kElems = 16 / int(sizeof(T));
  static constexpr int kLanes = kD / kElems;                 // lanes to a row
  static constexpr int kRowsPerLoad = 32 / kLanes;
  static constexpr int kRows = kLoads * kRowsPerLoad;        // rows a warp holds
};

// Largest magnitude of a lane's elements as fp32 bits (0x7f800000 or more if one of them is not
// finite), and the same without the non-finite ones.
__device__ __forceinline__ uint32_t top_bits(const uint4& x, float) {
  const uint32_t k = 0x7fffffffu;
  return max(max(x.x & k, x.y & k), max(x.z & k, x.w & k));
}
__device__ __forceinline__ uint32_t top_bits(const uint4& x, __nv_bfloat16) {
  const uint32_t k = 0x7fff7fffu;
  const uint32_t m = __vmaxu2(__vmaxu2(x.x & k, x.y & k), __vmaxu2(x.z & k, x.w & k));
  return max(m << 16, m & 0xffff0000u);
}
template <int E>
__device__ __forceinline__ uint32_t top_finite(const float (&v)[E]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) m = fmaxf(m, finite_abs(v[i]));
  return __float_as_uint(m);
}

__device__ __forceinline__ void elements(const uint4& x, float (&v)[4]) {
  v[0] = __uint_as_float(x.x);
  v[1] = __uint_as_float(x.y);
  v[2] = __uint_as_float(x.z);
  v[3] = __uint_as_float(x.w);
}
__device__ __forceinline__ void elements(const uint4& x, float (&v)[8]) {
  bf16x2_to_f32(x.x, v[0], v[1]);
  bf16x2_to_f32(x.y, v[2], v[3]);
  bf16x2_to_f32(x.z, v[4], v[5]);
  bf16x2_to_f32(x.w, v[6], v[7]);
}

// Key code of a row held E elements to a lane (element E l + i in lane l of the row): the
// orthonormal Walsh-Hadamard transform in natural order, index bits below log2 E inside the lane,
// the others across the row's lanes; then 2 bits per coordinate as warp_fwht_code gives them.
template <int E>
__device__ __forceinline__ uint32_t row_code(float (&v)[E], float t, float ratio, int lane) {
#pragma unroll
  for (int s = 1; s < E; s <<= 1)
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (!(i & s)) {
        const float a = v[i], b = v[i | s];
        v[i] = a + b;
        v[i | s] = a - b;
      }
#pragma unroll
  for (int s = 1; s < kD / E; s <<= 1) {
    const float sg = (lane & s) ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = fmaf(v[i], sg, __shfl_xor_sync(0xffffffffu, v[i], s));
  }
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] *= 0.088388347648318440550f;   // 1 / sqrt(128)
  if (ratio > 0.0f) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
    for (int s = kD / E / 2; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    t = ratio * m;
  }
  uint32_t code = 0;
#pragma unroll
  for (int i = 0; i < E; ++i)
    code |= (uint32_t(v[i] >= -t) + uint32_t(v[i] >= 0.0f) + uint32_t(v[i] >= t)) << (2 * i);
  return code;
}

// kCodes: the cache keeps key codes.
template <typename T, int FMT, bool kCodes>
__global__ void __launch_bounds__(256 * int(sizeof(T)), 4 / int(sizeof(T))) kv8_append_kernel(
    Kv8 c, const T* __restrict__ kn, const T* __restrict__ vn, int64_t n_new, int64_t sb,
    int64_t sh, int64_t sn, const int32_t* __restrict__ starts,
    const int32_t* __restrict__ counts, float t, float ratio, int team, uint32_t blocks_per_seq,
    uint32_t items, uint32_t* err) {
  using V = Vec<T>;
  __shared__ uint32_t warp_top[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int teams = (blockDim.x >> 5) / team;
  const int wt = warp % team;
  const uint32_t item = blockIdx.x * teams + warp / team;
  // kv heads innermost: neighbouring teams read neighbouring rows of token-major input
  const int h = int(item % uint32_t(c.Hkv));
  uint32_t r = item / uint32_t(c.Hkv);
  const bool is_v = r & 1;
  r >>= 1;
  const int b = int(r / blocks_per_seq);
  const int nth = int(r - b * blocks_per_seq);
  pdl_wait();
  pdl_trigger();
  bool active = item < items;
  int64_t start = 0, end = 0, first = 0, row0 = 0;
  if (active) {
    start = starts[b];
    const int64_t cnt = counts != nullptr ? int64_t(counts[b]) : n_new;
    if (start < 0 || cnt < 0 || cnt > n_new || start + cnt > c.Lmax) {
      if (lane == 0 && wt == 0) atomicOr(err, kErrInput);
      active = false;
    } else {
      end = start + cnt;
      first = ((start >> c.bshift) + nth) << c.bshift;   // this block's first position
      active = cnt > 0 && first < end;
    }
  }
  if (active) {
    row0 = kv8_row(c, b, h, first);
    if (row0 < 0) {
      if (lane == 0 && wt == 0) atomicOr(err, kErrInput);
      active = false;
    }
  }
  // rows of the block, relative to `first`: new ones are [lo, hi), older ones lie below lo
  const int bs = 1 << c.bshift;
  const int lo = int(max(start - first, int64_t(0)));
  const int hi = active ? int(min(end - first, int64_t(bs))) : 0;
  const int mine = wt * V::kRows + lane / V::kLanes;         // this lane's first row
  const int part = lane % V::kLanes;                         // its 16 bytes of a row
  float* const scale_at = (is_v ? c.vs : c.ks) + (row0 >> c.bshift);
  const float old_s = active && lo > 0 ? *scale_at : 0.0f;
  const T* const src = (is_v ? vn : kn) + int64_t(b) * sb + int64_t(h) * sh +
                       (first - start + mine) * sn + part * V::kElems;
  const auto piece = [&](int u) {   // the u-th of this lane's 16-byte pieces
    return __ldg(reinterpret_cast<const uint4*>(src + int64_t(u) * V::kRowsPerLoad * sn));
  };
  const auto is_new = [&](int u) {
    const int row = mine + u * V::kRowsPerLoad;
    return row >= lo && row < hi;
  };
  // a warp whose rows are all new needs no checks
  const bool whole = wt * V::kRows >= lo && (wt + 1) * V::kRows <= hi;
  uint4 x[kLoads];
  if (whole) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) x[u] = piece(u);
  } else {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      if (is_new(u)) x[u] = piece(u);
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < kLoads; ++u) top = max(top, top_bits(x[u], T{}));
  top = __reduce_max_sync(0xffffffffu, top);
  const bool odd = top >= 0x7f800000u;
  if (odd) {   // rare: the maximum again, without what is not finite
    top = 0;
#pragma unroll 1
    for (int u = 0; u < kLoads; ++u) {
      if (!is_new(u)) continue;
      float v[V::kElems];
      elements(piece(u), v);
      top = max(top, top_finite(v));
    }
    top = __reduce_max_sync(0xffffffffu, top);
  }
  if (team > 1) {
    if (lane == 0) warp_top[warp] = top;
    __syncthreads();   // also: every warp of the team has read the old scale
    top = __reduce_max_sync(0xffffffffu, lane < team ? warp_top[warp - wt + lane] : 0u);
  }
  if (hi == 0) return;
  const int e = scale_exponent<FMT>(__uint_as_float(top));
  float s = pow2i(e), inv = pow2i(-e);
  uint8_t* const dst = (is_v ? c.v : c.k) + row0 * kD;
  if (lo > 0) {
    if (old_s >= s) {
      s = old_s;
      inv = 1.0f / s;   // exact for the powers of two that this kernel writes
    } else {
      // the present rows move to the larger scale: v * old rounded to the new grid
      const int r1 = min(lo, (wt + 1) * V::kRows);
#pragma unroll 1
      for (int row = wt * V::kRows; row < r1; ++row) {
        uint32_t* const w = reinterpret_cast<uint32_t*>(dst + row * kD) + lane;
        float v[4];
        unpack8<FMT>(*w, v);
        *w = pack8<FMT>(v[0] * old_s * inv, v[1] * old_s * inv, v[2] * old_s * inv,
                        v[3] * old_s * inv);
      }
    }
  }
  if (wt == 0 && lane == 0) *scale_at = s;
  const auto store = [&](int u, const uint32_t (&w)[V::kElems / 4]) {
    uint8_t* const o = dst + (mine + u * V::kRowsPerLoad) * kD + part * V::kElems;
    if constexpr (V::kElems == 8) *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(o) = w[0];
  };
  if (odd || (__float_as_uint(s) & 0x7fffffu) != 0) {
    // not all elements are finite, or the block keeps a scale of another quantiser
#pragma unroll 1
    for (int u = 0; u < kLoads; ++u) {
      if (!is_new(u)) continue;
      float v[V::kElems];
      elements(piece(u), v);
      uint32_t w[V::kElems / 4];
#pragma unroll
      for (int i = 0; i < V::kElems / 4; ++i)
        w[i] = pack8<FMT>(v[4 * i] / s, v[4 * i + 1] / s, v[4 * i + 2] / s, v[4 * i + 3] / s);
      store(u, w);
    }
  } else {
    const auto round_rows = [&](auto all) {
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        if (!decltype(all)::value && !is_new(u)) continue;
        float v[V::kElems];
        elements(x[u], v);
        uint32_t w[V::kElems / 4];
#pragma unroll
        for (int i = 0; i < V::kElems / 4; ++i)
          w[i] = pack8_scaled<FMT>(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], inv);
        store(u, w);
      }
    };
    if (whole) round_rows(std::true_type{});
    else round_rows(std::false_type{});
  }
  if constexpr (kCodes) {
    if (is_v) return;
#pragma unroll 2
    for (int u = 0; u < kLoads; ++u) {
      // every lane of the warp takes part in the transform's exchanges
      const bool there = is_new(u);
      if (!__any_sync(0xffffffffu, there)) continue;
      float v[V::kElems];
      uint4 y = make_uint4(0u, 0u, 0u, 0u);
      if (there) y = piece(u);   // in L1 or L2 since the first pass
      elements(y, v);
      const uint32_t code = row_code<V::kElems>(v, t, ratio, lane);
      uint8_t* const o = c.codes + (row0 + mine + u * V::kRowsPerLoad) * kCodeBytes +
                         part * (V::kElems / 4);
      if (there) {
        if constexpr (V::kElems == 8) *reinterpret_cast<uint16_t*>(o) = uint16_t(code);
        else *o = uint8_t(code);
      }
    }
  }
}

template <typename T>
static cudaError_t append_t(const Kv8& c, int fmt, const void* kn, const void* vn, int64_t n_new,
                            int64_t sb, int64_t sh, int64_t sn, const int32_t* starts,
                            const int32_t* counts, float t, float ratio, uint32_t* err,
                            cudaStream_t stream) {
  const int bs = 1 << c.bshift;
  const int team = bs <= Vec<T>::kRows ? 1 : bs / Vec<T>::kRows;
  const int warps = team > 8 ? team : 8;
  const int teams = warps / team;
  // the blocks n_new positions can touch when they start anywhere in a block
  const int64_t per_seq = (n_new + 2 * int64_t(bs) - 2) / bs;
  const int64_t items = int64_t(c.B) * c.Hkv * 2 * per_seq;
  const int64_t grid = (items + teams - 1) / teams;
  if (items + teams > INT32_MAX) return cudaErrorNotSupported;   // more blocks than a grid holds
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(warps * 32));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto run = [&](auto kernel) {
    return cudaLaunchKernelEx(&cfg, kernel, c, static_cast<const T*>(kn),
                              static_cast<const T*>(vn), n_new, sb, sh, sn, starts, counts, t,
                              ratio, team, uint32_t(per_seq), uint32_t(items), err);
  };
  if (c.codes != nullptr)
    return fmt == kFmtE4m3 ? run(kv8_append_kernel<T, kFmtE4m3, true>)
                           : run(kv8_append_kernel<T, kFmtInt8, true>);
  return fmt == kFmtE4m3 ? run(kv8_append_kernel<T, kFmtE4m3, false>)
                         : run(kv8_append_kernel<T, kFmtInt8, false>);
}

cudaError_t launch_kv8_append(const Kv8& c, int fmt, const void* kn, const void* vn,
                              adamas_dtype dt, int64_t n_new, int64_t sb, int64_t sh, int64_t sn,
                              const int32_t* starts, const int32_t* counts, float t, float ratio,
                              uint32_t* err, cudaStream_t stream) {
  if (dt == ADAMAS_BF16)
    return append_t<__nv_bfloat16>(c, fmt, kn, vn, n_new, sb, sh, sn, starts, counts, t, ratio,
                                   err, stream);
  return append_t<float>(c, fmt, kn, vn, n_new, sb, sh, sn, starts, counts, t, ratio, err, stream);
}

// ------------------------------------------------------------------------- read
// A thread turns 8 bytes (a sixteenth of a row) into 8 values, so that a warp's bf16 stores are
// contiguous; a block covers kReadRows consecutive rows of one (sequence, kv head) of K
// (blockIdx.y = 0) or V.  32K rows of 8 kv heads take 32.5 us to bf16 (201 MB, 6.2 TB/s of the
// 6.55 that a copy reaches; issue slots 74 %, and part of what is written is still in L2 when the kernel
// ends), 78 us to fp32 from flushed caches (336 MB, 37 us to bf16 then).
constexpr int kReadThreads = 256;
constexpr int kReadPer = 8;                                   // pieces in flight per thread
constexpr int kReadRows = kReadThreads * kReadPer / 16;

__device__ __forceinline__ void store8(float* o, const float v[8]) {
  *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* o, const float v[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kReadThreads) kv8_read_kernel(
    Kv8 c, const int32_t* __restrict__ starts, int64_t n, int tiles, T* __restrict__ ko,
    T* __restrict__ vo, uint32_t* err) {
  pdl_wait();
  pdl_trigger();
  const uint32_t unit = blockIdx.x / uint32_t(tiles);
  const int64_t i0 = int64_t(blockIdx.x - unit * tiles) * kReadRows;
  const int b = int(unit / uint32_t(c.Hkv)), h = int(unit - b * c.Hkv);
  const uint8_t* const src = blockIdx.y ? c.v : c.k;
  const float* const sc = blockIdx.y ? c.vs : c.ks;
  const int piece = threadIdx.x & 15, row_in = threadIdx.x >> 4;
  T* const dst = (blockIdx.y ? vo : ko) + (int64_t(unit) * n + i0) * kD + 8 * piece;
  const int64_t start = starts[b];
  const UnitRows rows(c, b, h);
  uint2 w[kReadPer];
  float s[kReadPer];
  bool bad = false;
#pragma unroll
  for (int u = 0; u < kReadPer; ++u) {
    const int64_t i = i0 + u * (kReadThreads / 16) + row_in;
    w[u] = make_uint2(0u, 0u);
    s[u] = -1.0f;                                             // no such row: zeros
    if (i < n) {
      const int64_t p = start + i;
      const int row = p >= 0 && p < c.Lmax ? rows.row(int(p)) : -1;
      if (row >= 0) {
        // volatile: all of a thread's loads go out before the first is waited for
        asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];"
                     : "=r"(w[u].x), "=r"(w[u].y)
                     : "l"(src + int64_t(row) * kD + 8 * piece));
        asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(s[u]) : "l"(sc + (row >> c.bshift)));
      } else {
        bad = true;
      }
    }
  }
  if (bad) atomicOr(err, kErrInput);
  const auto write = [&](auto pow2) {
#pragma unroll
    for (int u = 0; u < kReadPer; ++u) {
      const int i = u * (kReadThreads / 16) + row_in;
      if (i0 + i >= n) continue;
      float v[8];
      const float f = s[u] == -1.0f ? 0.0f : s[u];            // no such row: zero bytes, scale 0
      scaled8<FMT, decltype(pow2)::value>(w[u].x, f, v);
      scaled8<FMT, decltype(pow2)::value>(w[u].y, f, v + 4);
      store8(dst + i * kD, v);
    }
  };
  uint32_t odd = 0;
#pragma unroll
  for (int u = 0; u < kReadPer; ++u)
    odd |= (__float_as_uint(s[u]) & 0x7fffffu) | uint32_t(fabsf(s[u]) > kLargestShifted);
  if (odd == 0) write(std::true_type{});
  else write(std::false_type{});
}

template <typename T>
static cudaError_t read_t(const Kv8& c, int fmt, const int32_t* starts, int64_t n, void* ko,
                          void* vo, uint32_t* err, cudaStream_t stream) {
  const int64_t tiles = (n + kReadRows - 1) / kReadRows;
  const int64_t grid = int64_t(c.B) * c.Hkv * tiles;
  if (grid > INT32_MAX) return cudaErrorNotSupported;   // more blocks than a grid holds
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid), 2);
  cfg.blockDim = dim3(kReadThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto run = [&](auto kernel) {
    return cudaLaunchKernelEx(&cfg, kernel, c, starts, n, int(tiles), static_cast<T*>(ko),
                              static_cast<T*>(vo), err);
  };
  return fmt == kFmtE4m3 ? run(kv8_read_kernel<T, kFmtE4m3>) : run(kv8_read_kernel<T, kFmtInt8>);
}

cudaError_t launch_kv8_read(const Kv8& c, int fmt, const int32_t* starts, int64_t n,
                            adamas_dtype out_dt, void* ko, void* vo, uint32_t* err,
                            cudaStream_t stream) {
  if (out_dt == ADAMAS_BF16) return read_t<__nv_bfloat16>(c, fmt, starts, n, ko, vo, err, stream);
  return read_t<float>(c, fmt, starts, n, ko, vo, err, stream);
}

}  // namespace adamas
