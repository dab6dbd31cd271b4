// 8-bit caches: append (quantise with block scales, optionally the key codes) and read.
//
// Both move bytes (256 B in, 128 B out per bf16 row and the reverse) with a handful of
// instructions per value, so HBM bounds them at length and latency at a few rows.
#include "kv8_internal.cuh"

namespace adamas {

// A team of `team` warps owns one block of one (sequence, kv head) of K or of V: 8 rows
// per warp (block size if smaller), held in registers between the maximum and the
// rounding, so new rows are read once.  A lane holds elements 4l .. 4l+3 of a row (the
// layout of the warp transform, which makes the key codes from the same registers).
// Several teams share a CTA when blocks are small.
constexpr int kRowsPerWarp = 8;

template <typename T, int FMT>
__global__ void __launch_bounds__(1024) kv8_append_kernel(
    Kv8 c, const T* __restrict__ kn, const T* __restrict__ vn, int64_t n_new, int64_t sb,
    int64_t sh, int64_t sn, const int32_t* __restrict__ starts,
    const int32_t* __restrict__ counts, float t, float ratio, int team, int blocks_per_seq,
    int64_t items, uint32_t* err) {
  __shared__ float warp_max[32];
  using R = Raw4<T>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int teams = (blockDim.x >> 5) / team;
  const int wt = warp % team;
  const int64_t item = int64_t(blockIdx.x) * teams + warp / team;
  // kv heads innermost: neighbouring teams read neighbouring rows of token-major input
  const int h = int(item % c.Hkv);
  int64_t r = item / c.Hkv;
  const bool is_v = r & 1;
  r >>= 1;
  const int nth = int(r % blocks_per_seq);
  const int b = int(r / blocks_per_seq);
  pdl_wait();
  pdl_trigger();
  const int bs = 1 << c.bshift;
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
  float* const scale_at = (is_v ? c.vs : c.ks) + (row0 >> c.bshift);
  const bool has_old = first < start;
  const float old_s = active && has_old ? *scale_at : 0.0f;
  const T* const src = (is_v ? vn : kn) + int64_t(b) * sb + int64_t(h) * sh;
  const int rw = bs < kRowsPerWarp ? bs : kRowsPerWarp;
  const int64_t p0 = first + wt * rw;                     // this warp's first position
  typename R::type x[kRowsPerWarp];
  float mx = 0.0f;
#pragma unroll
  for (int u = 0; u < kRowsPerWarp; ++u) {
    const int64_t p = p0 + u;
    if (active && u < rw && p >= start && p < end) {
      x[u] = R::load(src + (p - start) * sn, lane);
      float v[4];
      R::decode(x[u], v);
      mx = fmaxf(mx, fmaxf(fmaxf(finite_abs(v[0]), finite_abs(v[1])),
                           fmaxf(finite_abs(v[2]), finite_abs(v[3]))));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) warp_max[warp] = mx;
  __syncthreads();   // also: every warp of the team has read the old scale
  if (!active) return;
  // the team's maximum: lane i takes warp i's
  mx = lane < team ? warp_max[warp - wt + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const int e = scale_exponent<FMT>(mx);
  float s = pow2i(e), inv = pow2i(-e);
  uint8_t* const dst = (is_v ? c.v : c.k) + row0 * kD;
  if (has_old) {
    if (old_s >= s) {
      s = old_s;
      // 1/s: exact for the powers of two this kernel writes (never a smaller one than
      // 2^-126, so the reciprocal is finite); a foreign scale's is rounded once
      inv = 1.0f / s;
    } else {
      // the present rows move to the larger scale: v * old rounded to the new grid
#pragma unroll
      for (int u = 0; u < kRowsPerWarp; ++u) {
        const int64_t p = p0 + u;
        if (u < rw && p < start) {
          uint32_t* const w = reinterpret_cast<uint32_t*>(dst + (p - first) * kD) + lane;
          float v[4];
          unpack8<FMT>(*w, v);
          *w = pack8<FMT>(v[0] * old_s * inv, v[1] * old_s * inv, v[2] * old_s * inv,
                          v[3] * old_s * inv);
        }
      }
    }
  }
  if (wt == 0 && lane == 0) *scale_at = s;
  const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0;
#pragma unroll
  for (int u = 0; u < kRowsPerWarp; ++u) {
    const int64_t p = p0 + u;
    if (u < rw && p >= start && p < end) {
      float v[4];
      R::decode(x[u], v);
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = pow2 ? v[i] * inv : v[i] / s;
      reinterpret_cast<uint32_t*>(dst + (p - first) * kD)[lane] =
          pack8<FMT>(y[0], y[1], y[2], y[3]);
      if (!is_v && c.codes != nullptr)
        c.codes[(row0 + (p - first)) * kCodeBytes + lane] =
            static_cast<uint8_t>(warp_fwht_code(v, t, lane, ratio));
    }
  }
}

template <typename T>
static cudaError_t append_t(const Kv8& c, int fmt, const void* kn, const void* vn, int64_t n_new,
                            int64_t sb, int64_t sh, int64_t sn, const int32_t* starts,
                            const int32_t* counts, float t, float ratio, uint32_t* err,
                            cudaStream_t stream) {
  const int bs = 1 << c.bshift;
  const int team = bs < kRowsPerWarp ? 1 : bs / kRowsPerWarp;
  const int warps = team > 8 ? team : 8;
  const int teams = warps / team;
  // the blocks n_new positions can touch when they start anywhere in a block
  const int64_t per_seq = (n_new + 2 * int64_t(bs) - 2) / bs;
  const int64_t items = int64_t(c.B) * c.Hkv * 2 * per_seq;
  const int64_t grid = (items + teams - 1) / teams;
  if (per_seq > INT32_MAX || grid > INT32_MAX) return cudaErrorInvalidValue;
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
                              ratio, team, int(per_seq), items, err);
  };
  return fmt == kFmtE4m3 ? run(kv8_append_kernel<T, kFmtE4m3>)
                         : run(kv8_append_kernel<T, kFmtInt8>);
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
// A thread turns 16 bytes (an eighth of a row) into 16 values; a block covers kReadRows
// consecutive rows of one (sequence, kv head) of K (blockIdx.y = 0) or V.
constexpr int kReadThreads = 256;
constexpr int kReadPer = 4;                                   // pieces in flight per thread
constexpr int kReadRows = kReadThreads * kReadPer / 8;

__device__ __forceinline__ void store16(float* o, const float v[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 4)
    *reinterpret_cast<float4*>(o + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* o, const float v[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  reinterpret_cast<uint4*>(o)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(o)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kReadThreads) kv8_read_kernel(
    Kv8 c, const int32_t* __restrict__ starts, int64_t n, int tiles, T* __restrict__ ko,
    T* __restrict__ vo, uint32_t* err) {
  pdl_wait();
  pdl_trigger();
  const int64_t unit = blockIdx.x / tiles;
  const int64_t i0 = int64_t(blockIdx.x % tiles) * kReadRows;
  const int b = int(unit / c.Hkv), h = int(unit % c.Hkv);
  const uint8_t* const src = blockIdx.y ? c.v : c.k;
  const float* const sc = blockIdx.y ? c.vs : c.ks;
  T* const dst = (blockIdx.y ? vo : ko) + unit * n * kD;
  const int64_t start = starts[b];
  const int piece = threadIdx.x & 7;
  uint4 w[kReadPer];
  float s[kReadPer];
  bool bad = false;
#pragma unroll
  for (int u = 0; u < kReadPer; ++u) {
    const int64_t i = i0 + u * (kReadThreads / 8) + (threadIdx.x >> 3);
    w[u] = make_uint4(0u, 0u, 0u, 0u);
    s[u] = -1.0f;                                             // no such row: zeros
    if (i < n) {
      const int64_t p = start + i;
      const int64_t row = p >= 0 && p < c.Lmax ? kv8_row(c, b, h, p) : -1;
      if (row >= 0) {
        w[u] = __ldg(reinterpret_cast<const uint4*>(src + row * kD) + piece);
        s[u] = __ldg(sc + (row >> c.bshift));
      } else {
        bad = true;
      }
    }
  }
  if (bad) atomicOr(err, kErrInput);
#pragma unroll
  for (int u = 0; u < kReadPer; ++u) {
    const int64_t i = i0 + u * (kReadThreads / 8) + (threadIdx.x >> 3);
    if (i >= n) continue;
    float v[16];
    if (s[u] == -1.0f) {
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = 0.0f;
    } else {
      unpack8<FMT>(w[u].x, v);
      unpack8<FMT>(w[u].y, v + 4);
      unpack8<FMT>(w[u].z, v + 8);
      unpack8<FMT>(w[u].w, v + 12);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] *= s[u];
    }
    store16(dst + i * kD + 16 * piece, v);
  }
}

template <typename T>
static cudaError_t read_t(const Kv8& c, int fmt, const int32_t* starts, int64_t n, void* ko,
                          void* vo, uint32_t* err, cudaStream_t stream) {
  const int64_t tiles = (n + kReadRows - 1) / kReadRows;
  const int64_t grid = int64_t(c.B) * c.Hkv * tiles;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
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
