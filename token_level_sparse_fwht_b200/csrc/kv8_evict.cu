// Eviction by accumulated attention weight: selection of the positions that stay, and the
// move that closes the gaps (in place or into another cache).
#include "kv8_internal.cuh"

#include <cooperative_groups.h>

namespace adamas {

namespace {
namespace cg = cooperative_groups;

// ---------------------------------------------------------------------- selection
// One thread-block cluster per (batch, kv head).  Each CTA keeps its share of the weights
// in shared memory (read once).  The threshold, the n-th largest weight, is found by a
// radix search over the 32-bit order-preserving keys, 11 + 11 + 10 bits: every CTA
// histograms the next digit of the keys that share the prefix found so far, reads its
// peers' histograms from distributed shared memory and finds the digit.  Then every CTA
// counts what it keeps, learns its offset from its peers, and writes positions and weights
// in order.  Protected positions (first `sink`, last `recent`) are kept besides.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxShare = 49152;                     // weights per CTA (192 KiB)
constexpr int kMaxCluster = 16;

struct SelSmem {
  uint32_t hist[2][kBins];
  uint32_t warp_a[kSelWarps], warp_b[kSelWarps];
  uint32_t kept, ties;                               // this CTA's counts (read by peers)
  uint32_t digit, above;                             // result of a search step
};

// Larger weight, larger key; -0 as +0, NaN as -inf.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (!(x == x)) x = -INFINITY;
  if (x == 0.0f) x = 0.0f;
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(
    const float* w_in, int Hkv, int64_t Lmax, const int32_t* __restrict__ seq_lens, int budget,
    int sink, int recent, int32_t* __restrict__ keep, float* w_out, int64_t Lmax_out, int cs,
    int share, uint32_t* err) {
  extern __shared__ __align__(16) uint8_t sel_raw[];
  SelSmem& sm = *reinterpret_cast<SelSmem*>(sel_raw);
  float* const val = reinterpret_cast<float*>(sel_raw + sizeof(SelSmem));
  const cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % cs;
  const int64_t unit = blockIdx.x / cs;
  pdl_wait();
  pdl_trigger();
  const int len = int(checked_len(seq_lens[unit / Hkv], Lmax, err, rank == 0 && tid == 0));
  const int lo = min(len, rank * share), n = min(len, lo + share) - lo;
  const float* const w = w_in + unit * Lmax + lo;
  int32_t* const out = keep + unit * int64_t(budget);
  for (int i = tid; i < n; i += kSelThreads) val[i] = w[i];
  for (int i = tid; i < kBins; i += kSelThreads) sm.hist[0][i] = 0u;
  __syncthreads();

  const bool cut = len > budget;
  const int mid_lo = sink, mid_hi = len - recent;    // candidates: [mid_lo, mid_hi)
  uint32_t need = cut ? uint32_t(budget - sink - recent) : 0u;
  uint32_t thr = 0xffffffffu;                        // keys above it are kept ...
  uint32_t ties = 0;                                 // ... and so many of the equal ones
  if (cut && need > 0) {
    uint32_t prefix = 0;
    int shift = 32;
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10;
      uint32_t* const hist = sm.hist[pass & 1];
      const int below = shift - bits;
      for (int i = tid; i < n; i += kSelThreads) {
        const int pos = lo + i;
        if (pos < mid_lo || pos >= mid_hi) continue;
        const uint32_t key = order_key(val[i]);
        if (pass == 0 || (key >> shift) == prefix)
          atomicAdd(&hist[(key >> below) & ((1u << bits) - 1u)], 1u);
      }
      cluster.sync();
      // all CTAs sum the cluster's histograms, four bins per thread, from the top bin down
      const int bin0 = kBins - 4 * (tid + 1);
      uint4 c = make_uint4(0u, 0u, 0u, 0u);
      for (int r = 0; r < cs; ++r) {
        const uint4 y = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(hist, r) + bin0);
        c.x += y.x;
        c.y += y.y;
        c.z += y.z;
        c.w += y.w;
      }
      const uint32_t mine = c.x + c.y + c.z + c.w;
      uint32_t inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) sm.warp_a[warp] = inc;
      // the other buffer was last read before this pass's cluster barrier
      for (int i = tid; i < kBins; i += kSelThreads) sm.hist[(pass + 1) & 1][i] = 0u;
      __syncthreads();
      uint32_t before = inc - mine;
      for (int x = 0; x < warp; ++x) before += sm.warp_a[x];
      if (before < need && before + mine >= need) {   // one thread
        uint32_t a = before;
        const uint32_t v[4] = {c.w, c.z, c.y, c.x};
        int d = bin0 + 3;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (a + v[j] >= need) break;
          a += v[j];
          --d;
        }
        sm.digit = uint32_t(d);
        sm.above = a;
      }
      __syncthreads();
      prefix = (prefix << bits) | sm.digit;
      need -= sm.above;
      shift = below;
      __syncthreads();
    }
    thr = prefix;
    ties = need;
  }
  // which positions of this share stay: 0 no, 1 yes, 2 a tie at the threshold
  const auto state = [&](int i) -> int {
    const int pos = lo + i;
    if (!cut || pos < mid_lo || pos >= mid_hi) return 1;
    if (budget == sink + recent) return 0;
    const uint32_t key = order_key(val[i]);
    return key > thr ? 1 : key == thr ? 2 : 0;
  };
  // each warp owns a run of whole 32-position groups
  const int groups = (n + 31) / 32;
  const int per = (groups + kSelWarps - 1) / kSelWarps;
  const int g0 = min(groups, warp * per), g1 = min(groups, g0 + per);
  uint32_t cnt = 0, tie = 0;
  for (int g = g0; g < g1; ++g) {
    const int i = 32 * g + lane;
    const int s = i < n ? state(i) : 0;
    cnt += __popc(__ballot_sync(0xffffffffu, s == 1));
    tie += __popc(__ballot_sync(0xffffffffu, s == 2));
  }
  if (lane == 0) {
    sm.warp_a[warp] = cnt;
    sm.warp_b[warp] = tie;
  }
  __syncthreads();
  if (tid == 0) {
    uint32_t a = 0, b = 0;
    for (int x = 0; x < kSelWarps; ++x) {
      a += sm.warp_a[x];
      b += sm.warp_b[x];
    }
    sm.kept = a;
    sm.ties = b;
  }
  cluster.sync();   // counts are out; also: every CTA of the unit has read its weights
  uint32_t ties_before = 0, at = 0;
  for (int r = 0; r < rank; ++r) {
    const SelSmem* const p = cluster.map_shared_rank(&sm, r);
    ties_before += p->ties;
    at += p->kept;
  }
  for (int x = 0; x < warp; ++x) {
    at += sm.warp_a[x];
    ties_before += sm.warp_b[x];
  }
  at += min(ties_before, ties);
  float* const wo = w_out != nullptr ? w_out + unit * Lmax_out : nullptr;
  for (int g = g0; g < g1; ++g) {
    const int i = 32 * g + lane;
    const int s = i < n ? state(i) : 0;
    const uint32_t lt = (1u << lane) - 1u;
    const uint32_t tmask = __ballot_sync(0xffffffffu, s == 2);
    const bool stay = s == 1 || (s == 2 && ties_before + __popc(tmask & lt) < ties);
    const uint32_t kmask = __ballot_sync(0xffffffffu, stay);
    if (stay) {
      const uint32_t o = at + __popc(kmask & lt);
      out[o] = lo + i;
      if (wo != nullptr) wo[o] = val[i];
    }
    at += __popc(kmask);
    ties_before += __popc(tmask);
  }
  // the rest of the list, and the weights the move leaves behind
  const int kept = min(len, budget);
  for (int i = kept + rank * kSelThreads + tid; i < budget; i += cs * kSelThreads) out[i] = -1;
  if (wo != nullptr) {
    const int top = int(min(int64_t(len), Lmax_out));
    for (int i = kept + rank * kSelThreads + tid; i < top; i += cs * kSelThreads) wo[i] = 0.0f;
  }
  cluster.sync();   // a CTA's counts stay readable until its peers have read them
}

// ----------------------------------------------------------------------- moving
// Row i of a unit comes from row keep[i] >= i (the list ascends), so moving rows down is
// safe in place if a round's rows [i, i + c) are all read, by every CTA that works on the
// unit, before any row below i + c is overwritten: later rounds read rows at or above
// i + c only.  One cluster works on one unit's K, V or codes; a round is cluster size x kMoveRows rows, held
// in registers across the cluster barrier, and the next round's rows are requested before
// this round's are written.
constexpr int kMoveThreads = 512;
constexpr int kMoveRows = 256;                       // 8-bit rows per CTA and round
constexpr int kMovePer = kMoveRows * 8 / kMoveThreads;   // 16-byte pieces per thread: 4

struct Round {
  uint4 w[kMovePer];
  float s[kMovePer];          // -1: no row
};

template <int FMT>
__device__ __forceinline__ uint32_t largest_byte(uint32_t w) {
  // magnitudes of four bytes, as bytes; an e4m3 NaN does not count
  if constexpr (FMT == kFmtE4m3) {
    w &= 0x7f7f7f7fu;
    return w & ~__vcmpeq4(w, 0x7f7f7f7fu);
  } else {
    return __vabsss4(w);
  }
}

// the magnitude a byte stands for
template <int FMT>
__device__ __forceinline__ float magnitude(uint32_t byte) {
  float v[4];
  unpack8<FMT>(byte, v);
  return v[0];
}

// blockIdx.x = ((unit * parts) + part) * cs + rank; part 0: K, 1: V, 2: codes.
template <int FMT>
__global__ void __launch_bounds__(kMoveThreads) kv8_move_kernel(
    Kv8 src, Kv8 dst, const int32_t* __restrict__ keep, int n_keep,
    const int32_t* seq_lens, int32_t* lens_out, int parts, int cs, bool in_place,
    uint32_t* err) {
  __shared__ uint32_t top[kMoveRows];                // largest value per block of the round
  __shared__ uint32_t same[kMoveRows];               // rows of the block that stay in place
  const cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x;
  const int rank = blockIdx.x % cs;
  const int part = (blockIdx.x / cs) % parts;
  const int64_t unit = blockIdx.x / (cs * parts);
  const int b = int(unit / src.Hkv), h = int(unit % src.Hkv);
  pdl_wait();
  pdl_trigger();
  const int n = min(int(checked_len(seq_lens[b], src.Lmax, err, false)), n_keep);
  // every CTA that reads seq_lens[b] takes its minimum with n_keep, so it does not matter
  // whether it sees the old length or this
  if (lens_out != nullptr && h == 0 && part == 0 && rank == 0 && tid == 0) lens_out[b] = n;
  const int32_t* const list = keep + unit * int64_t(n_keep);
  if (part == 2) {
    // codes: rows of 32 bytes, two pieces each
    constexpr int kRows = kMoveThreads * kMovePer / 2;
    for (int i0 = 0; i0 < n; i0 += kRows * cs) {
      uint4 w[kMovePer];
      int64_t to[kMovePer];
#pragma unroll
      for (int u = 0; u < kMovePer; ++u) {
        const int i = i0 + rank * kRows + (u * kMoveThreads + tid) / 2;
        to[u] = -1;
        if (i < n) {
          const int p = list[i];
          const int64_t from = p >= 0 && p < src.Lmax ? kv8_row(src, b, h, p) : -1;
          const int64_t at = kv8_row(dst, b, h, i);
          if (from >= 0 && at >= 0) {
            w[u] = *(reinterpret_cast<const uint4*>(src.codes + from * kCodeBytes) + (tid & 1));
            to[u] = at;
          } else {
            atomicOr(err, kErrInput);
          }
        }
      }
      if (in_place) cluster.sync();
#pragma unroll
      for (int u = 0; u < kMovePer; ++u)
        if (to[u] >= 0)
          *(reinterpret_cast<uint4*>(dst.codes + to[u] * kCodeBytes) + (tid & 1)) = w[u];
    }
    return;
  }
  const uint8_t* const from8 = part ? src.v : src.k;
  const float* const from_s = part ? src.vs : src.ks;
  uint8_t* const to8 = part ? dst.v : dst.k;
  float* const to_s = part ? dst.vs : dst.ks;
  const int piece = tid & 7;
  const int bs = 1 << dst.bshift;
  const auto load = [&](int i0, Round& r) {
#pragma unroll
    for (int u = 0; u < kMovePer; ++u) {
      const int i = i0 + u * (kMoveThreads / 8) + (tid >> 3);
      r.s[u] = -1.0f;
      if (i < n) {
        const int p = list[i];
        const int64_t row = p >= 0 && p < src.Lmax ? kv8_row(src, b, h, p) : -1;
        if (row >= 0) {
          r.w[u] = *(reinterpret_cast<const uint4*>(from8 + row * kD) + piece);
          r.s[u] = from_s[row >> src.bshift];
        } else {
          atomicOr(err, kErrInput);
        }
      }
    }
  };
  Round cur, nxt;
  const int stride = kMoveRows * cs;
  load(rank * kMoveRows, cur);
  for (int i0 = rank * kMoveRows; i0 - rank * kMoveRows < n; i0 += stride) {
    // the largest magnitude of every block of this CTA's rows
    for (int i = tid; i < kMoveRows; i += kMoveThreads) top[i] = same[i] = 0u;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMovePer; ++u) {
      const int r = u * (kMoveThreads / 8) + (tid >> 3);
      uint32_t m = 0;
      if (cur.s[u] != -1.0f) {
        m = __vmaxu4(__vmaxu4(largest_byte<FMT>(cur.w[u].x), largest_byte<FMT>(cur.w[u].y)),
                     __vmaxu4(largest_byte<FMT>(cur.w[u].z), largest_byte<FMT>(cur.w[u].w)));
        m = max(max(m & 0xffu, (m >> 8) & 0xffu), max((m >> 16) & 0xffu, m >> 24));
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (piece == 0 && cur.s[u] != -1.0f) {
        atomicMax(&top[r >> dst.bshift], __float_as_uint(finite_abs(magnitude<FMT>(m) * cur.s[u])));
        if (in_place && list[i0 + r] == i0 + r) atomicAdd(&same[r >> dst.bshift], 1u);
      }
    }
    if (i0 + stride - rank * kMoveRows < n) load(i0 + stride, nxt);
    if (in_place) cluster.sync();   // all rows (and scales) of this round have been read
    else __syncthreads();
#pragma unroll
    for (int u = 0; u < kMovePer; ++u) {
      const int r = u * (kMoveThreads / 8) + (tid >> 3);
      const int i = i0 + r;
      if (cur.s[u] == -1.0f) continue;
      // a block whose rows all stay keeps its bytes and its scale
      const int first = i >> dst.bshift << dst.bshift;
      if (in_place && same[r >> dst.bshift] == uint32_t(min(bs, n - first))) continue;
      const int64_t at = kv8_row(dst, b, h, i);
      if (at < 0) {
        atomicOr(err, kErrInput);
        continue;
      }
      const int e = scale_exponent<FMT>(__uint_as_float(top[r >> dst.bshift]));
      const float s = pow2i(e);
      if (piece == 0 && i == first) to_s[at >> dst.bshift] = s;
      uint32_t w[4] = {cur.w[u].x, cur.w[u].y, cur.w[u].z, cur.w[u].w};
      if (cur.s[u] != s) {
        const float inv = pow2i(-e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v[4];
          unpack8<FMT>(w[j], v);
          w[j] = pack8<FMT>(v[0] * cur.s[u] * inv, v[1] * cur.s[u] * inv, v[2] * cur.s[u] * inv,
                            v[3] * cur.s[u] * inv);
        }
      }
      *(reinterpret_cast<uint4*>(to8 + at * kD) + piece) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();   // top / same are free again
    cur = nxt;
  }
}

// Rows of kPieces 16-byte pieces, moved as they are.
__global__ void __launch_bounds__(kMoveThreads) move_rows_kernel(
    Kv8 lay, const uint4* src, uint4* dst, int pshift, const int32_t* __restrict__ keep,
    int n_keep, const int32_t* __restrict__ seq_lens, int cs, bool in_place, uint32_t* err) {
  constexpr int kPer = 8;
  const cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x;
  const int rank = blockIdx.x % cs;
  const int64_t unit = blockIdx.x / cs;
  const int b = int(unit / lay.Hkv), h = int(unit % lay.Hkv);
  pdl_wait();
  pdl_trigger();
  const int n = min(int(checked_len(seq_lens[b], lay.Lmax, err, rank == 0 && tid == 0)), n_keep);
  const int32_t* const list = keep + unit * int64_t(n_keep);
  const int rows = (kMoveThreads * kPer) >> pshift;
  const int piece = tid & ((1 << pshift) - 1);
  for (int i0 = 0; i0 < n; i0 += rows * cs) {
    uint4 w[kPer];
    int64_t to[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = i0 + rank * rows + ((u * kMoveThreads + tid) >> pshift);
      to[u] = -1;
      if (i < n) {
        const int p = list[i];
        const int64_t from = p >= 0 && p < lay.Lmax ? kv8_row(lay, b, h, p) : -1;
        const int64_t at = kv8_row(lay, b, h, i);
        if (from >= 0 && at >= 0) {
          w[u] = src[(from << pshift) + piece];
          to[u] = at;
        } else {
          atomicOr(err, kErrInput);
        }
      }
    }
    if (in_place) cluster.sync();
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (to[u] >= 0) dst[(to[u] << pshift) + piece] = w[u];
  }
}

void cluster_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], int cs) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(cs);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
}

// Cluster size of a move: as many CTAs as a unit's rows fill, at most 8 (the portable size),
// and no more than the device can use for all units at once.
int move_cluster(int64_t rows, int rows_per_cta, int64_t clusters) {
  int cs = 1;
  while (cs < 8 && int64_t(cs) * rows_per_cta < rows && clusters * cs < 2 * device_sms()) cs *= 2;
  return cs;
}

}  // namespace

bool evict_fits(int64_t Lmax) { return Lmax <= int64_t(kMaxShare) * kMaxCluster; }

cudaError_t launch_evict_select(const float* w, int B, int Hkv, int64_t Lmax,
                                const int32_t* seq_lens, int budget, int sink, int recent,
                                int32_t* keep, float* w_out, int64_t Lmax_out, uint32_t* err,
                                cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e =
      allow_smem(reinterpret_cast<const void*>(evict_select_kernel),
                 int(sizeof(SelSmem)) + kMaxShare * 4, done, true);
  if (e != cudaSuccess) return e;
  // shares of at least 4096 weights while the units leave SMs free, and of at most what
  // shared memory holds
  const int64_t units = int64_t(B) * Hkv;
  int cs = 1;
  while (cs < 8 && Lmax > int64_t(cs) * 4096 && units * cs * 2 <= 2 * device_sms()) cs *= 2;
  while (Lmax > int64_t(cs) * kMaxShare) cs *= 2;
  const int share = int((Lmax + cs - 1) / cs + 31) / 32 * 32;
  if (units * cs > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cluster_config(cfg, attr, cs);
  cfg.gridDim = dim3(unsigned(units * cs));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = sizeof(SelSmem) + size_t(share) * 4;
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel, w, Hkv, Lmax, seq_lens, budget, sink,
                            recent, keep, w_out, Lmax_out, cs, share, err);
}

cudaError_t launch_kv8_compact(const Kv8& src, const Kv8& dst, int fmt, const int32_t* keep,
                               int n_keep, const int32_t* seq_lens, int32_t* lens_out,
                               uint32_t* err, cudaStream_t stream) {
  const int parts = dst.codes != nullptr ? 3 : 2;
  const int64_t units = int64_t(src.B) * src.Hkv;
  const int cs = move_cluster(n_keep, kMoveRows, units * parts);
  if (units * parts * cs > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cluster_config(cfg, attr, cs);
  cfg.gridDim = dim3(unsigned(units * parts * cs));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = stream;
  const bool in_place = src.k == dst.k;
  if (fmt == kFmtE4m3)
    return cudaLaunchKernelEx(&cfg, kv8_move_kernel<kFmtE4m3>, src, dst, keep, n_keep, seq_lens,
                              lens_out, parts, cs, in_place, err);
  return cudaLaunchKernelEx(&cfg, kv8_move_kernel<kFmtInt8>, src, dst, keep, n_keep, seq_lens,
                            lens_out, parts, cs, in_place, err);
}

cudaError_t launch_compact_rows(const Kv8& lay, const void* src, void* dst, int row_bytes,
                                const int32_t* keep, int n_keep, const int32_t* seq_lens,
                                uint32_t* err, cudaStream_t stream) {
  int pshift = 0;
  while ((16 << pshift) < row_bytes) ++pshift;
  const int64_t units = int64_t(lay.B) * lay.Hkv;
  const int cs = move_cluster(n_keep, (kMoveThreads * 8) >> pshift, units);
  if (units * cs > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cluster_config(cfg, attr, cs);
  cfg.gridDim = dim3(unsigned(units * cs));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, move_rows_kernel, lay, static_cast<const uint4*>(src),
                            static_cast<uint4*>(dst), pshift, keep, n_keep, seq_lens, cs,
                            src == dst, err);
}

}  // namespace adamas
