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
// histograms the next digit of the keys that share the prefix found so far and sends its
// sums of 64 bins to its peers; the 64 bins where the count is reached are then read from all
// (reading whole histograms, 64 KB per CTA, took 2 us a step).  Then every CTA
// counts what it keeps, learns its offset from its peers, and writes positions and weights
// in order.  Protected positions (first `sink`, last `recent`) are kept besides.
// The chain of three steps bounds it (histogram in shared memory, cluster barrier, search of the
// bins): 8 units of 32K weights take 14 us.  128 units of up to 16K take 33 us: they get two CTAs
// each, and as a CTA's 1024 threads take an SM, 256 CTAs on 148 SMs are two waves.
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
static_assert(kSelWarps == 32 && kBins == 64 * kSelWarps, "a warp sums 64 bins, a lane holds a warp's");
constexpr int kMaxShare = 49152;                     // weights per CTA (192 KiB, + 12 KiB of masks)
constexpr int kMaxCluster = 16;

struct SelSmem {
  uint32_t hist[2][kBins];
  uint32_t coarse[3][kMaxCluster][kSelWarps];        // per search step: every CTA's sums of 64 bins
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
  uint2* const masks = reinterpret_cast<uint2*>(val + share);   // per 32 positions: stay, tie
  const cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t chunk = blockIdx.x / uint32_t(cs);
  const int rank = int(blockIdx.x - chunk * cs);
  const int64_t unit = chunk;
  pdl_wait();
  pdl_trigger();
  cluster.barrier_arrive();
  const int len = int(checked_len(seq_lens[chunk / uint32_t(Hkv)], Lmax, err, rank == 0 && tid == 0));
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
      __syncthreads();
      // warp w sums bins 64 w .. + 63 and sends the sum to every CTA of the unit
      const uint2 two = reinterpret_cast<const uint2*>(hist)[tid];
      const uint32_t sum = __reduce_add_sync(0xffffffffu, two.x + two.y);
      if (pass == 0) cluster.barrier_wait();   // every CTA of the cluster has started
      if (lane < cs) cluster.map_shared_rank(&sm, lane)->coarse[pass][rank][warp] = sum;
      cluster.sync();
      if (warp == 0) {
        // lane l: the unit's sum of chunk 31 - l; the chunk where the count from the top
        // reaches `need`
        uint32_t c = 0;
        for (int r = 0; r < cs; ++r) c += sm.coarse[pass][r][31 - lane];
        uint32_t inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        const int l = __ffs(__ballot_sync(0xffffffffu, inc >= need)) - 1;
        const uint32_t above = __shfl_sync(0xffffffffu, inc - c, l);
        // that chunk's bins, two per lane from the top, from all CTAs
        const int bin0 = 64 * (31 - l) + 62 - 2 * lane;
        uint2 b = make_uint2(0u, 0u);
        for (int r0 = 0; r0 < cs; r0 += 8) {
          uint2 y[8];   // requested together: a read of a peer's memory takes about 0.3 us
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            y[r] = make_uint2(0u, 0u);
            if (r0 + r < cs)
              y[r] = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(hist, r0 + r) + bin0);
          }
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            b.x += y[r].x;
            b.y += y[r].y;
          }
        }
        uint32_t in2 = b.x + b.y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, in2, o);
          if (lane >= o) in2 += y;
        }
        in2 += above;
        const uint32_t before = in2 - b.x - b.y;
        if (before < need && in2 >= need) {   // one lane
          const bool second = before + b.y < need;
          sm.digit = uint32_t(bin0 + (second ? 0 : 1));
          sm.above = second ? before + b.y : before;
        }
      } else {
        // the other buffer was last read before this step's cluster barrier
        for (int i = tid - 32; i < kBins; i += kSelThreads - 32) sm.hist[(pass + 1) & 1][i] = 0u;
      }
      __syncthreads();
      prefix = (prefix << bits) | sm.digit;
      need -= sm.above;
      shift = below;
      __syncthreads();
    }
    thr = prefix;
    ties = need;
  } else {
    cluster.barrier_wait();
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
#pragma unroll 4
  for (int g = g0; g < g1; ++g) {
    const int i = 32 * g + lane;
    const int s = i < n ? state(i) : 0;
    const uint32_t yes = __ballot_sync(0xffffffffu, s == 1), eq = __ballot_sync(0xffffffffu, s == 2);
    if (lane == 0) masks[g] = make_uint2(yes, eq);
    cnt += __popc(yes);
    tie += __popc(eq);
  }
  if (lane == 0) {
    sm.warp_a[warp] = cnt;
    sm.warp_b[warp] = tie;
  }
  __syncthreads();
  const uint32_t wa = sm.warp_a[lane], wb = sm.warp_b[lane];   // one warp per lane
  if (warp == 0) {
    const uint32_t a = __reduce_add_sync(0xffffffffu, wa), b = __reduce_add_sync(0xffffffffu, wb);
    if (lane == 0) {
      sm.kept = a;
      sm.ties = b;
    }
  }
  cluster.sync();   // counts are out; also: every CTA of the unit has read its weights
  uint32_t at = 0, ties_before = 0;
  if (lane < rank) {   // rank < 16
    const SelSmem* const p = cluster.map_shared_rank(&sm, lane);
    at = p->kept;
    ties_before = p->ties;
  }
  if (lane < warp) {
    at += wa;
    ties_before += wb;
  }
  at = __reduce_add_sync(0xffffffffu, at);
  ties_before = __reduce_add_sync(0xffffffffu, ties_before);
  at += min(ties_before, ties);
  float* const wo = w_out != nullptr ? w_out + unit * Lmax_out : nullptr;
  const uint32_t lt = (1u << lane) - 1u;
#pragma unroll 4
  for (int g = g0; g < g1; ++g) {
    const uint2 m = masks[g];
    // ties are taken in order while there is room
    const uint32_t room = ties > ties_before ? ties - ties_before : 0u;
    const bool stay = (m.x >> lane & 1u) || ((m.y >> lane & 1u) && uint32_t(__popc(m.y & lt)) < room);
    const uint32_t before = __popc(m.x & lt) + min(uint32_t(__popc(m.y & lt)), room);
    if (stay) {
      const int i = 32 * g + lane;
      out[at + before] = lo + i;
      if (wo != nullptr) wo[at + before] = val[i];
    }
    at += __popc(m.x) + min(uint32_t(__popc(m.y)), room);
    ties_before += __popc(m.y);
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
// Row i of a unit comes from row keep[i] >= i (the list ascends).  Into another cache the chunks of
// rows are independent: a CTA takes up to kMoveRun of them, looks up the next one's places (list, pages)
// while it waits for the rows of the present one, and asks the next rows into L2 before it stores
// (16 ragged sequences x 8 heads to 6K rows, pages of 16, selection included: 102 us without runs, 90
// with lookups ahead, 87.4 with the rows asked for; runs of 8 90.3).
// In place one cluster works on one unit's K, V or codes in rounds of (cluster size) chunks, kept in registers across the cluster's barrier: when
// rows [i, i + c) are written, every row below i + c has been read by every CTA that needs it, and
// later rounds read rows at or above i + c only; so the next round is requested before this one's
// barrier.
constexpr int kMoveThreads = 512;
// A thread holds a quarter of a row (32 bytes; what is done per row, its address, scale and ratio,
// is then done four times, not eight as with 16 bytes: 133 -> 115 us when it was taken,
// for 16 x 8 units cut from 16K to 6K rows).
// Rows per thread: in place every round costs a cluster barrier, so it takes more rows (at 128
// registers about 90 bytes of the next round's rows are spilled; 8 units cut from 32K to 8K rows take 44 us with
// the selection, into another cache 28, caches flushed).  Into
// another cache a CTA is as small as a block allows (at least 64 rows), so that few warps wait at
// its barrier; before the runs, one row per thread took 131 us instead of 103 (the whole call), four
// 124.  Bound by the dependent loads at up to 32 warps per SM: what is moved there, 321 MB, would take
// 49 us at the copy rate.
constexpr int kMoveRun = 4;
constexpr int move_per(bool in_place) { return in_place ? 4 : 2; }
inline int move_threads(bool in_place, int bshift) {
  return in_place ? kMoveThreads : (2 << bshift) > 128 ? 2 << bshift : 128;
}

template <int kPer>
struct Round {
  uint4 w[kPer][2];
  float s[kPer];              // -1: no row
  uint32_t stays;             // bit u: row u comes from its own place
};
// Where a thread's rows come from and (into another cache) go; -1: nowhere.
template <int kPer>
struct Spots {
  int from[kPer], at[kPer];
  uint32_t stays;
};

// blockIdx.x = (unit * parts + part) * cs + rank; part 0: K, 1: V, 2: codes.  In place: cs CTAs
// (one cluster) per unit and part; else cs independent ones.  Each takes every cs-th chunk.
template <int FMT, bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads, kInPlace ? 1 : 2) kv8_move_kernel(
    Kv8 src, Kv8 dst, const int32_t* __restrict__ keep, int n_keep,
    const int32_t* seq_lens, int32_t* lens_out, int parts, int cs, uint32_t* err) {
  constexpr int kMovePer = move_per(kInPlace), kMaxRows = kMovePer * kMoveThreads / 4;
  const int threads = blockDim.x, rows = kMovePer * threads / 4;   // rows per CTA and round
  // per block of a round: 0 if no row of it came, else the bits of the largest value plus 1
  __shared__ uint32_t top[2][kMaxRows];
  __shared__ uint32_t same[kInPlace ? 2 : 1][kMaxRows];   // rows of the block that stay in place
  const int tid = threadIdx.x;
  const uint32_t chunk = blockIdx.x / uint32_t(cs);
  const int rank = int(blockIdx.x - chunk * cs);
  const uint32_t unit = chunk / uint32_t(parts);
  const int part = int(chunk - unit * parts);
  const int b = int(unit / uint32_t(src.Hkv)), h = int(unit - b * src.Hkv);
  pdl_wait();
  pdl_trigger();
  const int n = min(int(checked_len(seq_lens[b], src.Lmax, err, false)), n_keep);
  // every CTA that reads seq_lens[b] takes its minimum with n_keep, so it does not matter
  // whether it sees the old length or this
  if (lens_out != nullptr && h == 0 && part == 0 && rank == 0 && tid == 0) lens_out[b] = n;
  const int32_t* const list = keep + int64_t(unit) * n_keep;
  const UnitRows from_rows(src, b, h), to_rows(dst, b, h);
  if (part == 2) {
    // codes: rows of 32 bytes, two pieces each
    constexpr int kCodePer = 4;
    const int per_cta = threads * kCodePer / 2;
    for (int i0 = 0; i0 < n; i0 += per_cta * cs) {
      uint4 w[kCodePer];
      int to[kCodePer];
#pragma unroll
      for (int u = 0; u < kCodePer; ++u) {
        const int i = i0 + rank * per_cta + (u * threads + tid) / 2;
        to[u] = -1;
        if (i < n) {
          const int p = list[i];
          const int from = p >= 0 && p < src.Lmax ? from_rows.row(p) : -1;
          const int at = to_rows.row(i);
          if (from >= 0 && at >= 0) {
            w[u] = *(reinterpret_cast<const uint4*>(src.codes + int64_t(from) * kCodeBytes) + (tid & 1));
            to[u] = at;
          } else {
            atomicOr(err, kErrInput);
          }
        }
      }
      if (kInPlace) cg::this_cluster().sync();
#pragma unroll
      for (int u = 0; u < kCodePer; ++u)
        if (to[u] >= 0)
          *(reinterpret_cast<uint4*>(dst.codes + int64_t(to[u]) * kCodeBytes) + (tid & 1)) = w[u];
    }
    return;
  }
  if (!kInPlace && rank * rows >= n) return;
  const uint8_t* const from8 = part ? src.v : src.k;
  const float* const from_s = part ? src.vs : src.ks;
  uint8_t* const to8 = part ? dst.v : dst.k;
  float* const to_s = part ? dst.vs : dst.ks;
  const int piece = tid & 3;
  const int bs = 1 << dst.bshift;
  const auto locate = [&](int i0, Spots<kMovePer>& t) {
    int p[kMovePer];
    t.stays = 0;
#pragma unroll
    for (int u = 0; u < kMovePer; ++u) {
      const int i = i0 + u * (threads / 4) + (tid >> 2);
      // entries from n on are not used: loaded without waiting for n
      p[u] = i < n_keep ? list[i] : -1;
    }
#pragma unroll
    for (int u = 0; u < kMovePer; ++u) {
      const int i = i0 + u * (threads / 4) + (tid >> 2);
      t.from[u] = t.at[u] = -1;
      if (i >= n) continue;
      if (!kInPlace) t.at[u] = to_rows.row(i);
      t.from[u] = p[u] >= 0 && p[u] < src.Lmax ? from_rows.row(p[u]) : -1;
      if (t.from[u] < 0) atomicOr(err, kErrInput);
      if (kInPlace && p[u] == i) t.stays |= 1u << u;
    }
  };
  const auto load = [&](const Spots<kMovePer>& t, Round<kMovePer>& r) {
    r.stays = t.stays;
#pragma unroll
    for (int u = 0; u < kMovePer; ++u) {
      r.s[u] = -1.0f;
      r.w[u][0] = r.w[u][1] = make_uint4(0u, 0u, 0u, 0u);
      if (t.from[u] >= 0) {
        const uint4* const p4 = reinterpret_cast<const uint4*>(from8 + int64_t(t.from[u]) * kD) + piece;
        r.w[u][0] = p4[0];
        r.w[u][1] = p4[4];
        r.s[u] = from_s[t.from[u] >> src.bshift];
      }
    }
  };
  Round<kMovePer> cur, nxt;
  Spots<kMovePer> here, ahead;
  const int stride = rows * cs;
  int buf = 0;
  locate(rank * rows, here);
  load(here, cur);
  for (int i = tid; i < rows; i += threads) {
    top[0][i] = 0u;
    if (kInPlace) same[0][i] = 0u;
  }
  __syncthreads();
  for (int i0 = rank * rows; i0 - rank * rows * kInPlace < n; i0 += stride, buf ^= 1) {
    const bool more = i0 - rank * rows * kInPlace + stride < n;
    if (!kInPlace && more) locate(i0 + stride, ahead);
    // the largest magnitude of every block of this CTA's rows
#pragma unroll
    for (int u = 0; u < kMovePer; ++u) {
      const int r = u * (threads / 4) + (tid >> 2);
      __half2 m2 = __float2half2_rn(0.0f);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m2 = max_magnitude<FMT>(cur.w[u][j].x, m2);
        m2 = max_magnitude<FMT>(cur.w[u][j].y, m2);
        m2 = max_magnitude<FMT>(cur.w[u][j].z, m2);
        m2 = max_magnitude<FMT>(cur.w[u][j].w, m2);
      }
      const float m = __half2float(__hmax(__low2half(m2), __high2half(m2)));
      // (256 x 2^120 stands for a value of up to fp32's largest that was rounded up)
      uint32_t v = cur.s[u] != -1.0f ? __float_as_uint(fminf(m * cur.s[u], 0x1.fffffep127f)) + 1u : 0u;
      if (bs >= 8) {
        // the warp's eight rows lie in one block
        v = __reduce_max_sync(0xffffffffu, v);
        if ((tid & 31) == 0) atomicMax(&top[buf][r >> dst.bshift], v);
      } else {
        atomicMax(&top[buf][r >> dst.bshift], v);
      }
      if (kInPlace && piece == 0 && (cur.stays >> u & 1u))
        atomicAdd(&same[kInPlace ? buf : 0][r >> dst.bshift], 1u);
    }
    if (kInPlace && more) {
      locate(i0 + stride, here);
      load(here, nxt);
    }
    if (kInPlace) cg::this_cluster().sync();   // this round's rows and scales have been read
    else __syncthreads();
    if (more)
      for (int i = tid; i < rows; i += threads) {
        top[buf ^ 1][i] = 0u;
        if (kInPlace) same[kInPlace ? buf ^ 1 : 0][i] = 0u;
      }
    if (!kInPlace && more && piece == 0) {
      // the next rows come into L2 meanwhile
#pragma unroll
      for (int u = 0; u < kMovePer; ++u)
        if (ahead.from[u] >= 0)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(from8 + int64_t(ahead.from[u]) * kD));
    }
#pragma unroll
    for (int u = 0; u < kMovePer; ++u) {
      const int r = u * (threads / 4) + (tid >> 2);
      const int i = i0 + r;
      const int first = i >> dst.bshift << dst.bshift;
      const bool here_first = piece == 0 && i == first;
      const uint32_t largest = top[buf][r >> dst.bshift];
      // a row that did not come is left out, but a block's first one writes the scale of those that did
      if (cur.s[u] == -1.0f && !(here_first && largest != 0u)) continue;
      // a block whose rows all stay keeps its bytes and its scale
      if (kInPlace && same[kInPlace ? buf : 0][r >> dst.bshift] == uint32_t(min(bs, n - first)))
        continue;
      const int at = kInPlace ? to_rows.row(i) : here.at[u];
      if (at < 0) {
        atomicOr(err, kErrInput);
        continue;
      }
      bool odd_ratio = false;
      const int e = scale_exponent<FMT>(__uint_as_float(largest - 1u));
      const float s = pow2i(e);
      if (here_first) to_s[at >> dst.bshift] = s;
      if (cur.s[u] == -1.0f) continue;
      uint32_t w[8] = {cur.w[u][0].x, cur.w[u][0].y, cur.w[u][0].z, cur.w[u][0].w,
                       cur.w[u][1].x, cur.w[u][1].y, cur.w[u][1].z, cur.w[u][1].w};
      if (cur.s[u] != s) {
        const float ratio = cur.s[u] * pow2i(-e);   // exact, e being a power of two's exponent
        if ((__float_as_uint(ratio) & 0x807fffffu) == 0 && ratio >= 0x1p-14f && ratio <= 0x1p14f) {
          const __half2 r2 = __float2half2_rn(ratio);
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = rescale8<FMT>(w[j], r2);
        } else {
          odd_ratio = true;
        }
      }
      if (odd_ratio) {
        // a scale of another quantiser, or one far from the new one
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
          float v[4];
          uint32_t x = w[0];
#pragma unroll
          for (int i = 1; i < 8; ++i) x = j == i ? w[i] : x;
          unpack8<FMT>(x, v);
          const float f = pow2i(-e);
          reinterpret_cast<uint32_t*>(to8 + int64_t(at) * kD)[4 * piece + (j & 3) + 16 * (j >> 2)] =
              pack8<FMT>(v[0] * cur.s[u] * f, v[1] * cur.s[u] * f, v[2] * cur.s[u] * f,
                         v[3] * cur.s[u] * f);
        }
        continue;
      }
      uint4* const o = reinterpret_cast<uint4*>(to8 + int64_t(at) * kD) + piece;
      o[0] = make_uint4(w[0], w[1], w[2], w[3]);
      o[4] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    if (!more) return;
    __syncthreads();   // the other buffers are clear, this one is read
    if (kInPlace) {
      cur = nxt;
    } else {
      here = ahead;
      load(here, cur);
    }
  }
}

// Rows of kPieces 16-byte pieces, moved as they are.
__global__ void __launch_bounds__(kMoveThreads) move_rows_kernel(
    Kv8 lay, const uint4* src, uint4* dst, int pshift, const int32_t* __restrict__ keep,
    int n_keep, const int32_t* __restrict__ seq_lens, int cs, bool in_place, uint32_t* err) {
  constexpr int kPer = 8;
  const cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x;
  const uint32_t unit = blockIdx.x / uint32_t(cs);
  const int rank = int(blockIdx.x - unit * cs);
  const int b = int(unit / uint32_t(lay.Hkv)), h = int(unit - b * lay.Hkv);
  pdl_wait();
  pdl_trigger();
  const int n = min(int(checked_len(seq_lens[b], lay.Lmax, err, rank == 0 && tid == 0)), n_keep);
  const int32_t* const list = keep + int64_t(unit) * n_keep;
  const UnitRows rows_of(lay, b, h);
  const int rows = (kMoveThreads * kPer) >> pshift;
  const int piece = tid & ((1 << pshift) - 1);
  for (int i0 = 0; i0 < n; i0 += rows * cs) {
    uint4 w[kPer];
    int to[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = i0 + rank * rows + ((u * kMoveThreads + tid) >> pshift);
      to[u] = -1;
      if (i < n) {
        const int p = list[i];
        const int from = p >= 0 && p < lay.Lmax ? rows_of.row(p) : -1;
        const int at = rows_of.row(i);
        if (from >= 0 && at >= 0) {
          w[u] = src[(int64_t(from) << pshift) + piece];
          to[u] = at;
        } else {
          atomicOr(err, kErrInput);
        }
      }
    }
    if (in_place) cluster.sync();
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (to[u] >= 0) dst[(int64_t(to[u]) << pshift) + piece] = w[u];
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

// CTAs of a unit's part, moving into another cache: runs of chunks only where two waves of CTAs (8 per
// SM) are left.
int64_t move_ctas(int64_t chunks, int64_t units) {
  int64_t run = units * chunks / (device_sms() * int64_t(16));
  run = run < 1 ? 1 : run > kMoveRun ? kMoveRun : run;
  return (chunks + run - 1) / run;
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
                 int(sizeof(SelSmem)) + kMaxShare * 4 + kMaxShare / 4, done, true);
  if (e != cudaSuccess) return e;
  // shares of at least 4096 weights while the units leave SMs free, and of at most what
  // shared memory holds
  const int64_t units = int64_t(B) * Hkv;
  int cs = 1;
  while (cs < 8 && Lmax > int64_t(cs) * 4096 && units * cs * 2 <= 2 * device_sms()) cs *= 2;
  while (Lmax > int64_t(cs) * kMaxShare) cs *= 2;
  const int share = int((Lmax + cs - 1) / cs + 31) / 32 * 32;
  if (units * cs > INT32_MAX) return cudaErrorNotSupported;   // more blocks than a grid holds
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cluster_config(cfg, attr, cs);
  cfg.gridDim = dim3(unsigned(units * cs));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = sizeof(SelSmem) + size_t(share) * 4 + size_t(share) / 4;
  cfg.stream = stream;
  if (cs > 8) {
    // above the portable size whether 16 such CTAs find room in one GPC is the device's affair
    int fit = 0;
    cfg.numAttrs = 1;   // the cluster's shape alone
    const cudaError_t q = cudaOccupancyMaxActiveClusters(&fit, evict_select_kernel, &cfg);
    if (q != cudaSuccess) return q;
    if (fit < 1) return cudaErrorNotSupported;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, evict_select_kernel, w, Hkv, Lmax, seq_lens, budget, sink,
                            recent, keep, w_out, Lmax_out, cs, share, err);
}

cudaError_t launch_kv8_compact(const Kv8& src, const Kv8& dst, int fmt, const int32_t* keep,
                               int n_keep, const int32_t* seq_lens, int32_t* lens_out,
                               uint32_t* err, cudaStream_t stream) {
  const int parts = dst.codes != nullptr ? 3 : 2;
  const int64_t units = int64_t(src.B) * src.Hkv;
  const bool in_place = src.k == dst.k;
  const int threads = move_threads(in_place, dst.bshift);
  const int rows = move_per(in_place) * threads / 4;
  const int64_t cs = in_place ? move_cluster(n_keep, rows, units * parts)
                              : move_ctas((int64_t(n_keep) + rows - 1) / rows, units * parts);
  if (units * parts * cs > INT32_MAX) return cudaErrorNotSupported;   // more blocks than a grid holds
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cluster_config(cfg, attr, in_place ? int(cs) : 1);
  cfg.gridDim = dim3(unsigned(units * parts * cs));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.stream = stream;
  const auto run = [&](auto kernel) {
    return cudaLaunchKernelEx(&cfg, kernel, src, dst, keep, n_keep, seq_lens, lens_out, parts,
                              int(cs), err);
  };
  if (fmt == kFmtE4m3)
    return in_place ? run(kv8_move_kernel<kFmtE4m3, true>) : run(kv8_move_kernel<kFmtE4m3, false>);
  return in_place ? run(kv8_move_kernel<kFmtInt8, true>) : run(kv8_move_kernel<kFmtInt8, false>);
}

cudaError_t launch_compact_rows(const Kv8& lay, const void* src, void* dst, int row_bytes,
                                const int32_t* keep, int n_keep, const int32_t* seq_lens,
                                uint32_t* err, cudaStream_t stream) {
  int pshift = 0;
  while ((16 << pshift) < row_bytes) ++pshift;
  const int64_t units = int64_t(lay.B) * lay.Hkv;
  const int cs = move_cluster(n_keep, (kMoveThreads * 8) >> pshift, units);
  if (units * cs > INT32_MAX) return cudaErrorNotSupported;   // more blocks than a grid holds
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
