// Single-token attention over an 8-bit cache: dense (every position of a sequence) or
// sparse (given positions), one kernel, plus the pass that adds attention weights to a
// running sum.
//
// Mathematics.  For a unit (a kv head with its G query heads; in the per-head sparse form
// one query head) and its list of keys j with bytes k_j, v_j and scales a_j, c_j:
//   x_j = (q . k_j) a_j log2(e) / sqrt(d),  out = sum_j 2^(x_j - M) c_j v_j / sum_j 2^(x_j - M).
// One pass over the keys with running references instead of maxima: m is an INTEGER at or
// above every x_j seen (so 2^(x - m) is formed by one fused multiply-add and every change
// of reference, in a warp or between partial results, is an exact power of two), and
// m2 bounds x_j + log2 c_j the same way for the value sum, whose terms
// w_j = 2^(x_j - m2) c_j then lie in [0, 1] whatever the scales are.
//
// The work is 256 bytes of cache per key against 4 G d operations: HBM bounds it.  The
// tensor cores (mma.m16n8k16, fp16 operands, fp32 sums) keep the arithmetic out of the
// way; a byte of either format is exact in fp16.  Precision stays that of fp32: q is split
// into two fp16 parts (fp32 queries; a bf16 value is exact in one), scaled by a power of
// two per head, and so is w_j (times 2^14), each sum taking both parts.
//   scores: A = q (16 rows: 8 head rows, high parts; 8 rows of low parts), B = K^T.
//   values: A = V^T (16 dimensions x 16 keys), B = w^T (16 keys x 8 columns).
// The score fragment a lane gets (its head row, keys 2q, 2q+1 of two 8-key tiles) is the
// B fragment it needs for the values, so nothing is exchanged between the products.  The
// order of dimensions inside a product is free: a lane takes 16 contiguous bytes of a K
// row per load, and 16 contiguous dimensions of a V row (its outputs), pairs of keys
// interleaved by byte permutes.  With G <= 4 the 8 columns hold the high and the low parts of w
// for four heads (head rows repeated); with G <= 8 there are two column tiles.
//
// Layout of the work.  A step is 128 keys of a unit: 16 per warp, 8 warps.  The steps of all
// units form one line that is cut evenly over the CTAs (lengths are read on the device),
// so unequal sequences balance; a CTA's cut may hold the end of one unit, whole units and
// the start of another.  Each warp streams its own keys through a ring of kStages tiles in
// shared memory (16-byte asynchronous copies, rows swizzled in 16-byte chunks so that both
// products read without bank conflicts), the copies running ahead over unit borders.
// At a unit's end the 8 warps' states are merged; a unit cut between CTAs is merged from the
// partial results in the workspace, in CTA order, by the last CTA to finish its part.
#include "kv8_internal.cuh"

namespace adamas {

namespace {

constexpr int kAtWarps = 8;
constexpr int kAtThreads = kAtWarps * 32;
constexpr int kTile = 16;                        // keys per warp and step
constexpr int kStep = kAtWarps * kTile;          // keys per step
constexpr int kTileBytes = 2 * kTile * kD;       // K rows, then V rows
constexpr float kWBias = 14.0f;                  // w is held times 2^14
constexpr int kPart = 4 + kD;                    // floats of a partial: m, l, m2, 0, sums

// Shared memory of a CTA.
template <int NT, int ST>
struct Smem {
  static constexpr int kSums = NT == 1 ? 16 : 32;   // values per lane when warps are merged
  uint8_t ring[kAtWarps][ST][kTileBytes];
  float scale[kAtWarps][ST][2 * kTile];             // K scales, then V scales
  float sums[kAtWarps / 2][kSums][32];              // merge of the warps; combine scratch
  float stat[kAtWarps][8][4];                       // m, l, m2 per warp and head
  uint32_t mask[kAtWarps][ST];                      // which of a tile's keys exist
  float fin[8][2];                                  // M2 and the output factor per head
  long long base;                                   // steps before the first sequence
  long long total;
  int first_b;
  int last;
};

struct Args {
  Kv8 c;
  const void* q;
  const int32_t* seq_lens;
  const int32_t* idx;       // nullptr: dense
  float* out;
  float* part;              // [2 CTAs][G][kPart]
  float* stats;             // [B * Hq][2]: M, 1 / l (nullptr: not wanted)
  float* scores;            // [B * Hq][score_stride] (nullptr: not wanted)
  uint32_t* count;          // [units] parts done
  uint32_t* err;
  int64_t score_stride;
  float scale_log2;
  int U;                    // units per sequence
  int G;                    // query heads per unit
  int heads_per_kv;         // units per kv head (1, or the group size for per-head lists)
  int k;                    // list length (sparse)
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^(from - to) for a change of reference from <= to (integers or -inf); references that
// are equal, -inf included, change nothing.
__device__ __forceinline__ float ref_change(float from, float to) {
  return from == to ? 1.0f : ex2(from - to);
}

// cp.async that fills with zeros when !ok (nothing is read then)
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_4_or_zero(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 4 : 0)
               : "memory");
}

// 16-byte chunk ch of row r of a tile is stored at chunk ch ^ swz(r): the 8 lanes of a
// load phase (two K rows 2i, 2i + 1 and four neighbouring chunks; four V rows 2i or 2i + 1
// and two neighbouring chunks) then cover all 32 banks.
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r & 1) << 2); }

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16_rest(float lo, float hi, uint32_t taken) {
  const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&taken));
  return pack_f16(lo - t.x, hi - t.y);
}

// One step's place: unit u = (b, j), its step ls of ns.
struct Place {
  int b, j;
  int ls, ns;
  int len;
};

__device__ __forceinline__ int unit_len(const Args& a, int b, bool report) {
  if (a.idx != nullptr) return a.k;
  if (a.seq_lens == nullptr) return int(a.c.Lmax);
  return int(checked_len(a.seq_lens[b], a.c.Lmax, a.err, report));
}
__device__ __forceinline__ int steps_of(int len) { return (len + kStep - 1) / kStep; }

__device__ __forceinline__ void next_place(const Args& a, Place& p) {
  if (++p.ls < p.ns) return;
  p.ls = 0;
  if (++p.j < a.U) return;
  p.j = 0;
  do {
    ++p.b;
    p.len = unit_len(a, p.b, false);
    p.ns = steps_of(p.len);
  } while (p.ns == 0);   // the caller only moves on while steps remain
}

// Row of key `n` (0 .. 15) of this warp's tile at place p, or -1.
__device__ __forceinline__ int64_t key_row(const Args& a, const Place& p, int warp, int n) {
  const int i = p.ls * kStep + warp * kTile + n;
  if (i >= p.len) return -1;
  int64_t pos = i;
  const int h = p.j / a.heads_per_kv;
  if (a.idx != nullptr) {
    pos = a.idx[(int64_t(p.b) * a.U + p.j) * a.k + i];
    if (pos < 0) return -1;
    if (pos >= a.c.Lmax) {
      atomicOr(a.err, kErrInput);
      return -1;
    }
  }
  const int64_t row = kv8_row(a.c, p.b, h, pos);
  if (row < 0) atomicOr(a.err, kErrInput);
  return row;
}

// The query rows of a unit as A fragments.  Lane (gid, q) holds head row gid: elements
// 4 i .. 4 i + 3 of its 16-dimension runs (chunk c: dimensions 64 (c / 4) + 16 q +
// 4 (c % 4) + 0..3), scaled by 2^-e so that the head's largest element lies in [1, 2) x 2^14;
// the returned factor undoes it: x = dot * a_j * factor.
template <typename T, bool kLo>
__device__ __forceinline__ float load_q(const Args& a, int64_t row, bool exists, int q,
                                        uint32_t (&hi)[8][2], uint32_t (&lo)[kLo ? 8 : 1][2]) {
  float v[8][4];
  float mx = 0.0f;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[c][i] = 0.0f;
    if (exists)
      load4(static_cast<const T*>(a.q) + row * kD, 16 * (c >> 2) + 4 * q + (c & 3), v[c]);
#pragma unroll
    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fabsf(v[c][i]));
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  // exponent of the largest element, at least -98 (zero rows, all but denormal ones), so
  // that both powers of two are normal; infinities stay infinite
  const int e = max(int(__float_as_uint(mx) >> 23) - 127, -98);
  const float down = pow2i(14 - e);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[c][i] *= down;
    hi[c][0] = pack_f16(v[c][0], v[c][1]);
    hi[c][1] = pack_f16(v[c][2], v[c][3]);
    if constexpr (kLo) {
      lo[c][0] = pack_f16_rest(v[c][0], v[c][1], hi[c][0]);
      lo[c][1] = pack_f16_rest(v[c][2], v[c][3], hi[c][1]);
    }
  }
  return a.scale_log2 * pow2i(e - 14);
}

// FMT: byte format; NT: column tiles of the value product (1: G <= 4, 2: G <= 8); kLo: fp32
// queries; ST: ring stages.
template <typename T, int FMT, int NT, int ST, int kMinBlocks>
__global__ void __launch_bounds__(kAtThreads, kMinBlocks) kv8_attention_kernel(const Args a) {
  constexpr bool kLo = sizeof(T) == 4;
  using S = Smem<NT, ST>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, q = lane & 3;
  const int C0 = gridDim.x;
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's steps [s0, s1) of the line of all units' steps
  long long T_all, s0, s1;
  int C;
  Place pf;
  if (a.idx != nullptr || a.seq_lens == nullptr) {
    pf.len = unit_len(a, 0, false);
    pf.ns = steps_of(pf.len);
    T_all = (long long)(a.c.B) * a.U * pf.ns;
    C = int(min((long long)C0, T_all));
    const int cta = min(int(blockIdx.x), C);
    s0 = T_all * cta / C;
    s1 = T_all * min(cta + 1, C) / C;
    const long long u = s0 / pf.ns;
    pf.ls = int(s0 - u * pf.ns);
    pf.b = int(u / a.U);
    pf.j = int(u - (long long)(pf.b) * a.U);
  } else {
    long long mine = 0;
    for (int b = tid; b < a.c.B; b += kAtThreads)
      mine += steps_of(unit_len(a, b, blockIdx.x == 0));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    long long* const tot = reinterpret_cast<long long*>(&sm.sums[0][0][0]);
    if (lane == 0) tot[warp] = mine;
    __syncthreads();
    T_all = 0;
#pragma unroll
    for (int w = 0; w < kAtWarps; ++w) T_all += tot[w];
    T_all *= a.U;
    C = int(min((long long)C0, T_all));
    const int cta = min(int(blockIdx.x), C);
    s0 = C > 0 ? T_all * cta / C : 0;
    s1 = C > 0 ? T_all * min(cta + 1, C) / C : 0;
    if (warp == 0 && s0 < s1) {
      // the sequence that holds step s0: prefix sums, 32 sequences at a time
      long long before = 0;
      for (int b0 = 0;; b0 += 32) {
        const int b = b0 + lane;
        const long long n = b < a.c.B ? (long long)(steps_of(unit_len(a, b, false))) * a.U : 0;
        long long inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + inc > s0);
        if (hit) {
          const int l = __ffs(hit) - 1;
          if (lane == l) {
            sm.first_b = b;
            sm.base = before + inc - n;
          }
          break;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    __syncthreads();
    if (s0 < s1) {
      pf.b = sm.first_b;
      pf.len = unit_len(a, pf.b, false);
      pf.ns = steps_of(pf.len);
      const long long r = s0 - sm.base;
      pf.j = int(r / pf.ns);
      pf.ls = int(r - (long long)(pf.j) * pf.ns);
    }
    // sequences of length zero: their outputs are zero
    for (int b = blockIdx.x; b < a.c.B; b += C0) {
      if (unit_len(a, b, false) != 0) continue;
      for (int i = tid; i < a.U * a.G * kD; i += kAtThreads)
        a.out[int64_t(b) * a.U * a.G * kD + i] = 0.0f;
      if (a.stats != nullptr)
        for (int i = tid; i < a.U * a.G * 2; i += kAtThreads)
          a.stats[int64_t(b) * a.U * a.G * 2 + i] = 0.0f;
    }
  }
  if (s0 >= s1) return;

  // ---- ring: fetch rows one tile ahead of their copies, copies ST - 1 tiles ahead
  const uint32_t ring0 = smem_addr(&sm.ring[warp][0][0]);
  const uint32_t scale0 = smem_addr(&sm.scale[warp][0][0]);
  long long fetched = s0;
  int64_t row_next = key_row(a, pf, warp, lane & 15);
  const auto issue = [&](int st) {
    const int64_t row = row_next;
    const unsigned there = __ballot_sync(0xffffffffu, row >= 0) & 0xffffu;
    if (lane == 0) sm.mask[warp][st] = there;
    const uint32_t base = ring0 + st * kTileBytes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * i + (lane >> 3);
      const int64_t rr = __shfl_sync(0xffffffffu, row, r);
      const bool ok = rr >= 0;
      const int64_t off = (ok ? rr : 0) * kD + 16 * (lane & 7);
      const uint32_t dst = base + r * kD + 16 * ((lane & 7) ^ swz(r));
      cp_async_16_or_zero(dst, a.c.k + off, ok);
      cp_async_16_or_zero(dst + kTile * kD, a.c.v + off, ok);
    }
    const bool ok = row >= 0;
    cp_async_4_or_zero(scale0 + (st * 2 * kTile + lane) * 4,
                       (lane < 16 ? a.c.ks : a.c.vs) + ((ok ? row : 0) >> a.c.bshift), ok);
    cp_async_commit();
  };
  const auto fetch = [&]() {
    ++fetched;
    if (fetched < s1) {
      next_place(a, pf);
      row_next = key_row(a, pf, warp, lane & 15);
    }
  };
  Place cur = pf;
#pragma unroll
  for (int st = 0; st < ST - 1; ++st) {
    if (fetched < s1) {
      issue(st);
      fetch();
    } else {
      cp_async_commit();
    }
  }

  uint32_t qh[8][2], ql[kLo ? 8 : 1][2];
  float factor = 0.0f;
  float m = -INFINITY, m2 = -INFINITY, l = 0.0f;
  float acc[NT][8][4];
  const int head = NT == 1 ? (gid & 3) : gid;       // this lane's head row
  const bool head_ok = head < a.G;
  bool fresh = true;
  int st = 0;
  for (long long s = s0; s < s1; ++s) {
    {
      int sn = st + ST - 1;
      if (sn >= ST) sn -= ST;
      if (fetched < s1) {
        issue(sn);
        fetch();
      } else {
        cp_async_commit();
      }
    }
    const int64_t unit = int64_t(cur.b) * a.U + cur.j;
    if (fresh) {
      factor = load_q<T, kLo>(a, unit * a.G + head, head_ok, q, qh, ql);
      m = m2 = -INFINITY;
      l = 0.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][t][i] = 0.0f;
      fresh = false;
    }
    cp_async_wait_pending(ST - 1);
    __syncwarp();
    const uint32_t mask = sm.mask[warp][st];
    if (mask != 0) {
      const uint8_t* const tile = sm.ring[warp][st];
      const float* const sc = sm.scale[warp][st];
      // ---- scores of keys 8 tau + 2 q + {0, 1}, tau = 0, 1
      float x[4], sf[4];
#pragma unroll
      for (int tau = 0; tau < 2; ++tau) {
        const int r = 8 * tau + gid;
        float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 w =
              *reinterpret_cast<const uint4*>(tile + r * kD + 16 * ((4 * j + q) ^ swz(r)));
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = 4 * j + i;
            const uint32_t b0 = half2_of<FMT>(ww[i], 0), b1 = half2_of<FMT>(ww[i], 1);
            const uint32_t l0 = kLo ? ql[kLo ? c : 0][0] : 0u, l1 = kLo ? ql[kLo ? c : 0][1] : 0u;
            if (j == 0) mma_f16(c0, qh[c][0], l0, qh[c][1], l1, b0, b1);
            else mma_f16(c1, qh[c][0], l0, qh[c][1], l1, b0, b1);
          }
        }
        const float2 ks = *reinterpret_cast<const float2*>(sc + 8 * tau + 2 * q);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float dot = kLo ? (c0[e] + c1[e]) + (c0[2 + e] + c1[2 + e]) : c0[e] + c1[e];
          sf[2 * tau + e] = (e ? ks.y : ks.x) * factor;
          x[2 * tau + e] = dot;
        }
      }
      // ---- references
      float vs[4];
      *reinterpret_cast<float2*>(vs) = *reinterpret_cast<const float2*>(sc + kTile + 2 * q);
      *reinterpret_cast<float2*>(vs + 2) = *reinterpret_cast<const float2*>(sc + kTile + 8 + 2 * q);
      bool there[4];
      float mn = m, m2n = m2;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        there[i] = (mask >> (8 * (i >> 1) + 2 * q + (i & 1))) & 1u;
        const float up = there[i] ? ceilf(x[i] * sf[i]) : -INFINITY;
        mn = fmaxf(mn, up);
        // exponent of the value scale, rounded up, at least -112 so that 2^14 times its
        // reciprocal is finite
        m2n = fmaxf(m2n, up + float(max(int(__float_as_uint(vs[i]) >> 23) - 126, -112)));
      }
      if (a.scores != nullptr && (NT == 2 || gid < 4) && head_ok) {
        float* const o = a.scores + (unit * a.G + head) * a.score_stride + cur.ls * kStep +
                         warp * kTile + 2 * q;
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = there[i] ? x[i] * sf[i] : -INFINITY;
        *reinterpret_cast<float2*>(o) = make_float2(y[0], y[1]);
        *reinterpret_cast<float2*>(o + 8) = make_float2(y[2], y[3]);
      }
      mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 1));
      m2n = fmaxf(m2n, __shfl_xor_sync(0xffffffffu, m2n, 1));
      mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 2));
      m2n = fmaxf(m2n, __shfl_xor_sync(0xffffffffu, m2n, 2));
      if (__any_sync(0xffffffffu, mn > m || m2n > m2)) {
        l *= ref_change(m, mn);
        const float r = ref_change(m2, m2n);
        const float r0 = __shfl_sync(0xffffffffu, r, 8 * q);       // column 2 q
        const float r1 = __shfl_sync(0xffffffffu, r, 8 * q + 4);   // column 2 q + 1
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            acc[n][t][0] *= r0;
            acc[n][t][1] *= r1;
            acc[n][t][2] *= r0;
            acc[n][t][3] *= r1;
          }
        m = mn;
        m2 = m2n;
      }
      // w = 2^(x - m) c 2^(m - m2 + 14)
      const float lift = m2 == -INFINITY ? 1.0f : ex2(m - m2 + kWBias);
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = there[i] ? ex2(fmaf(x[i], sf[i], -m)) : 0.0f;
        l += p;
        w[i] = p * (vs[i] * lift);
      }
      uint32_t b0[NT], b1[NT];
      b0[0] = pack_f16(w[0], w[1]);
      b1[0] = pack_f16(w[2], w[3]);
      if constexpr (NT == 1) {
        if (gid >= 4) {   // columns 4..7: the low parts of heads 0..3
          b0[0] = pack_f16_rest(w[0], w[1], b0[0]);
          b1[0] = pack_f16_rest(w[2], w[3], b1[0]);
        }
      } else {
        b0[NT - 1] = pack_f16_rest(w[0], w[1], b0[0]);
        b1[NT - 1] = pack_f16_rest(w[2], w[3], b1[0]);
      }
      // ---- values: lane (gid, q): dimensions 16 gid .. + 15 of keys 2q, 2q+1, 8+2q, 9+2q
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * (i >> 1) + 2 * q + (i & 1);
        v[i] = *reinterpret_cast<const uint4*>(tile + (kTile + r) * kD + 16 * (gid ^ swz(r)));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t ka = i == 0 ? v[0].x : i == 1 ? v[0].y : i == 2 ? v[0].z : v[0].w;
        const uint32_t kb = i == 0 ? v[1].x : i == 1 ? v[1].y : i == 2 ? v[1].z : v[1].w;
        const uint32_t kc = i == 0 ? v[2].x : i == 1 ? v[2].y : i == 2 ? v[2].z : v[2].w;
        const uint32_t kd = i == 0 ? v[3].x : i == 1 ? v[3].y : i == 2 ? v[3].z : v[3].w;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t ab = __byte_perm(ka, kb, hf ? 0x7362 : 0x5140);
          const uint32_t cd = __byte_perm(kc, kd, hf ? 0x7362 : 0x5140);
          const uint32_t a0 = half2_of<FMT>(ab, 0), a1 = half2_of<FMT>(ab, 1);
          const uint32_t a2 = half2_of<FMT>(cd, 0), a3 = half2_of<FMT>(cd, 1);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(acc[n][2 * i + hf], a0, a1, a2, a3, b0[n], b1[n]);
        }
      }
    }
    if (mask == 0 && a.scores != nullptr && cur.ls * kStep + warp * kTile < cur.len) {
      // entries without a key (skipped, or a bad page) have no weight
      for (int i = lane; i < a.G * kTile; i += 32)
        a.scores[(unit * a.G + i / kTile) * a.score_stride + cur.ls * kStep + warp * kTile +
                 i % kTile] = -INFINITY;
    }
    __syncwarp();   // the tile's buffer is refilled by the next iteration
    if (++st == ST) st = 0;

    const bool unit_ends = cur.ls + 1 == cur.ns;
    if (unit_ends || s + 1 == s1) {
      // ---- merge the warps' states
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (q == 0 && (NT == 2 || gid < 4)) {
        sm.stat[warp][head][0] = m;
        sm.stat[warp][head][1] = l;
        sm.stat[warp][head][2] = m2;
      }
      __syncthreads();
      float M = -INFINITY, M2 = -INFINITY, Ls = 0.0f;
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) {
        M = fmaxf(M, sm.stat[w][head][0]);
        M2 = fmaxf(M2, sm.stat[w][head][2]);
      }
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) Ls += sm.stat[w][head][1] * ref_change(sm.stat[w][head][0], M);
      {
        const float r = ref_change(m2, M2);
        const float r0 = __shfl_sync(0xffffffffu, r, 8 * q);
        const float r1 = __shfl_sync(0xffffffffu, r, 8 * q + 4);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            acc[n][t][0] *= r0;
            acc[n][t][1] *= r1;
            acc[n][t][2] *= r0;
            acc[n][t][3] *= r1;
          }
      }
      // high and low parts together: NT = 1, lanes q and q ^ 2 hold the two parts of two
      // heads; each keeps half of the dimensions (value 4 t + i: tile t + 4 (q >> 1)).
      // NT = 2: both parts are in the lane (value 4 t + i: tile t).
      float val[S::kSums];
      if constexpr (NT == 1) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float keep = (q & 2) ? acc[0][t + 4][i] : acc[0][t][i];
            const float give = (q & 2) ? acc[0][t][i] : acc[0][t + 4][i];
            val[4 * t + i] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
          }
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) val[4 * t + i] = acc[0][t][i] + acc[NT - 1][t][i];
      }
#pragma unroll
      for (int h = kAtWarps / 2; h > 0; h >>= 1) {
        if (warp >= h && warp < 2 * h) {
#pragma unroll
          for (int i = 0; i < S::kSums; ++i) sm.sums[warp - h][i][lane] = val[i];
        }
        __syncthreads();
        if (warp < h) {
#pragma unroll
          for (int i = 0; i < S::kSums; ++i) val[i] += sm.sums[warp][i][lane];
        }
        __syncthreads();
      }
      // ---- the unit's parts: CTAs c0 .. c1 hold steps of it
      const long long u0 = s - cur.ls;                          // the unit's first step
      const int c0 = int(((u0 + 1) * C + T_all - 1) / T_all) - 1;
      const int c1 = int(((u0 + cur.ns) * C + T_all - 1) / T_all) - 1;
      const int parts = c1 - c0 + 1;
      const int cta = blockIdx.x;
      if (warp == 0) {
        // dimensions of this lane's values: 16 gid + d0 + 0..7 for NT = 1, + 0..15 for NT = 2;
        // head of column 2 (q or q & 1) + (i & 1)
        constexpr int kRun = S::kSums / 2;
        const int col = NT == 1 ? 2 * (q & 1) : 2 * q;
        const int dim = 16 * gid + (NT == 1 ? 8 * (q >> 1) : 0);
        if (parts == 1) {
          // factor of head `head`, held by the lanes of row gid = head
          const float f = Ls > 0.0f || !(Ls == Ls) ? ex2(M2 - M - kWBias) / Ls : 0.0f;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float fe = __shfl_sync(0xffffffffu, f, 4 * (col + e));
            if (col + e < a.G) {
              float* const o = a.out + (unit * a.G + col + e) * kD + dim;
#pragma unroll
              for (int d = 0; d < kRun; d += 4)
                *reinterpret_cast<float4*>(o + d) =
                    make_float4(val[2 * d + e] * fe, val[2 * d + 2 + e] * fe,
                                val[2 * d + 4 + e] * fe, val[2 * d + 6 + e] * fe);
            }
          }
          if (a.stats != nullptr && q == 0 && gid < a.G && (NT == 2 || gid < 4)) {
            float* const o = a.stats + (unit * a.G + gid) * 2;
            const bool some = Ls > 0.0f || !(Ls == Ls);
            o[0] = some ? M : 0.0f;
            o[1] = some ? 1.0f / Ls : 0.0f;
          }
        } else {
          // slot 0: the CTA's first unit, slot 1: its last when that is another one
          const int slot = 2 * cta + (u0 > s0 ? 1 : 0);
          float* const base = a.part + int64_t(slot) * a.G * kPart;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (col + e < a.G) {
              float* const o = base + (col + e) * kPart + 4 + dim;
#pragma unroll
              for (int d = 0; d < kRun; d += 4)
                *reinterpret_cast<float4*>(o + d) =
                    make_float4(val[2 * d + e], val[2 * d + 2 + e], val[2 * d + 4 + e],
                                val[2 * d + 6 + e]);
            }
          }
          if (q == 0 && gid < a.G && (NT == 2 || gid < 4)) {
            float* const o = base + gid * kPart;
            o[0] = M;
            o[1] = Ls;
            o[2] = M2;
          }
          __threadfence();
          __syncwarp();
          if (lane == 0)
            sm.last = atomicAdd(a.count + unit, 1u) + 1u == uint32_t(parts) ? 1 : 0;
        }
      }
      if (parts > 1) {
        __syncthreads();
        if (sm.last) {
          __threadfence();
          const auto slot_of = [&](int p) {
            const int c = c0 + p;
            return 2 * c + (p == 0 && T_all * c / C < u0 ? 1 : 0);
          };
          if (warp < a.G) {   // head `warp`: references and the sum of weights
            float hM = -INFINITY, hM2 = -INFINITY;
            for (int p = lane; p < parts; p += 32) {
              const float* const o = a.part + (int64_t(slot_of(p)) * a.G + warp) * kPart;
              hM = fmaxf(hM, __ldcg(o));
              hM2 = fmaxf(hM2, __ldcg(o + 2));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
              hM = fmaxf(hM, __shfl_xor_sync(0xffffffffu, hM, o));
              hM2 = fmaxf(hM2, __shfl_xor_sync(0xffffffffu, hM2, o));
            }
            float hl = 0.0f;
            for (int p = lane; p < parts; p += 32) {
              const float* const o = a.part + (int64_t(slot_of(p)) * a.G + warp) * kPart;
              hl += __ldcg(o + 1) * ref_change(__ldcg(o), hM);
            }
            hl = warp_sum(hl);
            if (lane == 0) {
              const bool some = hl > 0.0f || !(hl == hl);
              sm.fin[warp][0] = hM2;
              sm.fin[warp][1] = some ? ex2(hM2 - hM - kWBias) / hl : 0.0f;
              if (a.stats != nullptr) {
                float* const o = a.stats + (unit * a.G + warp) * 2;
                o[0] = some ? hM : 0.0f;
                o[1] = some ? 1.0f / hl : 0.0f;
              }
            }
          }
          __syncthreads();
          // sums: thread = (part group, head, 4 dimensions)
          const int cols = a.G * (kD / 4);
          const int groups = kAtThreads / cols;
          const int gr = tid / cols, ci = tid % cols;
          const int hh = ci / (kD / 4), d4 = ci % (kD / 4);
          float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
          if (gr < groups) {
            const float hM2 = sm.fin[hh][0];
#pragma unroll 4
            for (int p = gr; p < parts; p += groups) {
              const float* const o = a.part + (int64_t(slot_of(p)) * a.G + hh) * kPart;
              const float f = ref_change(__ldcg(o + 2), hM2);
              const float4 y = __ldcg(reinterpret_cast<const float4*>(o + 4) + d4);
              t.x = fmaf(y.x, f, t.x);
              t.y = fmaf(y.y, f, t.y);
              t.z = fmaf(y.z, f, t.z);
              t.w = fmaf(y.w, f, t.w);
            }
          }
          float4* const scratch = reinterpret_cast<float4*>(&sm.sums[0][0][0]);
          if (gr < groups) scratch[tid] = t;
          __syncthreads();
          if (gr == 0) {
            for (int g = 1; g < groups; ++g) {
              const float4 y = scratch[g * cols + ci];
              t.x += y.x;
              t.y += y.y;
              t.z += y.z;
              t.w += y.w;
            }
            const float f = sm.fin[hh][1];
            reinterpret_cast<float4*>(a.out + (unit * a.G + hh) * kD)[d4] =
                make_float4(t.x * f, t.y * f, t.z * f, t.w * f);
          }
          if (tid == 0) a.count[unit] = 0u;
        }
        __syncthreads();   // sm.last and the scratch are free again
      }
      fresh = true;
    }
    if (s + 1 < s1) next_place(a, cur);
  }
}

// ------------------------------------------------------------- attention weights
// Dense: w_out[unit][j] = w_in[unit][j] + sum_g 2^(x_gj - M_g) / l_g, from the scores the
// attention kernel left in the workspace (4 G bytes per key written and read against 128 G
// if K were scored again).
constexpr int kWPer = 4;

__global__ void __launch_bounds__(256) kv8_weights_kernel(
    const float* __restrict__ scores, int64_t score_stride, const float* __restrict__ stats,
    const int32_t* __restrict__ seq_lens, int Hkv, int G, int64_t Lmax, int tiles,
    const float* w_in, float* w_out, uint32_t* err) {
  pdl_wait();
  pdl_trigger();
  const int64_t unit = blockIdx.x / tiles;
  const int64_t j0 = int64_t(blockIdx.x % tiles) * (256 * kWPer) + threadIdx.x;
  const int64_t len =
      seq_lens == nullptr ? Lmax : checked_len(seq_lens[unit / Hkv], Lmax, err, false);
  // the heads' weights are summed first: the (larger) running sum is rounded once
  float in[kWPer], s[kWPer];
#pragma unroll
  for (int u = 0; u < kWPer; ++u) {
    const int64_t j = j0 + u * 256;
    in[u] = j < len ? w_in[unit * Lmax + j] : 0.0f;
    s[u] = 0.0f;
  }
  for (int g = 0; g < G; ++g) {
    const float M = __ldg(stats + (unit * G + g) * 2), inv = __ldg(stats + (unit * G + g) * 2 + 1);
    const float* const x = scores + (unit * G + g) * score_stride;
#pragma unroll
    for (int u = 0; u < kWPer; ++u) {
      const int64_t j = j0 + u * 256;
      if (j < len) s[u] = fmaf(ex2(__ldcs(x + j) - M), inv, s[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < kWPer; ++u) {
    const int64_t j = j0 + u * 256;
    if (j < len) w_out[unit * Lmax + j] = in[u] + s[u];
  }
}

// Sparse: a CTA owns kSlice consecutive positions of one (b, kv head) and walks through the
// lists of its heads one after another, adding the weights that fall into its slice in
// shared memory; a list without repeats adds at most once per position and head, so the
// order of the sums does not depend on timing.
constexpr int kSlice = 8192;

__global__ void __launch_bounds__(512) kv8_sparse_weights_kernel(
    const int32_t* __restrict__ idx, int k, const float* __restrict__ scores,
    int64_t score_stride, const float* __restrict__ stats, int lists, int G, int64_t Lmax,
    int slices, const float* w_in, float* w_out) {
  extern __shared__ float sum[];
  pdl_wait();
  pdl_trigger();
  const int64_t unit = blockIdx.x / slices;                     // (b, kv head)
  const int64_t base = int64_t(blockIdx.x % slices) * kSlice;
  const int n = int(min(int64_t(kSlice), Lmax - base));
  for (int i = threadIdx.x; i < n; i += 512) sum[i] = 0.0f;
  __syncthreads();
  // `lists` lists (G per-head ones, or one for all G heads)
  for (int li = 0; li < lists; ++li) {
    const int32_t* const list = idx + (unit * lists + li) * k;
    for (int i = threadIdx.x; i < k; i += 512) {
      const int64_t p = int64_t(list[i]) - base;
      if (list[i] >= 0 && p >= 0 && p < n) {
        float w = 0.0f;
        const int heads = G / lists;
        for (int g = 0; g < heads; ++g) {
          const int64_t r = unit * G + li * heads + g;
          w = fmaf(ex2(scores[r * score_stride + i] - __ldg(stats + 2 * r)), __ldg(stats + 2 * r + 1),
                   w);
        }
        atomicAdd(&sum[p], w);
      }
    }
    __syncthreads();
  }
  const float* const in = w_in + unit * Lmax + base;
  float* const out = w_out + unit * Lmax + base;
  for (int i = threadIdx.x; i < n; i += 512) {
    const float x = sum[i];
    if (in != out || x != 0.0f) out[i] = in[i] + x;
  }
}

constexpr int kStages1 = 3;   // G <= 4: two CTAs of 8 warps per SM
constexpr int kStages2 = 3;

// CTAs of the attention kernel: the co-resident ones, no more than there can be steps.
int attention_ctas(int G, int64_t units, int64_t len, int sms) {
  const int64_t steps = units * ((len + kStep - 1) / kStep);
  const int64_t room = int64_t(sms) * (G <= 4 ? 2 : 1);
  return int(steps < room ? steps : room);
}

struct Room {
  size_t count, part, stats, scores, total;
  int64_t stride;
};
Room workspace_room(int B, int Hq, int Hkv, int64_t Lmax, int k, bool shared, bool weights) {
  const bool sparse = k > 0;
  const int64_t U = sparse && !shared ? Hq : Hkv;
  const int G = int(Hq / U);
  Room r;
  r.count = 256;
  r.part = r.count + align_up(size_t(B) * U * 4, 256);
  const int ctas = attention_ctas(G, B * U, sparse ? k : Lmax, device_sms());
  r.stats = r.part + align_up(size_t(ctas) * 2 * G * kPart * 4, 256);
  r.scores = r.stats + (weights ? align_up(size_t(B) * Hq * 8, 256) : 0);
  // rows padded to whole warp tiles: the kernel stores scores tile by tile
  r.stride = ((sparse ? int64_t(k) : Lmax) + kTile - 1) / kTile * kTile;
  r.total = r.scores + (weights ? align_up(size_t(B) * Hq * size_t(r.stride) * 4, 256) : 0);
  return r;
}

template <typename T, int FMT, int NT, int ST, int MB>
cudaError_t run_attention(const Args& a, int ctas, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const auto kernel = kv8_attention_kernel<T, FMT, NT, ST, MB>;
  const int bytes = int(sizeof(Smem<NT, ST>));
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), bytes, done, false);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kAtThreads);
  cfg.dynamicSmemBytes = size_t(bytes);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T, int FMT>
cudaError_t run_attention_g(const Args& a, int ctas, cudaStream_t stream) {
  if (a.G <= 4) return run_attention<T, FMT, 1, kStages1, 2>(a, ctas, stream);
  return run_attention<T, FMT, 2, kStages2, 1>(a, ctas, stream);
}

}  // namespace

size_t kv8_attention_workspace(int B, int Hq, int Hkv, int64_t Lmax, int k, bool shared,
                               bool weights) {
  return workspace_room(B, Hq, Hkv, Lmax, k, shared, weights).total;
}

cudaError_t launch_kv8_attention(const Kv8& c, int fmt, const void* q, adamas_dtype dt, int Hq,
                                 const int32_t* seq_lens, const int32_t* idx, int k, bool shared,
                                 void* ws, const float* w_in, float* w_out, float* out,
                                 cudaStream_t stream) {
  const bool weights = w_out != nullptr;
  const Room r = workspace_room(c.B, Hq, c.Hkv, c.Lmax, idx ? k : 0, shared, weights);
  uint8_t* const base = static_cast<uint8_t*>(ws);
  Args a = {};
  a.c = c;
  a.q = q;
  a.seq_lens = idx ? nullptr : seq_lens;
  a.idx = idx;
  a.out = out;
  a.err = reinterpret_cast<uint32_t*>(base + decode_workspace_error_offset());
  a.count = reinterpret_cast<uint32_t*>(base + r.count);
  a.part = reinterpret_cast<float*>(base + r.part);
  a.stats = weights ? reinterpret_cast<float*>(base + r.stats) : nullptr;
  a.scores = weights ? reinterpret_cast<float*>(base + r.scores) : nullptr;
  a.score_stride = r.stride;
  a.scale_log2 = float(1.4426950408889634 / 11.313708498984761);
  a.U = idx && !shared ? Hq : c.Hkv;
  a.G = Hq / a.U;
  a.heads_per_kv = a.U / c.Hkv;
  a.k = k;
  const int ctas = attention_ctas(a.G, int64_t(c.B) * a.U, idx ? k : c.Lmax, device_sms());
  cudaError_t e;
  if (dt == ADAMAS_BF16)
    e = fmt == kFmtE4m3 ? run_attention_g<__nv_bfloat16, kFmtE4m3>(a, ctas, stream)
                        : run_attention_g<__nv_bfloat16, kFmtInt8>(a, ctas, stream);
  else
    e = fmt == kFmtE4m3 ? run_attention_g<float, kFmtE4m3>(a, ctas, stream)
                        : run_attention_g<float, kFmtInt8>(a, ctas, stream);
  if (e != cudaSuccess || !weights) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int64_t units = int64_t(c.B) * c.Hkv;
  const int G = Hq / c.Hkv;
  if (idx == nullptr) {
    const int64_t tiles = (c.Lmax + 256 * kWPer - 1) / (256 * kWPer);
    if (units * tiles > INT32_MAX) return cudaErrorInvalidValue;
    cfg.gridDim = dim3(unsigned(units * tiles));
    cfg.blockDim = dim3(256);
    return cudaLaunchKernelEx(&cfg, kv8_weights_kernel, static_cast<const float*>(a.scores),
                              a.score_stride, static_cast<const float*>(a.stats), seq_lens, c.Hkv,
                              G, c.Lmax, int(tiles), w_in, w_out, a.err);
  }
  const int64_t slices = (c.Lmax + kSlice - 1) / kSlice;
  if (units * slices > INT32_MAX) return cudaErrorInvalidValue;
  cfg.gridDim = dim3(unsigned(units * slices));
  cfg.blockDim = dim3(512);
  cfg.dynamicSmemBytes = size_t(kSlice) * 4;
  return cudaLaunchKernelEx(&cfg, kv8_sparse_weights_kernel, idx, k,
                            static_cast<const float*>(a.scores), a.score_stride,
                            static_cast<const float*>(a.stats), shared ? 1 : G, G, c.Lmax,
                            int(slices), w_in, w_out);
}

}  // namespace adamas
