// Single-token attention over an 8-bit cache: dense (every position of a sequence) or
// sparse (given positions), one kernel, plus the pass that adds attention weights to a
// running sum.
//
// Mathematics.  For a unit (a kv head with its G query heads; in the per-head sparse form
// one query head) and its list of keys j with bytes k_j, v_j and scales a_j, c_j:
//   x_j = (q . k_j) a_j log2(e) / sqrt(d),  out = sum_j 2^(x_j - M) c_j v_j / sum_j 2^(x_j - M).
// One pass over the keys with running references instead of maxima: m is an INTEGER at or
// above every x_j seen (so 2^(x - m) is formed by one fused multiply-add and every change
// of reference, in a warp or between partial results, is an exact power of two), and the
// integer r bounds x_j - m + log2 c_j the same way for the value sum, whose terms
// w_j = 2^(x_j - m - r) c_j then lie in [0, 1] whatever the scales are.  r is relative to m, since a
// sum m + r of a large m would lose r's last bits.
//
// The work is 256 bytes of cache per key against 4 G d operations: HBM bounds it.  The
// tensor cores (mma.m16n8k16, fp16 operands, fp32 sums) keep the arithmetic out of the
// way; a byte of either format is exact in fp16.  q and w_j are split into two fp16 parts (a bf16
// q takes one), scaled by powers of two so that a head's largest |q| lies in [2^14, 2^15) and its
// largest w in (2^12, 2^14]; each sum takes both parts.  The parts hold 2^-22 of a value, and
// never less than fp16's half step 2^-25: an element of q is off by at most 2^-22 of itself
// or 2^-39 of its head's largest, a product p_j c_j by 2^-22 of itself or 2^-37 of its
// head's largest.  So what a block adds to a dimension loses bits where another block's p c is
// 2^15 and more times larger, and shows only if that block holds zeros there.  Three parts,
// or bf16 ones (no conversion from e4m3), would cost registers that the loop does not have.
//   scores: A = q (16 rows: 8 head rows, high parts; 8 rows of low parts), B = K^T.
//   values: A = V^T (16 dimensions x 16 keys), B = w^T (16 keys x 8 columns).
// The score fragment a lane gets (its head row, keys 2q, 2q+1 of two 8-key tiles) is the
// B fragment it needs for the values, so nothing is exchanged between the products.  The
// order of dimensions inside a product is free: a lane takes 16 contiguous bytes of a K
// row per load, and 16 contiguous dimensions of a V row (its outputs), pairs of keys
// interleaved by byte permutes.  With G <= 4 (NT = 1) the 8 columns hold the high and the low
// parts of w for four heads (head rows repeated); with G <= 8 (NT = 2) each product is taken
// twice, with the high and with the low parts.
//
// Layout of the work.  A step is 128 keys of a unit: 32 per warp, 4 warps.  The steps of all
// units form one line (with kUnitCost places more per unit, for what its start and its merge cost)
// that is cut evenly over the CTAs; lengths are read on the device, so unequal sequences balance;
// a CTA's cut may hold the end of one unit, whole units and the start of another.  At a unit's end
// the warps' states are merged; a unit cut between CTAs leaves its parts in the workspace, and a
// second kernel, which is launched early and waits, merges them in CTA order.
//
// kUni: 16 rows of a tile follow one another and share one scale (contiguous caches and pages of
// at least 16 rows, blocks of at least 16 positions).  Each lane loads the 16-byte pieces of K and
// V rows that its fragments need straight into registers: a tile's K registers are refilled (with
// the next tile, of the next unit if need be) as soon as its scores are formed, the V registers
// after its value product, so 8 KB per warp stay under way through the rest of the work, and the
// tile behind it has been asked into L2.
// Otherwise (given positions, small pages or blocks) rows and scales are looked up key by key, three
// tiles ahead, and the rows come by cp.async through a ring of three tiles per warp: a tile has a
// whole tile's time more to arrive, and a row's address is formed once instead of by every lane
// that holds a piece of it (8 sequences x 32 lists of 1024 keys: 22 us; straight into registers 25.6).
//
// Measured, e4m3 and bf16 queries: 32 kv heads x 128K keys 187 us in single passes (1.074 GB, 5.7
// TB/s of the 6.55 that a copy reaches), 197 with running sums (1.108 GB); call after call, when the
// card sits at its power limit, 206 to 214 with sums.  8 kv heads x 32K keys, 4 query heads each,
// 19.5 us (3.4 TB/s: about 8 us go to the launches, the first loads and the merges, which 1000 keys take
// as well: 8.2 us).  Of the register-path variants the one for bf16 queries, e4m3 and G <= 4 spills
// nothing, the others 12 to 72 bytes; the ring variants nothing.
#include <type_traits>

#include "kv8_internal.cuh"

namespace adamas {

namespace {

constexpr int kWarps = 4;                        // two CTAs per SM: up to 255 registers a thread
constexpr int kCtasPerSm = 2;
constexpr int kThr = kWarps * 32;
constexpr int kTile = 32;                        // keys per warp and step, in two halves of 16
constexpr int kStep = kWarps * kTile;            // keys per step
constexpr int kUnitCost = 1;                     // steps that a unit's start and merge take as long as
constexpr int kStages = 3;                       // tiles of a warp's ring (gathered keys)
constexpr int kStage = 2 * kTile * kD;            // bytes: K rows, then V rows
constexpr int kMaxParts = 512;                   // CTAs, and so parts of a unit
constexpr float kWBias = 14.0f;                  // w is held times 2^14
constexpr int kPart = 4 + kD;                    // floats of a partial: m, l, r, 0, sums

// Shared memory of a CTA.
template <int NT>
struct Smem {
  static constexpr int kSums = NT == 1 ? 16 : 32;   // values per lane when warps are merged
  float sums[kWarps][kSums][32];                    // merge of the warps
  float stat[kWarps][8][4];                         // m, l, r per warp and head
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
  int4* cuts;               // [CTAs]: the unit that ends behind this CTA: unit (2 words), parts,
                            // which of them this CTA's is (0: the unit begins here)
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

// the first product of a chain: no sum to add to
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
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

// How far reference m lies below the common one M >= m (0 if equal, also where both are -inf).
__device__ __forceinline__ float ref_step(float m, float M) { return m == M ? 0.0f : m - M; }

// The references (m, r) of two sets of terms become those of both: r is relative to m.
__device__ __forceinline__ void ref_join(float& m, float& r, float m1, float r1) {
  const float top = fmaxf(m, m1);
  r = fmaxf(r + ref_step(m, top), r1 + ref_step(m1, top));
  m = top;
}

// What turns a head's value sum t into its output t 2^(r - 14) / l, in two factors: with small value
// scales r is as low as -126, and the whole factor below fp32's normal numbers although t times
// it may not.  The second is 1 but for exponents below -100.
struct OutScale {
  float f, g;
  __device__ __forceinline__ OutScale(float r, float l, bool some) {
    const float e = r - kWBias, e1 = fmaxf(e, -100.0f);
    f = some ? ex2(e1) / l : 0.0f;
    g = some ? ex2(e - e1) : 0.0f;
  }
  __device__ __forceinline__ float4 of(float a, float b, float c, float d) const {
    return make_float4(a * f * g, b * f * g, c * f * g, d * f * g);
  }
};

// 16 bytes that are read once (kept out of L1); zeros if !ok (nothing is read then).
__device__ __forceinline__ uint4 load_row16(const uint8_t* p, bool ok = true) {
  uint4 v;
  if (!ok)
    v = make_uint4(0u, 0u, 0u, 0u);
  else
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
  return v;
}

// cp.async that fills with zeros when !ok (nothing is read then)
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}

// 16-byte chunk ch of row r of a ring's tile is stored at chunk ch ^ swz(r): the 8 lanes of a
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

// One step's place: unit (b, j), its step ls of ns.
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

// This warp's tile at a place, found in three stages an iteration apart, because each may wait
// for a load: the positions (given lists), the pages (block tables), the rows.
struct Tile {
  int b, j, i0, n;      // unit, first key, keys (0 .. 32)
  int pos;              // lane i: key i's position
  int page[2];          // kUni: of each half; else lane i: key i's, in [0]
};
// A cache has fewer than 2^31 rows, so a row index is an int.  kUni: the row of the first key of
// each half, in every lane; else lane i holds key i's row.  mask: which of the keys are there.
struct Rows {
  int row[2];
  uint32_t mask;
  float ks, vs;         // !kUni: the scales of key i in lane i
};

__device__ __forceinline__ Tile no_tile() { return Tile{0, 0, 0, 0, -1, {0, 0}}; }

template <bool kUni>
__device__ __forceinline__ Tile tile_positions(const Args& a, const Place& p, int warp, int lane) {
  Tile t;
  t.b = p.b;
  t.j = p.j;
  t.i0 = p.ls * kStep + warp * kTile;
  t.n = max(0, min(kTile, p.len - t.i0));
  t.pos = -1;
  t.page[0] = t.page[1] = 0;
  if constexpr (!kUni) {
    if (lane < t.n)
      t.pos = a.idx != nullptr ? a.idx[(int64_t(p.b) * a.U + p.j) * a.k + t.i0 + lane]
                               : t.i0 + lane;
  }
  return t;
}

template <bool kUni>
__device__ __forceinline__ void tile_pages(const Args& a, Tile& t) {
  if (a.c.table == nullptr) return;
  const int32_t* const table = a.c.table + int64_t(t.b) * a.c.max_blocks;
  if constexpr (kUni) {
    if (t.n > 0) t.page[0] = table[t.i0 >> a.c.page_shift];
    if (t.n > 16) t.page[1] = table[(t.i0 + 16) >> a.c.page_shift];
  } else {
    if (t.pos >= 0 && t.pos < a.c.Lmax) t.page[0] = table[t.pos >> a.c.page_shift];
  }
}

template <bool kUni>
__device__ __forceinline__ Rows tile_rows(const Args& a, const Tile& t) {
  Rows r;
  r.row[0] = r.row[1] = -1;
  r.ks = r.vs = 0.0f;
  r.mask = t.n >= 32 ? 0xffffffffu : (1u << t.n) - 1u;
  if constexpr (kUni) {
    if (a.c.table == nullptr) {
      r.row[0] = (t.b * a.c.Hkv + t.j) * int(a.c.Lmax) + t.i0;
      r.row[1] = r.row[0] + 16;
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (t.page[u] < 0 || t.page[u] >= a.c.num_pages) {
          if (t.n > 16 * u) atomicOr(a.err, kErrInput);
          r.mask &= u ? 0x0000ffffu : 0xffff0000u;
        } else {
          r.row[u] = ((t.page[u] * a.c.Hkv + t.j) << a.c.page_shift) +
                     ((t.i0 + 16 * u) & ((1 << a.c.page_shift) - 1));
        }
      }
    }
  } else {
    if (t.pos >= 0) {
      const int h = t.j / a.heads_per_kv;
      if (t.pos >= a.c.Lmax || t.page[0] < 0 || t.page[0] >= (a.c.table ? a.c.num_pages : 1))
        atomicOr(a.err, kErrInput);
      else if (a.c.table == nullptr)
        r.row[0] = (t.b * a.c.Hkv + h) * int(a.c.Lmax) + t.pos;
      else
        r.row[0] = ((t.page[0] * a.c.Hkv + h) << a.c.page_shift) +
                   (t.pos & ((1 << a.c.page_shift) - 1));
    }
    r.mask = __ballot_sync(0xffffffffu, r.row[0] >= 0);
    r.ks = r.row[0] >= 0 ? __ldg(a.c.ks + (r.row[0] >> a.c.bshift)) : 0.0f;
    r.vs = r.row[0] >= 0 ? __ldg(a.c.vs + (r.row[0] >> a.c.bshift)) : 0.0f;
  }
  return r;
}

// The query rows of a unit.  Lane (gid, q) holds head row gid: elements 4 i .. 4 i + 3 of its
// 16-dimension runs (chunk c: dimensions 64 (c / 4) + 16 q + 4 (c % 4) + 0..3).
template <typename T>
struct QueryRow {
  typename Raw4<T>::type raw[8];
  __device__ __forceinline__ void load(const void* base, int64_t row, bool exists, int q) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      raw[c] = {};
      if (exists)
        raw[c] = Raw4<T>::load(static_cast<const T*>(base) + row * kD, 16 * (c >> 2) + 4 * q + (c & 3));
    }
  }
};

// The rows as A fragments, scaled by 2^-e so that the head's largest element lies in
// [1, 2) x 2^14; the returned factor undoes it: x = dot * a_j * factor.
template <typename T, bool kLo>
__device__ __forceinline__ float query_fragments(const QueryRow<T>& qr, float scale_log2,
                                                 uint32_t (&hi)[8][2],
                                                 uint32_t (&lo)[kLo ? 8 : 1][2]) {
  float mx = 0.0f;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    float v[4];
    Raw4<T>::decode(qr.raw[c], v);
#pragma unroll
    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fabsf(v[i]));
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  // exponent of the largest element, at least -98 (zero rows, all but denormal ones), so
  // that both powers of two are normal; infinities stay infinite
  const int e = max(int(__float_as_uint(mx) >> 23) - 127, -98);
  const float down = pow2i(14 - e);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    float v[4];
    Raw4<T>::decode(qr.raw[c], v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= down;
    hi[c][0] = pack_f16(v[0], v[1]);
    hi[c][1] = pack_f16(v[2], v[3]);
    if constexpr (kLo) {
      lo[c][0] = pack_f16_rest(v[0], v[1], hi[c][0]);
      lo[c][1] = pack_f16_rest(v[2], v[3], hi[c][1]);
    }
  }
  return scale_log2 * pow2i(e - 14);
}

// The even cut of a line over C CTAs, in grains (places, or whole units): the first CTAs take one
// grain more where it does not come out even.
struct Cut {
  int q, r, grain;
  __device__ __forceinline__ int start(int c) const { return (c * q + min(c, r)) * grain; }
  __device__ __forceinline__ int owner(int place) const {
    const int s = grain == 1 ? place : place / grain;
    const int wide = r * (q + 1);
    return s < wide ? s / (q + 1) : r + (s - wide) / q;
  }
};

// Whole units per CTA (equal units only) where that keeps 3 in 4 CTAs busy, since a unit in one piece
// needs no second merge: 256 lists of 1024 positions on 296 CTAs take 22.0 us, cut evenly 24.6.
// 0: cut evenly.
__host__ __device__ inline int whole_units(int units, int steps_per_unit, int grid) {
  const int each = (units + grid - 1) / grid;
  const bool few = int64_t(units) * steps_per_unit <= grid;
  return !few && int64_t(units) * 4 >= int64_t(each) * grid * 3 ? each : 0;
}

// Merges the parts (in CTA order) of the units that were cut; block c looks at what CTA c left.  A
// unit of at most kFewParts parts is merged by the block of its first CTA, a warp per head; of one in more
// (so cut into at least a first, 7 inner and a last part) the block of part h takes head h, thread p
// finding part p's reference before warp w sums parts w, w + 8, ..., 4 dimensions per lane.  So one
// long sequence among many short ones is not left to a warp.  (With blocks for all heads of every CTA
// one sequence of 1000 keys took 0.5 us more and one of 32K 0.2.)  The launch bound of 2 blocks is for
// the 80 registers that hold a warp's 8 parts at once: left to itself the compiler took 64 and two
// rounds of loads, 6.3 us instead of 5.6 by itself.
constexpr int kCombineThreads = 256, kFewParts = 8;

__global__ void __launch_bounds__(kCombineThreads, 2) kv8_combine_kernel(
    const int4* __restrict__ cuts, const float* __restrict__ part, int G, float* __restrict__ stats,
    float* __restrict__ out) {
  constexpr int kBatch = 10, kW = kCombineThreads / 32;
  __shared__ float ref[kMaxParts];
  __shared__ float red[3][kW];
  __shared__ float4 sums[kW][32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int4 cut = cuts[blockIdx.x];
  const int parts = cut.z;
  const bool by_warp = parts <= kFewParts;
  if (parts < 2 || (by_warp ? cut.w != 0 || warp >= G : cut.w >= G)) return;
  const int h = by_warp ? warp : cut.w, c = blockIdx.x - cut.w;
  const int64_t unit = (int64_t(uint32_t(cut.y)) << 32) | uint32_t(cut.x);
  const auto finish = [&](float l, float M, float R, const float4& t) {
    const bool some = l > 0.0f || !(l == l);   // an empty list: zeros
    reinterpret_cast<float4*>(out + (unit * G + h) * kD)[lane] =
        OutScale(R, l, some).of(t.x, t.y, t.z, t.w);
    if (stats != nullptr && lane == 0) {
      float* const o = stats + (unit * G + h) * 2;
      o[0] = some ? M : 0.0f;
      o[1] = some ? 1.0f / l : 0.0f;
    }
  };
  // a CTA's slot 1 holds the part of a unit that begins there, slot 0 that of one that goes on
  const auto at = [&](int p) {
    return reinterpret_cast<const float4*>(
        part + (int64_t(2 * (c + p) + (p == 0 ? 1 : 0)) * G + h) * kPart);
  };
  if (by_warp) {
    float4 w[kFewParts], y[kFewParts];
#pragma unroll
    for (int p = 0; p < kFewParts; ++p) {
      const bool ok = p < parts;
      w[p] = ok ? __ldcg(at(p)) : make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
      y[p] = ok ? __ldcg(at(p) + 1 + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float M = -INFINITY, R = -INFINITY, l = 0.0f;
#pragma unroll
    for (int p = 0; p < kFewParts; ++p) M = fmaxf(M, w[p].x);
#pragma unroll
    for (int p = 0; p < kFewParts; ++p) R = fmaxf(R, w[p].z + ref_step(w[p].x, M));
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 0; p < kFewParts; ++p) {
      const float step = ref_step(w[p].x, M);
      l += w[p].y * ex2(step);
      const float f = ref_change(w[p].z + step, R);
      t.x = fmaf(y[p].x, f, t.x);
      t.y = fmaf(y[p].y, f, t.y);
      t.z = fmaf(y[p].z, f, t.z);
      t.w = fmaf(y[p].w, f, t.w);
    }
    finish(l, M, R, t);
    return;
  }
  float4 y[kBatch];
  const auto load = [&](int p0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int p = p0 + u * kW;
      y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p < parts) y[u] = __ldcg(at(p) + 1 + lane);
    }
  };
  load(warp);   // under way while the references are found
  constexpr int kSt = (kMaxParts + kCombineThreads - 1) / kCombineThreads;
  float M = -INFINITY, R = -INFINITY;
  float4 st[kSt];
#pragma unroll
  for (int i = 0; i < kSt; ++i) {
    const int p = tid + i * kCombineThreads;
    st[i] = make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
    if (p < parts) st[i] = __ldcg(at(p));
    M = fmaxf(M, st[i].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) red[0][warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kW; ++w) M = fmaxf(M, red[0][w]);
  float l = 0.0f;
#pragma unroll
  for (int i = 0; i < kSt; ++i) {
    const int p = tid + i * kCombineThreads;
    const float step = ref_step(st[i].x, M), r = st[i].z + step;
    l += st[i].y * ex2(step);
    R = fmaxf(R, r);
    if (p < parts) ref[p] = r;
  }
  l = warp_sum(l);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) R = fmaxf(R, __shfl_xor_sync(0xffffffffu, R, o));
  if (lane == 0) {
    red[1][warp] = R;
    red[2][warp] = l;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kW; ++w) R = fmaxf(R, red[1][w]);
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = warp; p0 < parts; p0 += kBatch * kW) {
    if (p0 != warp) load(p0);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int p = p0 + u * kW;
      if (p < parts) {
        const float f = ref_change(ref[p], R);
        t.x = fmaf(y[u].x, f, t.x);
        t.y = fmaf(y[u].y, f, t.y);
        t.z = fmaf(y[u].z, f, t.z);
        t.w = fmaf(y[u].w, f, t.w);
      }
    }
  }
  sums[warp][lane] = t;
  __syncthreads();
  if (warp != 0) return;
  l = red[2][0];
  t = sums[0][lane];
#pragma unroll
  for (int w = 1; w < kW; ++w) {
    const float4 x = sums[w][lane];
    l += red[2][w];
    t.x += x.x;
    t.y += x.y;
    t.z += x.z;
    t.w += x.w;
  }
  finish(l, M, R, t);
}

// FMT: byte format; NT: value products per 16 keys (1: G <= 4, 2: G <= 8).
template <typename T, int FMT, int NT, bool kUni>
__global__ void __launch_bounds__(kThr, kCtasPerSm) kv8_attention_kernel(const Args a) {
  constexpr bool kLo = sizeof(T) == 4;   // fp32 queries take two fp16 parts
  using S = Smem<NT>;
  __shared__ __align__(16) S sm;
  extern __shared__ __align__(128) uint8_t ring[];   // !kUni: [kWarps][kStages][kStage]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, q = lane & 3;
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's part [x0, x1) of the line: per unit `cost` places that stand for its start and
  // merge, then its steps
  int x0, x1, cost;
  Cut cut;
  Place pf;
  const auto cut_over = [&](int grains, int ctas) {
    const int C = min(ctas, grains);
    cut.q = C > 0 ? grains / C : 0;
    cut.r = grains - cut.q * C;
    const int cta = min(int(blockIdx.x), C);
    x0 = cut.start(cta);
    x1 = cut.start(min(cta + 1, C));
  };
  const int grid = int(gridDim.x);
  int v = 0;   // place of the current step
  // the first step at or after place x0 of a sequence of `len` keys whose first unit is at `base`
  const auto begin = [&](int b, int len, int base) {
    pf.b = b;
    pf.len = len;
    pf.ns = steps_of(len);
    const int r = x0 - base, per = pf.ns + cost;
    pf.j = r / per;
    pf.ls = max(r - pf.j * per - cost, 0);
    v = base + pf.j * per + cost + pf.ls;
  };
  cut.grain = 1;
  if (a.idx != nullptr || a.seq_lens == nullptr) {
    const int len = unit_len(a, 0, false), ns = steps_of(len), units = a.c.B * a.U;
    // fewer steps than CTAs: one each, and no places for starts and merges
    cost = units * ns > grid ? kUnitCost : 0;
    const int each = whole_units(units, ns, grid);
    if (each > 0) {
      cut.grain = ns + cost;
      cut_over(units, (units + each - 1) / each);
    } else {
      cut_over(units * (ns + cost), cost > 0 ? grid : units * ns);
    }
    const int per = a.U * (ns + cost), b = x0 / per;
    begin(b, len, b * per);
  } else {
    // every warp for itself: lane l sums sequences l, l + 32, ..., then prefix sums over 32
    // sequences at a time find the one that holds place x0
    int mine = 0, some = 0;
    for (int b = lane; b < a.c.B; b += 32) {
      const int n = steps_of(unit_len(a, b, blockIdx.x == 0 && warp == 0));
      mine += n;
      some += n > 0;
    }
    const int steps = __reduce_add_sync(0xffffffffu, mine) * a.U;
    cost = steps > grid ? kUnitCost : 0;
    cut_over(steps + cost * __reduce_add_sync(0xffffffffu, some) * a.U, cost > 0 ? grid : steps);
    int before = 0;
    for (int b0 = 0; x0 < x1; b0 += 32) {
      const int b = b0 + lane;
      const int full = b < a.c.B ? unit_len(a, b, false) : 0;
      const int ns = steps_of(full);
      const int n = ns > 0 ? (ns + cost) * a.U : 0;
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + inc > x0);
      if (hit) {
        const int at = __ffs(hit) - 1;
        begin(b0 + at, __shfl_sync(0xffffffffu, full, at),
              before + __shfl_sync(0xffffffffu, inc - n, at));
        break;
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
    // sequences of length zero: their outputs are zero
    for (int b = blockIdx.x; b < a.c.B; b += gridDim.x) {
      if (unit_len(a, b, false) != 0) continue;
      for (int i = tid; i < a.U * a.G * kD; i += kThr)
        a.out[int64_t(b) * a.U * a.G * kD + i] = 0.0f;
      if (a.stats != nullptr)
        for (int i = tid; i < a.U * a.G * 2; i += kThr)
          a.stats[int64_t(b) * a.U * a.G * 2 + i] = 0.0f;
    }
  }
  if (x0 >= x1 || v >= x1) {
    if (tid == 0) a.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  const int head = NT == 1 ? (gid & 3) : gid;       // this lane's head row
  const bool head_ok = head < a.G;
  // the queries first: they are needed as soon as the first keys are
  QueryRow<T> qrow;
  qrow.load(a.q, (int64_t(pf.b) * a.U + pf.j) * a.G + head, head_ok, q);

  // ---- loads.  kUni: straight into registers; half u of a tile: kreg[u][2 tau + j] is key
  // 8 tau + gid, bytes 16 (4 j + q); vreg[u][i] key 8 (i / 2) + 2 q + i % 2, bytes 16 gid.
  // kSc: scales of a half that a lane needs.
  constexpr int kSc = kUni ? 1 : 4;
  uint4 kreg[kUni ? 2 : 1][4], vreg[2][4];
  float ks_in[2], vs_in[2];
  const auto load_k_of = [&](const Rows& r, auto full) {
    [[maybe_unused]] constexpr bool kFull = decltype(full)::value;
    if constexpr (kUni) {
      // both scales with the keys: they are needed together, before the values
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool some = kFull || ((r.mask >> (16 * u)) & 0xffffu) != 0;
        ks_in[u] = some ? __ldg(a.c.ks + (r.row[u] >> a.c.bshift)) : 0.0f;
        vs_in[u] = some ? __ldg(a.c.vs + (r.row[u] >> a.c.bshift)) : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t there = r.mask >> (16 * u);
        const uint8_t* const p = a.c.k + int64_t(r.row[u]) * kD + gid * kD + 16 * q;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          kreg[kUni ? u : 0][i] =
              load_row16(p + (i >> 1) * 8 * kD + (i & 1) * 64,
                         kFull || ((there >> (8 * (i >> 1) + gid)) & 1u));
      }
    }
  };
  const auto load_v_of = [&](const Rows& r, auto full) {
    [[maybe_unused]] constexpr bool kFull = decltype(full)::value;
    if constexpr (kUni) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t there = r.mask >> (16 * u);
        const uint8_t* const p = a.c.v + int64_t(r.row[u]) * kD + 2 * q * kD + 16 * gid;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          vreg[u][i] = load_row16(
              p + (i >> 1) * 8 * kD + (i & 1) * kD,
              kFull || ((there >> (8 * (i >> 1) + 2 * q + (i & 1))) & 1u));
      }
    }
  };
  const auto load_k = [&](const Rows& r) {
    if (r.mask == 0xffffffffu) load_k_of(r, std::true_type{});
    else load_k_of(r, std::false_type{});
  };
  const auto load_v = [&](const Rows& r) {
    if (r.mask == 0xffffffffu) load_v_of(r, std::true_type{});
    else load_v_of(r, std::false_type{});
  };
  // kUni: lane i pulls key i's K and V rows (one 128-byte line each) into L2.  Else the rows are
  // copied into stage st of the ring, 8 lanes to a row.
  const auto request = [&](const Rows& r, [[maybe_unused]] int st) {
    if constexpr (kUni) {
      const int row = (lane < 16 ? r.row[0] : r.row[1] - 16) + lane;
      if ((r.mask >> lane) & 1u) {
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.c.k + int64_t(row) * kD));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.c.v + int64_t(row) * kD));
      }
    } else {
      __syncwarp();   // the stage has been read by every lane
      if (r.mask != 0u) {
        const uint32_t base = smem_addr(ring + (warp * kStages + st) * kStage);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int n = 4 * i + (lane >> 3);
          const int row = __shfl_sync(0xffffffffu, r.row[0], n);
          const int64_t off = int64_t(max(row, 0)) * kD + 16 * (lane & 7);
          const uint32_t dst = base + n * kD + 16 * ((lane & 7) ^ swz(n));
          cp_async_16_or_zero(dst, a.c.k + off, row >= 0);
          cp_async_16_or_zero(dst + kTile * kD, a.c.v + off, row >= 0);
        }
      }
      cp_async_commit();
    }
  };

  // Tiles under way: r0 in registers or in the ring (or coming), r1 the next one (pulled into L2,
  // or on its way into the ring), tb with its pages and ta with its positions coming.
  Place cur = pf;
  int placed = v;   // place of pf's step
  const auto next_tile = [&]() {
    placed += pf.ls + 1 < pf.ns ? 1 : 1 + cost;
    if (placed >= x1) return no_tile();
    next_place(a, pf);
    return tile_positions<kUni>(a, pf, warp, lane);
  };
  Rows r0, r1;
  Tile ta, tb;
  {
    Tile t0 = tile_positions<kUni>(a, pf, warp, lane), t1 = next_tile();
    tb = next_tile();
    ta = next_tile();
    tile_pages<kUni>(a, t0);
    tile_pages<kUni>(a, t1);
    tile_pages<kUni>(a, tb);
    r0 = tile_rows<kUni>(a, t0);
    load_k(r0);
    load_v(r0);
    if (!kUni) request(r0, 0);
    r1 = tile_rows<kUni>(a, t1);
    request(r1, 1);
  }
  int st = 0;   // r0's stage of the ring
  const auto fetch = [&]() {
    const Rows r = tile_rows<kUni>(a, tb);
    request(r, st == 0 ? kStages - 1 : st - 1);
    tb = ta;
    tile_pages<kUni>(a, tb);
    ta = next_tile();
    return r;
  };

  uint32_t qh[8][2], ql[kLo ? 8 : 1][2];
  float factor = 0.0f;
  float m = -INFINITY, r = -INFINITY, l = 0.0f;
  bool big = false;   // this lane's m is at least 256 in magnitude
  float acc[8][4];
  bool fresh = true;
  int4 cut_here = make_int4(0, 0, 0, 0);   // the unit that ends in a later CTA
  for (;;) {
    const int64_t unit = int64_t(cur.b) * a.U + cur.j;
    if (fresh) {
      factor = query_fragments<T, kLo>(qrow, a.scale_log2, qh, ql);
      m = r = -INFINITY;
      big = false;
      l = 0.0f;
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
      fresh = false;
    }
    Rows r2;
    // kFull: all 32 keys are there
    const auto attend = [&](auto full) {
      constexpr bool kFull = decltype(full)::value;
      const uint32_t mask = r0.mask >> (2 * q);
      const auto there = [&](int u, int i) {   // key 16 u + 8 (i / 2) + 2 q + i % 2
        return kFull || ((mask >> (16 * u + 8 * (i >> 1) + (i & 1))) & 1u);
      };
      // ---- scores x (before scaling) of keys 16 u + 8 tau + 2 q + {0, 1}
      float x[2][4], sf[2][kSc], ksc[2][kSc], vsc[2][kSc];
      [[maybe_unused]] const uint8_t* const tile = ring + (warp * kStages + st) * kStage;
      if constexpr (!kUni) {
        cp_async_wait_pending(1);
        __syncwarp();
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < kSc; ++i) {
          const int from = 16 * u + 8 * (i >> 1) + 2 * q + (i & 1);
          ksc[u][i] = kUni ? ks_in[u] : __shfl_sync(0xffffffffu, r0.ks, from);
          vsc[u][i] = kUni ? vs_in[u] : __shfl_sync(0xffffffffu, r0.vs, from);
        }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int tau = 0; tau < 2; ++tau) {
          float cc[2][4];   // two chains: dimensions 0..63 and 64..127
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int n = 16 * u + 8 * tau + gid;
            const uint4 w = kUni ? kreg[kUni ? u : 0][2 * tau + j]
                                 : *reinterpret_cast<const uint4*>(
                                       tile + n * kD + 16 * ((4 * j + q) ^ swz(n)));
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int c = 4 * j + i;
              const uint32_t b0 = half2_of<FMT>(ww[i], 0), b1 = half2_of<FMT>(ww[i], 1);
              const uint32_t l0 = kLo ? ql[kLo ? c : 0][0] : 0u;
              const uint32_t l1 = kLo ? ql[kLo ? c : 0][1] : 0u;
              if (i == 0) mma_f16_first(cc[j], qh[c][0], l0, qh[c][1], l1, b0, b1);
              else mma_f16(cc[j], qh[c][0], l0, qh[c][1], l1, b0, b1);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
            x[u][2 * tau + e] =
                kLo ? (cc[0][e] + cc[1][e]) + (cc[0][2 + e] + cc[1][2 + e]) : cc[0][e] + cc[1][e];
        }
#pragma unroll
        for (int i = 0; i < kSc; ++i) sf[u][i] = ksc[u][i] * factor;
      }
      load_k(r1);
      // ---- references.  ve: the value scale's exponent plus 1, so that c < 2^ve.
      float up = -INFINITY, up2 = -INFINITY, ve[2][kSc];
      const auto y = [&](int u, int i) {
        return there(u, i) ? x[u][i] * sf[u][kUni ? 0 : i] : -INFINITY;
      };
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float half = -INFINITY;
#pragma unroll
        for (int i = 0; i < kSc; ++i) ve[u][i] = float(int(__float_as_uint(vsc[u][i]) >> 23) - 126);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          half = fmaxf(half, y(u, i));
          if (!kUni) up2 = fmaxf(up2, y(u, i) + ve[u][kUni ? 0 : i]);
        }
        up = fmaxf(up, half);
        if (kUni) up2 = fmaxf(up2, half + ve[u][0]);
      }
      if (a.scores != nullptr && (NT == 2 || gid < 4) && head_ok) {
        float* const o = a.scores + (unit * a.G + head) * a.score_stride + cur.ls * kStep +
                         warp * kTile + 2 * q;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          *reinterpret_cast<float2*>(o + 16 * u) = make_float2(y(u, 0), y(u, 1));
          *reinterpret_cast<float2*>(o + 16 * u + 8) = make_float2(y(u, 2), y(u, 3));
        }
      }
      if (__any_sync(0xffffffffu, up > m || up2 > m + r || big)) {
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, o));
          up2 = fmaxf(up2, __shfl_xor_sync(0xffffffffu, up2, o));
        }
        const float mn = fmaxf(m, ceilf(up)), step = ref_step(m, mn);
        up2 -= mn;
        // Scores of 256 and more are rounded before m is subtracted, and ve is added to the
        // difference: fp32 cannot place m within 1 of an exact x of 2^24 and more, nor add ve to
        // it; and the sums kernel, which gets rounded scores, forms the same weights.
        big = big || (fabsf(mn) >= 256.0f && mn != -INFINITY);
        if (__any_sync(0xffffffffu, big)) {
          float rt = -INFINITY;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              rt = fmaxf(rt, (y(u, i) - mn) + ve[u][kUni ? 0 : i]);
              if (big) x[u][i] *= sf[u][kUni ? 0 : i];
            }
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < kSc; ++i) sf[u][i] = big ? 1.0f : sf[u][i];
          rt = fmaxf(rt, __shfl_xor_sync(0xffffffffu, rt, 1));
          up2 = fmaxf(rt, __shfl_xor_sync(0xffffffffu, rt, 2));
        }
        const float rn = fmaxf(r + step, ceilf(up2));
        m = mn;
        l *= ex2(step);
        const float f = ref_change(r + step, rn);
        r = rn;
        const float f0 = __shfl_sync(0xffffffffu, f, 8 * q);       // column 2 q
        const float f1 = __shfl_sync(0xffffffffu, f, 8 * q + 4);   // column 2 q + 1
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          acc[t][0] *= f0;
          acc[t][1] *= f1;
          acc[t][2] *= f0;
          acc[t][3] *= f1;
        }
      }
      // w = 2^(d + E - r) (c / 2^E) 2^14, d = x - m, E = ve - 1: formed by itself, since p = 2^d and
      // 2^-r c can each leave the range of fp32 where w does not (a block of zeros may lead by
      // 100 and more, and r then lies as low).  c / 2^E is c's mantissa, but for scales below
      // 2^-126 (and 0).
      uint32_t b[2][NT][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float up_w[kSc], mant[kSc];
#pragma unroll
        for (int i = 0; i < kSc; ++i) {
          const uint32_t bits = __float_as_uint(vsc[u][i]);
          up_w[i] = ve[u][i] + (-1.0f - r);
          mant[i] = bits < 0x800000u ? vsc[u][i] * 0x1p126f * 0x1p15f
                                     : __uint_as_float((bits & 0x7fffffu) | 0x46800000u);
        }
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // a key that is not there has d = -inf, and p = w = 0
          const float d = there(u, i) ? fmaf(x[u][i], sf[u][kUni ? 0 : i], -m) : -INFINITY;
          l += ex2(d);
          w[i] = ex2(d + up_w[kUni ? 0 : i]) * mant[kUni ? 0 : i];
        }
        b[u][0][0] = pack_f16(w[0], w[1]);
        b[u][0][1] = pack_f16(w[2], w[3]);
        if constexpr (NT == 1) {
          // columns 4..7: the low parts of heads 0..3
          const uint32_t e0 = pack_f16_rest(w[0], w[1], b[u][0][0]);
          const uint32_t e1 = pack_f16_rest(w[2], w[3], b[u][0][1]);
          b[u][0][0] = gid >= 4 ? e0 : b[u][0][0];
          b[u][0][1] = gid >= 4 ? e1 : b[u][0][1];
        } else {
          b[u][NT - 1][0] = pack_f16_rest(w[0], w[1], b[u][0][0]);
          b[u][NT - 1][1] = pack_f16_rest(w[2], w[3], b[u][0][1]);
        }
      }
      r2 = fetch();
      // ---- values: lane (gid, q): dimensions 16 gid .. + 15 of keys 2q, 2q+1, 8+2q, 9+2q
      // A tile's product is formed by itself and added in fp32: the tensor cores' own sums drop
      // bits below the sum's last, always towards zero, which over thousands of keys shows (2.1e-6
      // of the result at 128K keys per head against 1.0e-6 of fp32 sums).
      if constexpr (!kUni) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = 16 * u + 8 * (i >> 1) + 2 * q + (i & 1);
            vreg[u][i] =
                *reinterpret_cast<const uint4*>(tile + (kTile + n) * kD + 16 * (gid ^ swz(n)));
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float part[4];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const auto word = [&](int v) {
              return i == 0 ? vreg[u][v].x : i == 1 ? vreg[u][v].y : i == 2 ? vreg[u][v].z
                                                                            : vreg[u][v].w;
            };
            const uint32_t ab = __byte_perm(word(0), word(1), hf ? 0x7362 : 0x5140);
            const uint32_t cd = __byte_perm(word(2), word(3), hf ? 0x7362 : 0x5140);
            const uint32_t a0 = half2_of<FMT>(ab, 0), a1 = half2_of<FMT>(ab, 1);
            const uint32_t a2 = half2_of<FMT>(cd, 0), a3 = half2_of<FMT>(cd, 1);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (u == 0 && n == 0) mma_f16_first(part, a0, a1, a2, a3, b[u][n][0], b[u][n][1]);
              else mma_f16(part, a0, a1, a2, a3, b[u][n][0], b[u][n][1]);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[2 * i + hf][e] += part[e];
        }
      }
      load_v(r1);
    };
    if (r0.mask == 0xffffffffu) {
      attend(std::true_type{});
    } else if (r0.mask != 0u) {
      attend(std::false_type{});
    } else {
      if (a.scores != nullptr) {
        // entries without a key (skipped, or a bad page) have no weight
        for (int i = lane; i < a.G * kTile; i += 32) {
          const int at = cur.ls * kStep + warp * kTile + i % kTile;
          if (at < cur.len)
            a.scores[(unit * a.G + i / kTile) * a.score_stride + at] = -INFINITY;
        }
      }
      load_k(r1);
      r2 = fetch();
      load_v(r1);
    }
    r0 = r1;
    r1 = r2;
    if (!kUni) st = st + 1 == kStages ? 0 : st + 1;

    const int u0 = v - cur.ls;                  // the place of the unit's first step
    const int unit_end = u0 + cur.ns;
    if (v + 1 < x1 && v + 1 < unit_end) {
      ++cur.ls;
      ++v;
    } else {
      const int next_v = unit_end + cost;
      const bool more = next_v < x1;
      if (more) {
        // the next unit's queries come while this one's states are merged
        next_place(a, cur);
        qrow.load(a.q, (int64_t(cur.b) * a.U + cur.j) * a.G + head, head_ok, q);
      }
      // ---- merge the warps' states
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (q == 0 && (NT == 2 || gid < 4)) {
        sm.stat[warp][head][0] = m;
        sm.stat[warp][head][1] = l;
        sm.stat[warp][head][2] = r;
      }
      // High and low parts together.  NT = 1: lanes q and q ^ 2 hold the two parts of two
      // heads; each keeps half of the dimensions (value 4 t + i: tile t + 4 (q / 2)).
      // NT = 2: value 4 t + i: tile t.
      if constexpr (NT == 1) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float keep = (q & 2) ? acc[t + 4][i] : acc[t][i];
            const float give = (q & 2) ? acc[t][i] : acc[t + 4][i];
            sm.sums[warp][4 * t + i][lane] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
          }
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) sm.sums[warp][4 * t + i][lane] = acc[t][i];
      }
      __syncthreads();
      // ---- the unit's parts: CTAs c0 .. c0 + parts - 1 hold steps of it
      const int c0 = cut.owner(u0);
      const int parts = cut.owner(unit_end - 1) - c0 + 1;
      // slot 0: the part of a unit that began before, slot 1: of one that begins here
      const int which = u0 >= x0 ? 1 : 0;
      float* const slot = a.part + int64_t(2 * blockIdx.x + which) * a.G * kPart;
      // value v of lane (gid, q) of the fragments: head 2 q (NT = 1: 2 (q % 2)) + v % 2,
      // dimension 16 gid (+ 8 (q / 2)) + v / 2; thread (head, 4 dimensions) sums the warps
      for (int i = tid; i < a.G * (kD / 4); i += kThr) {
        const int hh = i / (kD / 4), d = 4 * (i % (kD / 4));
        float hM = -INFINITY, hR = -INFINITY, hl = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) hM = fmaxf(hM, sm.stat[w][hh][0]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          hR = fmaxf(hR, sm.stat[w][hh][2] + ref_step(sm.stat[w][hh][0], hM));
        const int ln = 4 * (d >> 4) + (NT == 1 ? (hh >> 1) + 2 * ((d >> 3) & 1) : hh >> 1);
        const int v0 = 2 * (NT == 1 ? d & 7 : d & 15) + (hh & 1);
        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float step = ref_step(sm.stat[w][hh][0], hM);
          hl += sm.stat[w][hh][1] * ex2(step);
          const float f = ref_change(sm.stat[w][hh][2] + step, hR);
#pragma unroll
          for (int e = 0; e < 4; ++e) t[e] = fmaf(sm.sums[w][v0 + 2 * e][ln], f, t[e]);
        }
        if (parts == 1) {
          const bool some = hl > 0.0f || !(hl == hl);   // an empty list: zeros
          *reinterpret_cast<float4*>(a.out + (unit * a.G + hh) * kD + d) =
              OutScale(hR, hl, some).of(t[0], t[1], t[2], t[3]);
          if (d == 0 && a.stats != nullptr) {
            float* const o = a.stats + (unit * a.G + hh) * 2;
            o[0] = some ? hM : 0.0f;
            o[1] = some ? 1.0f / hl : 0.0f;
          }
        } else {
          *reinterpret_cast<float4*>(slot + hh * kPart + 4 + d) =
              make_float4(t[0], t[1], t[2], t[3]);
          if (d == 0)
            *reinterpret_cast<float4*>(slot + hh * kPart) = make_float4(hM, hl, hR, 0.0f);
        }
      }
      __syncthreads();   // the part is written; sums and stat are free again
      const int nth = int(blockIdx.x) - c0;
      if (nth + 1 < parts) cut_here = make_int4(int(unit), int(unit >> 32), parts, nth);
      fresh = true;
      if (!more) break;
      v = next_v;
    }
  }
  if (tid == 0) a.cuts[blockIdx.x] = cut_here;
}

// ------------------------------------------------------------- attention weights
// The running sums' traffic (8 bytes a position) and the scores bound these passes: 32 kv heads x
// 128K positions take 11 us, 17 ragged sequences of up to 8K and 4 kv heads 7 us (latency).
// Dense: w_out[unit][j] = w_in[unit][j] + sum_g 2^(x_gj - M_g) / l_g, from the scores the
// attention kernel left in the workspace (4 G bytes per key written and read against 128 G
// if K were scored again).
constexpr int kWPer = 4;

template <int kHeads>
__global__ void __launch_bounds__(256) kv8_weights_kernel(
    const float* __restrict__ scores, int64_t score_stride, const float* __restrict__ stats,
    const int32_t* __restrict__ seq_lens, int Hkv, int G, int64_t Lmax, int tiles,
    const float* w_in, float* w_out, uint32_t* err) {
  pdl_wait();
  pdl_trigger();
  const uint32_t un = blockIdx.x / uint32_t(tiles);
  const int64_t unit = un;
  const int64_t j0 = int64_t(blockIdx.x - un * tiles) * (256 * kWPer) + threadIdx.x;
  const int64_t len =
      seq_lens == nullptr ? Lmax : checked_len(seq_lens[un / uint32_t(Hkv)], Lmax, err, false);
  // the heads' weights are summed first: the (larger) running sum is rounded once
  float in[kWPer], s[kWPer];
#pragma unroll
  for (int u = 0; u < kWPer; ++u) {
    const int64_t j = j0 + u * 256;
    in[u] = j < len ? w_in[unit * Lmax + j] : 0.0f;
    s[u] = 0.0f;
  }
  // kHeads heads' scores at once (G = 1: 1, G <= 4: 4, else 8), so that their latencies overlap: 17
  // ragged sequences with 8 heads to a kv head take 1.3 us less in all than one by one (of 32), 32K with
  // 4 heads 0.5 (of 23).
  for (int g0 = 0; g0 < G; g0 += kHeads) {
    float x[kHeads][kWPer], M[kHeads], inv[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const bool there = g0 + i < G;
      const int64_t row = unit * G + g0 + (there ? i : 0);
      M[i] = __ldg(stats + row * 2);
      inv[i] = there ? __ldg(stats + row * 2 + 1) : 0.0f;
#pragma unroll
      for (int u = 0; u < kWPer; ++u) {
        const int64_t j = j0 + u * 256;
        x[i][u] = there && j < len ? __ldcs(scores + row * score_stride + j) : -INFINITY;
      }
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
#pragma unroll
      for (int u = 0; u < kWPer; ++u) s[u] = fmaf(ex2(x[i][u] - M[i]), inv[i], s[u]);
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
// Every slice reads the whole lists, so slices are wide (and the old sums requested before the
// lists, their latency being in the way then) when they still fill the device, and narrow
// otherwise: 8 sequences of 32K, 8 kv heads, 4 lists of 1024 each take 9.0 us wide against 10.8 narrow;
// one sequence 4.8 against 4.2.
constexpr int kWideSlice = 8192, kNarrowSlice = 4096;

template <int kSlice>
__global__ void __launch_bounds__(512, kSlice == kWideSlice ? 2 : 1) kv8_sparse_weights_kernel(
    const int32_t* __restrict__ idx, int k, const float* __restrict__ scores,
    int64_t score_stride, const float* __restrict__ stats, int lists, int G, int64_t Lmax,
    int slices, const float* w_in, float* w_out) {
  __shared__ float sum[kSlice];
  pdl_wait();
  pdl_trigger();
  constexpr int kPer = 2;                                       // entries per thread and round
  const int tid = threadIdx.x;
  const uint32_t un = blockIdx.x / uint32_t(slices);
  const int64_t unit = un;                                      // (b, kv head)
  const int64_t base = int64_t(blockIdx.x - un * slices) * kSlice;
  const int n = int(min(int64_t(kSlice), Lmax - base));
  const int heads = G / lists;   // `lists` lists: G per-head ones, or one for all G heads
  // entries of a round: position in the slice (-1: not in it) and the first head's score; requested
  // a round ahead, over the border of lists
  int pos[kPer], next_pos[kPer];
  float x[kPer], next_x[kPer];
  const auto load = [&](int li, int i0, int (&p)[kPer], float (&s)[kPer]) {
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = i0 + tid + u * 512;
      p[u] = -1;
      s[u] = 0.0f;
      if (li < lists && i < k) {
        p[u] = __ldg(idx + (unit * lists + li) * k + i);
        s[u] = __ldg(scores + (unit * G + li * heads) * score_stride + i);
      }
    }
  };
  load(0, 0, pos, x);
  const float* const in = w_in + unit * Lmax + base;
  float* const out = w_out + unit * Lmax + base;
  constexpr bool kEarly = kSlice == kWideSlice;
  [[maybe_unused]] float old[kSlice / 512];
  if (kEarly && in != out) {
#pragma unroll
    for (int u = 0; u < kSlice / 512; ++u)
      if (tid + u * 512 < n) old[u] = __ldg(in + tid + u * 512);
  }
  for (int i = tid; i < n; i += 512) sum[i] = 0.0f;
  __syncthreads();
  for (int li = 0, i0 = 0; li < lists;) {
    const bool ends = i0 + 512 * kPer >= k;
    const int nl = ends ? li + 1 : li, ni = ends ? 0 : i0 + 512 * kPer;
    load(nl, ni, next_pos, next_x);
    const int64_t r0 = unit * G + li * heads;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int64_t p = int64_t(pos[u]) - base;
      if (pos[u] < 0 || p < 0 || p >= n) continue;
      float w = ex2(x[u] - __ldg(stats + 2 * r0)) * __ldg(stats + 2 * r0 + 1);
      for (int g = 1; g < heads; ++g)
        w = fmaf(ex2(__ldg(scores + (r0 + g) * score_stride + i0 + tid + u * 512) -
                     __ldg(stats + 2 * (r0 + g))),
                 __ldg(stats + 2 * (r0 + g) + 1), w);
      atomicAdd(&sum[p], w);
    }
    if (ends) __syncthreads();
    li = nl;
    i0 = ni;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      pos[u] = next_pos[u];
      x[u] = next_x[u];
    }
  }
  if (in == out) {
    for (int i = tid; i < n; i += 512)
      if (sum[i] != 0.0f) out[i] = in[i] + sum[i];
  } else if constexpr (kEarly) {
#pragma unroll
    for (int u = 0; u < kSlice / 512; ++u)
      if (tid + u * 512 < n) out[tid + u * 512] = old[u] + sum[tid + u * 512];
  } else {
#pragma unroll 8
    for (int i = tid; i < n; i += 512) out[i] = __ldg(in + i) + sum[i];
  }
}

// CTAs of the attention kernel: the co-resident ones, no more than there can be steps.
int attention_ctas(int64_t units, int64_t len, int sms) {
  const int64_t steps = units * ((len + kStep - 1) / kStep);
  const int64_t room = sms * kCtasPerSm < kMaxParts ? sms * kCtasPerSm : kMaxParts;
  return int(steps < room ? steps : room);
}

// Whether units may be cut between CTAs (then the combine kernel follows).
bool cuts_units(int64_t units, int64_t len, bool equal, int ctas) {
  const int64_t per = (len + kStep - 1) / kStep;
  return per > 1 && !(equal && whole_units(int(units), int(per), ctas));
}

struct Room {
  size_t cuts, part, stats, scores, total;
  int64_t stride;
};
Room workspace_room(int B, int Hq, int Hkv, int64_t Lmax, int k, bool shared, bool weights) {
  const bool sparse = k > 0;
  const int64_t U = sparse && !shared ? Hq : Hkv;
  const int G = int(Hq / U);
  Room r;
  const int ctas = attention_ctas(B * U, sparse ? k : Lmax, device_sms());
  r.cuts = 256;
  r.part = r.cuts + align_up(size_t(ctas) * sizeof(int4), 256);
  r.stats = r.part + align_up(size_t(ctas) * 2 * G * kPart * 4, 256);
  r.scores = r.stats + (weights ? align_up(size_t(B) * Hq * 8, 256) : 0);
  // rows padded to whole warp tiles: the kernel stores scores tile by tile
  r.stride = ((sparse ? int64_t(k) : Lmax) + kTile - 1) / kTile * kTile;
  r.total = r.scores + (weights ? align_up(size_t(B) * Hq * size_t(r.stride) * 4, 256) : 0);
  return r;
}

template <typename T, int FMT, int NT>
cudaError_t run_attention(const Args& a, int ctas, bool uni, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const auto given = kv8_attention_kernel<T, FMT, NT, false>;
  if (!uni) {
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(given),
                                     kWarps * kStages * kStage, done, false);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kThr);
  cfg.dynamicSmemBytes = uni ? 0 : kWarps * kStages * kStage;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return uni ? cudaLaunchKernelEx(&cfg, kv8_attention_kernel<T, FMT, NT, true>, a)
             : cudaLaunchKernelEx(&cfg, given, a);
}

template <typename T, int FMT>
cudaError_t run_attention_g(const Args& a, int ctas, bool uni, cudaStream_t stream) {
  return a.G <= 4 ? run_attention<T, FMT, 1>(a, ctas, uni, stream)
                  : run_attention<T, FMT, 2>(a, ctas, uni, stream);
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
  a.cuts = reinterpret_cast<int4*>(base + r.cuts);
  a.part = reinterpret_cast<float*>(base + r.part);
  a.stats = weights ? reinterpret_cast<float*>(base + r.stats) : nullptr;
  a.scores = weights ? reinterpret_cast<float*>(base + r.scores) : nullptr;
  a.score_stride = r.stride;
  a.scale_log2 = float(1.4426950408889634 / 11.313708498984761);
  a.U = idx && !shared ? Hq : c.Hkv;
  a.G = Hq / a.U;
  a.heads_per_kv = a.U / c.Hkv;
  a.k = k;
  const int ctas = attention_ctas(int64_t(c.B) * a.U, idx ? k : c.Lmax, device_sms());
  const bool uni = idx == nullptr && c.bshift >= 4;   // pages are no smaller than blocks
  cudaError_t e;
  if (dt == ADAMAS_BF16)
    e = fmt == kFmtE4m3 ? run_attention_g<__nv_bfloat16, kFmtE4m3>(a, ctas, uni, stream)
                        : run_attention_g<__nv_bfloat16, kFmtInt8>(a, ctas, uni, stream);
  else
    e = fmt == kFmtE4m3 ? run_attention_g<float, kFmtE4m3>(a, ctas, uni, stream)
                        : run_attention_g<float, kFmtInt8>(a, ctas, uni, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cuts_units(int64_t(c.B) * a.U, idx ? k : c.Lmax, idx != nullptr || seq_lens == nullptr, ctas)) {
    cfg.gridDim = dim3(unsigned(ctas));
    cfg.blockDim = dim3(kCombineThreads);
    e = cudaLaunchKernelEx(&cfg, kv8_combine_kernel, static_cast<const int4*>(a.cuts),
                           static_cast<const float*>(a.part), a.G, a.stats, out);
    if (e != cudaSuccess) return e;
  }
  if (!weights) return cudaSuccess;
  const int64_t units = int64_t(c.B) * c.Hkv;
  const int G = Hq / c.Hkv;
  if (idx == nullptr) {
    const int64_t tiles = (c.Lmax + 256 * kWPer - 1) / (256 * kWPer);
    if (units * tiles > INT32_MAX) return cudaErrorNotSupported;   // more blocks than a grid holds
    cfg.gridDim = dim3(unsigned(units * tiles));
    cfg.blockDim = dim3(256);
    const auto kernel = G == 1   ? kv8_weights_kernel<1>
                        : G <= 4 ? kv8_weights_kernel<4>
                                 : kv8_weights_kernel<8>;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<const float*>(a.scores),
                              a.score_stride, static_cast<const float*>(a.stats), seq_lens, c.Hkv,
                              G, c.Lmax, int(tiles), w_in, w_out, a.err);
  }
  const bool wide = units * ((c.Lmax + kWideSlice - 1) / kWideSlice) >= device_sms();
  const int64_t slice = wide ? kWideSlice : kNarrowSlice;
  const int64_t slices = (c.Lmax + slice - 1) / slice;
  if (units * slices > INT32_MAX) return cudaErrorNotSupported;   // more blocks than a grid holds
  cfg.gridDim = dim3(unsigned(units * slices));
  cfg.blockDim = dim3(512);
  return cudaLaunchKernelEx(&cfg, wide ? kv8_sparse_weights_kernel<kWideSlice>
                                       : kv8_sparse_weights_kernel<kNarrowSlice>, idx, k,
                            static_cast<const float*>(a.scores), a.score_stride,
                            static_cast<const float*>(a.stats), shared ? 1 : G, G, c.Lmax,
                            int(slices), w_in, w_out);
}

}  // namespace adamas
