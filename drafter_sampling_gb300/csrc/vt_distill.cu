// Distillation of the drafter from a teacher's k best ids on sm_103a: loss and
// gradient of rows of logits.
//
// A row has the drafter's logits z over K ids and the teacher's list of (id, ln t).
// Kept are the entries that the drafter has: id given, in its vocabulary, z > -inf.
// With p = softmax(z / T), a = sum t over the kept, q = sum p over the unlisted:
//
//   rest:          b = max(0, 1 - a), A = a + b
//     loss = sum t_i (ln t_i - ln p_i) + b (ln b - ln q)
//     T dloss/dz_j = A p_j - t_j (listed),  (A - b / q) p_j (unlisted)
//   renormalised:  t' = t / a
//     loss = sum t'_i (ln t'_i - ln p_i)
//     T dloss/dz_j = p_j - t'_j (listed),  p_j (unlisted)
//
// b is what is left of 1, so a is summed with pairs of fp32 values; q is summed
// from the unlisted ids alone, never as a difference.  A gradient is then
//
//   g (c_all 2^((z_j - m) c) - c_t t_j) (listed),  g c_rest 2^((z_j - mr) c) (unlisted)
//
// with m the largest logit of all, mr that of the unlisted ids (two, because either
// may be out of fp32's range relative to the other) and the three factors kept
// per row by the loss.
//
// The loss reads R K logits once and is bound by HBM in the middle of a launch: 2304 rows of 38016
// bf16 logits 39.8 us (4.4 TB/s; 25.9 at the measured copy rate), of which 3 to the first chunk, 3 for
// the last rows' statistics and losses, and a sixth round of rows for 24 of 456 blocks.  112
// rows of 128256 fp32, 59 of them scored: 12.5 (latencies; 4.5 by bytes).  The gradient alone reads and
// writes them: the same bf16 rows 54.9 (6.4 TB/s), 58.8 in the logits' place.  Both in one call read and
// write once: 2048 rows of 32768 fp32 92.4 us (5.8 TB/s; 79 by bytes), in place 93.4; 1024 rows of 128256 bf16,
// 576 scored, 104 (60.9 by bytes), in place as well: there a row's two passes of exponentials take 2/3 of its
// turn, a block's warps idle in the rest.  All in graphs of calls.
#include <algorithm>
#include <atomic>
#include <cmath>

#include <cooperative_groups.h>

#include "vt_internal.h"
#include "vt_rows.cuh"
#include "vt_umma.cuh"

namespace cg = cooperative_groups;

namespace vt {
namespace {

constexpr int kDsMaxK = 128;
constexpr int kDsNT = 128;              // threads of the gradient kernel, one per list entry at least

// what takes an element out of a sum
template <typename T> struct Mask;
template <> struct Mask<float> {
  __device__ static uint32_t bits() { return 0xff800000u; }  // -infinity
};
template <> struct Mask<uint16_t> {
  __device__ static uint16_t bits() { return 0xff80u; }
};

struct DsStats {
  float m, mr, c_all, c_rest, c_t;
};

// (128 bytes: with more of them the row kernels spill, 107 instead of 104 us for 1024 rows of 128256 bf16)
struct DsArgs {
  const void* logits;
  int64_t ld;
  int R, K, V, k;
  bool rest;
  bool own_status;         // one row: its block stores the status word; else it is zeroed beforehand
  float c;                 // log2(e) / T
  Pair twice;              // 2 / T in units of `unit`, a power of two such that it is at most 1
  float unit, inv_t;       // inv_t: 1 / T
  const int* ids;          // [R][k]
  const float* logp;       // [R][k]
  const int* inv_map;      // [V] or nullptr (V == K)
  const float* weight;     // [R] or nullptr: dL/dloss
  float* out_loss;         // [R]
  DsStats* stats;          // [R]
  void* grad;
  int64_t ld_grad;
  int* dev_status;
};

static_assert(sizeof(DsArgs) <= 128, "");
// 1 / a.unit
__device__ __forceinline__ float ds_per_unit(const DsArgs& a) {
  return __int_as_float(0x7f000000 - __float_as_int(a.unit));
}

// the place of list entry i in the drafter's vocabulary, -1 where it has none,
// -2 where the id or the map is out of range
__device__ __forceinline__ int ds_place(const DsArgs& a, int64_t i) {
  const int id = a.ids[i];
  if (id == -1) return -1;
  if (id < 0 || id >= a.V) return -2;
  if (!a.inv_map) return id;
  const int p = a.inv_map[id];
  return p >= -1 && p < a.K ? p : -2;
}

// A row's list as the block's warps share it
struct DsList {
  int pos[kDsMaxK];    // bytes from the start of what this block reads of the row, -1: not there
  float val[kDsMaxK];  // the gradient there
  int any;             // an id is given
};

// What one warp holds of a row's list: its lanes have entries lane, lane + 32, ..., H each
template <int H>
struct DsEntries {
  int p[H];           // first the ids, then places in the drafter's vocabulary: -1 none, -2 out of range
  float z[H], lp[H];  // of kept entries; z = -infinity: not kept
  bool any;           // an id is given
};
// (loads that stay where they are issued: a turn ahead of their use)
__device__ __forceinline__ uint32_t load_ahead(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
// A logit.  Not by a load that promises that nothing writes there while the kernel runs: the gradient
// may take the logits' place.
template <typename T>
__device__ __forceinline__ float logit(const T* p) {
  if constexpr (sizeof(T) == 4) {
    uint32_t v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return __uint_as_float(v);
  } else {
    uint16_t v;
    asm volatile("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
    return bf16_bits_to_float(v);
  }
}
template <int H>
__device__ __forceinline__ void ds_ids(const DsArgs& a, int64_t row, int lane, int (&id)[H]) {
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int i = lane + 32 * h;
    id[h] = row < a.R && i < a.k ? (int)load_ahead(a.ids + row * a.k + i) : -1;
  }
}
template <int H>
__device__ __forceinline__ void ds_map(const DsArgs& a, const int (&id)[H], DsEntries<H>& e) {
  e.any = false;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    int p = id[h];
    e.any |= p != -1;
    if (p != -1 && (p < 0 || p >= a.V)) p = -2;
    if (p >= 0 && a.inv_map) {
      const int q = (int)load_ahead(a.inv_map + p);
      p = q >= -1 && q < a.K ? q : -2;
    }
    e.p[h] = p;
  }
  e.any = __any_sync(0xffffffffu, e.any);
}
template <typename T, int H>
__device__ __forceinline__ void ds_values(const DsArgs& a, int64_t row, int lane, DsEntries<H>& e) {
  const T* l = static_cast<const T*>(a.logits) + row * a.ld;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    e.z[h] = e.p[h] >= 0 ? logit(l + e.p[h]) : -INFINITY;
    e.lp[h] = e.p[h] >= 0 ? __uint_as_float(load_ahead(a.logp + row * a.k + lane + 32 * h)) : 0.f;
  }
}
// whether one of a row's ids is given; all lanes of a warp call it
template <int H>
__device__ __forceinline__ bool ds_any(const int (&id)[H]) {
  bool any = false;
#pragma unroll
  for (int h = 0; h < H; ++h) any |= id[h] != -1;
  return __any_sync(0xffffffffu, any);
}

// a row's edge element that place p is, or -1
template <int VE>
__device__ __forceinline__ int ds_edge(const Span& sp, int p) {
  if (p < 0) return -1;
  if (p < sp.head) return p;
  const int t = p - sp.nvec * VE;
  return t >= sp.head ? t : -1;
}

// Flags of the entries' values; two kept entries of one place among them: each leaves its number
// in a cell that its place gives, and one that finds another there has the same place, or
// tries again with other cells.
constexpr int kDsCells = 512;
struct DsCells {
  int place[kDsMaxK];
  uint8_t tag[kDsCells];
};
template <int H>
__device__ __forceinline__ int ds_flags(const DsEntries<H>& e, DsCells& sh, int lane) {
  int flags = 0;
  unsigned open = 0;  // of this lane's entries, those not yet told apart from the others
#pragma unroll
  for (int h = 0; h < H; ++h) {
    if (e.p[h] == -2) flags |= VT_DEV_BAD_ID;
    if (e.z[h] != -INFINITY) {
      if (!(e.z[h] < INFINITY) || !(e.lp[h] < 80.f)) flags |= VT_DEV_NONFINITE;
      open |= 1u << h;
    }
    sh.place[lane + 32 * h] = e.p[h];
  }
  for (uint32_t mix = 1; __any_sync(0xffffffffu, open != 0); mix = mix * 0x9E3779B1u + 2) {
    const auto cell = [&](int p) { return ((uint32_t)p * mix >> (mix == 1 ? 0 : 20)) & (kDsCells - 1); };
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (open >> h & 1) sh.tag[cell(e.p[h])] = (uint8_t)(lane + 32 * h);
    __syncwarp();
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (open >> h & 1) {
        const int i = lane + 32 * h, o = sh.tag[cell(e.p[h])];
        const bool same = sh.place[o] == e.p[h];
        if (o != i && same) flags |= VT_DEV_DUPLICATE_ID;
        if (same) open &= ~(1u << h);
      }
    __syncwarp();
  }
  return __reduce_or_sync(0xffffffffu, flags);
}

__device__ __forceinline__ Pair pair_from_lane(Pair v, int lane) {
  return Pair{__shfl_sync(0xffffffffu, v.h, lane), __shfl_sync(0xffffffffu, v.l, lane)};
}
__device__ __forceinline__ Pair pair_xor(Pair v, int o) {
  return Pair{__shfl_xor_sync(0xffffffffu, v.h, o), __shfl_xor_sync(0xffffffffu, v.l, o)};
}
__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// the lanes' sums as one (their five additions round: 2^-24 each)
__device__ __forceinline__ RowSum warp_join(RowSum a, float c) {
  const float m = warp_max_nan(a.m);
  return RowSum{m, warp_add((a.s + a.e) * exp2_approx((a.m - m) * c)), 0.f};
}

// What a row's list says by itself, the same in all lanes of the warp that holds it
struct DsHead {
  bool kept;    // an entry is
  int flags;
  float m;      // largest kept logit
  Pair S;       // sum of e^((z - m) / T) over the kept
  Pair mass;    // sum of t
  Pair cross;   // sum of t (ln t - (z - m) / T), in units of DsArgs::unit
};

// (z - m) / T in units of a.unit: z - m may lie beyond fp32, its quotient too where T < 1, and what the
// loss makes of them not.  (Halves differ exactly.)
__device__ __forceinline__ Pair ds_below(const DsArgs& a, float z, float m) {
  Pair d;
  two_sum(0.5f * z, -0.5f * m, d.h, d.l);
  return pair_mul(d, a.twice);
}
__device__ __forceinline__ Pair pair_scale(Pair v, float f) { return Pair{v.h * f, v.l * f}; }  // f: a power of two
// e^(y a.unit); 0 where fp32 has no such number
__device__ __forceinline__ Pair ds_exp(const DsArgs& a, Pair y) { return pair_exp(pair_scale(y, a.unit)); }

// (leaves the entries' weights 2^((z - m) c) in z and t in lp; both 0 where not kept)
template <int H>
__device__ __forceinline__ DsHead ds_head(const DsArgs& a, DsEntries<H>& e, int flags) {
  DsHead r;
  float m = -INFINITY;
#pragma unroll
  for (int h = 0; h < H; ++h) m = max_nan(m, e.z[h]);
  r.m = m = warp_max_nan(m);
  r.kept = !(m == -INFINITY);
  r.flags = flags;
  r.S = r.mass = r.cross = Pair{0.f, 0.f};
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const bool kept = e.z[h] != -INFINITY;
    const float z = kept ? e.z[h] : m;
    const Pair lnt{kept ? e.lp[h] : -INFINITY, 0.f}, t = pair_exp(lnt);
    const Pair y = ds_below(a, z, m), d = pair_add(Pair{t.h > 0.f ? lnt.h * ds_per_unit(a) : 0.f, 0.f}, pair_neg(y));
    const Pair x = pair_mul(t, d);
    r.mass = pair_add(r.mass, t);
    r.cross = pair_add(r.cross, t.h > 0.f ? x : Pair{0.f, 0.f});
    e.lp[h] = t.h;
    // (a listed id's weight to its last place: the list usually has most of S)
    const Pair w = kept ? ds_exp(a, y) : Pair{0.f, 0.f};
    r.S = pair_add(r.S, w);
    e.z[h] = w.h;
  }
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
    r.S = pair_add(r.S, pair_xor(r.S, o));
    r.mass = pair_add(r.mass, pair_xor(r.mass, o));
    r.cross = pair_add(r.cross, pair_xor(r.cross, o));
  }
  return r;
}

// What the consuming warps leave of a row: the sum over its unlisted ids (s = 0: there
// are none above -infinity)
struct DsSum {
  float m, s;
  int late;
};
// The row's statistics from both, and what the loss takes of them
struct DsTotal {
  Pair w;      // e^((l - m) / T) of the lower of the list's and the others' maxima
  Pair b;      // the teacher's rest: what the list leaves of 1, good to 2^-28
  int flags;
  bool learns;
};
// The consuming warps wait for this, so it is plain fp32 but for the exponential and b: a few roundings.  Those
// of c_all and c_rest are common to a row; where drafter and teacher agree on the rest, c_rest is a small difference and
// every unlisted id's gradient is off by them, and by the sums' own roundings, in one direction.
__device__ __forceinline__ DsTotal ds_stats(const DsArgs& a, const DsHead& hd, const DsSum& un, DsStats& st) {
  DsTotal r{Pair{0.f, 0.f}, Pair{0.f, 0.f}, hd.flags | (un.late ? VT_DEV_TIMEOUT : 0), false};
  const bool rest = !(un.s == 0.f);  // (NaN: flagged below)
  const float m = rest ? max_nan(hd.m, un.m) : hd.m, inv_t = a.inv_t;
  st = DsStats{0.f, 0.f, 0.f, 0.f, 0.f};
  if (hd.kept && !(m < INFINITY)) r.flags |= VT_DEV_NONFINITE;
  if (r.flags) {
    const float nan = __int_as_float(0x7fc00000);
    st = DsStats{nan, nan, nan, nan, nan};
    return r;
  }
  if (a.rest && rest) r.b = pair_add(Pair{1.f, 0.f}, pair_neg(hd.mass));
  if (!(r.b.h > 0.f)) r.b = Pair{0.f, 0.f};
  const float A = hd.mass.h + r.b.h;
  if (!hd.kept || !(A > 0.f)) return r;  // nothing to learn from this row
  r.learns = true;
  // one of the two maxima is m
  const float lower = rest ? fminf(hd.m, un.m) : m;
  r.w = ds_exp(a, ds_below(a, lower, m));
  const float top = rest ? un.m < m ? r.w.h : 1.f : 0.f;
  const float S = fmaf(un.s, top, hd.m < m ? hd.S.h * r.w.h : hd.S.h);
  st.m = m;
  st.mr = rest ? un.m : 0.f;
  const float all = inv_t / S, each = inv_t / un.s;
  if (a.rest) {
    st.c_all = A * all;
    st.c_rest = rest ? fmaf(A * all, top, -(r.b.h * each)) : 0.f;
    st.c_t = inv_t;
  } else {
    st.c_all = all;
    st.c_rest = all * top;
    st.c_t = inv_t / hd.mass.h;
  }
  return r;
}

// The loss, by the warp that holds the list (sr: the unlisted ids' sum again, with what rounding took)
__device__ __forceinline__ float ds_loss(const DsArgs& a, const DsHead& hd, const DsSum& un, Pair sr,
                                         const DsStats& st, const DsTotal& r, int lane) {
  if (r.flags) return __int_as_float(0x7fc00000);
  if (!r.learns) return 0.f;
  Pair S = hd.m < st.m ? pair_mul(hd.S, r.w) : hd.S;
  if (un.s > 0.f) S = pair_add(S, un.m < st.m ? pair_mul(sr, r.w) : sr);
  // four logarithms at once, one per lane
  Pair v = lane == 0 ? S : lane == 1 ? sr : lane == 2 ? r.b : hd.mass;
  v = v.h > 0.f ? pair_scale(pair_log(v), ds_per_unit(a)) : Pair{0.f, 0.f};
  const Pair lnS = pair_from_lane(v, 0), lnr = pair_from_lane(v, 1), lnb = pair_from_lane(v, 2);
  const Pair lna = pair_from_lane(v, 3);
  // ln p = (z - hd.m) / T + shift
  const Pair shift = pair_add(ds_below(a, hd.m, st.m), pair_neg(lnS));
  Pair sum = pair_add(hd.cross, pair_neg(pair_mul(hd.mass, shift)));
  if (!a.rest) {
    sum = pair_add(pair_div(sum, hd.mass), pair_neg(lna));
  } else if (r.b.h > 0.f) {
    const Pair lnq = pair_add(pair_add(lnr, ds_below(a, un.m, st.m)), pair_neg(lnS));
    sum = pair_add(sum, pair_mul(r.b, pair_add(lnb, pair_neg(lnq))));
  }
  return sum.h != sum.h ? INFINITY : sum.h * a.unit;  // (NaN: a term beyond fp32; they are positive)
}

// Loss, statistics and flags of a row to where they go, by one thread
__device__ __forceinline__ void ds_put(const DsArgs& a, int row, float loss, const DsStats& st, int flags) {
  a.out_loss[row] = loss;
  a.stats[row] = st;
  if (a.own_status) {
    *a.dev_status = flags;
    return;
  }
  griddep_wait();  // the status word is clear
  if (flags) atomicOr(a.dev_status, flags);
}

// Calls f(entry, byte position) for the listed elements of `bytes` bytes of the row that begin `first`
// bytes into the block's part, in the vectors of this warp (they go to threads in turn).
template <int NW, typename F>
__device__ __forceinline__ void ds_each(const DsList& sh, int first, int bytes, int k, int warp, int lane, F f) {
  for (int i = lane; i < k; i += 32) {
    const int p = sh.pos[i] - first;
    if (p >= 0 && p < bytes && ((p >> 9) & (NW - 1)) == warp) f(i, p);
  }
  __syncwarp();
}

// -------------------------------------------------------------- the gradient
template <typename T> struct Store;
template <> struct Store<float> {
  __device__ static void put(float* p, float v) { *p = v; }
  // factor * 2^((x - m) c) of a vector's elements
  __device__ static uint4 grad(uint4 v, float m, float c, float factor) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      float t0, t1;
      unpack2(mul2(Vec<float>::diff2(v, e, -m), pack2(c, c)), t0, t1);
      unpack2(mul2(pack2(exp2_approx(t0), exp2_approx(t1)), pack2(factor, factor)), t0, t1);
      w[e] = __float_as_uint(t0);
      w[e + 1] = __float_as_uint(t1);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Store<uint16_t> {
  // round to nearest even; NaN stays NaN
  __device__ static void put(uint16_t* p, float v) {
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(*p) : "f"(v));
  }
  __device__ static uint4 grad(uint4 v, float m, float c, float factor) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      float t0, t1;
      unpack2(mul2(Vec<uint16_t>::diff2(v, e, -m), pack2(c, c)), t0, t1);
      unpack2(mul2(pack2(exp2_approx(t0), exp2_approx(t1)), pack2(factor, factor)), t0, t1);
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e / 2]) : "f"(t1), "f"(t0));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// the gradient at a listed id
__device__ __forceinline__ float ds_listed(const DsArgs& a, const DsStats& st, float g, float z, float t) {
  return g * (st.c_all * exp2_approx((z - st.m) * a.c) - st.c_t * t);
}
__device__ __forceinline__ bool ds_nothing(const DsStats& st) { return st.c_all == 0.f && st.c_t == 0.f; }

// A vector's elements to an address that need not be aligned to it
template <typename T>
__device__ __forceinline__ void store_vec(T* d, uint4 v, bool aligned) {
  if (aligned) {
    *reinterpret_cast<uint4*>(d) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (sizeof(T) == 4) {
      reinterpret_cast<uint32_t*>(d)[e] = w[e];
    } else {
      d[2 * e] = (T)(w[e] & 0xffffu);
      d[2 * e + 1] = (T)(w[e] >> 16);
    }
  }
}

constexpr int kDgU = 8;  // vectors per thread

// Each block takes kDsNT * kDgU vectors of a row; the first also the row's edges.  What
// it reads is in registers before it writes, so the gradient may take the logits' place.  The blocks
// wait for their list's three loads in a row, so many small ones are better: 2304 rows of 38016 bf16
// logits take 55.1 us with 128 threads of 8 vectors, 56.9 of 4, 59.0 with 256 of 4, 65 with 256 of 2.
template <typename T>
__global__ void __launch_bounds__(kDsNT) distill_grad_kernel(DsArgs a, int pieces) {
  constexpr int VE = Elem<T>::kVec;
  const int row = blockIdx.x / pieces, piece = blockIdx.x - row * pieces, tid = threadIdx.x;
  const T* l = static_cast<const T*>(a.logits) + (int64_t)row * a.ld;
  T* d = static_cast<T*>(a.grad) + (int64_t)row * a.ld_grad;
  const Span sp = span_of<T>(l, a.K, 0, 1);
  const DsStats st = a.stats[row];
  const float g = a.weight ? a.weight[row] : 1.f;
  const bool nothing = ds_nothing(st);
  const bool aligned = (reinterpret_cast<uintptr_t>(d + sp.head) & 15) == 0;
  const uint4* l4 = reinterpret_cast<const uint4*>(l + sp.head);
  const int q0 = piece * (kDsNT * kDgU) + tid;
  uint4 v[kDgU];
  if (!nothing) {
#pragma unroll
    for (int u = 0; u < kDgU; ++u)
      if (q0 + u * kDsNT < sp.nvec) v[u] = l4[q0 + u * kDsNT];
  }
  // the edges, and the listed ids that this block has
  const bool edge = piece == 0 && tid < 2 * VE && edge_id<VE>(sp, tid) < a.K;
  float xe = 0.f, z = 0.f, lp = 0.f;
  int p = -1;
  if (!nothing) {
    if (edge) xe = logit(l + edge_id<VE>(sp, tid));
    if (tid < a.k) {
      p = ds_place(a, (int64_t)row * a.k + tid);
      const int q = (p - sp.head) / VE;
      const bool inner = p >= sp.head && q < sp.nvec;
      if (p >= 0 && (inner ? q / (kDsNT * kDgU) != piece : piece != 0)) p = -1;
      if (p >= 0) {
        lp = a.logp[(int64_t)row * a.k + tid];
        z = logit(l + p);
        if (z == -INFINITY) p = -1;
      }
    }
    if (a.grad == a.logits) __syncthreads();
  }
  const float factor = g * st.c_rest;
#pragma unroll
  for (int u = 0; u < kDgU; ++u) {
    const int q = q0 + u * kDsNT;
    if (q < sp.nvec)
      store_vec(d + sp.head + (int64_t)q * VE,
                nothing ? make_uint4(0, 0, 0, 0) : Store<T>::grad(v[u], st.mr, a.c, factor), aligned);
  }
  if (edge) Store<T>::put(d + edge_id<VE>(sp, tid), nothing ? 0.f : factor * exp2_approx((xe - st.mr) * a.c));
  if (nothing) return;
  __syncthreads();
  if (p >= 0) Store<T>::put(d + p, ds_listed(a, st, g, z, pair_exp(Pair{lp, 0.f}).h));
}

// ------------------------------------------------------- loss, and with it the gradient
constexpr int kDtLists = 2;             // warps for the lists
template <int NW>
constexpr int kDtThreads = 32 * (NW + 1 + kDtLists);
constexpr int kDtU = 4;                 // vectors that a thread takes together
constexpr int kDtMaxC = 8;
constexpr int kDtZero = 2048;
constexpr int kDtRing = 4;              // rows whose lists and sums are in hand
constexpr int kDtStages = 4;

// a sum on its way between blocks; s = -1: a wait has run out
struct alignas(8) DtPart {
  float m, s;
};

template <int NW>
struct DtShared {
  DsList list[kDtRing];
  DsStats st[kDtRing];
  DsCells cells[kDtLists];
  DtPart got[kDtRing][kDtMaxC * (NW + 1)];  // the blocks' sums: their consuming warps', their edges'
  alignas(16) uint8_t zero[kDtZero];
  alignas(8) uint64_t full[kDtStages], done[kDtStages];  // chunks of the row in shared memory
  alignas(8) uint64_t listed[kDtRing], summed[kDtRing], ready[kDtRing], used[kDtRing];
  int timeout;
};

// an address in shared memory of a block of the cluster
__device__ __forceinline__ uint32_t map_block(const void* p, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(umma::smem_u32(p)), "r"(rank));
  return a;
}
// a sum to a block of the cluster, counted by its barrier
__device__ __forceinline__ void send_part(const DtPart& v, DtPart* to, uint64_t* bar, int rank) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(
                   map_block(to, rank)),
               "r"(__float_as_uint(v.m)), "r"(__float_as_uint(v.s)), "r"(map_block(bar, rank))
               : "memory");
}
__device__ __forceinline__ void arrive_block(uint64_t* bar, int rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(map_block(bar, rank)) : "memory");
}
// one poll for what other blocks have done
__device__ __forceinline__ bool try_parts(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(umma::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(umma::smem_u32(src)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }

struct DtSplit {
  int share, chunk, stages;  // vectors of a row in each block, bytes of a chunk, chunks in shared memory
};

// The row that a cluster has in turn n, of `stride` clusters: another place among that turn's rows each
// time, so that rows that take longer in a regular pattern (first positions of sequences) are shared out.
__device__ __forceinline__ int64_t dt_row(int cluster, int n, int stride) {
  return (int64_t)n * stride + (cluster + ((uint32_t)n * 0x9E3779B1u >> 16)) % (uint32_t)stride;
}

// A row per cluster and turn.  Each block has `share` of its vectors, in chunks: one warp
// copies them, NW sum the unlisted ids and send their sums to the blocks that need them, and
// of two more each has the list of every other row, which it reads ahead; it takes the sums
// together and finishes the row.
// With the gradient a part is one chunk, and stays in shared memory until the statistics are there,
// which takes longer than a sum: the consuming warps sum the next row meanwhile, then put the
// gradient in the logits' place, and the copying warp takes it out.  Every block finishes every row
// for itself.  Without the gradient the blocks finish rows in turn.
template <typename T, bool kGrad, int H, int NW>
__global__ void __launch_bounds__(kDtThreads<NW>, NW > kLpWarps ? 1 : H == 1 ? 3 : 2)
    distill_rows_kernel(DsArgs a, DtSplit split) {
  constexpr int NT = 32 * NW;    // consuming threads
  constexpr int kParts = NW + 1;
  constexpr int VE = Elem<T>::kVec;
  extern __shared__ __align__(16) uint8_t buf[];
  __shared__ DtShared<NW> sh;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cluster = blockIdx.x / C, stride = gridDim.x / C;
  const auto row_of = [&](int n) { return dt_row(cluster, n, stride); };
  const int turns = a.R / stride + (row_of(a.R / stride) < a.R ? 1 : 0);
  const auto row_at = [&](int n) { return n < turns ? row_of(n) : (int64_t)a.R; };  // (R: none)
  const int chunk = split.chunk, NS = split.stages;
  const bool first = rank == 0;  // has the rows' edges
  uint32_t limit = umma::kWaitLimit;
  // a bounded wait of a whole warp; one that gives up is noted and the next ones are short
  const auto late = [&](bool ok) {
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      limit = 1;
      if (lane == 0) atomicExch(&sh.timeout, 1);
    }
    return ok;
  };
  const auto wait = [&](uint64_t* bar, int phase) { return late(umma::mbar_wait(bar, phase & 1, limit)); };
  const auto wait_blocks = [&](uint64_t* bar, int phase) {
    bool ok = false;
    for (uint32_t i = 0; i < limit && !ok; ++i) ok = try_parts(bar, phase & 1);
    return late(ok);
  };
  const auto logits = [&](int row) { return static_cast<const T*>(a.logits) + (int64_t)row * a.ld; };
  const auto grads = [&](int row) { return static_cast<T*>(a.grad) + (int64_t)row * a.ld_grad; };
  // this block's vectors of a row
  struct Mine {
    int v0, n;
  };
  const auto mine_of = [&](const Span& sp) {
    const int v0 = min(rank * split.share, sp.nvec);
    return Mine{v0, min(split.share, sp.nvec - v0)};
  };
  if (tid == 0) {
    for (int s = 0; s < kDtStages; ++s) {
      umma::mbar_init(&sh.full[s], 1);
      umma::mbar_init(&sh.done[s], NW);
    }
    for (int s = 0; s < kDtRing; ++s) {
      umma::mbar_init(&sh.listed[s], 1);
      umma::mbar_init(&sh.summed[s], 1);
      umma::mbar_init(&sh.ready[s], 1);
      umma::mbar_init(&sh.used[s], NW);
    }
    sh.timeout = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (kGrad) {
    for (int i = tid; i < kDtZero / 4; i += kDtThreads<NW>) reinterpret_cast<uint32_t*>(sh.zero)[i] = 0;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (C > 1)
    cl.sync();  // every block's barriers are there
  else
    __syncthreads();

  if (warp == NW) {
    // copies, as far ahead of the consumers as there are chunks
    bool ok = true;
    int id[H], id1[H];           // the ids of this turn's row, and the next one's
    ds_ids<H>(a, row_at(0), lane, id);
    ds_ids<H>(a, row_at(1), lane, id1);
    int s = 0, lap = 0;          // the next chunk's place, and how often that has been gone round
    int held[kDtStages];         // the rows whose gradients the chunks will hold
#pragma unroll
    for (int i = 0; i < kDtStages; ++i) held[i] = -1;
    const auto put = [&](int at) {
      int row = -1;
#pragma unroll
      for (int i = 0; i < kDtStages; ++i)
        if (i == at) row = held[i];
      const Span sp = span_of<T>(logits(row), a.K, 0, 1);
      const Mine me = mine_of(sp);
      T* d = grads(row) + sp.head + (int64_t)me.v0 * VE;
      if ((reinterpret_cast<uintptr_t>(d) & 15) == 0) bulk_store(d, buf + (size_t)at * chunk, me.n * 16);
      bulk_commit();
    };
    for (int n = 0; n < turns; ++n) {
      const bool any = ds_any<H>(id);
      if (ok && lane == 0) {
        const int row = (int)row_of(n);
        const T* l = logits(row);
        const Span sp = span_of<T>(l, a.K, 0, 1);
        const Mine me = mine_of(sp);
        if (any) {
          const uint8_t* src = reinterpret_cast<const uint8_t*>(l + sp.head) + (int64_t)me.v0 * 16;
          for (int at = 0; at < me.n * 16; at += chunk) {
            if (lap > 0) {
              ok = umma::mbar_wait(&sh.done[s], (lap - 1) & 1);
              if (!ok) break;
              if (kGrad) {
                put(s);
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
              }
            }
#pragma unroll
            for (int i = 0; i < kDtStages; ++i)
              if (i == s) held[i] = row;
            const uint32_t bytes = (uint32_t)min(chunk, me.n * 16 - at);
            umma::mbar_expect_tx(&sh.full[s], bytes);
            umma::bulk_load(buf + (size_t)s * chunk, src + at, bytes, &sh.full[s]);
            if (++s == NS) s = 0, ++lap;
          }
        } else if (kGrad) {
          T* d = grads(row) + sp.head + (int64_t)me.v0 * VE;
          if ((reinterpret_cast<uintptr_t>(d) & 15) == 0)
            for (int at = 0; at < me.n * 16; at += kDtZero)
              bulk_store(reinterpret_cast<uint8_t*>(d) + at, sh.zero, min(kDtZero, me.n * 16 - at));
          bulk_commit();
        }
      }
#pragma unroll
      for (int h = 0; h < H; ++h) id[h] = id1[h];
      ds_ids<H>(a, row_at(n + 2), lane, id1);
    }
    if (kGrad && lane == 0) {
      // the last rows' gradients, oldest first
      const int filled = lap > 0 ? NS : s;
      for (int i = 0; i < filled && ok; ++i) {
        const int at = lap > 0 ? (s + i) % NS : i;
        ok = umma::mbar_wait(&sh.done[at], (at < s ? lap : lap - 1) & 1);
        if (ok) put(at);
      }
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    if (!ok) {
      atomicExch(&sh.timeout, 1);
      // every copy issued has landed before this block may exit
      for (int i = 0; i < kDtStages; ++i)
        for (int par = 0; par < 2; ++par) umma::mbar_wait(&sh.full[i], par, 1u << 12);
    }
    __syncwarp();
  } else if (warp > NW) {
    // the lists: one warp has the even turns, the other the odd ones.  A row's statistics are what the
    // consuming warps wait for, so all else of a turn is done ahead: at row n's turn its own list has
    // been taken in, the values of row n + 2 arrive, and row n + 4's ids.  (Long code here costs the
    // consuming warps their instruction cache: with the loops over pairs unrolled and the exponential
    // inlined the training batch of 2048 rows took 102 instead of 92.5 us.)
    const int mod = C % 4 == 0 ? C : C % 2 == 0 ? 2 * C : 4 * C;  // turns between two uses of a sums' place
    DsCells& cells = sh.cells[warp - NW - 1];
    int n = warp - NW - 1;
    const auto finishes = [&](int n) { return kGrad || n % C == rank; };
    // row n's places to the consuming warps
    const auto publish = [&](const DsEntries<H>& e, int64_t row, int n) {
      if (row >= a.R) return;
      DsList& list = sh.list[n & 3];
      const Span sp = span_of<T>(logits((int)row), a.K, 0, 1);
      const Mine me = mine_of(sp);
      if (n >= kDtRing) wait(&sh.used[n & 3], (n >> 2) - 1);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int i = lane + 32 * h, x = e.p[h] - sp.head, v = x / VE - me.v0;
        if (i < a.k)
          list.pos[i] = e.p[h] < 0 || x < 0 || v < 0 || v >= me.n ? -1 : v * 16 + (x % VE) * (int)sizeof(T);
      }
      if (lane == 0) list.any = e.any;
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(&sh.listed[n & 3]);
    };
    // what row n's list says, and the row's edges, one per lane: their sum goes to where the others
    // go.  (When all sums are there this warp has read what it reads of the row, and the gradient may
    // take the logits' place.)
    struct Edges {
      float x;      // -infinity: none
      bool here, unlisted;
    };
    const auto send_ends = [&](const DsEntries<H>& e, int64_t row, int n, Edges& edge) {
      if (row >= a.R) return;
      DtPart ends{-INFINITY, 0.f};
      edge = Edges{-INFINITY, false, false};
      if (first) {
        const T* l = logits((int)row);
        const Span sp = span_of<T>(l, a.K, 0, 1);
        edge.here = lane < 2 * VE && edge_id<VE>(sp, lane) < a.K;
        if (e.any && __any_sync(0xffffffffu, edge.here)) {
          unsigned listed = 0;
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const int t = ds_edge<VE>(sp, e.p[h]);
            if (t >= 0) listed |= 1u << t;
          }
          listed = __reduce_or_sync(0xffffffffu, listed);
          edge.unlisted = edge.here && !(listed >> lane & 1);
          if (edge.unlisted) edge.x = logit(l + edge_id<VE>(sp, lane));
          ends.m = warp_max_nan(edge.x);
          const float w = exp2_approx((edge.x - ends.m) * a.c);
          ends.s = ends.m == -INFINITY ? 0.f : warp_add(w);
        }
      }
      const int slot = n & 3;
      if (finishes(n) && lane == 0)
        umma::mbar_expect_tx(&sh.summed[slot], (uint32_t)(C * kParts * sizeof(DtPart)));
      // A place for sums is taken again after four turns, when all blocks have read it: as each has said
      // (without the gradient), or as those have that have sent their sums of row n - 2, which this warp has
      if (!kGrad && n >= kDtRing) wait_blocks(&sh.ready[slot], (n >> 2) - 1);
      if (kGrad ? lane < C : lane == 0)
        send_part(ends, &sh.got[slot][rank * kParts + NW], &sh.summed[slot], kGrad ? lane : n % C);
    };
    DsEntries<H> e{}, next;
    int id[H];
    ds_ids<H>(a, row_at(n), lane, id);
    ds_map<H>(a, id, next);
    ds_ids<H>(a, row_at(n + 2), lane, id);
    Edges edge{};
    DsHead hd{};
    for (n -= 2; n < turns; n += 2) {  // (the first time round takes in the first row alone)
      const int row = n < 0 ? 0 : (int)row_of(n), slot = n & 3;
      const int64_t after = row_at(n + 2);
      if (finishes(n + 2)) ds_values<T, H>(a, after, lane, next);
      DsStats st{0.f, 0.f, 0.f, 0.f, 0.f};
      DsTotal r{};
      DsSum un{-INFINITY, 0.f, 0};
      constexpr int kMost = (kDtMaxC * kParts + 31) / 32;
      float pm[kMost], ps[kMost];
      if (n >= 0 && finishes(n)) {
        const float g = kGrad && a.weight ? __ldg(a.weight + row) : 1.f;
        un.late = !wait_blocks(&sh.summed[slot], kGrad ? n >> 2 : n / mod);
#pragma unroll
        for (int h = 0; h < kMost; ++h) {
          const int i = lane + 32 * h;
          DtPart v{-INFINITY, 0.f};
          if (i < C * kParts) v = sh.got[slot][i];
          un.late |= v.s < 0.f;
          pm[h] = v.m;
          ps[h] = v.s;
          un.m = max_nan(un.m, v.m);
        }
        un.m = warp_max_nan(un.m);
        un.late = __any_sync(0xffffffffu, un.late != 0);
        // (0 and -infinity where nothing was summed)
#pragma unroll
        for (int h = 0; h < kMost; ++h) {
          ps[h] = ps[h] == 0.f ? 0.f : ps[h] * exp2_approx((pm[h] - un.m) * a.c);
          un.s += ps[h];
        }
        un.s = warp_add(un.s);
        if (!kGrad && lane < C) arrive_block(&sh.ready[slot], lane);  // the sums' place is free
        if (e.any) r = ds_stats(a, hd, un, st);
        if (kGrad) {
          const float all = g * st.c_all * (r.learns ? exp2_approx((hd.m - st.m) * a.c) : 1.f), ct = g * st.c_t;
#pragma unroll
          for (int h = 0; h < H; ++h) {
            e.lp[h] = all * e.z[h] - ct * e.lp[h];
            if (lane + 32 * h < a.k) sh.list[slot].val[lane + 32 * h] = e.lp[h];
          }
          if (lane == 0) sh.st[slot] = st;
          __syncwarp();
          if (lane == 0) umma::mbar_arrive(&sh.ready[slot]);
          if (first) {
            // the edges' gradients
            T* d = grads(row);
            const Span sp = span_of<T>(logits(row), a.K, 0, 1);
            const bool nothing = ds_nothing(st);
            if (edge.here && (nothing || edge.unlisted))
              Store<T>::put(d + edge_id<VE>(sp, lane),
                            nothing ? 0.f : g * st.c_rest * exp2_approx((edge.x - st.mr) * a.c));
            if (!nothing)
#pragma unroll
              for (int h = 0; h < H; ++h)
                if (ds_edge<VE>(sp, e.p[h]) >= 0) Store<T>::put(d + e.p[h], e.lp[h]);
          }
        }
      }
      // the next row's places, and what its sums wait for, ahead of this row's loss
      publish(next, after, n + 2);
      const bool learns = e.any, counts = n >= 0 && n % C == rank;
      e = next;
      ds_map<H>(a, id, next);
      ds_ids<H>(a, row_at(n + 6), lane, id);
      const bool more = finishes(n + 2) && e.any;
      const int flags = more ? ds_flags<H>(e, cells, lane) : 0;
      send_ends(e, after, n + 2, edge);
      if (counts) {
        Pair sr{0.f, 0.f};
#pragma unroll
        for (int h = 0; h < kMost; ++h) sr = pair_add(sr, Pair{ps[h], 0.f});
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1) sr = pair_add(sr, pair_xor(sr, o));
        const float loss = learns ? ds_loss(a, hd, un, sr, st, r, lane) : 0.f;
        if (lane == 0) ds_put(a, row, loss, st, r.flags);
        __syncwarp();
      }
      hd = more ? ds_head<H>(a, e, flags) : DsHead{};
    }
  } else {
    int in_at = 0, in_lap = 0, out_at = 0;  // chunks' places
    // sums row n and sends the sum
    const auto sum_row = [&](int row, int n) {
      const int slot = n & 3;
      const DsList& list = sh.list[slot];
      const Span sp = span_of<T>(logits(row), a.K, 0, 1);
      const Mine me = mine_of(sp);
      wait(&sh.listed[slot], n >> 2);
      RowSum sum{kNegBig, 0.f, 0.f};
      if (list.any)
        for (int at = 0; at < me.n * 16; at += chunk) {
          const int s = in_at, have = min(chunk, me.n * 16 - at) / 16;
          uint8_t* const b = buf + (size_t)s * chunk;
          const uint4* in = reinterpret_cast<const uint4*>(b);
          wait(&sh.full[s], in_lap);
          if (++in_at == NS) in_at = 0, ++in_lap;
          ds_each<NW>(list, at, chunk, a.k, warp, lane, [&](int, int q) {
            *reinterpret_cast<decltype(Mask<T>::bits())*>(b + q) = Mask<T>::bits();
            // ahead of the next copy into this place
            if (!kGrad) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          });
          const auto add = [&](const auto& v) {
            const float pm = Vec<T>::top(v);
            if (!(pm <= sum.m)) sum_rescale(sum, max_nan(sum.m, pm), a.c);
            sum_add<T>(sum, v, a.c);
          };
          int q = tid;
          for (; q + (kDtU - 1) * NT < have; q += kDtU * NT) {
            uint4 v[kDtU];
#pragma unroll
            for (int u = 0; u < kDtU; ++u) v[u] = in[q + u * NT];
            add(v);
          }
          for (; q < have; q += NT) {
            const uint4 v[1] = {in[q]};
            add(v);
          }
          if (!kGrad) {
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&sh.done[s]);
          }
        }
      // (a row that is not read is exchanged too, so that no block gets ahead of another: a place for
      // sums is taken again after four turns, when all blocks have read it)
      const RowSum w = warp_join(sum, a.c);
      if (!kGrad && n >= kDtRing) wait_blocks(&sh.ready[slot], (n >> 2) - 1);
      const DtPart part{w.m, *reinterpret_cast<volatile int*>(&sh.timeout) ? -1.f : w.s};
      if (kGrad ? lane < C : lane == 0)
        send_part(part, &sh.got[slot][rank * kParts + warp], &sh.summed[slot], kGrad ? lane : n % C);
      if (!kGrad) {
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&sh.used[slot]);
      }
    };
    // the gradient of row n
    const auto grad_row = [&](int row, int n) {
      const int slot = n & 3;
      const DsList& list = sh.list[slot];
      const Span sp = span_of<T>(logits(row), a.K, 0, 1);
      const Mine me = mine_of(sp);
      T* const out = grads(row) + sp.head + (int64_t)me.v0 * VE;
      const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
      const float g = a.weight ? __ldg(a.weight + row) : 1.f;
      wait(&sh.ready[slot], n >> 2);
      if (list.any && me.n > 0) {
        const int s = out_at;
        if (++out_at == NS) out_at = 0;
        uint8_t* const b = buf + (size_t)s * chunk;
        uint4* const in = reinterpret_cast<uint4*>(b);
        const DsStats st = sh.st[slot];
        const bool nothing = ds_nothing(st);
        const float factor = g * st.c_rest;
#pragma unroll 4
        for (int q = tid; q < me.n; q += NT)
          in[q] = nothing ? make_uint4(0, 0, 0, 0) : Store<T>::grad(in[q], st.mr, a.c, factor);
        __syncwarp();
        if (!nothing)
          ds_each<NW>(list, 0, chunk, a.k, warp, lane,
                  [&](int i, int q) { Store<T>::put(reinterpret_cast<T*>(b + q), list.val[i]); });
        if (!aligned)
          for (int q = tid; q < me.n; q += NT) store_vec(out + (int64_t)q * VE, in[q], false);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&sh.done[s]);
      } else if (!list.any && !aligned) {
        for (int q = tid; q < me.n; q += NT) store_vec(out + (int64_t)q * VE, make_uint4(0, 0, 0, 0), false);
      }
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(&sh.used[slot]);
    };
    if (kGrad && turns > 0) sum_row((int)row_of(0), 0);
    for (int n = 0; n < turns; ++n) {
      if (!kGrad) {
        sum_row((int)row_of(n), n);
      } else {
        if (n + 1 < turns) sum_row((int)row_of(n + 1), n + 1);
        grad_row((int)row_of(n), n);
      }
    }
  }
  if (C > 1) cl.sync();  // nothing more is sent to a block that has left
}

// arguments that the three calls share
int ds_check(const void* logits, int32_t dtype, int64_t R, int32_t K, int64_t ld, const int32_t* ids,
             const float* logp, int32_t k, int32_t V, const int32_t* inv_map, float T, const float* stats) {
  if (!logits || !ids || !logp || !stats) return VT_ERR_INVALID_ARG;
  if (dtype != VT_F32 && dtype != VT_BF16) return VT_ERR_INVALID_ARG;
  if (R < 1 || R > (1 << 24) || K < 1 || K > (1 << 22) || ld < K) return VT_ERR_INVALID_ARG;
  if (k < 1 || k > kDsMaxK || V < 1 || (!inv_map && V != K)) return VT_ERR_INVALID_ARG;
  if (!(T >= 1e-30f && T <= 1e30f)) return VT_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == VT_F32 ? 4 : 2) != 0) return VT_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(stats) % 4 != 0) return VT_ERR_INVALID_ARG;
  return VT_OK;
}
// the gradient's buffer: the logits' own, or apart from them
int ds_check_grad(const void* logits, int32_t dtype, int64_t R, int32_t K, int64_t ld, const void* grad,
                  int64_t ld_grad) {
  const int elem = dtype == VT_F32 ? 4 : 2;
  if (!grad || ld_grad < K || reinterpret_cast<uintptr_t>(grad) % elem != 0) return VT_ERR_INVALID_ARG;
  if (grad == logits && (ld_grad == ld || R == 1)) return VT_OK;
  const uintptr_t l0 = reinterpret_cast<uintptr_t>(logits), g0 = reinterpret_cast<uintptr_t>(grad);
  const uintptr_t l1 = l0 + (uintptr_t)((R - 1) * ld + K) * elem, g1 = g0 + (uintptr_t)((R - 1) * ld_grad + K) * elem;
  return l0 < g1 && g0 < l1 ? VT_ERR_INVALID_ARG : VT_OK;
}

DsArgs ds_args(const void* logits, int64_t R, int32_t K, int64_t ld, const int32_t* ids, const float* logp,
               int32_t k, int32_t V, const int32_t* inv_map, int32_t rest, float T, const float* weight,
               float* out_loss, float* stats, void* grad, int64_t ld_grad, int32_t* dev_status) {
  DsArgs a;
  a.logits = logits;
  a.ld = ld;
  a.R = (int)R;
  a.K = K;
  a.V = V;
  a.k = k;
  a.rest = rest != 0;
  a.c = VT_LOG2E / T;
  double twice = 2.0 / (double)T;
  a.unit = 1.f;
  for (; twice > 1.0; twice *= 0.5) a.unit *= 2.f;
  a.inv_t = (float)(1.0 / (double)T);
  a.twice.h = (float)twice;
  a.twice.l = (float)(twice - (double)a.twice.h);
  a.ids = ids;
  a.logp = logp;
  a.inv_map = inv_map;
  a.weight = weight;
  a.out_loss = out_loss;
  a.stats = reinterpret_cast<DsStats*>(stats);
  a.grad = grad;
  a.ld_grad = ld_grad;
  a.dev_status = dev_status;
  a.own_status = R == 1;
  return a;
}

int ds_launch_grad(const DsArgs& a, int32_t dtype, cudaStream_t s) {
  const int elem = dtype == VT_F32 ? 4 : 2;
  const int pieces = std::max(1, (int)(((int64_t)a.K * elem / 16 + kDsNT * kDgU - 1) / (kDsNT * kDgU)));
  if ((int64_t)a.R * pieces > 0x7fffffff) return VT_ERR_UNSUPPORTED;
  if (elem == 4)
    distill_grad_kernel<float><<<(unsigned)a.R * pieces, kDsNT, 0, s>>>(a, pieces);
  else
    distill_grad_kernel<uint16_t><<<(unsigned)a.R * pieces, kDsNT, 0, s>>>(a, pieces);
  VT_RETURN_IF_LAUNCH_FAILED();
  return VT_OK;
}

// How a row is spread: C blocks with `share` vectors each, in chunks; kDtBytes[tier] bytes of them
// leave room for 3 - tier blocks on an SM.
struct DtPlan {
  int C, tier;
  DtSplit split;
};
constexpr int kDtBytes[3] = {64 << 10, 100 << 10, 200 << 10};

// With the gradient a part is one chunk, two or three of them are in work.  A turn costs about 2500
// cycles besides its bytes, and clusters of many blocks do not fill the device (76 pairs fit where 51
// clusters of eight do), so: whole rows in one block where they fit (several on an SM), else few large
// parts.  us, before the loss's sums were pairs, at 2048 rows of 32768 fp32 logits: 2 blocks with 3 x 64 KB 89, 4 with 3 x 32 89 (two on an
// SM), 4 with 2 x 32 102 (three), 6 with 3 x 21 127.  2304 rows of 32003 bf16: 1 with 3 x 64 62, 2 with
// 3 x 32 75, 3 with 3 x 21 80.  4000 rows of 2000 fp32: three blocks on an SM 34, two 39, one 57.
// false: the row does not fit.
bool dt_plan_grad(int64_t R, int64_t bytes, DtPlan& p) {
  const auto fits = [&](int tier, int stages, int C) {
    p.tier = tier;
    p.split.stages = stages;
    p.C = C;
    return (bytes / 16 + C - 1) / C * 16 * stages <= kDtBytes[tier];
  };
  bool ok = fits(0, 3, 1) || fits(1, 3, 1) || fits(1, 2, 1);
  for (int stages = 3; stages >= 2 && !ok; --stages)
    for (int C = 1; C <= kDtMaxC && !ok; ++C) ok = fits(2, stages, C);
  if (!ok) return false;
  // few rows: more blocks to each
  while (p.C < kDtMaxC && R * p.C * 2 <= num_sms() * (3 - p.tier) && bytes / p.C > (4 << 10))
    p.C = std::min(p.C * 2, kDtMaxC);
  p.split.share = std::max(1, (int)((bytes / 16 + p.C - 1) / p.C));
  p.split.chunk = p.split.share * 16;
  return true;
}

// Without it a block streams its part through two chunks of 32 KB, three blocks on an SM.  The number of
// blocks to a row is the one with the shortest schedule, a turn taking its chunks and one more, or two
// where sums go between blocks (before the loss's sums were pairs, 2304 rows of 38016 bf16 logits: 1 block
// 37 us, 2 43, 3 47; 112 rows of 128256 fp32, 59 of them scored: 3 blocks 11.8 us, 4 10.4, 8 11.2).  Lists of
// more than 32 leave room for two blocks on an SM only.  The schedule counts three for them too: counted as two, 160 rows
// of 38016 bf16 take 10.6 instead of 11.4 us and 60 of 128256 12.5 instead of 11.5.
DtPlan dt_plan_loss(int64_t R, int64_t bytes) {
  DtPlan p;
  p.tier = 0;
  p.split.stages = 2;
  const int part = kDtBytes[0] / p.split.stages;
  const int64_t slots = num_sms() * 3;
  double least = 0.0;
  for (int C = 1; C <= kDtMaxC && (C == 1 || bytes / C > (4 << 10)); ++C) {
    const double t = (double)((R * C + slots - 1) / slots) * ((double)bytes / C / part + (C == 1 ? 1 : 2));
    if (C == 1 || t < least) {
      least = t;
      p.C = C;
    }
  }
  p.split.share = std::max(1, (int)((bytes / 16 + p.C - 1) / p.C));
  const int chunks = (int)(((int64_t)p.split.share * 16 + part - 1) / part);
  p.split.chunk = (p.split.share + chunks - 1) / chunks * 16;  // evenly
  return p;
}

template <typename T, bool kGrad, int H, int NW>
int ds_launch_rows(const DsArgs& a, cudaStream_t s, const DtPlan& p) {
  auto kern = distill_rows_kernel<T, kGrad, H, NW>;
  VT_RETURN_IF_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kDtBytes[2]));
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kDtThreads<NW>);
  cfg.dynamicSmemBytes = (size_t)kDtBytes[p.tier];
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // clusters that run at once, by device and spread: a property of the device, asked once
  static std::atomic<int> cache[64][3][kDtMaxC];
  int dev = 0;
  VT_RETURN_IF_CUDA(cudaGetDevice(&dev));
  int clusters = dev < 64 ? cache[dev][p.tier][p.C - 1].load(std::memory_order_relaxed) : 0;
  if (clusters == 0) {
    cfg.gridDim = dim3((unsigned)(p.C * num_sms() * 3));
    VT_RETURN_IF_CUDA(cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg));
    if (clusters < 1) return VT_ERR_CUDA;
    if (dev < 64) cache[dev][p.tier][p.C - 1].store(clusters, std::memory_order_relaxed);
  }
  if (!a.own_status) {
    const int st = clear_status(s, a.dev_status);
    if (st != VT_OK) return st;
  }
  cfg.gridDim = dim3((unsigned)(std::min(a.R, clusters) * p.C));
  cfg.numAttrs = a.own_status ? 1 : 2;
  VT_RETURN_IF_CUDA(cudaLaunchKernelEx(&cfg, kern, a, p.split));
  return VT_OK;
}
template <typename T, bool kGrad, int H>
int ds_launch_rows(const DsArgs& a, cudaStream_t s, const DtPlan& p) {
  // one block on an SM: twice the warps
  if (kGrad && p.tier == 2) return ds_launch_rows<T, kGrad, H, kGrad ? 2 * kLpWarps : kLpWarps>(a, s, p);
  return ds_launch_rows<T, kGrad, H, kLpWarps>(a, s, p);
}
template <bool kGrad>
int ds_launch_rows(const DsArgs& a, int32_t dtype, cudaStream_t s, const DtPlan& p) {
  if (a.k <= 32)
    return dtype == VT_F32 ? ds_launch_rows<float, kGrad, 1>(a, s, p) : ds_launch_rows<uint16_t, kGrad, 1>(a, s, p);
  return dtype == VT_F32 ? ds_launch_rows<float, kGrad, kDsMaxK / 32>(a, s, p)
                         : ds_launch_rows<uint16_t, kGrad, kDsMaxK / 32>(a, s, p);
}

int ds_launch_loss(const DsArgs& a, int32_t dtype, cudaStream_t s) {
  const DtPlan p = dt_plan_loss(a.R, (int64_t)a.K * (dtype == VT_F32 ? 4 : 2));
  return ds_launch_rows<false>(a, dtype, s, p);
}

// Rows that the blocks of a cluster hold between them are read once; longer ones take the two calls.
int ds_launch_both(const DsArgs& a, int32_t dtype, cudaStream_t s) {
  DtPlan p;
  if (!dt_plan_grad(a.R, (int64_t)a.K * (dtype == VT_F32 ? 4 : 2), p)) {
    const int rc = ds_launch_loss(a, dtype, s);
    return rc != VT_OK ? rc : ds_launch_grad(a, dtype, s);
  }
  return ds_launch_rows<true>(a, dtype, s, p);
}

}  // namespace
}  // namespace vt

extern "C" int vt_distill_loss(const void* logits, int32_t logits_dtype, int64_t R, int32_t K,
                               int64_t ld_logits, const int32_t* top_ids, const float* top_logp, int32_t k,
                               const int32_t* inv_map, int32_t V, int32_t rest, float temperature,
                               float* out_loss, float* out_stats, int32_t* dev_status, void* stream) {
  using namespace vt;
  const int st = ds_check(logits, logits_dtype, R, K, ld_logits, top_ids, top_logp, k, V, inv_map, temperature,
                          out_stats);
  if (st != VT_OK) return st;
  if (!out_loss || !dev_status || (rest != 0 && rest != 1)) return VT_ERR_INVALID_ARG;
  return ds_launch_loss(ds_args(logits, R, K, ld_logits, top_ids, top_logp, k, V, inv_map, rest, temperature,
                                nullptr, out_loss, out_stats, nullptr, 0, dev_status),
                        logits_dtype, static_cast<cudaStream_t>(stream));
}

extern "C" int vt_distill_grad(const void* logits, int32_t logits_dtype, int64_t R, int32_t K,
                               int64_t ld_logits, const int32_t* top_ids, const float* top_logp, int32_t k,
                               const int32_t* inv_map, int32_t V, float temperature, const float* stats,
                               const float* grad_loss, void* out_grad, int64_t ld_grad, void* stream) {
  using namespace vt;
  int st = ds_check(logits, logits_dtype, R, K, ld_logits, top_ids, top_logp, k, V, inv_map, temperature, stats);
  if (st == VT_OK) st = ds_check_grad(logits, logits_dtype, R, K, ld_logits, out_grad, ld_grad);
  if (st != VT_OK) return st;
  return ds_launch_grad(ds_args(logits, R, K, ld_logits, top_ids, top_logp, k, V, inv_map, 0, temperature,
                                grad_loss, nullptr, const_cast<float*>(stats), out_grad, ld_grad, nullptr),
                        logits_dtype, static_cast<cudaStream_t>(stream));
}

extern "C" int vt_distill_loss_grad(const void* logits, int32_t logits_dtype, int64_t R, int32_t K,
                                    int64_t ld_logits, const int32_t* top_ids, const float* top_logp, int32_t k,
                                    const int32_t* inv_map, int32_t V, int32_t rest, float temperature,
                                    const float* grad_loss, float* out_loss, float* out_stats, void* out_grad,
                                    int64_t ld_grad, int32_t* dev_status, void* stream) {
  using namespace vt;
  int st = ds_check(logits, logits_dtype, R, K, ld_logits, top_ids, top_logp, k, V, inv_map, temperature,
                    out_stats);
  if (st == VT_OK) st = ds_check_grad(logits, logits_dtype, R, K, ld_logits, out_grad, ld_grad);
  if (st != VT_OK) return st;
  if (!out_loss || !dev_status || (rest != 0 && rest != 1)) return VT_ERR_INVALID_ARG;
  const DsArgs a = ds_args(logits, R, K, ld_logits, top_ids, top_logp, k, V, inv_map, rest, temperature, grad_loss,
                           out_loss, out_stats, out_grad, ld_grad, dev_status);
  return ds_launch_both(a, logits_dtype, static_cast<cudaStream_t>(stream));
}
