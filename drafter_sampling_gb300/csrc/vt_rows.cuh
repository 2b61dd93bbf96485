// Streaming of rows of logits by thread blocks, and their k best ids, shared by the
// kernels that read whole rows (log probabilities, beam search, distillation).
//
// A row is taken in 32 KB chunks that one warp copies into a ring of shared
// memory and kLpWarps warps consume; ids are kept as 64-bit keys ordered by (value,
// lower id first).
#pragma once

#include "vt_internal.h"
#include "vt_pair.cuh"
#include "vt_verify_common.cuh"

namespace vt {

constexpr int kLpNT = 256;           // consuming threads
constexpr int kLpWarps = kLpNT / 32;
constexpr int kLpU = 8;              // 16-byte vectors per thread and chunk
constexpr int kLpChunk = kLpNT * kLpU * 16;  // bytes
constexpr int kLpStages = 2;
constexpr int kLpMaxK = 32;
constexpr int kLpList = 64;          // entries of a warp's list (2 * kLpMaxK: a cut leaves room)
constexpr int kLpMaxC = 8;
constexpr int kLpSmem = kLpStages * kLpChunk;
constexpr int kLpPerSm = 3;          // resident blocks per SM (shared memory)

// Order key of (value, id): higher value first, then lower id; 0 is after
// every key.  -0 counts as 0.
typedef unsigned long long lp_key;
__device__ __forceinline__ uint32_t lp_ord(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ lp_key key_of(float v, int id) {
  return (lp_key)lp_ord(v) << 32 | (uint32_t)~id;
}
__device__ __forceinline__ float key_value(lp_key q) {
  const uint32_t o = (uint32_t)(q >> 32);
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ int key_id(lp_key q) { return (int)~(uint32_t)q; }

// how many of the n keys at `keys` come before q; keys is 16-byte aligned and
// zero from n up to the next multiple of 8
__device__ __forceinline__ int count_before(const lp_key* keys, int n, lp_key q) {
  int r = 0;
  for (int o = 0; o < n; o += 8) {
#pragma unroll
    for (int h = 0; h < 8; h += 2) {
      const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(keys + o + h);
      r += (two.x > q ? 1 : 0) + (two.y > q ? 1 : 0);
    }
  }
  return r;
}

// larger of two, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// two fp32 values in one 64-bit register, and arithmetic on both at once
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// the largest of a 16-byte vector's elements, NaN if one is
template <typename T> struct Vec;
template <> struct Vec<float> {
  __device__ static float top(uint4 v) {
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                   max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  template <int U>
  __device__ static float top(const uint4 (&v)[U]) {
    float m = top(v[0]);
#pragma unroll
    for (int u = 1; u < U; ++u) m = max_nan(m, top(v[u]));
    return m;
  }
  // elements e, e + 1 of a vector, plus s
  __device__ static f32x2 diff2(uint4 v, int e, float s) {
    return add2(e == 0 ? pack2(__uint_as_float(v.x), __uint_as_float(v.y))
                       : pack2(__uint_as_float(v.z), __uint_as_float(v.w)),
                pack2(s, s));
  }
  static constexpr uint32_t kMasked = 0xff800000u;  // -infinity
};
template <> struct Vec<uint16_t> {
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ static float top(uint4 v) {
    const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  template <int U>
  __device__ static float top(const uint4 (&v)[U]) {
    uint32_t m = max2(max2(v[0].x, v[0].y), max2(v[0].z, v[0].w));
#pragma unroll
    for (int u = 1; u < U; ++u)
      m = max2(m, max2(max2(v[u].x, v[u].y), max2(v[u].z, v[u].w)));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  // elements e, e + 1 of a vector, plus s: bf16 operands widened by the addition
  __device__ static f32x2 diff2(uint4 v, int e, float s) {
    const uint32_t w = e == 0 ? v.x : e == 2 ? v.y : e == 4 ? v.z : v.w;
    float a, b;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "add.rn.f32.bf16 %0, lo, %3;\n\tadd.rn.f32.bf16 %1, hi, %3;\n\t}"
        : "=f"(a), "=f"(b)
        : "r"(w), "f"(s));
    return pack2(a, b);
  }
  static constexpr uint32_t kMasked = 0xff80ff80u;
};

// Ranks a warp's list of n keys by counting and cuts it to its k best, in
// order; returns how many are left.
static __device__ __noinline__ int list_cut(lp_key* list, int n, int k) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  lp_key q[kLpList / 32];
  int r[kLpList / 32];
#pragma unroll
  for (int h = 0; h < kLpList / 32; ++h) {
    const int j = lane + 32 * h;
    q[h] = j < n ? list[j] : 0;
    r[h] = j < n ? 0 : k;
  }
  for (int o = 0; o < n; ++o) {
    const lp_key other = list[o];
#pragma unroll
    for (int h = 0; h < kLpList / 32; ++h) r[h] += other > q[h] ? 1 : 0;
  }
  __syncwarp();
#pragma unroll
  for (int h = 0; h < kLpList / 32; ++h)
    if (r[h] < k) list[r[h]] = q[h];
  __syncwarp();
  return min(n, k);
}

// the k-th largest of the 32 lanes' values (1 <= k <= 32), by a bitonic sort
__device__ __forceinline__ float kth_of_lanes(float v, int k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      const float o = __shfl_xor_sync(0xffffffffu, v, stride);
      v = ((lane & size) == 0) == ((lane & stride) == 0) ? fmaxf(v, o) : fminf(v, o);
    }
  return __shfl_sync(0xffffffffu, v, k - 1);
}

// the consuming warps' barrier
__device__ __forceinline__ void lp_bar() {
  asm volatile("bar.sync 1, %0;" ::"n"(kLpNT) : "memory");
}

// A row's layout for one block: ids [0, head) precede the first 16-byte
// boundary, nvec whole vectors follow, then the rest; mine of the vectors'
// chunks are this block's.
struct Span {
  int head, nvec, mine;
};
template <typename T>
__device__ __forceinline__ Span span_of(const T* l, int V, int rank, int C) {
  constexpr int VE = Elem<T>::kVec;
  const int off = (int)((reinterpret_cast<uintptr_t>(l) & 15) / sizeof(T));
  Span sp;
  sp.head = min(V, off ? VE - off : 0);
  sp.nvec = (V - sp.head) / VE;
  const int chunks = (sp.nvec + kLpNT * kLpU - 1) / (kLpNT * kLpU);
  sp.mine = chunks > rank ? (chunks - rank + C - 1) / C : 0;
  return sp;
}

// the id of a row's edge element t: first those before the vectors, then those behind
template <int VE>
__device__ __forceinline__ int edge_id(const Span& sp, int t) {
  return t < sp.head ? t : sp.nvec * VE + t;
}

// What the consuming warps share of a row's best ids
struct RowLists {
  alignas(16) lp_key list[kLpWarps][kLpList];        // the warps' lists
  alignas(16) lp_key all[kLpWarps * kLpList + 8];    // all lists, joined
  alignas(16) lp_key best[kLpMaxK];                  // this block's k best, as published
  alignas(16) float group[32];                       // largest logit of each of 32 groups of threads
  int n[kLpWarps];
};

// Joins the warps' lists (n entries in this warp's, of which those not after
// `bound` count) into the block's k best, ranked in sh.best (zero behind the
// last).  All consuming warps call it.
__device__ __forceinline__ void lists_join(RowLists& sh, int n, lp_key bound, int k, int warp,
                                           int lane) {
  lp_key mine[kLpList / 32];
  __syncwarp();
#pragma unroll
  for (int h = 0; h < kLpList / 32; ++h) {
    const int j = lane + 32 * h;
    mine[h] = j < n ? sh.list[warp][j] : 0;
    if (mine[h] < bound) mine[h] = 0;
  }
  unsigned has[kLpList / 32];
  n = 0;
#pragma unroll
  for (int h = 0; h < kLpList / 32; ++h) {
    has[h] = __ballot_sync(0xffffffffu, mine[h] != 0);
    n += __popc(has[h]);
  }
  if (lane == 0) sh.n[warp] = n;
  if (warp == 0) sh.best[lane] = 0;
  lp_bar();
  int at = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kLpWarps; ++w) {
    const int nw = sh.n[w];
    at += w < warp ? nw : 0;
    total += nw;
  }
#pragma unroll
  for (int h = 0; h < kLpList / 32; ++h) {
    if (mine[h] != 0) sh.all[at + __popc(has[h] & ((1u << lane) - 1u))] = mine[h];
    at += __popc(has[h]);
  }
  if (warp == kLpWarps - 1 && lane < 8) sh.all[total + lane] = 0;
  lp_bar();
  for (int j = warp * 32 + lane; j < total; j += kLpNT) {
    const lp_key q = sh.all[j];
    const int r = count_before(sh.all, total, q);
    if (r < k) sh.best[r] = q;
  }
}

// A warp's list: n keys that are not after `bound`, whose value is tv
struct TopList {
  lp_key* list;
  int n;
  lp_key bound;
  float tv;

  // one id per lane
  __device__ __forceinline__ void add(float x, int id, bool valid, int k, int lane) {
    if (!__any_sync(0xffffffffu, valid && x >= tv)) return;  // a NaN is none
    const lp_key q = key_of(x, id);
    const bool take = valid && x >= tv && q >= bound;
    const unsigned m = __ballot_sync(0xffffffffu, take);
    if (n + __popc(m) > kLpList) {
      n = list_cut(list, n, k);  // n > 32: k keys are left
      if (list[k - 1] > bound) {
        bound = list[k - 1];
        tv = key_value(bound);
      }
    }
    if (take) list[n + __popc(m & ((1u << lane) - 1u))] = q;
    n += __popc(m);
  }

  // After 1, 2, 4 ... of a block's `mine` chunks, while more are to come than have been, the
  // bound: the k-th largest of 32 groups' (8 lanes each) largest logits so far, this
  // thread's being g.  Only the first chunk needs every group's value; later a value of
  // another warp may be an older one, which is as valid.
  __device__ __forceinline__ void renew(float g, int i, int mine, volatile float* group, int k, int tid) {
    const int lane = tid & 31;
    if ((i & (i + 1)) != 0 || (i != 0 && mine - 1 - i <= i + 1)) return;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    if ((lane & 7) == 0) group[tid >> 3] = g;
    if (i == 0)
      lp_bar();
    else
      __syncwarp();
    const float gk = kth_of_lanes(group[lane], k, lane);
    const lp_key b = (lp_key)lp_ord(gk) << 32;
    if (b > bound) {
      bound = b;
      tv = gk;
    }
  }

  // The lanes whose largest logit pm of a chunk reaches the bound, usually few, one by one:
  // the warp looks at that lane's vectors together, a word per lane.  st4: this thread's
  // first vector, the row's q0-th after its head.
  template <typename T>
  __device__ __forceinline__ void scan(float pm, const uint4* st4, int q0, const Span& sp, int k, int lane) {
    constexpr int VE = Elem<T>::kVec;
    unsigned holders = __ballot_sync(0xffffffffu, pm >= tv);
    while (holders) {
      const int src = __ffs(holders) - 1;
      holders &= holders - 1;
      const int qv = q0 - lane + src + (lane >> 2) * kLpNT;
      const uint32_t word =
          reinterpret_cast<const uint32_t*>(st4 - lane + src + (lane >> 2) * kLpNT)[lane & 3];
      const int id = sp.head + qv * VE + (lane & 3) * (VE / 4);
      if constexpr (VE == 4) {
        add(__uint_as_float(word), id, qv < sp.nvec, k, lane);
      } else {
        add(__uint_as_float(word << 16), id, qv < sp.nvec, k, lane);
        add(__uint_as_float(word & 0xffff0000u), id + 1, qv < sp.nvec, k, lane);
      }
    }
  }
};

// running sum of weights: the maximum m and S = s + e (e: what rounding took from s)
struct RowSum {
  float m, s, e;
};
// relative to a maximum m >= a.m
__device__ __forceinline__ void sum_rescale(RowSum& a, float m, float c) {
  const float f = exp2_approx((a.m - m) * c);
  a.s *= f;
  a.e *= f;
  a.m = m;
}
__device__ __forceinline__ RowSum sum_join(RowSum a, RowSum b, float c) {
  const float m = max_nan(a.m, b.m);
  sum_rescale(a, m, c);
  sum_rescale(b, m, c);
  RowSum r;
  r.m = m;
  two_sum(a.s, b.s, r.s, r.e);
  r.e += a.e + b.e;
  return r;
}
// joins those of n lanes, a power of two
__device__ __forceinline__ RowSum sum_lanes(RowSum a, int n, float c) {
  for (int o = n >> 1; o > 0; o >>= 1) {
    RowSum b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.e = __shfl_xor_sync(0xffffffffu, a.e, o);
    a = sum_join(a, b, c);
  }
  return a;
}
// adds a chunk's vectors, none of which is above a.m
template <typename T, int U>
__device__ __forceinline__ void sum_add(RowSum& a, const uint4 (&v)[U], float c) {
  const f32x2 c2 = pack2(c, c);
  f32x2 sum[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < Elem<T>::kVec; e += 2) {
      float t0, t1;
      unpack2(mul2(Vec<T>::diff2(v[u], e, -a.m), c2), t0, t1);
      const f32x2 w = pack2(exp2_approx(t0), exp2_approx(t1));
      sum[u] = e == 0 ? w : add2(sum[u], w);
    }
#pragma unroll
  for (int h = U / 2; h > 0; h >>= 1)
#pragma unroll
    for (int u = 0; u < h; ++u) sum[u] = add2(sum[u], sum[u + h]);
  float s0, s1, er;
  unpack2(sum[0], s0, s1);
  two_sum(a.s, s0 + s1, a.s, er);
  a.e += er;
}

// Thread blocks per row: the count that gives the shortest schedule, taking a
// block's time as its chunks plus three more for its start and its join, and
// kLpPerSm blocks of each SM running at once.
inline int lp_cluster(int64_t R, int V, int elem) {
  const int64_t chunks = ((int64_t)V * elem + kLpChunk - 1) / kLpChunk;
  const int64_t slots = (int64_t)num_sms() * kLpPerSm;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int C = 1; C <= kLpMaxC && C <= chunks; C *= 2) {
    const int64_t waves = (R * C + slots - 1) / slots;
    const int64_t t = waves * ((chunks + C - 1) / C + 3);
    if (t < least) {
      least = t;
      best = C;
    }
  }
  return best;
}

}  // namespace vt
