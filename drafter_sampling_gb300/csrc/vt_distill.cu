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
#include <algorithm>
#include <cmath>

#include <cooperative_groups.h>

#include "vt_internal.h"
#include "vt_rows.cuh"
#include "vt_umma.cuh"

namespace cg = cooperative_groups;

namespace vt {
namespace {

constexpr int kDsMaxK = 128;
constexpr int kDsLane = kDsMaxK / 32;      // list entries of a lane
constexpr int kDsNT = 256;
constexpr int kDsThreads = kLpNT + 64;     // consuming warps, one that copies, one for the list

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

struct DsArgs {
  const void* logits;
  int64_t ld;
  int R, K, V, k;
  int rest;
  float c;                 // log2(e) / T
  Pair inv_t;              // 1 / T
  const int* ids;          // [R][k]
  const float* logp;       // [R][k]
  const int* inv_map;      // [V] or nullptr (V == K)
  const float* weight;     // [R] or nullptr: dL/dloss
  float* out_loss;         // [R]
  DsStats* stats;          // [R]
  void* grad;
  int64_t ld_grad;
  int* dev_status;
  int own_status;          // one row: its block stores the status word; else it is zeroed beforehand
};

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
  int place[kDsMaxK];  // of entries that the drafter has, else -1
  int pos[kDsMaxK];    // bytes from the start of what this block reads of the row, -1: not there
  float z[kDsMaxK], logp[kDsMaxK];
  unsigned edges;      // the row's edge elements that are listed
  int any;             // an id is given
  int flags;
};
// What the consuming warps leave of a row: the sum over its unlisted ids
struct DsSum {
  RowSum sum;
  int late;
};

// The list of a row, read by one warp in two steps: the places, which the consuming
// warps wait for, and what stands there.  at(place): the byte position in what this
// block reads, or -1.
template <typename T, typename At>
__device__ __forceinline__ void ds_places(const DsArgs& a, int row, const Span& sp, bool edges, DsList& sh, int lane,
                                          At at) {
  int p[kDsLane];
  bool any = false;
#pragma unroll
  for (int h = 0; h < kDsLane; ++h) {
    const int i = lane + 32 * h;
    p[h] = -1;
    if (i < a.k) {
      const int id = __ldg(a.ids + (int64_t)row * a.k + i);
      any |= id != -1;
      p[h] = id == -1 ? -1 : id < 0 || id >= a.V ? -2 : id;
    }
  }
  bool bad = false;
  unsigned edge = 0;
#pragma unroll
  for (int h = 0; h < kDsLane; ++h) {
    const int i = lane + 32 * h;
    if (p[h] >= 0 && a.inv_map) {
      const int q = __ldg(a.inv_map + p[h]);
      p[h] = q >= -1 && q < a.K ? q : -2;
    }
    bad |= p[h] == -2;
    if (i < a.k) {
      sh.place[i] = max(p[h], -1);
      sh.pos[i] = p[h] >= 0 ? at(p[h]) : -1;
    }
    if (p[h] >= 0 && edges) {
      const int t = p[h] < sp.head ? p[h] : p[h] - sp.nvec * Elem<T>::kVec;
      if (p[h] < sp.head || t >= sp.head) edge |= 1u << t;
    }
  }
  any = __any_sync(0xffffffffu, any);
  bad = __any_sync(0xffffffffu, bad);
  edge = __reduce_or_sync(0xffffffffu, edge);
  if (lane == 0) {
    sh.any = any;
    sh.flags = bad ? VT_DEV_BAD_ID : 0;
    sh.edges = edge;
  }
  __syncwarp();
}
template <typename T>
__device__ __forceinline__ void ds_entries(const DsArgs& a, int row, const T* l, DsList& sh, int lane) {
  int flags = 0;
#pragma unroll
  for (int h = 0; h < kDsLane; ++h) {
    const int i = lane + 32 * h;
    if (i >= a.k) break;
    const int p = sh.place[i];
    const float lp = __ldg(a.logp + (int64_t)row * a.k + i);
    const float z = p >= 0 ? Elem<T>::load(l + p) : -INFINITY;
    if (p >= 0 && z != -INFINITY) {  // kept
      if (!(z < INFINITY) || !(lp < 80.f)) flags = VT_DEV_NONFINITE;
      int twice = 0;
      for (int o = 0; o < i; ++o) twice |= sh.place[o] == p;
      if (twice) flags |= VT_DEV_DUPLICATE_ID;
    }
    sh.z[i] = z;
    sh.logp[i] = lp;
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (lane == 0) sh.flags |= flags;
  __syncwarp();
}

__device__ __forceinline__ Pair pair_warp_sum(Pair v) {
  for (int o = 16; o > 0; o >>= 1) {
    Pair w;
    w.h = __shfl_xor_sync(0xffffffffu, v.h, o);
    w.l = __shfl_xor_sync(0xffffffffu, v.l, o);
    v = pair_add(v, w);
  }
  return v;
}
__device__ __forceinline__ Pair pair_from_lane(Pair v, int lane) {
  return Pair{__shfl_sync(0xffffffffu, v.h, lane), __shfl_sync(0xffffffffu, v.l, lane)};
}

// Loss, statistics and flags of a row, by one warp: from its list and the sum of its
// unlisted ids (s = 0: there are none above -infinity).
__device__ void ds_finish(const DsArgs& a, const DsList& sh, const DsSum& un, int lane, float& loss, DsStats& st,
                          int& flags) {
  const float mr = un.sum.m;
  const bool rest = !(un.sum.s == 0.f);  // (NaN: flagged below)
  bool kept = false;
  float m = rest ? mr : -INFINITY;
  Pair mass{0.f, 0.f};
#pragma unroll
  for (int h = 0; h < kDsLane; ++h) {
    const int i = lane + 32 * h;
    if (i < a.k && sh.z[i] != -INFINITY) {
      kept = true;
      m = max_nan(m, sh.z[i]);
      mass = pair_add(mass, pair_exp(Pair{sh.logp[i], 0.f}));
    }
  }
  kept = __any_sync(0xffffffffu, kept);
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  mass = pair_warp_sum(mass);
  loss = 0.f;
  st = DsStats{0.f, 0.f, 0.f, 0.f, 0.f};
  flags = sh.flags | (un.late ? VT_DEV_TIMEOUT : 0);
  if (kept && !(m < INFINITY)) flags |= VT_DEV_NONFINITE;
  if (flags) {
    loss = __int_as_float(0x7fc00000);
    st = DsStats{loss, loss, loss, loss, loss};
    return;
  }
  // (z - m) / T; nothing of e^ it is left below -87
  const auto below = [&](float z) {
    Pair d;
    two_sum(z, -m, d.h, d.l);
    return pair_mul(d, a.inv_t);
  };
  const auto weight = [&](float z) {
    return (z - m) * a.inv_t.h < -87.f ? Pair{0.f, 0.f} : pair_exp(below(z));
  };
  Pair b{0.f, 0.f};
  if (a.rest && rest) b = pair_add(Pair{1.f, 0.f}, pair_neg(mass));
  if (!(b.h > 0.f)) b = Pair{0.f, 0.f};
  const Pair A = pair_add(mass, b);
  if (!kept || !(A.h > 0.f)) return;  // nothing to learn from this row
  Pair S{0.f, 0.f};
#pragma unroll
  for (int h = 0; h < kDsLane; ++h) {
    const int i = lane + 32 * h;
    if (i < a.k && sh.z[i] != -INFINITY) S = pair_add(S, weight(sh.z[i]));
  }
  S = pair_warp_sum(S);
  const Pair sr = pair_of(un.sum.s, un.sum.e);
  const Pair top = rest ? weight(mr) : Pair{0.f, 0.f};  // of the largest unlisted logit
  S = pair_add(S, pair_mul(sr, top));
  // four logarithms at once, one per lane
  Pair v = lane == 0 ? S : lane == 1 ? sr : lane == 2 ? b : mass;
  v = v.h > 0.f ? pair_log(v) : Pair{0.f, 0.f};
  const Pair lnS = pair_from_lane(v, 0), lnr = pair_from_lane(v, 1), lnb = pair_from_lane(v, 2);
  const Pair lna = pair_from_lane(v, 3);
  Pair sum{0.f, 0.f};
#pragma unroll
  for (int h = 0; h < kDsLane; ++h) {
    const int i = lane + 32 * h;
    if (i < a.k && sh.z[i] != -INFINITY && sh.logp[i] > -INFINITY) {
      const Pair lnp = pair_add(below(sh.z[i]), pair_neg(lnS));
      const Pair lnt{sh.logp[i], 0.f};
      sum = pair_add(sum, pair_mul(pair_exp(lnt), pair_add(lnt, pair_neg(lnp))));
    }
  }
  sum = pair_warp_sum(sum);
  const Pair all = pair_div(a.inv_t, S);
  st.m = m;
  st.mr = rest ? mr : 0.f;
  if (a.rest) {
    if (b.h > 0.f) {
      const Pair lnq = pair_add(pair_add(lnr, below(mr)), pair_neg(lnS));
      sum = pair_add(sum, pair_mul(b, pair_add(lnb, pair_neg(lnq))));
    }
    st.c_all = pair_mul(A, all).h;
    Pair c = pair_mul(A, pair_mul(all, top));
    if (b.h > 0.f) c = pair_add(c, pair_neg(pair_div(pair_mul(a.inv_t, b), sr)));
    st.c_rest = c.h;
    st.c_t = a.inv_t.h;
  } else {
    sum = pair_add(pair_div(sum, mass), pair_neg(lna));
    st.c_all = all.h;
    st.c_rest = pair_mul(all, top).h;
    st.c_t = pair_div(a.inv_t, mass).h;
  }
  loss = sum.h;
  if (loss != loss) loss = INFINITY;  // a term beyond fp32: they are positive
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

// Takes the listed elements out of what this warp is about to read: `first` bytes into
// the block's part of the row begin `bytes` of it, at `buf`; vectors go to threads in turn.
template <typename T>
__device__ __forceinline__ void ds_mask(const DsList& sh, uint8_t* buf, int first, int bytes, int k, int warp, int lane) {
  for (int i = lane; i < k; i += 32) {
    const int p = sh.pos[i] - first;
    if (p >= 0 && p < bytes && ((p >> 9) & (kLpWarps - 1)) == warp) {
      *reinterpret_cast<decltype(Mask<T>::bits())*>(buf + p) = Mask<T>::bits();
      // ahead of the next copy into this place
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
  }
  __syncwarp();
}

// ------------------------------------------------------------------ the loss
struct DsShared {
  DsList list[2];  // of the row in hand and the next one
  DsSum sum[2];
  RowSum red[2][kLpWarps];
  RowSum blk;      // this block's sum, as published
  float edge[2][16];
  alignas(8) uint64_t full[kLpStages], empty[kLpStages], listed[2], summed[2];
  int timeout;
};

// whether a row has an id listed; all lanes of a warp call it
__device__ __forceinline__ bool ds_any(const DsArgs& a, int row, int lane) {
  bool any = false;
  for (int i = lane; i < a.k; i += 32) any |= __ldg(a.ids + (int64_t)row * a.k + i) != -1;
  return __any_sync(0xffffffffu, any);
}

// Rows are streamed as the log probabilities' kernel does it: one warp copies, eight sum the
// unlisted ids; another reads the next row's list meanwhile and finishes the last one.
template <typename T>
__global__ void __launch_bounds__(kDsThreads, kLpPerSm) distill_loss_kernel(DsArgs a) {
  constexpr int VE = Elem<T>::kVec;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ DsShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row0 = blockIdx.x / C, stride = gridDim.x / C;
  if (tid == 0) {
    for (int s = 0; s < kLpStages; ++s) {
      umma::mbar_init(&sh.full[s], 1);
      umma::mbar_init(&sh.empty[s], kLpWarps);
    }
    for (int s = 0; s < 2; ++s) {
      umma::mbar_init(&sh.listed[s], 1);
      umma::mbar_init(&sh.summed[s], kLpWarps);
    }
    sh.timeout = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  if (warp == kLpWarps) {
    // the copying warp runs ahead of the consumers, into their next rows
    bool ok = true, any = ds_any(a, row0, lane);
    const bool first = any;
    int it = 0;  // chunks requested so far
    for (int row = row0; row < a.R; row += stride) {
      if (any && ok && lane == 0) {
        const T* l = static_cast<const T*>(a.logits) + (int64_t)row * a.ld;
        const Span sp = span_of<T>(l, a.K, rank, C);
        const uint8_t* src = reinterpret_cast<const uint8_t*>(l + sp.head);
        for (int i = 0; i < sp.mine; ++i, ++it) {
          const int s = it % kLpStages;
          if (it >= kLpStages) ok = umma::mbar_wait(&sh.empty[s], ((it / kLpStages) - 1) & 1);
          if (!ok) break;
          const int64_t at = (int64_t)(rank + i * C) * kLpChunk;
          const uint32_t bytes = (uint32_t)min((int64_t)kLpChunk, (int64_t)sp.nvec * 16 - at);
          umma::mbar_expect_tx(&sh.full[s], bytes);
          umma::bulk_load(ring + s * kLpChunk, src + at, bytes, &sh.full[s]);
        }
      }
      if (row + stride < a.R) any = ds_any(a, row + stride, lane);
    }
    if (!ok) {
      atomicExch(&sh.timeout, 1);
      // every copy issued has landed before this block may exit
      for (int s = 0; s < kLpStages; ++s)
        for (int par = 0; par < 2; ++par) umma::mbar_wait(&sh.full[s], par, 1u << 12);
    }
    __syncwarp();
    if (C > 1 && first) {
      cl.sync();
      cl.sync();
    }
    return;
  }

  if (warp == kLpWarps + 1) {
    // the list's warp: row r is finished after row r + 1's list has been read
    uint32_t limit = umma::kWaitLimit;
    const auto read = [&](int row, int slot) {
      DsList& list = sh.list[slot];
      const T* l = static_cast<const T*>(a.logits) + (int64_t)row * a.ld;
      const Span sp = span_of<T>(l, a.K, rank, C);
      ds_places<T>(a, row, sp, rank == 0, list, lane, [&](int p) {
        const int e = p - sp.head, v = e / VE;
        if (e < 0 || v >= sp.nvec) return -1;
        const int chunk = v / (kLpNT * kLpU), mine = chunk / C;
        if (chunk - mine * C != rank) return -1;
        return mine * kLpChunk + (v - chunk * (kLpNT * kLpU)) * 16 + (e - v * VE) * (int)sizeof(T);
      });
      if (lane == 0) umma::mbar_arrive(&sh.listed[slot]);
      if (list.any && rank == 0) ds_entries<T>(a, row, l, list, lane);
    };
    read(row0, 0);
    int n = 0;
    bool first = sh.list[0].any;
    for (int row = row0; row < a.R; row += stride, ++n) {
      const int slot = n & 1;
      if (row + stride < a.R) read(row + stride, slot ^ 1);
      if (C > 1) break;  // (one row, finished below)
      const bool any = sh.list[slot].any;
      if (!__all_sync(0xffffffffu, umma::mbar_wait(&sh.summed[slot], (n >> 1) & 1, limit))) {
        limit = 1;
        if (lane == 0) atomicExch(&sh.timeout, 1);
        sh.sum[slot].late = 1;
      }
      __syncwarp();
      float loss = 0.f;
      DsStats st{0.f, 0.f, 0.f, 0.f, 0.f};
      int flags = 0;
      if (any) ds_finish(a, sh.list[slot], sh.sum[slot], lane, loss, st, flags);
      if (lane == 0) ds_put(a, row, loss, st, flags);
      __syncwarp();
    }
    if (C > 1) {
      float loss = 0.f;
      DsStats st{0.f, 0.f, 0.f, 0.f, 0.f};
      int flags = 0;
      if (first) {
        cl.sync();
        if (rank == 0) {
          // all blocks' sums, one per lane
          const int from = lane < C ? lane : 0;
          RowSum r = *cl.map_shared_rank(&sh.blk, from);
          const bool late = *cl.map_shared_rank(&sh.timeout, from) != 0;
          if (lane >= C) r.s = r.e = 0.f;
          r = sum_lanes(r, kLpMaxC, a.c);
          DsSum un{r, __any_sync(0xffffffffu, late)};
          un.sum.m = __shfl_sync(0xffffffffu, r.m, 0);
          un.sum.s = __shfl_sync(0xffffffffu, r.s, 0);
          un.sum.e = __shfl_sync(0xffffffffu, r.e, 0);
          ds_finish(a, sh.list[0], un, lane, loss, st, flags);
        }
        cl.sync();  // the first block has read the others' memory
      }
      if (rank == 0 && lane == 0) ds_put(a, row0, loss, st, flags);
    }
    return;
  }

  int it = 0, n = 0;  // chunks and rows consumed so far
  uint32_t limit = umma::kWaitLimit;
  for (int row = row0; row < a.R; row += stride, ++n) {
    const int slot = n & 1;
    const DsList& list = sh.list[slot];
    const T* l = static_cast<const T*>(a.logits) + (int64_t)row * a.ld;
    const Span sp = span_of<T>(l, a.K, rank, C);
    const bool edge = rank == 0 && tid < 2 * VE;
    float xe = -INFINITY;
    if (edge) {
      const int id = edge_id<VE>(sp, tid);
      if (id < a.K) xe = Elem<T>::load(l + id);
    }
    if (!__all_sync(0xffffffffu, umma::mbar_wait(&sh.listed[slot], (n >> 1) & 1, limit))) {
      limit = 1;
      if (lane == 0) atomicExch(&sh.timeout, 1);
    }
    if (!list.any) {
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(&sh.summed[slot]);
      continue;
    }
    RowSum st{kNegBig, 0.f, 0.f};
    for (int i = 0; i < sp.mine; ++i, ++it) {
      const int s = it % kLpStages;
      if (!__all_sync(0xffffffffu, umma::mbar_wait(&sh.full[s], (it / kLpStages) & 1, limit))) {
        // gave up: go on without the data, so that no barrier is missed
        limit = 1;
        if (lane == 0) atomicExch(&sh.timeout, 1);
      }
      ds_mask<T>(list, ring + s * kLpChunk, i * kLpChunk, kLpChunk, a.k, warp, lane);
      const int q0 = (rank + i * C) * (kLpNT * kLpU) + tid;  // first vector of this thread
      const uint4* st4 = reinterpret_cast<const uint4*>(ring + s * kLpChunk) + tid;
      const int have = min(kLpU, max(0, (sp.nvec - q0 + kLpNT - 1) / kLpNT));  // vectors in the row
      uint4 v[kLpU];
#pragma unroll
      for (int u = 0; u < kLpU; ++u)
        v[u] = u < have ? st4[u * kLpNT]
                        : make_uint4(Vec<T>::kMasked, Vec<T>::kMasked, Vec<T>::kMasked, Vec<T>::kMasked);
      const float pm = Vec<T>::top(v);
      if (!(pm <= st.m)) sum_rescale(st, max_nan(st.m, pm), a.c);
      sum_add<T>(st, v, a.c);
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(&sh.empty[s]);
    }
    if (edge && !(list.edges >> tid & 1)) {
      if (!(xe <= st.m)) sum_rescale(st, max_nan(st.m, xe), a.c);
      float er;
      two_sum(st.s, exp2_approx((xe - st.m) * a.c), st.s, er);
      st.e += er;
    }
    st = sum_lanes(st, 32, a.c);
    if (lane == 0) sh.red[slot][warp] = st;
    lp_bar();
    if (warp == 0) {
      // (a warp that is ahead writes the other slot; it cannot reach the next but one
      // row before this one has passed the next row's barrier)
      const RowSum r = sum_lanes(sh.red[slot][lane % kLpWarps], kLpWarps, a.c);
      if (lane == 0) {
        sh.sum[slot] = DsSum{r, sh.timeout};
        sh.blk = r;
      }
    }
    __syncwarp();
    if (lane == 0) umma::mbar_arrive(&sh.summed[slot]);
    if (C > 1) {
      cl.sync();
      cl.sync();
    }
  }
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
__device__ __forceinline__ float ds_listed(const DsArgs& a, const DsStats& st, float g, float z, float logp) {
  return g * (st.c_all * exp2_approx((z - st.m) * a.c) - st.c_t * pair_exp(Pair{logp, 0.f}).h);
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

constexpr int kDgU = 4;  // vectors per thread

// Each block takes kDsNT * kDgU vectors of a row; the first also the row's edges.  What
// it reads is in registers before it writes, so the gradient may take the logits' place.
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
    if (edge) xe = Elem<T>::load(l + edge_id<VE>(sp, tid));
    if (tid < a.k) {
      p = ds_place(a, (int64_t)row * a.k + tid);
      const int q = (p - sp.head) / VE;
      const bool inner = p >= sp.head && q < sp.nvec;
      if (p >= 0 && (inner ? q / (kDsNT * kDgU) != piece : piece != 0)) p = -1;
      if (p >= 0) {
        lp = a.logp[(int64_t)row * a.k + tid];
        z = Elem<T>::load(l + p);
        if (z == -INFINITY) p = -1;
      }
    }
    __syncthreads();
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
  if (p >= 0) Store<T>::put(d + p, ds_listed(a, st, g, z, lp));
}

// ------------------------------------------------------- loss and gradient
constexpr int kDtThreads = kLpNT + 32;  // consuming warps and one for the list
constexpr int kDtPieces = 8;            // copies of kLpChunk bytes a block
constexpr int kDtMaxC = 8;

struct DtShared {
  DsList list;
  RowSum red[kLpWarps];
  DsStats st;
  float edge[16];
  alignas(8) uint64_t full[kDtPieces];
  int timeout;
};

// One row per cluster, kept in its blocks' shared memory between the sum and the
// gradient: `share` vectors in each block.  Every block finishes the row for itself.
template <typename T>
__global__ void __launch_bounds__(kDtThreads) distill_train_kernel(DsArgs a, int share) {
  constexpr int VE = Elem<T>::kVec;
  extern __shared__ __align__(16) uint8_t part[];
  __shared__ DtShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / C;
  const T* l = static_cast<const T*>(a.logits) + (int64_t)row * a.ld;
  T* d = static_cast<T*>(a.grad) + (int64_t)row * a.ld_grad;
  const Span sp = span_of<T>(l, a.K, 0, 1);
  const int v0 = min(rank * share, sp.nvec), mine = min(share, sp.nvec - v0);  // this block's vectors
  const int pieces = (mine * 16 + kLpChunk - 1) / kLpChunk;
  const bool edges = rank == 0;
  if (tid == kLpNT) {
    for (int i = 0; i < kDtPieces; ++i) umma::mbar_init(&sh.full[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    sh.timeout = 0;
  }
  __syncthreads();
  float xe = -INFINITY;
  if (warp == kLpWarps) {
    const bool any = ds_any(a, row, lane);
    if (any && lane == 0) {
      const uint8_t* src = reinterpret_cast<const uint8_t*>(l + sp.head) + (int64_t)v0 * 16;
      for (int i = 0; i < pieces; ++i) {
        const uint32_t bytes = (uint32_t)min(kLpChunk, mine * 16 - i * kLpChunk);
        umma::mbar_expect_tx(&sh.full[i], bytes);
        umma::bulk_load(part + i * kLpChunk, src + (int64_t)i * kLpChunk, bytes, &sh.full[i]);
      }
    }
    __syncwarp();
    ds_places<T>(a, row, sp, edges, sh.list, lane, [&](int p) {
      const int e = p - sp.head, v = e / VE - v0;
      return e < 0 || v < 0 || v >= mine ? -1 : v * 16 + (e % VE) * (int)sizeof(T);
    });
  } else if (edges && tid < 2 * VE) {
    const int id = edge_id<VE>(sp, tid);
    if (id < a.K) xe = Elem<T>::load(l + id);
  }
  __syncthreads();  // the places
  const float g = a.weight ? a.weight[row] : 1.f;
  const bool any = sh.list.any;
  bool nothing = !any;
  if (any) {
    if (warp == kLpWarps) {
      ds_entries<T>(a, row, l, sh.list, lane);
    } else {
      RowSum st{kNegBig, 0.f, 0.f};
      for (int i = 0; i < pieces; ++i) {
        if (!__all_sync(0xffffffffu, umma::mbar_wait(&sh.full[i], 0)) && lane == 0) atomicExch(&sh.timeout, 1);
        ds_mask<T>(sh.list, part + i * kLpChunk, i * kLpChunk, kLpChunk, a.k, warp, lane);
        const uint4* st4 = reinterpret_cast<const uint4*>(part + i * kLpChunk) + tid;
        const int have = min(kLpU, max(0, (mine - i * (kLpNT * kLpU) - tid + kLpNT - 1) / kLpNT));
        uint4 v[kLpU];
#pragma unroll
        for (int u = 0; u < kLpU; ++u)
          v[u] = u < have ? st4[u * kLpNT]
                          : make_uint4(Vec<T>::kMasked, Vec<T>::kMasked, Vec<T>::kMasked, Vec<T>::kMasked);
        const float pm = Vec<T>::top(v);
        if (!(pm <= st.m)) sum_rescale(st, max_nan(st.m, pm), a.c);
        sum_add<T>(st, v, a.c);
      }
      if (edges && tid < 2 * VE && !(sh.list.edges >> tid & 1)) {
        if (!(xe <= st.m)) sum_rescale(st, max_nan(st.m, xe), a.c);
        float er;
        two_sum(st.s, exp2_approx((xe - st.m) * a.c), st.s, er);
        st.e += er;
      }
      st = sum_lanes(st, 32, a.c);
      if (lane == 0) sh.red[warp] = st;
    }
    if (C > 1)
      cl.sync();  // every block's sums; and what is read of the row has been read
    else
      __syncthreads();
    if (warp == kLpWarps) {
      DsSum un{RowSum{kNegBig, 0.f, 0.f}, 0};
      for (int i = lane; i < C * kLpWarps; i += 32) {
        const int from = i / kLpWarps;
        un.sum = sum_join(un.sum, cl.map_shared_rank(sh.red, from)[i % kLpWarps], a.c);
        un.late |= *cl.map_shared_rank(&sh.timeout, from);
      }
      un.sum = sum_lanes(un.sum, 32, a.c);
      un.late = __any_sync(0xffffffffu, un.late != 0);
      float loss;
      DsStats st;
      int flags;
      ds_finish(a, sh.list, un, lane, loss, st, flags);
      if (lane == 0) {
        sh.st = st;
        if (edges) ds_put(a, row, loss, st, flags);
      }
    }
    __syncthreads();
    if (C > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");  // done with the others' memory
    nothing = ds_nothing(sh.st);
  } else if (edges && tid == 0) {
    ds_put(a, row, 0.f, DsStats{0.f, 0.f, 0.f, 0.f, 0.f}, 0);
  }
  const DsStats st = any ? sh.st : DsStats{0.f, 0.f, 0.f, 0.f, 0.f};
  const float factor = g * st.c_rest;
  if (warp < kLpWarps) {
    T* out = d + sp.head + (int64_t)v0 * VE;
    const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    const uint4* in = reinterpret_cast<const uint4*>(part);
#pragma unroll 4
    for (int q = tid; q < mine; q += kLpNT)
      store_vec(out + (int64_t)q * VE,
                nothing ? make_uint4(0, 0, 0, 0) : Store<T>::grad(in[q], st.mr, a.c, factor), aligned);
    if (edges && tid < 2 * VE && edge_id<VE>(sp, tid) < a.K)
      Store<T>::put(d + edge_id<VE>(sp, tid), nothing ? 0.f : factor * exp2_approx((xe - st.mr) * a.c));
  }
  if (!nothing) {
    __syncthreads();
    if (warp == kLpWarps)
      for (int i = lane; i < a.k; i += 32) {
        const int p = sh.list.place[i];
        const bool here = sh.list.pos[i] >= 0 || (edges && p >= 0 && (p < sp.head || p >= sp.head + sp.nvec * VE));
        const float z = sh.list.z[i];
        if (here && z != -INFINITY) Store<T>::put(d + p, ds_listed(a, st, g, z, sh.list.logp[i]));
      }
  }
  if (sh.timeout && tid == 0)  // every copy issued has landed before this block may exit
    for (int i = 0; any && i < pieces; ++i) umma::mbar_wait(&sh.full[i], 0, 1u << 12);
  if (C > 1 && any) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
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
  a.rest = rest;
  a.c = VT_LOG2E / T;
  a.inv_t.h = (float)(1.0 / (double)T);
  a.inv_t.l = (float)(1.0 / (double)T - (double)a.inv_t.h);
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

template <typename T>
int ds_launch_loss(const DsArgs& a, cudaStream_t s) {
  auto kern = distill_loss_kernel<T>;
  VT_RETURN_IF_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kLpSmem));
  if (!a.own_status) {
    const int st = clear_status(s, a.dev_status);
    if (st != VT_OK) return st;
  }
  const int C = lp_cluster(a.R, a.K, (int)sizeof(T));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(C > 1 ? a.R * C : std::min(a.R, num_sms() * kLpPerSm)));
  cfg.blockDim = dim3(kDsThreads);
  cfg.dynamicSmemBytes = kLpSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.own_status ? 1 : 2;
  VT_RETURN_IF_CUDA(cudaLaunchKernelEx(&cfg, kern, a));
  return VT_OK;
}
int ds_launch_loss(const DsArgs& a, int32_t dtype, cudaStream_t s) {
  return dtype == VT_F32 ? ds_launch_loss<float>(a, s) : ds_launch_loss<uint16_t>(a, s);
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

// bytes of shared memory that a row's part may take: three blocks on an SM, or one
constexpr int kDtThree = 68 << 10, kDtOne = 200 << 10;

template <typename T>
int ds_launch_train(const DsArgs& a, cudaStream_t s, int C, int share) {
  auto kern = distill_train_kernel<T>;
  VT_RETURN_IF_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kDtOne));
  if (!a.own_status) {
    const int st = clear_status(s, a.dev_status);
    if (st != VT_OK) return st;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.R * C));
  cfg.blockDim = dim3(kDtThreads);
  cfg.dynamicSmemBytes = (size_t)share * 16;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.own_status ? 1 : 2;
  VT_RETURN_IF_CUDA(cudaLaunchKernelEx(&cfg, kern, a, share));
  return VT_OK;
}

// Rows that the blocks of a cluster hold between them are read once; longer ones take the two calls.
int ds_launch_both(const DsArgs& a, int32_t dtype, cudaStream_t s) {
  const int64_t bytes = (int64_t)a.K * (dtype == VT_F32 ? 4 : 2);
  int C = (int)std::min<int64_t>((bytes + kDtThree - 1) / kDtThree, kDtMaxC);
  const int64_t vecs = bytes / 16, share = (vecs + C - 1) / C;
  if (share * 16 > kDtOne || (int64_t)a.R * C > 0x7fffffff) {
    const int rc = ds_launch_loss(a, dtype, s);
    return rc != VT_OK ? rc : ds_launch_grad(a, dtype, s);
  }
  return dtype == VT_F32 ? ds_launch_train<float>(a, s, C, (int)share) : ds_launch_train<uint16_t>(a, s, C, (int)share);
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
