// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits on sm_103a.
//
// With p = softmax(l / T) over the V ids of a row and c = log2(e) / T:
//   m = max l,  y_i = l_i - m,  S = sum 2^(y_i c),  D = sum 2^(y_i c) y_i
//   log p_x = y_x / T - ln S
//   entropy = ln S - D / (T S)
// and the k largest l (ties to the lower id) with their log p.  The maximum is
// subtracted before the scale, so a row of the type's lowest value still gives
// the uniform distribution; ids at -inf have p = 0 and add nothing.
//
// One pass over a row by a cluster of C thread blocks: block r takes the 32 KB
// chunks r, r + C, ... .  One warp streams them by bulk copies into a ring of
// two shared-memory stages, eight warps consume them, so the bytes in flight
// do not depend on what the consumers are doing; a row's elements before its
// first and after its last 16-byte boundary are loaded one by one.
// A thread keeps a running (m, S, D) of what it has seen.  S is a sum of
// chunks' sums carried with its rounding error, so that it does not lose with
// the row's length, and ln S is taken as log1p(S - 1).  A chunk's own sum (32 or 64
// weights of a thread) is a plain fp32 one: next to a peak's weight of 1 it loses
// up to 16 roundings of 2^-24, so ln S and a peaked row's entropy are good to
// 1e-6, not to all their digits.  Adding the peak's chunk once more with the 1
// apart keeps them, and makes one row take 7.7 instead of 6.8 us and many rows 2%
// longer.
//
// The k best are kept as 64-bit keys, ordered by (value, lower id first).  A
// warp lists in shared memory the ids whose key reaches a bound that at least
// k ids seen reach: the k-th best of 32 disjoint groups' largest logits,
// renewed after 2, 4 ... chunks.  So little more than k ids of the first
// chunk are listed and few later ones; the lists are ranked by counting at the
// end.  A list that fills (ties, masks, ordered rows) is cut to its k best
// keys, the last of which is a bound too.  Blocks join through distributed
// shared memory.
//
// Bound by HBM without alternatives (2304 rows of 152064 bf16 logits: 111 us, 6.3
// TB/s).  With them (k = 1: 121 us, k = 20: 145) no unit is saturated, issue slots are
// 66% busy: the warps that stream a row also rank and join its lists (16 KB chunks
// were 199 against 182 us at an earlier step).  Latency when rows are few: one
// row of 128256 fp32 logits takes 5.0 us at k = 0 and 6.8 at k = 5; 112 rows, of which
// 59 are scored, 14.3 at k = 8: 4 to the first chunk, 5.7 of stream, 3 of join.
#include <algorithm>
#include <cmath>

#include <cooperative_groups.h>

#include "vt_internal.h"
#include "vt_rows.cuh"
#include "vt_umma.cuh"

namespace cg = cooperative_groups;

namespace vt {
namespace {

struct LpArgs {
  const void* logits;
  int64_t ld;
  int R, V, k;
  float c, inv_t;        // log2(e) / T and 1 / T
  const int* tokens;     // [R]
  float* out_logp;       // [R]
  float* out_entropy;    // [R] or nullptr
  int* out_ids;          // [R][k]
  float* out_top;        // [R][k]
  int* dev_status;
  int own_status;        // one row: its block stores the status word; else it is zeroed beforehand
};

// (x - m) / T, where x - m itself may lie beyond fp32 (halves differ exactly)
__device__ __forceinline__ float scaled_diff(float x, float m, float inv_t) {
  return (0.5f * x - 0.5f * m) * (2.f * inv_t);
}

// running statistics: the maximum m, S = s + e (e: what rounding took from s)
// and d = sum w y, with y = x - m and w = 2^(y c)
struct Lse {
  float m, s, e, d;
};

// y is bounded below at -kLpLow / c: 2^(y c) is zero there, and -inf times a
// zero weight is not formed
constexpr float kLpLow = 200.f;

// the same statistics relative to a maximum m >= a.m
__device__ __forceinline__ void lse_rescale(Lse& a, float m, float c, float low) {
  const float y = fmaxf(a.m - m, low);
  const float f = exp2_approx(y * c);
  a.d = f * fmaf(y, a.s, a.d);
  a.s *= f;
  a.e *= f;
  a.m = m;
}
__device__ __forceinline__ Lse lse_join(Lse a, Lse b, float c, float low) {
  const float m = max_nan(a.m, b.m);
  lse_rescale(a, m, c, low);
  lse_rescale(b, m, c, low);
  Lse r;
  r.m = m;
  two_sum(a.s, b.s, r.s, r.e);
  r.e += a.e + b.e;
  r.d = a.d + b.d;
  return r;
}

// Adds one chunk's vectors to a thread's statistics (their maximum is at most
// st.m).  A chunk that holds -inf, or values so far below st.m that the
// difference overflows, leaves st.d NaN.
template <typename T>
__device__ __forceinline__ Lse lse_add(Lse st, const uint4 (&v)[kLpU], float c) {
  constexpr int VE = Elem<T>::kVec;
  const f32x2 c2 = pack2(c, c);
  f32x2 sum[kLpU], d = pack2(st.d, 0.f);
#pragma unroll
  for (int u = 0; u < kLpU; ++u) {
#pragma unroll
    for (int e = 0; e < VE; e += 2) {
      const f32x2 y = Vec<T>::diff2(v[u], e, -st.m);
      float t0, t1;
      unpack2(mul2(y, c2), t0, t1);
      const f32x2 w = pack2(exp2_approx(t0), exp2_approx(t1));
      sum[u] = e == 0 ? w : add2(sum[u], w);
      d = fma2(w, y, d);
    }
  }
#pragma unroll
  for (int h = kLpU / 2; h > 0; h >>= 1)
#pragma unroll
    for (int u = 0; u < h; ++u) sum[u] = add2(sum[u], sum[u + h]);
  float s0, s1, d0, d1, er;
  unpack2(sum[0], s0, s1);
  unpack2(d, d0, d1);
  two_sum(st.s, s0 + s1, st.s, er);
  st.e += er;
  st.d = d0 + d1;
  return st;
}

// The same with y bounded below, from the vectors at `src` (every kLpNT-th;
// those from index `have` on hold nothing).
template <typename T>
__device__ __noinline__ Lse lse_add_bounded(Lse st, const uint4* src, int have, float c, float low) {
  constexpr int VE = Elem<T>::kVec;
  float s = 0.f;
#pragma unroll 1
  for (int u = 0; u < have; ++u) {
    float x[VE], part = 0.f;
    Elem<T>::unpack16(src[u * kLpNT], x);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float y = fmaxf(x[e] - st.m, low), w = exp2_approx(y * c);
      part += w;
      st.d = fmaf(w, y, st.d);
    }
    s += part;
  }
  float er;
  two_sum(st.s, s, st.s, er);
  st.e += er;
  return st;
}

struct LpShared {
  RowLists top;
  alignas(8) uint64_t full[kLpStages], empty[kLpStages];
  Lse red[kLpWarps];
  Lse blk;                                           // this block's statistics, as published
  float edge[16], xt;                                // the row's edges; the given token's logit
  int timeout;
};

template <typename T>
__global__ void __launch_bounds__(kLpNT + 32, kLpPerSm) token_logprobs_kernel(LpArgs a) {
  constexpr int VE = Elem<T>::kVec;           // ids per 16-byte vector
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ LpShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int k = a.k;
  const float nan = __int_as_float(0x7fc00000);
  // this cluster's rows (more than one only when C == 1)
  const int row0 = blockIdx.x / C, stride = gridDim.x / C;
  if (tid == 0) {
    for (int s = 0; s < kLpStages; ++s) {
      umma::mbar_init(&sh.full[s], 1);
      umma::mbar_init(&sh.empty[s], kLpWarps);
    }
    sh.timeout = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  if (warp == kLpWarps) {
    // the producing warp runs ahead of the consumers, into their next rows
    if (lane == 0) {
      bool ok = true;
      int it = 0;  // chunks requested so far
      for (int row = row0; row < a.R && ok; row += stride) {
        if (a.tokens[row] == -1) continue;
        const Span sp = span_of<T>(static_cast<const T*>(a.logits) + (int64_t)row * a.ld, a.V, rank, C);
        const uint8_t* src = reinterpret_cast<const uint8_t*>(
            static_cast<const T*>(a.logits) + (int64_t)row * a.ld + sp.head);
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
      if (!ok) {
        atomicExch(&sh.timeout, 1);
        // every copy issued has landed before this block may exit
        for (int s = 0; s < kLpStages; ++s)
          for (int par = 0; par < 2; ++par) umma::mbar_wait(&sh.full[s], par, 1u << 12);
      }
    }
    __syncwarp();
    if (C > 1 && a.tokens[row0] != -1) {
      cl.sync();
      cl.sync();
    }
    return;
  }

  if (tid == 0 && !a.own_status) griddep_wait();  // the status word is clear
  int it = 0;  // chunks consumed so far
  uint32_t limit = umma::kWaitLimit;
  int next_token = a.tokens[row0];
  for (int row = row0; row < a.R; row += stride) {
    const int token = next_token;
    if (row + stride < a.R) next_token = a.tokens[row + stride];
    if (token == -1) {  // not scored: the row is not read
      if (rank == 0) {
        if (tid == 0) {
          a.out_logp[row] = nan;
          if (a.out_entropy) a.out_entropy[row] = nan;
          if (a.own_status) *a.dev_status = 0;
        }
        if (tid < k) {
          a.out_ids[(int64_t)row * k + tid] = -1;
          a.out_top[(int64_t)row * k + tid] = nan;
        }
      }
      continue;
    }
    const T* l = static_cast<const T*>(a.logits) + (int64_t)row * a.ld;
    const Span sp = span_of<T>(l, a.V, rank, C);
    const int nvec = sp.nvec, mine = sp.mine;
    // the given token's logit and the row's edges, one element per thread of
    // block 0, kept in shared memory until the end: registers are short
    const bool edge = rank == 0 && tid < 2 * VE;
    if (edge) {
      if (tid == 0) sh.xt = token >= 0 && token < a.V ? Elem<T>::load(l + token) : 0.f;
      const int id = edge_id<VE>(sp, tid);
      sh.edge[tid] = id < a.V ? Elem<T>::load(l + id) : -INFINITY;
    }
    const float c = a.c, low = -kLpLow / c;
    Lse st{kNegBig, 0.f, 0.f, 0.f};
    TopList top{sh.top.list[warp], 0, 0, -INFINITY};
    bool bounded = false;

    for (int i = 0; i < mine; ++i, ++it) {
      const int s = it % kLpStages;
      if (!__all_sync(0xffffffffu, umma::mbar_wait(&sh.full[s], (it / kLpStages) & 1, limit))) {
        // gave up: go on without the data, so that no barrier is missed
        limit = 1;
        if (lane == 0) atomicExch(&sh.timeout, 1);
      }
      const int q0 = (rank + i * C) * (kLpNT * kLpU) + tid;  // first vector of this thread
      const uint4* st4 = reinterpret_cast<const uint4*>(ring + s * kLpChunk) + tid;
      const int have = min(kLpU, max(0, (nvec - q0 + kLpNT - 1) / kLpNT));  // vectors in the row
      float pm;
      {
        uint4 v[kLpU];
        if (have == kLpU) {
#pragma unroll
          for (int u = 0; u < kLpU; ++u) v[u] = st4[u * kLpNT];
        } else {
#pragma unroll
          for (int u = 0; u < kLpU; ++u)
            v[u] = u < have ? st4[u * kLpNT]
                            : make_uint4(Vec<T>::kMasked, Vec<T>::kMasked, Vec<T>::kMasked,
                                         Vec<T>::kMasked);
        }
        pm = Vec<T>::top(v);
        if (!(pm <= st.m)) lse_rescale(st, max_nan(st.m, pm), c, low);
        if (!bounded) {
          const Lse next = lse_add<T>(st, v, c);
          if (__any_sync(0xffffffffu, next.d != next.d))
            bounded = true;  // this warp's later chunks too: masks come in numbers
          else
            st = next;
        }
        if (bounded) st = lse_add_bounded<T>(st, st4, have, c, low);
      }
      if (k == 0) {
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&sh.empty[s]);
        continue;
      }

      top.renew(st.s > 0.f ? st.m : -INFINITY, i, mine, sh.top.group, k, tid);
      top.scan<T>(pm, st4, q0, sp, k, lane);
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(&sh.empty[s]);
    }

    // the edges
    if (rank == 0) {
      const float xe = edge ? sh.edge[tid] : -INFINITY;
      if (!(xe <= st.m)) lse_rescale(st, max_nan(st.m, xe), c, low);
      const float y = fmaxf(xe - st.m, low), w = exp2_approx(y * c);
      float er;
      two_sum(st.s, w, st.s, er);
      st.e += er;
      st.d = fmaf(w, y, st.d);
      if (k > 0) {
        const int id = edge_id<VE>(sp, tid);
        top.add(xe, id, edge && id < a.V && xe == xe, k, lane);
      }
    }
    // this block's statistics and ranked keys
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Lse w;
      w.m = __shfl_xor_sync(0xffffffffu, st.m, o);
      w.s = __shfl_xor_sync(0xffffffffu, st.s, o);
      w.e = __shfl_xor_sync(0xffffffffu, st.e, o);
      w.d = __shfl_xor_sync(0xffffffffu, st.d, o);
      st = lse_join(st, w, c, low);
    }
    if (lane == 0) sh.red[warp] = st;
    if (k > 0) lists_join(sh.top, top.n, top.bound, k, warp, lane);
    lp_bar();
    Lse r = sh.red[lane % kLpWarps];
#pragma unroll
    for (int o = kLpWarps / 2; o > 0; o >>= 1) {
      Lse w;
      w.m = __shfl_xor_sync(0xffffffffu, r.m, o);
      w.s = __shfl_xor_sync(0xffffffffu, r.s, o);
      w.e = __shfl_xor_sync(0xffffffffu, r.e, o);
      w.d = __shfl_xor_sync(0xffffffffu, r.d, o);
      r = lse_join(r, w, c, low);
    }
    lp_key q = 0;  // this thread's key of the row's candidates for the k best
    int rk = 0;    // ... and its rank
    bool late;
    if (C == 1) {
      if (warp == 0 && lane < k) q = sh.top.best[lane];
      rk = lane;
      late = sh.timeout != 0;
    } else {
      if (tid == 0) sh.blk = r;
      cl.sync();
      if (rank != 0) {
        // the first block reads this one's memory before it arrives in turn
        cl.sync();
        return;
      }
      // all blocks' statistics, one per lane, and keys; warp w holds block w's
      const int from = lane < C ? lane : 0;
      r = *cl.map_shared_rank(&sh.blk, from);
      if (lane >= C) r.s = r.e = r.d = 0.f;
      const bool gave_up = *cl.map_shared_rank(&sh.timeout, from) != 0;
      if (warp < C) {
        if (lane < k) {
          q = cl.map_shared_rank(sh.top.best, warp)[lane];
          sh.top.all[warp * k + lane] = q;
        }
        if (warp == 0 && lane < 8) sh.top.all[C * k + lane] = 0;
      }
      late = __any_sync(0xffffffffu, gave_up);
#pragma unroll
      for (int o = kLpMaxC / 2; o > 0; o >>= 1) {
        Lse w;
        w.m = __shfl_xor_sync(0xffffffffu, r.m, o);
        w.s = __shfl_xor_sync(0xffffffffu, r.s, o);
        w.e = __shfl_xor_sync(0xffffffffu, r.e, o);
        w.d = __shfl_xor_sync(0xffffffffu, r.d, o);
        r = lse_join(r, w, c, low);
      }
      r.m = __shfl_sync(0xffffffffu, r.m, 0);
      r.s = __shfl_sync(0xffffffffu, r.s, 0);
      r.e = __shfl_sync(0xffffffffu, r.e, 0);
      r.d = __shfl_sync(0xffffffffu, r.d, 0);
      lp_bar();  // every read of the other blocks' memory has returned
      asm volatile("barrier.cluster.arrive.release;" ::: "memory");  // they may exit
      if (q != 0) rk = count_before(sh.top.all, C * k, q);
    }
    const bool ok = !late && r.s > 0.f && isfinite(r.s) && isfinite(r.m);
    const float lnS = log1pf((r.s - 1.f) + r.e);  // the largest logit's weight is exactly 1
    if (tid == 0) {
      const bool in = token >= 0 && token < a.V;
      a.out_logp[row] = ok && in ? scaled_diff(sh.xt, r.m, a.inv_t) - lnS : nan;
      if (a.out_entropy) a.out_entropy[row] = ok ? lnS - a.inv_t * (r.d / r.s) : nan;
      const int flags =
          (late ? VT_DEV_TIMEOUT : ok ? 0 : VT_DEV_NONFINITE) | (in ? 0 : VT_DEV_BAD_ID);
      if (a.own_status)
        *a.dev_status = flags;
      else if (flags)
        atomicOr(a.dev_status, flags);
    }
    if (ok && q != 0 && rk < k) {
      a.out_ids[(int64_t)row * k + rk] = key_id(q);
      a.out_top[(int64_t)row * k + rk] = scaled_diff(key_value(q), r.m, a.inv_t) - lnS;
    }
    if (!ok && tid < k) {
      a.out_ids[(int64_t)row * k + tid] = -1;
      a.out_top[(int64_t)row * k + tid] = nan;
    }
    if (C > 1)
      asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    else
      lp_bar();  // the next row writes what this one has read
  }
}

template <typename T>
int launch_logprobs(cudaStream_t s, const LpArgs& a, int C) {
  auto kern = token_logprobs_kernel<T>;
  VT_RETURN_IF_CUDA(
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kLpSmem));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(C > 1 ? a.R * C : std::min(a.R, num_sms() * kLpPerSm)));
  cfg.blockDim = dim3(kLpNT + 32);
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

}  // namespace
}  // namespace vt

extern "C" int vt_token_logprobs(const void* logits, int32_t logits_dtype, int64_t R, int32_t V,
                                 int64_t ld_logits, const int32_t* tokens, int32_t k,
                                 float temperature, float* out_logp, float* out_entropy,
                                 int32_t* out_top_ids, float* out_top_logp, int32_t* dev_status,
                                 void* stream) {
  using namespace vt;
  if (!logits || !tokens || !out_logp || !dev_status) return VT_ERR_INVALID_ARG;
  if (logits_dtype != VT_F32 && logits_dtype != VT_BF16) return VT_ERR_INVALID_ARG;
  if (R < 1 || R > (1 << 24) || V < 1 || V > (1 << 22) || ld_logits < V) return VT_ERR_INVALID_ARG;
  if (k < 0 || k > kLpMaxK || k > V || (k > 0 && (!out_top_ids || !out_top_logp)))
    return VT_ERR_INVALID_ARG;
  if (!(temperature >= 1e-30f && temperature <= 1e30f)) return VT_ERR_INVALID_ARG;
  const int elem = logits_dtype == VT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % elem != 0) return VT_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  LpArgs a;
  a.own_status = R == 1;
  if (R > 1) {
    const int st = clear_status(s, dev_status);
    if (st != VT_OK) return st;
  }
  a.logits = logits;
  a.R = (int)R;
  a.ld = ld_logits;
  a.V = V;
  a.k = k;
  a.c = VT_LOG2E / temperature;
  a.inv_t = 1.f / temperature;
  a.tokens = tokens;
  a.out_logp = out_logp;
  a.out_entropy = out_entropy;
  a.out_ids = out_top_ids;
  a.out_top = out_top_logp;
  a.dev_status = dev_status;
  const int C = lp_cluster(R, V, elem);
  return elem == 4 ? launch_logprobs<float>(s, a, C) : launch_logprobs<uint16_t>(s, a, C);
}
