// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits on sm_103a.
//
// With p = softmax(l / T) over the V ids of a row and c = log2(e) / T:
//   m = max l,  d_i = (l_i - m) c,  S = sum 2^d_i,  D = sum 2^d_i d_i
//   log p_x = (l_x - m) / T - ln S
//   entropy = ln S - ln2 D / S
// and the k largest l (ties to the lower id) with their log p.  The maximum is
// subtracted before the scale, so a row of the type's lowest value still gives
// the uniform distribution; ids at -inf have p = 0 and add nothing.
//
// One pass over a row: one cluster of C thread blocks per row; block r takes the chunks r, r + C, ...
// of a row.  A thread keeps a running (m, S, D) of what it has seen; the
// candidates for the k best are the ids not after a bound tau that at least k
// of the ids seen reach: the k-th best of 32 disjoint groups' best ids at
// first, then the k-th best found.  About k pass; they are gathered in
// shared memory and ranked by counting.  Blocks join through distributed
// shared memory.
#include <algorithm>
#include <cmath>

#include <cooperative_groups.h>

#include "vt_verify_common.cuh"

namespace cg = cooperative_groups;

namespace vt {
namespace {

constexpr int kLpNT = 256;
constexpr int kLpWarps = kLpNT / 32;
constexpr int kLpU = 8;            // 16-byte loads in flight per thread
constexpr int kLpMaxK = 32;
constexpr int kLpCap = 1024;       // candidates gathered before a fallback
constexpr int kLpCompact = 160;    // candidates kept before they are ranked
constexpr int kLpMaxC = 8;
constexpr int kNoId = 0x7fffffff;

struct LpArgs {
  const void* logits;
  int64_t R, ld;
  int V, k;
  float c, inv_t;        // log2(e) / T and 1 / T
  const int* tokens;     // [R]
  float* out_logp;       // [R]
  float* out_entropy;    // [R] or nullptr
  int* out_ids;          // [R][k]
  float* out_top;        // [R][k]
  int* dev_status;
};

// (value, id) order of the alternatives: higher value, then lower id
__device__ __forceinline__ bool lp_before(float av, int ai, float bv, int bi) {
  return av > bv || (av == bv && ai < bi);
}

// larger of two, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// running statistics: maximum, sum 2^d and sum 2^d d with d = (x - m) c
struct Lse {
  float m, s, d;
};

// exponents below this contribute exactly nothing in fp32; bounding them keeps
// -inf - m and its product with a zero weight finite
constexpr float kLpLow = -1.0e4f;

__device__ __forceinline__ void lse_rescale(Lse& a, float m, float c) {
  const float u = fmaxf((a.m - m) * c, kLpLow);
  const float f = exp2_approx(u);
  a.d = f * fmaf(u, a.s, a.d);
  a.s *= f;
  a.m = m;
}
__device__ __forceinline__ Lse lse_join(Lse a, Lse b, float c) {
  const float m = max_nan(a.m, b.m);
  lse_rescale(a, m, c);
  lse_rescale(b, m, c);
  return Lse{m, a.s + b.s, a.d + b.d};
}

template <typename T>
__global__ void __launch_bounds__(kLpNT) token_logprobs_kernel(LpArgs a) {
  constexpr int VE = Elem<T>::kVec;           // ids per 16-byte load
  constexpr int CHUNK = kLpNT * kLpU * VE;    // ids per pass
  __shared__ float cv[kLpCap];                // candidates; the list of the k best at the front
  __shared__ int ci[kLpCap];
  __shared__ float lv[kLpMaxK];               // ranked list, as published to the cluster
  __shared__ int li[kLpMaxK];
  __shared__ float gv[32];                    // best id of each of 32 groups of threads
  __shared__ int gi[32];
  __shared__ Lse red[kLpWarps];
  __shared__ Lse blk;                         // this block's statistics, as published
  __shared__ int s_n, s_listed;
  __shared__ float s_tv;
  __shared__ int s_ti;
  __shared__ float wv[kLpWarps];
  __shared__ int wi[kLpWarps];
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int64_t row = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int token = a.tokens[row];
  const int k = a.k;
  const float nan = __int_as_float(0x7fc00000);
  if (token == -1) {  // not scored: the row is not read
    if (rank == 0) {
      if (tid == 0) {
        a.out_logp[row] = nan;
        if (a.out_entropy) a.out_entropy[row] = nan;
      }
      if (tid < k) {
        a.out_ids[row * k + tid] = -1;
        a.out_top[row * k + tid] = nan;
      }
    }
    return;
  }
  const T* l = static_cast<const T*>(a.logits) + row * a.ld;
  // ids of the row that precede its first 16-byte boundary are counted from a
  // negative position: vector q of the aligned row holds ids q VE - off ...
  const int off = (int)((reinterpret_cast<uintptr_t>(l) & 15) / sizeof(T));
  const int total = a.V + off;  // aligned positions of the row
  float xt = 0.f;
  if (rank == 0 && tid == 0 && token >= 0 && token < a.V) xt = Elem<T>::load(l + token);
  if (tid == 0) {
    s_n = 0;
    s_listed = 0;
  }

  Lse st{kNegBig, 0.f, 0.f};
  bool first = true;
  __syncthreads();
  for (int64_t base = (int64_t)rank * CHUNK; base < total; base += (int64_t)C * CHUNK) {
    float x[kLpU][VE];
#pragma unroll
    for (int u = 0; u < kLpU; ++u) {
      const int64_t id0 = base + (int64_t)(u * kLpNT + tid) * VE - off;
      if (id0 >= 0 && id0 + VE <= a.V) {
        Elem<T>::unpack16(__ldg(reinterpret_cast<const uint4*>(l + id0)), x[u]);
      } else {
#pragma unroll
        for (int e = 0; e < VE; ++e)
          x[u][e] = (id0 + e >= 0 && id0 + e < a.V) ? Elem<T>::load(l + id0 + e) : -INFINITY;
      }
    }
    // statistics
    float pm = -INFINITY;
#pragma unroll
    for (int u = 0; u < kLpU; ++u)
#pragma unroll
      for (int e = 0; e < VE; ++e) pm = max_nan(pm, x[u][e]);
    if (!(pm <= st.m)) lse_rescale(st, pm, a.c);
#pragma unroll
    for (int u = 0; u < kLpU; ++u)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float d = fmaxf((x[u][e] - st.m) * a.c, kLpLow);
        const float w = exp2_approx(d);
        st.s += w;
        st.d = fmaf(w, d, st.d);
      }
    if (k == 0) continue;

    auto id_of = [&](int u, int e) {
      return (int)(base + (int64_t)(u * kLpNT + tid) * VE - off) + e;
    };
    if (first) {
      // bound: the k-th best of 32 groups' best ids (8 lanes each)
      float bv = -INFINITY;
      int bi = kNoId;
#pragma unroll
      for (int u = 0; u < kLpU; ++u)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const int id = id_of(u, e);
          if (id >= 0 && id < a.V && lp_before(x[u][e], id, bv, bi)) {
            bv = x[u][e];
            bi = id;
          }
        }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
        const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
        if (lp_before(ov, oi, bv, bi)) {
          bv = ov;
          bi = oi;
        }
      }
      if ((lane & 7) == 0) {
        gv[tid >> 3] = bv;
        gi[tid >> 3] = bi;
      }
      __syncthreads();
      if (warp == 0) {
        const float v = gv[lane];
        const int i = gi[lane];
        int r = 0;
        for (int o = 0; o < 32; ++o) r += lp_before(gv[o], gi[o], v, i) || (gv[o] == v && gi[o] == i && o < lane);
        if (r == k - 1) {
          s_tv = v;
          s_ti = i;
        }
      }
      __syncthreads();
      first = false;
    }
    const float tv = s_tv;
    const int ti = s_ti;
    if (pm >= tv) {
#pragma unroll
      for (int u = 0; u < kLpU; ++u)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const int id = id_of(u, e);
          if (x[u][e] >= tv && id >= 0 && id < a.V && !lp_before(tv, ti, x[u][e], id)) {
            const int slot = atomicAdd(&s_n, 1);
            if (slot < kLpCap) {
              cv[slot] = x[u][e];
              ci[slot] = id;
            }
          }
        }
    }
    __syncthreads();
    int n = s_n;
    if (n > kLpCap) {
      // too many reach the bound: take this chunk's k best one by one, each
      // the best after the one before, and join them to the list
      const int n0 = s_listed;
      float pv = INFINITY;
      int pi = -1;
      int got = 0;
      for (; got < k; ++got) {
        float bv = -INFINITY;
        int bi = kNoId;
#pragma unroll
        for (int u = 0; u < kLpU; ++u)
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const int id = id_of(u, e);
            if (id >= 0 && id < a.V && lp_before(pv, pi, x[u][e], id) &&
                lp_before(x[u][e], id, bv, bi)) {
              bv = x[u][e];
              bi = id;
            }
          }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
          const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
          if (lp_before(ov, oi, bv, bi)) {
            bv = ov;
            bi = oi;
          }
        }
        if (lane == 0) {
          wv[warp] = bv;
          wi[warp] = bi;
        }
        __syncthreads();
        bv = wv[0];
        bi = wi[0];
        for (int w = 1; w < kLpWarps; ++w)
          if (lp_before(wv[w], wi[w], bv, bi)) {
            bv = wv[w];
            bi = wi[w];
          }
        __syncthreads();
        if (bi == kNoId) break;
        if (tid == 0) {
          cv[n0 + got] = bv;
          ci[n0 + got] = bi;
        }
        pv = bv;
        pi = bi;
      }
      n = n0 + got;
      __syncthreads();
    }
    if (n > kLpCompact) {
      // rank by counting; the k best, in order, become the list
      float mv[kLpCap / kLpNT];
      int mi[kLpCap / kLpNT], mr[kLpCap / kLpNT];
#pragma unroll
      for (int q = 0; q < kLpCap / kLpNT; ++q) {
        const int j = tid + q * kLpNT;
        mr[q] = k;
        if (j < n) {
          mv[q] = cv[j];
          mi[q] = ci[j];
          int r = 0;
          for (int o = 0; o < n; ++o) r += lp_before(cv[o], ci[o], mv[q], mi[q]) ? 1 : 0;
          mr[q] = r;
        }
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kLpCap / kLpNT; ++q)
        if (mr[q] < k) {
          cv[mr[q]] = mv[q];
          ci[mr[q]] = mi[q];
          if (mr[q] == k - 1) {
            s_tv = mv[q];
            s_ti = mi[q];
          }
        }
      if (tid == 0) s_n = s_listed = min(n, k);
    } else if (tid == 0) {
      s_n = s_listed = n;
    }
    __syncthreads();
  }

  // this block's statistics and ranked list
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Lse w;
    w.m = __shfl_xor_sync(0xffffffffu, st.m, o);
    w.s = __shfl_xor_sync(0xffffffffu, st.s, o);
    w.d = __shfl_xor_sync(0xffffffffu, st.d, o);
    st = lse_join(st, w, a.c);
  }
  if (lane == 0) red[warp] = st;
  if (tid < kLpMaxK) {
    lv[tid] = -INFINITY;
    li[tid] = kNoId;
  }
  __syncthreads();
  if (tid == 0) {
    Lse r = red[0];
    for (int w = 1; w < kLpWarps; ++w) r = lse_join(r, red[w], a.c);
    blk = r;
  }
  if (k > 0) {
    const int n = s_n;
    for (int j = tid; j < n; j += kLpNT) {
      int r = 0;
      for (int o = 0; o < n; ++o) r += lp_before(cv[o], ci[o], cv[j], ci[j]) ? 1 : 0;
      if (r < k) {
        lv[r] = cv[j];
        li[r] = ci[j];
      }
    }
  }
  cl.sync();
  if (rank == 0) {
    // all blocks' lists, ranked; thread (q, j) holds entry j of block q
    const int q = tid >> 5, j = tid & 31;
    float v = -INFINITY;
    int i = kNoId;
    if (q < C && j < k) {
      v = cl.map_shared_rank(lv, q)[j];
      i = cl.map_shared_rank(li, q)[j];
    }
    cv[tid] = v;
    ci[tid] = i;
    if (tid < C && tid > 0) red[tid] = *cl.map_shared_rank(&blk, tid);
    if (tid == 0) red[0] = blk;
  }
  cl.sync();  // the other blocks' memory has been read; they may exit
  if (rank != 0) return;
  Lse r = red[0];
  for (int w = 1; w < C; ++w) r = lse_join(r, red[w], a.c);
  const bool ok = r.s > 0.f && isfinite(r.s) && isfinite(r.m);
  const float ln2 = 0.6931471805599453f;
  const float lnS = logf(r.s);
  if (tid == 0) {
    const bool in = token >= 0 && token < a.V;
    a.out_logp[row] = ok && in ? (xt - r.m) * a.inv_t - lnS : nan;
    if (a.out_entropy) a.out_entropy[row] = ok ? lnS - ln2 * (r.d / r.s) : nan;
    const int flags = (ok ? 0 : VT_DEV_NONFINITE) | (in ? 0 : VT_DEV_BAD_ID);
    if (flags) atomicOr(a.dev_status, flags);
  }
  if (k > 0) {
    const float v = cv[tid];
    const int i = ci[tid];
    if (i != kNoId) {
      int rk = 0;
      for (int o = 0; o < 32 * C; ++o) rk += lp_before(cv[o], ci[o], v, i) ? 1 : 0;
      if (rk < k && ok) {
        a.out_ids[row * k + rk] = i;
        a.out_top[row * k + rk] = (v - r.m) * a.inv_t - lnS;
      }
    }
    if (!ok && tid < k) {
      a.out_ids[row * k + tid] = -1;
      a.out_top[row * k + tid] = nan;
    }
  }
}

// Thread blocks per row: enough rows fill the GPU with one block each; fewer
// are cut into up to eight.
int lp_cluster(int64_t R, int V, int elem) {
  const int64_t chunks = ((int64_t)V * elem + 15) / 16 / (kLpNT * kLpU) + 1;
  int C = 1;
  while (C < kLpMaxC && R * C < 608 && C < chunks) C *= 2;
  return C;
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
  if (!std::isfinite(temperature) || temperature <= 0.f || !std::isfinite(VT_LOG2E / temperature))
    return VT_ERR_INVALID_ARG;
  const int elem = logits_dtype == VT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % elem != 0) return VT_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  VT_RETURN_IF_CUDA(cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s));
  LpArgs a;
  a.logits = logits;
  a.R = R;
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(R * C));
  cfg.blockDim = dim3(kLpNT);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (elem == 4)
    VT_RETURN_IF_CUDA(cudaLaunchKernelEx(&cfg, token_logprobs_kernel<float>, a));
  else
    VT_RETURN_IF_CUDA(cudaLaunchKernelEx(&cfg, token_logprobs_kernel<uint16_t>, a));
  return VT_OK;
}
