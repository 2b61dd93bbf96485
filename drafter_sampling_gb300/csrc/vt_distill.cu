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
#include <cmath>

#include "vt_internal.h"
#include "vt_pair.cuh"
#include "vt_verify_common.cuh"

namespace vt {
namespace {

constexpr int kDsMaxK = 128;
constexpr int kDsNT = 256;
constexpr int kDsWarps = kDsNT / 32;

struct DsStats {
  float m, mr, c_all, c_rest, c_t;
};

struct DsArgs {
  const void* logits;
  int64_t ld;
  int R, K, V, k;
  int rest;
  float c;                 // log2(e) / T
  double inv_t;            // 1 / T
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

struct DsList {
  int place[kDsMaxK];  // of kept entries, -1 of others
  float z[kDsMaxK], logp[kDsMaxK];
  int flags, kept;
};

// Reads a row's list; all threads of the block call it.
template <typename T>
__device__ void ds_read_list(const DsArgs& a, int row, const T* l, DsList& sh) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (tid == 0) sh.flags = sh.kept = 0;
  __syncthreads();
  int p = -1;
  if (tid < a.k) {
    const int64_t i = (int64_t)row * a.k + tid;
    p = ds_place(a, i);
    float z = 0.f;
    const float lp = a.logp[i];
    if (p == -2) atomicOr(&sh.flags, VT_DEV_BAD_ID);
    if (p >= 0) {
      z = Elem<T>::load(l + p);
      if (z == -INFINITY) p = -1;
    }
    if (p >= 0 && !(lp < 80.f)) atomicOr(&sh.flags, VT_DEV_NONFINITE);
    if (p >= 0) atomicAdd(&sh.kept, 1);
    sh.place[tid] = p < 0 ? -1 : p;
    sh.z[tid] = z;
    sh.logp[tid] = lp;
  }
  __syncthreads();
  if (p >= 0)
    for (int i = 0; i < tid; ++i)
      if (sh.place[i] == p) atomicOr(&sh.flags, VT_DEV_DUPLICATE_ID);
  __syncthreads();
}

__device__ __forceinline__ double warp_sum(double v) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Loss and statistics of a row, by one warp: from its list and the largest logit
// mr and sum sr (relative to mr; 0: none) of the unlisted ids.
__device__ void ds_finish(const DsArgs& a, const DsList& sh, float mr, double sr, int lane, float& loss,
                          DsStats& st) {
  float m = sr > 0.0 ? mr : -INFINITY;
  for (int i = lane; i < a.k; i += 32)
    if (sh.place[i] >= 0) m = fmaxf(m, sh.z[i]);
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  double S = 0.0, mass = 0.0;
  for (int i = lane; i < a.k; i += 32)
    if (sh.place[i] >= 0) {
      S += (double)exp2_approx((sh.z[i] - m) * a.c);
      const Pair t = pair_exp(Pair{sh.logp[i], 0.f});
      mass += (double)t.h + (double)t.l;
    }
  S = warp_sum(S);
  mass = warp_sum(mass);
  // ln of the unlisted ids' sum, relative to m, which may be far above mr
  const double inv_t = a.inv_t;
  double down = 0.0;
  if (sr > 0.0) {
    down = ((double)mr - (double)m) * inv_t;
    S += sr * exp(down);
  }
  const double b = a.rest && sr > 0.0 ? fmax(0.0, 1.0 - mass) : 0.0;
  const double A = mass + b;
  if (!(A > 0.0)) {  // nothing to learn from this row
    loss = 0.f;
    st = DsStats{0.f, 0.f, 0.f, 0.f, 0.f};
    return;
  }
  // four logarithms at once, one per lane
  double v = lane == 0 ? S : lane == 1 ? sr : lane == 2 ? b : mass;
  v = v > 0.0 ? log(v) : 0.0;
  const double lnS = __shfl_sync(0xffffffffu, v, 0), lnr = __shfl_sync(0xffffffffu, v, 1);
  const double lnb = __shfl_sync(0xffffffffu, v, 2), lna = __shfl_sync(0xffffffffu, v, 3);
  double sum = 0.0;
  for (int i = lane; i < a.k; i += 32)
    if (sh.place[i] >= 0 && sh.logp[i] > -INFINITY) {
      const Pair t = pair_exp(Pair{sh.logp[i], 0.f});
      const double lnp = ((double)sh.z[i] - (double)m) * inv_t - lnS;
      sum += ((double)t.h + (double)t.l) * ((double)sh.logp[i] - lnp);
    }
  sum = warp_sum(sum);
  const double lnq = lnr + down - lnS;
  const double all = inv_t / S, rest = sr > 0.0 ? all * exp(down) : 0.0;
  if (a.rest) {
    if (b > 0.0) sum += b * (lnb - lnq);
    loss = (float)sum;
    st.c_all = (float)(A * all);
    st.c_rest = (float)(A * rest - (b > 0.0 ? inv_t * b / sr : 0.0));
    st.c_t = (float)inv_t;
  } else {
    loss = (float)(sum / mass - lna);
    st.c_all = (float)all;
    st.c_rest = (float)rest;
    st.c_t = (float)(inv_t / mass);
  }
  st.m = m;
  st.mr = sr > 0.0 ? mr : 0.f;
}

__device__ __forceinline__ float nan_f() { return __int_as_float(0x7fc00000); }

template <typename T>
__global__ void __launch_bounds__(kDsNT) distill_loss_kernel(DsArgs a) {
  __shared__ DsList sh;
  __shared__ int hash[4 * kDsMaxK];
  __shared__ float red[kDsWarps], red_s[kDsWarps], red_e[kDsWarps];
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* l = static_cast<const T*>(a.logits) + (int64_t)row * a.ld;
  ds_read_list<T>(a, row, l, sh);
  int flags = sh.flags;
  if (sh.kept == 0 && flags == 0) {  // nothing listed: the row is not read
    if (tid == 0) {
      a.out_loss[row] = 0.f;
      a.stats[row] = DsStats{0.f, 0.f, 0.f, 0.f, 0.f};
    }
    return;
  }
  for (int i = tid; i < 4 * kDsMaxK; i += kDsNT) hash[i] = -1;
  __syncthreads();
  if (tid < a.k && sh.place[tid] >= 0) {
    int h = sh.place[tid] & (4 * kDsMaxK - 1);
    while (atomicCAS(&hash[h], -1, sh.place[tid]) != -1) h = (h + 1) & (4 * kDsMaxK - 1);
  }
  __syncthreads();
  auto listed = [&](int j) {
    for (int h = j & (4 * kDsMaxK - 1); hash[h] != -1; h = (h + 1) & (4 * kDsMaxK - 1))
      if (hash[h] == j) return true;
    return false;
  };
  float m = -INFINITY;
  bool bad = false;
  for (int j = tid; j < a.K; j += kDsNT) {
    const float x = Elem<T>::load(l + j);
    bad |= !(x < INFINITY);
    if (!listed(j)) m = fmaxf(m, x);
  }
  if (__syncthreads_or(bad)) flags |= VT_DEV_NONFINITE;
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  for (int w = 0; w < kDsWarps; ++w) m = fmaxf(m, red[w]);
  float s = 0.f, e = 0.f;
  if (m > -INFINITY)
    for (int j = tid; j < a.K; j += kDsNT) {
      if (listed(j)) continue;
      float t;
      two_sum(s, exp2_approx((Elem<T>::load(l + j) - m) * a.c), s, t);
      e += t;
    }
  for (int o = 16; o > 0; o >>= 1) {
    const float s2 = __shfl_xor_sync(0xffffffffu, s, o), e2 = __shfl_xor_sync(0xffffffffu, e, o);
    float t;
    two_sum(s, s2, s, t);
    e += e2 + t;
  }
  if (lane == 0) red_s[warp] = s, red_e[warp] = e;
  __syncthreads();
  if (warp != 0) return;
  float loss = nan_f();
  DsStats st{loss, loss, loss, loss, loss};
  if (flags == 0) {
    double sr = 0.0;
    for (int w = 0; w < kDsWarps; ++w) sr += (double)red_s[w] + (double)red_e[w];
    ds_finish(a, sh, m, sr, lane, loss, st);
  }
  if (lane == 0) {
    a.out_loss[row] = loss;
    a.stats[row] = st;
    if (flags) atomicOr(a.dev_status, flags);
  }
}

template <typename T> struct Store;
template <> struct Store<float> {
  __device__ static void put(float* p, float v) { *p = v; }
};
template <> struct Store<uint16_t> {
  // round to nearest even; NaN stays NaN
  __device__ static void put(uint16_t* p, float v) {
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(*p) : "f"(v));
  }
};

template <typename T>
__global__ void __launch_bounds__(kDsNT) distill_grad_kernel(DsArgs a) {
  __shared__ DsList sh;
  const int row = blockIdx.x, tid = threadIdx.x;
  const T* l = static_cast<const T*>(a.logits) + (int64_t)row * a.ld;
  T* d = static_cast<T*>(a.grad) + (int64_t)row * a.ld_grad;
  const DsStats st = a.stats[row];
  const float g = a.weight ? a.weight[row] : 1.f;
  if (st.c_all == 0.f && st.c_t == 0.f) {  // nothing to learn: not read
    for (int j = tid; j < a.K; j += kDsNT) Store<T>::put(d + j, 0.f);
    return;
  }
  ds_read_list<T>(a, row, l, sh);  // ahead of the first store: d may be l
  const float cr = g * st.c_rest;
  for (int j = tid; j < a.K; j += kDsNT)
    Store<T>::put(d + j, cr * exp2_approx((Elem<T>::load(l + j) - st.mr) * a.c));
  __syncthreads();
  if (tid < a.k && sh.place[tid] >= 0) {
    const Pair t = pair_exp(Pair{sh.logp[tid], 0.f});
    Store<T>::put(d + sh.place[tid],
                  g * (st.c_all * exp2_approx((sh.z[tid] - st.m) * a.c) - st.c_t * t.h));
  }
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
  a.inv_t = 1.0 / (double)T;
  a.ids = ids;
  a.logp = logp;
  a.inv_map = inv_map;
  a.weight = weight;
  a.out_loss = out_loss;
  a.stats = reinterpret_cast<DsStats*>(stats);
  a.grad = grad;
  a.ld_grad = ld_grad;
  a.dev_status = dev_status;
  return a;
}

int ds_launch_loss(const DsArgs& a, int32_t dtype, cudaStream_t s) {
  VT_RETURN_IF_CUDA(cudaMemsetAsync(a.dev_status, 0, sizeof(int), s));
  if (dtype == VT_F32)
    distill_loss_kernel<float><<<a.R, kDsNT, 0, s>>>(a);
  else
    distill_loss_kernel<uint16_t><<<a.R, kDsNT, 0, s>>>(a);
  VT_RETURN_IF_LAUNCH_FAILED();
  return VT_OK;
}

int ds_launch_grad(const DsArgs& a, int32_t dtype, cudaStream_t s) {
  if (dtype == VT_F32)
    distill_grad_kernel<float><<<a.R, kDsNT, 0, s>>>(a);
  else
    distill_grad_kernel<uint16_t><<<a.R, kDsNT, 0, s>>>(a);
  VT_RETURN_IF_LAUNCH_FAILED();
  return VT_OK;
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
  const int rc = ds_launch_loss(a, logits_dtype, static_cast<cudaStream_t>(stream));
  return rc != VT_OK ? rc : ds_launch_grad(a, logits_dtype, static_cast<cudaStream_t>(stream));
}
