// One step of beam search on sm_103a: the N best continuations of each
// sequence's W beams over the vocabulary, and the states that follow them.
//
// Candidate j of beam w scores s_w + (l_wj - m_w) / T - ln S_w, with m_w = max l
// and S_w = sum 2^((l_wj - m_w) c), c = log2(e) / T.  Within a beam the order is
// that of the logits (ties to the lower id), so N candidates of each beam are
// enough: the row kernel leaves each beam's m, S and N best, the merge takes
// the N best of the W ordered lists.
//
// Scores are compared in fp64.  S itself is a sum of fp32 exponentials, so two
// beams' candidates nearer than kNear are not yet told apart: the merge then
// sums those beams' rows again with pairs of fp32 values, in an order that
// depends on the ids alone (equal beams give equal scores, whatever their rows'
// alignment), and takes the lists again.
#include <cmath>

#include "vt_internal.h"
#include "vt_pair.cuh"
#include "vt_verify_common.cuh"

namespace vt {
namespace {

constexpr int kBsMaxBeams = 32;
constexpr int kBsMaxN = 32;
constexpr int kBsNT = 256;

// Two scores further apart than this are in their true order.  An fp32 weight
// 2^((l - m) c) is off by 2^-22 (the exponential) and by three roundings of its
// argument, whose mean under the softmax is at most ln V <= 15.3: 3e-6 in ln S;
// the sums add 1e-6; twice that for two rows.
constexpr double kNear = 1e-5;

typedef unsigned long long bs_key;
__device__ __forceinline__ bs_key bs_key_of(float v, int id) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return (bs_key)(b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u)) << 32 | (uint32_t)~id;
}
__device__ __forceinline__ float bs_value(bs_key q) {
  const uint32_t o = (uint32_t)(q >> 32);
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ int bs_id(bs_key q) { return (int)~(uint32_t)q; }

// What the row kernel leaves of a beam: its largest logit, S = s + e, how many
// candidates follow and the VT_DEV_* flags of its row
struct BeamRow {
  float m, s, e;
  int n, flags;
};

struct BsArgs {
  const void* logits;
  int64_t ld;
  int B, W, K, N;
  float c;
  double inv_t;
  const float* scores;     // [B][W]
  const uint8_t* done;     // [B][W] or nullptr
  int end_id;
  const int* trim_ids;     // [K] or nullptr
  float* out_scores;       // [B][N]
  int* out_parent;
  int* out_tokens;
  uint8_t* out_done;       // [B][N] or nullptr
  int* dev_status;
  BeamRow* rows;           // [B * W]
  bs_key* best;            // [B * W][N], best first
};

// whether a beam's row of logits is to be read
__device__ __forceinline__ bool bs_live(const BsArgs& a, int row) {
  const float s = a.scores[row];
  return s > -INFINITY && s < INFINITY && !(a.done && a.done[row]);
}

template <typename T>
__global__ void __launch_bounds__(kBsNT) beam_rows_kernel(BsArgs a) {
  __shared__ float red_m[kBsNT / 32], red_s[kBsNT / 32], red_e[kBsNT / 32];
  __shared__ bs_key red_k[kBsNT / 32];
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!bs_live(a, row)) {
    if (tid == 0) {
      const float s = a.scores[row];
      a.rows[row] = BeamRow{0.f, 1.f, 0.f, 0, s == -INFINITY || fabsf(s) < INFINITY ? 0 : VT_DEV_NONFINITE};
    }
    return;
  }
  const T* l = static_cast<const T*>(a.logits) + (int64_t)row * a.ld;
  float m = -INFINITY;
  bool nan = false;
  for (int j = tid; j < a.K; j += kBsNT) {
    const float x = Elem<T>::load(l + j);
    nan |= x != x;
    m = fmaxf(m, x);
  }
  if (nan) m = INFINITY;
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red_m[warp] = m;
  __syncthreads();
  for (int w = 0; w < kBsNT / 32; ++w) m = fmaxf(m, red_m[w]);
  if (!(fabsf(m) < INFINITY)) {  // uniform in the block
    if (tid == 0) a.rows[row] = BeamRow{0.f, 1.f, 0.f, 0, m > 0.f ? VT_DEV_NONFINITE : 0};
    return;
  }
  float s = 0.f, e = 0.f;
  for (int j = tid; j < a.K; j += kBsNT) {
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
  bs_key last = ~0ull;
  int n = 0;
  for (; n < a.N; ++n) {
    bs_key top = 0;
    for (int j = tid; j < a.K; j += kBsNT) {
      const float x = Elem<T>::load(l + j);
      const bs_key q = x > -INFINITY ? bs_key_of(x, j) : 0;
      if (q < last && q > top) top = q;
    }
    for (int o = 16; o > 0; o >>= 1) {
      const bs_key q = __shfl_xor_sync(0xffffffffu, top, o);
      top = q > top ? q : top;
    }
    __syncthreads();
    if (lane == 0) red_k[warp] = top;
    __syncthreads();
    for (int w = 0; w < kBsNT / 32; ++w) top = red_k[w] > top ? red_k[w] : top;
    if (top == 0) break;
    if (tid == 0) a.best[(int64_t)row * a.N + n] = top;
    last = top;
  }
  if (tid == 0) {
    float S = 0.f, E = 0.f;
    for (int w = 0; w < kBsNT / 32; ++w) {
      float t;
      two_sum(S, red_s[w], S, t);
      E += red_e[w] + t;
    }
    a.rows[row] = BeamRow{m, S, E, n, 0};
  }
}

// order of fp64 scores as unsigned integers; 0 comes after every finite score
__device__ __forceinline__ bs_key bs_order(double v) {
  const long long b = __double_as_longlong(v + 0.0);
  return (bs_key)(b ^ ((b >> 63) | (1ll << 63)));
}
__device__ __forceinline__ double bs_score(bs_key q) {
  const long long b = (long long)q;
  return __longlong_as_double(b < 0 ? b ^ (1ll << 63) : ~b);
}

// S of one row again, by all threads of the block: the exponentials and their sum
// as pairs, good to 2^-27.  Thread t takes ids t, t + kBsNT, ...
template <typename T>
__device__ double bs_exact_sum(const BsArgs& a, int row, float m, Pair inv_t, Pair* red) {
  const T* l = static_cast<const T*>(a.logits) + (int64_t)row * a.ld;
  Pair sum{0.f, 0.f};
  for (int j = threadIdx.x; j < a.K; j += kBsNT) {
    const float x = Elem<T>::load(l + j);
    float d, e;
    two_sum(x, -m, d, e);
    if (!((double)d * a.inv_t > -80.0)) continue;  // e^-80 of 2^22 ids is nothing to S >= 1
    const Pair y = pair_exp(pair_mul(Pair{d, e}, inv_t));
    sum = pair_add(sum, y);
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int o = 16; o > 0; o >>= 1) {
    Pair w;
    w.h = __shfl_xor_sync(0xffffffffu, sum.h, o);
    w.l = __shfl_xor_sync(0xffffffffu, sum.l, o);
    sum = pair_add(sum, w);
  }
  __syncthreads();
  if (lane == 0) red[warp] = sum;
  __syncthreads();
  sum = red[0];
  for (int w = 1; w < kBsNT / 32; ++w) sum = pair_add(sum, red[w]);
  return (double)sum.h + (double)sum.l;
}

template <typename T>
__global__ void __launch_bounds__(kBsNT) beam_merge_kernel(BsArgs a) {
  __shared__ bs_key key[kBsMaxBeams][kBsMaxN];
  __shared__ double off[kBsMaxBeams];  // score minus ln S of each beam
  __shared__ float top[kBsMaxBeams];
  __shared__ int count[kBsMaxBeams];
  __shared__ Pair red[kBsNT / 32];
  __shared__ unsigned again;           // beams whose S is summed again
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int W = a.W, N = a.N, row0 = b * W;
  if (b == 0) {  // the call's status word
    __shared__ int flags;
    if (tid == 0) flags = 0;
    __syncthreads();
    int f = 0;
    for (int r = tid; r < a.B * W; r += kBsNT) f |= a.rows[r].flags;
    if (f) atomicOr(&flags, f);
    __syncthreads();
    if (tid == 0) *a.dev_status = flags;
  }
  if (tid < W) {
    const int row = row0 + tid;
    const BeamRow r = a.rows[row];
    const float s = a.scores[row];
    count[tid] = r.n;
    top[tid] = r.m;
    off[tid] = (double)s - log((double)r.s + (double)r.e);
    if (a.done && a.done[row] && fabsf(s) < INFINITY) {
      // a beam that has ended continues once, as it is
      count[tid] = 1;
      key[tid][0] = bs_order((double)s);
    }
  }
  __syncthreads();
  Pair inv_t;
  inv_t.h = (float)a.inv_t;
  inv_t.l = (float)(a.inv_t - (double)inv_t.h);
  unsigned exact = 0;  // beams whose S is the precise one
  for (;;) {
    for (int i = tid; i < W * N; i += kBsNT) {
      const int w = i / N, j = i - w * N;
      if (j < count[w] && !(a.done && a.done[row0 + w])) {
        const float v = bs_value(a.best[(int64_t)(row0 + w) * N + j]);
        key[w][j] = bs_order(((double)v - (double)top[w]) * a.inv_t + off[w]);
      }
    }
    __syncthreads();
    if (warp == 0) {
      // lane w holds beam w's place in its list
      const int mine = lane < W ? count[lane] : 0;
      int at = 0, before = -1;
      double above = 0.0;
      unsigned near = 0;
      for (int n = 0; n <= N; ++n) {
        const bs_key q = at < mine ? key[lane][at] : 0;
        const unsigned hi = __reduce_max_sync(0xffffffffu, (unsigned)(q >> 32));
        const bool h = q != 0 && (unsigned)(q >> 32) == hi;
        const unsigned lo = __reduce_max_sync(0xffffffffu, h ? (unsigned)q : 0u);
        const unsigned who = __ballot_sync(0xffffffffu, h && (unsigned)q == lo);
        if (who == 0) {
          if (lane == 0)
            for (; n < N; ++n) {
              const int64_t o = (int64_t)b * N + n;
              a.out_scores[o] = -INFINITY;
              a.out_parent[o] = a.out_tokens[o] = -1;
              if (a.out_done) a.out_done[o] = 0;
            }
          break;
        }
        const int w = __ffs(who) - 1;  // ties to the lower beam
        const double score = bs_score((bs_key)hi << 32 | lo);
        if (n > 0 && w != before && above - score < kNear) near |= 1u << w | 1u << before;
        above = score;
        before = w;
        if (lane == w && n < N) {
          const int row = row0 + w;
          const bool over = a.done && a.done[row];
          int token = a.end_id;
          if (!over) {
            token = bs_id(a.best[(int64_t)row * N + at]);
            if (a.trim_ids) token = a.trim_ids[token];
          }
          const int64_t o = (int64_t)b * N + n;
          a.out_scores[o] = (float)score;
          a.out_parent[o] = w;
          a.out_tokens[o] = token;
          if (a.out_done) a.out_done[o] = over || token == a.end_id;
        }
        at += lane == w;
      }
      if (lane == 0) again = near;
    }
    __syncthreads();
    // beams that have ended have their scores exactly
    unsigned todo = again & ~exact;
    if (a.done)
      for (int w = 0; w < W; ++w)
        if (a.done[row0 + w]) todo &= ~(1u << w);
    if (todo == 0) break;
    exact |= todo;
    while (todo) {
      const int w = __ffs(todo) - 1;
      todo &= todo - 1;
      const double S = bs_exact_sum<T>(a, row0 + w, top[w], inv_t, red);
      if (tid == 0) off[w] = (double)a.scores[row0 + w] - log(S);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- reordering
constexpr int kBrNT = 128;

// A state's parts: O x B x W x P segments of up to S positions of `row` bytes
struct BrLayout {
  int64_t o, b, w, p, s;  // strides in bytes
};
struct BrArgs {
  const uint8_t* src;
  uint8_t* dst;
  BrLayout from, to;
  int64_t O, P, S, row;
  int B, W, N;
  const int* parent;   // [B][N]
  const int* lengths;  // [B] or nullptr
  int* dev_status;
  int inplace;
};

template <typename V>
__global__ void __launch_bounds__(kBrNT) beam_reorder_kernel(BrArgs a, int64_t pieces) {
  extern __shared__ __align__(16) uint8_t raw[];
  V* const col = reinterpret_cast<V*>(raw) + threadIdx.x;  // this thread's column of W vectors
  __shared__ int par[kBsMaxBeams];
  __shared__ unsigned need;
  __shared__ int flags;
  const int tid = threadIdx.x;
  if (blockIdx.x == 0) {
    if (tid == 0) flags = 0;
    __syncthreads();
    for (int64_t i = tid; i < (int64_t)a.B * a.N; i += kBrNT) {
      const int p = a.parent[i];
      if (p < -1 || p >= a.W) flags = VT_DEV_BAD_ID;
    }
    __syncthreads();
    if (tid == 0) *a.dev_status = flags;
  }
  const int64_t seg = blockIdx.x / pieces, piece = blockIdx.x - seg * pieces;
  const int64_t p = seg % a.P, ob = seg / a.P;
  const int b = (int)(ob % a.B);
  const int64_t o = ob / a.B;
  if (tid < 32) {
    int q = tid < a.N ? a.parent[(int64_t)b * a.N + tid] : -1;
    if (q < 0 || q >= a.W || (a.inplace && q == tid)) q = -1;  // nothing to write
    par[tid] = q;
    const unsigned m = __reduce_or_sync(0xffffffffu, q >= 0 ? 1u << q : 0u);
    if (tid == 0) need = m;
  }
  __syncthreads();
  const unsigned used = need;
  if (used == 0) return;
  int64_t len = a.S;
  if (a.lengths) len = min(len, (int64_t)max(a.lengths[b], 0));
  const int64_t per = a.row / (int64_t)sizeof(V);  // vectors of a position
  const int64_t i = piece * kBrNT + tid;
  const int64_t pos = i / per, rest = (i - pos * per) * (int64_t)sizeof(V);
  if (pos >= len) return;
  const uint8_t* src = a.src + o * a.from.o + b * a.from.b + p * a.from.p + pos * a.from.s + rest;
  uint8_t* dst = a.dst + o * a.to.o + b * a.to.b + p * a.to.p + pos * a.to.s + rest;
  for (int w = 0; w < a.W; ++w)
    if (used >> w & 1) col[w * kBrNT] = *reinterpret_cast<const V*>(src + w * a.from.w);
  for (int n = 0; n < a.N; ++n)
    if (par[n] >= 0) *reinterpret_cast<V*>(dst + n * a.to.w) = col[par[n] * kBrNT];
}

template <typename V>
int launch_reorder(cudaStream_t s, const BrArgs& a) {
  const int64_t per = a.S * (a.row / (int64_t)sizeof(V));
  const int64_t pieces = (per + kBrNT - 1) / kBrNT, blocks = a.O * a.B * a.P * pieces;
  if (blocks > 0x7fffffff) return VT_ERR_UNSUPPORTED;
  const int smem = a.W * kBrNT * (int)sizeof(V);
  VT_RETURN_IF_CUDA(cudaFuncSetAttribute(beam_reorder_kernel<V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kBsMaxBeams * kBrNT * (int)sizeof(V)));
  beam_reorder_kernel<V><<<(unsigned)blocks, kBrNT, smem, s>>>(a, pieces);
  VT_RETURN_IF_LAUNCH_FAILED();
  return VT_OK;
}

size_t select_bytes(int64_t B, int64_t W, int64_t N) {
  return align_up((size_t)(B * W) * sizeof(BeamRow), 256) + (size_t)(B * W * N) * sizeof(bs_key);
}

bool select_sizes_ok(int32_t B, int32_t W, int32_t K, int32_t N) {
  return B >= 1 && W >= 1 && W <= kBsMaxBeams && N >= 1 && N <= kBsMaxN && K >= 1 && K <= (1 << 22) &&
         (int64_t)B * W <= (1 << 24);
}

}  // namespace
}  // namespace vt

extern "C" size_t vt_beam_select_workspace_bytes(int32_t B, int32_t W, int32_t K, int32_t n) {
  if (!vt::select_sizes_ok(B, W, K, n)) return 0;
  return vt::select_bytes(B, W, n);
}

extern "C" int vt_beam_select(const void* logits, int32_t logits_dtype, int32_t B, int32_t W, int32_t K,
                              int64_t ld_logits, const float* scores, const uint8_t* done, int32_t end_id,
                              const int32_t* trim_ids, int32_t n, float temperature, float* out_scores,
                              int32_t* out_parent, int32_t* out_tokens, uint8_t* out_done,
                              int32_t* dev_status, void* workspace, size_t workspace_bytes,
                              void* stream) {
  using namespace vt;
  if (!logits || !scores || !out_scores || !out_parent || !out_tokens || !dev_status)
    return VT_ERR_INVALID_ARG;
  if (logits_dtype != VT_F32 && logits_dtype != VT_BF16) return VT_ERR_INVALID_ARG;
  if (!select_sizes_ok(B, W, K, n) || ld_logits < K) return VT_ERR_INVALID_ARG;
  if (end_id < -1 || ((done || out_done) && end_id < 0) || (done && !out_done)) return VT_ERR_INVALID_ARG;
  if (!(temperature >= 1e-30f && temperature <= 1e30f)) return VT_ERR_INVALID_ARG;
  const int elem = logits_dtype == VT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % elem != 0) return VT_ERR_INVALID_ARG;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 ||
      workspace_bytes < select_bytes(B, W, n))
    return VT_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  BsArgs a;
  a.logits = logits;
  a.ld = ld_logits;
  a.B = B;
  a.W = W;
  a.K = K;
  a.N = n;
  a.c = VT_LOG2E / temperature;
  a.inv_t = 1.0 / (double)temperature;
  a.scores = scores;
  a.done = done;
  a.end_id = end_id;
  a.trim_ids = trim_ids;
  a.out_scores = out_scores;
  a.out_parent = out_parent;
  a.out_tokens = out_tokens;
  a.out_done = out_done;
  a.dev_status = dev_status;
  a.rows = static_cast<BeamRow*>(workspace);
  a.best = reinterpret_cast<bs_key*>(static_cast<uint8_t*>(workspace) +
                                     align_up((size_t)B * W * sizeof(BeamRow), 256));
  if (elem == 4) {
    beam_rows_kernel<float><<<B * W, kBsNT, 0, s>>>(a);
    VT_RETURN_IF_LAUNCH_FAILED();
    beam_merge_kernel<float><<<B, kBsNT, 0, s>>>(a);
  } else {
    beam_rows_kernel<uint16_t><<<B * W, kBsNT, 0, s>>>(a);
    VT_RETURN_IF_LAUNCH_FAILED();
    beam_merge_kernel<uint16_t><<<B, kBsNT, 0, s>>>(a);
  }
  VT_RETURN_IF_LAUNCH_FAILED();
  return VT_OK;
}

extern "C" int vt_beam_reorder(const void* state, void* out, const int64_t* strides,
                               const int64_t* out_strides, int64_t outer, int32_t B, int32_t W, int32_t n,
                               int64_t inner, int64_t positions, int64_t row_bytes,
                               const int32_t* parent, const int32_t* lengths, int32_t* dev_status,
                               void* stream) {
  using namespace vt;
  if (!state || !out || !strides || !out_strides || !parent || !dev_status) return VT_ERR_INVALID_ARG;
  if (B < 1 || W < 1 || W > kBsMaxBeams || n < 1 || n > kBsMaxN || outer < 1 || inner < 1 || positions < 1 ||
      row_bytes < 1)
    return VT_ERR_INVALID_ARG;
  const int64_t big = (int64_t)1 << 40;  // no product below leaves 64 bits
  if (outer > big || inner > big || positions > big || row_bytes > big) return VT_ERR_UNSUPPORTED;
  BrArgs a;
  a.src = static_cast<const uint8_t*>(state);
  a.dst = static_cast<uint8_t*>(out);
  a.from = BrLayout{strides[0], strides[1], strides[2], strides[3], strides[4]};
  a.to = BrLayout{out_strides[0], out_strides[1], out_strides[2], out_strides[3], out_strides[4]};
  a.inplace = state == out;
  uint64_t align = reinterpret_cast<uintptr_t>(state) | reinterpret_cast<uintptr_t>(out) | (uint64_t)row_bytes;
  for (int i = 0; i < 5; ++i) {
    if (strides[i] < 0 || out_strides[i] < 0 || strides[i] > big || out_strides[i] > big)
      return VT_ERR_INVALID_ARG;
    if (a.inplace && strides[i] != out_strides[i]) return VT_ERR_INVALID_ARG;
    align |= (uint64_t)strides[i] | (uint64_t)out_strides[i];
  }
  if (a.inplace && n > W) return VT_ERR_INVALID_ARG;
  // a position that follows the last without a gap is more of the same row
  a.O = outer;
  a.B = B;
  a.W = W;
  a.N = n;
  a.P = inner;
  a.S = positions;
  a.row = row_bytes;
  a.parent = parent;
  a.lengths = lengths;
  a.dev_status = dev_status;
  const double total = (double)outer * B * inner * positions * row_bytes;
  if (total > 1e15) return VT_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (align % 16 == 0) return launch_reorder<uint4>(s, a);
  if (align % 4 == 0) return launch_reorder<uint32_t>(s, a);
  return launch_reorder<uint8_t>(s, a);
}
