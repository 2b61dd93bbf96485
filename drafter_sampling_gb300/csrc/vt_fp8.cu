// The drafter's head in 8-bit floating point (e4m3) on sm_103a.
//
//   quantise   W8[j, h] = e4m3(W[j, h] / s), s = w_scale[j / 128, h / 128] the
//              smallest power of two >= 2^-126 with max |block| <= 448 s
//   product    z[b, j] = out_scale * sum_g sw[j / 128, g] sx[b, g]
//                                    * sum_{h in group g} x8[b, h] W8[j, h]
//              with x8, sx the hidden states quantised by the same rule per
//              row and group of 128 columns
//
// Power-of-two scales make every division exact, so the 8-bit values do not
// depend on how a division rounds, and cost no precision: a floating-point
// format has the same relative step at any scale (a block's largest value
// lands in (224, 448] rather than on 448; at worst one of e4m3's 18 binades
// is not used).  The product takes any fp32 weight scales.
#include <algorithm>
#include <cmath>

#include <cudaTypedefs.h>

#include "vt_common.cuh"
#include "vt_internal.h"
#include "vt_umma.cuh"

namespace vt {
namespace {

constexpr int kQB = 128;  // side of a scale block
// largest K: the quantiser's grid, and far from where 32-bit row counts overflow
constexpr int kMaxRows = 65535 * kQB;

// Exponent e of a block's scale 2^e from the bf16 bits of its largest
// magnitude (sign cleared): the smallest e >= -126 with amax <= 448 * 2^e.
// amax = f 2^p, 1 <= f < 2, 448 = 1.75 * 2^8: e = p - 8, one more when
// f > 1.75 (bf16 mantissa above 0x60).
__device__ __forceinline__ int scale_exponent(uint32_t amax_bf16) {
  const int e = (int)(amax_bf16 >> 7) - 127 - 8 + ((amax_bf16 & 0x7fu) > 0x60u ? 1 : 0);
  return max(e, -126);
}
__device__ __forceinline__ float exact_pow2(int e) {  // -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// two floats to two e4m3 bytes, round to nearest even: a in the low byte
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// one word of two bf16 values times inv (a power of two: exact)
__device__ __forceinline__ uint32_t scale_e4m3x2(uint32_t w, float inv) {
  return e4m3x2(__uint_as_float(w << 16) * inv, __uint_as_float(w & 0xffff0000u) * inv);
}

// ------------------------------------------------------------ weights
constexpr int kQuantNT = 256;
constexpr int kQuantU = kQB * kQB / 8 / kQuantNT;  // 16-byte loads per thread (8)

// The eight bf16 values from column h of row r (zero past the row) as four
// words.  `by` 16: rows of whole 16-byte vectors; 4: W is 4-byte aligned, rows
// may start in the middle of a word, so five words are read and shifted; 2:
// value by value, as is what the words would reach past the matrix.
__device__ __forceinline__ uint4 load_bf16x8(const uint16_t* __restrict__ W, int K, int H, int r,
                                             int h, int by) {
  if (r >= K || h >= H) return make_uint4(0, 0, 0, 0);
  const int64_t at = (int64_t)r * H + h;
  if (by == 16) return __ldg(reinterpret_cast<const uint4*>(W + at));
  uint32_t w[5];
  if (by == 4 && at + 10 <= (int64_t)K * H) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(W) + (at >> 1);
    const unsigned shift = (unsigned)(at & 1) * 16;
#pragma unroll
    for (int e = 0; e < 5; ++e) w[e] = __ldg(p + e);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = __funnelshift_r(w[e], w[e + 1], shift);
    const int left = H - h;  // values of this row
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (2 * e + 2 > left) w[e] = 2 * e + 1 > left ? 0u : w[e] & 0xffffu;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (h + e < H) w[e >> 1] |= (uint32_t)__ldg(W + at + e) << (16 * (e & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One CTA per 128 x 128 block: the block is read once (eight 16-byte loads
// in flight per thread), its largest magnitude reduced, and the registers
// scaled, rounded and stored.  HBM-bound: 2 bytes read, 1 written per weight
// (K = 128256, H = 4096: 219 us, 7.2 TB/s; K = 32768, H = 2048: 32 us, 6.3 TB/s;
// rows that are read by shifted words, H = 2047: 53 us).
__global__ void __launch_bounds__(kQuantNT)
quantize_head_kernel(const uint16_t* __restrict__ W, int K, int H, uint8_t* __restrict__ W8,
                     int64_t ldw, float* __restrict__ w_scale, int* __restrict__ dev_status,
                     int by) {
  __shared__ uint32_t smax[kQuantNT / 32];
  const int tid = threadIdx.x;
  const int r0 = blockIdx.y * kQB, h = blockIdx.x * kQB + (tid & 15) * 8;
  uint4 v[kQuantU];
  uint32_t mx = 0;  // largest magnitudes of the even and odd columns, packed
#pragma unroll
  for (int i = 0; i < kQuantU; ++i)
    v[i] = load_bf16x8(W, K, H, r0 + i * (kQuantNT / 16) + (tid >> 4), h, by);
#pragma unroll
  for (int i = 0; i < kQuantU; ++i) {
    mx = __vmaxu2(mx, v[i].x & 0x7fff7fffu);
    mx = __vmaxu2(mx, v[i].y & 0x7fff7fffu);
    mx = __vmaxu2(mx, v[i].z & 0x7fff7fffu);
    mx = __vmaxu2(mx, v[i].w & 0x7fff7fffu);
  }
  uint32_t m = max(mx >> 16, mx & 0xffffu);
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) smax[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQuantNT / 32; ++w) m = max(m, smax[w]);
  const int e = scale_exponent(m);
  const float inv = exact_pow2(-e);
  if (tid == 0) {
    griddep_wait();  // the status word is clear
    w_scale[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = exact_pow2(e);
    if (m >= 0x7f80u) atomicOr(dev_status, VT_DEV_NONFINITE);
  }
#pragma unroll
  for (int i = 0; i < kQuantU; ++i) {
    const int r = r0 + i * (kQuantNT / 16) + (tid >> 4);
    if (r >= K || h >= H) continue;
    uint2 o;
    o.x = scale_e4m3x2(v[i].x, inv) | scale_e4m3x2(v[i].y, inv) << 16;
    o.y = scale_e4m3x2(v[i].z, inv) | scale_e4m3x2(v[i].w, inv) << 16;
    uint8_t* q = W8 + (int64_t)r * ldw + h;
    if (h + 8 <= H) {  // ldw % 16 == 0 and W8 is 16-byte aligned
      *reinterpret_cast<uint2*>(q) = o;
    } else {
#pragma unroll
      for (int b = 0; b < 8; ++b)
        if (h + b < H) q[b] = (uint8_t)((b < 4 ? o.x >> (8 * b) : o.y >> (8 * (b - 4))) & 0xffu);
    }
  }
}

// ------------------------------------------------------- hidden states
// Quantises hidden [B, H] to x8 [B, ldx] (columns H..ldx zero) and sx
// [groups][Bp] (rows B..Bp zero), one warp per (row, group of 128 columns).
// A group with a NaN or an infinity gets the scale NaN, so that row's logits
// are NaN.  The product starts over it and loads weights meanwhile, so that it
// adds 0.3 to 0.5 us to a call of 16 rows.
__global__ void __launch_bounds__(256)
quantize_hidden_kernel(const uint16_t* __restrict__ hidden, int B, int H, uint8_t* __restrict__ x8,
                       int ldx, float* __restrict__ sx, int Bp, int groups, int vec_ok,
                       int* __restrict__ status, int status_reset) {
  griddep_launch_dependents();  // the product prefetches weights before its own wait
  griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0 && status_reset) *status = 0;
  const int64_t wid = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int b = (int)(wid / groups), g = (int)(wid % groups);
  if (b >= Bp) return;
  if (b >= B) {
    if (lane == 0) sx[(int64_t)g * Bp + b] = 0.f;
    return;
  }
  const int h = g * kQB + 4 * lane;
  const uint16_t* p = hidden + (int64_t)b * H + h;
  uint2 v = make_uint2(0, 0);
  if (vec_ok) {  // H % 4 == 0 and 8-byte aligned rows
    if (h < H) v = *reinterpret_cast<const uint2*>(p);
  } else {
    if (h < H) v.x = p[0];
    if (h + 1 < H) v.x |= (uint32_t)p[1] << 16;
    if (h + 2 < H) v.y = p[2];
    if (h + 3 < H) v.y |= (uint32_t)p[3] << 16;
  }
  const uint32_t mx = __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu);
  const uint32_t m = __reduce_max_sync(0xffffffffu, max(mx >> 16, mx & 0xffffu));
  const int e = scale_exponent(m);
  const float inv = exact_pow2(-e);
  *reinterpret_cast<uint32_t*>(x8 + (int64_t)b * ldx + h) =
      scale_e4m3x2(v.x, inv) | scale_e4m3x2(v.y, inv) << 16;
  if (lane == 0)
    sx[(int64_t)g * Bp + b] = m >= 0x7f80u ? __int_as_float(0x7fc00000) : exact_pow2(e);
}

// --------------------------------------------------------------- product
struct Fp8Args {
  umma::HeadArgs h;     // batch, sizes, outputs and partials as in the bf16 projection
  const float* sw;      // [K / 128][groups]
  const float* sx;      // [groups][Bp]
  int Bp, groups, nchunk;
  int items;            // blocks of W8 rows times batch chunks
  int give_up;          // self-test: from this item of a CTA on, the promoting threads act as if
                        // a wait had run out (-1: never)
  int vec_out;          // the output's rows are 16-byte aligned
};

constexpr int kMaxGroups = 512;   // H <= 65536
constexpr int kScaleSlots = 8;    // groups whose sx are in shared memory at once

// Two kernels, by the batch.  Up to 64 rows (head_fp8_kernel) the batch is the
// MMA's N operand, 128 rows of W8 its M: the weights are streamed at N = 16,
// 32 or 64, whichever holds the batch.  Wider batches (batch_fp8_kernel) are
// the M operand and 256 rows of W8 the N: a promoting thread then has one
// batch row, so one factor sw * sx a group instead of one per column (the
// factors' shared-memory reads cost as much as the MMAs otherwise).

// z of row j as a key that ascends with z and, at equal z, with descending j
// (-0 counts as +0); a non-finite z is above all.  No key of a row is 0.
constexpr uint32_t kKeyNonFinite = 0xffffffffu;
__device__ __forceinline__ uint64_t greedy_key(float z, int j) {
  const uint32_t u = __float_as_uint(z + 0.f);
  const uint32_t o = !isfinite(z) ? kKeyNonFinite : (u >> 31) ? ~u : u | 0x80000000u;
  return (uint64_t)o << 32 | (uint32_t)~j;
}
__device__ __forceinline__ uint64_t max_key(uint64_t x, uint64_t y) { return x > y ? x : y; }

// Folds N columns' keys over the 8 lanes that share lane % 4, halving the
// columns that a lane holds while it can: lane l ends with the keys of
// max(1, N / 8) columns, the first of which is returned.
template <int N>
__device__ __forceinline__ int fold_keys(uint64_t (&key)[N], int lane) {
  int first = 0, n = N;
#pragma unroll
  for (int o = 16; o >= 4; o >>= 1) {
    if (n > 1) {
      n /= 2;
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        if (j >= n) break;
        const uint64_t send = up ? key[j] : key[j + n], keep = up ? key[j + n] : key[j];
        key[j] = max_key(keep, __shfl_xor_sync(0xffffffffu, send, o));
      }
      first += up ? n : 0;
    } else {
      key[0] = max_key(key[0], __shfl_xor_sync(0xffffffffu, key[0], o));
    }
  }
  return first;
}

// columns (batch rows) and warps that promote a narrow tile
template <int BN>
constexpr int kPartCols = BN < 32 ? BN : 32;  // columns whose partials are reduced at once
constexpr int kNarrowBufs = 4;                // accumulator buffers in tensor memory
constexpr int kNarrowNP = 128;                // promoting threads
constexpr int kNarrowNT = kNarrowNP + 64;     // and a warp for the loads, one for the MMAs

template <bool kTwo>
__device__ __forceinline__ void mma_e4m3(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  if constexpr (kTwo)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor of kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), e4m3
// A and B (7-9 and 10-12 = 0), both K-major, N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Counterparts for a pair of CTAs (a cluster of two) of the single-CTA helpers.
// Barriers of the pair's first CTA are named by their cluster address.
__device__ __forceinline__ uint32_t first_cta(const void* p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(umma::smem_u32(p)));
  return r;
}
__device__ __forceinline__ void pair_load_2d(void* dst, const CUtensorMap* map, int x, int y,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(umma::smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// arrive on `bar` of both CTAs once every MMA issued so far has completed
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(umma::smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// What is handed over with this arrival is tensor memory only: accumulators that
// have been read, and scales that have been written, for the first CTA's MMAs.
// A caller has waited for its loads and stores of tensor memory to complete
// (tcgen05.wait::ld, ::st) and ordered them before the arrival
// (tcgen05.fence::before_thread_sync; the issuing warp has the ::after one), so
// it needs no release at cluster scope, which is for other memory and would cost
// some 1000 cycles a group.
__device__ __forceinline__ void remote_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   umma::smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// one thread of a converged warp, the same at every call
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}

// two fp32 values in one 64-bit register
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(uint32_t a, uint32_t b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void add2(f32x2& acc, f32x2 a) {
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(acc) : "l"(a));
}
__device__ __forceinline__ void fma2(f32x2& acc, f32x2 a, f32x2 b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}

// 8 NB consecutive columns of this warp's 32 TMEM lanes, spread over the warp
// so that a thread has few columns and several rows (so few scales): thread t
// gets of column block k the columns 8 k + 2 (t % 4) + {0, 1} of the rows
// t / 4 + 8 i: pairs r[i / 2][4 k + 2 (i % 2)], + 1.  The registers hold them
// after tmem_ld_wait.
template <int NB>
__device__ __forceinline__ void tmem_ld_spread(uint32_t taddr, uint32_t (&r)[2][NB * 4]) {
  static_assert(NB == 2 || NB == 4, "16 or 32 columns");
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // lanes 0-15 and 16-31
    const uint32_t at = taddr + ((uint32_t)(16 * h) << 16);
    if constexpr (NB == 4) {
      asm volatile(
          "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
          "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
          : "=r"(r[h][0]), "=r"(r[h][1]), "=r"(r[h][2]), "=r"(r[h][3]), "=r"(r[h][4]),
            "=r"(r[h][5]), "=r"(r[h][6]), "=r"(r[h][7]), "=r"(r[h][8]), "=r"(r[h][9]),
            "=r"(r[h][10]), "=r"(r[h][11]), "=r"(r[h][12]), "=r"(r[h][13]), "=r"(r[h][14]),
            "=r"(r[h][15])
          : "r"(at)
          : "memory");
    } else {
      asm volatile(
          "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
          : "=r"(r[h][0]), "=r"(r[h][1]), "=r"(r[h][2]), "=r"(r[h][3]), "=r"(r[h][4]),
            "=r"(r[h][5]), "=r"(r[h][6]), "=r"(r[h][7])
          : "r"(at)
          : "memory");
    }
  }
}
// Waits for this thread's TMEM loads; it names the registers of one, so that
// no use of them can precede it.
template <int NB>
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[2][NB * 4]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < NB * 4; ++e) asm volatile("" : "+r"(r[h][e])::"memory");
}

// Moves registers between the warpgroups of a block: the sum over the
// warpgroups stays what the block was launched with.
template <int N>
__device__ __forceinline__ void regs_give() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Narrow batches: tiles of 128 rows of W8, taken by a persistent CTA one after
// another, with the batch (BN rows) as the N operand.  Each group of 128
// reduction columns is one shared-memory stage (W8 128 x 128 bytes, x8 BN x 128
// bytes, both K-major with the 128-byte swizzle) and one tcgen05 accumulation of four K = 32 steps
// into one of the tensor-memory buffers.  The promoting warps read each
// finished buffer, give it back at once, and add it, times sw * sx, to fp32
// sums in registers: the scales of a group multiply its partial sum only, and
// the long sum is held in 32 bits by the CUDA cores.  One warp issues the TMA
// loads (and the copies of sx, in a ring of its own, so that a stage is free
// as soon as its MMAs are done) and one the MMAs; both run ahead into the next
// tile while the promoting warps store the last one.
//
// Bound by HBM and by how a call starts: B = 16, K = 32768, H = 2048 takes 13.7 us
// (5.0 TB/s; the weights alone are 9.9), of which 1.5 are the launch, 2.3 pass
// from the first request for weights to the first MMA, 7 are the stream (6.7 of
// HBM at its copy rate) and 0.6 the last tile's rows.  B = 1: 13.6, B = 64: 15.6.
// One row and all columns per promoting thread, rather than four rows and a
// quarter of the columns, cost as much time in broadcast reads of the columns'
// scales as the MMAs take.  One CTA per SM with twice the ring: 16.3.
template <int BN>
__global__ void __launch_bounds__(kNarrowNT, 2)
head_fp8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                Fp8Args fa) {
  using namespace umma;
  const HeadArgs& a = fa.h;
  static_assert(BN <= 64, "wider batches have their own kernel");
  constexpr int NP = kNarrowNP;
  constexpr int kPromWarps = NP / 32;
  constexpr int NBUF = kNarrowBufs;
  constexpr int CW = BN;                // columns of a promoting warp, which has 32 of the rows
  constexpr int NB = CW >= 32 ? 4 : 2;  // 8-column blocks read at once
  constexpr int PC = kPartCols<BN>;
  constexpr uint32_t kCols = (uint32_t)(NBUF * BN);  // 64..256, a power of two
  constexpr int stage_bytes = kABytes + BN * 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t full_bar[kMaxStages], empty_bar[kMaxStages];
  __shared__ __align__(8) uint64_t sx_full[kScaleSlots], sx_empty[kScaleSlots];
  __shared__ __align__(8) uint64_t acc_full[NBUF], acc_empty[NBUF];
  __shared__ __align__(8) uint64_t done_bar;
  __shared__ __align__(16) float sx_sh[kScaleSlots][BN];
  __shared__ float sw_sh[kMaxGroups];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int s_err;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = a.stages;
  const int nk = fa.groups;
  const int items = fa.items;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(&sx_full[s], 1);
      mbar_init(&sx_empty[s], kPromWarps);
    }
    for (int p = 0; p < NBUF; ++p) {
      mbar_init(&acc_full[p], 1);
      mbar_init(&acc_empty[p], kPromWarps);
    }
    mbar_init(&done_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_err = 0;
    tma_prefetch_map(&map_w);
    tma_prefetch_map(&map_x);
  }
  if (warp == kPromWarps + 1) {
    tmem_alloc(&tmem_base_sh, kCols);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = tmem_base_sh;

  // Tiles start their reduction at different groups, so the rows streamed at
  // any moment are spread over column offsets (DRAM channels).  The loops below
  // count stages, slots and groups up by hand: a division by a runtime value in
  // each would be most of the time between two groups.
  if (warp >= kPromWarps) {
    const bool leader = elect_one();  // one thread issues; the warp stays together
    if (warp == kPromWarps) {
      // TMA producer: the first stages' weights before the wait on the
      // kernel that quantises the hidden states
      const int pre = min(S, nk);
      if (leader) {
        int g = (int)blockIdx.x % nk;
        for (int kb = 0; kb < pre; ++kb) {
          mbar_expect_tx(&full_bar[kb], (uint32_t)stage_bytes);
          tma_load_2d(smem + (size_t)kb * stage_bytes, &map_w, g * 128, (int)blockIdx.x * kBM,
                      &full_bar[kb]);
          g = g + 1 == nk ? 0 : g + 1;
        }
      }
      griddep_wait();
      int it = 0;                     // groups requested so far
      int s = 0, q = 0;               // stage and scale slot of the next one
      uint32_t sphase = 1, qphase = 1;  // parity that says they are free
      bool ok = true;
      for (int tile = blockIdx.x; tile < items && ok; tile += gridDim.x) {
        int g = tile % nk;
        for (int kb = 0; kb < nk; ++kb, ++it) {
          uint8_t* st = smem + (size_t)s * stage_bytes;
          if (it >= pre) {
            // a fresh barrier counts as having completed the phase before
            ok = mbar_wait(&empty_bar[s], sphase);
            if (!ok) break;
            if (leader) {
              mbar_expect_tx(&full_bar[s], (uint32_t)stage_bytes);
              tma_load_2d(st, &map_w, g * 128, tile * kBM, &full_bar[s]);
            }
          }
          if (leader) tma_load_2d(st + kABytes, &map_x, g * 128, 0, &full_bar[s]);
          ok = mbar_wait(&sx_empty[q], qphase);
          if (!ok) {
            ++it;
            break;
          }
          if (leader) {
            mbar_expect_tx(&sx_full[q], BN * 4);
            bulk_load(sx_sh[q], fa.sx + (int64_t)g * fa.Bp, BN * 4, &sx_full[q]);
          }
          if (++s == S) {
            s = 0;
            sphase ^= 1;
          }
          if (++q == kScaleSlots) {
            q = 0;
            qphase ^= 1;
          }
          g = g + 1 == nk ? 0 : g + 1;
        }
      }
      if (!ok) atomicExch(&s_err, 1);
      // drain: every issued copy has landed before this CTA may exit
      for (int k = max(0, it - S); k < it; ++k) mbar_wait(&full_bar[k % S], (k / S) & 1);
      for (int k = max(0, it - kScaleSlots); k < it; ++k)
        mbar_wait(&sx_full[k % kScaleSlots], (k / kScaleSlots) & 1, ok ? kWaitLimit : 1u << 12);
    } else if (warp == kPromWarps + 1) {
      // MMA issuer.  The limits of its waits do not count what the kernels ahead take.
      griddep_wait();
      constexpr uint32_t idesc = idesc_e4m3(kBM, BN);
      const uint64_t desc0 = sw128_desc(smem_u32(smem));
      int s = 0, p = 0;
      uint32_t sphase = 0, pphase = 1;
      bool ok = true;
      for (int tile = blockIdx.x; tile < items && ok; tile += gridDim.x)
        for (int kb = 0; kb < nk; ++kb) {
          ok = __all_sync(0xffffffffu,
                          mbar_wait(&acc_empty[p], pphase) && mbar_wait(&full_bar[s], sphase)) != 0;
          if (!ok) break;
          fence_after_sync();
          if (leader) {
            const uint64_t adesc = desc0 + (uint64_t)(s * (stage_bytes >> 4));
            const uint64_t bdesc = adesc + (kABytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 32 elements = 32 bytes per step
              mma_e4m3<false>(tmem + (uint32_t)(p * BN), adesc + 2 * kk, bdesc + 2 * kk, idesc,
                              kk > 0 ? 1u : 0u);
            mma_commit(&empty_bar[s]);
            mma_commit(&acc_full[p]);
          }
          if (++s == S) {
            s = 0;
            sphase ^= 1;
          }
          if (++p == NBUF) {
            p = 0;
            pphase ^= 1;
          }
        }
      if (!ok) atomicExch(&s_err, 1);
      if (leader) mma_commit(&done_bar);
    }
  } else {
    griddep_wait();
    const int quad = warp;
    // this thread's first row of the tile (TMEM lane) and first column; it
    // has the rows row0 + 8 i and the columns 8 k + cpair + {0, 1}
    const int row0 = quad * 32 + (lane >> 2), cpair = 2 * (lane & 3);
    // one block of columns transposed, for the partials
    float* zt = reinterpret_cast<float*>(smem + (size_t)S * stage_bytes);
    int it = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < items; tile += gridDim.x) {
      const int m0 = tile * kBM;
      // the last item's weights' scales have been read by all
      asm volatile("bar.sync 1, %0;" ::"n"(NP) : "memory");
      for (int g = tid; g < nk; g += NP) sw_sh[g] = fa.sw[(int64_t)tile * nk + g];
      asm volatile("bar.sync 1, %0;" ::"n"(NP) : "memory");
      // greedy: the tile's part of the one-hot q, while the first weights are
      // on their way; the 1 follows once all tiles are done
      if (a.greedy) {
        for (int b = warp; b < a.B; b += kPromWarps) {
          float* to = a.out + (int64_t)b * a.ldo + m0;
          if (fa.vec_out && m0 + kBM <= a.K) {
            reinterpret_cast<float4*>(to)[lane] = make_float4(0.f, 0.f, 0.f, 0.f);
          } else {
#pragma unroll
            for (int e = 0; e < kBM; e += 32)
              if (m0 + e + lane < a.K) to[e + lane] = 0.f;
          }
        }
      }
      f32x2 acc[CW / 8][4];  // [column block][row]
#pragma unroll
      for (int k = 0; k < CW / 8; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[k][i] = 0;
      if (tile == (int)blockIdx.x + fa.give_up * (int)gridDim.x) ok = false;
      int g = tile % nk;
      for (int kb = 0; kb < nk && ok; ++kb, ++it) {
        const int q = it % kScaleSlots, p = it % NBUF;
        ok = mbar_wait(&sx_full[q], (it / kScaleSlots) & 1) &&
             mbar_wait(&acc_full[p], (it / NBUF) & 1);
        ok = __all_sync(0xffffffffu, ok) != 0;
        if (!ok) break;
        fence_after_sync();
        const uint32_t swb = __float_as_uint(sw_sh[g]);
        g = g + 1 == nk ? 0 : g + 1;
        const f32x2 sw = pack2(swb, swb);
        const float* sxq = sx_sh[q] + cpair;
        const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(p * BN);
        uint32_t raw[2][2][NB * 4];
        tmem_ld_spread<NB>(taddr, raw[0]);
#pragma unroll
        for (int k0 = 0; k0 < CW / 8; k0 += NB) {
          // the next block's load overlaps this one's arithmetic
          uint32_t (&v)[2][NB * 4] = raw[(k0 / NB) & 1];
          tmem_ld_wait<NB>(v);
          if (k0 + NB < CW / 8) {
            tmem_ld_spread<NB>(taddr + 8 * (k0 + NB), raw[(k0 / NB + 1) & 1]);
          } else {  // all of this warp's columns are in registers
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[p]);
          }
#pragma unroll
          for (int k = 0; k < NB; ++k) {
            const f32x2 f =
                mul2(*reinterpret_cast<const f32x2*>(sxq + 8 * (k0 + k)), sw);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t* e = &v[i / 2][4 * k + 2 * (i % 2)];
              fma2(acc[k0 + k][i], pack2(e[0], e[1]), f);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sx_empty[q]);
      }
      // a warp that gave up misses no barrier; logits, whose call returns no
      // status word, are NaN then, and with one nothing more is stored
      if (a.part == nullptr) {
        const float scale = ok ? a.out_scale : __int_as_float(0x7fc00000);
#pragma unroll
        for (int k = 0; k < CW / 8; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 z = unpack2(acc[k][i]);
            const int b = 8 * k + cpair, j = m0 + row0 + 8 * i;
            if (j < a.K) {
              if (b < a.B) a.out[(int64_t)b * a.ldo + j] = z.x * scale;
              if (b + 1 < a.B) a.out[(int64_t)(b + 1) * a.ldo + j] = z.y * scale;
            }
          }
      } else if (a.greedy) {
        // each column's best key: over this thread's rows, the warp's, the tile's
        uint64_t* best = reinterpret_cast<uint64_t*>(zt);  // [warp][column]
#pragma unroll
        for (int c = 0; c < BN; c += PC) {
          uint64_t key[PC / 4];
#pragma unroll
          for (int k = 0; k < PC / 4; ++k) {
            // seen is NaN once a z is not finite
            float top = -INFINITY, seen = 0.f;
            int j = m0 + row0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 zz = unpack2(acc[c / 8 + k / 2][i]);
              const float z = (k % 2 ? zz.y : zz.x) * a.out_scale;
              if (m0 + row0 + 8 * i < a.K) {
                seen = fmaf(z, 0.f, seen);
                if (z > top) {
                  top = z;
                  j = m0 + row0 + 8 * i;
                }
              }
            }
            key[k] = m0 + row0 < a.K ? greedy_key(top + seen, j) : 0;
          }
          const int n = fold_keys(key, lane);
          best[warp * BN + c + 8 * (n / 2) + cpair + n % 2] = key[0];
        }
        asm volatile("bar.sync 1, %0;" ::"n"(NP) : "memory");
        if (tid < a.B) {
          uint64_t key = best[tid];
#pragma unroll
          for (int w = 1; w < kPromWarps; ++w) key = max_key(key, best[w * BN + tid]);
          reinterpret_cast<uint64_t*>(a.part)[(int64_t)tile * a.B + tid] = key;
        }
      } else {
#pragma unroll
        for (int c = 0; c < BN; c += PC) {
#pragma unroll
          for (int k = 0; k < PC / 8; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float2 z = unpack2(acc[c / 8 + k][i]);
              z.x *= a.out_scale;
              z.y *= a.out_scale;
              const int col = 8 * k + cpair, b = c + col, r = row0 + 8 * i;
              if (ok && m0 + r < a.K) {
                if (b < a.B) a.out[(int64_t)b * a.ldo + m0 + r] = z.x;
                if (b + 1 < a.B) a.out[(int64_t)(b + 1) * a.ldo + m0 + r] = z.y;
              }
              zt[col * zt_pitch<PC, NP>() + r] = z.x;
              zt[(col + 1) * zt_pitch<PC, NP>() + r] = z.y;
            }
          asm volatile("bar.sync 1, %0;" ::"n"(NP) : "memory");
          tile_partials<PC, NP>(zt, a, min(kBM, a.K - m0), m0, tile, tid, c);
          asm volatile("bar.sync 1, %0;" ::"n"(NP) : "memory");
        }
      }
    }
    if (!ok && lane == 0) atomicExch(&s_err, 1);
  }
  __syncwarp();
  __syncthreads();  // every role has finished or given up: no wait counts another's work
  // the MMAs have completed
  const bool all_ok = __syncthreads_and(mbar_wait(&done_bar, 0) && s_err == 0 ? 1 : 0) != 0;
  griddep_launch_dependents();
  fence_after_sync();
  if (tid == 0 && !all_ok) atomicOr(a.status, VT_DEV_TIMEOUT);
  if (warp == kPromWarps + 1) tmem_dealloc(tmem, kCols);
}

// Threads of batch_fp8_kernel: two promoting warpgroups, and a third of which
// one warp issues the loads and one the MMAs.  A promoting thread sums 128
// values and reads another 32 at a time, more registers than an even split over
// the block gives, so the third warpgroup gives most of its own to the others:
// 3 x 168 = 2 x 224 + 56 a thread, with which neither side's loops spill (with 2 x
// 232 + 40 the issuing warp's did; B = 1000: 124 against 119 us).
constexpr int kBatchNP = 256;                // promoting threads
constexpr int kBatchNT = kBatchNP + 128;     // and a warpgroup: loads, MMAs, two idle warps
constexpr int kBatchRowsW = 256;             // rows of W8 of an item: two tiles of 128
constexpr int kTurn = 4;                     // groups whose scales are handed over at once
constexpr int kUnit = 16;                    // groups that the tensor cores sum up
constexpr int kTurns = 4;                    // turns whose scales are in tensor memory at once
constexpr int kGroupCols = 16;               // tensor-memory columns of a group's scales
// floats: a warp's 32 x 32 block on its way out; 16-byte accesses by row and by
// column of eight lanes then meet all banks
constexpr int kOutPitch = 36;

// MMA whose products of 32 elements are scaled by a power of two per row of A and
// per row of B: one byte each, the exponent plus 127, in tensor memory (bits 4-5
// and 29-30 of the descriptor name the byte of a word; all four hold the same
// here).
template <bool kTwo>
__device__ __forceinline__ void mma_e4m3_scaled(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                                uint32_t idesc, uint32_t scale_a, uint32_t scale_b,
                                                uint32_t accumulate) {
  if constexpr (kTwo)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(scale_a), "r"(scale_b), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(scale_a), "r"(scale_b), "r"(accumulate)
        : "memory");
}
// Its instruction descriptor: e4m3 A and B, both K-major, N >> 3 at bit 17,
// scales in ue8m0 (bit 23), M >> 7 at bit 27.
__host__ __device__ constexpr uint32_t idesc_e4m3_scaled(int M, int N) {
  return ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27);
}
// The scales of 128 rows of an operand and one group: row 32 c + l is in lane l
// of column c, and in the same lane of the other three quarters of the lanes.
// This writes A's four columns and B's eight, whose rows have one scale per 128.
__device__ __forceinline__ void tmem_st_scales(uint32_t taddr, const uint32_t (&x)[4], uint32_t w0,
                                               uint32_t w1) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %5, %5, %5};" ::"r"(taddr),
      "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(w0)
      : "memory");
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %1, %1, %1};" ::"r"(taddr + 8),
               "r"(w1)
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// a normal power of two, which ue8m0 holds as the float's exponent bits
__device__ __forceinline__ bool is_pow2(float s) {
  const uint32_t u = __float_as_uint(s);
  return (u & 0x807fffffu) == 0 && u - 0x00800000u < 0x7f000000u;
}
// four times the exponent byte of a power of two (or of NaN, which is ue8m0's too)
__device__ __forceinline__ uint32_t ue8m0x4(float s) {
  return (__float_as_uint(s) >> 23 & 0xffu) * 0x01010101u;
}
// Tensor-memory columns of a turn's scales: those of even and odd turns are where
// the accumulators of the two halves are in units of one group.
__device__ __forceinline__ uint32_t scale_cols(int t) {
  static_assert(kTurns * kTurn * kGroupCols == kBatchRowsW, "they share an accumulator's columns");
  return (uint32_t)(kBatchRowsW + (t & 1) * 128 + (t % kTurns / 2) * kTurn * kGroupCols);
}
// barrier of n threads that also tells whether x holds in all of them
__device__ __forceinline__ bool barrier_and(int id, int n, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

// Wide batches: items of 256 rows of W8 x 128 batch rows, or, as a pair of CTAs
// (TWO), x 256 batch rows with one MMA of 256 x 256: each CTA of a pair stages
// its 128 batch rows and half of the weights, two thirds of the shared-memory
// traffic of the same work on one CTA.  The roles are those of
// head_fp8_kernel; in a pair the first CTA issues the MMAs for both and holds
// the barriers that they wait on.
//
// Single CTAs promote every group: its sums are read, and added times sw * sx to
// fp32 sums in registers, while the next group is summed in the other of two
// accumulators.  So do pairs with any scales that are not powers of two.
// Where all weight scales of an item are powers of two, as this library's
// quantiser leaves them, a pair has the tensor cores scale the products: both
// scales of a group are then bytes in tensor memory (where the second accumulator
// would be), written by the promoting warps up to four turns of four groups
// ahead, and a unit of up to 16 groups is summed there before it is read.  MMAs
// stand still while tensor memory is read, some 380 cycles for a group's sums; a
// pair is bound by its MMAs and gains from fewer reads (K = 38016, H = 4096: B = 256
// 40.2 against 44.5 us, B = 1000 119 against 156), a single CTA, whose three
// stages leave it waiting for loads, does not (K = 20000, H = 8192, B = 128: 40.7
// against 44.0 scaled; B = 300: 59.9 against 60.3).
//
// The tensor cores hold the running sum in fp32 but cut off, rather than round,
// each addition, so the unit's length is a choice between digits and speed.  Off
// in the 2-norm at H = 4096 / 8192, and us at B = 256 / 1000 (K = 38016, H = 4096):
// units of 8 groups 0.7 / 0.8e-7, 44.9 / 144; of 16, 1.1 / 1.1e-7, 40.2 / 119; of 32,
// 2.1 / 2.1e-7, 39.8 / 112.  A plain fp32 product is off by 0.8 / 1.2e-7, groups that
// are promoted one by one by 0.7 / 1.0e-7, so 16 keeps fp32's digits.
//
// What bounds it, at B = 1000, K = 38016, H = 4096 (119 us, 2620 TFLOP/s): the loads'
// latency.  A group is 513 cycles of MMAs, about 660 pass, of which 180 are waits for
// the loads.  No unit is saturated (tensor pipe 60%, L2 44%), but 160 KB on their way
// to each SM at 10.5 TB/s over all are 2.3 us of loaded latency; four stages
// instead of five cost 5%.  Two accumulators of 128 columns in turn, to hide the
// reads, made every MMA slower: they read the batch's stage twice, and shared
// memory has the loads' traffic too (161 against 129 us, at an earlier step).  A
// row's 64 instead of 128 bytes out in one piece, for a sixth stage: 10 us slower.
template <bool TWO, bool PART>
__global__ void __launch_bounds__(kBatchNT, 1)
batch_fp8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                 Fp8Args fa) {
  using namespace umma;
  const HeadArgs& a = fa.h;
  constexpr int kPromWarps = kBatchNP / 32;
  constexpr int NR = kBatchRowsW;
  constexpr int kXBytes = kBM * 128;      // 128 batch rows
  constexpr int WR = TWO ? NR / 2 : NR;   // and as many rows of W8
  constexpr int stage_bytes = kXBytes + WR * 128;
  constexpr int kCtas = TWO ? 2 : 1;
  constexpr uint32_t kCols = 512;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t full_bar[kMaxStages], empty_bar[kMaxStages];
  // [unit & 1]: a unit may be summed; its sums are complete
  __shared__ __align__(8) uint64_t ready[2], acc_full[2];
  // [turn % kTurns]: a turn's scales are in tensor memory; its MMAs are done with them
  __shared__ __align__(8) uint64_t scales_full[kTurns], scales_free[kTurns];
  __shared__ __align__(8) uint64_t done_bar;
  __shared__ float sw_sh[2][2][kMaxGroups];  // [item & 1][half]
  __shared__ int scaled_sh[2];               // [item & 1]
  __shared__ uint32_t tmem_base_sh;
  __shared__ int s_err;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = a.stages;
  const int nk = fa.groups;
  const int items = fa.items;
  // this CTA's part of a pair; the items of a CTA or pair: first, first + step ...
  const int part = TWO ? (int)(blockIdx.x & 1) : 0;
  const int first = (int)blockIdx.x / kCtas, step = (int)gridDim.x / kCtas;
  // the first item's weight scales come from HBM while the block is set up
  {
    const int tile = first / fa.nchunk * (NR / 128) + (tid >> 7), g = 32 * (tid & 127);
    if (tid < kBatchNP && tile * 128 < a.K && g < nk)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(fa.sw + (uint32_t)(tile * nk + g)));
  }

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int p = 0; p < 2; ++p) {
      mbar_init(&ready[p], kPromWarps * kCtas);
      mbar_init(&acc_full[p], 1);
    }
    for (int p = 0; p < kTurns; ++p) {
      mbar_init(&scales_full[p], kPromWarps / 2 * kCtas);  // four warps of each CTA
      mbar_init(&scales_free[p], 1);
    }
    mbar_init(&done_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_err = 0;
    tma_prefetch_map(&map_w);
    tma_prefetch_map(&map_x);
  }
  if (warp == kPromWarps + 1) {
    if constexpr (TWO) {
      pair_tmem_alloc(&tmem_base_sh, kCols);
    } else {
      tmem_alloc(&tmem_base_sh, kCols);
      tmem_relinquish();
    }
  }
  fence_before_sync();
  __syncthreads();
  if constexpr (TWO) cluster_sync_all();  // both CTAs' barriers are ready
  fence_after_sync();
  const uint32_t tmem = tmem_base_sh;

  // item -> block of W8 rows, batch chunk.  The chunks of a block are
  // neighbours, so its weights are read from HBM once.
  if (warp >= kPromWarps) {
    regs_give<56>();
    const bool leader = elect_one();  // one thread issues; the warp stays together
    if (warp == kPromWarps) {
      // TMA producer: the first stages' weights before the wait on the kernel
      // that quantises the hidden states.  A stage is announced by the (first)
      // CTA, for both, and loaded by each.
      auto announce = [&](int s) {
        if (part == 0) mbar_expect_tx(&full_bar[s], (uint32_t)(stage_bytes * kCtas));
      };
      auto load = [&](void* dst, const CUtensorMap* map, int x, int y, int s) {
        if constexpr (TWO)
          pair_load_2d(dst, map, x, y, first_cta(&full_bar[s]));
        else
          tma_load_2d(dst, map, x, y, &full_bar[s]);
      };
      auto load_w = [&](int s, int g, int blk) {
        load(smem + (size_t)s * stage_bytes + kXBytes, &map_w, g * 128, blk * NR + part * WR, s);
      };
      const int pre = min(S, nk);
      if (leader) {
        const int blk = first / fa.nchunk;
        int g = blk % nk;
        for (int kb = 0; kb < pre; ++kb) {
          announce(kb);
          load_w(kb, g, blk);
          g = g + 1 == nk ? 0 : g + 1;
        }
      }
      griddep_wait();
      int it = 0;           // groups requested so far
      int s = 0;            // stage of the next one
      uint32_t sphase = 1;  // parity that says it is free
      bool ok = true;
      for (int item = first; item < items && ok; item += step) {
        const int blk = item / fa.nchunk;
        const int b0 = (item - blk * fa.nchunk) * kCtas * kBM + part * kBM;
        int g = blk % nk;
        for (int kb = 0; kb < nk; ++kb, ++it) {
          if (it >= pre) {
            // a fresh barrier counts as having completed the phase before
            ok = mbar_wait(&empty_bar[s], sphase);
            if (!ok) break;
            if (leader) {
              announce(s);
              load_w(s, g, blk);
            }
          }
          if (leader)
            load(smem + (size_t)s * stage_bytes, &map_x, g * 128, b0, s);
          if (++s == S) {
            s = 0;
            sphase ^= 1;
          }
          g = g + 1 == nk ? 0 : g + 1;
        }
      }
      if (!ok) atomicExch(&s_err, 1);
      // drain: every issued copy has landed before this CTA may exit (a pair's
      // second CTA: the first waits for its copies too, and it for the first)
      if (part == 0)
        for (int k = max(0, it - S); k < it; ++k) mbar_wait(&full_bar[k % S], (k / S) & 1);
    } else if (warp == kPromWarps + 1 && part == 0) {
      // MMA issuer.  The limits of its waits do not count what the kernels ahead take.
      griddep_wait();
      constexpr uint32_t idesc = idesc_e4m3(kCtas * kBM, NR);
      constexpr uint32_t idesc_scaled = idesc_e4m3_scaled(kCtas * kBM, NR);
      auto commit = [&](uint64_t* bar) {
        if constexpr (TWO)
          pair_commit(bar);
        else
          mma_commit(bar);
      };
      const uint64_t desc0 = sw128_desc(smem_u32(smem));
      int u = 0, t = 0, s = 0;  // units and turns so far; the next group's stage
      uint32_t sphase = 0;
      bool ok = true;
      // one group's MMAs, once its operands are there
      auto sum_group = [&](auto mma) {
        fence_after_sync();
        if (leader) {
          const uint64_t xdesc = desc0 + (uint64_t)(s * (stage_bytes >> 4));
          const uint64_t wdesc = xdesc + (kXBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 32 elements = 32 bytes per step
            mma(kk, xdesc + 2 * kk, wdesc + 2 * kk);
          commit(&empty_bar[s]);
        }
        if (++s == S) {
          s = 0;
          sphase ^= 1;
        }
      };
      int at = 0;
      for (int item = first; item < items && ok; item += step, at ^= 1) {
        bool scaled = false;
        if constexpr (TWO) {
          ok = __all_sync(0xffffffffu, mbar_wait(&ready[u & 1], (u >> 1) & 1)) != 0;
          if (!ok) break;
          scaled = scaled_sh[at] != 0;
        }
        // a loop for either kind of scales: with the choice inside, MMAs were issued
        // so much later that units of one group took a quarter longer
        if (!scaled) {
          for (int k = 0; k < nk; ++k, ++u) {
            const int p = u & 1;
            ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[s], sphase) &&
                                             mbar_wait(&ready[p], (u >> 1) & 1)) != 0;
            if (!ok) break;
            const uint32_t acc = tmem + (uint32_t)(p * NR);
            sum_group([&](int kk, uint64_t x, uint64_t w) {
              mma_e4m3<TWO>(acc, x, w, idesc, kk > 0 ? 1u : 0u);
            });
            if (leader) commit(&acc_full[p]);
          }
          continue;
        }
        for (int k = 0; k < nk && ok; ++u) {
          ok = __all_sync(0xffffffffu, mbar_wait(&ready[u & 1], (u >> 1) & 1)) != 0;
          uint32_t add = 0;
          for (const int end = min(nk, k + kUnit); k < end && ok; ++k) {
            const int turn = t % kTurns;
            ok = __all_sync(0xffffffffu, mbar_wait(&scales_full[turn], t / kTurns & 1) &&
                                             mbar_wait(&full_bar[s], sphase)) != 0;
            if (!ok) break;
            const uint32_t scales = tmem + scale_cols(t) + (uint32_t)(k % kTurn * kGroupCols);
            sum_group([&](int, uint64_t x, uint64_t w) {
              mma_e4m3_scaled<TWO>(tmem, x, w, idesc_scaled, scales, scales + 4, add);
              add = 1;
            });
            if (k % kTurn == kTurn - 1 || k + 1 == nk) {
              if (leader) commit(&scales_free[turn]);
              ++t;
            }
          }
          if (ok && leader) commit(&acc_full[u & 1]);
        }
      }
      if (!ok) atomicExch(&s_err, 1);
      if (leader) commit(&done_bar);
    }
  } else {
    regs_take<224>();
    // this thread's batch row (TMEM lane) and its half of the W8 rows
    const int quad = warp & 3, half = warp >> 2, row = quad * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(half * 128);
    float* ob = reinterpret_cast<float*>(smem + (size_t)S * stage_bytes) + warp * 32 * kOutPitch;  // 16-byte aligned
    int u = 0, t = 0;  // units read, and turns whose scales have been written, so far
    bool ok = true;  // once false it stays so: what a late wait would find belongs to another item
    auto chunk_of = [&](int item) { return (item - item / fa.nchunk * fa.nchunk) * kCtas * kBM + part * kBM; };
    // One of this warp's arrivals.  Its loads and stores of tensor memory have
    // completed (tmem_ld32 waits, tmem_st_wait); the fence orders them before it.
    auto give = [&](uint64_t* bar) {
      fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (!TWO || part == 0)
          mbar_arrive(bar);
        else
          remote_arrive(first_cta(bar));
      }
    };
    // an item's weight scales; whether all are powers of two
    auto fetch = [&](int item, int at) {
      const int tile = item / fa.nchunk * (NR / 128) + half;
      bool two = true;
      for (int g = tid & 127; g < nk; g += 128) {
        const float s = tile * 128 < a.K ? fa.sw[(uint32_t)(tile * nk + g)] : 1.f;
        two = two && is_pow2(s);
        sw_sh[at][half][g] = s;
      }
      two = barrier_and(1, kBatchNP, two);
      return TWO && two;
    };
    // The scales of the next turn, of up to n groups from group g on.  Turns
    // alternate between the two halves' warps, each of which writes where its own
    // accumulator is in units of one group.
    auto put_scales = [&](int b0, int at, int g, int n) {
      if ((t & 1) == half) {
        float x[kTurn][4], w[kTurn][2];  // loaded together, groups past n too
#pragma unroll
        for (int i = 0; i < kTurn; ++i) {
          const float* sx = fa.sx + (uint32_t)(g * fa.Bp + b0 + lane);  // B <= 4096, 512 groups
#pragma unroll
          for (int c = 0; c < 4; ++c) x[i][c] = sx[32 * c];
          w[i][0] = sw_sh[at][0][g];
          w[i][1] = sw_sh[at][1][g];
          g = g + 1 == nk ? 0 : g + 1;
        }
        // a fresh barrier counts as having completed the phase before
        ok = __all_sync(0xffffffffu, mbar_wait(&scales_free[t % kTurns], (t / kTurns & 1) ^ 1)) != 0;
        fence_after_sync();
        if (ok) {
#pragma unroll
          for (int i = 0; i < kTurn; ++i) {
            uint32_t xb[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) xb[c] = ue8m0x4(x[i][c]);
            if (i < n)
              tmem_st_scales(tmem + ((uint32_t)(quad * 32) << 16) + scale_cols(t) + (uint32_t)(kGroupCols * i),
                             xb, ue8m0x4(w[i][0]), ue8m0x4(w[i][1]));
          }
          tmem_st_wait();
          give(&scales_full[t % kTurns]);
        }
      }
      ++t;
    };
    int at = 0;
    bool scaled = false;
    if (first < items) {
      scaled = fetch(first, 0);  // like the weights, before the wait
      if (part == 0 && tid == 0) scaled_sh[0] = scaled;
      give(&ready[0]);
      if (!scaled && nk > 1) give(&ready[1]);
    }
    griddep_wait();
    int ahead = 0;  // groups of the item whose scales have been written
    for (int item = first; item < items; item += step) {
      const int blk = item / fa.nchunk, b0 = chunk_of(item);
      const int tile = blk * (NR / 128) + half, j0 = tile * 128;  // 128-row tile of W8
      const int nvalid = min(128, a.K - j0);                      // <= 0: past the end
      const int next = item + step;
      int g = blk % nk;                                           // of group `kb`, or `ahead`
      if (scaled) {
        for (; ahead < min(nk, kTurns * kTurn) && ok; ahead += kTurn) {
          int ga = g + ahead;
          if (ga >= nk) ga -= nk;
          put_scales(b0, at, ga, nk - ahead);
        }
        g += ahead;
        if (g >= nk) g -= nk;
      }
      // the last item's scales have been read by all
      asm volatile("bar.sync 1, %0;" ::"n"(kBatchNP) : "memory");
      const bool next_scaled = next < items && fetch(next, at ^ 1);
      if (item == first + fa.give_up * step) ok = false;
      f32x2 acc[64];  // sums of this batch row and 128 rows of W8
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0;
      if (scaled) {
        for (int kb = 0; kb < nk && ok; kb += kUnit) {
          // with the scales of the next unit's first turns, but for the one that
          // would wait for this unit's last MMAs: its sums come first
          const int upto = min(nk, kb + kUnit + (kTurns - 1) * kTurn);
          for (; ahead < upto && ok; ahead += kTurn) {
            put_scales(b0, at, g, nk - ahead);
            g += kTurn;
            if (g >= nk) g -= nk;
          }
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[u & 1], (u >> 1) & 1)) != 0;
          if (!ok) break;
          fence_after_sync();
          ++u;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float v[32];
            tmem_ld32(lanes + 32 * c, v);
            // all of this warp's columns are in registers: on to the next unit
            if (c == 3 && kb + kUnit < nk) give(&ready[u & 1]);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              add2(acc[16 * c + e], pack2(__float_as_uint(v[2 * e]), __float_as_uint(v[2 * e + 1])));
          }
        }
      } else {
        float sx = fa.sx[(uint32_t)(g * fa.Bp + b0 + row)];
        for (int kb = ok ? 0 : nk; kb < nk; ++kb, ++u) {
          const uint32_t fb = __float_as_uint(sw_sh[at][half][g] * sx);
          const f32x2 f = pack2(fb, fb);
          g = g + 1 == nk ? 0 : g + 1;
          sx = fa.sx[(uint32_t)(g * fa.Bp + b0 + row)];  // the next group's
          ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[u & 1], (u >> 1) & 1)) != 0;
          if (!ok) break;
          fence_after_sync();
          const uint32_t taddr = lanes + (uint32_t)((u & 1) * NR);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float v[32];
            tmem_ld32(taddr + 32 * c, v);
            // all of this warp's columns are in registers: on to the next group but one
            if (c == 3 && kb + 2 < nk) give(&ready[u & 1]);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              fma2(acc[16 * c + e], pack2(__float_as_uint(v[2 * e]), __float_as_uint(v[2 * e + 1])), f);
          }
        }
      }
      // the next item's sums start while this one's rows go out
      ahead = 0;
      if (ok && next < items) {
        if (part == 0 && tid == 0) scaled_sh[at ^ 1] = next_scaled;
        give(&ready[u & 1]);
        if (!next_scaled && nk > 1) give(&ready[(u + 1) & 1]);
        if (next_scaled) {
          const int bn = chunk_of(next);
          int gn = next / fa.nchunk % nk;
          for (; ahead < min(nk, kTurns * kTurn) && ok; ahead += kTurn) {
            put_scales(bn, at ^ 1, gn, nk - ahead);
            gn += kTurn;
            if (gn >= nk) gn -= nk;
          }
        }
      }
      at ^= 1;
      scaled = next_scaled;
      // a warp that gave up misses no barrier; logits, whose call returns no
      // status word, are NaN then, and with one nothing more is stored
      if (nvalid <= 0 || (PART && !ok)) continue;
      const float scale = PART || ok ? a.out_scale : __int_as_float(0x7fc00000);
      const int b = b0 + row;
      // this row's partial over the tile's rows: greedy, its best key (the rows
      // out are q's zeros then); sampling, like tile_partials', (max, sum
      // 2^(z - max)), a NaN or +inf z leaving the sum NaN
      float pm = kNegBig, ps = 0.f;
      uint64_t key = 0;
      const bool zero = PART && a.greedy;
      // 32 batch rows x 32 columns at a time through shared memory, so that a
      // row's 128 bytes leave in one piece: four rows in an instruction where
      // the output's rows are 16-byte aligned, one otherwise
      float* out = a.out + (int64_t)(b0 + quad * 32) * a.ldo + j0;
      const int rows = a.B - (b0 + quad * 32);
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        __syncwarp();
        // the MMAs may be through with the next item's first turns, up to three of
        // them while its first unit's sums are not read
        static_assert(3 * kTurn <= kUnit, "a turn of the next unit would be waited for");
        if (!PART && c > 0 && ok && scaled && ahead > 0 && ahead < nk) {
          const int chunk = chunk_of(next);
          int ga = next / fa.nchunk % nk + ahead;
          if (ga >= nk) ga -= nk;
          put_scales(chunk, at, ga, nk - ahead);
          ahead += kTurn;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 x = unpack2(acc[c / 2 + 2 * i]), y = unpack2(acc[c / 2 + 2 * i + 1]);
          *reinterpret_cast<float4*>(ob + lane * kOutPitch + 4 * i) = make_float4(
              x.x * scale, x.y * scale, y.x * scale, y.y * scale);
        }
        __syncwarp();
        if constexpr (PART) {
          // from this thread's row in shared memory, 32 values at a time
          const float* mine = ob + lane * kOutPitch;
          const int some = min(32, nvalid - c);
          if (a.greedy) {
            for (int i = 0; i < some; ++i) key = max_key(key, greedy_key(mine[i], j0 + c + i));
          } else if (some > 0) {
            float top = pm;
            for (int i = 0; i < some; ++i) top = fmaxf(top, mine[i]);
            ps *= exp2_approx(pm - top);
            pm = top;
            for (int i = 0; i < some; ++i) ps += exp2_approx(mine[i] - pm);
          }
        }
        if (fa.vec_out && c + 32 <= nvalid) {
          const int r0 = lane >> 3, col = 4 * (lane & 7);
          float4 t[8];
#pragma unroll
          for (int r = 0; r < 8; ++r)
            t[r] = zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                        : *reinterpret_cast<const float4*>(ob + (4 * r + r0) * kOutPitch + col);
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (4 * r + r0 < rows)
              *reinterpret_cast<float4*>(out + (int64_t)(4 * r + r0) * a.ldo + c + col) = t[r];
        } else if (c + lane < nvalid) {
          float* o = out + c + lane;
#pragma unroll 8
          for (int r = 0; r < 32; ++r) {
            if (r < rows) *o = zero ? 0.f : ob[r * kOutPitch + lane];
            o += a.ldo;
          }
        }
      }
      if (PART && b < a.B) {
        const int64_t at = (int64_t)tile * a.B + b;
        if (a.greedy)
          reinterpret_cast<uint64_t*>(a.part)[at] = key;
        else
          a.part[at] = make_float2(pm, ps);
      }
    }
    if (!ok && lane == 0) atomicExch(&s_err, 1);
  }
  __syncwarp();
  __syncthreads();  // every role has finished or given up: no wait counts another's work
  // the MMAs have completed
  const bool all_ok = __syncthreads_and(mbar_wait(&done_bar, 0) && s_err == 0 ? 1 : 0) != 0;
  griddep_launch_dependents();
  fence_after_sync();
  if (tid == 0 && !all_ok) atomicOr(a.status, VT_DEV_TIMEOUT);
  if constexpr (TWO) {
    fence_before_sync();
    __syncwarp();
    cluster_sync_all();  // nothing of the pair's is on its way to either CTA
    fence_after_sync();
    if (warp == kPromWarps + 1) pair_tmem_dealloc(tmem, kCols);
  } else {
    if (warp == kPromWarps + 1) tmem_dealloc(tmem, kCols);
  }
}

struct Fp8Ws {
  uint8_t* x8;
  float* sx;
  float2* part;
  int* status_sink;  // status word of calls that report none (vt_draft_logits_fp8)
  size_t bytes;
};

int pad_batch(int B) { return B <= 16 ? 16 : B <= 32 ? 32 : B <= 64 ? 64 : (B + 127) / 128 * 128; }

// Wide batches of an even number of 128-row chunks go to pairs of CTAs, an odd
// number to single ones (K = 38016, H = 4096, B = 300: 59.9 us against 62.5 padded
// to pairs; K = 32768, H = 2048, B = 128: 17.9 against 22.4)
bool paired(int Bp) { return Bp % 256 == 0; }

Fp8Ws carve_fp8(void* base, int B, int H, int K) {
  Fp8Ws w;
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t o = off;
    off = align_up(off + n, 256);
    return o;
  };
  const size_t groups = (H + kQB - 1) / kQB;
  const size_t o_x = take((size_t)B * groups * kQB);
  const size_t o_sx = take(groups * pad_batch(B) * sizeof(float));
  const size_t o_part = take((size_t)((K + umma::kBM - 1) / umma::kBM) * B * sizeof(float2));
  const size_t o_s = take(sizeof(int));
  char* p = static_cast<char*>(base);
  w.x8 = reinterpret_cast<uint8_t*>(p + o_x);
  w.sx = reinterpret_cast<float*>(p + o_sx);
  w.part = reinterpret_cast<float2*>(p + o_part);
  w.status_sink = reinterpret_cast<int*>(p + o_s);
  w.bytes = off;
  return w;
}

// 2-D tensor map of a row-major byte matrix [rows, cols] with a row stride of
// ld bytes, boxes of 128 columns (128-byte swizzle) x box_rows rows
bool make_e4m3_map(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint64_t ld,
                   uint32_t box_rows) {
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, ptr, {cols, rows}, ld,
                           {128, box_rows});
}

// a launch that overlaps the kernel that quantises the hidden states, as a
// grid of clusters of `cluster` CTAs.  smem_max is the most that this kernel is
// ever launched with: the kernel's limit is set to the same value by every
// call, as another host thread may set it between here and the launch.
template <typename K>
int launch_product(cudaStream_t s, K kern, int grid, int threads, size_t smem, size_t smem_max,
                   int cluster, const CUtensorMap& mw, const CUtensorMap& mx, const Fp8Args& fa) {
  VT_RETURN_IF_CUDA(
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_max));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  VT_RETURN_IF_CUDA(cudaLaunchKernelEx(&cfg, kern, mw, mx, fa));
  return VT_OK;
}

template <int BN>
int launch_narrow(cudaStream_t s, const CUtensorMap& mw, const CUtensorMap& mx, Fp8Args fa) {
  constexpr int stage = umma::kABytes + BN * 128;
  constexpr size_t kZt =
      (size_t)kPartCols<BN> * umma::zt_pitch<kPartCols<BN>, kNarrowNP>() * sizeof(float);
  const size_t zt = fa.h.part == nullptr ? 0
                    : fa.h.greedy        ? (size_t)kNarrowNP / 32 * BN * sizeof(uint64_t)
                                         : kZt;
  fa.items = (fa.h.K + umma::kBM - 1) / umma::kBM;
  // Two CTAs per SM.  Where no SM gets a second tile, a tile of 64 columns has a
  // longer ring (B = 50, K = 10007, H = 1500, greedy: 11.6 against 12.9 us; B = 64,
  // K = 19000, H = 4096: 19.0 against 20.0); with fewer columns that was slower by
  // up to 4%, the next call's product then starting later.
  constexpr int kRing = 96 * 1024, kLongRing = 150 * 1024;
  const int sms = num_sms();
  const int ring = fa.items > sms || BN < 64 ? kRing : kLongRing;
  fa.h.stages = std::max(2, std::min(umma::kMaxStages, (int)((ring - zt) / stage)));
  return launch_product(s, head_fp8_kernel<BN>, std::min(fa.items, 2 * sms), kNarrowNT,
                        (size_t)fa.h.stages * stage + zt + 1024,
                        (BN < 64 ? kRing : kLongRing) + 1024, 1, mw, mx, fa);
}

template <bool TWO>
int launch_wide(cudaStream_t s, const CUtensorMap& mw, const CUtensorMap& mx, Fp8Args fa) {
  constexpr int stage = umma::kBM * 128 + (TWO ? 128 : 256) * 128, ctas = TWO ? 2 : 1;
  constexpr int stages = 160 * 1024 / stage;  // five of a pair, three of a single CTA
  constexpr size_t out = (size_t)(kBatchNP / 32) * 32 * kOutPitch * sizeof(float);
  constexpr size_t smem = stages * stage + out + 1024;
  fa.h.stages = stages;
  fa.nchunk = fa.Bp / (128 * ctas);
  fa.items = (fa.h.K + kBatchRowsW - 1) / kBatchRowsW * fa.nchunk;
  return launch_product(s, fa.h.part != nullptr ? batch_fp8_kernel<TWO, true> : batch_fp8_kernel<TWO, false>,
                        ctas * std::min(fa.items, num_sms() / ctas), kBatchNT, smem, smem, ctas, mw,
                        mx, fa);
}

// z = out_scale * hidden @ (scaled W8)^T; part[tile][b] partials of 128-row
// tiles; greedy, out is q without its ones and part holds each tile's best keys
int launch_head_fp8(cudaStream_t s, const uint16_t* hidden, int B, int H, const uint8_t* W8,
                    int64_t ldw, const float* w_scale, int K, float out_scale, float* out,
                    int64_t ldo, const Fp8Ws& ws, float2* part, int* status, int status_reset,
                    int greedy, int give_up = -1) {
  const int groups = (H + kQB - 1) / kQB, Bp = pad_batch(B), ldx = groups * kQB;
  CUtensorMap mw, mx;
  // the boxes: the rows that one CTA stages
  if (!make_e4m3_map(&mw, W8, (uint64_t)K, (uint64_t)H, (uint64_t)ldw,
                     Bp > 64 && !paired(Bp) ? 256 : 128))
    return VT_ERR_CUDA;
  if (!make_e4m3_map(&mx, ws.x8, (uint64_t)B, (uint64_t)ldx, (uint64_t)ldx,
                     (uint32_t)std::min(Bp, 128)))
    return VT_ERR_CUDA;
  {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((int64_t)Bp * groups + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int vec_ok = H % 4 == 0 && (reinterpret_cast<uintptr_t>(hidden) & 7) == 0;
    VT_RETURN_IF_CUDA(cudaLaunchKernelEx(&cfg, quantize_hidden_kernel, hidden, B, H, ws.x8, ldx,
                                         ws.sx, Bp, groups, vec_ok, status, status_reset));
  }
  Fp8Args fa;
  fa.h = umma::HeadArgs{};
  fa.h.B = B;
  fa.h.H = H;
  fa.h.K = K;
  fa.h.out_scale = out_scale;
  fa.h.out = out;
  fa.h.ldo = ldo;
  fa.h.part = part;
  fa.h.status = status;
  fa.h.greedy = greedy;
  fa.sw = w_scale;
  fa.sx = ws.sx;
  fa.Bp = Bp;
  fa.groups = groups;
  fa.nchunk = 1;
  fa.give_up = give_up;
  fa.vec_out = (reinterpret_cast<uintptr_t>(out) & 15) == 0 && ldo % 4 == 0;
  switch (Bp) {
    case 16: return launch_narrow<16>(s, mw, mx, fa);
    case 32: return launch_narrow<32>(s, mw, mx, fa);
    case 64: return launch_narrow<64>(s, mw, mx, fa);
    default: return paired(Bp) ? launch_wide<true>(s, mw, mx, fa) : launch_wide<false>(s, mw, mx, fa);
  }
}

// The greedy step's token of a batch row (grid B): the best key of all tiles.
// The product has left q's zeros, so that only the one is written here; a row
// with a non-finite z stays all zero and gets the token -1.  Bound by its latency:
// the step takes 2.4 us more than the logits at B = 16, K = 32768, H = 2048 (3.8
// when all of q was written behind the product, and 7.5 at B = 64).
constexpr int kTokenNT = 256;
__global__ void __launch_bounds__(kTokenNT)
greedy_token_kernel(const uint64_t* __restrict__ part, int B, int G, int K,
                    const int* __restrict__ trim_ids, float* __restrict__ q, int64_t ldq,
                    int* __restrict__ tokens, int64_t ldt, int* __restrict__ status) {
  __shared__ uint64_t of_warp[kTokenNT / 32];
  const int b = blockIdx.x, tid = threadIdx.x;
  griddep_launch_dependents();  // the next kernel waits for this grid before reading
  griddep_wait();
  uint64_t key = 0;
  for (int t = tid; t < G; t += kTokenNT) key = max_key(key, part[(int64_t)t * B + b]);
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32));
  const uint32_t lo =
      __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32) == hi ? (uint32_t)key : 0u);
  if ((tid & 31) == 0) of_warp[tid >> 5] = (uint64_t)hi << 32 | lo;
  __syncthreads();
  if (tid != 0) return;
  key = of_warp[0];
#pragma unroll
  for (int w = 1; w < kTokenNT / 32; ++w) key = max_key(key, of_warp[w]);
  const int j = (int)~(uint32_t)key;
  const bool ok = (uint32_t)(key >> 32) != kKeyNonFinite && j >= 0 && j < K;
  if (ok) q[(int64_t)b * ldq + j] = 1.f;
  tokens[(int64_t)b * ldt] = ok ? trim_ids[j] : -1;
  if (!ok) atomicOr(status, VT_DEV_NONFINITE);
}

// T > 0, or T == 0 where greedy drafting is allowed
int check_fp8_args(const uint16_t* hidden, int B, int H, const uint8_t* W8, int64_t ldw,
                   const float* w_scale, int K, float T, bool allow_greedy) {
  if (!hidden || !W8 || !w_scale) return VT_ERR_INVALID_ARG;
  if (B < 1 || B > 4096 || H < 1 || H > 65536 || K < 1) return VT_ERR_INVALID_ARG;
  if (K > kMaxRows) return VT_ERR_UNSUPPORTED;
  if (ldw < H || ldw % 16 != 0 || (reinterpret_cast<uintptr_t>(W8) & 15) != 0)
    return VT_ERR_INVALID_ARG;
  if (!std::isfinite(T) || T < 0.f || (T == 0.f && !allow_greedy)) return VT_ERR_INVALID_ARG;
  return VT_OK;
}

}  // namespace
}  // namespace vt

extern "C" int vt_quantize_head(const uint16_t* W, int32_t K, int32_t H, uint8_t* W8, int64_t ldw,
                                float* w_scale, int32_t* dev_status, void* stream) {
  using namespace vt;
  if (!W || !W8 || !w_scale || !dev_status || K < 1 || H < 1 || H > 65536)
    return VT_ERR_INVALID_ARG;
  if (ldw < H || ldw % 16 != 0 || (reinterpret_cast<uintptr_t>(W8) & 15) != 0)
    return VT_ERR_INVALID_ARG;
  if (K > kMaxRows) return VT_ERR_UNSUPPORTED;
  const int rows = (K + kQB - 1) / kQB;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int st = clear_status(s, dev_status);
  if (st != VT_OK) return st;
  const uintptr_t wa = reinterpret_cast<uintptr_t>(W);
  const int by = H % 8 == 0 && (wa & 15) == 0 ? 16 : (wa & 3) == 0 ? 4 : 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((H + kQB - 1) / kQB), (unsigned)rows);
  cfg.blockDim = dim3(kQuantNT);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  VT_RETURN_IF_CUDA(cudaLaunchKernelEx(&cfg, quantize_head_kernel, W, K, H, W8, ldw, w_scale,
                                       dev_status, by));
  return VT_OK;
}

extern "C" size_t vt_draft_fp8_workspace_bytes(int32_t B, int32_t H, int32_t K) {
  if (B < 1 || B > 4096 || H < 1 || H > 65536 || K < 1 || K > vt::kMaxRows) return 0;
  return vt::carve_fp8(nullptr, B, H, K).bytes;
}

extern "C" int vt_draft_logits_fp8(const uint16_t* hidden, int32_t B, int32_t H, const uint8_t* W8,
                                   int64_t ldw, const float* w_scale, int32_t K, float temperature,
                                   float* logits, int64_t ld_logits, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  using namespace vt;
  const int st = check_fp8_args(hidden, B, H, W8, ldw, w_scale, K, temperature, false);
  if (st != VT_OK) return st;
  if (!logits || ld_logits < K) return VT_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)) return VT_ERR_WORKSPACE;
  const Fp8Ws ws = carve_fp8(workspace, B, H, K);
  if (workspace_bytes < ws.bytes) return VT_ERR_WORKSPACE;
  return launch_head_fp8(static_cast<cudaStream_t>(stream), hidden, B, H, W8, ldw, w_scale, K,
                         1.0f / temperature, logits, ld_logits, ws, nullptr, ws.status_sink, 1, 0);
}

extern "C" int vt_selftest_draft_fp8(int32_t give_up, const uint16_t* hidden, int32_t B, int32_t H,
                                     const uint8_t* W8, int64_t ldw, const float* w_scale,
                                     int32_t K, float temperature, float* logits,
                                     int64_t ld_logits, int32_t* dev_status, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  using namespace vt;
  const int st = check_fp8_args(hidden, B, H, W8, ldw, w_scale, K, temperature, false);
  if (st != VT_OK) return st;
  if (give_up < -1 || give_up > 65535 || !logits || ld_logits < K || !dev_status)
    return VT_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)) return VT_ERR_WORKSPACE;
  const Fp8Ws ws = carve_fp8(workspace, B, H, K);
  if (workspace_bytes < ws.bytes) return VT_ERR_WORKSPACE;
  return launch_head_fp8(static_cast<cudaStream_t>(stream), hidden, B, H, W8, ldw, w_scale, K,
                         1.0f / temperature, logits, ld_logits, ws, nullptr, dev_status, 1, 0,
                         give_up);
}

extern "C" int vt_draft_step_fp8(const uint16_t* hidden, int32_t B, int32_t H, const uint8_t* W8,
                                 int64_t ldw, const float* w_scale, const int32_t* trim_ids,
                                 int32_t K, const float* uniforms, float temperature, float* q,
                                 int64_t ldq, int32_t* tokens, int64_t ld_tokens,
                                 int32_t* dev_status, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  return vt::draft_step_fp8_impl(hidden, B, H, W8, ldw, w_scale, trim_ids, K, uniforms, temperature,
                                 q, ldq, tokens, ld_tokens, dev_status, workspace, workspace_bytes,
                                 stream, 1);
}

int vt::draft_step_fp8_impl(const uint16_t* hidden, int32_t B, int32_t H, const uint8_t* W8,
                            int64_t ldw, const float* w_scale, const int32_t* trim_ids, int32_t K,
                            const float* uniforms, float temperature, float* q, int64_t ldq,
                            int32_t* tokens, int64_t ld_tokens, int32_t* dev_status,
                            void* workspace, size_t workspace_bytes, void* stream,
                            int status_reset) {
  const int st = check_fp8_args(hidden, B, H, W8, ldw, w_scale, K, temperature, true);
  if (st != VT_OK) return st;
  const bool greedy = temperature == 0.f;
  if (!trim_ids || (!uniforms && !greedy) || !q || ldq < K || !tokens || ld_tokens < 1 ||
      !dev_status)
    return VT_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)) return VT_ERR_WORKSPACE;
  const Fp8Ws ws = carve_fp8(workspace, B, H, K);
  if (workspace_bytes < ws.bytes) return VT_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int rc = launch_head_fp8(s, hidden, B, H, W8, ldw, w_scale, K,
                                 greedy ? 1.0f : VT_LOG2E / temperature, q, ldq, ws, ws.part,
                                 dev_status, status_reset, greedy ? 1 : 0);
  if (rc != VT_OK) return rc;
  if (greedy) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)B);
    cfg.blockDim = dim3(kTokenNT);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    VT_RETURN_IF_CUDA(cudaLaunchKernelEx(&cfg, greedy_token_kernel,
                                         reinterpret_cast<const uint64_t*>(ws.part), B,
                                         (K + umma::kBM - 1) / umma::kBM, K, trim_ids, q, ldq,
                                         tokens, ld_tokens, dev_status));
    return VT_OK;
  }
  return draft_finish(s, B, K, false, ws.part, (K + umma::kBM - 1) / umma::kBM, umma::kBM,
                      uniforms, trim_ids, q, ldq, tokens, ld_tokens, dev_status);
}

extern "C" size_t vt_draft_topk_fp8_workspace_bytes(int32_t B, int32_t H, int32_t K, int32_t k) {
  if (B < 1 || B > 4096 || H < 1 || H > 65536 || K < 1 || K > vt::kMaxRows || k < 1 ||
      k > vt::kDraftTopkMax || k > K)
    return 0;
  return vt::align_up(vt_draft_fp8_workspace_bytes(B, H, K), 256) +
         vt::align_up((size_t)B * K * 4, 256);
}

extern "C" int vt_draft_topk_fp8(const uint16_t* hidden, int32_t B, int32_t H, const uint8_t* W8,
                                 int64_t ldw, const float* w_scale, const int32_t* trim_ids,
                                 int32_t K, int32_t k, float temperature, int32_t* out_ids,
                                 float* out_logq, int32_t* dev_status, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  using namespace vt;
  const int st = check_fp8_args(hidden, B, H, W8, ldw, w_scale, K, temperature, false);
  if (st != VT_OK) return st;
  if (!trim_ids || !out_ids || !out_logq || !dev_status || k < 1 || k > kDraftTopkMax || k > K)
    return VT_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)) return VT_ERR_WORKSPACE;
  if (workspace_bytes < vt_draft_topk_fp8_workspace_bytes(B, H, K, k)) return VT_ERR_WORKSPACE;
  char* base = static_cast<char*>(workspace);
  const Fp8Ws ws = carve_fp8(base, B, H, K);
  float* z2 = reinterpret_cast<float*>(base + align_up(ws.bytes, 256));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int rc = launch_head_fp8(s, hidden, B, H, W8, ldw, w_scale, K, VT_LOG2E / temperature, z2,
                                 K, ws, ws.part, dev_status, 1, 0);
  if (rc != VT_OK) return rc;
  return draft_topk_finish(s, z2, B, K, k, ws.part, (K + umma::kBM - 1) / umma::kBM, trim_ids,
                           out_ids, out_logq, dev_status);
}
