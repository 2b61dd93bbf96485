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
// sums those beams' rows again, exponentials as pairs of fp32 values added as integers
// (equal beams give equal scores, whatever their rows' alignment or the order of their logits),
// and takes the lists again.  That is one block, row after row: for a row of 38016 fp32 logits some 50 us, and
// the whole call waits.  256 x 8 beams over 38016 take 159 us with one near pair among them, 692 where all beams
// of each sequence are equal (55 without); 16 x 8 over 32768 82 and 288 (11); 16 x 32 over 38016 with 32
// continuations 144 and 1490 (55); 16 x 8 over 152064 bf16 315 and 1280 (18).
//
// The rows are streamed as the log probabilities' are: a cluster of up to 8 blocks to a row where rows
// are few, one persistent block for row after row where they are many.  256 x 8 beams over 38016 fp32
// logits, 8 best: 55.2 us in a graph of calls (5.6 TB/s; 45.9 at the measured copy rate): 53.8 of rows alone
// (DRAM at 74%, issue slots at 58%; 4.5 rows a block are five rounds) and what the merge's start under
// them does not hide of its 7.  16 x 8 beams over 32768: 11.2, one row of 32768: 7.9, latencies:
// 5 to 8 of rows, 3 of the merge, whose lists start with logarithms by pairs of fp32 values (in fp64 it
// took 6).  The merge inside the rows' kernel, a sequence's beams one cluster, was built and is slower
// (13.0 and 8.5 us), as a beam then has one block instead of two to eight.
#include <algorithm>
#include <cmath>

#include <cooperative_groups.h>

#include "vt_internal.h"
#include "vt_rows.cuh"
#include "vt_umma.cuh"

namespace cg = cooperative_groups;

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

typedef unsigned long long bs_key;  // an fp64 score, or a row's (value, id)

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
  double t, inv_t;         // T and 1 / T
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

struct BsShared {
  RowLists top;
  alignas(8) uint64_t full[kLpStages], empty[kLpStages];
  RowSum red[kLpWarps];
  RowSum blk;      // this block's, as published
  float edge[16];  // the row's edges
  int timeout;
};

// Each cluster takes rows of logits as the log probabilities' kernel does (one warp
// copies, eight consume), and leaves m, S and the N best.
template <typename T>
__global__ void __launch_bounds__(kLpNT + 32, kLpPerSm) beam_rows_kernel(BsArgs a) {
  constexpr int VE = Elem<T>::kVec;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ BsShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int N = a.N, R = a.B * a.W;
  const int row0 = blockIdx.x / C, stride = gridDim.x / C;
  griddep_launch_dependents();  // the merge waits for this grid before it reads
  if (tid == 0) {
    for (int s = 0; s < kLpStages; ++s) {
      umma::mbar_init(&sh.full[s], 1);
      umma::mbar_init(&sh.empty[s], kLpWarps);
    }
    sh.timeout = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (blockIdx.x == 0) *a.dev_status = 0;  // the merge adds the rows' flags
  }
  __syncthreads();

  if (warp == kLpWarps) {
    // the copying warp runs ahead of the consumers, into their next rows
    if (lane == 0) {
      bool ok = true;
      int it = 0;  // chunks requested so far
      for (int row = row0; row < R && ok; row += stride) {
        if (!bs_live(a, row)) continue;
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
      if (!ok) {
        atomicExch(&sh.timeout, 1);
        // every copy issued has landed before this block may exit
        for (int s = 0; s < kLpStages; ++s)
          for (int par = 0; par < 2; ++par) umma::mbar_wait(&sh.full[s], par, 1u << 12);
      }
    }
    __syncwarp();
    if (C > 1 && bs_live(a, row0)) {
      cl.sync();
      cl.sync();
    }
    return;
  }

  int it = 0;  // chunks consumed so far
  uint32_t limit = umma::kWaitLimit;
  for (int row = row0; row < R; row += stride) {
    if (!bs_live(a, row)) {
      if (rank == 0 && tid == 0) {
        const float s = a.scores[row];
        a.rows[row] = BeamRow{0.f, 1.f, 0.f, 0, s == -INFINITY || fabsf(s) < INFINITY ? 0 : VT_DEV_NONFINITE};
      }
      continue;
    }
    const T* l = static_cast<const T*>(a.logits) + (int64_t)row * a.ld;
    const Span sp = span_of<T>(l, a.K, rank, C);
    // the row's edges, one element per thread of block 0, kept in shared memory until the end
    const bool edge = rank == 0 && tid < 2 * VE;
    if (edge) {
      const int id = edge_id<VE>(sp, tid);
      sh.edge[tid] = id < a.K ? Elem<T>::load(l + id) : -INFINITY;
    }
    RowSum st{kNegBig, 0.f, 0.f};
    // an id at -infinity is no candidate: the bound starts above it
    TopList top{sh.top.list[warp], 0, (lp_key)(lp_ord(-INFINITY) + 1) << 32, kNegBig};

    for (int i = 0; i < sp.mine; ++i, ++it) {
      const int s = it % kLpStages;
      if (!__all_sync(0xffffffffu, umma::mbar_wait(&sh.full[s], (it / kLpStages) & 1, limit))) {
        // gave up: go on without the data, so that no barrier is missed
        limit = 1;
        if (lane == 0) atomicExch(&sh.timeout, 1);
      }
      const int q0 = (rank + i * C) * (kLpNT * kLpU) + tid;  // first vector of this thread
      const uint4* st4 = reinterpret_cast<const uint4*>(ring + s * kLpChunk) + tid;
      const int have = min(kLpU, max(0, (sp.nvec - q0 + kLpNT - 1) / kLpNT));  // vectors in the row
      float pm;
      {
        uint4 v[kLpU];
#pragma unroll
        for (int u = 0; u < kLpU; ++u)
          v[u] = u < have ? st4[u * kLpNT]
                          : make_uint4(Vec<T>::kMasked, Vec<T>::kMasked, Vec<T>::kMasked, Vec<T>::kMasked);
        pm = Vec<T>::top(v);
        if (!(pm <= st.m)) sum_rescale(st, max_nan(st.m, pm), a.c);
        sum_add<T, kLpU>(st, v, a.c);
      }
      top.renew(st.s > 0.f ? st.m : -INFINITY, i, sp.mine, sh.top.group, N, tid);
      top.scan<T>(pm, st4, q0, sp, N, lane);
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(&sh.empty[s]);
    }

    if (rank == 0) {
      const float xe = edge ? sh.edge[tid] : -INFINITY;
      if (!(xe <= st.m)) sum_rescale(st, max_nan(st.m, xe), a.c);
      float er;
      two_sum(st.s, exp2_approx((xe - st.m) * a.c), st.s, er);
      st.e += er;
      top.add(xe, edge_id<VE>(sp, tid), edge, N, lane);
    }
    st = sum_lanes(st, 32, a.c);
    if (lane == 0) sh.red[warp] = st;
    lists_join(sh.top, top.n, top.bound, N, warp, lane);
    lp_bar();
    RowSum r = sum_lanes(sh.red[lane % kLpWarps], kLpWarps, a.c);
    lp_key q = 0;  // this thread's candidate for the N best
    int rk = lane, n = 0;
    bool late;
    if (C == 1) {
      if (warp == 0 && lane < N) q = sh.top.best[lane];
      n = __popc(__ballot_sync(0xffffffffu, q != 0));
      late = sh.timeout != 0;
    } else {
      if (tid == 0) sh.blk = r;
      cl.sync();
      if (rank != 0) {
        // the first block reads this one's memory before it arrives in turn
        cl.sync();
        return;
      }
      // all blocks' sums, one per lane, and keys; warp w holds block w's
      const int from = lane < C ? lane : 0;
      r = *cl.map_shared_rank(&sh.blk, from);
      if (lane >= C) r.s = r.e = 0.f;
      const bool gave_up = *cl.map_shared_rank(&sh.timeout, from) != 0;
      if (warp < C) {
        if (lane < N) {
          q = cl.map_shared_rank(sh.top.best, warp)[lane];
          sh.top.all[warp * N + lane] = q;
        }
        if (warp == 0 && lane < 8) sh.top.all[C * N + lane] = 0;
      }
      const unsigned has = __ballot_sync(0xffffffffu, q != 0);
      if (lane == 0) sh.top.n[warp] = __popc(has);
      late = __any_sync(0xffffffffu, gave_up);
      r = sum_lanes(r, kLpMaxC, a.c);
      lp_bar();  // every read of the other blocks' memory has returned
      asm volatile("barrier.cluster.arrive.release;" ::: "memory");  // they may exit
      if (q != 0) rk = count_before(sh.top.all, C * N, q);
      for (int w = 0; w < kLpWarps; ++w) n += sh.top.n[w];
      n = min(n, N);
    }
    const bool ok = !late && r.m < INFINITY;  // no NaN, no +infinity
    if (tid == 0)
      a.rows[row] = BeamRow{r.m, r.s, r.e, ok && r.s > 0.f ? n : 0, late ? VT_DEV_TIMEOUT : ok ? 0 : VT_DEV_NONFINITE};
    if (q != 0 && rk < N) a.best[(int64_t)row * N + rk] = q;
    if (C > 1)
      asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    else
      lp_bar();  // the next row writes what this one has read
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

// S of one row again, by all threads of the block.  The exponentials are pairs, good to 2^-28,
// and are added as integers in units of 2^-54: a weight's multiples of 2^-30 and what it has beyond
// them apart, each below 2^30 in size, so that 2^22 of them fit 64 bits.  So S is the same in whatever order
// it is added: rows of the same logits in other places, or behind a constant, have equal sums.
template <typename T>
__device__ __noinline__ double bs_exact_sum(const BsArgs& a, int row, float m, Pair inv_t, long long (*red)[2]) {
  constexpr int U = 4;  // ids of a thread in flight
  const T* l = static_cast<const T*>(a.logits) + (int64_t)row * a.ld;
  long long hi = 0, lo = 0;
  for (int j = threadIdx.x; j < a.K; j += U * kBsNT) {
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = j + u * kBsNT < a.K ? Elem<T>::load(l + j + u * kBsNT) : -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Pair d;
      two_sum(x[u], -m, d.h, d.l);
      if (!(d.h * inv_t.h > -80.f)) continue;  // e^-80 of 2^22 ids is nothing to S >= 1
      const Pair w = pair_exp(pair_mul(d, inv_t));
      const float y = w.h * 0x1p30f;
      const int whole = __float2int_rz(y);
      hi += whole;
      lo += __float2int_rn(((y - (float)whole) + w.l * 0x1p30f) * 0x1p24f);  // (off by two units at most)
    }
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int o = 16; o > 0; o >>= 1) {
    hi += __shfl_xor_sync(0xffffffffu, hi, o);
    lo += __shfl_xor_sync(0xffffffffu, lo, o);
  }
  __syncthreads();
  if (lane == 0) {
    red[warp][0] = hi;
    red[warp][1] = lo;
  }
  __syncthreads();
  hi = lo = 0;
  for (int w = 0; w < kBsNT / 32; ++w) {
    hi += red[w][0];
    lo += red[w][1];
  }
  return (double)hi * 0x1p-30 + (double)lo * 0x1p-54;
}

// What the merge's threads share
struct BsMerge {
  bs_key key[kBsMaxBeams][kBsMaxN + 1];
  double off[kBsMaxBeams];       // score minus ln S of each beam
  float top[kBsMaxBeams];
  int count[kBsMaxBeams];
  long long red[kBsNT / 32][2];
  unsigned again;                // beams whose S is summed again
};

// Sums the rows of the beams in `todo` again and scores their candidates from these sums.  (Apart from the kernel,
// which seldom comes here and is slower with this code among its own.)
template <typename T>
__device__ __noinline__ void bs_again(const BsArgs& a, int row0, unsigned todo, BsMerge& sh) {
  Pair inv_t;
  inv_t.h = (float)a.inv_t;
  inv_t.l = (float)(a.inv_t - (double)inv_t.h);
  for (; todo; todo &= todo - 1) {
    const int w = __ffs(todo) - 1;
    const double lnS = log(bs_exact_sum<T>(a, row0 + w, sh.top[w], inv_t, sh.red));
    const double score = (double)a.scores[row0 + w];
    for (int j = threadIdx.x; j < sh.count[w]; j += kBsNT) {
      const double d = (double)key_value(a.best[(int64_t)(row0 + w) * a.N + j]) - (double)sh.top[w];
      // d / T, after a Newton step, so that a quotient that fp64 has is that one, and ln S last, so
      // that totals of score and logit that are equal stay so
      double x = d * a.inv_t;
      x = fma(fma(-x, a.t, d), a.inv_t, x);
      sh.key[w][j] = bs_order((x + score) - lnS);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kBsNT) beam_merge_kernel(BsArgs a) {
  __shared__ BsMerge sh;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int W = a.W, N = a.N, row0 = b * W;
  const int w0 = tid / N, j0 = tid - w0 * N;
  const bool ended = tid < W && a.done && a.done[row0 + tid];
  const unsigned over = __ballot_sync(0xffffffffu, ended);  // (of the first warp's use)
  const float score = tid < W ? a.scores[row0 + tid] : 0.f;
  griddep_wait();
  // this thread's first candidate, asked for together with the rows
  bs_key first = 0;
  if (w0 < W) first = a.best[(int64_t)(row0 + w0) * N + j0];
  if (tid < W) {
    const BeamRow r = a.rows[row0 + tid];
    if (r.flags) atomicOr(a.dev_status, r.flags);
    sh.count[tid] = r.n;
    sh.top[tid] = r.m;
    const Pair lnS = pair_log(pair_of(r.s, r.e));
    sh.off[tid] = ((double)score - (double)lnS.h) - (double)lnS.l;
    if (ended && fabsf(score) < INFINITY) {
      // a beam that has ended continues once, as it is
      sh.count[tid] = 1;
      sh.key[tid][0] = bs_order((double)score);
    }
  }
  __syncthreads();
  for (int i = tid, w = w0, j = j0; i < W * N; i += kBsNT, w = i / N, j = i - w * N)
    if (j < sh.count[w] && !(a.done && a.done[row0 + w])) {
      const float v = key_value(i == tid ? first : a.best[(int64_t)(row0 + w) * N + j]);
      sh.key[w][j] = bs_order(((double)v - (double)sh.top[w]) * a.inv_t + sh.off[w]);
    }
  unsigned exact = 0;  // beams whose S is the precise one
  for (;;) {
    __syncthreads();
    if (warp == 0) {
      // lane w holds beam w's place in its list, lane n the n-th chosen
      const int mine = lane < W ? sh.count[lane] : 0;
      int at = 0, from = -1, place = 0;
      bs_key q = mine > 0 ? sh.key[lane][0] : 0, won = 0;
      for (int n = 0; n < N; ++n) {
        const unsigned hi = __reduce_max_sync(0xffffffffu, (unsigned)(q >> 32));
        if (hi == 0) break;  // (no finite score has a zero there)
        const bool h = (unsigned)(q >> 32) == hi;
        unsigned who = __ballot_sync(0xffffffffu, h);
        if (who & (who - 1)) {
          const unsigned lo = __reduce_max_sync(0xffffffffu, h ? (unsigned)q : 0u);
          who = __ballot_sync(0xffffffffu, h && (unsigned)q == lo);
        }
        const int w = __ffs(who) - 1;  // ties to the lower beam
        const bs_key best = __shfl_sync(0xffffffffu, q, w);
        const int best_at = __shfl_sync(0xffffffffu, at, w);
        if (lane == n) won = best, from = w, place = best_at;
        if (lane == w) q = ++at < mine ? sh.key[lane][at] : 0;
      }
      // Beams that are too near to be told apart: neighbours among the chosen, and the last chosen
      // with every other beam that has a candidate left (its best is q).  A beam that should
      // change places with another is within kNear of it, so of all chosen between them.
      const bs_key below = __shfl_down_sync(0xffffffffu, won, 1);
      const int next = __shfl_down_sync(0xffffffffu, from, 1);
      const bs_key end = __shfl_sync(0xffffffffu, won, N - 1);
      const int end_from = __shfl_sync(0xffffffffu, from, N - 1);
      unsigned near = 0;
      if (lane < N - 1 && below != 0 && next != from && bs_score(won) - bs_score(below) < kNear)
        near = 1u << from | 1u << next;
      if (end != 0 && q != 0 && lane != end_from && bs_score(end) - bs_score(q) < kNear)
        near |= 1u << lane | 1u << end_from;
      near = __reduce_or_sync(0xffffffffu, near) & ~over;  // beams that have ended have their scores exactly
      if (lane == 0) sh.again = near;
      if ((near & ~exact) == 0 && lane < N) {
        const int64_t o = (int64_t)b * N + lane;
        int token = -1;
        bool done = false;
        if (won != 0) {
          done = over >> from & 1;
          token = a.end_id;
          if (!done) {
            token = key_id(a.best[(int64_t)(row0 + from) * N + place]);
            if (a.trim_ids) token = a.trim_ids[token];
            done = token == a.end_id;
          }
        }
        a.out_scores[o] = won != 0 ? (float)bs_score(won) : -INFINITY;
        a.out_parent[o] = won != 0 ? from : -1;
        a.out_tokens[o] = token;
        if (a.out_done) a.out_done[o] = done;
      }
    }
    __syncthreads();
    const unsigned todo = sh.again & ~exact;
    if (todo == 0) break;
    exact |= todo;
    bs_again<T>(a, row0, todo, sh);
  }
}

// ---------------------------------------------------------------- reordering
// A thread has one vector of all W beams of a sequence: it reads those that continue, by asynchronous
// copies to shared memory so that all are on their way together, and then writes; so the move may
// be in place, whatever the parents.  Bound by HBM: a cache of 268 MB of which 5 of 8 beams continue, half
// full, takes 37.5 us (6.2 TB/s; plain loads one after another 39.4), in place, where 14% of the slots keep
// their beam, 35.2.  Positions are moved one by one, a vector being no longer than a position: contiguous
// histories of 4-byte ids move 4 bytes a thread and beam.
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

// a vector to shared memory; asynchronous where there is such a copy of its size
template <typename V>
__device__ __forceinline__ void fetch(V* to, const uint8_t* from) {
  if constexpr (sizeof(V) == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(umma::smem_u32(to)), "l"(from) : "memory");
  else if constexpr (sizeof(V) >= 4)
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(umma::smem_u32(to)), "l"(from), "n"(sizeof(V))
                 : "memory");
  else
    *to = *reinterpret_cast<const V*>(from);
}

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
    if (used >> w & 1) fetch(col + w * kBrNT, src + w * a.from.w);
  asm volatile("cp.async.wait_all;" ::: "memory");
  for (int n = 0; n < a.N; ++n)
    if (par[n] >= 0) *reinterpret_cast<V*>(dst + n * a.to.w) = col[par[n] * kBrNT];
}

template <typename V>
int launch_reorder(cudaStream_t s, const BrArgs& a) {
  const int64_t per = a.S * (a.row / (int64_t)sizeof(V));
  const int64_t pieces = (per + kBrNT - 1) / kBrNT, blocks = a.O * a.B * a.P * pieces;
  if (blocks > 0x7fffffff) return VT_ERR_UNSUPPORTED;
  const int smem = a.W * kBrNT * (int)sizeof(V);
  // what a launch may take without asking is 48 KB together with the kernel's own few hundred bytes
  if (smem > 47 << 10)
    VT_RETURN_IF_CUDA(cudaFuncSetAttribute(beam_reorder_kernel<V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           kBsMaxBeams * kBrNT * (int)sizeof(V)));
  beam_reorder_kernel<V><<<(unsigned)blocks, kBrNT, smem, s>>>(a, pieces);
  VT_RETURN_IF_LAUNCH_FAILED();
  return VT_OK;
}

template <typename T>
int launch_select(cudaStream_t s, const BsArgs& a) {
  auto rows = beam_rows_kernel<T>;
  VT_RETURN_IF_CUDA(cudaFuncSetAttribute(rows, cudaFuncAttributeMaxDynamicSharedMemorySize, kLpSmem));
  const int64_t R = (int64_t)a.B * a.W;
  const int C = lp_cluster(R, a.K, (int)sizeof(T));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(C > 1 ? R * C : std::min<int64_t>(R, num_sms() * kLpPerSm)));
  cfg.blockDim = dim3(kLpNT + 32);
  cfg.dynamicSmemBytes = kLpSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  VT_RETURN_IF_CUDA(cudaLaunchKernelEx(&cfg, rows, a));
  cfg = {};
  cfg.gridDim = dim3((unsigned)a.B);
  cfg.blockDim = dim3(kBsNT);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  VT_RETURN_IF_CUDA(cudaLaunchKernelEx(&cfg, beam_merge_kernel<T>, a));
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
  a.t = (double)temperature;
  a.inv_t = 1.0 / a.t;
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
  return elem == 4 ? launch_select<float>(s, a) : launch_select<uint16_t>(s, a);
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
  if (align % 8 == 0) return launch_reorder<uint2>(s, a);
  if (align % 4 == 0) return launch_reorder<uint32_t>(s, a);
  if (align % 2 == 0) return launch_reorder<uint16_t>(s, a);
  return launch_reorder<uint8_t>(s, a);
}
