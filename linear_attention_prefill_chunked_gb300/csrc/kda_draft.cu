// kda_draft.cu -- what follows a pass over drafted tokens: verification against the target's
// probabilities, and the commit of the accepted step's state into the pool.
#include <cooperative_groups.h>

#include <utility>

#include "kda_internal.cuh"

namespace kda {
namespace {

KDA_DEBUG_FLAG_DEFINE();
namespace cg = cooperative_groups;

// ---- verification --------------------------------------------------------------------------
// The draw is a race: with noise e ~ Exp(1), argmax w / e falls on an entry in proportion to w.
// Each entry's score is one subtraction and one rounded division, so the drawn token does not
// depend on the order of any sum.
//
// Bound by HBM (a request reads one row of p and noise, and of q after a refusal: 8..12 bytes an
// entry), or by latency for few requests: a cluster of CTAs shares a request's row, reads it once
// with 16-byte loads and joins its best entries through distributed shared memory.
//
// 64 requests of 131072 entries (82 MB) take 16.7 us, 4.9 TB/s; 12.4 us is a copy's rate, and the
// chain before the row (lengths, tokens, their probabilities) is three trips to memory.  Loads are
// issued three rows of 16 bytes an operand ahead of their use (one: 21 us; four need 72 registers: 23 us).
// CTAs of 256 threads let all 512 of those be resident (512 threads: two waves, 20.1 us); requests too
// few to fill the GPU so take 512 (one of 32003 entries: 5.9 us against 7.4 us).
constexpr int kMaxRanks = 8, kBatch = 3;

struct Best {
  float score;
  int at;
};
__device__ __forceinline__ Best better(Best a, Best b) {
  return (b.score > a.score || (b.score == a.score && b.at < a.at)) ? b : a;
}

// w / e against the best so far; entries come in rising order, so an equal one never replaces it.
__device__ __forceinline__ void race(Best& best, float w, float e, int at) {
  // the product rules most entries out without a division; it is a few roundings off at most
  if (!(w > 0.f) || !(w >= best.score * e * 0.99999f)) return;
  const float s = __fdiv_rn(w, e);
  if (s > best.score) best = {s, at};
}

// The best entry of this CTA's share of the row.  kDiff: w = max(p - q, 0).
template <int kThreads, bool kDiff>
__device__ __forceinline__ Best scan_row(const float* __restrict__ p, const float* __restrict__ q,
                                         int hot, const float* __restrict__ e, int vocab, int rank,
                                         int ranks) {
  Best best{-1.f, 0x7fffffff};
  auto one = [&](int i, float pv, float qv, float ev) {
    if (kDiff) pv -= q ? qv : (i == hot ? 1.f : 0.f);
    race(best, pv, ev, i);
  };
  const bool wide = vocab % 4 == 0 && (((uintptr_t)p | (uintptr_t)e | (uintptr_t)(kDiff && q ? q : p)) % 16) == 0;
  const int stride = ranks * kThreads;
  if (wide) {
    const int nv = vocab / 4;
    const float4* p4 = reinterpret_cast<const float4*>(p);
    const float4* q4 = reinterpret_cast<const float4*>(q);
    const float4* e4 = reinterpret_cast<const float4*>(e);
    for (int i0 = rank * kThreads + threadIdx.x; i0 < nv; i0 += kBatch * stride) {
      float4 a[kBatch], b[kBatch], c[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {  // a batch's loads before its first use
        const int i = i0 + k * stride;
        a[k] = b[k] = c[k] = make_float4(0.f, 0.f, 0.f, 0.f);  // a weight of zero never wins
        if (i < nv) {
          a[k] = p4[i];
          c[k] = e4[i];
          if (kDiff && q) b[k] = q4[i];
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = 4 * (i0 + k * stride);
        one(i, a[k].x, b[k].x, c[k].x);
        one(i + 1, a[k].y, b[k].y, c[k].y);
        one(i + 2, a[k].z, b[k].z, c[k].z);
        one(i + 3, a[k].w, b[k].w, c[k].w);
      }
    }
  } else {
#pragma unroll 4
    for (int i = rank * kThreads + threadIdx.x; i < vocab; i += stride)
      one(i, p[i], kDiff && q ? q[i] : 0.f, e[i]);
  }
  return best;
}

// Joins the cluster's best entries: each CTA puts its own into every CTA's `all`, so that one barrier
// of the cluster suffices and what is read after it is the CTA's own.
template <int kThreads>
__device__ __forceinline__ Best join(Best b, Best* s_warp, Best* all, cg::cluster_group& cl) {
  auto across = [](Best x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      Best other{__shfl_xor_sync(0xffffffffu, x.score, o), __shfl_xor_sync(0xffffffffu, x.at, o)};
      x = better(x, other);
    }
    return x;
  };
  b = across(b);
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = b;
  __syncthreads();
  if (threadIdx.x < 32) {
    b = across(threadIdx.x < kThreads / 32 ? s_warp[threadIdx.x] : Best{-1.f, 0x7fffffff});
    if (threadIdx.x < cl.num_blocks()) cl.map_shared_rank(all, threadIdx.x)[cl.block_rank()] = b;
  }
  cl.sync();
  b = all[0];
  for (unsigned r = 1; r < cl.num_blocks(); ++r) b = better(b, all[r]);
  return b;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads)
verify_kernel(const int32_t* __restrict__ tokens, const float* __restrict__ p,
              const float* __restrict__ q, const float* __restrict__ u,
              const float* __restrict__ noise, const int32_t* __restrict__ cu,
              int32_t* __restrict__ kept, int32_t* __restrict__ next,
              uint32_t* __restrict__ status, int N, int64_t T, int vocab, uint32_t flags) {
  __shared__ Best s_warp[kThreads / 32], s_all[2][kMaxRanks];
  __shared__ int s_stop, s_bad;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), ranks = (int)cl.num_blocks();
  const int n = (int)(blockIdx.x / ranks) - 1, tid = threadIdx.x;

  if (n < 0) {  // the first cluster's: the status word, bad lengths and drafted tokens outside the vocabulary
    if (rank != 0) return;
    uint32_t bits = 0;
    for (int i = tid; i < N; i += kThreads) {
      int64_t a, b;
      if (!seq_bounds(cu, i, T, &a, &b)) {
        bits |= KDA_DEVICE_BAD_SEQLENS;
        continue;
      }
      for (int64_t t = a + 1; t < b; ++t)
        if (tokens[t] < 0 || tokens[t] >= vocab) bits |= KDA_DEVICE_BAD_TOKEN;
    }
    const int s = __syncthreads_or((int)(bits & KDA_DEVICE_BAD_SEQLENS));
    const int k = __syncthreads_or((int)(bits & KDA_DEVICE_BAD_TOKEN));
    if (tid == 0)
      set_status(status, (s ? KDA_DEVICE_BAD_SEQLENS : 0u) | (k ? KDA_DEVICE_BAD_TOKEN : 0u));
    return;
  }

  // this CTA's part of the noise is wanted whatever is accepted: on its way while that is found out (without
  // a token in the batch there may be no noise)
  if (T > 0)
    for (int64_t i = ((int64_t)rank * kThreads + tid) * 32; i < vocab; i += (int64_t)ranks * kThreads * 32)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(noise + (int64_t)n * vocab + i));

  // every CTA of the cluster has to have started before another writes into its shared memory: said
  // here and waited for after the accepted tokens are known
  auto started = cl.barrier_arrive();
  auto skipped = [&] {
    if (rank != 0 || tid != 0) return;
    if (flags & KDA_VERIFY_MARK_COUNT) kept[n] = 0;
    if (flags & KDA_VERIFY_MARK_TOKEN) next[n] = -1;
  };
  int64_t bos, eos;
  if (!seq_bounds(cu, n, T, &bos, &eos)) {  // the whole cluster, as at each return below
    cl.barrier_wait(std::move(started));
    skipped();
    return;
  }
  const int len = (int)(eos - bos);
  if (len == 0) {
    cl.barrier_wait(std::move(started));
    if (rank == 0 && tid == 0) {
      kept[n] = 0;
      next[n] = -1;
    }
    return;
  }
  // the first drafted token that is refused (position of the token before it)
  if (tid == 0) {
    s_stop = len - 1;
    s_bad = 0;
  }
  __syncthreads();
  for (int j = tid; j < len - 1; j += kThreads) {
    const int64_t t = bos + j;
    const int d = tokens[t + 1];
    if (d < 0 || d >= vocab) {
      s_bad = 1;
    } else {
      const float qd = q ? q[t * vocab + d] : 1.f;
      if (!(__fmul_rn(u[t], qd) < p[t * vocab + d])) atomicMin(&s_stop, j);
    }
  }
  __syncthreads();
  cl.barrier_wait(std::move(started));
  if (s_bad) {  // the whole cluster read the same tokens
    skipped();
    return;
  }
  const int stop = s_stop;
  const int64_t r = bos + stop;
  const float* pr = p + r * vocab;
  const float* e = noise + (int64_t)n * vocab;
  Best best{-1.f, 0x7fffffff};
  if (stop < len - 1) {
    best = scan_row<kThreads, true>(pr, q ? q + r * vocab : nullptr, tokens[r + 1], e, vocab, rank, ranks);
    best = join<kThreads>(best, s_warp, s_all[0], cl);
  }
  if (best.score < 0.f) {  // every draft kept, or nothing left of the difference
    best = scan_row<kThreads, false>(pr, nullptr, 0, e, vocab, rank, ranks);
    best = join<kThreads>(best, s_warp, s_all[1], cl);
  }
  if (rank == 0 && tid == 0) {
    kept[n] = stop + 1;
    next[n] = best.score < 0.f ? -1 : best.at;
  }
}

// ---- commit --------------------------------------------------------------------------------
// A gathered copy, bound by HBM: a block moves kCommitThreads x kCommitLoads vectors of a row, all its
// loads issued before its stores.  Requests' states of 32 x 128 x 128 in fp32 (128 of them, 447 MB read and
// written) take 70 us, 94 % of a copy's rate.
constexpr int kCommitThreads = 256, kCommitLoads = 8;

template <typename V>
__global__ void __launch_bounds__(kCommitThreads)
commit_kernel(const V* __restrict__ cache, int64_t pitch, int64_t row, int max_steps,
              const int32_t* __restrict__ kept, V* __restrict__ pool, int64_t num_slots,
              int64_t slot_stride, const int32_t* __restrict__ idx, uint32_t* __restrict__ status,
              int N) {
  const int n = blockIdx.x, tid = threadIdx.x;
  if (n == 0 && blockIdx.y == 0) {
    uint32_t bits = 0;
    for (int i = tid; i < N; i += kCommitThreads) {
      if (kept[i] < 0 || kept[i] > max_steps) bits |= KDA_DEVICE_BAD_COUNT;
      if (idx ? resolve_slot(idx, i, num_slots) < 0 : i >= num_slots) bits |= KDA_DEVICE_BAD_SLOT;
    }
    const int c = __syncthreads_or((int)(bits & KDA_DEVICE_BAD_COUNT));
    const int s = __syncthreads_or((int)(bits & KDA_DEVICE_BAD_SLOT));
    if (tid == 0)
      set_status(status, (c ? KDA_DEVICE_BAD_COUNT : 0u) | (s ? KDA_DEVICE_BAD_SLOT : 0u));
  }
  const int a = kept[n];
  if (a <= 0 || a > max_steps) return;
  const int64_t slot = idx ? resolve_slot(idx, n, num_slots) : (n < num_slots ? n : -1);
  if (slot < 0) return;
  const V* src = cache + n * pitch + (a - 1) * row;
  V* dst = pool + slot * slot_stride;
  for (int64_t base = (int64_t)blockIdx.y * kCommitThreads * kCommitLoads; base < row;
       base += (int64_t)gridDim.y * kCommitThreads * kCommitLoads) {
    V v[kCommitLoads];
#pragma unroll
    for (int i = 0; i < kCommitLoads; ++i) {
      const int64_t k = base + i * kCommitThreads + tid;
      if (k < row) v[i] = src[k];
    }
#pragma unroll
    for (int i = 0; i < kCommitLoads; ++i) {
      const int64_t k = base + i * kCommitThreads + tid;
      if (k < row && KDA_CHECK(slot * slot_stride + k < num_slots * slot_stride)) dst[k] = v[i];
    }
  }
  KDA_DEBUG_FOLD(status);
}

template <typename V>
cudaError_t commit_as(int N, int64_t row, const void* cache, int64_t pitch, int max_steps,
                      const int32_t* kept, void* pool, int64_t num_slots, int64_t slot_stride,
                      const int32_t* idx, uint32_t* status, cudaStream_t st) {
  const int64_t per = (int64_t)kCommitThreads * kCommitLoads;
  const int64_t y = (row + per - 1) / per;
  dim3 grid((unsigned)N, (unsigned)(y < 65535 ? y : 65535));
  commit_kernel<V><<<grid, kCommitThreads, 0, st>>>((const V*)cache, pitch, row, max_steps, kept,
                                                    (V*)pool, num_slots, slot_stride, idx, status, N);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_verify(int N, int64_t T, int vocab, const int32_t* tokens, const float* p,
                          const float* q, const float* u, const float* noise, const int32_t* cu,
                          int32_t* kept, int32_t* next, uint32_t* status, uint32_t flags, cudaStream_t st) {
  // a CTA a request fills the GPU from two an SM on; below that the row is shared
  const int sms = gpu_sms();
  int ranks = 1;
  while (ranks < kMaxRanks && (int64_t)N * ranks < 2 * sms && (int64_t)ranks * 4096 < vocab) ranks *= 2;
  const bool few = (int64_t)N * ranks <= sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((N + 1) * ranks));  // (num_seqs is at most 2^27)
  cfg.blockDim = dim3(few ? 512 : 256);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few ? verify_kernel<512> : verify_kernel<256>, tokens, p, q, u, noise, cu, kept, next, status, N,
                            T, vocab, flags);
}

cudaError_t launch_commit(int N, int elem_bytes, int64_t row, const void* cache, int64_t pitch,
                          int max_steps, const int32_t* kept, void* pool, int64_t num_slots,
                          int64_t slot_stride, const int32_t* idx, uint32_t* status,
                          cudaStream_t st) {
  const int64_t e = elem_bytes;
  // 16 bytes at a time where every row starts and ends on such a boundary, else by elements
  if (row * e % 16 == 0 && pitch * e % 16 == 0 && slot_stride * e % 16 == 0 &&
      ((uintptr_t)cache | (uintptr_t)pool) % 16 == 0)
    return commit_as<uint4>(N, row * e / 16, cache, pitch * e / 16, max_steps, kept, pool, num_slots,
                            slot_stride * e / 16, idx, status, st);
  if (e == 2)
    return commit_as<uint16_t>(N, row, cache, pitch, max_steps, kept, pool, num_slots, slot_stride,
                               idx, status, st);
  return commit_as<uint32_t>(N, row, cache, pitch, max_steps, kept, pool, num_slots, slot_stride,
                             idx, status, st);
}

}  // namespace kda
