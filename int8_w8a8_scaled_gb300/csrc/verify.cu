// verify.cu -- verification of drafted tokens (sm_103a).
//
// Request b drafted n tokens x_0..x_{n-1} from distributions q_i; the target
// model gave p_0..p_n.  Token i is kept while u_i q_i(x_i) < p_i(x_i), u_i
// given.  At the first token j that is not kept the replacement is drawn
// from max(p_j - q_j, 0); with all kept the extra token comes from p_n.  The
// draw is the lowest v with C_v > u C_total, C the running sum of the
// unnormalised weights, u given.  The result then has the target's
// distribution whatever the draft was.
//
// Sums and comparisons are made in 64 bits: a 32-bit running sum over 10^5
// weights is off by more than most of them.  u q is a product of two 24-bit
// numbers, which 64 bits hold exactly.
#include "internal.h"
#include "kv4.cuh"

namespace w8a8 {

namespace {

constexpr int kVerifyThreads = 1024;

template <int DT>
__device__ __forceinline__ float prob(const void* p, size_t i) {
  float x;
  if (DT == W8A8_FP32) x = __ldg(static_cast<const float*>(p) + i);
  else if (DT == W8A8_BF16) x = __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else x = __half2float(static_cast<const __half*>(p)[i]);
  return x > 0.f ? x : 0.f;  // a NaN or a negative number weighs nothing
}

struct Weights {
  const void* p;
  const void* q;  // null: none
  size_t p_at, q_at;
  int hole;       // a token of weight 0 (-1: none)
};

template <int DT>
__device__ __forceinline__ double weight(const Weights& w, int v) {
  double x = prob<DT>(w.p, w.p_at + v);
  if (w.q) x = fmax(x - static_cast<double>(prob<DT>(w.q, w.q_at + v)), 0.0);
  return v == w.hole ? 0.0 : x;
}

// Sums over the block's threads up to this one: without it (the returned
// value; the same bits as its neighbour's *upto) and with it.
__device__ __forceinline__ double block_scan(double x, double* s_warp, double* upto, double* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  double run = x;
  for (int off = 1; off < 32; off <<= 1) {
    const double o = __shfl_up_sync(0xffffffffu, run, off);
    if (lane >= off) run += o;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = run;
  __syncthreads();
  double before = 0.0, all = 0.0;
  for (int w = 0; w < kVerifyThreads / 32; ++w) {
    if (w == warp) before = all;
    all += s_warp[w];
  }
  *total = all;
  *upto = before + run;
  const double left = __shfl_up_sync(0xffffffffu, run, 1);
  return lane ? before + left : before;
}

template <int DT>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyArgs a) {
  __shared__ double s_warp[kVerifyThreads / 32];
  __shared__ int s_accepted, s_pick, s_first, s_last;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int first = min(max(__ldg(a.draft_start + b), 0), a.rows);
  const int n = min(min(max(__ldg(a.draft_start + b + 1) - first, 0), a.rows - first), a.max_drafts);
  if (tid == 0) {
    int i = 0;
    for (; i < n; ++i) {
      const int x = __ldg(a.draft_tokens + first + i);
      if (x < 0 || x >= a.vocab) break;
      const double p = prob<DT>(a.target, static_cast<size_t>(first + b + i) * a.target_ld + x);
      const double q = a.draft ? prob<DT>(a.draft, static_cast<size_t>(first + i) * a.draft_ld + x) : 1.0;
      if (!(static_cast<double>(__ldg(a.uniform + first + i)) * q < p)) break;
    }
    s_accepted = i;
    s_pick = -1;
    s_first = kVerifyThreads;
    s_last = -1;
    a.num_accepted[b] = i;
  }
  __syncthreads();
  const int kept = s_accepted;
  for (int i = tid; i <= a.max_drafts; i += kVerifyThreads)
    if (i != kept)
      a.out_tokens[static_cast<size_t>(b) * (a.max_drafts + 1) + i] = i < kept ? __ldg(a.draft_tokens + first + i) : -1;
  Weights w;
  w.p = a.target;
  w.p_at = static_cast<size_t>(first + b + kept) * a.target_ld;
  w.q = kept < n ? a.draft : nullptr;
  w.q_at = static_cast<size_t>(first + kept) * a.draft_ld;
  w.hole = kept < n && !a.draft ? __ldg(a.draft_tokens + first + kept) : -1;
  // each thread sums a run of consecutive tokens
  const int per = (a.vocab + kVerifyThreads - 1) / kVerifyThreads;
  const int v0 = min(a.vocab, tid * per), v1 = min(a.vocab, v0 + per);
  double mine = 0.0, total, upto;
  for (int v = v0; v < v1; ++v) mine += weight<DT>(w, v);
  double c = block_scan(mine, s_warp, &upto, &total);
  if (!(total > 0.0)) {  // nothing left of the target: draw from all of it
    w.q = nullptr;
    w.hole = -1;
    mine = 0.0;
    for (int v = v0; v < v1; ++v) mine += weight<DT>(w, v);
    c = block_scan(mine, s_warp, &upto, &total);
  }
  const double goal = static_cast<double>(__ldg(a.sample_uniform + b)) * total;
  // the first run that passes the goal; with none (a rounding) the last that has any weight
  if (mine > 0.0) {
    if (upto > goal) atomicMin(&s_first, tid);
    atomicMax(&s_last, tid);
  }
  __syncthreads();
  if (tid == (s_first < kVerifyThreads ? s_first : s_last)) {
    int pick = -1;
    for (int v = v0; v < v1 && !(pick >= 0 && c > goal); ++v) {
      const double x = weight<DT>(w, v);
      c += x;
      if (x > 0.0) pick = v;
    }
    s_pick = pick;
  }
  __syncthreads();
  if (tid == 0) a.out_tokens[static_cast<size_t>(b) * (a.max_drafts + 1) + kept] = s_pick;
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int, cudaStream_t stream) {
  switch (a.dtype) {
    case W8A8_FP32: verify_kernel<W8A8_FP32><<<a.batch, kVerifyThreads, 0, stream>>>(a); break;
    case W8A8_BF16: verify_kernel<W8A8_BF16><<<a.batch, kVerifyThreads, 0, stream>>>(a); break;
    default: verify_kernel<W8A8_FP16><<<a.batch, kVerifyThreads, 0, stream>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace w8a8
