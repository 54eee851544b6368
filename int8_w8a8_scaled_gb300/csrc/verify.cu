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
// Bound by the bytes of one target and one draft row for each request.  A row
// is shared by a cluster of CTAs (8 for a few requests: one SM alone draws
// about 100 GB/s; one where there are as many requests as SMs), whose warps
// sum consecutive pieces.  The piece that holds
// the draw follows from all pieces' sums, exchanged through distributed
// shared memory; its CTA reads it once more (from L2) and narrows it down.
//
// Sums and comparisons have to be good to about 48 bits: a 32-bit running sum
// over 10^5 weights is off by more than most of them.  A GB300 SM adds two
// 64-bit numbers a cycle, so the long sums are made in pairs of 32-bit ones:
// with p > q >= 0 the difference is p - q = h + (p - h - q) exactly, h
// rounded, and each addition keeps its rounding error (Knuth's two-sum).  64
// bits proper are left to the few sums of pieces and to the walk.  u q is a
// product of two 24-bit numbers, which 64 bits hold exactly.
//
// Measured (device time): 128 requests of 131072 tokens 40 us, 3.3 TB/s (sums in 64
// bits: 249 us); 4 of 32000 15-18 us, a chain of latencies.
#include <algorithm>

#include "internal.h"
#include "kv4.cuh"
#include "sm103_ptx.cuh"

namespace w8a8 {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kStride = 128;  // tokens a warp takes at once: 4 of each lane

template <int DT>
__device__ __forceinline__ float widen(uint32_t bits) {
  if (DT == W8A8_FP32) return __uint_as_float(bits);
  if (DT == W8A8_BF16) return __uint_as_float(bits << 16);
  return __half2float(__ushort_as_half(static_cast<uint16_t>(bits)));
}

// a NaN or a negative number weighs nothing
__device__ __forceinline__ float clean(float x) { return x > 0.f ? x : 0.f; }

template <int DT>
__device__ __forceinline__ float prob(const void* p, size_t i) {
  if (DT == W8A8_FP32) return clean(__ldg(static_cast<const float*>(p) + i));
  return clean(widen<DT>(__ldg(static_cast<const uint16_t*>(p) + i)));
}

// 4 consecutive probabilities, 16 (8) bytes aligned.
template <int DT>
__device__ __forceinline__ void prob4(const void* p, size_t i, float (&x)[4]) {
  if (DT == W8A8_FP32) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
    x[0] = clean(v.x);
    x[1] = clean(v.y);
    x[2] = clean(v.z);
    x[3] = clean(v.w);
  } else {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i));
    x[0] = clean(widen<DT>(v.x & 0xFFFFu));
    x[1] = clean(widen<DT>(v.x >> 16));
    x[2] = clean(widen<DT>(v.y & 0xFFFFu));
    x[3] = clean(widen<DT>(v.y >> 16));
  }
}

// The weights of a draw.
struct Weights {
  const void* p;
  const void* q;  // null: none
  size_t p_at, q_at;
  int hole;       // a token of weight 0 (-1: none)
};

// A sum as two fp32 numbers.
struct Pair {
  float h = 0.f, l = 0.f;
  // + (a + e), e small against a
  __device__ __forceinline__ void add(float a, float e) {
    const float s = __fadd_rn(h, a), b = __fsub_rn(s, h);
    l = __fadd_rn(l, __fadd_rn(__fadd_rn(__fsub_rn(h, __fsub_rn(s, b)), __fsub_rn(a, b)), e));
    h = s;
  }
  // + max(p - q, 0)
  __device__ __forceinline__ void add_difference(float p, float q) {
    q = fminf(p, q);
    const float d = __fsub_rn(p, q);
    add(d, __fsub_rn(__fsub_rn(p, d), q));
  }
};

// Sum of the tokens [v0, v1) over a warp, in every lane.  kQ: less a second
// row.
template <int DT, bool kVec, bool kQ>
__device__ __forceinline__ double warp_sum(const Weights& w, int v0, int v1, int lane) {
  Pair sum;
  if (kVec) {
    int v = v0 + 4 * lane;
    auto take = [&](int at, const float (&p)[4], const float (&q)[4]) {
      float x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = p[k];
      if (!kQ && static_cast<unsigned>(w.hole - at) < 4u) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (at + k == w.hole) x[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) sum.add_difference(x[k], q[k]);
    };
    // four loads of each row in flight (a loop left after any of its loads would not have them)
    constexpr int kAhead = 4;
    for (; v + (kAhead - 1) * kStride + 4 <= v1; v += kAhead * kStride) {
      float p[kAhead][4], q[kAhead][4];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        prob4<DT>(w.p, w.p_at + v + i * kStride, p[i]);
        q[i][0] = q[i][1] = q[i][2] = q[i][3] = 0.f;
        if (kQ) prob4<DT>(w.q, w.q_at + v + i * kStride, q[i]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) take(v + i * kStride, p[i], q[i]);
    }
    for (; v + 4 <= v1; v += kStride) {
      float p[4], q[4] = {0.f, 0.f, 0.f, 0.f};
      prob4<DT>(w.p, w.p_at + v, p);
      if (kQ) prob4<DT>(w.q, w.q_at + v, q);
      take(v, p, q);
    }
    for (int k = v; k < min(v1, v + 4); ++k)  // the row's end
      sum.add_difference(k == w.hole ? 0.f : prob<DT>(w.p, w.p_at + k), kQ ? prob<DT>(w.q, w.q_at + k) : 0.f);
  } else {
#pragma unroll 4
    for (int v = v0 + lane; v < v1; v += 32)
      sum.add_difference(v == w.hole ? 0.f : prob<DT>(w.p, w.p_at + v), kQ ? prob<DT>(w.q, w.q_at + v) : 0.f);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    sum.add(__shfl_xor_sync(0xffffffffu, sum.h, off), __shfl_xor_sync(0xffffffffu, sum.l, off));
  // the lanes add in different orders: all take lane 0's
  return static_cast<double>(__shfl_sync(0xffffffffu, sum.h, 0)) + static_cast<double>(__shfl_sync(0xffffffffu, sum.l, 0));
}

template <int DT, bool kVec>
__global__ void __launch_bounds__(kThreads, 1) verify_kernel(const VerifyArgs a) {
  __shared__ double s_sum[kWarps];
  __shared__ double s_before, s_goal;
  __shared__ int s_kept, s_owner;  // s_owner: the piece that holds the draw
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int rank = static_cast<int>(cluster_ctarank()), b = static_cast<int>(cluster_id_x());
  const int first = min(max(__ldg(a.draft_start + b), 0), a.rows);
  const int n = min(min(max(__ldg(a.draft_start + b + 1) - first, 0), a.rows - first), a.max_drafts);
  // ---- the first token that is not kept: 32 at a time, by every CTA for itself
  if (warp == 0) {
    int kept = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      bool keep = false;
      if (i < n) {
        const int x = __ldg(a.draft_tokens + first + i);
        const double u = __ldg(a.uniform + first + i);
        if (x >= 0 && x < a.vocab) {
          const double p = prob<DT>(a.target, static_cast<size_t>(first + b + i) * a.target_ld + x);
          const double q = a.draft ? prob<DT>(a.draft, static_cast<size_t>(first + i) * a.draft_ld + x) : 1.0;
          keep = u * q < p;
        }
      }
      const uint32_t lost = ~__ballot_sync(0xffffffffu, keep);
      kept = i0 + (lost ? __ffs(lost) - 1 : 32);
      if (lost) break;
    }
    if (lane == 0) s_kept = min(kept, n);
  }
  __syncthreads();
  const int kept = s_kept;
  int* out = a.out_tokens + static_cast<size_t>(b) * (a.max_drafts + 1);
  if (rank == 0) {
    if (tid == 0) a.num_accepted[b] = kept;
    for (int i = tid; i <= a.max_drafts; i += kThreads)
      if (i != kept) out[i] = i < kept ? __ldg(a.draft_tokens + first + i) : -1;
  }
  Weights w;
  w.p = a.target;
  w.p_at = static_cast<size_t>(first + b + kept) * a.target_ld;
  w.q = kept < n ? a.draft : nullptr;
  w.q_at = static_cast<size_t>(first + kept) * a.draft_ld;
  w.hole = kept < n && !a.draft ? __ldg(a.draft_tokens + first + kept) : -1;
  const double u = __ldg(a.sample_uniform + b);
  // ---- the pieces' sums; a second time over the target alone if nothing is left of it
  static_assert(kWarps == 32, "a warp looks at one sum in each lane");
  const int pieces = a.cluster * kWarps, mine = rank * kWarps + warp;
  const int per = ((a.vocab + pieces - 1) / pieces + kStride - 1) / kStride * kStride;
  const int v0 = static_cast<int>(min(static_cast<long long>(a.vocab), static_cast<long long>(mine) * per));
  const int v1 = min(a.vocab, v0 + per);
  constexpr int kLanePieces = kMaxCluster * kWarps / 32;
  for (int pass = 0;; ++pass) {
    const double sum = w.q ? warp_sum<DT, kVec, true>(w, v0, v1, lane) : warp_sum<DT, kVec, false>(w, v0, v1, lane);
    if (lane == 0) s_sum[warp] = sum;
    cluster_sync();
    // one warp of each CTA looks at all pieces: lane l at pieces 4 l .. 4 l + 3
    if (warp == 0) {
      double piece[kLanePieces], run = 0.0;
#pragma unroll
      for (int k = 0; k < kLanePieces; ++k) {
        const int i = lane * kLanePieces + k;
        piece[k] = 0.0;
        if (i < pieces) {
          const uint32_t at = mapa_shared(smem_addr(&s_sum[i % kWarps]), i / kWarps);
          const uint32_t lo = ld_dsmem_u32(at), hi = ld_dsmem_u32(at + 4);
          piece[k] = __hiloint2double(static_cast<int>(hi), static_cast<int>(lo));
        }
        run += piece[k];
      }
      double upto = run;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += o;
      }
      const double goal = u * __shfl_sync(0xffffffffu, upto, 31);
      // the first piece that passes the goal; with none (a rounding) the last of any weight
      double c = upto - run, c_first = 0.0, c_last = 0.0;
      int i_first = 1 << 20, i_last = -1;
#pragma unroll
      for (int k = 0; k < kLanePieces; ++k) {
        const int i = lane * kLanePieces + k;
        if (piece[k] > 0.0) {
          if (c + piece[k] > goal && i < i_first) {
            i_first = i;
            c_first = c;
          }
          i_last = i;
          c_last = c;
        }
        c += piece[k];
      }
      const int lowest = __reduce_min_sync(0xffffffffu, i_first), highest = __reduce_max_sync(0xffffffffu, i_last);
      const int owner = lowest < (1 << 20) ? lowest : highest;
      if (lane == max(owner, 0) / kLanePieces) {
        s_owner = owner;
        s_before = lowest < (1 << 20) ? c_first : c_last;
        s_goal = goal;
      }
    }
    cluster_sync();  // the sums have been read: they may change, and CTAs may end
    if (s_owner >= 0 || pass == 1) break;
    w.q = nullptr;
    w.hole = -1;
  }
  const int owner = s_owner;
  if (owner < 0) {  // no token has any probability
    if (rank == 0 && tid == 0) out[kept] = -1;
    return;
  }
  if (owner / kWarps != rank) return;
  // ---- the owner's CTA narrows the piece down to 128 tokens, its warps summing
  // a 32nd of what is left each time
  const double goal = s_goal;
  int lo = static_cast<int>(min(static_cast<long long>(a.vocab), static_cast<long long>(owner) * per));
  int hi = min(a.vocab, lo + per);
  double c = s_before;
  while (hi - lo > kStride) {
    const int part = ((hi - lo + kWarps - 1) / kWarps + kStride - 1) / kStride * kStride;
    const int p0 = static_cast<int>(min(static_cast<long long>(hi), lo + static_cast<long long>(warp) * part)), p1 = min(hi, p0 + part);
    const double sum = w.q ? warp_sum<DT, kVec, true>(w, p0, p1, lane) : warp_sum<DT, kVec, false>(w, p0, p1, lane);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    // every warp for itself: the first part that passes the goal, or the last of any weight
    const double mine_sum = s_sum[lane];
    double upto = mine_sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const double o = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += o;
    }
    const uint32_t any = __ballot_sync(0xffffffffu, mine_sum > 0.0);
    const uint32_t passes = __ballot_sync(0xffffffffu, mine_sum > 0.0 && c + upto > goal);
    const int pick = passes ? __ffs(passes) - 1 : any ? 31 - __clz(any) : 0;
    const double front = __shfl_sync(0xffffffffu, upto - mine_sum, pick);
    c += front;
    lo = static_cast<int>(min(static_cast<long long>(hi), lo + static_cast<long long>(pick) * part));
    hi = min(hi, lo + part);
    __syncthreads();  // the sums have been read
  }
  if (warp != 0) return;
  double x[4], run = 0.0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int t = lo + 4 * lane + k;
    x[k] = 0.0;
    if (t < hi && t != w.hole) {
      const float p = prob<DT>(w.p, w.p_at + t);
      x[k] = w.q ? fmax(static_cast<double>(p) - static_cast<double>(prob<DT>(w.q, w.q_at + t)), 0.0) : p;
    }
    run += x[k];
  }
  double upto = run;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const double o = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += o;
  }
  double at = c + (upto - run);
  int found = 1 << 30, some = -1;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    at += x[k];
    const int t = lo + 4 * lane + k;
    if (x[k] > 0.0) {
      if (at > goal && found == (1 << 30)) found = t;
      some = t;
    }
  }
  found = __reduce_min_sync(0xffffffffu, found);
  some = __reduce_max_sync(0xffffffffu, some);  // nothing passes (a rounding): the last of any weight
  if (lane == 0) out[kept] = found < (1 << 30) ? found : some;
}

template <int DT, bool kVec>
cudaError_t launch_t(const VerifyArgs& a, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(a.cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * a.cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, verify_kernel<DT, kVec>, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int DT>
cudaError_t launch_dt(const VerifyArgs& a, cudaStream_t stream) {
  // 4 probabilities in one load where every row begins aligned
  const size_t bytes = DT == W8A8_FP32 ? 16 : 8;
  const bool vec = reinterpret_cast<uintptr_t>(a.target) % bytes == 0 && reinterpret_cast<uintptr_t>(a.draft) % bytes == 0 &&
                   a.target_ld % 4 == 0 && (!a.draft || a.draft_ld % 4 == 0);
  return vec ? launch_t<DT, true>(a, stream) : launch_t<DT, false>(a, stream);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& args, int num_sms, cudaStream_t stream) {
  VerifyArgs a = args;
  // as many CTAs to a row as there are SMs for, while a warp keeps 128 tokens
  // (128 rows of 131072: one CTA each; 4 CTAs of 512 threads each took twice as long)
  a.cluster = kMaxCluster;
  while (a.cluster > 1 && (static_cast<long long>(a.batch) * a.cluster > num_sms ||
                           a.vocab < a.cluster * kWarps * kStride))
    a.cluster /= 2;
  switch (a.dtype) {
    case W8A8_FP32: return launch_dt<W8A8_FP32>(a, stream);
    case W8A8_BF16: return launch_dt<W8A8_BF16>(a, stream);
    default: return launch_dt<W8A8_FP16>(a, stream);
  }
}

}  // namespace w8a8
