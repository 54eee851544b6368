// kv4_prompt.cu -- attention over the 4-bit KV cache, many rows a request
// (sm_103a).
//
// Row i of the n new rows of a request of length L sees its tokens
// t <= L - n + i:  out = sum_t softmax(sm_scale q . K_t) V_t, with the cache
// decoded as it is read.  A row that sees nothing gives zeros.
//
// One CTA takes one row and one query head, 128 tokens at a time: a thread
// scores a token, the block shares the running maximum and sum, and a thread
// then sums a dim over the tokens.
#include "internal.h"
#include "kv4.cuh"

namespace w8a8 {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float load16(const void* p, int fp16, size_t i) {
  if (fp16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

template <int KIND>
__device__ __forceinline__ float code_value(const uint8_t* row, const uint8_t* scales, int d) {
  uint32_t h[4];
  kv4_decode8<KIND>(row[d / 2] >> (4 * (d & 1)), kv4_scale<KIND>(e4m3x2_to_half2(scales[d / kKv4Group] * 0x101u)), h);
  const __half2 v = *reinterpret_cast<const __half2*>(&h[0]);
  return __low2float(v);
}

template <int KIND>
__global__ void __launch_bounds__(kThreads) kv4_prompt_kernel(const Kv4AttnParams p) {
  __shared__ float s_q[128], s_p[kThreads];
  __shared__ float s_red[kThreads / 32];
  __shared__ long long s_rec[kThreads];
  const int h = blockIdx.x % p.num_q_heads, i = blockIdx.x / p.num_q_heads, b = blockIdx.y, tid = threadIdx.x;
  const int first = p.query_start ? min(max(__ldg(p.query_start + b), 0), p.tokens) : b;
  const int n = p.query_start ? min(max(__ldg(p.query_start + b + 1) - first, 0), min(p.tokens - first, p.max_query_len)) : 1;
  if (i >= n) return;
  const int kvh = h / (p.num_q_heads / p.num_kv_heads), d = p.head_dim;
  const long long room = static_cast<long long>(p.max_blocks) * p.block_size;
  const int len = static_cast<int>(min(static_cast<long long>(max(__ldg(p.seq_lens + b), 0)), room));
  const int seen = max(0, len - n + i + 1);
  if (tid < d) s_q[tid] = load16(p.q, p.q_fp16, static_cast<size_t>(first + i) * p.q_token_stride + h * p.q_head_stride + tid);
  const float cs = p.sm_scale * __ldg(p.k_scale) * 1.4426950408889634f;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int t0 = 0; t0 < seen; t0 += kThreads) {
    __syncthreads();
    const int t = t0 + tid;
    float s = -INFINITY;
    s_rec[tid] = -1;
    if (t < seen) {
      const int blk = __ldg(p.block_table + static_cast<size_t>(b) * p.max_blocks + t / p.block_size);
      if (blk >= 0 && blk < p.num_blocks) {
        const int off = t % p.block_size;
        const size_t rec = kv4_record_of(blk, kvh, p.num_kv_heads, p.block_size, off) * kv4_record_bytes(d);
        s_rec[tid] = static_cast<long long>(rec);
        const uint8_t* base = static_cast<const uint8_t*>(p.cache) + rec;
        const int row = off % kKv4Tokens;
        s = 0.f;
        for (int j = 0; j < d; ++j)
          s += s_q[j] * code_value<KIND>(base + row * (d / 2), base + kv4_scales_at(d, 0) + row * (d / 16), j);
        s *= cs;
      }
    }
    float mx = s;
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    if (tid % 32 == 0) s_red[tid / 32] = mx;
    __syncthreads();
    mx = m;
    for (int w = 0; w < kThreads / 32; ++w) mx = fmaxf(mx, s_red[w]);
    const float alpha = mx == -INFINITY ? 1.f : exp2f(m - mx);
    m = mx;
    const float w = s == -INFINITY ? 0.f : exp2f(s - mx);
    s_p[tid] = w;
    l = l * alpha + w;
    o *= alpha;
    __syncthreads();
    if (tid < d) {
      for (int j = 0; j < kThreads && t0 + j < seen; ++j) {
        if (s_rec[j] < 0) continue;
        const uint8_t* base = static_cast<const uint8_t*>(p.cache) + s_rec[j];
        const int row = (t0 + j) % p.block_size % kKv4Tokens;
        o += s_p[j] * code_value<KIND>(base + kv4_codes_at(d, 1) + row * (d / 2),
                                       base + kv4_scales_at(d, 1) + row * (d / 16), tid);
      }
    }
  }
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  __syncthreads();
  if (tid % 32 == 0) s_red[tid / 32] = l;
  __syncthreads();
  l = 0.f;
  for (int w = 0; w < kThreads / 32; ++w) l += s_red[w];
  if (tid < d) {
    const float y = l > 0.f ? o / l * __ldg(p.v_scale) : 0.f;
    const size_t at = static_cast<size_t>(first + i) * p.out_token_stride + h * p.out_head_stride + tid;
    if (p.out_fp16) static_cast<__half*>(p.out)[at] = __float2half_rn(y);
    else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
  }
}

}  // namespace

cudaError_t launch_kv4_prompt(const Kv4AttnParams& p, cudaStream_t stream) {
  const dim3 grid(p.num_q_heads * p.max_query_len, p.batch);
  if (p.kind == W8A8_KV4_E2M1) kv4_prompt_kernel<W8A8_KV4_E2M1><<<grid, kThreads, 0, stream>>>(p);
  else kv4_prompt_kernel<W8A8_KV4_INT4><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace w8a8
