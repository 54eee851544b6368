// fp8_attention.cu -- attention of a step's new tokens over the paged fp8
// cache, over all of it or over the blocks selected for each token (sm_103a).
//
// The simplest form that is right for every case: one CTA to a row of the
// query, a warp to a token, running maximum and sum per warp, joined at the
// end.
#include <algorithm>

#include "fp8_paged.cuh"

namespace w8a8 {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;

__device__ __forceinline__ float e4m3_value(uint8_t code) {
  uint32_t h;
  const uint16_t two = code;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}

template <int D>
__global__ void __launch_bounds__(kThreads) fp8_attention_simple_kernel(const Fp8AttnParams p) {
  constexpr int kPer = D / 32;
  __shared__ int s_found;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  fp8_let_dependents_start();
  fp8_wait_for_predecessor();
  const int token = blockIdx.x, head = blockIdx.y, kvh = head / p.share;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int b = fp8_request_of_row(p.c, token, &s_found);
  if (b < 0) return;
  const Fp8Request r = fp8_request(p.c, b);
  const int pos = r.len - r.all + token - r.first;
  const float scale = p.sm_scale * __ldg(p.k_scale) * kFp8Log2e, vscale = __ldg(p.v_scale);
  float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
  bool bad = false;
  for (int i = 0; i < kPer; ++i) {
    const uint32_t x = static_cast<const uint16_t*>(p.q)[token * p.q_token_stride + head * p.q_head_stride + lane * kPer + i];
    q[i] = fp8_to_float2(x, p.q_fp16).x;
    bad |= !(fabsf(q[i]) < INFINITY);
    o[i] = 0.f;
  }
  bad = __any_sync(0xffffffffu, bad);
  auto attend = [&](long long t) {
    const int blk = __ldg(p.c.block_table + static_cast<size_t>(b) * p.c.max_blocks + t / p.c.block_size);
    if (blk < 0 || blk >= p.c.num_blocks) return;
    const size_t at = ((static_cast<size_t>(blk) * p.c.block_size + t % p.c.block_size) * p.c.num_kv_heads + kvh) * D + lane * kPer;
    float s = 0.f;
    for (int i = 0; i < kPer; ++i) s = fmaf(q[i], e4m3_value(static_cast<const uint8_t*>(p.k_cache)[at + i]), s);
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s = bad ? __int_as_float(0x7fffffff) : s * scale;
    const float mn = s > m ? s : m;
    const float f = mn == -INFINITY ? 1.f : exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = l * f + w;
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * f + w * e4m3_value(static_cast<const uint8_t*>(p.v_cache)[at + i]);
  };
  if (p.selected) {
    const int* cols = p.selected + (static_cast<size_t>(token) * p.c.num_kv_heads + kvh) * p.budget;
    for (int j = warp; j < p.budget; j += kWarps) {
      const long long col = __ldg(cols + j), t0 = col * p.c.block_size;
      if (col < 0 || col >= p.c.max_blocks) continue;
      for (int i = 0; i < p.c.block_size && t0 + i <= pos; ++i) attend(t0 + i);
    }
  } else {
    for (int t = warp; t <= pos; t += kWarps) attend(t);
  }
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
  for (int i = 0; i < kPer; ++i) s_o[warp][lane * kPer + i] = o[i];
  __syncthreads();
  if (threadIdx.x >= D) return;
  float mx = s_m[0];
  for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, s_m[w]);
  float sum = 0.f, y = 0.f;
  for (int w = 0; w < kWarps; ++w) {
    const float f = s_m[w] == -INFINITY ? (s_l[w] == 0.f ? 0.f : 1.f) : exp2f(s_m[w] - mx);
    sum += f * s_l[w];
    y += f * s_o[w][threadIdx.x];
  }
  y = sum != 0.f ? y / sum * vscale : 0.f;
  const uint32_t u = fp8_pack2(y, 0.f, p.out_fp16);
  static_cast<uint16_t*>(p.out)[token * p.out_token_stride + head * p.out_head_stride + threadIdx.x] = static_cast<uint16_t>(u);
}

}  // namespace

namespace {
// Rows up to which the few-rows kernel takes a call.
constexpr int kFewRows = 32;
}  // namespace

size_t fp8_paged_attention_workspace(int share, long long max_query_len, int head_dim, int num_sms) {
  const long long rows = share * max_query_len;
  return fp8_rows_workspace(static_cast<int>(std::min<long long>(rows, kFewRows)), head_dim, num_sms);
}

size_t fp8_sparse_attention_workspace(int share, int head_dim, int num_sms) {
  return fp8_rows_workspace(std::min(share, kFewRows), head_dim, num_sms);
}

cudaError_t read_clear_fp8_status(int* flags) { return read_clear_fp8_rows_status(flags); }

cudaError_t launch_fp8_attention(const Fp8AttnParams& args, const CUtensorMap& map_k, const CUtensorMap& map_v, int num_sms,
                                 void* workspace, cudaStream_t stream) {
  Fp8AttnParams p = args;
  p.counters = static_cast<unsigned*>(workspace);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kFp8CounterBytes);
  p.few_rows = kFewRows;
  const long long rows = p.selected ? std::min(p.share, kFewRows) : static_cast<long long>(p.share) * p.c.max_query_len;
  if (rows <= kFewRows) return launch_fp8_rows(p, static_cast<int>(rows), map_k, map_v, num_sms, stream);
  const dim3 grid(p.c.tokens, p.num_q_heads);
  if (p.c.head_dim == 64) return fp8_launch(fp8_attention_simple_kernel<64>, grid, dim3(kThreads), 0, stream, p);
  return fp8_launch(fp8_attention_simple_kernel<128>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace w8a8
