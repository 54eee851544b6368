// fp8_paged.cuh -- a step's rows over the paged fp8 cache, as its kernels see
// them (internal.h has the structures, include/w8a8.h their meaning).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace w8a8 {
namespace {  // each translation unit keeps its own copy

constexpr float kFp8Log2e = 1.4426950408889634f;

struct Fp8Request {
  int first, n;  // its rows in q that are looked at
  int all;       // its new tokens (more than n only past max_query_len)
  int len;       // tokens, the new ones among them
};

__device__ __forceinline__ Fp8Request fp8_request(const Fp8Paged& c, int b) {
  Fp8Request r;
  r.first = b;
  r.all = 1;
  if (c.query_start) {
    r.first = min(max(__ldg(c.query_start + b), 0), c.tokens);
    r.all = max(min(__ldg(c.query_start + b + 1), c.tokens) - r.first, 0);
  }
  r.n = min(r.all, c.max_query_len);
  const long long room = static_cast<long long>(c.max_blocks) * c.block_size;
  r.len = static_cast<int>(min(static_cast<long long>(max(__ldg(c.seq_lens + b), 0)), room));
  return r;
}

// The request that row `token` belongs to (the first, should the starts not
// rise), -1 if none; every thread of the block takes part, `found` is shared.
// The threads look at all requests at once: a bisection would be a chain of
// loads.
__device__ __forceinline__ int fp8_request_of_row(const Fp8Paged& c, int token, int* found) {
  if (!c.query_start) return token < c.batch ? token : -1;
  if (threadIdx.x == 0) *found = 0x7fffffff;
  __syncthreads();
  for (int b = threadIdx.x; b < c.batch; b += blockDim.x) {
    const int first = min(max(__ldg(c.query_start + b), 0), c.tokens);
    const int end = min(__ldg(c.query_start + b + 1), c.tokens);
    if (token >= first && token < end && token - first < c.max_query_len) atomicMin(found, b);
  }
  __syncthreads();
  const int b = *found;
  return b == 0x7fffffff ? -1 : b;
}

__device__ __forceinline__ float2 fp8_to_float2(uint32_t two, int fp16) {
  return fp16 ? __half22float2(*reinterpret_cast<const __half2*>(&two))
              : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&two));
}

__device__ __forceinline__ uint32_t fp8_pack2(float a, float b, int fp16) {
  if (fp16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 8 16-bit values at `src`.
__device__ __forceinline__ uint4 fp8_load8(const uint16_t* src, int vec) {
  if (vec) return __ldg(reinterpret_cast<const uint4*>(src));
  uint32_t u[4];
#pragma unroll
  for (int x = 0; x < 4; ++x)
    u[x] = static_cast<uint32_t>(__ldg(src + 2 * x)) | (static_cast<uint32_t>(__ldg(src + 2 * x + 1)) << 16);
  return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ void fp8_store8(uint16_t* dst, const float (&y)[8], int fp16, int vec) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = fp8_pack2(y[2 * i], y[2 * i + 1], fp16);
  if (vec) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dst[2 * i] = static_cast<uint16_t>(w[i]);
      dst[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
    }
  }
}

// Clears the bytes of a word that are e4m3 NaN codes (0x7F, 0xFF).
__device__ __forceinline__ uint32_t fp8_nan_to_zero(uint32_t w) {
  const uint32_t nan_top = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return w & ~((nan_top >> 7) * 0xFFu);
}

template <typename... Params, typename... Args>
cudaError_t fp8_launch(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

__device__ __forceinline__ void fp8_wait_for_predecessor() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void fp8_let_dependents_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace
}  // namespace w8a8
