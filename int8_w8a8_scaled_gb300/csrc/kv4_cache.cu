// kv4_cache.cu -- writing and reading the 4-bit KV cache, and the block
// tables, slots and positions of a serving step's tokens (sm_103a).
#include "internal.h"
#include "kv4.cuh"
#include "quant_math.cuh"

namespace w8a8 {

namespace {

// ------------------------------------------------------------------ cache write
//
// One thread takes one group: 16 dims of one head of one token's key or
// value.  a = max |x| (NaN ignored), s = e4m3(clamp(a / (M g), 2^-9, 448))
// with M the largest code, codes = nearest(x / (s g)), ties to even; a NaN
// becomes code 0 and an infinity the largest code.  Both divisions are
// correctly rounded in fp32, as the 8-bit quantiser's are.

constexpr int kCacheThreads = 256;

// 8 quotients -> a word of codes.
template <int KIND>
__device__ __forceinline__ uint32_t kv4_encode8(float (&y)[8]) {
  uint32_t w = 0u;
  if (KIND == W8A8_KV4_E2M1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = y[i] != y[i] ? 0.f : y[i];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int c;
      asm("cvt.rni.s32.f32 %0, %1;" : "=r"(c) : "f"(y[i]));  // half to even, NaN -> 0, saturating
      w |= static_cast<uint32_t>(max(-7, min(7, c)) & 15) << (4 * i);
    }
  }
  return w;
}

template <int KIND>
__device__ __forceinline__ uint2 kv4_encode16(const float (&x)[16], float sg) {
  float r, lo[8], hi[8];
  const bool ok = recip_ok(sg, &r);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = div_by<false>(x[i], sg, r, ok);
    hi[i] = div_by<false>(x[8 + i], sg, r, ok);
  }
  return make_uint2(kv4_encode8<KIND>(lo), kv4_encode8<KIND>(hi));
}

template <int KIND>
__global__ void __launch_bounds__(kCacheThreads) kv4_write_kernel(const Kv4CacheArgs p) {
  const int groups = p.head_dim / kKv4Group;
  const long long per_token = 2LL * p.heads * groups;
  const long long i = static_cast<long long>(blockIdx.x) * kCacheThreads + threadIdx.x;
  if (i >= p.tokens * per_token) return;
  const long long token = i / per_token;
  int r = static_cast<int>(i % per_token);
  const int which = r / (p.heads * groups);
  r -= which * p.heads * groups;
  const int head = r / groups, grp = r % groups;
  const long long slot = __ldg(p.slots + token);
  if (slot < 0 || slot / p.block_size >= p.num_blocks) return;
  const float g = __ldg(which ? p.v_scale : p.k_scale);
  const uint16_t* src = static_cast<const uint16_t*>(which ? p.v : p.k) +
                        token * (which ? p.v_token_stride : p.k_token_stride) +
                        head * (which ? p.v_head_stride : p.k_head_stride) + grp * kKv4Group;
  uint4 raw[2];
  if (p.vec) {
    raw[0] = __ldg(reinterpret_cast<const uint4*>(src));
    raw[1] = __ldg(reinterpret_cast<const uint4*>(src) + 1);
  } else {
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      u[j] = static_cast<uint32_t>(__ldg(src + 2 * j)) | (static_cast<uint32_t>(__ldg(src + 2 * j + 1)) << 16);
    raw[0] = make_uint4(u[0], u[1], u[2], u[3]);
    raw[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
  float x[16];
  {
    float lo[8], hi[8];
    if (p.fp16) {
      unpack8<1>(raw[0], lo);
      unpack8<1>(raw[1], hi);
    } else {
      unpack8<0>(raw[0], lo);
      unpack8<0>(raw[1], hi);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = lo[j];
      x[8 + j] = hi[j];
    }
  }
  float a = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) a = fmaxf(a, fabsf(x[j]));  // fmaxf drops a NaN
  const float ratio = __fdiv_rn(a, __fmul_rn(kv4_largest(KIND), g));
  const uint32_t scale = e4m3x2(fminf(fmaxf(ratio, 0.001953125f), 448.f), 0.f) & 0xFFu;
  const uint2 codes = kv4_encode16<KIND>(x, __fmul_rn(e4m3_to_float(static_cast<uint8_t>(scale)), g));
  const int off = static_cast<int>(slot % p.block_size), row = off % kKv4Tokens;
  uint8_t* rec = static_cast<uint8_t*>(p.cache) +
                 kv4_record_of(slot / p.block_size, head, p.heads, p.block_size, off) * kv4_record_bytes(p.head_dim);
  *reinterpret_cast<uint2*>(rec + kv4_codes_at(p.head_dim, which) + row * (p.head_dim / 2) + grp * 8) = codes;
  rec[kv4_scales_at(p.head_dim, which) + row * groups + grp] = static_cast<uint8_t>(scale);
}

// ------------------------------------------------------------------ cache read
//
// The inverse: round16(code * s * g), zeros for a token without a slot.

template <int KIND>
__global__ void __launch_bounds__(kCacheThreads) kv4_read_kernel(const Kv4CacheArgs p) {
  const int groups = p.head_dim / kKv4Group;
  const long long per_token = 2LL * p.heads * groups;
  const long long i = static_cast<long long>(blockIdx.x) * kCacheThreads + threadIdx.x;
  if (i >= p.tokens * per_token) return;
  const long long token = i / per_token;
  int r = static_cast<int>(i % per_token);
  const int which = r / (p.heads * groups);
  r -= which * p.heads * groups;
  const int head = r / groups, grp = r % groups;
  const long long slot = __ldg(p.slots + token);
  uint32_t out[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
  if (slot >= 0 && slot / p.block_size < p.num_blocks) {
    const float g = __ldg(which ? p.v_scale : p.k_scale);
    const int off = static_cast<int>(slot % p.block_size), row = off % kKv4Tokens;
    const uint8_t* rec =
        static_cast<const uint8_t*>(p.cache) +
        kv4_record_of(slot / p.block_size, head, p.heads, p.block_size, off) * kv4_record_bytes(p.head_dim);
    const uint2 codes =
        *reinterpret_cast<const uint2*>(rec + kv4_codes_at(p.head_dim, which) + row * (p.head_dim / 2) + grp * 8);
    const float s = e4m3_to_float(rec[kv4_scales_at(p.head_dim, which) + row * groups + grp]);
    uint32_t h[2][4];
    const Kv4Scale one = kv4_scale<KIND>(__float2half2_rn(1.f));
    kv4_decode8<KIND>(codes.x, one, h[0]);
    kv4_decode8<KIND>(codes.y, one, h[1]);
    float y[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&h[j / 4][j % 4]));
      y[8 * (j / 4) + kv4_low<KIND>(j % 4)] = c.x * s * g;
      y[8 * (j / 4) + kv4_high<KIND>(j % 4)] = c.y * s * g;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = y[2 * j], b = y[2 * j + 1];
      if (p.fp16) {
        const __half2 y = __floats2half2_rn(a, b);
        out[j] = *reinterpret_cast<const uint32_t*>(&y);
      } else {
        const __nv_bfloat162 y = __floats2bfloat162_rn(a, b);
        out[j] = *reinterpret_cast<const uint32_t*>(&y);
      }
    }
  }
  uint16_t* dst = static_cast<uint16_t*>(which ? p.v_out : p.k_out) +
                  token * (which ? p.v_token_stride : p.k_token_stride) +
                  head * (which ? p.v_head_stride : p.k_head_stride) + grp * kKv4Group;
  if (p.vec) {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(out[0], out[1], out[2], out[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(out[4], out[5], out[6], out[7]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dst[2 * j] = static_cast<uint16_t>(out[j]);
      dst[2 * j + 1] = static_cast<uint16_t>(out[j] >> 16);
    }
  }
}

// ------------------------------------------------------------------ block tables
//
// need_b = ceil((ctx + new) / S) - ceil(ctx / S) blocks for request b (none
// if it would not fit its table), taken in request order from the end of the
// free list: block i of request b is free[count - 1 - before_b - i], before_b
// the sum of the needs in front of it.  A request is admitted if it fits and
// needs nothing or before_b + need_b <= count.
//
// Every thread block makes the two prefix sums (new tokens, needs; one scan
// of 64-bit pairs) over all requests for itself, in shared memory, and then
// places its own share of the packed tokens: a token's request is found by
// bisection, and a token of a new block names that block without reading the
// table, so that nothing waits for another thread block and one launch does.

constexpr int kTableThreads = 256;

__device__ __forceinline__ int blocks_for(long long tokens, int size) {
  return static_cast<int>((tokens + size - 1) / size);
}

__global__ void __launch_bounds__(kTableThreads) block_table_kernel(const BlockTableArgs p) {
  extern __shared__ int smem[];
  int* s_start = smem;                 // [batch + 1] first packed token of each request
  int* s_before = smem + p.batch + 1;  // [batch] blocks taken before it; -1: not admitted
  __shared__ unsigned long long s_warp[kTableThreads / 32];
  __shared__ unsigned s_used, s_upto;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int count = max(0, min(__ldg(p.free_count), p.free_capacity));
  if (tid == 0) s_used = s_upto = 0u;
  // each thread's run of requests
  const int per = (p.batch + kTableThreads - 1) / kTableThreads;
  const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
  const long long room = static_cast<long long>(p.max_blocks) * p.block_size;
  unsigned long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const long long ctx = max(0, __ldg(p.context_lens + b)), add = max(0, __ldg(p.new_lens + b));
    const unsigned need = ctx + add <= room ? blocks_for(ctx + add, p.block_size) - blocks_for(ctx, p.block_size) : 0;
    mine += (static_cast<unsigned long long>(need) << 32) + add;
  }
  unsigned long long run = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned long long o = __shfl_up_sync(0xffffffffu, run, off);
    if (lane >= off) run += o;
  }
  if (lane == 31) s_warp[warp] = run;
  __syncthreads();
  run -= mine;
  for (int w = 0; w < warp; ++w) run += s_warp[w];
  unsigned used = 0u, upto = 0u;
  for (int b = b0; b < b1; ++b) {
    const long long ctx = max(0, __ldg(p.context_lens + b)), add = max(0, __ldg(p.new_lens + b));
    const bool fits = ctx + add <= room;
    const unsigned need = fits ? blocks_for(ctx + add, p.block_size) - blocks_for(ctx, p.block_size) : 0;
    const unsigned before = static_cast<unsigned>(run >> 32);
    const bool ok = fits && (need == 0 || static_cast<unsigned long long>(before) + need <= static_cast<unsigned>(count));
    const int start = static_cast<int>(run & 0xffffffffu);
    s_start[b] = start;
    s_before[b] = ok ? static_cast<int>(min(before, 0x7fffffffu)) : -1;
    if (ok) upto = max(upto, before + need);
    if (ok && need) used = max(used, before + need);
    if (blockIdx.x == 0) {
      p.query_start[b] = start;
      p.seq_lens[b] = ok ? static_cast<int>(ctx + add) : 0;
    }
    run += (static_cast<unsigned long long>(need) << 32) + add;
  }
  if (b1 == p.batch && b0 < b1) {
    s_start[p.batch] = static_cast<int>(run & 0xffffffffu);
    if (blockIdx.x == 0) p.query_start[p.batch] = static_cast<int>(run & 0xffffffffu);
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    used = __reduce_max_sync(0xffffffffu, used);
    upto = __reduce_max_sync(0xffffffffu, upto);
    if (lane == 0) {
      atomicMax(&s_used, used);
      atomicMax(&s_upto, upto);
    }
    __syncthreads();
    if (tid == 0) {
      *p.free_left = static_cast<int>(max(static_cast<long long>(count) - s_upto, -2147483648LL));
      if (p.free_count_out) *p.free_count_out = count - static_cast<int>(s_used);
    }
  }
  const int total = s_start[p.batch];
  for (long long t = static_cast<long long>(blockIdx.x) * kTableThreads + tid; t < p.tokens;
       t += static_cast<long long>(gridDim.x) * kTableThreads) {
    long long slot = -1;
    int pos = 0;
    if (t < total) {
      int lo = 0, hi = p.batch - 1;  // the last request that starts at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (s_start[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      const int ctx = max(0, __ldg(p.context_lens + lo)), add = max(0, __ldg(p.new_lens + lo));
      const int i = static_cast<int>(t - s_start[lo]), before = s_before[lo];
      pos = ctx + i;
      if (before >= 0 && i < add) {
        const int col = pos / p.block_size, first = blocks_for(ctx, p.block_size);
        int* entry = p.block_table + static_cast<size_t>(lo) * p.max_blocks + col;
        int block;
        if (col >= first) {
          block = __ldg(p.free_blocks + (count - 1 - before - (col - first)));
          if (pos % p.block_size == 0) *entry = block;
        } else {
          block = *entry;
        }
        if (block >= 0) slot = static_cast<long long>(block) * p.block_size + pos % p.block_size;
      }
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
}

}  // namespace

cudaError_t launch_kv4_cache(const Kv4CacheArgs& a, bool write, cudaStream_t stream) {
  const long long n = a.tokens * 2 * a.heads * (a.head_dim / kKv4Group);
  const unsigned grid = static_cast<unsigned>((n + kCacheThreads - 1) / kCacheThreads);
  if (write) {
    if (a.kind == W8A8_KV4_E2M1) kv4_write_kernel<W8A8_KV4_E2M1><<<grid, kCacheThreads, 0, stream>>>(a);
    else kv4_write_kernel<W8A8_KV4_INT4><<<grid, kCacheThreads, 0, stream>>>(a);
  } else {
    if (a.kind == W8A8_KV4_E2M1) kv4_read_kernel<W8A8_KV4_E2M1><<<grid, kCacheThreads, 0, stream>>>(a);
    else kv4_read_kernel<W8A8_KV4_INT4><<<grid, kCacheThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_block_tables(const BlockTableArgs& a, int num_sms, cudaStream_t stream) {
  const int smem = static_cast<int>((2LL * a.batch + 1) * sizeof(int));
  cudaError_t e = cudaFuncSetAttribute(block_table_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  long long grid = (a.tokens + kTableThreads - 1) / kTableThreads;
  if (grid > 2LL * num_sms) grid = 2LL * num_sms;
  if (grid < 1) grid = 1;
  block_table_kernel<<<static_cast<unsigned>(grid), kTableThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace w8a8
