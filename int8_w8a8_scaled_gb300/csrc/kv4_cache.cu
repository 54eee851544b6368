// kv4_cache.cu -- writing and reading the 4-bit KV cache, and the block
// tables, slots and positions of a serving step's tokens (sm_103a).
#include <algorithm>

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
//
// Bound by the bytes, 2 + 0.5625 an element, once an element takes about ten
// instructions.  So: a block's threads are laid out (groups of a token) x
// (tokens), and nothing is divided to find one's place; a group is looked
// through for NaN by its maximum (max.NaN) and mended apart; the quotient's
// guard against overflow is left out where the group's scale bounds it.
// Measured (device time): 16384 tokens of 8 heads of 128 written and read back
// 54 us, 3.2 TB/s (78 us before).

constexpr int kCacheThreads = 256;

__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// 8 quotients (no NaN) -> a word of codes.
template <int KIND>
__device__ __forceinline__ uint32_t kv4_encode8(const float* y) {
  uint32_t w = 0u;
  if (KIND == W8A8_KV4_E2M1) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  } else {
    // adding 1.5 * 2^23 rounds to the nearest whole number, half to even, and
    // leaves its two's complement in the low bits
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w |= (__float_as_uint(__fadd_rn(fminf(fmaxf(y[i], -7.f), 7.f), 12582912.f)) & 15u) << (4 * i);
  }
  return w;
}

template <int KIND, bool kBounded>
__device__ __forceinline__ uint2 kv4_encode16(const float (&x)[16], float sg) {
  float r, y[16];
  const bool ok = recip_ok(sg, &r);
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = div_by<kBounded>(x[i], sg, r, ok);
  return make_uint2(kv4_encode8<KIND>(y), kv4_encode8<KIND>(y + 8));
}

// A token's record for one head, and its row in it; false: no such slot.
__device__ __forceinline__ bool kv4_place(const Kv4CacheArgs& p, long long slot, int head, int record_bytes,
                                          size_t* record, int* row) {
  if (slot < 0) return false;
  long long block;
  int off;
  if (p.block_shift >= 0) {
    block = slot >> p.block_shift;
    off = static_cast<int>(slot) & (p.block_size - 1);
  } else if (slot < (1LL << 32)) {
    block = static_cast<unsigned>(slot) / static_cast<unsigned>(p.block_size);
    off = static_cast<int>(static_cast<unsigned>(slot) - static_cast<unsigned>(block) * static_cast<unsigned>(p.block_size));
  } else {
    block = slot / p.block_size;
    off = static_cast<int>(slot - block * p.block_size);
  }
  if (block >= p.num_blocks) return false;
  *row = off % kKv4Tokens;
  *record = kv4_record_of(block, head, p.heads, p.block_size, off) * record_bytes;
  return true;
}

template <int KIND, int D>
__global__ void __launch_bounds__(kCacheThreads) kv4_write_kernel(const Kv4CacheArgs p) {
  constexpr int kGroups = D / kKv4Group;
  const long long token = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (token >= p.tokens) return;
  const long long slot = __ldg(p.slots + token);
  const int per_half = p.heads * kGroups;
  for (int i = threadIdx.x; i < 2 * per_half; i += blockDim.x) {
    const int which = i >= per_half, r = i - (which ? per_half : 0);
    const int head = r / kGroups, grp = r % kGroups;
    size_t record;
    int row;
    if (!kv4_place(p, slot, head, kv4_record_bytes(D), &record, &row)) return;
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
    for (int j = 0; j < 16; ++j) a = max_nan(a, fabsf(x[j]));
    if (a != a) {
      a = 0.f;
      for (int j = 0; j < 16; ++j) {
        x[j] = x[j] != x[j] ? 0.f : x[j];
        a = fmaxf(a, fabsf(x[j]));
      }
    }
    const float ratio = __fdiv_rn(a, __fmul_rn(kv4_largest(KIND), g));
    const uint32_t scale = e4m3x2(fminf(fmaxf(ratio, 0.001953125f), 448.f), 0.f) & 0xFFu;
    const float sg = __fmul_rn(e4m3_to_float(static_cast<uint8_t>(scale)), g);
    // with its scale not cut off no quotient passes the largest code by more than a rounding
    const uint2 codes = ratio <= 448.f ? kv4_encode16<KIND, true>(x, sg) : kv4_encode16<KIND, false>(x, sg);
    uint8_t* rec = static_cast<uint8_t*>(p.cache) + record;
    *reinterpret_cast<uint2*>(rec + kv4_codes_at(D, which) + row * (D / 2) + grp * 8) = codes;
    rec[kv4_scales_at(D, which) + row * kGroups + grp] = static_cast<uint8_t>(scale);
  }
}

// ------------------------------------------------------------------ cache read
//
// The inverse: round16(code * s * g), zeros for a token without a slot.

template <int KIND, int D>
__global__ void __launch_bounds__(kCacheThreads) kv4_read_kernel(const Kv4CacheArgs p) {
  constexpr int kGroups = D / kKv4Group;
  const long long token = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (token >= p.tokens) return;
  const long long slot = __ldg(p.slots + token);
  const int per_half = p.heads * kGroups;
  for (int i = threadIdx.x; i < 2 * per_half; i += blockDim.x) {
    const int which = i >= per_half, r = i - (which ? per_half : 0);
    const int head = r / kGroups, grp = r % kGroups;
    uint32_t out[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    size_t record;
    int row;
    if (kv4_place(p, slot, head, kv4_record_bytes(D), &record, &row)) {
      const float g = __ldg(which ? p.v_scale : p.k_scale);
      const uint8_t* rec = static_cast<const uint8_t*>(p.cache) + record;
      const uint2 codes = *reinterpret_cast<const uint2*>(rec + kv4_codes_at(D, which) + row * (D / 2) + grp * 8);
      // code * s is an exact f16 number
      const Kv4Scale s = kv4_scale<KIND>(
          __half2half2(__low2half(e4m3x2_to_half2(rec[kv4_scales_at(D, which) + row * kGroups + grp]))));
      uint32_t h[2][4];
      kv4_decode8<KIND>(codes.x, s, h[0]);
      kv4_decode8<KIND>(codes.y, s, h[1]);
      float y[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&h[j / 4][j % 4]));
        y[8 * (j / 4) + kv4_low<KIND>(j % 4)] = c.x * g;
        y[8 * (j / 4) + kv4_high<KIND>(j % 4)] = c.y * g;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (p.fp16) {
          const __half2 v = __floats2half2_rn(y[2 * j], y[2 * j + 1]);
          out[j] = *reinterpret_cast<const uint32_t*>(&v);
        } else {
          const __nv_bfloat162 v = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
          out[j] = *reinterpret_cast<const uint32_t*>(&v);
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
}

// ------------------------------------------------------------------ block tables
//
// need_b = ceil((ctx + new) / S) - ceil(ctx / S) blocks for request b (none
// if it would not fit its table), taken in request order from the end of the
// free list: block i of request b is free[count - 1 - before_b - i], before_b
// the sum of the needs in front of it.  A request is admitted if it fits its
// table and the packed tokens, and needs nothing or before_b + need_b <= count.
//
// Every thread block makes the two prefix sums (new tokens, needs; one scan
// of 64-bit pairs) over all requests for itself, in shared memory, and then
// places its own share of the packed tokens: a token's request is found by
// bisection, and a token of a new block names that block without reading the
// table, so that nothing waits for another thread block and one launch does.
// A chain of latencies (lengths, scans, free ids): 8 us between events for 8 requests, 10
// for 1000 with 39000 new tokens.

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
    const int start = static_cast<int>(run & 0xffffffffu);
    // its tokens past the packed arrays would leave blocks without an entry
    const bool packed = add == 0 || start + add <= p.tokens;
    const bool ok = fits && packed && (need == 0 || static_cast<unsigned long long>(before) + need <= static_cast<unsigned>(count));
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

namespace {

template <int KIND, int D>
cudaError_t launch_cache_t(const Kv4CacheArgs& a, bool write, cudaStream_t stream) {
  const int per_token = 2 * a.heads * (D / kKv4Group);
  const dim3 block(std::min(per_token, kCacheThreads), std::max(1, kCacheThreads / per_token));
  const unsigned grid = static_cast<unsigned>((a.tokens + block.y - 1) / block.y);
  if (write) kv4_write_kernel<KIND, D><<<grid, block, 0, stream>>>(a);
  else kv4_read_kernel<KIND, D><<<grid, block, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_cache(const Kv4CacheArgs& args, bool write, cudaStream_t stream) {
  Kv4CacheArgs a = args;
  a.block_shift = -1;
  for (int i = 0; i < 31; ++i)
    if ((1 << i) == a.block_size) a.block_shift = i;
  if (a.head_dim == 64)
    return a.kind == W8A8_KV4_E2M1 ? launch_cache_t<W8A8_KV4_E2M1, 64>(a, write, stream)
                                   : launch_cache_t<W8A8_KV4_INT4, 64>(a, write, stream);
  return a.kind == W8A8_KV4_E2M1 ? launch_cache_t<W8A8_KV4_E2M1, 128>(a, write, stream)
                                 : launch_cache_t<W8A8_KV4_INT4, 128>(a, write, stream);
}

cudaError_t launch_block_tables(const BlockTableArgs& a, int num_sms, cudaStream_t stream) {
  const int smem = static_cast<int>((2LL * a.batch + 1) * sizeof(int));
  // the attribute belongs to the function, for all host threads: always the
  // largest batch's, so that no thread lowers it in front of another's launch
  constexpr int kMost = static_cast<int>((2LL * kMaxTableBatch + 1) * sizeof(int));
  cudaError_t e = cudaFuncSetAttribute(block_table_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  if (e != cudaSuccess) return e;
  long long grid = (a.tokens + kTableThreads - 1) / kTableThreads;
  if (grid > 2LL * num_sms) grid = 2LL * num_sms;
  if (grid < 1) grid = 1;
  block_table_kernel<<<static_cast<unsigned>(grid), kTableThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace w8a8
