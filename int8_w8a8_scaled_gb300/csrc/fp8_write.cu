// fp8_write.cu -- queries and keys rotated by their positions, keys and values
// into the paged fp8 cache (sm_103a).
//
// Pair i of a head, (x, y), turns by the angle whose cosine and sine stand in
// row position of a table: (x cos - y sin, y cos + x sin), each product and
// sum rounded to fp32.  The keys' rotated values go to e4m3 without another
// rounding between, by the quantiser's own division (quant_math.cuh).
//
// Bound by its bytes: queries in and out, keys and values in and as codes.
// One thread takes 16 elements of a head (8 pairs, or 16 values), by vectors
// of 16 bytes; a CTA takes heads of one token, so that a thread meets the same
// pairs in each of its heads and loads their angles once.  With few tokens the
// heads of one go to several CTAs, a unit to a thread; with many a thread has
// kBatch units' loads in flight and the next token's position and slot.
// Measured: 16384 tokens, 32 query and 8 KV heads of 128: 72.5 us, 5.2 TB/s, 77 % of what
// a copy reaches (a CTA for each token, without looking ahead: 85); 64 tokens: 3.2 us.  The
// form for any alignment and rot_dim, two bytes at a time: 255 us (rot_dim 120).
#include <algorithm>

#include "fp8_paged.cuh"
#include "quant_math.cuh"

namespace w8a8 {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, int fp16, float (&x)[16]) {
  const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = fp8_to_float2(u[i], fp16);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ int axis_of(const Fp8WriteArgs& a, int pair) {
  int axis = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i) axis += i + 1 < a.axes && pair >= a.section_end[i];
  return axis;
}

// cos and sin of one pair of a token, NaN for a position outside the table.
__device__ __forceinline__ void angle_of(const Fp8WriteArgs& a, long long token, int pair, float& c, float& s) {
  const int pos = __ldg(a.positions + axis_of(a, pair) * a.tokens + token);
  c = s = __int_as_float(0x7fffffff);
  if (pos >= 0 && pos < a.max_position) {
    const float* row = a.cos_sin + static_cast<long long>(pos) * a.rot_dim + pair;
    c = __ldg(row);
    s = __ldg(row + a.rot_dim / 2);
  }
}

__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float u = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  x = u;
}

// What a head of a token is: its kind, its input and where it goes.
struct Head {
  int kind;  // 0 query, 1 key, 2 value, 3 none
  const uint16_t* src;
  void* dst;
};

__device__ __forceinline__ Head head_of(const Fp8WriteArgs& a, long long token, long long slot, int head) {
  Head r;
  r.kind = 3;
  r.src = nullptr;
  r.dst = nullptr;
  if (head < a.num_q_heads) {
    r.kind = 0;
    r.src = static_cast<const uint16_t*>(a.q) + token * a.q_token_stride + head * a.q_head_stride;
    r.dst = static_cast<uint16_t*>(a.q_out) + token * a.q_out_token_stride + head * a.q_out_head_stride;
    return r;
  }
  const int h = head - a.num_q_heads;
  if (h >= 2 * a.num_kv_heads || slot < 0 || slot >= a.cache_rows) return r;
  const bool value = h >= a.num_kv_heads;
  const int kv = value ? h - a.num_kv_heads : h;
  r.kind = value ? 2 : 1;
  r.src = value ? static_cast<const uint16_t*>(a.v) + token * a.v_token_stride + kv * a.v_head_stride
                : static_cast<const uint16_t*>(a.k) + token * a.k_token_stride + kv * a.k_head_stride;
  r.dst = static_cast<uint8_t*>(value ? a.v_cache : a.k_cache) + (slot * a.num_kv_heads + kv) * a.head_dim;
  return r;
}

// kBatch: units a thread loads before it works on them.
template <int D, bool kInterleaved, int kBatch>
__global__ void __launch_bounds__(kThreads, kBatch > 1 ? 5 : 1) fp8_rotate_write_kernel(const Fp8WriteArgs a, int heads_per_cta) {
  constexpr int kUnits = D / 16;              // of a head
  constexpr int kAtOnce = kThreads / kUnits;  // heads
  fp8_let_dependents_start();
  fp8_wait_for_predecessor();
  const int unit = threadIdx.x % kUnits, mine = threadIdx.x / kUnits;
  const int all = a.num_q_heads + 2 * a.num_kv_heads;
  const int first = blockIdx.y * heads_per_cta, end = min(all, first + heads_per_cta);

  // the unit's elements: 8 at `lo` and 8 at `hi`
  const bool rotated = unit < a.rot_dim / 16;
  const int lo = kInterleaved || !rotated ? 16 * unit : 8 * unit;
  const int hi = kInterleaved || !rotated ? lo + 8 : a.rot_dim / 2 + lo;
  float scale[2], inv[2];
  bool fine[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    scale[i] = __ldg(i ? a.v_scale : a.k_scale);
    fine[i] = recip_ok(scale[i], &inv[i]);
  }

  // the token after this one has its position and slot looked up meanwhile: they stand in
  // front of its angles and of where it goes
  long long next_slot = __ldg(a.slots + blockIdx.x);
  int next_pos = a.axes == 1 ? __ldg(a.positions + blockIdx.x) : 0;
#pragma unroll 1
  for (long long token = blockIdx.x; token < a.tokens; token += gridDim.x) {
    const long long slot = next_slot;
    const int this_pos = next_pos;
    if (token + gridDim.x < a.tokens) {
      next_slot = __ldg(a.slots + token + gridDim.x);
      if (a.axes == 1) next_pos = __ldg(a.positions + token + gridDim.x);
    }
    // angles of its pairs, which are 8 * unit + 0..7 either way
    float c[8], s[8];
    if (rotated && first < a.num_q_heads + a.num_kv_heads) {
      if (a.axes == 1) {
        const int pos = this_pos;
        if (pos >= 0 && pos < a.max_position) {
          const float* row = a.cos_sin + static_cast<long long>(pos) * a.rot_dim + 8 * unit;
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(row + i));
            const float4 y = __ldg(reinterpret_cast<const float4*>(row + a.rot_dim / 2 + i));
            c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
            s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) c[i] = s[i] = __int_as_float(0x7fffffff);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) angle_of(a, token, 8 * unit + i, c[i], s[i]);
      }
    }
#pragma unroll 1
    for (int h0 = first + mine; h0 < end; h0 += kBatch * kAtOnce) {
      Head head[kBatch];
      uint4 w[kBatch][2];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + i * kAtOnce;
        head[i] = head_of(a, token, slot, h < end ? h : all);
        if (head[i].kind != 3) {
          w[i][0] = *reinterpret_cast<const uint4*>(head[i].src + lo);  // (q may be written in place)
          w[i][1] = *reinterpret_cast<const uint4*>(head[i].src + hi);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (head[i].kind == 3) continue;
        float x[16];
        unpack16(w[i][0], w[i][1], a.fp16, x);
        if (rotated && head[i].kind != 2) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (kInterleaved) turn(x[2 * j], x[2 * j + 1], c[j], s[j]);
            else turn(x[j], x[8 + j], c[j], s[j]);
          }
        }
        if (head[i].kind == 0) {
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = fp8_pack2(x[2 * j], x[2 * j + 1], a.fp16);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(head[i].dst) + lo) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(head[i].dst) + hi) = make_uint4(o[4], o[5], o[6], o[7]);
        } else {
          const int v = head[i].kind - 1;
          const uint4 q = v ? quant16<0>(x, scale[1], inv[1], fine[1], false) : quant16<0>(x, scale[0], inv[0], fine[0], false);
          uint8_t* dst = static_cast<uint8_t*>(head[i].dst);
          if (hi == lo + 8) {
            *reinterpret_cast<uint4*>(dst + lo) = q;
          } else {
            *reinterpret_cast<uint2*>(dst + lo) = make_uint2(q.x, q.y);
            *reinterpret_cast<uint2*>(dst + hi) = make_uint2(q.z, q.w);
          }
        }
      }
    }
  }
}

// Any alignment and rot_dim: a thread takes two elements, a pair or two behind
// the rotated ones.
__global__ void __launch_bounds__(kThreads) fp8_rotate_write_any_kernel(const Fp8WriteArgs a) {
  fp8_let_dependents_start();
  fp8_wait_for_predecessor();
  const long long token = blockIdx.x;
  const int pairs = a.head_dim / 2, all = a.num_q_heads + 2 * a.num_kv_heads;
  const long long slot = __ldg(a.slots + token);
  const float ks = __ldg(a.k_scale), vs = __ldg(a.v_scale);
  for (int item = threadIdx.x; item < all * pairs; item += kThreads) {
    const Head head = head_of(a, token, slot, item / pairs);
    if (head.kind == 3) continue;
    const int pair = item % pairs;
    const bool rotated = pair < a.rot_dim / 2;
    const int lo = rotated && !a.interleaved ? pair : 2 * pair;
    const int hi = rotated && !a.interleaved ? a.rot_dim / 2 + pair : lo + 1;
    const float2 f = fp8_to_float2(static_cast<uint32_t>(head.src[lo]) | (static_cast<uint32_t>(head.src[hi]) << 16), a.fp16);
    float x = f.x, y = f.y;
    if (rotated && head.kind != 2) {
      float c, s;
      angle_of(a, token, pair, c, s);
      turn(x, y, c, s);
    }
    if (head.kind == 0) {
      const uint32_t o = fp8_pack2(x, y, a.fp16);
      static_cast<uint16_t*>(head.dst)[lo] = static_cast<uint16_t>(o);
      static_cast<uint16_t*>(head.dst)[hi] = static_cast<uint16_t>(o >> 16);
    } else {
      const float scale = head.kind == 1 ? ks : vs;
      static_cast<uint8_t*>(head.dst)[lo] = enc1<0>(__fdiv_rn(x, scale));
      static_cast<uint8_t*>(head.dst)[hi] = enc1<0>(__fdiv_rn(y, scale));
    }
  }
}

template <int D, bool kInterleaved>
cudaError_t launch_t(const Fp8WriteArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int kAtOnce = kThreads / (D / 16);
  const int all = a.num_q_heads + 2 * a.num_kv_heads, turns = (all + kAtOnce - 1) / kAtOnce;
  const dim3 block(kThreads);
  const unsigned tokens = static_cast<unsigned>(a.tokens);
  // one unit to a thread while that leaves the CTAs below 16 an SM, all resident
  if (a.tokens * turns <= 16LL * num_sms)
    return fp8_launch(fp8_rotate_write_kernel<D, kInterleaved, 1>, dim3(tokens, turns), block, 0, stream, a, kAtOnce);
  // a resident grid (5 CTAs of 96 registers an SM) goes over the tokens
  return fp8_launch(fp8_rotate_write_kernel<D, kInterleaved, 3>, dim3(std::min(tokens, 5u * num_sms)), block, 0, stream, a, all);
}

}  // namespace

cudaError_t launch_fp8_rotate_write(const Fp8WriteArgs& a, int num_sms, cudaStream_t stream) {
  if (!a.vec)
    return fp8_launch(fp8_rotate_write_any_kernel, dim3(static_cast<unsigned>(a.tokens)), dim3(kThreads), 0, stream, a);
  if (a.head_dim == 64) return a.interleaved ? launch_t<64, true>(a, num_sms, stream) : launch_t<64, false>(a, num_sms, stream);
  return a.interleaved ? launch_t<128, true>(a, num_sms, stream) : launch_t<128, false>(a, num_sms, stream);
}

}  // namespace w8a8
