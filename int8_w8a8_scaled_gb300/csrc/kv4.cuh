// kv4.cuh -- the 4-bit KV cache: its layout, and the arithmetic of its codes.
//
// A cache is [num_blocks, num_kv_heads, block_size / 16] records of 16
// tokens, 18 * head_dim bytes each:
//   key codes    16 rows of head_dim / 2 bytes (two codes a byte, even dim low)
//   key scales   16 rows of head_dim / 16 bytes (one e4m3 scale for 16 dims)
//   value codes, value scales   the same
// One block and head's records are consecutive, so that any run of records is
// one untiled bulk copy, whose offsets are multiples of 16 bytes.
//
// An element stands for code * group scale * g, with g the tensor's fp32
// scale, one for K and one for V.  Codes are e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6
// and their negatives) or int4 (two's complement, -7..7).  code * group scale
// has at most 3 + 4 significant bits and lies in [2^-10, 7 * 448]: an exact
// f16 number, so a matrix product over f16 operands sees the cache without
// a rounding, and g is applied in fp32 to its result.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace w8a8 {
namespace {  // each translation unit keeps its own copy

constexpr int kKv4Tokens = 16;  // tokens of a record
constexpr int kKv4Group = 16;   // dims that share a scale

// Byte offsets within a record.
__host__ __device__ constexpr int kv4_record_bytes(int d) { return 18 * d; }
__host__ __device__ constexpr int kv4_codes_at(int d, int which) { return which ? 9 * d : 0; }
__host__ __device__ constexpr int kv4_scales_at(int d, int which) { return which ? 17 * d : 8 * d; }

// The record of token `off` of a block, for one head.
__device__ __forceinline__ size_t kv4_record_of(long long block, int head, int heads, int block_size, int off) {
  return (static_cast<size_t>(block) * heads + head) * (block_size / kKv4Tokens) + off / kKv4Tokens;
}

__host__ __device__ constexpr float kv4_largest(int kind) { return kind == W8A8_KV4_E2M1 ? 6.f : 7.f; }

// A pair of group scales as kv4_decode8 takes them: the scales, and for int4
// also -72 times them (4 + 4 significant bits: exact).
struct Kv4Scale {
  __half2 s, bias;
};
template <int KIND>
__device__ __forceinline__ Kv4Scale kv4_scale(__half2 s) {
  return {s, KIND == W8A8_KV4_INT4 ? __hmul2(s, __float2half2_rn(-72.f)) : s};
}

// (x & mask) ^ flip in one instruction (two immediates would make it two).
__device__ __forceinline__ uint32_t and_xor(uint32_t x, uint32_t mask, uint32_t flip) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(y) : "r"(x), "r"(mask), "r"(flip));
  return y;
}

// Where the two codes of f16x2 value i of a decoded word sit in it.  An e2m1
// conversion takes a byte; int4's arithmetic takes nibbles 16 bits apart.
template <int KIND>
__host__ __device__ constexpr int kv4_low(int i) {
  return KIND == W8A8_KV4_E2M1 ? 2 * i : i;
}
template <int KIND>
__host__ __device__ constexpr int kv4_high(int i) {
  return KIND == W8A8_KV4_E2M1 ? 2 * i + 1 : i + 4;
}

// The 8 codes of a word times a pair of scales, as 4 f16x2 values: h[i] =
// (code kv4_low(i) * low scale, code kv4_high(i) * high scale), exactly.
// Four conversions and four products for e2m1; for int4 three shifts, four
// logical operations and four FMAs.
template <int KIND>
__device__ __forceinline__ void kv4_decode8(uint32_t w, const Kv4Scale& sc, uint32_t (&h)[4]) {
  if (KIND == W8A8_KV4_E2M1) {
    uint32_t c[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&c[i]), sc.s);
      h[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  } else {
    // a nibble n in bits 4..7 of the f16 64 (whose steps are 1/16 there), its
    // sign bit flipped, is 72 + n; s (72 + n) - 72 s is one exact FMA
    const uint32_t at[4] = {w << 4, w, w >> 4, w >> 8};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = and_xor(at[i], 0x00F000F0u, 0x54805480u);
      const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&r), sc.s, sc.bias);
      h[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
}

// A word for kv4_decode8 whose value i pairs code 4 q + i of `a` (low) with
// the same of `b`, q = 0 or 1; for e2m1 the codes come in the order kv4_pair_dim.
template <int KIND>
__device__ __forceinline__ uint32_t kv4_interleave(uint32_t a, uint32_t b, int q) {
  if (KIND == W8A8_KV4_E2M1) {
    constexpr uint32_t kLow = 0x0F0F0F0Fu;
    return q == 0 ? (a & kLow) | ((b << 4) & ~kLow) : ((a >> 4) & kLow) | (b & ~kLow);
  }
  return __byte_perm(a, b, q == 0 ? 0x5410 : 0x7632);
}
// The code (of 8) that value i of kv4_interleave(.., q) holds.
template <int KIND>
__host__ __device__ constexpr int kv4_pair_dim(int q, int i) {
  return KIND == W8A8_KV4_E2M1 ? 2 * i + q : 4 * q + i;
}

// The factor of the outputs: v_scale, or NaN where the scores' scale is one (their
// own arithmetic takes it for a small number, to keep a masked score's infinity).
__device__ __forceinline__ float kv4_out_scale(float sm_scale, const float* k_scale, const float* v_scale) {
  const float s = sm_scale * __ldg(k_scale);
  return s == s ? __ldg(v_scale) : s;
}

// Two e4m3 bytes as f16x2.
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return *reinterpret_cast<const __half2*>(&h);
}

__device__ __forceinline__ float e4m3_to_float(uint8_t s) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(s)));
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace
}  // namespace w8a8
