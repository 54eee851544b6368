// fp8_rows.cu -- attention over the paged fp8 cache for few rows: single tokens,
// drafts, and every token of a sparse selection (sm_103a).
//
// The rows of a unit (a request or a token, a KV head, up to R of its tokens
// times query heads) are the N of both products, the cache their M, straight
// from its e4m3 codes:
//   S^T[128 tokens x N] = K[128 x D] . Q^T       O^T[D x N] += V^T[D x 128] . P^T
// by tcgen05 kind::f8f6f4 with fp32 sums in TMEM.  No code is decoded: tiles of
// 128 tokens go from HBM to the tensor cores by TMA, V as it lies (dims
// contiguous, so V^T is an operand with M contiguous).  What is not e4m3 is
// made of several e4m3 numbers, which cost columns of N only:
//   a query element is q 2^e = a + b 2^-4 + c 2^-8, with e such that the row's
//     largest element lies in [2^7, 2^8): exact for bf16 and fp16 (4 bits a
//     part) down to 2^-13 of that element, rounded at 2^-24 of it below;
//   a weight is f16(2^(s - m + 6)) = a + b 2^-4 + c 2^-8 + d 2^-12, exact (11
//     bits) for weights above 2^-17 of the largest, rounded at 2^-28 below (the last
//     part's steps are 2^-21, an f16's 2^-21 from 2^-11 on); the
//     sum that divides is of the weights before that rounding.
// The maximum m is raised, and O rescaled, only when a score passes it by 2^2.
//
// Bound by the cache's bytes, 2 D a token: the MMAs of a tile take about half of
// the time that HBM needs for it, and its softmax (128 tokens x R rows) less.
//
// One CTA to an SM, 12 warps: one copies tiles ahead into a ring, one prepares the next
// unit's query (the first one's all softmax warps: by one warp it was 5 us) and with 8
// rows takes over the copies of V, and two groups of four warps take the tiles in
// turn, each with scores, weights and sums O of its own, joined at the unit's end, and
// each with a warp that issues its MMAs (one for both spent 1300 cycles a tile on waits
// that were over and on issuing, more than HBM's time for it).  A thread is a token: the
// weights of a token need nothing of another but the maximum, which all agree on by
// one vote.
//
// All units' tiles in a row are cut into equal runs, one for each CTA, so that ragged
// lengths load the SMs evenly (CTAs side by side take neighbouring KV heads of the same
// tokens: a head's rows are 128-byte pieces of the cache's); a cut unit leaves a part
// in the workspace from each of its CTAs, joined by the last to arrive, in their
// order: results do not depend on timing.
//
// Measured (calls in a row in a graph): 64 requests up to 8192 tokens, 8 KV
// heads of 128, 4 query heads each: 121 us, 5.3 TB/s, 79 % of what a copy reaches (128
// requests: 214 us, 5.6 TB/s); blocks of 16 in place of 64: 135 (four times the copies);
// heads of 64: 101; 16 / 32 query heads: 173 / 283; one request of 2003 tokens: 16, of
// which about 2 us each go to the launch, the first copies, the first tile, the unit's end
// and the joining.  On the way there: one MMA warp for both groups 166 us; K and V fetched
// together 166, apart 136; the query's rows loaded one after another by one warp 5 us at
// the start.
//
// Weights of 0 do not cancel a NaN code, so the rows of V that no row of the unit
// sees are cleared in shared memory before the product, and NaN codes of tokens
// that only some rows see are taken out and put into those rows' results.
#include <algorithm>

#include "fp8_paged.cuh"
#include "sm103_ptx.cuh"

namespace w8a8 {

namespace {

constexpr int kTile = 128;                    // tokens
constexpr int kGroupThreads = 128;            // a softmax group
constexpr int kCopyWarp = 8, kMmaWarp = 9, kQueryWarp = 11;
constexpr int kThreads = 32 * (kQueryWarp + 1);
constexpr int kQueryArrivals = 8;             // the first query is made by the softmax warps
constexpr float kHeadroom = 2.f;
constexpr float kNoScore = -1e25f;
// Tiles whose places are kept: keys are sent for at most half as many tiles ahead of the
// values, and values at most a ring (8 tiles) ahead of the products, which come after
// the places have been read.
constexpr int kPlaces = 32;
constexpr int kDead = kFp8MostTokens;         // the position of a token that is not there
constexpr size_t kSmemMost = 227 * 1024;

template <int D, int R>
struct Few {
  static constexpr int kQParts = 3, kPParts = 4;
  static constexpr int kNS = (kQParts * R + 15) / 16 * 16;  // columns of the scores (M = 128: a multiple of 16)
  static constexpr int kNP = kPParts * R;                   // columns of the output
  static constexpr int kHalf = kTile * D;                   // K or V of a tile
  static constexpr int kQ = kNS * D, kP = kNP * kTile, kDump = R * D * 4, kRawQ = R * D * 2;
  static constexpr int kFixed = 2 * kQ + 2 * kP + kDump + kRawQ + 1024;  // + alignment
  static constexpr int kStatic = 8 * 1024;                  // room for the kernel's static shared memory
  static constexpr int kFit = static_cast<int>((kSmemMost - kStatic - kFixed) / (2 * kHalf));
  // even, and the groups take every second tile of the run, so that the tile before in a
  // stage was the same group's: no wait for a stage can mistake another phase for its own
  static constexpr int kStages = kFit > 8 ? 8 : kFit / 2 * 2;
  static_assert(kStages >= 4, "the ring holds two tiles of each group");
  static constexpr int kSmem = kStages * 2 * kHalf + kFixed;
  static constexpr uint32_t kCols = 2 * (kNS + kNP);
  static constexpr uint32_t kTmem = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512, "scores and outputs of both groups fit TMEM");
  static constexpr int kPart = R * (D + 2);                 // floats: o [R][D], m [R], l [R]
  // V by a warp of its own, the query's: one warp's copies do not keep up with HBM (64
  // single tokens, 8 rows: 116 us for 126).  With more rows a tile's softmax takes longer
  // than that, the query too, and V would wait for it (32 x 5 drafts: 97 us for 80)
  static constexpr bool kSplit = R == 8;
};

__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

// Two f16 numbers to e4m3 codes (the low one in the low byte), and back.
__device__ __forceinline__ uint32_t to_e4m3x2(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
__device__ __forceinline__ uint32_t from_e4m3x2(uint32_t codes) {
  uint32_t r;
  const uint16_t c = static_cast<uint16_t>(codes);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

// Parts of two f16 numbers of at most 448: x = p0 + p1 2^-4 + p2 2^-8 ...; what
// a part leaves over is at most 2^-4 of a power of two above it, and exact.
template <int N>
__device__ __forceinline__ void parts_of(uint32_t x, uint32_t (&part)[N]) {
  const __half2 up = __float2half2_rn(16.f), down = __float2half2_rn(-16.f);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    part[i] = to_e4m3x2(x);
    if (i + 1 < N) x = as_u32(__hfma2(as_half2(from_e4m3x2(part[i])), down, __hmul2(as_half2(x), up)));
  }
}

__device__ __forceinline__ void mma_f8_by(uint32_t leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
}

// The largest of a warp's numbers (NaN has no part in it).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Descriptor of an operand tile of ROW-byte rows (32, 64 or 128) with the swizzle of
// that width, in atoms of 8 rows.  With M or N contiguous a row is one K index, and
// the next ROW elements of M or N are `next` bytes on.
template <int ROW>
__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr, uint32_t next) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((next >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((8u * ROW) >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(ROW == 128 ? 2u : ROW == 64 ? 4u : 6u) << 61;
  return d;
}

// Where the 16-byte chunk `chunk` of row `row` lies in such a tile.
template <int ROW>
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
  const int turn = ROW == 128 ? row & 7 : ROW == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
  return static_cast<uint32_t>(row * ROW + ((chunk ^ turn) << 4));
}

__device__ __forceinline__ bool mbar_is_over(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Whether a phase is over, for every lane.
__device__ __forceinline__ bool warp_over(uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_is_over(bar, parity)); }
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity)); }

// Whether a warp that polls several barriers may go on: bounded like every wait, from
// the first look that found nothing.  The timer is read now and then.
struct Patience {
  uint64_t since = 0;
  uint32_t looks = 0;
  __device__ __forceinline__ void again() { looks = 0; }
  __device__ __forceinline__ bool left() {
    if (++looks & 255u) return true;
    const uint64_t now = global_timer_ns();
    if (looks == 256u) since = now;
    if (!__any_sync(0xffffffffu, now - since > W8A8_WAIT_NS)) return true;
    if (threadIdx.x % 32 == 0) atomicOr(&g_device_status, 1);
    return false;
  }
};

// A count that one warp raises and another follows.
__device__ __forceinline__ void publish(int* to, int x) {
  asm volatile("st.release.cta.shared.u32 [%0], %1;" ::"r"(smem_addr(to)), "r"(x) : "memory");
}
__device__ __forceinline__ int follow(const int* from) {
  int x;
  asm volatile("ld.acquire.cta.shared.u32 %0, [%1];" : "=r"(x) : "r"(smem_addr(from)) : "memory");
  return __shfl_sync(0xffffffffu, x, 0);
}

__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ void mbar_arrive_many(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

// Named barriers: 1 + g a group's own; 3 group 1's state is there, 4 it has been read.
__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kGroupThreads) : "memory"); }
__device__ __forceinline__ bool group_any(int group, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(1 + group), "n"(kGroupThreads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void both_sync(int id) { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(2 * kGroupThreads) : "memory"); }
__device__ __forceinline__ void both_arrive(int id) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(2 * kGroupThreads) : "memory"); }

// ------------------------------------------------------------------ units

// A unit: rows over the same tokens.  Dense: one request, KV head and R of its
// rows (row r: token r / share, head r % share).  Sparse: one token, KV head and R
// of its heads; its tokens are those of the selected columns, in their order.
struct Unit {
  int b;               // request, -1: a row of q that belongs to none
  int first;           // first row of q of the request (sparse: the token's row)
  int kvh, row0, rows; // rows of the unit: row0 .. row0 + rows - 1
  int base;            // position of the request's new token 0 (sparse: the token's position)
  int len;             // tokens of the request
  int tiles;
};

// A place in the row of all units' tiles.
template <int R, bool SPARSE>
struct Cursor {
  Unit u;
  int lane;                 // the CTA's place among those that go side by side over the KV heads
  int group, groups, tile;  // row group of the unit, groups of the request; next tile
  int token;                // sparse: the row of q

  // Sparse: the request of `token`, looked for from request `from` on where starts rise;
  // where they do not (a batch padded by zeros), among all of them, as the selection does.
  __device__ __forceinline__ void find(const Fp8AttnParams& p, int from) {
    const Fp8Paged& c = p.c;
    u.b = u.base = -1;
    u.len = 0;
    // (one loop for both: it is inlined where the tiles are counted, and the code of those
    // loops has to stay in the instruction cache)
#pragma unroll 1
    for (int b = falls ? 0 : from; b < c.batch; ++b) {
      const Fp8Request r = fp8_request(c, b);
      const int row = token - r.first;
      if (row < 0 && !falls) break;
      seen = b;
      if (row < 0 || row >= (falls ? r.n : r.all)) continue;
      if (row < r.n) {
        u.b = b;
        u.len = r.len;
        u.base = r.len - r.all + row;
      }
      return;
    }
  }
  int seen;                 // sparse: requests in front of this one end before `token`
  bool falls;               // sparse: some start is below the one in front of it

  __device__ __forceinline__ void dense(const Fp8AttnParams& p, int b) {
    const Fp8Request r = fp8_request(p.c, b);
    u.b = b;
    u.first = r.first;
    u.len = r.len;
    u.base = r.len - r.all;
    rows_all = r.n * p.share;
    groups = tiles_of(p, r) == 0 ? 0 : (rows_all + R - 1) / R;
    u.tiles = tiles_of(p, r);
  }
  int rows_all;

  // Tiles of each of a request's units, 0 if it is not this kernel's.
  static __device__ __forceinline__ int tiles_of(const Fp8AttnParams& p, const Fp8Request& r) {
    const int rows = r.n * p.share;
    if (rows == 0 || rows > p.few_rows) return 0;
    return max(1, (r.len + kTile - 1) / kTile);
  }

  __device__ __forceinline__ void set_rows(const Fp8AttnParams& p) {
    u.row0 = group * R;
    u.rows = min(R, (SPARSE ? p.share : rows_all) - u.row0);
  }

  __device__ __forceinline__ void next_unit(const Fp8AttnParams& p) {
    tile = 0;
    if (++group < groups) {
      set_rows(p);
      return;
    }
    group = 0;
    u.kvh += p.side;
    if (u.kvh >= p.c.num_kv_heads) {
      u.kvh = lane;
      if (SPARSE) {
        u.first = ++token;
        find(p, seen);
      } else {
        int b = u.b;
        do dense(p, ++b);
        while (groups == 0);
      }
    }
    set_rows(p);
  }
};

// A unit that goes on in other CTAs.
struct Open {
  int b, first, rows, row0, kvh;
  long long unit;  // its first tile; -1: none
  int tiles;
};

__device__ __forceinline__ size_t out_at(const Fp8AttnParams& p, bool sparse, int first, int kvh, int row) {
  const int token = sparse ? first : first + row / p.share, head = kvh * p.share + (sparse ? row : row % p.share);
  return token * p.out_token_stride + head * p.out_head_stride;
}

__device__ __forceinline__ void store1(const Fp8AttnParams& p, size_t at, float y) {
  if (p.out_fp16) static_cast<__half*>(p.out)[at] = __float2half_rn(y);
  else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
}

// The query of a unit as the scores' N operand, its rows' factors and limits: rows w,
// w + warps, ... by this warp, converted a row at a time (a rolled loop: code that
// runs once is paid for in instruction fetches).
template <int D, int R, bool SPARSE>
__device__ __forceinline__ void write_query(const Fp8AttnParams& p, const Unit& u, uint8_t* rows, uint8_t* dst, float* cs,
                                            int* lim, int* limits, int w, int warps) {
  using C = Few<D, R>;
  constexpr int kPer = D / 32;  // elements of a lane
  const int lane = threadIdx.x % 32;
  const float to_log2 = p.sm_scale * __ldg(p.k_scale) * kFp8Log2e;
  // the rows as they are first, many loads in flight: with the cache streaming a load
  // takes 2 us, and row after row a unit's query took longer than the unit
  constexpr int kPerRow = D / 8, kBatch = 8;
  const int pieces = (R - w + warps - 1) / warps * kPerRow;
#pragma unroll 1
  for (int i0 = lane; i0 < pieces; i0 += 32 * kBatch) {
    uint4 x[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + 32 * k, r = w + i / kPerRow * warps;
      x[k] = make_uint4(0u, 0u, 0u, 0u);
      if (i >= pieces || r >= u.rows || u.b < 0) continue;
      const int row = u.row0 + r, token = SPARSE ? u.first : u.first + row / p.share;
      const int head = u.kvh * p.share + (SPARSE ? row : row % p.share);
      x[k] = fp8_load8(static_cast<const uint16_t*>(p.q) + token * p.q_token_stride + head * p.q_head_stride + 8 * (i % kPerRow),
                       p.q_vec);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + 32 * k, r = w + i / kPerRow * warps;
      if (i < pieces) reinterpret_cast<uint4*>(rows)[r * kPerRow + i % kPerRow] = x[k];
    }
  }
  __syncwarp();
#pragma unroll 1
  for (int r = w; r < R; r += warps) {
    uint32_t raw[kPer / 2];
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k) raw[k] = reinterpret_cast<const uint32_t*>(rows)[(r * D + kPer * lane) / 2 + k];
    float x[kPer], top = 0.f;
    bool odd = false;
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k) {
      const float2 f = fp8_to_float2(raw[k], p.q_fp16);
      x[2 * k] = f.x;
      x[2 * k + 1] = f.y;
      top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
      odd = odd || !(fabsf(f.x) < INFINITY) || !(fabsf(f.y) < INFINITY);
    }
    top = warp_max(top);
    odd = __any_sync(0xffffffffu, odd);
    // 2^e brings the largest element into [2^7, 2^8)
    int e = 0;
    if (top > 0.f && !odd) e = min(100, 7 + 127 - static_cast<int>(__float_as_uint(top) >> 23));
    const float down = to_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    // the scale's sign goes to the query: the largest product is the largest score
    const float up = copysignf(__uint_as_float(static_cast<uint32_t>(127 + e) << 23), down);
    if (lane == 0) {
      // a row with a NaN or an infinity, or any row under a NaN scale, has NaN scores
      cs[r] = odd || !(fabsf(down) <= INFINITY) ? __int_as_float(0x7fffffff) : fmaxf(fabsf(down), 1e-37f);
      lim[r] = r < u.rows ? u.base + (SPARSE ? 0 : (u.row0 + r) / p.share) : -1;
    }
    uint32_t code[C::kQParts][kPer / 2];
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k) {
      uint32_t part[C::kQParts];
      parts_of(as_u32(__floats2half2_rn(odd ? 0.f : x[2 * k] * up, odd ? 0.f : x[2 * k + 1] * up)), part);
#pragma unroll
      for (int j = 0; j < C::kQParts; ++j) code[j][k] = part[j];
    }
#pragma unroll
    for (int j = 0; j < C::kQParts; ++j) {
      const int byte = kPer * lane;
      uint8_t* to = dst + chunk_at<D>(j * R + r, byte >> 4) + (byte & 15);
      if (D == 128) *reinterpret_cast<uint32_t*>(to) = code[j][0] | (code[j][kPer / 2 - 1] << 16);
      else *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(code[j][0]);
    }
  }
  // (columns past the last part are not looked at, but are finite)
  for (int i = 32 * w + lane; i < (C::kNS - C::kQParts * R) * D / 4; i += 32 * warps)
    reinterpret_cast<uint32_t*>(dst + C::kQParts * R * D)[i] = 0u;
  if (w == 0 && lane == 0) {
    limits[0] = u.base + (SPARSE ? 0 : u.row0 / p.share);
    limits[1] = SPARSE ? limits[0] : u.base + (u.row0 + u.rows - 1) / p.share;
  }
  fence_proxy_async_shared();
  __syncwarp();
}

template <int D, int R, bool SPARSE>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_rows_kernel(const Fp8AttnParams p, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using C = Few<D, R>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const s_ring = smem;                               // [stage] K, V
  uint8_t* const s_p = smem + C::kStages * 2 * C::kHalf;      // [group] weights
  uint8_t* const s_q = s_p + 2 * C::kP;                       // [2] queries
  float* const s_dump = reinterpret_cast<float*>(s_q + 2 * C::kQ);  // group 1's outputs [R][D]
  uint8_t* const s_rows = reinterpret_cast<uint8_t*>(s_dump) + C::kDump;  // a query as it is given
  __shared__ uint64_t s_kfull[C::kStages], s_vfull[C::kStages], s_kempty[C::kStages], s_vempty[C::kStages];
  __shared__ uint64_t s_qfull[2], s_qempty[2], s_sfull[2], s_sfree[2], s_pfull[2], s_pvdone[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_pos[kPlaces][8], s_row[kPlaces][8];  // of a tile's boxes: positions of the first tokens, rows of the cache
  __shared__ long long s_scan[kThreads / 32], s_before;
  __shared__ int s_item, s_found, s_last[2];
  __shared__ int s_jk, s_jv;                   // tiles whose K has been sent for, whose V has
  __shared__ Open s_open[2];
  __shared__ __align__(16) float s_cs[2][R];   // [query buffer] factor of each row's scores
  __shared__ __align__(16) int s_lim[2][R];    // last position that each row sees
  __shared__ int s_limits[2][2];               // smallest and largest of them
  __shared__ __align__(16) float s_m[2][R];    // [group] maxima
  __shared__ float s_red[2][4][R];             // [group][warp]
  __shared__ __align__(16) float s_alpha[2][R]; // [group] what a raised maximum makes of the sums so far
  __shared__ float s_state[2][2][R];           // [group] m in the log2 domain, l
  __shared__ __align__(16) float s_factor[3][R];  // of a unit's outputs: each group's, the whole's
  __shared__ __align__(16) long long s_to[R];  // where a unit's rows go, -1: nowhere
  __shared__ int s_nan[2][D];                  // [group] first token with a NaN in a dim
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int boxes = kTile / p.box;             // copies of a tile's K (or V)

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(smem_addr(&s_kfull[i]), boxes);
      mbar_init(smem_addr(&s_vfull[i]), boxes);
      mbar_init(smem_addr(&s_kempty[i]), 1);
      mbar_init(smem_addr(&s_vempty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&s_qfull[i]), kQueryArrivals);
      mbar_init(smem_addr(&s_qempty[i]), 10);  // the softmax warps, and the MMA warps, so that none falls a phase behind
      mbar_init(smem_addr(&s_sfull[i]), 1);
      mbar_init(smem_addr(&s_sfree[i]), 4);
      mbar_init(smem_addr(&s_pfull[i]), 4);
      mbar_init(smem_addr(&s_pvdone[i]), 1);
    }
    fence_barrier_init();
  }
  if (tid < 2) s_open[tid].unit = -1;
  if (tid == 0) s_jk = s_jv = 0;
  for (int i = tid; i < 2 * D; i += kThreads) (&s_nan[0][0])[i] = kDead;
  // TMEM only after the wait: a kernel in front may still need it.  Dependents start
  // only when it is taken: one that took it first and then waited for this kernel's
  // end would never see it.
  fp8_wait_for_predecessor();
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&s_tmem), C::kTmem);
    tmem_relinquish();
  }

  // ---- this CTA's run: number `nth` of those of its place `place`, over every side-th
  // KV head from that one on
  const int place = static_cast<int>(blockIdx.x) % p.side, nth = static_cast<int>(blockIdx.x) / p.side;
  const int runs = static_cast<int>(gridDim.x) / p.side;
  long long total = 0, share;
  if constexpr (!SPARSE) {
    const int per = (p.c.batch + kThreads - 1) / kThreads;
    const int b0 = min(p.c.batch, tid * per), b1 = min(p.c.batch, b0 + per);
    auto tiles_of = [&](int b) {
      const Fp8Request r = fp8_request(p.c, b);
      return static_cast<long long>(Cursor<R, SPARSE>::tiles_of(p, r)) * (p.c.num_kv_heads / p.side) * ((r.n * p.share + R - 1) / R);
    };
    long long mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) mine += tiles_of(b);
    long long run = mine;
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, run, off);
      if (lane >= off) run += o;
    }
    if (lane == 31) s_scan[warp] = run;
    __syncthreads();
    run -= mine;
#pragma unroll 1
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) run += s_scan[w];
      total += s_scan[w];
    }
    share = max(1LL, (total + runs - 1) / runs);
    const long long at = share * nth;
    if (at >= run && at < run + mine) {
#pragma unroll 1
      for (int b = b0; b < b1; ++b) {
        const long long w = tiles_of(b);
        if (at < run + w) {
          s_item = b;
          s_before = run;
          break;
        }
        run += w;
      }
    }
  }
  const int sparse_tiles = SPARSE ? static_cast<int>((static_cast<long long>(p.budget) * p.c.block_size + kTile - 1) / kTile) : 0;
  const int sparse_groups = SPARSE ? (p.share + R - 1) / R : 0;
  int sparse_seen = 0;
  bool sparse_falls = false;
  if constexpr (SPARSE) {
    const long long per_token = static_cast<long long>(sparse_tiles) * sparse_groups * (p.c.num_kv_heads / p.side);
    total = per_token * p.c.tokens;
    share = max(1LL, (total + runs - 1) / runs);
    // the request of the run's first token: all threads look at once
    const long long token = share * nth / per_token;
    if (tid == 0) s_found = 0;
    __syncthreads();
    bool fall = false;
    if (p.c.query_start && token < p.c.tokens)
      for (int b = tid; b < p.c.batch; b += kThreads) {
        const int start = __ldg(p.c.query_start + b);
        if (start <= token) atomicMax(&s_found, b);
        fall = fall || __ldg(p.c.query_start + b + 1) < start;
      }
    sparse_falls = __syncthreads_or(fall);
    sparse_seen = p.c.query_start ? s_found : static_cast<int>(min(token, static_cast<long long>(p.c.batch)));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  fp8_let_dependents_start();
  const uint32_t tmem = s_tmem;
  const long long r0 = share * nth;
  const int run_tiles = static_cast<int>(max(0LL, min(total - r0, min(share, 0x7fffffffLL))));
  Cursor<R, SPARSE> at;
  at.u.b = -1;
  at.lane = place;
  at.falls = sparse_falls;
  if (run_tiles > 0) {
    if constexpr (SPARSE) {
      const long long unit = r0 / sparse_tiles;
      at.groups = sparse_groups;
      at.group = static_cast<int>(unit % sparse_groups);
      const int heads = p.c.num_kv_heads / p.side;
      at.u.kvh = place + p.side * static_cast<int>(unit / sparse_groups % heads);
      at.token = at.u.first = static_cast<int>(unit / sparse_groups / heads);
      at.u.tiles = sparse_tiles;
      at.tile = static_cast<int>(r0 % sparse_tiles);
      at.find(p, at.seen = sparse_seen);
    } else {
      at.dense(p, s_item);
      const long long in = r0 - s_before;
      const int unit = static_cast<int>(in / at.u.tiles);
      at.tile = static_cast<int>(in % at.u.tiles);
      at.u.kvh = place + p.side * (unit / at.groups);
      at.group = unit % at.groups;
    }
    at.set_rows(p);
  }
  bool ok = true;

  const uint32_t bytes = static_cast<uint32_t>(p.box * D);  // of a copy
  const uint64_t pol = policy_evict_first();
  int jv = 0;  // the next tile whose V is to go out
  // sends for V of tile jv of the run (`head`) if K's copies have gone out as far, and its
  // place in the ring is free
  auto copy_v = [&](Cursor<R, SPARSE>& head, int sent) -> bool {
    const int stage = jv % C::kStages;
    if (jv >= min(sent, run_tiles)) return false;
    if (jv >= C::kStages && !warp_over(smem_addr(&s_vempty[stage]), ((jv / C::kStages) & 1) ^ 1u)) return false;
    if (lane < boxes) {
      const int row = s_row[jv % kPlaces][lane];
      const uint32_t bar = smem_addr(&s_vfull[stage]);
      fence_proxy_async_shared();  // what was written there by hand before the copy over it
      if (row >= 0) {
        mbar_arrive_expect_tx(bar, bytes);
        tma_load_2d_hint(smem_addr(s_ring) + stage * 2 * C::kHalf + C::kHalf + lane * bytes, &map_v, bar, head.u.kvh * D, row, pol);
      } else {
        mbar_arrive(bar);
      }
    }
    __syncwarp();
    if (++jv < run_tiles && ++head.tile == head.u.tiles) head.next_unit(p);
    return true;
  };
  // a wait gave up: the copies in flight land before shared memory is released
  auto land = [&](uint64_t* full, int sent) {
    for (int i = max(0, sent - C::kStages); i < sent; ++i) mbar_wait(smem_addr(&full[i % C::kStages]), (i / C::kStages) & 1);
  };

  if (run_tiles == 0) {
    // nothing to do
  } else if (warp == kCopyWarp) {
    // ================= copies: lane x has box x of the tile
    const uint32_t ring = smem_addr(s_ring);
    // the place of this lane's box of a tile, a batch of tiles at once
    const int ahead = 32 / boxes;          // tiles of a batch
    Cursor<R, SPARSE> mine = at;           // the tile this lane looks up
    int mine_at = 0;
    int row = -1, pos = kDead;
    auto look_up = [&](int tile_of_run) {
      row = -1;
      pos = kDead;
      if (tile_of_run >= run_tiles) return;
      int left = tile_of_run - mine_at;
      mine_at = tile_of_run;
      while (left > 0) {
        const int step = min(left, mine.u.tiles - mine.tile);
        left -= step;
        mine.tile += step;
        if (mine.tile == mine.u.tiles && left >= 0) mine.next_unit(p);
      }
      if (SPARSE && mine.u.b < 0) return;
      const long long t = static_cast<long long>(mine.tile) * kTile + (lane % boxes) * p.box;
      int col, off;
      if (SPARSE) {
        const int entry = static_cast<int>(t / p.c.block_size);
        off = static_cast<int>(t - static_cast<long long>(entry) * p.c.block_size);
        if (entry >= p.budget) return;
        col = __ldg(p.selected + (static_cast<size_t>(mine.token) * p.c.num_kv_heads + mine.u.kvh) * p.budget + entry);
        if (col < 0 || col >= p.c.max_blocks) return;
        const long long first = static_cast<long long>(col) * p.c.block_size + off;
        if (first > mine.u.base) return;
        pos = static_cast<int>(first);
      } else {
        if (t >= mine.u.len) return;
        col = static_cast<int>(t) / p.c.block_size;
        off = static_cast<int>(t) - col * p.c.block_size;
        pos = static_cast<int>(t);
      }
      const int block = __ldg(p.c.block_table + static_cast<size_t>(mine.u.b) * p.c.max_blocks + col);
      if (block < 0 || block >= p.c.num_blocks) {
        pos = kDead;
        return;
      }
      row = block * p.c.block_size + off;
    };
    // K and V each go out when their place in the ring is free: K's is long before V's
    Cursor<R, SPARSE> khead = at, vhead = at;  // their tiles: the KV heads
    int jk = 0;
    Patience patience;
#pragma unroll 1
    while (jk < run_tiles || (!C::kSplit && jv < run_tiles)) {
      bool moved = false;
      if (jk < run_tiles && jk < (C::kSplit ? follow(&s_jv) : jv) + kPlaces / 2 &&
          (jk < C::kStages || warp_over(smem_addr(&s_kempty[jk % C::kStages]), ((jk / C::kStages) & 1) ^ 1u))) {
        if (jk % ahead == 0) look_up(jk + lane / boxes);
        const int stage = jk % C::kStages, src = (jk % ahead) * boxes;
        const bool turn = lane >= src && lane < src + boxes;
        if (turn) {
          s_pos[jk % kPlaces][lane - src] = pos;
          s_row[jk % kPlaces][lane - src] = row;
        }
        __syncwarp();
        if (C::kSplit && lane == 0) publish(&s_jk, jk + 1);
        if (turn) {
          const uint32_t bar = smem_addr(&s_kfull[stage]);
          if (row >= 0) {
            mbar_arrive_expect_tx(bar, bytes);
            tma_load_2d_hint(ring + stage * 2 * C::kHalf + (lane - src) * bytes, &map_k, bar, khead.u.kvh * D, row, pol);
          } else {
            mbar_arrive(bar);
          }
        }
        if (++jk < run_tiles && ++khead.tile == khead.u.tiles) khead.next_unit(p);
        moved = true;
      }
      if (!C::kSplit) moved |= copy_v(vhead, jk);
      if (moved) patience.again();
      else if (!(ok = patience.left())) break;
    }
    if (!ok) {
      land(s_kfull, jk);
      if (!C::kSplit) land(s_vfull, jv);
    }
  } else if (warp >= kMmaWarp && warp < kQueryWarp) {
    // ================= MMAs, a warp for each group: every second tile of the run
    const int group = warp - kMmaWarp;
    const uint32_t leader = elect_one();
    constexpr uint32_t kIdescS = make_idesc(kTile, C::kNS, 0);
    // V^T and P^T: their tokens are the rows as they lie, M and N contiguous
    constexpr uint32_t kIdescO = make_idesc(128, C::kNP, 0) | (1u << 15) | (1u << 16);
    const uint32_t tm = uniform(tmem);
    const uint32_t ring = smem_addr(s_ring), qbuf = smem_addr(s_q);
    const uint32_t to_s = tm + group * C::kNS, to_o = tm + 2 * C::kNS + group * C::kNP;
    const uint64_t dp = desc_rows<C::kNP>(smem_addr(s_p) + group * C::kP, 16);
    // (heads of 64 fill half of M = 128; the other half reads what lies behind, the next
    // 8 KB, always within the ring or the weights, and is not looked at)
    constexpr uint32_t kNext = C::kHalf;
    const uint32_t sfree = smem_addr(&s_sfree[group]), sfull = smem_addr(&s_sfull[group]);
    const uint32_t pfull = smem_addr(&s_pfull[group]), pvdone = smem_addr(&s_pvdone[group]);
    const int all = uniform(run_tiles);
    uint32_t scount = 0u, pcount = 0u;
    int done = 0, units = 0;
    auto scores = [&](int tile, int q) {
      const int stage = tile % C::kStages;
      tc_fence_after();
      const uint64_t dk = desc_rows<D>(ring + stage * 2 * C::kHalf, 16), dq = desc_rows<D>(qbuf + q * C::kQ, 16);
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) mma_f8_by(leader, to_s, dk + 2 * kk, dq + 2 * kk, kIdescS, kk > 0);
      mma_commit_by(leader, sfull);
      mma_commit_by(leader, smem_addr(&s_kempty[stage]));
      ++scount;
    };
#pragma unroll 1
    while (done < all && ok) {
      const int nt = uniform(min(at.u.tiles - at.tile, all - done));
      const int q = units & 1;
      ok = warp_wait(smem_addr(&s_qfull[q]), (units / 2) & 1);
      tc_fence_after();
      const int j0 = (done ^ group) & 1;
      if (j0 < nt && ok) {
        if (scount > 0) ok = warp_wait(sfree, (scount - 1) & 1);
        ok = ok && warp_wait(smem_addr(&s_kfull[(done + j0) % C::kStages]), ((done + j0) / C::kStages) & 1);
        if (ok) scores(done + j0, q);
      }
#pragma unroll 1
      for (int j = j0; j < nt && ok; j += 2) {
        // the product with these weights, and the next scores as soon as the group has read
        // its own and their keys are there: whichever can go first
        const int stage = (done + j) % C::kStages, next = done + j + 2;
        bool product = true, more = j + 2 < nt;
        if (more) ok = warp_wait(sfree, (scount - 1) & 1);
        Patience patience;
        while ((product || more) && ok) {
          bool moved = false;
          if (more && warp_over(smem_addr(&s_kfull[next % C::kStages]), (next / C::kStages) & 1)) {
            scores(next, q);
            more = false;
            moved = true;
          }
          // (with many rows the softmax takes the time: one look that may sleep, all lanes', and
          // no polling beside it: 82.7 us for 84, 32 requests of 20 rows; 266 for 270, 64 of 32)
          if (product && (R > 8 ? __all_sync(0xffffffffu, mbar_try_wait(pfull, pcount & 1)) : warp_over(pfull, pcount & 1)) &&
              warp_over(smem_addr(&s_vfull[stage]), ((done + j) / C::kStages) & 1)) {
            tc_fence_after();
            const uint64_t dv = desc_rows<D>(ring + stage * 2 * C::kHalf + C::kHalf, kNext);
#pragma unroll
            for (int kk = 0; kk < kTile / 32; ++kk)
              mma_f8_by(leader, to_o, dv + kk * ((32 * D) >> 4), dp + kk * ((32 * C::kNP) >> 4), kIdescO, kk > 0 || j >= 2);
            mma_commit_by(leader, smem_addr(&s_vempty[stage]));
            mma_commit_by(leader, pvdone);
            ++pcount;
            product = false;
            moved = true;
          }
          if (moved) patience.again();
          else ok = patience.left();
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&s_qempty[q]));
      done += nt;
      ++units;
      at.tile += nt;
      if (done < all) at.next_unit(p);
    }
  } else if (warp >= kQueryWarp) {
    // ================= the queries of the units after the first (and copies of V)
    Cursor<R, SPARSE> head = at;
    int done = min(at.u.tiles - at.tile, run_tiles), units = 1;
    at.tile += done;
    if (done < run_tiles) at.next_unit(p);
    Patience patience;
#pragma unroll 1
    while (done < run_tiles || (C::kSplit && jv < run_tiles)) {
      bool moved = false;
      if (C::kSplit && copy_v(head, follow(&s_jk))) {
        if (lane == 0) publish(&s_jv, jv);
        moved = true;
      }
      const int buf = units & 1;
      if (done < run_tiles && (units < 2 || warp_over(smem_addr(&s_qempty[buf]), ((units / 2) & 1) ^ 1u))) {
        write_query<D, R, SPARSE>(p, at.u, s_rows, s_q + buf * C::kQ, s_cs[buf], s_lim[buf], s_limits[buf], 0, 1);
        if (lane == 0) mbar_arrive_many(smem_addr(&s_qfull[buf]), kQueryArrivals);
        const int nt = min(at.u.tiles - at.tile, run_tiles - done);
        done += nt;
        ++units;
        at.tile += nt;
        if (done < run_tiles) at.next_unit(p);
        moved = true;
      }
      if (moved) patience.again();
      else if (!(ok = patience.left())) break;
    }
    if (C::kSplit && !ok) land(s_vfull, jv);
  } else {
    // ================= softmax: thread = token of the tile (in the outputs: dim)
    const int group = warp / 4, quarter = warp % 4, token = 32 * quarter + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter) << 21);
    const uint32_t s_cols = lanes + group * C::kNS, o_cols = lanes + 2 * C::kNS + group * C::kNP;
    uint8_t* const weights = s_p + group * C::kP;  // a row of kNP bytes for each token
    float* const m = s_m[group];
    const float vscale = __ldg(p.v_scale);
    uint32_t count = 0u;  // tiles of this group
    int done = 0, units = 0;
    // nothing to do yet: the first unit's query
    // (by way of the outputs' place: the query warp may be at the second unit's already)
    write_query<D, R, SPARSE>(p, at.u, reinterpret_cast<uint8_t*>(s_dump), s_q, s_cs[0], s_lim[0], s_limits[0], warp, 8);
    if (lane == 0) mbar_arrive(smem_addr(&s_qfull[0]));
#pragma unroll 1
    while (done < run_tiles) {
      const int nt = min(at.u.tiles - at.tile, run_tiles - done);
      const int buf = units & 1;
      float l[R];
#pragma unroll
      for (int r = 0; r < R; ++r) l[r] = 0.f;
      if (ok) ok = warp_wait(smem_addr(&s_qfull[buf]), (units / 2) & 1);
      const int low = s_limits[buf][0], high = s_limits[buf][1];
      group_sync(group);  // the last unit's maxima have been read
      if (token < R) m[token] = kNoScore;
      group_sync(group);
      int mine = 0;
#pragma unroll 1
      for (int j = (done ^ group) & 1; j < nt; j += 2) {
        const int stage = (done + j) % C::kStages;
        if (ok) ok = warp_wait(smem_addr(&s_sfull[group]), count & 1);
        // (for s_pos and the rows of V that are cleared; the keys' barrier may be phases
        // ahead by now, V's waits for this tile's product)
        if (ok) ok = warp_wait(smem_addr(&s_vfull[stage]), ((done + j) / C::kStages) & 1);
        tc_fence_after();
        const int first = s_pos[(done + j) % kPlaces][token / p.box], pos = first + token % p.box;
        float s[R];
        constexpr int kAtOnce = R < 16 ? R : 16;
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += kAtOnce) {
          uint32_t x[C::kQParts][kAtOnce / 8][8];
#pragma unroll
          for (int i = 0; i < C::kQParts; ++i)
#pragma unroll
            for (int k = 0; k < kAtOnce / 8; ++k) tmem_ld8(s_cols + i * R + r0 + 8 * k, x[i][k]);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < C::kQParts; ++i)
#pragma unroll
            for (int k = 0; k < kAtOnce / 8; ++k) tmem_loaded(x[i][k]);
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i)
            s[r0 + i] = fmaf(fmaf(__uint_as_float(x[2][i / 8][i % 8]), 0.0625f, __uint_as_float(x[1][i / 8][i % 8])), 0.0625f,
                             __uint_as_float(x[0][i / 8][i % 8]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&s_sfree[group]));
        // tokens that some row does not see: the last ones, and places without a token
        const bool hidden = pos > low;
        uint32_t blind = 0u;
        const bool edge = __any_sync(0xffffffffu, hidden);
        if (edge) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if (pos > s_lim[buf][r]) {
              blind |= 1u << r;
              s[r] = -INFINITY;
            }
          }
          // V's row must not reach the rows that do not see it as 0 times NaN
          if (hidden && ok) {
            uint4* v = reinterpret_cast<uint4*>(s_ring + stage * 2 * C::kHalf + C::kHalf + token * D);
            if (pos > high) {
#pragma unroll
              for (int i = 0; i < D / 16; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
            } else {
#pragma unroll 1
              for (int i = 0; i < D / 16; ++i) {
                const uint4 x = v[i];
                const uint4 y = make_uint4(fp8_nan_to_zero(x.x), fp8_nan_to_zero(x.y), fp8_nan_to_zero(x.z), fp8_nan_to_zero(x.w));
                if (x.x == y.x && x.y == y.y && x.z == y.z && x.w == y.w) continue;
                v[i] = y;
                const int chunk = i ^ (D == 128 ? token & 7 : (token >> 1) & 3);  // of the row's dims
                const uint32_t from[4] = {x.x, x.y, x.z, x.w};
                for (int c = 0; c < 16; ++c)
                  if ((from[c / 4] >> (8 * (c % 4)) & 0x7Fu) == 0x7Fu) atomicMin(&s_nan[group][16 * chunk + c], pos);
              }
            }
          }
        }
        // ---- the maximum, raised when a weight would pass 2^kHeadroom
        float past = -INFINITY;
#pragma unroll
        for (int r = 0; r < R; r += 4) {
          const float4 m4 = *reinterpret_cast<const float4*>(m + r), c4 = *reinterpret_cast<const float4*>(&s_cs[buf][r]);
          past = fmaxf(fmaxf(past, (s[r] - m4.x) * c4.x), (s[r + 1] - m4.y) * c4.y);
          past = fmaxf(fmaxf(past, (s[r + 2] - m4.z) * c4.z), (s[r + 3] - m4.w) * c4.w);
        }
        if (group_any(group, past > kHeadroom)) {
          float top = 0.f;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float x = warp_max(s[r]);
            if (lane == r) top = x;
          }
          if (lane < R) s_red[group][quarter][lane] = top;
          group_sync(group);
          if (token < R) {
            const float old = m[token];
            const float now = fmaxf(old, fmaxf(fmaxf(s_red[group][0][token], s_red[group][1][token]),
                                               fmaxf(s_red[group][2][token], s_red[group][3][token])));
            s_alpha[group][token] = now > old ? ex2_fast((old - now) * s_cs[buf][token]) : 1.f;
            m[token] = now;
          }
          group_sync(group);
          if (mine > 0) {
            // the product before this one has to be in; rows are rescaled by 8 where one is raised
            if (ok) ok = warp_wait(smem_addr(&s_pvdone[group]), (count - 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int r0 = 0; r0 < R; r0 += 8) {
              float alpha[8], other = 0.f;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                alpha[i] = s_alpha[group][r0 + i];
                other += alpha[i];
              }
              if (other == 8.f) continue;
              uint32_t o[C::kPParts][8];
#pragma unroll
              for (int k = 0; k < C::kPParts; ++k) tmem_ld8(o_cols + k * R + r0, o[k]);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < C::kPParts; ++k) {
                tmem_loaded(o[k]);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[k][i] = __float_as_uint(__uint_as_float(o[k][i]) * alpha[i]);
                tmem_st8(o_cols + k * R + r0, o[k]);
              }
            }
            tmem_st_wait();
          }
#pragma unroll
          for (int r = 0; r < R; ++r) l[r] *= s_alpha[group][r];
        }
        // ---- weights times 2^6, and their parts; the last product has read its own
        if (count > 0 && ok) ok = warp_wait(smem_addr(&s_pvdone[group]), (count - 1) & 1);
        // (16 rows of a part, or 8 of two parts, are a 16-byte chunk)
        constexpr int kRows = R < 16 ? R : 16, kWords = kRows / 4;
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += kRows) {
          uint32_t code[C::kPParts][kWords];
#pragma unroll
          for (int r = 0; r < kRows; r += 2) {
            const float2 m2 = *reinterpret_cast<const float2*>(m + r0 + r), c2 = *reinterpret_cast<const float2*>(&s_cs[buf][r0 + r]);
            float w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              w[i] = ex2_fast(fmaf(s[r0 + r + i] - (i ? m2.y : m2.x), i ? c2.y : c2.x, 8.f - kHeadroom));
              if (edge && (blind >> (r0 + r + i) & 1u)) w[i] = 0.f;
              l[r0 + r + i] += w[i];
            }
            uint32_t part[C::kPParts];
            parts_of(as_u32(__floats2half2_rn(w[0], w[1])), part);
#pragma unroll
            for (int i = 0; i < C::kPParts; ++i) {
              if (r % 4 == 0) code[i][r / 4] = part[i];
              else code[i][r / 4] = __byte_perm(code[i][r / 4], part[i], 0x5410);
            }
          }
          if constexpr (R == 8) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              *reinterpret_cast<uint4*>(weights + chunk_at<C::kNP>(token, i)) =
                  make_uint4(code[2 * i][0], code[2 * i][1], code[2 * i + 1][0], code[2 * i + 1][1]);
          } else {
#pragma unroll
            for (int i = 0; i < C::kPParts; ++i)
              *reinterpret_cast<uint4*>(weights + chunk_at<C::kNP>(token, (i * R + r0) / 16)) =
                  make_uint4(code[i][0], code[i][1], code[i][kWords - 2], code[i][kWords - 1]);
          }
        }
        fence_proxy_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&s_pfull[group]));
        ++count;
        ++mine;
      }

      // ---- the unit's end, or the run's
      const bool whole = at.tile == 0 && nt == at.u.tiles;
      if (mine > 0 && ok) ok = warp_wait(smem_addr(&s_pvdone[group]), (count - 1) & 1);
      tc_fence_after();
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float x = l[r];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        if (lane == 0) s_red[group][quarter][r] = x;
      }
      group_sync(group);
      if (group == 1 && units > 0) both_sync(4);  // the last unit's state and outputs have been read
      if (token < R) {
        const float sum = (s_red[group][0][token] + s_red[group][1][token]) + (s_red[group][2][token] + s_red[group][3][token]);
        s_state[group][0][token] = sum != 0.f ? m[token] * s_cs[buf][token] : -INFINITY;  // a sum of 0: nothing seen
        s_state[group][1][token] = sum;
      }
      group_sync(group);
      const int nan_from = token < D ? s_nan[group][token] : kDead;
      // this group's output of dim `token` and row r
      auto output = [&](int r0, float (&y)[8]) {
        uint32_t o[C::kPParts][8];
#pragma unroll
        for (int i = 0; i < C::kPParts; ++i) tmem_ld8(o_cols + i * R + r0, o[i]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < C::kPParts; ++i) tmem_loaded(o[i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float x = __uint_as_float(o[C::kPParts - 1][i]);
#pragma unroll
          for (int k = C::kPParts - 2; k >= 0; --k) x = fmaf(x, 0.0625f, __uint_as_float(o[k][i]));
          y[i] = mine > 0 ? x : 0.f;
        }
        if (nan_from != kDead) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (nan_from <= s_lim[buf][r0 + i]) y[i] = __int_as_float(0x7fffffff);
        }
      };
      if (group == 1) {
#pragma unroll 1
        for (int r0 = 0; r0 < R && r0 < at.u.rows; r0 += 8) {
          float y[8];
          output(r0, y);
          if (token < D) {
#pragma unroll
            for (int i = 0; i < 8; ++i) s_dump[(r0 + i) * D + token] = y[i];
          }
        }
        tc_fence_before();
        __syncwarp();
        both_arrive(3);
      } else {
        both_sync(3);
        float* part = nullptr;
        const long long unit = r0 + done - at.tile;
        const bool begun = unit / share == nth;
        if (!whole) part = p.partial + (2 * static_cast<size_t>(blockIdx.x) + begun) * C::kPart;
        // a thread for each row: the groups' factors (negative: nothing seen, and what was never
        // written stays out of the sum), and where the row goes
        if (token < R) {
          const float m0 = s_state[0][0][token], m1 = s_state[1][0][token], l0 = s_state[0][1][token], l1 = s_state[1][1][token];
          const float mx = fmaxf(m0, m1);
          const float a0 = l0 != 0.f ? ex2_fast(m0 - mx) : -1.f, a1 = l1 != 0.f ? ex2_fast(m1 - mx) : -1.f;
          const float sum = (l0 != 0.f ? a0 * l0 : 0.f) + (l1 != 0.f ? a1 * l1 : 0.f);
          s_factor[0][token] = a0;
          s_factor[1][token] = a1;
          if (whole) {
            s_factor[2][token] = sum != 0.f ? vscale / sum : 0.f;
            s_to[token] = token < at.u.rows && (!SPARSE || at.u.b >= 0)
                              ? static_cast<long long>(out_at(p, SPARSE, at.u.first, at.u.kvh, at.u.row0 + token)) : -1;
          } else {
            __stcg(part + R * D + token, mx);
            __stcg(part + R * (D + 1) + token, sum);
          }
        }
        group_sync(0);
#pragma unroll 1
        for (int r0 = 0; r0 < R && r0 < at.u.rows; r0 += 8) {
          float y[8];
          output(r0, y);
          if (token < D) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float a0 = s_factor[0][r0 + i], a1 = s_factor[1][r0 + i], other = s_dump[(r0 + i) * D + token];
              y[i] = (a0 < 0.f ? 0.f : a0 * y[i]) + (a1 < 0.f ? 0.f : a1 * other);
            }
            if (whole) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const long long to = s_to[r0 + i];
                if (to >= 0) store1(p, to + token, y[i] * s_factor[2][r0 + i]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) __stcg(part + (r0 + i) * D + token, y[i]);
            }
          }
        }
        tc_fence_before();
        if (!whole && tid == 0) s_open[begun] = {at.u.b, at.u.first, at.u.rows, at.u.row0, at.u.kvh, unit, at.u.tiles};
        __syncwarp();
        both_arrive(4);
      }
      if (nan_from != kDead) s_nan[group][token] = kDead;  // (read by this thread alone)
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&s_qempty[buf]));
      done += nt;
      ++units;
      at.tile += nt;
      if (done < run_tiles) at.next_unit(p);
    }
    if (group == 1) both_sync(4);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
  if (s_open[0].unit < 0 && s_open[1].unit < 0) return;

  // ---- join the CTAs' parts of a unit, in the last CTA to arrive
  if (tid < 2) {
    const Open u = s_open[tid];
    s_last[tid] = 0;
    if (u.unit >= 0) {
      const long long c0 = u.unit / share, c1 = (u.unit + u.tiles - 1) / share;
      __threadfence();  // the CTA's stores, seen through the barrier, before the arrival
      s_last[tid] = atomicAdd(p.counters + c0 * p.side + place, 1u) == static_cast<unsigned>(c1 - c0);
      if (s_last[tid]) {
        p.counters[c0 * p.side + place] = 0u;
        __threadfence();
      }
    }
  }
  __syncthreads();
  const float vscale = __ldg(p.v_scale);
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    if (!s_last[which]) continue;
    const Open u = s_open[which];
    if (SPARSE && u.b < 0) continue;
    const long long c0 = u.unit / share;
    const int parts = static_cast<int>((u.unit + u.tiles - 1) / share - c0) + 1;
    // part 0 is the second place of run c0's CTA, part k the first of run c0 + k's
    const float* src = p.partial + 2 * (static_cast<size_t>(c0) * p.side + place) * C::kPart;
    const size_t next = 2 * static_cast<size_t>(p.side) * C::kPart;
    auto part_at = [&](int k) { return src + (k ? k * next : C::kPart); };
#pragma unroll 1
    for (int item = tid; item < u.rows * (D / 4); item += kThreads) {
      const int r = item / (D / 4), d = 4 * (item % (D / 4));
      float mx = -INFINITY, sum = 0.f;
#pragma unroll 8
      for (int k = 0; k < parts; ++k) mx = fmaxf(mx, __ldcg(part_at(k) + R * D + r));
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int k = 0; k < parts; ++k) {
        const float* s = part_at(k);
        const float l = __ldcg(s + R * (D + 1) + r), mk = __ldcg(s + R * D + r);
        const float4 v = __ldcg(reinterpret_cast<const float4*>(s + r * D + d));
        if (l == 0.f) continue;
        const float a = ex2_fast(mk - mx);
        sum = fmaf(a, l, sum);
        o = make_float4(fmaf(a, v.x, o.x), fmaf(a, v.y, o.y), fmaf(a, v.z, o.z), fmaf(a, v.w, o.w));
      }
      const float inv = sum != 0.f ? vscale / sum : 0.f;
      const size_t to = out_at(p, SPARSE, u.first, u.kvh, u.row0 + r) + d;
      store1(p, to, sum != 0.f ? o.x * inv : 0.f);
      store1(p, to + 1, sum != 0.f ? o.y * inv : 0.f);
      store1(p, to + 2, sum != 0.f ? o.z * inv : 0.f);
      store1(p, to + 3, sum != 0.f ? o.w * inv : 0.f);
    }
  }
}

template <int D, int R, bool SPARSE>
cudaError_t launch_t(const Fp8AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, int num_sms, cudaStream_t stream) {
  auto kern = fp8_rows_kernel<D, R, SPARSE>;
  // the attribute is per function and device; setting it again is harmless
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<D, R>::kSmem);
  if (e != cudaSuccess) return e;
  const int ctas = std::min(num_sms, kFp8MaxCtas) / p.side * p.side;
  return fp8_launch(kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), Few<D, R>::kSmem, stream, p, k, v);
}

template <int D, bool SPARSE>
cudaError_t launch_r(const Fp8AttnParams& p, int rows, const CUtensorMap& k, const CUtensorMap& v, int num_sms, cudaStream_t stream) {
  if (rows <= 8) return launch_t<D, 8, SPARSE>(p, k, v, num_sms, stream);
  if (rows <= 16) return launch_t<D, 16, SPARSE>(p, k, v, num_sms, stream);
  return launch_t<D, 32, SPARSE>(p, k, v, num_sms, stream);
}

}  // namespace

size_t fp8_rows_workspace(int rows, int head_dim, int num_sms) {
  const int r = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
  return kCounterRegion + static_cast<size_t>(std::min(num_sms, kFp8MaxCtas)) * 2 * r * (head_dim + 2) * sizeof(float);
}

cudaError_t read_clear_fp8_rows_status(int* flags) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_status, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  e = cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int));
  *flags = v;
  return e;
}

cudaError_t launch_fp8_rows(const Fp8AttnParams& args, int rows, const CUtensorMap& map_k, const CUtensorMap& map_v, int num_sms,
                            cudaStream_t stream) {
  Fp8AttnParams p = args;
  // A token's KV heads lie side by side in the cache, head_dim bytes each: as many as fill
  // 1 KB are read at the same time, by CTAs next to each other
  p.side = 1;
  for (int i = 2; i <= std::min(1024 / p.c.head_dim, num_sms); ++i)
    if (!p.selected && p.c.num_kv_heads % i == 0) p.side = i;
  if (p.selected)
    return p.c.head_dim == 64 ? launch_r<64, true>(p, rows, map_k, map_v, num_sms, stream)
                              : launch_r<128, true>(p, rows, map_k, map_v, num_sms, stream);
  return p.c.head_dim == 64 ? launch_r<64, false>(p, rows, map_k, map_v, num_sms, stream)
                            : launch_r<128, false>(p, rows, map_k, map_v, num_sms, stream);
}

}  // namespace w8a8
