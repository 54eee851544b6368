// kv4_attention.cu -- attention over the 4-bit KV cache (sm_103a).
//
// Row i of the n new rows of a request of length L sees its tokens
// t <= L - n + i:  out = sum_t softmax(sm_scale q . K_t) V_t, with the cache
// decoded as it is read.  A row that sees nothing gives zeros.
//
// ---- Work
// A unit is one request and KV head: its n new tokens times the G query heads
// that share the KV head are `rows` rows over the same tokens, taken 16 at a
// time (a tile: one record of the cache).  All units' tiles in a row, request
// by request and head by head, are cut into equal runs, one for each CTA, so
// that ragged lengths load the SMs evenly.  A unit that lies in one run is
// written out by its CTA.  One that is cut leaves a partial result (maximum,
// sum, unnormalised output of each row) in the workspace from each CTA, and
// the last of them to arrive joins the parts, in their order.  Every CTA
// makes the sum over the requests' lengths that finds its run itself, so the
// split follows the lengths on the device and one launch does it all.
//
// ---- Few rows (up to 16): mma.sync
// Bound by the cache's bytes, 18 head_dim a tile, as long as the decoding
// keeps up: per tile a warp issues about 250 instructions, of the 390 that
// the SM has slots for in the time that HBM takes to bring the tile.
//   scores  S^T[16 tokens x 8 rows] = K[16 x D] . q^T[D x 8]
//   output  O^T[D x 8 rows] += V^T[D x 16 tokens] . P^T[16 x 8]
// with f16 operands (the decoded cache is exact in f16, the query after
// scaling by a power of two) and fp32 sums.  The weights p = 2^(s - m) <= 1
// enter the second product as f16(p 2^15), 11 bits, and the sum that divides
// the result is taken over the rounded weights, so that the rounding's common
// part cancels.
//
// A producer warp copies tiles ahead into a ring (one untiled bulk copy each;
// lane l looks after slot l: block table, wait, copy); eight warps take the
// tiles in turn, each with a softmax state of its own, joined in shared memory
// at the end of a unit.  While they join, the producer is filling the ring
// with the next unit's tiles.
//
// Registers (lane = 4 g + t).  The dot product does not depend on the order
// of the dims, nor the sum over tokens on theirs, so both are permuted to
// make every shared-memory read one wide word of consecutive codes:
//   K: lane (g, t) holds dims [D/4 t, D/4 (t + 1)) of the tokens in rows g
//      and g + 8; k-block j takes dims D/4 t + 4 j .. + 3 of every lane.
//   V: lane (g, t) holds dims [D/8 g, D/8 (g + 1)) of four tokens, those of
//      rows 2t, 2t + 1, 2t + 8, 2t + 9; m-tile i takes dims D/8 g + 2 i (row
//      g) and + 2 i + 1 (row g + 8).  The codes of two tokens are interleaved
//      nibble by nibble, which makes each byte one operand register.
//   Row 2j of the tile is token j, row 2j + 1 token 4 + (j ^ 1), rows 8.. the
//      same + 8: the K reads are then free of bank conflicts (V's two-way).
#include <algorithm>

#include "internal.h"
#include "kv4.cuh"
#include "sm103_ptx.cuh"

namespace w8a8 {

namespace {

constexpr float kPScale = 32768.f;
constexpr float kLog2e = 1.4426950408889634f;

constexpr int kWarps = 8;                        // warps that compute
constexpr int kThreads = 32 * (kWarps + 1);      // and the producer
constexpr int kComputeThreads = 32 * kWarps;
constexpr int kSlots = 32;                       // ring slots, one for each lane of the producer
constexpr int kMinRun = kWarps;                  // tiles of a CTA's run: one a warp at least
constexpr int kSmallRows = 16;
constexpr int kMaxCounters = 1024;               // CTAs that may leave a unit open
constexpr size_t kCounterBytes = kMaxCounters * sizeof(unsigned);

// CTAs of the few-rows kernel that are resident at once (its registers and
// shared memory allow two of 8 rows to an SM, one of 16).
inline int few_rows_ctas(int nt, int num_sms) { return std::min(kMaxCounters, (nt == 1 ? 2 : 1) * num_sms); }

// ------------------------------------------------------------------ requests

struct Request {
  int first, n;  // its rows in q
  int len;       // tokens
  int tiles;     // 0: nothing to do here
};

// `only` 1: requests of up to kSmallRows rows, 0: larger ones, -1: all.
__device__ __forceinline__ Request request_of(const Kv4AttnParams& p, int b, int only) {
  Request r;
  r.first = b;
  r.n = 1;
  if (p.query_start) {
    r.first = min(max(__ldg(p.query_start + b), 0), p.tokens);
    r.n = min(max(__ldg(p.query_start + b + 1) - r.first, 0), min(p.tokens - r.first, p.max_query_len));
  }
  const long long room = static_cast<long long>(p.max_blocks) * p.block_size;
  r.len = static_cast<int>(min(static_cast<long long>(max(__ldg(p.seq_lens + b), 0)), room));
  const bool small = static_cast<long long>(r.n) * p.share <= kSmallRows;
  // an empty request has one tile, with no token in it, to write its zeros
  r.tiles = r.n > 0 && (only < 0 || small == (only > 0)) ? max(1, (r.len + kKv4Tokens - 1) / kKv4Tokens) : 0;
  return r;
}

// Where a CTA's run begins.
struct Start {
  long long total;  // tiles of all units
  long long before; // tiles in front of request b
  int b;
};

// ------------------------------------------------------------------ pieces

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kComputeThreads) : "memory"); }

__device__ __forceinline__ float load16(const void* p, int fp16, size_t i) {
  if (fp16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// 4 consecutive outputs.
__device__ __forceinline__ void store4(const Kv4AttnParams& p, size_t at, const float (&y)[4]) {
  uint32_t w[2];
  if (p.out_fp16) {
    w[0] = as_u32(__floats2half2_rn(y[0], y[1]));
    w[1] = as_u32(__floats2half2_rn(y[2], y[3]));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(y[0], y[1]), b = __floats2bfloat162_rn(y[2], y[3]);
    w[0] = *reinterpret_cast<const uint32_t*>(&a);
    w[1] = *reinterpret_cast<const uint32_t*>(&b);
  }
  uint16_t* dst = static_cast<uint16_t*>(p.out) + at;
  if (p.out_vec) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
    dst[0] = static_cast<uint16_t>(w[0]);
    dst[1] = static_cast<uint16_t>(w[0] >> 16);
    dst[2] = static_cast<uint16_t>(w[1]);
    dst[3] = static_cast<uint16_t>(w[1] >> 16);
  }
}

// ------------------------------------------------------------------ few rows

template <int D, int NT>
struct Small {
  static constexpr int kRows = 8 * NT;
  static constexpr int kTile = kv4_record_bytes(D);
  static constexpr int kRing = kSlots * kTile;
  static constexpr int kOStride = D + 4;                   // a row's o in shared memory
  static constexpr int kJoin = kWarps * kRows * kOStride * 4;
  static constexpr int kSmem = kRing + kJoin;
  static constexpr int kPart = kRows * (D + 4);            // floats of a partial result: o, then m, l of each row
};

template <int KIND, int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) kv4_few_rows_kernel(const Kv4AttnParams p) {
  using C = Small<D, NT>;
  constexpr int KW = D / 32;   // words of K codes a lane holds of a token
  constexpr int MT = D / 16;   // m-tiles of the output product, k-blocks of the scores'
  extern __shared__ __align__(128) uint8_t smem[];
  float* s_o = reinterpret_cast<float*>(smem + C::kRing);
  __shared__ uint64_t s_full[kSlots], s_empty[kSlots];
  __shared__ float s_m[kWarps][C::kRows], s_l[kWarps][C::kRows];
  __shared__ long long s_scan[kWarps + 1];
  __shared__ Start s_start;
  __shared__ int s_last;
  __shared__ uint8_t s_live[kSlots];  // the slot's tile lies in the cache
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

  if (tid < kSlots) {
    mbar_init(smem_addr(&s_full[tid]), 1);
    mbar_init(smem_addr(&s_empty[tid]), 1);
  }
  if (tid == 0) {
    fence_barrier_init();
    s_start.b = p.batch;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- this CTA's run of tiles
  const int hkv = p.num_kv_heads;
  {
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += static_cast<long long>(request_of(p, b, p.only).tiles) * hkv;
    long long run = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, run, off);
      if (lane >= off) run += o;
    }
    if (lane == 31) s_scan[warp] = run;
    __syncthreads();
    long long total = 0;
    run -= mine;
    for (int w = 0; w <= kWarps; ++w) {
      if (w < warp) run += s_scan[w];
      total += s_scan[w];
    }
    const long long share = max(static_cast<long long>(kMinRun), (total + gridDim.x - 1) / gridDim.x);
    const long long r0 = share * blockIdx.x;
    if (r0 >= run && r0 < run + mine) {
      for (int b = b0; b < b1; ++b) {
        const long long w = static_cast<long long>(request_of(p, b, p.only).tiles) * hkv;
        if (r0 < run + w) {
          s_start.b = b;
          s_start.before = run;
          break;
        }
        run += w;
      }
    }
    if (tid == 0) s_start.total = total;
  }
  __syncthreads();
  const long long total = s_start.total;
  const long long share = max(static_cast<long long>(kMinRun), (total + gridDim.x - 1) / gridDim.x);
  const long long r0 = share * blockIdx.x, r1 = min(total, r0 + share);
  if (r0 >= r1) return;
  int b = s_start.b;
  Request rq = request_of(p, b, p.only);
  int kvh = static_cast<int>((r0 - s_start.before) / rq.tiles);
  int tile = static_cast<int>((r0 - s_start.before) % rq.tiles);
  const int run_tiles = static_cast<int>(min(r1 - r0, 0x7fffffffLL));

  if (warp == kWarps) {
    // ---- producer: lane l fills slot l with tiles l, l + 32, ...; the lanes
    // poll, so that none waits for a slot that is not its own
    const int per_block = p.block_size / kKv4Tokens;
    const uint64_t pol = policy_evict_first();
    const uint32_t full = smem_addr(&s_full[lane]), empty = smem_addr(&s_empty[lane]);
    const uint32_t dst = smem_addr(smem) + lane * C::kTile;
    uint32_t use = 0, idle = 0;
    uint64_t since = 0;
    int f = lane;
    long long rec = -1;
    tile += lane;
    bool fresh = true;  // the next tile's place in the cache is not known yet
    while (__any_sync(0xffffffffu, f < run_tiles)) {
      bool moved = false;
      if (f < run_tiles) {
        if (fresh) {
          while (tile >= rq.tiles) {
            tile -= rq.tiles;
            if (++kvh == hkv) {
              kvh = 0;
              do rq = request_of(p, ++b, p.only);
              while (rq.tiles == 0);
            }
          }
          rec = -1;
          if (tile * kKv4Tokens < rq.len) {
            const int blk = __ldg(p.block_table + static_cast<size_t>(b) * p.max_blocks + tile / per_block);
            if (blk >= 0 && blk < p.num_blocks)
              rec = (static_cast<long long>(blk) * hkv + kvh) * per_block + tile % per_block;
          }
          fresh = false;
        }
        if (use == 0 || mbar_test_wait(empty, (use - 1) & 1)) {
          s_live[lane] = rec >= 0;
          if (rec >= 0) {
            mbar_arrive_expect_tx(full, C::kTile);
            bulk_load_hint(dst, static_cast<const uint8_t*>(p.cache) + rec * C::kTile, C::kTile, full, pol);
          } else {
            mbar_arrive(full);
          }
          ++use;
          f += kSlots;
          tile += kSlots;
          fresh = moved = true;
        }
      }
      if (__any_sync(0xffffffffu, moved)) {
        idle = 0;
      } else if ((++idle & 255u) == 0u) {  // bounded, like every wait
        const uint64_t now = global_timer_ns();
        if (idle == 256u) since = now;
        else if (now - since > W8A8_WAIT_NS) {
          atomicOr(&g_device_status, 1);
          break;
        }
      }
    }
    // the slot's last copy has landed before the CTA's shared memory is released
    if (use > 0) mbar_wait(full, (use - 1) & 1);
    return;
  }

  // ---- the warps that compute
  const int g = lane >> 2, t = lane & 3;
  const int tk = (g >> 1) + (g & 1 ? 4 - (g >> 1) + ((g >> 1) ^ 1) : 0);  // token of row g
  const int tv[4] = {t, 4 + (t ^ 1), 8 + t, 12 + (t ^ 1)};                // tokens of rows 2t, 2t + 1, 2t + 8, 2t + 9
  const float kscale = __ldg(p.k_scale), vscale = __ldg(p.v_scale);
  bool ok = true;
  int f = 0;  // tiles of the run in front of this unit
  long long at = r0;
  while (f < run_tiles) {
    const int seg = min(rq.tiles - tile, run_tiles - f);  // this unit's tiles in the run
    const int rows = rq.n * p.share;

    // the query: dims D/4 t .. of row g (and 8 + g), scaled by 2^e so that the largest lies in [2^14, 2^15)
    uint32_t qf[NT][MT][2];
    float cs;
    {
      float qmax = 0.f;
      uint32_t raw[NT][D / 8];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int c = 8 * nt + g;
        const int i = c / p.share, h = kvh * p.share + c % p.share;
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + (rq.first + i) * p.q_token_stride + h * p.q_head_stride +
                              (D / 4) * t;
#pragma unroll
        for (int j = 0; j < D / 8; j += 4) {
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (c < rows) {
            if (p.q_vec) {
              w = __ldg(reinterpret_cast<const uint4*>(src + 2 * j));
            } else {
              uint32_t u[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                u[x] = static_cast<uint32_t>(__ldg(src + 2 * (j + x))) |
                       (static_cast<uint32_t>(__ldg(src + 2 * (j + x) + 1)) << 16);
              w = make_uint4(u[0], u[1], u[2], u[3]);
            }
          }
          raw[nt][j] = w.x;
          raw[nt][j + 1] = w.y;
          raw[nt][j + 2] = w.z;
          raw[nt][j + 3] = w.w;
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const float2 v = p.q_fp16 ? __half22float2(*reinterpret_cast<const __half2*>(&raw[nt][j]))
                                    : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[nt][j]));
          qmax = fmaxf(qmax, fmaxf(fabsf(v.x), fabsf(v.y)));
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, off));
      // 2^e as a float: qmax in [2^x, 2^(x + 1)) has x + 127 in its exponent bits
      int e = 0;
      if (qmax > 0.f && qmax <= 3.0e38f) e = min(100, max(-100, 14 + 127 - static_cast<int>(__float_as_uint(qmax) >> 23)));
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      cs = p.sm_scale * kscale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const float2 v = p.q_fp16 ? __half22float2(*reinterpret_cast<const __half2*>(&raw[nt][j]))
                                    : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[nt][j]));
          qf[nt][j / 2][j & 1] = as_u32(__floats2half2_rn(v.x * up, v.y * up));
        }
    }
    // the last token that the columns 2t, 2t + 1 see
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 8 * nt + 2 * t + c;
        lim[nt][c] = col < rows ? rq.len - rq.n + col / p.share : rq.len - 1;
      }
    const int all_seen = rq.len - rq.n;  // tokens up to this one are seen by every row

    float m[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }

    // tiles f + x of the run, x < seg, with (f + x) % kWarps == warp
    for (int x = (warp - f % kWarps + kWarps) % kWarps; x < seg; x += kWarps) {
      const int slot = (f + x) % kSlots;
      const uint32_t parity = ((f + x) / kSlots) & 1;
      if (ok) ok = mbar_wait(smem_addr(&s_full[slot]), parity);
      const int t0 = (tile + x) * kKv4Tokens;
      if (ok && s_live[slot]) {
        const uint8_t* rec = smem + slot * C::kTile;
        // scores
        float sp[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sp[nt][0] = sp[nt][1] = sp[nt][2] = sp[nt][3] = 0.f;
        uint32_t kw[2][KW];
        Kv4Scale ks[2][D / 64];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = tk + 8 * r;
          if (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(rec + row * (D / 2) + 16 * t);
            kw[r][0] = v.x;
            kw[r][1] = v.y;
            kw[r][KW - 2] = v.z;
            kw[r][KW - 1] = v.w;
            const __half2 s = e4m3x2_to_half2(*reinterpret_cast<const uint16_t*>(rec + kv4_scales_at(D, 0) + row * (D / 16) + 2 * t));
            ks[r][0] = kv4_scale<KIND>(__low2half2(s));
            ks[r][D / 64 - 1] = kv4_scale<KIND>(__high2half2(s));
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(rec + row * (D / 2) + 8 * t);
            kw[r][0] = v.x;
            kw[r][1] = v.y;
            const __half2 s = e4m3x2_to_half2(rec[kv4_scales_at(D, 0) + row * (D / 16) + t]);
            ks[r][0] = kv4_scale<KIND>(__low2half2(s));
          }
        }
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          uint32_t a[2][4];
          kv4_decode8<KIND>(kw[0][w], ks[0][w / 2], a[0]);
          kv4_decode8<KIND>(kw[1][w], ks[1][w / 2], a[1]);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816(sp[nt], a[0][2 * j], a[1][2 * j], a[0][2 * j + 1], a[1][2 * j + 1], qf[nt][2 * w + j][0],
                       qf[nt][2 * w + j][1]);
        }
        // softmax weights
        const bool edge = t0 + kKv4Tokens - 1 > all_seen;
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float s[4], mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s[k] = sp[nt][k] * cs;
            if (edge && t0 + tk + 8 * (k >> 1) > lim[nt][k & 1]) s[k] = -INFINITY;
            mx[k & 1] = fmaxf(mx[k & 1], s[k]);
          }
          if (__any_sync(0xffffffffu, mx[0] > m[nt][0] || mx[1] > m[nt][1])) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], off));
              const float mn = fmaxf(m[nt][c], mx[c]);
              const float alpha = mn == -INFINITY ? 1.f : ex2_fast(m[nt][c] - mn);
              m[nt][c] = mn;
              l[nt][c] *= alpha;
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[nt][i][c] *= alpha;
                o[nt][i][2 + c] *= alpha;
              }
            }
          }
          float w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = m[nt][k & 1] == -INFINITY ? 0.f : ex2_fast(s[k] - m[nt][k & 1]) * kPScale;
          const __half2 h01 = __floats2half2_rn(w[0], w[1]), h23 = __floats2half2_rn(w[2], w[3]);
          const float2 f01 = __half22float2(h01), f23 = __half22float2(h23);
          l[nt][0] += f01.x + f23.x;
          l[nt][1] += f01.y + f23.y;
          pb[nt][0] = movmatrix_t(as_u32(h01));
          pb[nt][1] = movmatrix_t(as_u32(h23));
        }
        // output
        uint32_t vw[4][D / 64], vs[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint8_t* row = rec + kv4_codes_at(D, 1) + tv[r] * (D / 2);
          if (D == 128) {
            const uint2 v = *reinterpret_cast<const uint2*>(row + 8 * g);
            vw[r][0] = v.x;
            vw[r][D / 64 - 1] = v.y;
            vs[r] = rec[kv4_scales_at(D, 1) + tv[r] * (D / 16) + g];
          } else {
            vw[r][0] = *reinterpret_cast<const uint32_t*>(row + 4 * g);
            vs[r] = rec[kv4_scales_at(D, 1) + tv[r] * (D / 16) + (g >> 1)];
          }
          // past the end the scale may be anything, a NaN too: the weights there are 0
          if (t0 + kKv4Tokens > rq.len && t0 + tv[r] >= rq.len) vs[r] = 0u;
        }
        const Kv4Scale s01 = kv4_scale<KIND>(e4m3x2_to_half2(vs[0] | (vs[1] << 8)));
        const Kv4Scale s23 = kv4_scale<KIND>(e4m3x2_to_half2(vs[2] | (vs[3] << 8)));
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          constexpr uint32_t kLow = 0x0F0F0F0Fu;
          uint32_t e01[4], e23[4], d01[4], d23[4];  // even and odd dims of the token pairs
          kv4_decode8<KIND>((vw[0][w] & kLow) | ((vw[1][w] << 4) & ~kLow), s01, e01);
          kv4_decode8<KIND>((vw[2][w] & kLow) | ((vw[3][w] << 4) & ~kLow), s23, e23);
          kv4_decode8<KIND>(((vw[0][w] >> 4) & kLow) | (vw[1][w] & ~kLow), s01, d01);
          kv4_decode8<KIND>(((vw[2][w] >> 4) & kLow) | (vw[3][w] & ~kLow), s23, d23);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816(o[nt][4 * w + i], e01[i], d01[i], e23[i], d23[i], pb[nt][0], pb[nt][1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&s_empty[slot]));
    }

    // ---- join the warps' states
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], off);
        const int col = 8 * nt + 2 * t + c;
        if (g == 0) {
          s_m[warp][col] = m[nt][c];
          s_l[warp][col] = l[nt][c];
        }
        float* dst = s_o + (warp * C::kRows + col) * C::kOStride + (D / 8) * g;
#pragma unroll
        for (int i = 0; i < MT; ++i) *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(o[nt][i][c], o[nt][i][2 + c]);
      }
    compute_sync();
    const bool whole = tile == 0 && seg == rq.tiles;
    const long long unit = at - tile;  // the unit's first tile
    const long long c0 = unit / share;
    const int parts = static_cast<int>((unit + rq.tiles - 1) / share - c0) + 1;
    float* part = p.partial + (2 * static_cast<size_t>(blockIdx.x) + (c0 == blockIdx.x ? 1 : 0)) * C::kPart;
    for (int item = tid; item < C::kRows * (D / 4); item += kComputeThreads) {
      const int col = item / (D / 4), d = 4 * (item % (D / 4));
      if (col >= rows) continue;
      float mm = s_m[0][col];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, s_m[w][col]);
      float ll = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
      if (mm != -INFINITY) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float a = ex2_fast(s_m[w][col] - mm);
          const float4 v = *reinterpret_cast<const float4*>(s_o + (w * C::kRows + col) * C::kOStride + d);
          ll = fmaf(a, s_l[w][col], ll);
          y[0] = fmaf(a, v.x, y[0]);
          y[1] = fmaf(a, v.y, y[1]);
          y[2] = fmaf(a, v.z, y[2]);
          y[3] = fmaf(a, v.w, y[3]);
        }
      }
      if (whole) {
        const float inv = ll > 0.f ? vscale / ll : 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] *= inv;
        store4(p, (rq.first + col / p.share) * p.out_token_stride + (kvh * p.share + col % p.share) * p.out_head_stride + d, y);
      } else {
        __stcg(reinterpret_cast<float4*>(part + col * (D + 4) + d), make_float4(y[0], y[1], y[2], y[3]));
        if (d == 0) __stcg(reinterpret_cast<float2*>(part + col * (D + 4) + D), make_float2(mm, ll));
      }
    }
    if (!whole) {
      __threadfence();
      compute_sync();
      if (tid == 0) {
        const unsigned old = atomicAdd(p.counters + c0, 1u);
        s_last = old == static_cast<unsigned>(parts) - 1u;
        if (s_last) p.counters[c0] = 0u;
      }
      compute_sync();
      if (s_last) {
        __threadfence();
        for (int item = tid; item < C::kRows * (D / 4); item += kComputeThreads) {
          const int col = item / (D / 4), d = 4 * (item % (D / 4));
          if (col >= rows) continue;
          const float* src = p.partial + 2 * static_cast<size_t>(c0) * C::kPart + col * (D + 4);
          // part 0 is the second place of CTA c0, part j the first of CTA c0 + j
          float mm = -INFINITY;
#pragma unroll 8
          for (int j = 0; j < parts; ++j) mm = fmaxf(mm, __ldcg(src + (j ? 2 * j : 1) * static_cast<size_t>(C::kPart) + D));
          float ll = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
          if (mm != -INFINITY) {
#pragma unroll 8
            for (int j = 0; j < parts; ++j) {
              const float* q = src + (j ? 2 * j : 1) * static_cast<size_t>(C::kPart);
              const float2 ml = __ldcg(reinterpret_cast<const float2*>(q + D));
              const float4 v = __ldcg(reinterpret_cast<const float4*>(q + d));
              const float a = ex2_fast(ml.x - mm);
              ll = fmaf(a, ml.y, ll);
              y[0] = fmaf(a, v.x, y[0]);
              y[1] = fmaf(a, v.y, y[1]);
              y[2] = fmaf(a, v.z, y[2]);
              y[3] = fmaf(a, v.w, y[3]);
            }
          }
          const float inv = ll > 0.f ? vscale / ll : 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] *= inv;
          store4(p, (rq.first + col / p.share) * p.out_token_stride + (kvh * p.share + col % p.share) * p.out_head_stride + d, y);
        }
      }
    } else {
      compute_sync();  // the joined states have been read
    }

    // ---- the next unit
    f += seg;
    at += seg;
    tile = 0;
    if (f < run_tiles && ++kvh == hkv) {
      kvh = 0;
      do rq = request_of(p, ++b, p.only);
      while (rq.tiles == 0);
    }
  }
}

template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args) {
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

template <int KIND, int D, int NT>
cudaError_t launch_few(const Kv4AttnParams& p, int num_sms, cudaStream_t stream) {
  auto kern = kv4_few_rows_kernel<KIND, D, NT>;
  // the attribute is per function and device; setting it again is harmless
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Small<D, NT>::kSmem);
  if (e != cudaSuccess) return e;
  const long long most = static_cast<long long>(p.batch) * p.num_kv_heads *
                         ((static_cast<long long>(p.max_blocks) * p.block_size + kKv4Tokens - 1) / kKv4Tokens);
  const long long ctas = std::min<long long>((most + kMinRun - 1) / kMinRun, few_rows_ctas(NT, num_sms));
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), Small<D, NT>::kSmem, stream, p);
}

template <int KIND, int D>
cudaError_t launch_kind(const Kv4AttnParams& p, int num_sms, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.share) * p.max_query_len;
  if (rows <= 8) return launch_few<KIND, D, 1>(p, num_sms, stream);
  return launch_few<KIND, D, 2>(p, num_sms, stream);
}

}  // namespace

size_t kv4_attention_workspace(int share, long long max_query_len, int head_dim, int num_sms) {
  const int nt = share * max_query_len <= 8 ? 1 : 2;
  return kCounterBytes + static_cast<size_t>(few_rows_ctas(nt, num_sms)) * 2 * 8 * nt * (head_dim + 4) * sizeof(float);
}

cudaError_t read_clear_kv4_status(int* flags) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_status, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  e = cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int));
  *flags = v;
  return e;
}

cudaError_t launch_kv4_attention(const Kv4AttnParams& args, int num_sms, void* workspace, cudaStream_t stream) {
  Kv4AttnParams p = args;
  p.counters = static_cast<unsigned*>(workspace);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCounterBytes);
  p.share = p.num_q_heads / p.num_kv_heads;
  p.only = -1;
  if (static_cast<long long>(p.share) * p.max_query_len > kSmallRows) return launch_kv4_prompt(p, stream);
  if (p.head_dim == 64)
    return p.kind == W8A8_KV4_E2M1 ? launch_kind<W8A8_KV4_E2M1, 64>(p, num_sms, stream)
                                   : launch_kind<W8A8_KV4_INT4, 64>(p, num_sms, stream);
  return p.kind == W8A8_KV4_E2M1 ? launch_kind<W8A8_KV4_E2M1, 128>(p, num_sms, stream)
                                 : launch_kind<W8A8_KV4_INT4, 128>(p, num_sms, stream);
}

}  // namespace w8a8
