// kv4_attention.cu -- attention over the 4-bit KV cache (sm_103a).
//
// Row i of the n new rows of a request of length L sees its tokens
// t <= L - n + i:  out = sum_t softmax(sm_scale q . K_t) V_t, with the cache
// decoded as it is read.  A row that sees nothing gives zeros.
//
// ---- Work
// A unit is one request and KV head: its n new tokens times the G query heads
// that share the KV head are rows over the same tokens (up to 16; 17 to 32 make
// two units, the second of which finds the cache in L2), taken in steps of
// kStep tiles (a tile: the 16 tokens of one record).  All units' steps in a
// row, request by request and head by head, are cut into equal runs, one for
// each warp of the grid, so that ragged lengths load the SMs evenly.  A warp
// goes through its run alone: no barrier, no other warp's data.  A unit that
// lies in one run is written out by its warp; one that is cut leaves a piece
// (maximum, sum, unnormalised output of each row) with each of its warps.  At
// the end the CTA joins its warps' pieces; a unit that goes on in other CTAs
// leaves a part in the workspace, and the last CTA to arrive joins the parts.
// Pieces and parts are joined in the order of their tokens, so the result does
// not depend on timing.  Every CTA makes the sum over the requests' lengths
// that finds its run itself: the split follows the lengths on the device, and
// one launch does it all.
//
// ---- Few rows: mma.sync
// Bound by the cache's bytes, 18 head_dim a tile, as long as the decoding
// keeps up: per tile of head_dim 128 a warp issues about 330 instructions (70
// conversions, 64 products with the scales, 17 MMAs), of the 390 that the SM
// has slots for in the time that HBM takes to bring the tile.
//   scores  S^T[16 tokens x 8 rows] = K[16 x D] . q^T[D x 8]
//   output  O^T[D x 8 rows] += V^T[D x 16 tokens] . P^T[16 x 8]
// with f16 operands (the decoded cache is exact in f16, the query after
// scaling by a power of two) and fp32 sums.  The weights p = 2^(s - m)
// enter the second product as f16(p 2^13), 11 bits (fewer for weights below
// 2^-27 of the largest), and the sum that divides the result is taken over the
// rounded weights (by one more MMA, whose A is ones), so that the rounding's
// common part cancels.  The maximum m is raised only when a score passes it by
// more than 2 (2^15 then, f16's last power of two): the state is rescaled a few
// times a unit, not at every new maximum.  (A headroom of 8 was no faster and
// kept fewer bits of small weights.)
//
// A warp copies its next step's records (untiled bulk copies) as soon as it
// has read a slot of its ring, across the ends of units.  (A producer warp in
// place of that cost a fifth of the issue slots in polling, and its
// registers; units shared by a CTA's warps and joined one by one cost 10 us
// of barriers and cold loads each.)  The two tiles of a step are decoded
// together, so that one's latencies hide behind the other's.
//
// Registers (lane = 4 g + t).  The dot product does not depend on the order
// of the dims, nor the sum over tokens on theirs, so both are permuted to
// make every shared-memory read one wide word of consecutive codes:
//   K: lane (g, t) holds dims [D/4 t, D/4 (t + 1)) of the tokens in rows g
//      and g + 8; k-block j takes dims D/4 t + 4 j .. + 3 of every lane.
//   V: lane (g, t) holds dims [D/8 g, D/8 (g + 1)) of four tokens, those of
//      rows 2t, 2t + 1, 2t + 8, 2t + 9; m-tile i takes two of the dims (rows g
//      and g + 8).  The codes of two tokens are interleaved, which makes two
//      codes of one dim one operand register.
//   Row 2j of the tile is token j, row 2j + 1 token 4 + (j ^ 1), rows 8.. the
//      same + 8: the K reads are then free of bank conflicts (V's two-way).
//
// Measured (device time, cold L2): 64 requests up to 8192 tokens, 8 KV heads of
// 128, 4 query heads each: 88 us, 3.9 TB/s of the cache (58 % of the 6.7 TB/s that
// a copy reaches; the steps run at 88 % of it, the rest is the launch, the first
// copies and the joins); heads of 64: 62 us, 2.8 TB/s; 128 requests up to 16384:
// 269 us, 5.1 TB/s (77 %); one request of 1023: 17 us, of which the launch and the
// measurement are 6.
#include <algorithm>

#include "internal.h"
#include "kv4.cuh"
#include "sm103_ptx.cuh"

namespace w8a8 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// At most two groups of 16.  20 rows (32 requests of up to 4096 tokens, cold): 79 us
// here, 121 in the many-rows kernel, which takes 128 rows at a time; one group 57.
// A third group was not tried.
constexpr int kSmallRows = 32;
constexpr float kHeadroom = 2.f;
constexpr float kNoScore = -1e25f;               // below any product, and finite
constexpr int kMaxCounters = 1024;               // CTAs that may leave a unit open
constexpr size_t kCounterBytes = kMaxCounters * sizeof(unsigned);

// CTAs of the few-rows kernel that are resident at once (its registers and
// shared memory allow two of 8 rows to an SM, one of 16).
inline int few_rows_ctas(int nt, int num_sms) { return std::min(kMaxCounters, (nt == 1 ? 2 : 1) * num_sms); }

// ------------------------------------------------------------------ requests

struct Request {
  int first, n;  // its rows in q that are looked at
  int all;       // its new tokens (more than n only past max_query_len)
  int len;       // tokens
  int steps;     // steps of a unit; 0: nothing to do here
  int more;      // groups of its rows that a KV head has, less one (0 or 1)
  int units;
};

template <int kStep, int kRows>
__device__ __forceinline__ Request request_of(const Kv4AttnParams& p, int b) {
  Request r;
  r.first = b;
  r.all = 1;
  if (p.query_start) {
    r.first = min(max(__ldg(p.query_start + b), 0), p.tokens);
    r.all = max(min(__ldg(p.query_start + b + 1), p.tokens) - r.first, 0);
  }
  r.n = min(r.all, p.max_query_len);
  const long long room = static_cast<long long>(p.max_blocks) * p.block_size;
  r.len = static_cast<int>(min(static_cast<long long>(max(__ldg(p.seq_lens + b), 0)), room));
  // an empty request has one step, with no token in it, to write its zeros
  constexpr int kTokens = kStep * kKv4Tokens;
  r.more = r.n * p.share > kRows;
  r.units = p.num_kv_heads << r.more;
  r.steps = r.n > 0 ? max(1, (r.len + kTokens - 1) / kTokens) : 0;
  return r;
}

// Where a warp's run begins: the request, and the steps in front of it.
struct Start {
  int b, before;
};

// A cut unit's share of one run.
struct Piece {
  int unit;  // the unit's first step; -1: no piece
  int steps; // the unit's
  int first, kvh, row0, rows;
};

// ------------------------------------------------------------------ pieces

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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

// The first output element of a unit's row.
__device__ __forceinline__ size_t out_at(const Kv4AttnParams& p, int first, int kvh, int row) {
  return (first + row / p.share) * p.out_token_stride + (kvh * p.share + row % p.share) * p.out_head_stride;
}

// 4 consecutive outputs.
__device__ __forceinline__ void store4(const Kv4AttnParams& p, size_t at, float a, float b, float c, float d) {
  uint32_t w[2];
  if (p.out_fp16) {
    w[0] = as_u32(__floats2half2_rn(a, b));
    w[1] = as_u32(__floats2half2_rn(c, d));
  } else {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
    w[0] = *reinterpret_cast<const uint32_t*>(&x);
    w[1] = *reinterpret_cast<const uint32_t*>(&y);
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

// Softmax states of one row and 4 dims, joined: m their largest maximum,
// known first.
struct Joined {
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void add(float2 ml, float4 v) {
    const float a = ml.x == -INFINITY ? 0.f : ex2_fast(ml.x - m);
    l = fmaf(a, ml.y, l);
    o = make_float4(fmaf(a, v.x, o.x), fmaf(a, v.y, o.y), fmaf(a, v.z, o.z), fmaf(a, v.w, o.w));
  }
  __device__ __forceinline__ void store(const Kv4AttnParams& p, size_t at, float vscale) const {
    const float inv = l > 0.f ? vscale / l : 0.f;
    store4(p, at, o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  }
};

// ------------------------------------------------------------------ few rows

template <int D, int NT>
struct Small {
  static constexpr int kRows = 8 * NT;
  // 8 rows: 128 registers, two CTAs of 8 warps to an SM.  16 rows: the state
  // takes twice the registers (240), so one CTA (12 warps of 168 registers with
  // steps of one tile: 61 us for 55 at 32 requests of 12 rows, 2300 tokens)
  static constexpr int kWarps = 8, kThreads = 32 * kWarps;
  static constexpr int kCtas = NT == 1 ? 2 : 1;
  static constexpr int kStep = 2;            // tiles of a step
  static constexpr int kRing = 2;            // steps in a warp's ring
  static constexpr int kTile = kv4_record_bytes(D);
  static constexpr int kSlot = kStep * kTile;
  static constexpr int kRingBytes = kWarps * kRing * kSlot;
  static constexpr int kOStride = D + 4;                   // a row of a piece
  static constexpr int kPiece = kRows * kOStride;          // floats: o, m, l of each row
  static constexpr int kSmem = kRingBytes + kWarps * kPiece * 4;
  static_assert(kPiece * 4 <= kRing * kSlot, "a warp's ring holds its last piece");
};

template <int KIND, int D, int NT>
__global__ void __launch_bounds__(Small<D, NT>::kThreads, Small<D, NT>::kCtas) kv4_few_rows_kernel(const Kv4AttnParams p) {
  using C = Small<D, NT>;
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads, kStep = C::kStep, kRing = C::kRing;
  constexpr uint32_t kAll = (1u << kStep) - 1u;  // a step's records
  constexpr int KW = D / 32;   // words of K codes a lane holds of a token
  constexpr int MT = D / 16;   // m-tiles of the output product, k-blocks of the scores'
  extern __shared__ __align__(128) uint8_t smem[];
  float* const heads = reinterpret_cast<float*>(smem + C::kRingBytes);  // [kWarps] pieces of units begun in front of a run
  __shared__ uint64_t s_full[kWarps][kRing];
  __shared__ int s_scan[kWarps];
  __shared__ Start s_start[kWarps];
  __shared__ Piece s_piece[2 * kWarps];  // in the order of their tokens
  __shared__ int s_last[2];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < kWarps * kRing; ++i) mbar_init(smem_addr(&s_full[0][0] + i), kStep);
    fence_barrier_init();
  }
  if (tid < 2 * kWarps) s_piece[tid].unit = -1;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- the runs (all units' steps are fewer than 2^31, the launcher sees to it)
  const int workers = static_cast<int>(gridDim.x) * kWarps;
  int total = 0, share;
  {
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
    int mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const Request r = request_of<kStep, C::kRows>(p, b);
      mine += r.steps * r.units;
    }
    int run = mine;
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, run, off);
      if (lane >= off) run += o;
    }
    if (lane == 31) s_scan[warp] = run;
    __syncthreads();
    run -= mine;
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) run += s_scan[w];
      total += s_scan[w];
    }
    share = static_cast<int>((static_cast<unsigned>(total) + workers - 1u) / workers);
    // the runs of this CTA's warps that begin in the thread's requests
    if (mine > 0) {
#pragma unroll 1
      for (int w = 0; w < kWarps; ++w) {
        const long long at = static_cast<long long>(share) * (blockIdx.x * kWarps + w);
        if (at < run || at >= static_cast<long long>(run) + mine) continue;
        int before = run;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
          const Request r = request_of<kStep, C::kRows>(p, b);
          const int steps = r.steps * r.units;
          if (at < before + steps) {
            s_start[w] = {b, before};
            break;
          }
          before += steps;
        }
      }
    }
  }
  __syncthreads();
  const int cta_share = share * kWarps;  // at most total + workers
  if (static_cast<long long>(cta_share) * blockIdx.x >= total) return;
  const int r0 = static_cast<int>(min(static_cast<long long>(total), static_cast<long long>(share) * (blockIdx.x * kWarps + warp)));
  const int run_steps = min(total - r0, share);
  const float kscale = __ldg(p.k_scale), vscale = kv4_out_scale(p.sm_scale, p.k_scale, p.v_scale);
  const uint32_t full0 = smem_addr(&s_full[warp][0]);
  uint8_t* const ring = smem + warp * kRing * C::kSlot;
  bool ok = true;
  if (run_steps > 0) {
  int b = s_start[warp].b;
  Request rq = request_of<kStep, C::kRows>(p, b);
  int ui = (r0 - s_start[warp].before) / rq.steps;  // unit of the request: KV head, then group of rows
  int step = (r0 - s_start[warp].before) - ui * rq.steps;

  // ---- fetching, up to kRing steps ahead of the computation
  const uint64_t pol = policy_evict_first();
  // The places of a batch of 16 steps are looked up at once: lane 2 k + u has
  // record u of the batch's step k, and copies it when its turn comes.
  constexpr int kBatch = 32 / kStep;
  int fb = b, fui = ui, fpos = 0, fetched = 0;  // fpos: the position in the run that fstep stands for
  int fstep = step;
  Request frq = rq;
  const uint8_t* src = nullptr;  // this lane's record
  uint32_t found = 0u;           // the lanes whose record lies in the cache
  uint32_t live_bits = 0u;       // the same of the steps in the ring
  auto fetch = [&] {
    if (fetched >= run_steps) return;
    if (fetched % kBatch == 0) {
      const int want = fetched + lane / kStep;
      bool in = want < run_steps;
      if (in) {
        fstep += want - fpos;
        fpos = want;
        while (fstep >= frq.steps) {
          fstep -= frq.steps;
          if (++fui == frq.units) {
            fui = 0;
            do frq = request_of<kStep, C::kRows>(p, ++fb);
            while (frq.steps == 0);
          }
        }
        const int tile = fstep * kStep + lane % kStep;
        in = tile < (frq.len + kKv4Tokens - 1) / kKv4Tokens;
        if (in) {
          const int page = p.block_shift >= 0 ? tile >> p.block_shift : tile / p.per_block;
          const int blk = __ldg(p.block_table + static_cast<size_t>(fb) * p.max_blocks + page);
          in = blk >= 0 && blk < p.num_blocks;
          src = static_cast<const uint8_t*>(p.cache) +
                ((static_cast<long long>(blk) * p.num_kv_heads + (fui >> frq.more)) * p.per_block + (tile - page * p.per_block)) * C::kTile;
        }
      }
      found = __ballot_sync(0xffffffffu, in);
    }
    const int turn = fetched % kBatch, slot = fetched % kRing;
    const uint32_t live = (found >> (kStep * turn)) & kAll;
    live_bits = (live_bits & ~(kAll << (kStep * slot))) | (live << (kStep * slot));
    if (lane / kStep == turn) {
      const uint32_t full = full0 + 8 * slot;
      fence_proxy_async_shared();  // the reads of the slot's last step before the copies that overwrite it
      if (live >> (lane % kStep) & 1u) {
        mbar_arrive_expect_tx(full, C::kTile);
        const uint32_t dst = smem_addr(ring + slot * C::kSlot + (lane % kStep) * C::kTile);
        if (NT == 1) bulk_load_hint(dst, src, C::kTile, full, pol);
        else bulk_load(dst, src, C::kTile, full);  // a second group of rows may read it again
      } else {
        mbar_arrive(full);
      }
    }
    ++fetched;
  };
#pragma unroll 1
  for (int i = 0; i < kRing; ++i) fetch();

  const int g = lane >> 2, t = lane & 3;
  const int tk = (g >> 1) + (g & 1 ? 4 - (g >> 1) + ((g >> 1) ^ 1) : 0);  // token of row g
  const int tv[4] = {t, 4 + (t ^ 1), 8 + t, 12 + (t ^ 1)};                // tokens of rows 2t, 2t + 1, 2t + 8, 2t + 9
  int done = 0;  // steps computed
  while (done < run_steps) {
    const int seg = min(rq.steps - step, run_steps - done);  // this unit's steps in the run
    const int kvh = ui >> rq.more, row0 = (ui & rq.more) * C::kRows;
    const int rows = min(C::kRows, rq.n * p.share - row0);

    // the query: dims D/4 t .. of row g (and 8 + g), each row scaled by a 2^e that
    // brings its largest element into [2^14, 2^15); infinities stay what they are
    uint32_t qf[NT][MT][2];
    float cs[NT][2];  // scale of the scores of the columns 2t, 2t + 1
    {
      float up[NT];
      uint32_t raw[NT][D / 8];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float qmax = 0.f;
        const int c = 8 * nt + g;
        const int i = (row0 + c) / p.share, h = kvh * p.share + (row0 + c) % p.share;
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
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, off));
        // 2^e as a float: qmax in [2^x, 2^(x + 1)) has x + 127 in its exponent bits
        int e = 0;
        if (qmax > 0.f) e = min(100, 14 + 127 - static_cast<int>(__float_as_uint(qmax) >> 23));
        float down = p.sm_scale * kscale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        // the scale's sign goes to the query: the largest product is the largest score
        up[nt] = copysignf(__uint_as_float(static_cast<uint32_t>(127 + e) << 23), down);
        // (no zero, so that a masked score's infinity stays one)
        down = fmaxf(fabsf(down), 1e-37f);
        cs[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t);
        cs[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 x = p.q_fp16 ? __half22float2(*reinterpret_cast<const __half2*>(&raw[nt][4 * w + j]))
                                      : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[nt][4 * w + j]));
            v[2 * j] = x.x * up[nt];
            v[2 * j + 1] = x.y * up[nt];
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            qf[nt][2 * w + j / 2][j & 1] = as_u32(__floats2half2_rn(v[kv4_low<KIND>(j)], v[kv4_high<KIND>(j)]));
        }
    }
    // the last token that the columns 2t, 2t + 1 see
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 8 * nt + 2 * t + c;
        lim[nt][c] = col < rows ? rq.len - rq.all + (row0 + col) / p.share : rq.len - 1;
      }
    const int all_seen = rq.len - rq.all + row0 / p.share;  // tokens up to this one are seen by every row

    float m[NT][2], l[NT][4], o[NT][MT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kNoScore;
      l[nt][0] = l[nt][1] = l[nt][2] = l[nt][3] = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }

    for (int x = 0; x < seg; ++x) {
      const int slot = done % kRing;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(full0 + 8 * slot, (done / kRing) & 1));
      const uint32_t live = ok ? (live_bits >> (kStep * slot)) & kAll : 0u;
      const int t0 = (step + x) * kStep * kKv4Tokens;
      const uint8_t* rec0 = ring + slot * C::kSlot;
      if (live) {
        // scores
        float sp[kStep][NT][4];
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
          const uint8_t* rec = rec0 + u * C::kTile;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) sp[u][nt][0] = sp[u][nt][1] = sp[u][nt][2] = sp[u][nt][3] = 0.f;
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
              const __half2 s = e4m3x2_to_half2(
                  *reinterpret_cast<const uint16_t*>(rec + kv4_scales_at(D, 0) + row * (D / 16) + 2 * t));
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
                mma16816(sp[u][nt], a[0][2 * j], a[1][2 * j], a[0][2 * j + 1], a[1][2 * j + 1], qf[nt][2 * w + j][0],
                         qf[nt][2 * w + j][1]);
          }
        }
        // softmax weights
        const bool edge = t0 + kStep * kKv4Tokens - 1 > all_seen || live != kAll;
        if (edge) {
          asm volatile("");  // a branch, not a select for every score of every step
#pragma unroll
          for (int u = 0; u < kStep; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (t0 + u * kKv4Tokens + tk + 8 * (k >> 1) > lim[nt][k & 1] || !(live >> u & 1u)) sp[u][nt][k] = -INFINITY;
        }
        uint32_t pb[kStep][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int u = 0; u < kStep; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k & 1] = fmaxf(mx[k & 1], sp[u][nt][k]);
          // raised when a weight would pass 2^kHeadroom; weights come out times 2^(15 - kHeadroom) for f16
          if (__any_sync(0xffffffffu, (mx[0] - m[nt][0]) * cs[nt][0] > kHeadroom || (mx[1] - m[nt][1]) * cs[nt][1] > kHeadroom)) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], off));
              const float mn = fmaxf(m[nt][c], mx[c]);
              const float alpha = ex2_fast((m[nt][c] - mn) * cs[nt][c]);
              m[nt][c] = mn;
              l[nt][c] *= alpha;
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[nt][i][c] *= alpha;
                o[nt][i][2 + c] *= alpha;
              }
            }
          }
#pragma unroll
          for (int u = 0; u < kStep; ++u) {
            // (s - m) cs and not s cs - m cs: with scores of 2^26 and more the rounding of
            // m cs alone would push weights out of f16
            float w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = ex2_fast(fmaf(sp[u][nt][k] - m[nt][k & 1], cs[nt][k & 1], 15.f - kHeadroom));
            pb[u][nt][0] = movmatrix_t(as_u32(__floats2half2_rn(w[0], w[1])));
            pb[u][nt][1] = movmatrix_t(as_u32(__floats2half2_rn(w[2], w[3])));
            // the sum of the rounded weights, as one more row of ones
            constexpr uint32_t kOnes = 0x3C003C00u;
            mma16816(l[nt], kOnes, kOnes, kOnes, kOnes, pb[u][nt][0], pb[u][nt][1]);
          }
        }
        // output
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
          const uint8_t* rec = rec0 + u * C::kTile;
          const bool tail = t0 + (u + 1) * kKv4Tokens > rq.len || !(live >> u & 1u);
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
          }
          if (tail) {
            // where there is no token the scale may be anything, a NaN too: the weights there are 0
            asm volatile("");
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (t0 + u * kKv4Tokens + tv[r] >= rq.len || !(live >> u & 1u)) vs[r] = 0u;
          }
          const Kv4Scale s01 = kv4_scale<KIND>(e4m3x2_to_half2(__byte_perm(vs[0], vs[1], 0x0040)));
          const Kv4Scale s23 = kv4_scale<KIND>(e4m3x2_to_half2(__byte_perm(vs[2], vs[3], 0x0040)));
#pragma unroll
          for (int w = 0; w < D / 64; ++w) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t h01[4], h23[4];
              kv4_decode8<KIND>(kv4_interleave<KIND>(vw[0][w], vw[1][w], q), s01, h01);
              kv4_decode8<KIND>(kv4_interleave<KIND>(vw[2][w], vw[3][w], q), s23, h23);
#pragma unroll
              for (int i = 0; i < 4; i += 2)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma16816(o[nt][4 * w + 2 * q + i / 2], h01[i], h01[i + 1], h23[i], h23[i + 1], pb[u][nt][0], pb[u][nt][1]);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the slot
      ++done;
      fetch();
    }

    // ---- the unit's end, or the run's: lane (g, t) has dims D/8 g .. of the columns 2t, 2t + 1
    const bool ends = step + seg == rq.steps;
    const bool last = done == run_steps;
    const bool whole = step == 0 && ends;
    if (!whole && last) __syncwarp();  // the ring's last slot has been read: it takes the piece
    float* piece = last ? reinterpret_cast<float*>(ring) : heads + warp * C::kPiece;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 8 * nt + 2 * t + c;
        float y[D / 8];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          // m-tile i: values 2 (i % 2), + 1 of interleaved word i / 2
          const int w = i / 4, q = i / 2 % 2, v = 2 * (i % 2);
          y[8 * w + kv4_pair_dim<KIND>(q, v)] = o[nt][i][c];
          y[8 * w + kv4_pair_dim<KIND>(q, v + 1)] = o[nt][i][2 + c];
        }
        if (col >= rows) continue;
        if (whole) {
          const float inv = l[nt][c] > 0.f ? vscale / l[nt][c] : 0.f;
          const size_t at = out_at(p, rq.first, kvh, row0 + col) + (D / 8) * g;
#pragma unroll
          for (int i = 0; i < D / 8; i += 4) store4(p, at + i, y[i] * inv, y[i + 1] * inv, y[i + 2] * inv, y[i + 3] * inv);
        } else {
          float* dst = piece + col * C::kOStride + (D / 8) * g;
#pragma unroll
          for (int i = 0; i < D / 8; i += 4) *reinterpret_cast<float4*>(dst + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
          if (g == 0)  // m in the log2 domain
            *reinterpret_cast<float2*>(piece + col * C::kOStride + D) =
                make_float2(l[nt][c] > 0.f ? m[nt][c] * cs[nt][c] : -INFINITY, l[nt][c]);
        }
      }
    if (!whole && lane == 0) s_piece[2 * warp + last] = {r0 + done - seg - step, rq.steps, rq.first, kvh, row0, rows};

    // ---- the next unit
    step = 0;
    if (!last && ++ui == rq.units) {
      ui = 0;
      do rq = request_of<kStep, C::kRows>(p, ++b);
      while (rq.steps == 0);
    }
  }
  // a wait gave up (flagged in the device status): the copies still in flight
  // land before the CTA's shared memory is released
  if (!ok)
    for (int i = max(0, fetched - kRing); i < fetched; ++i) mbar_wait(full0 + 8 * (i % kRing), (i / kRing) & 1);
  }
  __syncthreads();

  // ---- join the warps' pieces
  auto piece_at = [&](int k) {
    return k & 1 ? reinterpret_cast<const float*>(smem + (k / 2) * kRing * C::kSlot) : heads + (k / 2) * C::kPiece;
  };
  Piece open0, open1;  // units that go on in other CTAs: the one begun in front of this CTA, the one begun here
  open0.unit = open1.unit = -1;
  for (int i = 0; i < 2 * kWarps;) {
    const Piece u = s_piece[i];
    if (u.unit < 0) {
      ++i;
      continue;
    }
    uint32_t mine = 0u;  // the unit's pieces
    int next = 2 * kWarps;
#pragma unroll 1
    for (int k = i; k < next; ++k) {
      const int unit = s_piece[k].unit;
      if (unit == u.unit) mine |= 1u << k;
      else if (unit >= 0) next = k;
    }
    const int c0 = u.unit / cta_share, c1 = (u.unit + u.steps - 1) / cta_share;
    const bool whole = c0 == c1, begun = c0 == static_cast<int>(blockIdx.x);
    float* part = p.partial + (2 * static_cast<size_t>(blockIdx.x) + begun) * C::kPiece;
    for (int item = tid; item < u.rows * (D / 4); item += kThreads) {
      const int col = item / (D / 4), d = 4 * (item % (D / 4));
      Joined sum;
      float2 ml[2 * kWarps];
#pragma unroll
      for (int k = 0; k < 2 * kWarps; ++k) {
        ml[k] = mine >> k & 1u ? *reinterpret_cast<const float2*>(piece_at(k) + col * C::kOStride + D)
                               : make_float2(-INFINITY, 0.f);
        sum.m = fmaxf(sum.m, ml[k].x);
      }
#pragma unroll
      for (int k = 0; k < 2 * kWarps; ++k)
        if (mine >> k & 1u) sum.add(ml[k], *reinterpret_cast<const float4*>(piece_at(k) + col * C::kOStride + d));
      if (whole) {
        sum.store(p, out_at(p, u.first, u.kvh, u.row0 + col) + d, vscale);
      } else {
        __stcg(reinterpret_cast<float4*>(part + col * C::kOStride + d), sum.o);
        if (d == 0) __stcg(reinterpret_cast<float2*>(part + col * C::kOStride + D), make_float2(sum.m, sum.l));
      }
    }
    if (!whole) {
      if (begun) open1 = u;
      else open0 = u;
    }
    i = next;
  }
  if (open0.unit < 0 && open1.unit < 0) return;

  // ---- join the CTAs' parts of a unit, in the last CTA to arrive
  __syncthreads();
  if (tid < 2) {
    const Piece u = tid ? open1 : open0;
    s_last[tid] = 0;
    if (u.unit >= 0) {
      const int c0 = u.unit / cta_share, c1 = (u.unit + u.steps - 1) / cta_share;
      __threadfence();  // the CTA's stores, seen through the barrier, before the arrival
      s_last[tid] = atomicAdd(p.counters + c0, 1u) == static_cast<unsigned>(c1 - c0);
      if (s_last[tid]) {
        p.counters[c0] = 0u;
        __threadfence();
      }
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    if (!s_last[which]) continue;
    const Piece u = which ? open1 : open0;
    const int c0 = u.unit / cta_share, parts = (u.unit + u.steps - 1) / cta_share - c0 + 1;
    for (int item = tid; item < u.rows * (D / 4); item += kThreads) {
      const int col = item / (D / 4), d = 4 * (item % (D / 4));
      // part 0 is the second place of CTA c0, part k the first of CTA c0 + k
      const float* src = p.partial + 2 * static_cast<size_t>(c0) * C::kPiece + col * C::kOStride;
      Joined sum;
#pragma unroll 8
      for (int k = 0; k < parts; ++k)
        sum.m = fmaxf(sum.m, __ldcg(src + (k ? 2 * k : 1) * static_cast<size_t>(C::kPiece) + D));
#pragma unroll 4
      for (int k = 0; k < parts; ++k) {
        const float* s = src + (k ? 2 * k : 1) * static_cast<size_t>(C::kPiece);
        sum.add(__ldcg(reinterpret_cast<const float2*>(s + D)), __ldcg(reinterpret_cast<const float4*>(s + d)));
      }
      sum.store(p, out_at(p, u.first, u.kvh, u.row0 + col) + d, vscale);
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
  using C = Small<D, NT>;
  const long long most = 2LL * p.batch * p.num_kv_heads *
                         ((static_cast<long long>(p.max_blocks) * p.per_block + C::kStep - 1) / C::kStep);
  const long long ctas = std::min<long long>((most + C::kWarps - 1) / C::kWarps, few_rows_ctas(NT, num_sms));
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(C::kThreads), Small<D, NT>::kSmem, stream, p);
}

template <int KIND, int D>
cudaError_t launch_kind(const Kv4AttnParams& p, int num_sms, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.share) * p.max_query_len;
  if (rows <= 8) return launch_few<KIND, D, 1>(p, num_sms, stream);
  return launch_few<KIND, D, 2>(p, num_sms, stream);
}

}  // namespace

size_t kv4_attention_workspace(int share, long long max_query_len, int head_dim, int num_sms) {
  if (share * max_query_len > kSmallRows) return kv4_prompt_workspace(head_dim, num_sms);
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
  if (e != cudaSuccess) return e;
  e = read_clear_kv4_prompt_status(&v);
  *flags |= v;
  return e;
}

cudaError_t launch_kv4_attention(const Kv4AttnParams& args, int num_sms, void* workspace, cudaStream_t stream) {
  Kv4AttnParams p = args;
  p.counters = static_cast<unsigned*>(workspace);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCounterBytes);
  p.share = p.num_q_heads / p.num_kv_heads;
  p.per_block = p.block_size / kKv4Tokens;
  p.block_shift = -1;
  for (int i = 0; i < 31; ++i)
    if ((1 << i) == p.per_block) p.block_shift = i;
  if (static_cast<long long>(p.share) * p.max_query_len > kSmallRows) return launch_kv4_prompt(p, num_sms, stream);
  if (p.head_dim == 64)
    return p.kind == W8A8_KV4_E2M1 ? launch_kind<W8A8_KV4_E2M1, 64>(p, num_sms, stream)
                                   : launch_kind<W8A8_KV4_INT4, 64>(p, num_sms, stream);
  return p.kind == W8A8_KV4_E2M1 ? launch_kind<W8A8_KV4_E2M1, 128>(p, num_sms, stream)
                                 : launch_kind<W8A8_KV4_INT4, 128>(p, num_sms, stream);
}

}  // namespace w8a8
