// kv4_prompt.cu -- attention over the 4-bit KV cache, many rows a request
// (prompts, prompt chunks, long drafts; sm_103a).
//
// The rows of a request and KV head are its n new tokens times the G query
// heads that share the KV head (row r: token r / G, head r % G), so that each
// decoded K and V serves all of them.  Both products run on the 5th-generation
// tensor cores with f16 operands and fp32 accumulators in TMEM:
//   S[128 rows x 128 tokens] = Q[128 x D] . K^T     (Q, K in shared memory)
//   O[128 rows x D]         += P[128 x 128] . V     (P in TMEM, over S; V in
//                                                    shared memory as it lies,
//                                                    dims contiguous)
// The decoded cache is exact in f16; a row of Q is scaled by a power of two
// before its conversion; the weights are f16(2^(s - m + 13)), with the maximum
// m raised (and O rescaled) only when a score passes it by 2^2.  The sum that
// divides is of the weights in fp32, each off by at most 2^-11 of itself from the
// one in the product: widening the rounded ones again would lengthen the softmax,
// which is what bounds this kernel (few rows get their sum from one more MMA).
//
// One CTA to an SM, 22 warps: two slots of 8 softmax warps, one warp that
// copies the codes, four that decode K and V into swizzled tiles two deep, one
// that issues the MMAs.  While one slot is at its softmax the tensor cores work
// for the other; the MMA warp serves them strictly in turn, which keeps them
// out of step (serving whichever is ready let their softmaxes collide: 920 us
// for 781 at 2 x 4000 new tokens).  With more than 128 rows the slots take 128
// rows each of the same tokens; with fewer both take the same rows, and the
// token tiles in turn, and their states are joined at the end.  Two threads
// share a softmax row, 64 tokens each: a tile's softmax is a chain of latencies,
// and halves (907 -> 801 us).  Its maximum comes with the TMEM load itself.
// The loops are kept short: together they have to fit the instruction cache
// (unrolled ones ran half as fast).
//
// Per 128 tokens and 256 rows the MMAs take 4 x 512 cycles (at 8192 flops a
// cycle) and the shared memory about 2300 for their operands and the decoded
// tiles; a turn takes about 4200: what bounds it now is the chain of one slot,
// softmax (1800) - product with V - next scores - softmax, as S and P share their
// TMEM columns (P fills half of them; scores into the other half meanwhile were not
// tried).  2 x 4000 new tokens after 4200, 32 query and 8 KV heads of 128: 801 us,
// 1.01 PFLOP/s, 52 % of the 1.97 that a bf16 matrix product reaches; heads of 64:
// 641 us, 0.63 PFLOP/s.
//
// A unit is one request, KV head and 256 rows; its work is the token tiles up
// to the last one that its last row sees.  All units' tiles in a row are cut
// into equal runs, one for each CTA; a cut unit leaves a part in the workspace
// from each of its CTAs, joined by the last to arrive, in their order.
#include <algorithm>

#include "internal.h"
#include "kv4.cuh"
#include "sm103_ptx.cuh"

namespace w8a8 {

namespace {

constexpr int kTileRows = 128, kTileTokens = 128;
constexpr int kUnitRows = 2 * kTileRows;
constexpr int kSoftmaxThreads = 512;                   // two slots of 8 warps, two threads to a row
constexpr int kSlotThreads = kSoftmaxThreads / 2;
constexpr int kDecodeThreads = 128;
constexpr int kDecodeWarp = kSoftmaxThreads / 32, kMmaWarp = kDecodeWarp + kDecodeThreads / 32, kCopyWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kCopyWarp + 1);
constexpr int kRaw = 3;                                // halves (K or V of a tile) of codes in flight
constexpr int kStages = 2;
constexpr int kRecords = kTileTokens / kKv4Tokens;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kHeadroom = 2.f;
constexpr float kNoScore = -1e25f;
// Scores (in the log2 domain) up to which a weight's exponent is one FMA,
// s cs + (13 - m cs): the rounding of m cs moves all weights of a row by the same
// 2^-9 at most.  From 2^26 on it would push them out of f16.
constexpr float kFar = 65536.f;
constexpr int kMaxCounters = 1024;
constexpr uint32_t kTmemCols = 512;

template <int D>
struct Big {
  static constexpr int kHalves = D / 64;                        // 128-byte column blocks of a row
  static constexpr int kBlockBytes = 128 * 128;                 // 128 rows x 128 bytes
  static constexpr int kTileBytes = kHalves * kBlockBytes;      // a Q, K or V tile
  static constexpr int kQ = 0, kK = 2 * kTileBytes, kV = kK + kStages * kTileBytes;
  static constexpr int kHalf = kv4_record_bytes(D) / 2;         // K or V of a record, codes and scales
  static constexpr int kCodes = kV + kStages * kTileBytes, kSmem = kCodes + kRaw * kRecords * kHalf + 1024;  // + alignment
  static constexpr int kPart = kUnitRows * (D + 2);             // floats: o [D / 4][256][4], m [256], l [256]
  static constexpr int kPieces = kTileTokens * D / 2 / 16 / kDecodeThreads;  // 16-byte pieces of K a thread decodes
};

struct Request {
  int first, n, all, len, rows;  // all: its new tokens, n: those looked at (fewer past max_query_len)
};

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
  r.rows = r.n * p.share;
  return r;
}

// Token tiles of row block `rt` of a request: up to the last token that its
// last row sees, at least one (to write the zeros of rows that see none); 0
// past its rows.
__device__ __forceinline__ int tiles_of(const Kv4AttnParams& p, const Request& r, int rt) {
  if (rt * kUnitRows >= r.rows) return 0;
  const int last = min(r.rows, (rt + 1) * kUnitRows) - 1;
  const int seen = min(r.len, max(0, r.len - r.all + last / p.share + 1));
  return max(1, (seen + kTileTokens - 1) / kTileTokens);
}

// A place in the row of all units' tiles.
struct Cursor {
  int b, rt, kvh;
  Request rq;
  int tiles;  // of the unit
  int tile;   // the next one
  __device__ __forceinline__ void next_unit(const Kv4AttnParams& p) {
    tile = 0;
    if (++kvh < p.num_kv_heads) return;
    kvh = 0;
    ++rt;
    while ((tiles = tiles_of(p, rq, rt)) == 0) {
      rt = 0;
      rq = request_of(p, ++b);
    }
  }
};

__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 numbers in one register pair, and their arithmetic.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory"); }

// The 8 warps of a slot, the two warps that share 32 rows.
__device__ __forceinline__ void slot_sync(int slot) {
  asm volatile("bar.sync %0, %1;" ::"r"(2 + slot), "n"(kSlotThreads) : "memory");
}
__device__ __forceinline__ void rows_sync(int slot, int quarter) {
  asm volatile("bar.sync %0, 64;" ::"r"(4 + 4 * slot + quarter) : "memory");
}

// Whether a warp's wait ended well: the same answer in every lane, since what
// follows is done by the whole warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

__device__ __forceinline__ float2 to_float2(uint32_t two, int fp16) {
  return fp16 ? __half22float2(*reinterpret_cast<const __half2*>(&two))
              : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&two));
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// A value that all lanes share, known as such to the compiler.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// 8 16-bit values at `src` (null: zeros).
__device__ __forceinline__ uint4 load8(const uint16_t* src, int vec) {
  if (!src) return make_uint4(0u, 0u, 0u, 0u);
  if (vec) return __ldg(reinterpret_cast<const uint4*>(src));
  uint32_t u[4];
#pragma unroll
  for (int x = 0; x < 4; ++x)
    u[x] = static_cast<uint32_t>(__ldg(src + 2 * x)) | (static_cast<uint32_t>(__ldg(src + 2 * x + 1)) << 16);
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// 8 consecutive outputs.
__device__ __forceinline__ void store8(const Kv4AttnParams& p, size_t at, const float (&y)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (p.out_fp16) {
      w[i] = as_u32(__floats2half2_rn(y[2 * i], y[2 * i + 1]));
    } else {
      const __nv_bfloat162 x = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&x);
    }
  }
  uint16_t* dst = static_cast<uint16_t*>(p.out) + at;
  if (p.out_vec) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dst[2 * i] = static_cast<uint16_t>(w[i]);
      dst[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
    }
  }
}

__device__ __forceinline__ size_t out_at(const Kv4AttnParams& p, int first, int kvh, int row) {
  return (first + row / p.share) * p.out_token_stride + (kvh * p.share + row % p.share) * p.out_head_stride;
}

// A unit that goes on in other CTAs.
struct Open {
  int first, rows, row0, kvh;
  long long unit;  // its first tile; -1: none
  int tiles;
};

// A unit whose results are still to be written.
struct Ended {
  int first, rows, row0, kvh, tiles;
  bool whole, begun, pair, both;
};

template <int KIND, int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_prompt_kernel(const Kv4AttnParams p) {
  using C = Big<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t s_kfull[kStages], s_kempty[kStages], s_vfull[kStages], s_vempty[kStages];
  __shared__ uint64_t s_rfull[kRaw], s_rempty[kRaw];
  __shared__ uint8_t s_live[kRaw];  // which of a half's records lie in the cache
  __shared__ uint64_t s_qfull, s_sfull[2], s_pfull[2], s_pvdone[2];
  __shared__ uint32_t s_tmem;
  __shared__ long long s_scan[kThreads / 32], s_before;
  __shared__ int s_item, s_last[2];
  __shared__ Open s_open[2];  // the unit begun in front of this CTA, the one begun here
  __shared__ float s_cs[2][kTileRows];         // scale of each row's scores
  __shared__ float s_mx[2][2][2][kTileRows];   // largest score: tile's parity, slot, half of the tokens
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&s_kfull[i]), kDecodeThreads / 32);
      mbar_init(smem_addr(&s_vfull[i]), kDecodeThreads / 32);
      mbar_init(smem_addr(&s_kempty[i]), 1);
      mbar_init(smem_addr(&s_vempty[i]), 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(smem_addr(&s_rfull[i]), kRecords);
      mbar_init(smem_addr(&s_rempty[i]), kDecodeThreads / 32);
    }
    mbar_init(smem_addr(&s_qfull), kSoftmaxThreads / 32);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&s_sfull[i]), 1);
      mbar_init(smem_addr(&s_pfull[i]), kSlotThreads / 32);
      mbar_init(smem_addr(&s_pvdone[i]), 1);
    }
    fence_barrier_init();
  }
  if (tid < 2) s_open[tid].unit = -1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // TMEM only now: a kernel in front may still need it.  Dependents start only
  // when it is taken: one that took it first and then waited for this kernel's
  // end would never see it.
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&s_tmem), kTmemCols);
    tmem_relinquish();
  }

  // ---- this CTA's run; an item is one request and row block, all KV heads
  const int blocks_max = static_cast<int>((static_cast<long long>(p.share) * p.max_query_len + kUnitRows - 1) / kUnitRows);
  const int items = p.batch * blocks_max;  // below 2^31, the launcher sees to it
  long long total = 0, share;
  {
    const int per = (items + kThreads - 1) / kThreads;
    const int i0 = min(items, tid * per), i1 = min(items, i0 + per);
    long long mine = 0;
#pragma unroll 1
    for (int i = i0; i < i1; ++i)
      mine += static_cast<long long>(tiles_of(p, request_of(p, i / blocks_max), i % blocks_max)) * p.num_kv_heads;
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
    share = max(1LL, (total + gridDim.x - 1) / gridDim.x);
    const long long at = share * blockIdx.x;
    if (at >= run && at < run + mine) {
#pragma unroll 1
      for (int i = i0; i < i1; ++i) {
        const long long w = static_cast<long long>(tiles_of(p, request_of(p, i / blocks_max), i % blocks_max)) * p.num_kv_heads;
        if (at < run + w) {
          s_item = i;
          s_before = run;
          break;
        }
        run += w;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = s_tmem;
  const long long r0 = share * blockIdx.x;
  const int run_tiles = static_cast<int>(max(0LL, min(total - r0, min(share, 0x7fffffffLL))));
  Cursor at;
  if (run_tiles > 0) {
    at.b = s_item / blocks_max;
    at.rt = s_item % blocks_max;
    at.rq = request_of(p, at.b);
    at.tiles = tiles_of(p, at.rq, at.rt);
    at.kvh = static_cast<int>((r0 - s_before) / at.tiles);
    at.tile = static_cast<int>((r0 - s_before) % at.tiles);
  }
  bool ok = true;

  if (run_tiles == 0) {
    // nothing to do
  } else if (warp >= kDecodeWarp && warp < kMmaWarp) {
    // ================= decoding: thread (token, piece) of each 16-byte piece of codes
    const int dt = tid - kSoftmaxThreads;
    constexpr int kPerRow = D / 32;                       // pieces of a token's row
    constexpr int kStride = kDecodeThreads / kPerRow;     // tokens between a thread's pieces
    const int piece = dt % kPerRow, token0 = dt / kPerRow;
    const uint32_t base = smem_addr(smem);
    // the second block's lanes store their words in another order: the eight
    // lanes of a store then meet eight different bank groups
    const bool turn = D == 128 && piece >= 2;
    // half h of the run: the keys (even) or values (odd) of tile h / 2
#pragma unroll 1
    for (int h = 0; h < 2 * run_tiles; ++h) {
      const int j = h / 2, w = h & 1, stage = j % kStages, slot = h % kRaw;
      if (!(ok = warp_wait(smem_addr(&s_rfull[slot]), (h / kRaw) & 1))) break;
      const uint8_t* half = smem + C::kCodes + slot * kRecords * C::kHalf;
      const uint32_t live = s_live[slot];
      const int end = at.rq.len - at.tile * kTileTokens;
      uint4 raw[C::kPieces];
      uint32_t sc[C::kPieces];
#pragma unroll
      for (int x = 0; x < C::kPieces; ++x) {
        const int token = token0 + x * kStride, row = token % kKv4Tokens;
        const uint8_t* rec = half + token / kKv4Tokens * C::kHalf;
        raw[x] = *reinterpret_cast<const uint4*>(rec + row * (D / 2) + 16 * piece);
        // what is not a token of the request becomes zeros, whatever the cache holds there
        sc[x] = token < end && (live >> (token / kKv4Tokens) & 1u)
                    ? *reinterpret_cast<const uint16_t*>(rec + kv4_scales_at(D, 0) + row * (D / 16) + 2 * piece)
                    : 0u;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&s_rempty[slot]));
      if (j >= kStages) ok = warp_wait(smem_addr(w ? &s_vempty[stage] : &s_kempty[stage]), ((j / kStages) & 1) ^ 1u);
      if (!ok) break;
      const uint32_t tile = base + (w ? C::kV : C::kK) + stage * C::kTileBytes + (D == 128 ? piece / 2 : 0) * C::kBlockBytes;
#pragma unroll
      for (int x = 0; x < C::kPieces; ++x) {
        const int token = token0 + x * kStride;
        const __half2 s = e4m3x2_to_half2(sc[x]);
        const Kv4Scale s0 = kv4_scale<KIND>(turn ? __high2half2(s) : __low2half2(s));
        const Kv4Scale s1 = kv4_scale<KIND>(turn ? __low2half2(s) : __high2half2(s));
        const uint32_t word[4] = {turn ? raw[x].z : raw[x].x, turn ? raw[x].w : raw[x].y, turn ? raw[x].x : raw[x].z,
                                  turn ? raw[x].y : raw[x].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t v[4];
          kv4_decode8<KIND>(word[i], i < 2 ? s0 : s1, v);
          const int chunk = (piece % 2) * 4 + (turn ? i ^ 2 : i);
          st_shared_v4(tile + token * 128 + ((chunk ^ (token & 7)) << 4), v[0], v[1], v[2], v[3]);
        }
      }
      fence_proxy_async_shared();  // the stores before the tensor cores' reads
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(w ? &s_vfull[stage] : &s_kfull[stage]));
      if (w && h + 1 < 2 * run_tiles && ++at.tile == at.tiles) at.next_unit(p);
    }
  } else if (warp == kCopyWarp) {
    // ================= copies: lane x has record x of the tile
    const uint32_t codes = smem_addr(smem) + C::kCodes + lane * C::kHalf;
    auto look_up = [&]() -> long long {
      const int tile = at.tile * kRecords + lane;
      if (lane >= kRecords || tile >= (at.rq.len + kKv4Tokens - 1) / kKv4Tokens) return -1;
      const int page = p.block_shift >= 0 ? tile >> p.block_shift : tile / p.per_block;
      const int blk = __ldg(p.block_table + static_cast<size_t>(at.b) * p.max_blocks + page);
      if (blk < 0 || blk >= p.num_blocks) return -1;
      return (static_cast<long long>(blk) * p.num_kv_heads + at.kvh) * p.per_block + (tile - page * p.per_block);
    };
    long long next = look_up(), rec = -1;
#pragma unroll 1
    for (int h = 0; h < 2 * run_tiles; ++h) {
      const int slot = h % kRaw;
      if (!(h & 1)) {
        rec = next;
        if (h + 2 < 2 * run_tiles) {  // the next tile's places, while this one's are copied
          if (++at.tile == at.tiles) at.next_unit(p);
          next = look_up();
        }
      }
      if (h >= kRaw && !(ok = warp_wait(smem_addr(&s_rempty[slot]), ((h / kRaw) & 1) ^ 1u))) break;
      const uint32_t live = __ballot_sync(0xffffffffu, rec >= 0);
      if (lane == 0) s_live[slot] = static_cast<uint8_t>(live);
      __syncwarp();
      if (lane < kRecords) {
        const uint32_t full = smem_addr(&s_rfull[slot]);
        fence_proxy_async_shared();  // the reads of the slot's last half before the copies over it
        if (rec >= 0) {
          mbar_arrive_expect_tx(full, C::kHalf);
          bulk_load(codes + slot * kRecords * C::kHalf,
                    static_cast<const uint8_t*>(p.cache) + rec * kv4_record_bytes(D) + (h & 1) * C::kHalf, C::kHalf, full);
        } else {
          mbar_arrive(full);
        }
      }
    }
    // a wait gave up: the copies in flight land before shared memory is released
    if (!ok)
      for (int i = 0; i < kRaw; ++i) mbar_wait(smem_addr(&s_rfull[i]), 0), mbar_wait(smem_addr(&s_rfull[i]), 1);
  } else if (warp == kMmaWarp) {
    // ================= MMAs: the warp runs converged on uniform values, one lane issues
    const uint32_t leader = elect_one();
    constexpr uint32_t kIdescS = make_idesc(kTileRows, kTileTokens, 0);
    constexpr uint32_t kIdescO = make_idesc(kTileRows, D, 0) | (1u << 16);  // V: dims contiguous
    const uint32_t tm = uniform(tmem);
    const uint64_t dq = smem_desc_sw128(smem_addr(smem) + C::kQ), dk = smem_desc_sw128(smem_addr(smem) + C::kK);
    const uint64_t dv = smem_desc_mn_sw128(smem_addr(smem) + C::kV, C::kBlockBytes);
    const int all = uniform(run_tiles);
    uint32_t pcount[2] = {0u, 0u};  // weight tiles taken, each slot
    int done = 0, units = 0;
    auto scores = [&](int tile, int slot, int q) {
      const int stage = tile % kStages;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk / 4) * (C::kBlockBytes >> 4) + 2 * (kk % 4);
        mma_f16_by(leader, tm + slot * kTileTokens, dq + q * (C::kTileBytes >> 4) + off,
                   dk + stage * (C::kTileBytes >> 4) + off, kIdescS, kk > 0);
      }
      mma_commit_by(leader, smem_addr(&s_sfull[slot]));
    };
    auto wait_k = [&](int tile) {
      if (ok) ok = warp_wait(smem_addr(&s_kfull[tile % kStages]), (tile / kStages) & 1);
      tc_fence_after();
    };
#pragma unroll 1
    while (done < all && ok) {
      const int nt = uniform(min(at.tiles - at.tile, all - done));
      const bool pair = uniform(at.rq.rows - at.rt * kUnitRows > kTileRows);
      const int ahead = pair ? 1 : 2;
      ok = warp_wait(smem_addr(&s_qfull), units & 1);
      tc_fence_after();
#pragma unroll 1
      for (int j = 0; j < ahead && j < nt && ok; ++j) {
        wait_k(done + j);
        if (!ok) break;
        for (int slot = pair ? 0 : j; slot < (pair ? 2 : j + 1) && ok; ++slot) {
          const uint32_t c = slot ? pcount[1] : pcount[0];
          if (c > 0) ok = warp_wait(smem_addr(&s_pvdone[slot]), (c - 1) & 1);
        }
        if (!ok) break;
#pragma unroll 1
        for (int slot = pair ? 0 : j; slot < (pair ? 2 : j + 1); ++slot) scores(done + j, slot, pair ? slot : 0);
        mma_commit_by(leader, smem_addr(&s_kempty[(done + j) % kStages]));
      }
#pragma unroll 1
      for (int j = 0; j < nt && ok; ++j) {
        const int stage = (done + j) % kStages;
        const bool more = j + ahead < nt;
        ok = warp_wait(smem_addr(&s_vfull[stage]), ((done + j) / kStages) & 1);
#pragma unroll 1
        for (int slot = pair ? 0 : j & 1, end = pair ? 2 : slot + 1; slot < end && ok; ++slot) {
          const uint32_t parity = (slot ? pcount[1] : pcount[0]) & 1u;
          if (slot) ++pcount[1];
          else ++pcount[0];
          if (!(ok = warp_wait(smem_addr(&s_pfull[slot]), parity))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kTileTokens / 16; ++kk)
            mma_f16_ts_by(leader, tm + 2 * kTileTokens + slot * D, tm + slot * kTileTokens + 64 * (kk / 4) + 8 * (kk % 4),
                          dv + stage * (C::kTileBytes >> 4) + kk * (2048 >> 4), kIdescO, kk > 0 || j >= ahead);
          mma_commit_by(leader, smem_addr(&s_pvdone[slot]));
          if (more) {
            if (slot == 0 || !pair) wait_k(done + j + ahead);
            // the scores overwrite the weights
            if (ok) ok = warp_wait(smem_addr(&s_pvdone[slot]), parity);
            if (ok) scores(done + j + ahead, slot, pair ? slot : 0);
          }
        }
        mma_commit_by(leader, smem_addr(&s_vempty[stage]));
        if (more) mma_commit_by(leader, smem_addr(&s_kempty[(done + j + ahead) % kStages]));
      }
      done += nt;
      ++units;
      at.tile += nt;
      if (done < all) at.next_unit(p);
    }
  } else {
    // ================= softmax: thread = row of slot `slot` and half of its tokens (or dims)
    const int slot = warp / 8, half = warp / 4 % 2, quarter = warp % 4, row = 32 * quarter + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter) << 21);  // this warp's 32 TMEM lanes
    const uint32_t s_cols = lanes + slot * kTileTokens, o_cols = lanes + 2 * kTileTokens + slot * D + half * (D / 2);
    const float vscale = kv4_out_scale(p.sm_scale, p.k_scale, p.v_scale), to_log2 = p.sm_scale * __ldg(p.k_scale) * kLog2e;
    uint32_t count = 0u;  // tiles of this slot
    int done = 0;
    // the unit before, whose results are written when the next one's query is on its way
    Ended old;
    old.tiles = 0;
    float m = kNoScore, l = 0.f, cs = 0.f;
    int mine = 0;  // tiles of this slot in the unit
#pragma unroll 1
    while (true) {
      const bool more = done < run_tiles;
      const int nt = more ? min(at.tiles - at.tile, run_tiles - done) : 0;
      const Request rq = at.rq;
      const int row0 = at.rt * kUnitRows;
      const bool pair = rq.rows - row0 > kTileRows;
      const int top = row0 + (pair ? slot * kTileRows : 0);  // the request's row in this slot's row 0
      const int my = top + row;
      const bool real = my < rq.rows;

      // both slots' last scores are there: the query may go.  With pairs that holds
      // for the warp's own slot already, but s_cs is another warp's to read: all of
      // the slot have taken the old unit's scales before one writes the next unit's
      // (a unit of one tile has no other wait between the two)
      if (old.tiles > 0) {
        if (old.pair) slot_sync(slot);
        else softmax_sync();
      }
      // ---- the warp's 16 query rows, a 16-byte piece for each lane, scaled by
      // 2^e so that a row's largest element lies in [2^14, 2^15); infinities stay
      if (more && (pair || slot == 0)) {
        constexpr int kPerRow = D / 8, kAtOnce = 32 / kPerRow;  // pieces of a row, rows of one load
        constexpr int kBatch = 4;                               // loads in flight
        const int c = lane % kPerRow, wrow = 16 * (warp % 8) + lane / kPerRow;
        const uint32_t dst = smem_addr(smem) + C::kQ + slot * C::kTileBytes + (c / 8) * C::kBlockBytes;
#pragma unroll 1
        for (int i0 = 0; i0 < 16 / kAtOnce; i0 += kBatch) {
          uint4 raw[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int r = top + wrow + (i0 + i) * kAtOnce;
            raw[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < rq.rows)
              raw[i] = load8(static_cast<const uint16_t*>(p.q) + (rq.first + r / p.share) * p.q_token_stride +
                                 (at.kvh * p.share + r % p.share) * p.q_head_stride + 8 * c,
                             p.q_vec);
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int r = wrow + (i0 + i) * kAtOnce;
            const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            float v[8], qmax = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 x = to_float2(u[k], p.q_fp16);
              v[2 * k] = x.x;
              v[2 * k + 1] = x.y;
              qmax = fmaxf(qmax, fmaxf(fabsf(x.x), fabsf(x.y)));
            }
#pragma unroll
            for (int off = 1; off < kPerRow; off <<= 1) qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, off));
            int e = 0;
            if (qmax > 0.f) e = min(100, 14 + 127 - static_cast<int>(__float_as_uint(qmax) >> 23));
            const float down = to_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            // the scale's sign goes to the query: the largest product is the largest score
            const float up = copysignf(__uint_as_float(static_cast<uint32_t>(127 + e) << 23), down);
            if (c == 0) s_cs[slot][r] = fmaxf(fabsf(down), 1e-37f);
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              h[k] = as_u32(__floats2half2_rn(v[kv4_low<KIND>(k)] * up, v[kv4_high<KIND>(k)] * up));
            st_shared_v4(dst + r * 128 + (((c % 8) ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
          }
        }
        fence_proxy_async_shared();
      }
      __syncwarp();
      if (more && lane == 0) mbar_arrive(smem_addr(&s_qfull));

      // ---- the results of the unit before
      if (old.tiles > 0) {
        if (mine > 0 && ok) ok = warp_wait(smem_addr(&s_pvdone[slot]), (count - 1) & 1);
        // sums by slot and half, and slot 1's maximum, where nobody reads scores any
        // more (with pairs the buffer that the next tile does not write to)
        float (&s_l)[2][2][kTileRows] = s_mx[old.pair ? (count + 1) & 1 : 0];
        float (&s_m)[kTileRows] = s_mx[1][0][0];
        s_l[slot][half][row] = l;
        if (!old.pair && half == 0 && slot == 1) s_m[row] = m * cs;
        tc_fence_before();
        if (old.pair) rows_sync(slot, quarter);
        else softmax_sync();
        tc_fence_after();
        float a0 = 1.f, a1 = 0.f;  // this slot's factor, the other's
        l = s_l[slot][0][row] + s_l[slot][1][row];
        // a sum of 0: nothing seen.  A NaN goes on into the row's results
        float ms = l != 0.f ? m * cs : -INFINITY;
        if (!old.pair && slot == 0) {
          const float l1 = s_l[1][0][row] + s_l[1][1][row], m1 = l1 != 0.f ? s_m[row] : -INFINITY;
          const float mn = fmaxf(ms, m1);
          a0 = l != 0.f ? ex2_fast(ms - mn) : 0.f;
          a1 = l1 != 0.f ? ex2_fast(m1 - mn) : 0.f;
          ms = mn;
          l = a0 * l + a1 * l1;
        }
        if (old.pair || slot == 0) {
          const float inv = l != 0.f ? vscale / l : 0.f;
          const int prow = row + (old.pair ? slot * kTileRows : 0), r = old.row0 + prow;
          const bool real_row = r < old.rows;
          const size_t to = real_row ? out_at(p, old.first, old.kvh, r) + half * (D / 2) : 0;
          float* part = p.partial + (2 * static_cast<size_t>(blockIdx.x) + old.begun) * C::kPart;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[16];
            float y[16];
            tmem_ld16(o_cols + 16 * c, o);
            tmem_ld_wait();
            tmem_loaded(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = l != 0.f ? __uint_as_float(o[i]) * a0 : 0.f;
            if (old.both) {
              tmem_ld16(o_cols + D + 16 * c, o);
              tmem_ld_wait();
              tmem_loaded(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = l != 0.f ? fmaf(__uint_as_float(o[i]), a1, y[i]) : 0.f;
            }
            if (!old.whole) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                __stcg(reinterpret_cast<float4*>(part) + (half * (D / 8) + 4 * c + q) * kUnitRows + prow,
                       make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]));
            } else if (real_row) {
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                float z[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  z[kv4_low<KIND>(i)] = y[8 * q + 2 * i] * inv;
                  z[kv4_high<KIND>(i)] = y[8 * q + 2 * i + 1] * inv;
                }
                store8(p, to + 16 * c + 8 * q, z);
              }
            }
          }
          if (!old.whole && half == 0) {
            __stcg(part + kUnitRows * D + prow, ms);
            __stcg(part + kUnitRows * (D + 1) + prow, l);
          }
        }
        tc_fence_before();
        if (!old.pair) softmax_sync();  // slot 1's accumulators and the states have been read
      }
      if (!more) break;
      if (pair) slot_sync(slot);
      else softmax_sync();
      cs = s_cs[pair ? slot : 0][row];
      const int lim = real ? rq.len - rq.all + my / p.share : rq.len - 1;  // the last token seen
      const float room = fminf(kHeadroom / cs, 1e38f);
      m = kNoScore;
      l = 0.f;
      mine = 0;

      // ---- its tiles
#pragma unroll 1
      for (int j = pair ? 0 : slot; j < nt; j += pair ? 1 : 2) {
        const int t0 = (at.tile + j) * kTileTokens + half * 64;  // this thread's 64 tokens
        // records that lie outside the cache: lane x looks record x up
        bool gone = false;
        {
          const int tile = (at.tile + j) * kRecords + lane;
          if (lane < kRecords && tile < (rq.len + kKv4Tokens - 1) / kKv4Tokens) {
            const int page = p.block_shift >= 0 ? tile >> p.block_shift : tile / p.per_block;
            const int blk = __ldg(p.block_table + static_cast<size_t>(at.b) * p.max_blocks + page);
            gone = blk < 0 || blk >= p.num_blocks;
          }
        }
        const uint32_t holes = __ballot_sync(0xffffffffu, gone) >> (4 * half);
        const bool edge = __any_sync(0xffffffffu, t0 + 63 > lim) || (holes & 15u);
        // (a wait that gave up ends no loop here: the barriers below want every warp)
        if (ok) ok = warp_wait(smem_addr(&s_sfull[slot]), count & 1);
        tc_fence_after();
        const uint32_t cols = s_cols + half * 64;
        if (edge) {
          // what a row does not see, written back as -infinity: rare, and apart
          // from the loops below, whose code has to stay in the instruction cache
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t s[16];
            tmem_ld16(cols + 16 * c, s);
            tmem_ld_wait();
            tmem_loaded(s);
            const int seen = holes >> c & 1u ? 0 : lim + 1 - t0 - 16 * c;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i >= seen) s[i] = __float_as_uint(-INFINITY);
            tmem_st16(cols + 16 * c, s);
          }
          tmem_st_wait();
        }
        // the maximum first, found by the load itself, then the weights
        float mx = kNoScore;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t s[32], big;
          tmem_ld32_max(cols + 32 * c, s, big);
          tmem_ld_wait();
          tmem_loaded(s);
          asm volatile("" : "+r"(big));
          mx = fmaxf(mx, __uint_as_float(big));
        }
        s_mx[count & 1][slot][half][row] = mx;
        rows_sync(slot, quarter);
        mx = fmaxf(mx, s_mx[count & 1][slot][half ^ 1][row]);
        if (__any_sync(0xffffffffu, mx > m + room)) {
          const float mn = fmaxf(m, mx);
          const float alpha = ex2_fast((m - mn) * cs);
          m = mn;
          l *= alpha;
          if (mine > 0) {
            if (ok) ok = warp_wait(smem_addr(&s_pvdone[slot]), (count - 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[16];
              tmem_ld16(o_cols + 16 * c, o);
              tmem_ld_wait();
              tmem_loaded(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st16(o_cols + 16 * c, o);
            }
            tmem_st_wait();
          }
        }
        // the tokens' weights, over this half's scores as they are read
        float bias = fmaf(-m, cs, 15.f - kHeadroom);
        if (__builtin_expect(__any_sync(0xffffffffu, fabsf(bias) > kFar), 0)) {
          // s - m in place of far scores s: rare, and apart as above (subtracting in
          // the loop below: 816 us, with this branch 808, without either 798)
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t s[16];
            tmem_ld16(cols + 16 * c, s);
            tmem_ld_wait();
            tmem_loaded(s);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = __float_as_uint(__uint_as_float(s[i]) - m);
            tmem_st16(cols + 16 * c, s);
          }
          tmem_st_wait();
          bias = 15.f - kHeadroom;
        }
        const uint64_t cs2 = pack2(cs, cs), bias2 = pack2(bias, bias);
        uint64_t sum = 0;
        auto weights = [&](const uint32_t (&s)[16], uint32_t* w) {
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            float a, b;
            unpack2(fma2(pack2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), cs2, bias2), a, b);
            a = ex2_fast(a);
            b = ex2_fast(b);
            sum = add2(sum, pack2(a, b));
            w[i / 2] = as_u32(__floats2half2_rn(a, b));
          }
        };
        uint32_t sx[16], sy[16], w[16];  // the next columns are on their way while these are worked on
        tmem_ld16(cols, sx);
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          tmem_ld_wait();
          tmem_loaded(sx);
          tmem_ld16(cols + 32 * c + 16, sy);
          weights(sx, w);
          tmem_ld_wait();
          tmem_loaded(sy);
          if (c == 0) tmem_ld16(cols + 32, sx);
          weights(sy, w + 8);
          tmem_st16(cols + 16 * c, w);
        }
        {
          float a, b;
          unpack2(sum, a, b);
          l += a + b;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&s_pfull[slot]));
        ++count;
        ++mine;
      }

      // ---- its end
      const long long unit = r0 + done - at.tile;
      old.whole = at.tile == 0 && nt == at.tiles;
      old.begun = unit / share == blockIdx.x;
      old.pair = pair;
      old.both = !pair && nt > 1;
      old.first = rq.first;
      old.rows = rq.rows;
      old.row0 = row0;
      old.kvh = at.kvh;
      old.tiles = nt;
      if (!old.whole && tid == 0) s_open[old.begun] = {rq.first, rq.rows, row0, at.kvh, unit, at.tiles};
      done += nt;
      at.tile += nt;
      if (done < run_tiles) at.next_unit(p);
    }
  }

  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid >= kSoftmaxThreads || (s_open[0].unit < 0 && s_open[1].unit < 0)) return;

  // ---- join the CTAs' parts of a unit, in the last CTA to arrive
  if (tid < 2) {
    const Open u = s_open[tid];
    s_last[tid] = 0;
    if (u.unit >= 0) {
      const long long c0 = u.unit / share, c1 = (u.unit + u.tiles - 1) / share;
      __threadfence();  // the CTA's stores, seen through the barrier, before the arrival
      s_last[tid] = atomicAdd(p.counters + c0, 1u) == static_cast<unsigned>(c1 - c0);
      if (s_last[tid]) {
        p.counters[c0] = 0u;
        __threadfence();
      }
    }
  }
  softmax_sync();
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    if (!s_last[which]) continue;
    const Open u = s_open[which];
    const int row = tid % kUnitRows, my = u.row0 + row;
    if (my >= u.rows) continue;
    const long long c0 = u.unit / share;
    const int parts = static_cast<int>((u.unit + u.tiles - 1) / share - c0) + 1;
    // part 0 is the second place of CTA c0, part k the first of CTA c0 + k
    const float* src = p.partial + 2 * static_cast<size_t>(c0) * C::kPart;
    float m = -INFINITY, l = 0.f;
#pragma unroll 4
    for (int k = 0; k < parts; ++k)
      m = fmaxf(m, __ldcg(src + (k ? 2 * k : 1) * static_cast<size_t>(C::kPart) + kUnitRows * D + row));
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
      const float* s = src + (k ? 2 * k : 1) * static_cast<size_t>(C::kPart) + kUnitRows * D + row;
      const float lk = __ldcg(s + kUnitRows);
      if (lk != 0.f) l = fmaf(ex2_fast(__ldcg(s) - m), lk, l);
    }
    const float inv = l != 0.f ? kv4_out_scale(p.sm_scale, p.k_scale, p.v_scale) / l : 0.f;
    const size_t to = out_at(p, u.first, u.kvh, my);
#pragma unroll 1
    for (int q = tid / kUnitRows; q < D / 8; q += kSoftmaxThreads / kUnitRows) {
      float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
      for (int k = 0; k < parts; ++k) {
        const float* s = src + (k ? 2 * k : 1) * static_cast<size_t>(C::kPart);
        const float mk = __ldcg(s + kUnitRows * D + row);
        const float a = mk == -INFINITY ? 0.f : ex2_fast(mk - m) * inv;
        const float4 v = __ldcg(reinterpret_cast<const float4*>(s) + (2 * q) * kUnitRows + row);
        const float4 w = __ldcg(reinterpret_cast<const float4*>(s) + (2 * q + 1) * kUnitRows + row);
        y[0] = fmaf(a, v.x, y[0]);
        y[1] = fmaf(a, v.y, y[1]);
        y[2] = fmaf(a, v.z, y[2]);
        y[3] = fmaf(a, v.w, y[3]);
        y[4] = fmaf(a, w.x, y[4]);
        y[5] = fmaf(a, w.y, y[5]);
        y[6] = fmaf(a, w.z, y[6]);
        y[7] = fmaf(a, w.w, y[7]);
      }
      float z[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[kv4_low<KIND>(i)] = y[2 * i];
        z[kv4_high<KIND>(i)] = y[2 * i + 1];
      }
      store8(p, to + 8 * q, z);
    }
  }
}

template <int KIND, int D>
cudaError_t launch_t(const Kv4AttnParams& p, int num_sms, cudaStream_t stream) {
  auto kern = kv4_prompt_kernel<KIND, D>;
  // the attribute is per function and device; setting it again is harmless
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Big<D>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min(num_sms, kMaxCounters)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Big<D>::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, kern, p)) != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

size_t kv4_prompt_workspace(int head_dim, int num_sms) {
  return kCounterRegion + static_cast<size_t>(std::min(num_sms, kMaxCounters)) * 2 * kUnitRows * (head_dim + 2) * sizeof(float);
}

cudaError_t read_clear_kv4_prompt_status(int* flags) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_status, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  e = cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int));
  *flags = v;
  return e;
}

cudaError_t launch_kv4_prompt(const Kv4AttnParams& p, int num_sms, cudaStream_t stream) {
  if (p.head_dim == 64)
    return p.kind == W8A8_KV4_E2M1 ? launch_t<W8A8_KV4_E2M1, 64>(p, num_sms, stream)
                                   : launch_t<W8A8_KV4_INT4, 64>(p, num_sms, stream);
  return p.kind == W8A8_KV4_E2M1 ? launch_t<W8A8_KV4_E2M1, 128>(p, num_sms, stream)
                                 : launch_t<W8A8_KV4_INT4, 128>(p, num_sms, stream);
}

}  // namespace w8a8
