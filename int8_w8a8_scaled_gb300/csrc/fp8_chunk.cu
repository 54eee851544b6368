// fp8_chunk.cu -- attention over the paged fp8 cache, many rows a request (prompts,
// prompt chunks, long drafts; sm_103a).
//
// The rows of a request and KV head are its n new tokens times the G query heads
// that share the KV head (row r: token r / G, head r % G), so that each K and V
// serves all of them.  Both products run on the tensor cores with f16 operands and
// fp32 accumulators in TMEM:
//   S[128 rows x 128 tokens] = Q[128 x D] . K^T     (Q, K in shared memory)
//   O[128 rows x D]         += P[128 x 128] . V     (P in TMEM, over S; V in
//                                                    shared memory as it lies,
//                                                    dims contiguous)
// e4m3 codes are exact in f16; a row of Q is scaled by a power of two before its
// conversion; the weights are f16(2^(s - m + 13)), with the maximum m raised (and O
// rescaled) only when a score passes it by 2^2.  The sum that divides is of the
// weights in fp32, each off by at most 2^-11 of itself from the one in the product.
// (e4m3 operands would need two or three parts of the query and of the weights:
// twice the rate, and as much more of it, with a longer softmax.)
//
// One CTA to an SM, 22 warps: two slots of 8 softmax warps, one that copies the codes
// by TMA, 64 tokens of K or V at a time, four that write them as swizzled f16 tiles,
// one that issues the MMAs.  While one slot is at its softmax the tensor cores work for the other; the
// MMA warp serves them strictly in turn, which keeps them out of step.  With more
// than 128 rows the slots take 128 rows each of the same tokens; with fewer both
// take the same rows, and the token tiles in turn, and their states are joined at
// the end.  Two threads share a softmax row, 64 tokens each.  The loops are kept
// short: together they have to fit the instruction cache.
//
// Measured: 2048 new tokens after 30000, 32 query and 8 KV heads of 128: 1022 us, 1.02
// PFLOP/s, 52 % of the 1.95 that a bf16 matrix product reaches.  A turn (256 rows, 128
// tokens) takes about 4700 cycles where the MMAs need 2050: what bounds it is the four
// warps that make f16 tiles (1100 cycles a quarter, most of it waiting for issue slots
// beside 16 softmax warps) together with the chain of a slot, softmax (1500) - product
// with V - next scores.  Before: codes loaded by the warps themselves 2052 us (spilled),
// three quarters in flight 1328, masks and selects in every quarter 1124.  Two of the
// four warps for K and two for V: 1098.
//
// A unit is one request, KV head and 256 rows; its work is the token tiles up to
// the last one that its last row sees.  All units' tiles in a row are cut into
// equal runs, one for each CTA; a cut unit leaves a part in the workspace from each
// of its CTAs, joined by the last to arrive, in their order.
//
// A weight of 0 does not cancel a NaN, so tokens that no row sees are written as
// zeros, and NaN codes of V in tokens that only some rows see are written as zeros
// too and put into those rows' results at the end.
#include <algorithm>

#include "fp8_paged.cuh"
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
constexpr int kRaw = 7;                                // quarters (64 tokens of K or V) of codes in flight
constexpr int kQuarter = kTileTokens / 2;
// f16 tiles: one of K, free again when the scores are made, long before the next ones are
// due; two of V.  The rest is for codes on their way.
constexpr int kKStages = 1, kVStages = 2;
constexpr int kPageTokens = 16, kRecords = kTileTokens / kPageTokens;  // tokens that surely share a block
constexpr int kDead = 0x7fffffff;
constexpr float kHeadroom = 2.f;
constexpr float kNoScore = -1e25f;
// Scores (in the log2 domain) up to which a weight's exponent is one FMA,
// s cs + (13 - m cs): the rounding of m cs moves all weights of a row by the same
// 2^-9 at most.  From 2^26 on it would push them out of f16.
constexpr float kFar = 65536.f;
constexpr uint32_t kTmemCols = 512;

template <int D>
struct Big {
  static constexpr int kHalves = D / 64;                        // 128-byte column blocks of a row
  static constexpr int kBlockBytes = 128 * 128;                 // 128 rows x 128 bytes
  static constexpr int kTileBytes = kHalves * kBlockBytes;      // a Q, K or V tile
  static constexpr int kQ = 0, kK = 2 * kTileBytes, kV = kK + kKStages * kTileBytes;
  static constexpr int kCodes = kV + kVStages * kTileBytes, kCodeBytes = kQuarter * D;
  static constexpr int kSmem = kCodes + kRaw * kCodeBytes + 1024;  // + alignment
  static constexpr int kPart = kUnitRows * (D + 2);             // floats: o [D / 4][256][4], m [256], l [256]
  static constexpr int kPieces = kQuarter * D / 16 / kDecodeThreads;  // 16-byte pieces of a quarter that a thread takes
};

struct Request : Fp8Request {
  int rows;  // 0: the few-rows kernel's
};

__device__ __forceinline__ Request request_of(const Fp8AttnParams& p, int b) {
  Request r;
  static_cast<Fp8Request&>(r) = fp8_request(p.c, b);
  r.rows = r.n * p.share;
  if (r.rows <= p.few_rows) r.rows = 0;
  return r;
}

// Token tiles of row block `rt` of a request: up to the last token that its
// last row sees, at least one (to write the zeros of rows that see none); 0
// past its rows.
__device__ __forceinline__ int tiles_of(const Fp8AttnParams& p, const Request& r, int rt) {
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
  __device__ __forceinline__ void next_unit(const Fp8AttnParams& p) {
    tile = 0;
    if (++kvh < p.c.num_kv_heads) return;
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

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// A value that all lanes share, known as such to the compiler.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ size_t out_at(const Fp8AttnParams& p, int first, int kvh, int row) {
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
  int base;  // position of the request's new token 0
  bool whole, begun, pair, both;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_chunk_kernel(const Fp8AttnParams p, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using C = Big<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t s_kfull[kKStages], s_kempty[kKStages], s_vfull[kVStages], s_vempty[kVStages];
  __shared__ uint64_t s_rfull[kRaw], s_rempty[kRaw];
  __shared__ uint8_t s_live[kRaw];  // which of a quarter's boxes lie in the cache
  __shared__ uint64_t s_qfull, s_sfull[2], s_pfull[2], s_pvdone[2];
  __shared__ uint32_t s_tmem;
  __shared__ long long s_scan[kThreads / 32], s_before;
  __shared__ int s_item, s_last[2];
  __shared__ Open s_open[2];  // the unit begun in front of this CTA, the one begun here
  __shared__ float s_cs[2][kTileRows];         // scale of each row's scores
  __shared__ float s_mx[2][2][2][kTileRows];   // largest score: tile's parity, slot, half of the tokens
  // the first token with a NaN in a dim that not all of a unit's rows see, for each slot to
  // read, by the unit's number: the tiles that are written as f16 are less than four units
  // ahead of the results
  __shared__ int s_nan[4][2][D];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

  if (tid == 0) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(smem_addr(&s_kfull[i]), kDecodeThreads / 32);
      mbar_init(smem_addr(&s_kempty[i]), 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(smem_addr(&s_vfull[i]), kDecodeThreads / 32);
      mbar_init(smem_addr(&s_vempty[i]), 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(smem_addr(&s_rfull[i]), kQuarter / p.box);
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
  for (int i = tid; i < 8 * D; i += kThreads) (&s_nan[0][0][0])[i] = kDead;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // TMEM only now: a kernel in front may still need it.  Dependents start only
  // when it is taken: one that took it first and then waited for this kernel's
  // end would never see it.
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&s_tmem), kTmemCols);
    tmem_relinquish();
  }

  // ---- this CTA's run; an item is one request and row block, all KV heads
  const int blocks_max = static_cast<int>((static_cast<long long>(p.share) * p.c.max_query_len + kUnitRows - 1) / kUnitRows);
  const int items = p.c.batch * blocks_max;  // below 2^31, the launcher sees to it
  long long total = 0, share;
  {
    const int per = (items + kThreads - 1) / kThreads;
    const int i0 = min(items, tid * per), i1 = min(items, i0 + per);
    long long mine = 0;
#pragma unroll 1
    for (int i = i0; i < i1; ++i)
      mine += static_cast<long long>(tiles_of(p, request_of(p, i / blocks_max), i % blocks_max)) * p.c.num_kv_heads;
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
        const long long w = static_cast<long long>(tiles_of(p, request_of(p, i / blocks_max), i % blocks_max)) * p.c.num_kv_heads;
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
    // ================= tiles of f16: thread (token, piece) of each 16-byte piece of codes
    const int dt = tid - kSoftmaxThreads;
    constexpr int kPerRow = D / 16;                       // pieces of a token's row
    constexpr int kStride = kDecodeThreads / kPerRow;     // tokens between a thread's pieces
    const int piece = dt % kPerRow, token0 = dt / kPerRow;
    const uint32_t base = smem_addr(smem);
    // the second block's lanes take their 8-dim halves in another order: the eight lanes
    // of a store then meet eight different bank groups
    const int turn = D == 128 && piece >= 4;
    const int box_shift = 31 - __clz(p.box);
    const uint32_t all_live = (1u << (kQuarter / p.box)) - 1u;
    // a thread's tokens are a multiple of 8 apart: one swizzle for all of them
    static_assert(kStride % 8 == 0, "tokens of a thread share their swizzle");
    const uint32_t from = C::kCodes + token0 * D + ((piece ^ (D == 128 ? token0 & 7 : (token0 >> 1) & 3)) << 4) + 8 * turn;
    const uint32_t block = base + (D == 128 ? piece / 4 : 0) * C::kBlockBytes + token0 * 128;
    const uint32_t to0 = block + ((((piece % 4) * 2 + turn) ^ (token0 & 7)) << 4), to1 = to0 ^ 16u;
    int unit = 0, slot = -1, turns = 0;
    // the last position that the unit's first row sees
    auto first_sees = [&] { return at.rq.len - at.rq.all + at.rt * kUnitRows / p.share; };
    int seen = first_sees();
    // quarter h of the run: tokens 64 (h % 2) .. of the keys, then the values, of tile h / 4
#pragma unroll 1
    for (int h = 0; h < 4 * run_tiles; ++h) {
      const int j = h / 4, w = h >> 1 & 1, part = h & 1;
      const int stages = w ? kVStages : kKStages, stage = j % stages;
      if (++slot == kRaw) {
        slot = 0;
        ++turns;
      }
      if (!(ok = warp_wait(smem_addr(&s_rfull[slot]), turns & 1))) break;
      const uint8_t* codes = smem + slot * C::kCodeBytes + from;
      uint2 raw[C::kPieces][2];  // dims 16 piece + 8 turn .., and the other 8
#pragma unroll
      for (int x = 0; x < C::kPieces; ++x) {
        raw[x][0] = *reinterpret_cast<const uint2*>(codes + x * kStride * D);
        raw[x][1] = *reinterpret_cast<const uint2*>(codes + x * kStride * D + (turn ? -8 : 8));
      }
      const uint32_t live = s_live[slot];
      const int end = at.rq.len - at.tile * kTileTokens - part * kQuarter;
      if (end < kQuarter || live != all_live) {
        asm volatile("");  // a branch, for few tiles
        // what is not a token of the request becomes zeros, whatever the cache holds there
#pragma unroll
        for (int x = 0; x < C::kPieces; ++x) {
          const int token = token0 + x * kStride;
          if (token >= end || !(live >> (token >> box_shift) & 1u)) raw[x][0] = raw[x][1] = make_uint2(0u, 0u);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&s_rempty[slot]));
      // tokens that the unit's first row does not see: NaN codes of V there go apart
      const int low = seen - at.tile * kTileTokens - part * kQuarter;
      if (w && low < kQuarter - 1) {
        asm volatile("");
#pragma unroll
        for (int x = 0; x < C::kPieces; ++x)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int token = token0 + x * kStride;
            const uint2 was = raw[x][i];
            if (token <= low) continue;
            raw[x][i] = make_uint2(fp8_nan_to_zero(was.x), fp8_nan_to_zero(was.y));
            if (raw[x][i].x == was.x && raw[x][i].y == was.y) continue;
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              if (((c < 4 ? was.x : was.y) >> (8 * (c % 4)) & 0x7Fu) != 0x7Fu) continue;
              const int dim = 16 * piece + 8 * (i ^ turn) + c, position = at.tile * kTileTokens + part * kQuarter + token;
              atomicMin(&s_nan[unit & 3][0][dim], position);
              atomicMin(&s_nan[unit & 3][1][dim], position);
            }
          }
      }
      if (j >= stages && part == 0) ok = warp_wait(smem_addr(w ? &s_vempty[stage] : &s_kempty[stage]), ((j / stages) & 1) ^ 1u);
      if (!ok) break;
      const uint32_t tile = (w ? C::kV : C::kK) + stage * C::kTileBytes + part * kQuarter * 128;
#pragma unroll
      for (int x = 0; x < C::kPieces; ++x) {
        uint32_t v[4];
        e4m3x4_to_f16x2x2(raw[x][0].x, v[0], v[1]);
        e4m3x4_to_f16x2x2(raw[x][0].y, v[2], v[3]);
        st_shared_v4(to0 + tile + x * kStride * 128, v[0], v[1], v[2], v[3]);
        e4m3x4_to_f16x2x2(raw[x][1].x, v[0], v[1]);
        e4m3x4_to_f16x2x2(raw[x][1].y, v[2], v[3]);
        st_shared_v4(to1 + tile + x * kStride * 128, v[0], v[1], v[2], v[3]);
      }
      if (part == 0) continue;
      fence_proxy_async_shared();  // the stores before the tensor cores' reads
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(w ? &s_vfull[stage] : &s_kfull[stage]));
      if (w && h + 1 < 4 * run_tiles && ++at.tile == at.tiles) {
        at.next_unit(p);
        seen = first_sees();
        ++unit;
      }
    }
  } else if (warp == kCopyWarp) {
    // ================= copies: lane x has box x of the tile's rows of the cache
    const uint32_t codes = smem_addr(smem) + C::kCodes;
    const int boxes = kQuarter / p.box;  // of a quarter
    const uint32_t bytes = static_cast<uint32_t>(p.box * D);
    auto look_up = [&]() -> int {
      const int t = at.tile * kTileTokens + lane * p.box;
      if (lane >= 2 * boxes || t >= at.rq.len) return -1;
      const int col = t / p.c.block_size;
      const int blk = __ldg(p.c.block_table + static_cast<size_t>(at.b) * p.c.max_blocks + col);
      if (blk < 0 || blk >= p.c.num_blocks) return -1;
      return blk * p.c.block_size + (t - col * p.c.block_size);
    };
    int next = look_up(), next_kvh = at.kvh, row = -1, kvh = 0, h = 0;
#pragma unroll 1
    for (; h < 4 * run_tiles; ++h) {
      const int slot = h % kRaw;
      if (!(h & 3)) {
        row = next;
        kvh = next_kvh;
        if (h + 4 < 4 * run_tiles) {  // the next tile's places, while this one's are copied
          if (++at.tile == at.tiles) at.next_unit(p);
          next = look_up();
          next_kvh = at.kvh;
        }
      }
      if (h >= kRaw && !(ok = warp_wait(smem_addr(&s_rempty[slot]), ((h / kRaw) & 1) ^ 1u))) break;
      const int x = lane - (h & 1) * boxes;  // this lane's box of the quarter
      const uint32_t live = __ballot_sync(0xffffffffu, row >= 0) >> ((h & 1) * boxes);
      if (lane == 0) s_live[slot] = static_cast<uint8_t>(live & ((1u << boxes) - 1u));
      __syncwarp();
      if (x >= 0 && x < boxes) {
        const uint32_t full = smem_addr(&s_rfull[slot]);
        fence_proxy_async_shared();  // the reads of the slot's last quarter before the copies over it
        if (row >= 0) {
          mbar_arrive_expect_tx(full, bytes);
          tma_load_2d(codes + slot * C::kCodeBytes + x * bytes, h & 2 ? &map_v : &map_k, full, kvh * D, row);
        } else {
          mbar_arrive(full);
        }
      }
    }
    // a wait gave up: the copies in flight land before shared memory is released
    if (!ok)
      for (int i = max(0, h - kRaw); i < h; ++i) mbar_wait(smem_addr(&s_rfull[i % kRaw]), (i / kRaw) & 1);
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
      const int stage = tile % kKStages;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk / 4) * (C::kBlockBytes >> 4) + 2 * (kk % 4);
        mma_f16_by(leader, tm + slot * kTileTokens, dq + q * (C::kTileBytes >> 4) + off,
                   dk + stage * (C::kTileBytes >> 4) + off, kIdescS, kk > 0);
      }
      mma_commit_by(leader, smem_addr(&s_sfull[slot]));
    };
    auto wait_k = [&](int tile) {
      if (ok) ok = warp_wait(smem_addr(&s_kfull[tile % kKStages]), (tile / kKStages) & 1);
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
        mma_commit_by(leader, smem_addr(&s_kempty[(done + j) % kKStages]));
      }
#pragma unroll 1
      for (int j = 0; j < nt && ok; ++j) {
        const int stage = (done + j) % kVStages;
        const bool more = j + ahead < nt;
        ok = warp_wait(smem_addr(&s_vfull[stage]), ((done + j) / kVStages) & 1);
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
        if (more) mma_commit_by(leader, smem_addr(&s_kempty[(done + j + ahead) % kKStages]));
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
    const float vscale = __ldg(p.v_scale), to_log2 = p.sm_scale * __ldg(p.k_scale) * kFp8Log2e;
    uint32_t count = 0u;  // tiles of this slot
    int done = 0, nth = 0;
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
      // 2^e so that a row's largest element lies in [2^14, 2^15)
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
              raw[i] = fp8_load8(static_cast<const uint16_t*>(p.q) + (rq.first + r / p.share) * p.q_token_stride +
                                     (at.kvh * p.share + r % p.share) * p.q_head_stride + 8 * c,
                                 p.q_vec);
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int r = wrow + (i0 + i) * kAtOnce;
            const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            float v[8], qmax = 0.f;
            bool odd = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 x = fp8_to_float2(u[k], p.q_fp16);
              v[2 * k] = x.x;
              v[2 * k + 1] = x.y;
              qmax = fmaxf(qmax, fmaxf(fabsf(x.x), fabsf(x.y)));
              odd = odd || !(fabsf(x.x) < INFINITY) || !(fabsf(x.y) < INFINITY);
            }
#pragma unroll
            for (int off = 1; off < kPerRow; off <<= 1) qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, off));
            odd = (__ballot_sync(0xffffffffu, odd) >> (lane / kPerRow * kPerRow) & ((1u << kPerRow) - 1u)) != 0u;
            int e = 0;
            if (qmax > 0.f && !odd) e = min(100, 14 + 127 - static_cast<int>(__float_as_uint(qmax) >> 23));
            const float down = to_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            // the scale's sign goes to the query: the largest product is the largest score
            const float up = copysignf(__uint_as_float(static_cast<uint32_t>(127 + e) << 23), down);
            // a row with a NaN or an infinity, or any row under a NaN scale, has NaN scores
            if (c == 0) s_cs[slot][r] = odd || !(fabsf(down) <= INFINITY) ? __int_as_float(0x7fffffff) : fmaxf(fabsf(down), 1e-37f);
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              h[k] = odd ? 0u : as_u32(__floats2half2_rn(v[2 * k] * up, v[2 * k + 1] * up));
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
            const int* nan_from = &s_nan[(nth - 1) & 3][slot][half * (D / 2) + 16 * c];
            const int seen = old.base + r / p.share;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (nan_from[i] <= seen) y[i] = __int_as_float(0x7fffffff);
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
                for (int i = 0; i < 8; ++i) z[i] = y[8 * q + i] * inv;
                fp8_store8(static_cast<uint16_t*>(p.out) + to + 16 * c + 8 * q, z, p.out_fp16, p.out_vec);
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
      // the last unit's NaN marks have been read (who writes this entry again comes four units on)
      if (old.tiles > 0 && tid % kSlotThreads < D) s_nan[(nth - 1) & 3][slot][tid % kSlotThreads] = kDead;
      const int lim = real ? rq.len - rq.all + my / p.share : rq.len - 1;  // the last token seen
      // (a row of NaN scores goes by those of its finite query: what it does not see has weight
      // 0 then, and its sum says at the end whether it saw anything)
      cs = s_cs[pair ? slot : 0][row];
      if (!(cs == cs)) cs = 1.f;
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
          const int t = (at.tile + j) * kTileTokens + lane * kPageTokens;
          if (lane < kRecords && t < rq.len) {
            const int blk = __ldg(p.c.block_table + static_cast<size_t>(at.b) * p.c.max_blocks + t / p.c.block_size);
            gone = blk < 0 || blk >= p.c.num_blocks;
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

      // ---- its end: NaN for such a row, if it saw a token (the next unit's scales are written
      // behind the next barrier)
      if (l != 0.f && !(s_cs[pair ? slot : 0][row] == s_cs[pair ? slot : 0][row])) l = __int_as_float(0x7fffffff);
      const long long unit = r0 + done - at.tile;
      old.whole = at.tile == 0 && nt == at.tiles;
      old.begun = unit / share == blockIdx.x;
      old.pair = pair;
      old.both = !pair && nt > 1;
      old.first = rq.first;
      old.base = rq.len - rq.all;
      old.rows = rq.rows;
      old.row0 = row0;
      old.kvh = at.kvh;
      old.tiles = nt;
      if (!old.whole && tid == 0) s_open[old.begun] = {rq.first, rq.rows, row0, at.kvh, unit, at.tiles};
      done += nt;
      at.tile += nt;
      ++nth;
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
    const float inv = l != 0.f ? __ldg(p.v_scale) / l : 0.f;
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
      fp8_store8(static_cast<uint16_t*>(p.out) + to + 8 * q, y, p.out_fp16, p.out_vec);
    }
  }
}

template <int D>
cudaError_t launch_t(const Fp8AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, int num_sms, cudaStream_t stream) {
  auto kern = fp8_chunk_kernel<D>;
  // the attribute is per function and device; setting it again is harmless
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Big<D>::kSmem);
  if (e != cudaSuccess) return e;
  return fp8_launch(kern, dim3(static_cast<unsigned>(std::min(num_sms, kFp8MaxCtas))), dim3(kThreads), Big<D>::kSmem, stream, p, k, v);
}

}  // namespace

size_t fp8_chunk_workspace(int head_dim, int num_sms) {
  return kCounterRegion + static_cast<size_t>(std::min(num_sms, kFp8MaxCtas)) * 2 * kUnitRows * (head_dim + 2) * sizeof(float);
}

cudaError_t read_clear_fp8_chunk_status(int* flags) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_status, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  e = cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int));
  *flags = v;
  return e;
}

cudaError_t launch_fp8_chunk(const Fp8AttnParams& p, const CUtensorMap& map_k, const CUtensorMap& map_v, int num_sms,
                             cudaStream_t stream) {
  return p.c.head_dim == 64 ? launch_t<64>(p, map_k, map_v, num_sms, stream) : launch_t<128>(p, map_k, map_v, num_sms, stream);
}

}  // namespace w8a8
