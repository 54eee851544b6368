// fp8_select.cu -- 8-bit means of the cache's blocks, and the blocks that
// matter most to each query by them (sm_103a).
//
// ---- Means
// One CTA for a written block and KV head sums the codes' values of its tokens.
// A value is a multiple of 2^-9 of at most 448, so 64 of them add exactly in
// fp32; what a thread has of them goes on as an integer (times 2^9).
//
// ---- Scores
// Products of int8 codes by mma.sync m16n8k32 with int32 sums, 16 blocks by 8
// query rows at a time.  A query's heads that share a KV head stand side by
// side in the 8 columns (padded to a power of two; more than 8 take several
// tiles), so that their maximum is a step or two of shuffles.  A CTA of 8 warps
// takes kColumns blocks of one request and KV head and all its rows, 64 at a
// time: the means, 132 bytes a block, are what it reads, and they stay in
// registers while the rows pass.  The dot product does not depend on the order
// of the dims: lane t of a group takes 32 consecutive ones.
// (tcgen05 has no int8 kind on this GPU.  The codes as f16 numbers, which would add as
// exactly, by m16n8k16: 16 tokens over 4096 blocks 39 us for the whole selection, not 32,
// for twice the instructions and half the blocks a warp holds.)
//
// ---- Selection
// One CTA to a token and KV head: its scores as sortable integers in shared
// memory, the budget's threshold found by three passes of 11, 11 and 10 bits
// over histograms (a pass looks only at keys that agree so far), then the
// columns above the threshold, and the lowest of those at it, written in rising
// order by ballots.  It leaves zeros where its scores lay in the workspace's first
// kCounterRegion bytes: other operators keep their arrival counters there and
// find them in the same workspace afterwards.
//
// Means and selection are latency, a chain of lengths, block ids, means and scores; so are
// the scores of few tokens, and those of several wait for the int8 matrix instruction
// (44 % of its rate).  32 requests up to 32768 tokens in blocks of 64, 8 KV heads: 22 us
// in a graph, of which the means take 4; 4 requests of 131071 in blocks of 32, 4 tokens
// and 8 x 8 heads: 36 (under the profiler 6.5, 21 and 15).  Rows of a prompt chunk are not
// divided over CTAs: 600 tokens after 30000, blocks of 64, 505 us; 2048 tokens 1703.
#include <algorithm>

#include "fp8_paged.cuh"
#include "quant_math.cuh"

namespace w8a8 {

namespace {

// The scale of 8-bit codes: absmax times 1/127, both in fp32, 1 for zeros (a
// product and not, as the quantiser's int8 scale, a quotient: a last bit apart, and the codes
// are of this one).
__device__ __forceinline__ float int8_scale(float top) { return top > 0.f ? __fmul_rn(top, 1.f / 127.f) : 1.f; }

// ------------------------------------------------------------------ means

constexpr int kMeanThreads = 128;

template <int D>
__global__ void __launch_bounds__(kMeanThreads) fp8_block_means_kernel(const Fp8MeansArgs a) {
  constexpr int kPieces = D / 16, kTokens = kMeanThreads / kPieces;  // tokens looked at side by side
  constexpr int kExact = 64;  // values of one thread that add exactly
  __shared__ int s_sum[D];
  __shared__ float s_top[D / 32];
  fp8_let_dependents_start();
  fp8_wait_for_predecessor();
  const int kvh = blockIdx.x % a.c.num_kv_heads, nth = blockIdx.x / a.c.num_kv_heads, b = blockIdx.y;
  const Fp8Request r = fp8_request(a.c, b);
  if (r.n <= 0 || r.len <= 0) return;
  const int tid = threadIdx.x, piece = tid % kPieces;
  const size_t row = static_cast<size_t>(a.c.num_kv_heads) * D;
  // (one turn, but where a request has more new tokens than max_query_len)
#pragma unroll 1
  for (long long col = max(0, r.len - r.all) / a.c.block_size + nth;; col += gridDim.x / a.c.num_kv_heads) {
    const long long t0 = col * a.c.block_size;
    if (t0 >= r.len) return;
    const int block = __ldg(a.c.block_table + static_cast<size_t>(b) * a.c.max_blocks + col);
    if (block < 0 || block >= a.c.num_blocks) continue;
    const int count = static_cast<int>(min(static_cast<long long>(a.c.block_size), r.len - t0));
    if (tid < D) s_sum[tid] = 0;
    __syncthreads();
    const uint8_t* src = static_cast<const uint8_t*>(a.k_cache) + static_cast<size_t>(block) * a.c.block_size * row +
                         static_cast<size_t>(kvh) * D + 16 * piece;
#pragma unroll 1
    for (int u0 = 0; u0 < count; u0 += kExact * kTokens) {
      float sum[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[i] = 0.f;
#pragma unroll 4
      for (int u = u0 + tid / kPieces; u < min(count, u0 + kExact * kTokens); u += kTokens) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(src + u * row));
        const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t h[2];
          const uint32_t clean = fp8_nan_to_zero(word[i]);
          asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
              "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
              : "=r"(h[0]), "=r"(h[1])
              : "r"(clean));
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
            sum[4 * i + 2 * k] += f.x;
            sum[4 * i + 2 * k + 1] += f.y;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        int x = __float2int_rn(sum[i] * 512.f);
        // lanes with the same piece first
#pragma unroll
        for (int off = kPieces; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        sum[i] = __int_as_float(x);
      }
      if (tid % 32 < kPieces) {
#pragma unroll
        for (int i = 0; i < 16; ++i) atomicAdd(&s_sum[16 * piece + i], __float_as_int(sum[i]));
      }
    }
    __syncthreads();
    float mean = 0.f;
    if (tid < D) {
      mean = __fdiv_rn(__int2float_rn(s_sum[tid]) * (1.f / 512.f), static_cast<float>(count));
      float top = fabsf(mean);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      if (tid % 32 == 0) s_top[tid / 32] = top;
    }
    __syncthreads();
    if (tid < D) {
      float top = s_top[0];
#pragma unroll
      for (int i = 1; i < D / 32; ++i) top = fmaxf(top, s_top[i]);
      const float scale = int8_scale(top);
      const size_t at = static_cast<size_t>(block) * a.c.num_kv_heads + kvh;
      a.means[at * D + tid] = static_cast<int8_t>(enc1<1>(__fdiv_rn(mean, scale)));
      if (tid == 0) a.mean_scales[at] = scale;
    }
  }
}

// ------------------------------------------------------------------ scores

constexpr int kScoreWarps = 8, kScoreThreads = 32 * kScoreWarps;
constexpr int kRowTile = 64;                   // padded query rows in shared memory
constexpr int kColumns = 2 * 16 * kScoreWarps; // blocks of a CTA

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Tokens [token0, token0 + slab) of q; p.scores is theirs.
template <int D>
__global__ void __launch_bounds__(kScoreThreads, 4) fp8_block_scores_kernel(const Fp8SelectArgs a, int token0) {
  constexpr int kStride = D + 16;   // bytes of a query row: 16-byte reads of 8 rows meet 8 bank groups
  constexpr int kSteps = D / 32;    // k-steps of an MMA
  constexpr int kPer = D / 4;       // dims of a lane
  __shared__ __align__(16) int8_t s_q[kRowTile * kStride];
  __shared__ float s_scale[kRowTile];
  fp8_let_dependents_start();
  fp8_wait_for_predecessor();
  const int b = blockIdx.z, kvh = blockIdx.y;
  const Fp8Request r = fp8_request(a.c, b);
  const int i0 = max(0, token0 - r.first), i1 = min(r.n, token0 + a.slab - r.first);  // its tokens in the slab
  const int blocks = (r.len + a.c.block_size - 1) / a.c.block_size;
  const int col0 = blockIdx.x * kColumns;
  if (i0 >= i1 || col0 >= blocks) return;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane >> 2, t = lane & 3;

  // ---- the means: two tiles of 16 blocks a warp, rows g and g + 8
  uint32_t m[2][2][kPer / 4];
  float ms[2][2];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = col0 + (x * kScoreWarps + warp) * 16 + g + 8 * h;
      int block = -1;
      if (col < blocks) block = __ldg(a.c.block_table + static_cast<size_t>(b) * a.c.max_blocks + col);
      const bool in = block >= 0 && block < a.c.num_blocks;
      const size_t at = static_cast<size_t>(in ? block : 0) * a.c.num_kv_heads + kvh;
      // (a block outside the cache: -1 marks it, true scales are not negative)
      ms[x][h] = in ? __ldg(a.mean_scales + at) : -1.f;
#pragma unroll
      for (int i = 0; i < kPer / 16; ++i) {
        const uint4 w = in ? __ldg(reinterpret_cast<const uint4*>(a.means + at * D + kPer * t) + i) : make_uint4(0u, 0u, 0u, 0u);
        m[x][h][4 * i] = w.x, m[x][h][4 * i + 1] = w.y, m[x][h][4 * i + 2] = w.z, m[x][h][4 * i + 3] = w.w;
      }
    }

  // ---- rows: token i's heads fill `pad` columns, a tile holds `side` tokens, or a
  // token `tiles` tiles
  const int pad = a.share > 4 ? 8 : a.share > 2 ? 4 : a.share;
  const int tiles = (a.share + 7) / 8, side = 8 / pad;
  const int per_pass = tiles > 1 ? kRowTile / 8 / tiles : kRowTile / pad;  // tokens (share <= 64: at least one)
  const int rows_of = tiles > 1 ? 8 * tiles : pad;                         // padded rows of a token
#pragma unroll 1
  for (int i = i0; i < i1; i += per_pass) {  // (i1 is at most kFp8MostRows)
    const int n = min(per_pass, i1 - i);
    __syncthreads();
    // a warp quantises its rows, D / 32 values a lane, four rows' loads in flight; zeros for
    // padding, up to a whole tile of 8
    const int rows = (n * rows_of + 7) / 8 * 8;
    constexpr int kAtOnce = 4;
#pragma unroll 1
    for (int first = warp; first < rows; first += kAtOnce * kScoreWarps) {
      uint32_t raw[kAtOnce][kPer / 16];
      bool real[kAtOnce];
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) {
        const int row = first + x * kScoreWarps, tok = row / rows_of, head = row % rows_of;
        real[x] = tok < n && head < a.share;
#pragma unroll
        for (int k = 0; k < kPer / 16; ++k) raw[x][k] = 0u;
        if (!real[x]) continue;
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + (r.first + i + tok) * a.q_token_stride +
                              (kvh * a.share + head) * a.q_head_stride + (kPer / 8) * lane;
#pragma unroll
        for (int k = 0; k < kPer / 16; ++k)
          raw[x][k] = a.q_vec ? __ldg(reinterpret_cast<const uint32_t*>(src) + k)
                              : static_cast<uint32_t>(__ldg(src + 2 * k)) | (static_cast<uint32_t>(__ldg(src + 2 * k + 1)) << 16);
      }
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) {
        const int row = first + x * kScoreWarps;
        if (row >= rows) break;
        float f[kPer / 8], top = 0.f;
#pragma unroll
        for (int k = 0; k < kPer / 16; ++k) {
          const float2 v = fp8_to_float2(raw[x][k], a.q_fp16);
          f[2 * k] = v.x, f[2 * k + 1] = v.y;
          top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float scale = int8_scale(top);
#pragma unroll
        for (int k = 0; k < kPer / 8; ++k)
          s_q[row * kStride + (kPer / 8) * lane + k] = static_cast<int8_t>(enc1<1>(__fdiv_rn(f[k], scale)));
        // (a padded head's NaN never is a maximum)
        if (lane == 0) s_scale[row] = real[x] ? scale : __int_as_float(0x7fffffff);
      }
    }
    __syncthreads();
    const int used = rows / 8;
    float best[2][2] = {{-INFINITY, -INFINITY}, {-INFINITY, -INFINITY}};
#pragma unroll 1
    for (int nt = 0; nt < used; ++nt) {
      uint32_t q[kPer / 4];
#pragma unroll
      for (int k = 0; k < kPer / 16; ++k) {
        const uint4 w = *reinterpret_cast<const uint4*>(s_q + (8 * nt + g) * kStride + kPer * t + 16 * k);
        q[4 * k] = w.x, q[4 * k + 1] = w.y, q[4 * k + 2] = w.z, q[4 * k + 3] = w.w;
      }
      const float sq[2] = {s_scale[8 * nt + 2 * t], s_scale[8 * nt + 2 * t + 1]};
      const bool last = tiles == 1 || nt % tiles == tiles - 1;  // of a token
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        int d[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
          mma_s8(d, m[x][0][2 * k], m[x][1][2 * k], m[x][0][2 * k + 1], m[x][1][2 * k + 1], q[2 * k], q[2 * k + 1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // columns 2t, 2t + 1 of row g + 8 h (fmaxf passes a NaN by)
          float v0 = fmaxf(__int2float_rn(d[2 * h]) * sq[0], -INFINITY), v1 = fmaxf(__int2float_rn(d[2 * h + 1]) * sq[1], -INFINITY);
          const int col = col0 + (x * kScoreWarps + warp) * 16 + g + 8 * h;
          auto put = [&](int tok, float v) {
            if (tok >= n || col >= blocks) return;
            const float y = ms[x][h] < 0.f ? -INFINITY : fmaxf(__fmul_rn(v, ms[x][h]), -INFINITY);
            a.scores[(static_cast<size_t>(r.first + i + tok - token0) * a.c.num_kv_heads + kvh) * a.c.max_blocks + col] = y;
          };
          if (pad == 1) {
            put(nt * side + 2 * t, v0);
            put(nt * side + 2 * t + 1, v1);
            continue;
          }
          v0 = fmaxf(v0, v1);
          if (pad >= 4) v0 = fmaxf(v0, __shfl_xor_sync(0xffffffffu, v0, 1));
          if (pad == 8) v0 = fmaxf(v0, __shfl_xor_sync(0xffffffffu, v0, 2));
          if (tiles > 1) {
            best[x][h] = v0 = fmaxf(v0, best[x][h]);
            if (!last) continue;
            best[x][h] = -INFINITY;
          }
          // one of the lanes that have the maximum
          if (pad == 2) put(nt * side + t, v0);
          else if (pad == 4 && t % 2 == 0) put(nt * side + t / 2, v0);
          else if (pad == 8 && t == 0) put(tiles > 1 ? nt / tiles : nt, v0);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ selection

constexpr int kBins = 2048;

// Order-preserving: a larger score, a larger key; the lowest score has key 0x007fffff.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 counts as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int kPickThreads>
__global__ void __launch_bounds__(kPickThreads) fp8_pick_blocks_kernel(const Fp8SelectArgs a, int token0) {
  constexpr int kPickWarps = kPickThreads / 32;
  extern __shared__ __align__(16) uint32_t s_key[];  // [max_blocks]
  __shared__ int s_hist[kBins];
  __shared__ int s_found, s_warp[kPickWarps], s_warp2[kPickWarps], s_bin, s_above;
  fp8_let_dependents_start();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int token = token0 + blockIdx.x, kvh = blockIdx.y;
  fp8_wait_for_predecessor();
  const int b = fp8_request_of_row(a.c, token, &s_found);
  if (b < 0) return;
  const Fp8Request r = fp8_request(a.c, b);
  const int pos = r.len - r.all + token - r.first;
  int* out = a.selected + (static_cast<size_t>(token) * a.c.num_kv_heads + kvh) * a.budget;
  const int n = pos < 0 ? 0 : pos / a.c.block_size + 1;  // blocks up to its own
  const size_t at_score = (static_cast<size_t>(token - token0) * a.c.num_kv_heads + kvh) * a.c.max_blocks;
  // the scores of this row that lie where other calls have their counters, once they have been read
  auto clear = [&] {
    const size_t region = kCounterRegion / sizeof(float);
    if (at_score >= region) return;
    const int end = static_cast<int>(min(region - at_score, static_cast<size_t>(a.c.max_blocks)));
    for (int c = tid; c < end; c += kPickThreads) a.scores[at_score + c] = 0.f;
  };
  if (n <= a.budget) {
    for (int i = tid; i < a.budget; i += kPickThreads) out[i] = i < n ? i : -1;
    clear();
    return;
  }
  const int lo = a.first_blocks, hi = n - a.last_blocks;  // columns [lo, hi) are chosen from
  const float* src = a.scores + at_score;
  for (int c = lo + tid; c < hi; c += kPickThreads) s_key[c] = key_of(src[c]);

  // ---- the threshold: `want` keys are taken, those above `prefix` and the first
  // at it; bits below `shift` are not fixed yet
  int want = a.budget - a.first_blocks - a.last_blocks;
  const bool none = want == 0;
  uint32_t prefix = 0u, mask = 0u;
#pragma unroll 1
  for (int pass = 0; pass < 3 && want > 0; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < kBins; i += kPickThreads) s_hist[i] = 0;
    __syncthreads();
    for (int c = lo + tid; c < hi; c += kPickThreads) {
      const uint32_t k = s_key[c];
      if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & ((1u << bits) - 1u)], 1);
    }
    __syncthreads();
    // from the top: a thread has kBins / kPickThreads bins, thread 0 the highest ones
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kBins / kPickThreads; ++i) mine += s_hist[kBins - 1 - (kBins / kPickThreads) * tid - i];
    int run = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, run, off);
      if (lane >= off) run += o;
    }
    if (lane == 31) s_warp[warp] = run;
    __syncthreads();
    run -= mine;
#pragma unroll
    for (int w = 0; w < kPickWarps; ++w)
      if (w < warp) run += s_warp[w];
    if (run < want && run + mine >= want) {
#pragma unroll 1
      for (int i = 0; i < kBins / kPickThreads; ++i) {
        const int bin = kBins - 1 - (kBins / kPickThreads) * tid - i, h = s_hist[bin];
        if (run + h >= want) {
          s_bin = bin;
          s_above = run;
          break;
        }
        run += h;
      }
    }
    __syncthreads();
    want -= s_above;
    prefix |= static_cast<uint32_t>(s_bin) << shift;
    mask |= ((1u << bits) - 1u) << shift;
    __syncthreads();
  }

  // ---- columns in rising order: each warp has a stretch of them
  const int per = ((n + kPickWarps - 1) / kPickWarps + 31) / 32 * 32;
  const int c0 = min(n, warp * per), c1 = min(n, c0 + per);
  __syncthreads();
  clear();
  // 2: taken, 1: at the threshold, 0: not taken
  auto state = [&](int c) {
    if (c >= c1) return 0;
    if (c < lo || c >= hi) return 2;
    if (none) return 0;
    const uint32_t k = s_key[c];
    return k > prefix ? 2 : k == prefix ? 1 : 0;
  };
  int sure = 0, ties = 0;
#pragma unroll 1
  for (int c = c0; c < c1; c += 32) {
    const int s = state(c + lane);
    sure += __popc(__ballot_sync(0xffffffffu, s == 2));
    ties += __popc(__ballot_sync(0xffffffffu, s == 1));
  }
  if (lane == 0) s_warp[warp] = sure, s_warp2[warp] = ties;
  __syncthreads();
  int at = 0, left = want;  // places before this warp's, ties still to take
#pragma unroll
  for (int w = 0; w < kPickWarps; ++w) {
    if (w >= warp) continue;
    const int taken = min(left, s_warp2[w]);
    at += s_warp[w] + taken;
    left -= taken;
  }
#pragma unroll 1
  for (int c = c0; c < c1; c += 32) {
    const int s = state(c + lane);
    const uint32_t tie = __ballot_sync(0xffffffffu, s == 1);
    const bool taken = s == 2 || (s == 1 && __popc(tie & ((1u << lane) - 1u)) < left);
    const uint32_t all = __ballot_sync(0xffffffffu, taken);
    if (taken) out[at + __popc(all & ((1u << lane) - 1u))] = c + lane;
    at += __popc(all);
    left -= min(left, __popc(tie));
  }
}

// Tokens whose scores the workspace holds: as many as fit 64 MB, at least one
// (a row of scores is at most 49152 * 4 bytes for each of 65535 KV heads).
int slab_of(long long tokens, long long num_kv_heads, long long max_blocks) {
  const long long row = num_kv_heads * max_blocks * 4;
  return static_cast<int>(std::max(1LL, std::min(tokens, (64LL << 20) / row)));
}

template <int D>
cudaError_t launch_scores(const Fp8SelectArgs& a, int token0, cudaStream_t stream) {
  const dim3 grid((a.c.max_blocks + kColumns - 1) / kColumns, a.c.num_kv_heads, a.c.batch);
  return fp8_launch(fp8_block_scores_kernel<D>, grid, dim3(kScoreThreads), 0, stream, a, token0);
}

}  // namespace

cudaError_t launch_fp8_block_means(const Fp8MeansArgs& a, cudaStream_t stream) {
  const int most = static_cast<int>(std::min<long long>((a.c.max_query_len - 1LL) / a.c.block_size + 2, a.c.max_blocks));
  // (at most max_blocks * num_kv_heads, which the sizes' limits keep below 2^29)
  const dim3 grid(static_cast<unsigned>(most) * a.c.num_kv_heads, a.c.batch);
  if (a.c.head_dim == 64) return fp8_launch(fp8_block_means_kernel<64>, grid, dim3(kMeanThreads), 0, stream, a);
  return fp8_launch(fp8_block_means_kernel<128>, grid, dim3(kMeanThreads), 0, stream, a);
}

size_t fp8_select_workspace(long long tokens, long long num_kv_heads, long long max_blocks) {
  return static_cast<size_t>(slab_of(tokens, num_kv_heads, max_blocks)) * num_kv_heads * max_blocks * sizeof(float);
}

cudaError_t launch_fp8_select(const Fp8SelectArgs& args, cudaStream_t stream) {
  Fp8SelectArgs a = args;
  const int slab = slab_of(a.c.tokens, a.c.num_kv_heads, a.c.max_blocks);
  const int smem = (a.c.max_blocks + 3) / 4 * 4 * static_cast<int>(sizeof(uint32_t));
  // more threads where there are many columns: 4096 of them (16 tokens, 8 heads) 12.8 us by 1024
  // threads, 16.5 by 256; 300 (32 tokens, 8 heads) 9.0 by 256.  (Ranks in place of the
  // threshold, every key against every other, were 15.8 there.)
  const bool wide = a.c.max_blocks > 2048;
  auto pick = wide ? fp8_pick_blocks_kernel<1024> : fp8_pick_blocks_kernel<256>;
  // one limit for every call, so that host threads with other sizes do not lower it
  cudaError_t e = cudaFuncSetAttribute(pick, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kMaxSelectBlocks * static_cast<int>(sizeof(uint32_t)));
  if (e != cudaSuccess) return e;
  for (long long t0 = 0; t0 < a.c.tokens; t0 += slab) {
    const int n = static_cast<int>(std::min<long long>(slab, a.c.tokens - t0));
    a.slab = n;  // (the last pass's own: the kernel's token0 + slab never passes the tokens, nor 2^31)
    e = a.c.head_dim == 64 ? launch_scores<64>(a, static_cast<int>(t0), stream) : launch_scores<128>(a, static_cast<int>(t0), stream);
    if (e != cudaSuccess) return e;
    e = fp8_launch(pick, dim3(n, a.c.num_kv_heads), dim3(wide ? 1024 : 256), smem, stream, a, static_cast<int>(t0));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace w8a8
