// fp8_attention.cu -- attention of a step's new tokens over the paged fp8 cache:
// which kernel takes which requests (sm_103a).
#include <algorithm>

#include "internal.h"

namespace w8a8 {

namespace {

// Rows (tokens times query heads of a KV head) up to which a call whose requests
// all have as few goes to the few-rows kernel.
constexpr int kFewRows = 32;

// In a call with larger requests: the rows up to which a request still goes there.
// The few-rows kernel's smallest tile that holds a token's heads, so that single
// tokens cost what they cost alone.  (32 requests to 4096 tokens with 2 to 5 drafts of 4
// heads: 90 us in the few-rows kernel, 129 where a limit above 8 tokens brings the larger
// ones here; in its form for 32 rows a single token costs twice what it does in that for 8.)
int few_beside_many(int share) { return share <= 8 ? 8 : share <= 16 ? 16 : kFewRows; }

}  // namespace

size_t fp8_paged_attention_workspace(int share, long long max_query_len, int head_dim, int num_sms) {
  const long long rows = share * max_query_len;
  if (rows <= kFewRows) return fp8_rows_workspace(static_cast<int>(rows), head_dim, num_sms);
  return std::max(fp8_chunk_workspace(head_dim, num_sms), fp8_rows_workspace(few_beside_many(share), head_dim, num_sms));
}

size_t fp8_sparse_attention_workspace(int share, int head_dim, int num_sms) {
  return fp8_rows_workspace(std::min(share, kFewRows), head_dim, num_sms);
}

cudaError_t read_clear_fp8_status(int* flags) {
  int rows = 0, chunk = 0;
  cudaError_t e = read_clear_fp8_rows_status(&rows);
  if (e == cudaSuccess) e = read_clear_fp8_chunk_status(&chunk);
  *flags = rows | chunk;
  return e;
}

cudaError_t launch_fp8_attention(const Fp8AttnParams& args, const CUtensorMap& map_k, const CUtensorMap& map_v, int num_sms,
                                 void* workspace, cudaStream_t stream) {
  Fp8AttnParams p = args;
  p.counters = static_cast<unsigned*>(workspace);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCounterRegion);
  p.few_rows = kFewRows;
  const long long rows = p.selected ? std::min(p.share, kFewRows) : static_cast<long long>(p.share) * p.c.max_query_len;
  if (rows <= kFewRows) return launch_fp8_rows(p, static_cast<int>(rows), map_k, map_v, num_sms, stream);
  // single tokens between chunks: 128 rows of the many-rows kernel would be theirs.  (Both
  // kernels use the workspace: the second begins when the first has ended.)  One request
  // alone is a chunk.
  p.few_rows = 0;
  if (p.c.batch > 1 && p.share <= kFewRows) {
    p.few_rows = few_beside_many(p.share);
    const cudaError_t e = launch_fp8_rows(p, p.few_rows, map_k, map_v, num_sms, stream);
    if (e != cudaSuccess) return e;
  }
  return launch_fp8_chunk(p, map_k, map_v, num_sms, stream);
}

}  // namespace w8a8
