// What the kernels of kvq_query_attention share: the queries of a call as rows of a
// (sequence, kv-head), and the choice of kernel.
//
// The n queries of a sequence and the n_rep query heads of a kv-head read the same keys,
// so they are rows of one matrix product: row i * n_rep + r is query i, head
// kvh * n_rep + r.  Row i sees the tokens [0, end): all T, or T - n + i + 1 of them under
// the causal mask.
#pragma once

#include "kvq_attn_plan.cuh"
#include "kvq_ptx.cuh"

namespace kvq {

// Queries of sequence b in this call.
__device__ __forceinline__ int query_count(const KvqView& v, const QueryArgs& a, int b) {
  if (!a.n_per_seq) return a.n_q;
  const int n = a.n_per_seq[b];
  if (n < 0 || n > a.n_q) {
    atomicOr(v.status, KVQ_DEV_BAD_LENGTH);
    return 0;
  }
  return n;
}

// Tokens that query i of n sees of T.
__device__ __forceinline__ int query_end(const QueryArgs& a, int T, int n, int i) {
  return a.causal ? max(0, T - n + i + 1) : T;
}

constexpr int kFewPass = 32;    // rows of the few-row kernel's widest pass
constexpr int kFewPasses = 8;   // and passes of a launch
constexpr int kFewSmallRows = 256;  // rows of a small call at most, in passes of 8
constexpr int kFewUnits = 7424;  // its runs at most: four for each of the 1,824 warps that head_dim 128 fills a GPU with
constexpr int kFewLeast = 1216;  // and the fewest that a call is cut down to: one for each warp at two CTAs an SM
int few_runs(const KvqView& v, int batch, long long rows, int out_f32);  // a call's
constexpr int kManyGrid = 160;  // CTAs of the many-row kernel at most (one per SM)

bool few_small(const KvqView& v, int batch, long long rows, long long tokens);  // whether passes of 8 rows take it
bool query_tc_shape(const KvqView& v);      // config only: the tensor-core kernels take it
bool query_tc_eligible(const KvqView& v);   // and the cache's pool

// The few-row kernel's workspace: its plan (4 ints), pref[B + 1], the counter, then records
// (M, l, 2 pad, o[D]) for each row of a pass.
__host__ __device__ inline size_t few_counter_offset(int B) { return (16 + ((size_t)B + 1) * 4 + 7) & ~(size_t)7; }
__host__ __device__ inline size_t few_header_bytes(int B) { return (few_counter_offset(B) + 8 + 255) / 256 * 256; }
size_t query_many_workspace_bytes(const KvqView& v, int batch, int n_q);
kvq_status launch_query_few_i8(const KvqView& v, const QueryArgs& a, void* ws, cudaStream_t st);
kvq_status launch_query_few_e4(const KvqView& v, const QueryArgs& a, void* ws, cudaStream_t st);
kvq_status launch_query_few_e5(const KvqView& v, const QueryArgs& a, void* ws, cudaStream_t st);
kvq_status launch_query_many(const KvqView& v, const QueryArgs& a, void* ws, cudaStream_t st);

}  // namespace kvq
