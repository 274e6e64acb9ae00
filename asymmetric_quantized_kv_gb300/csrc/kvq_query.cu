// kvq_query_attention: the choice of kernel, and the plain kernel that takes every
// configuration (any axis, format, window, pre-RoPE keys, head_dim, fp32 sources).
//
// The plain kernel: a CTA takes 8 rows (query, head) of one (sequence, kv-head) and walks
// the tokens in tiles of 32, dequantized into shared memory as fp32 by the rules of
// include/kvq.h, with the softmax's running maximum and sum in base 2.  It is bound by the
// per-element dequantization and by its one pass per 8 rows; it is what is right, not what
// is fast.
#include <math.h>

#include "kvq_dequant.cuh"
#include "kvq_query.cuh"
#include "kvq_tmap.h"

namespace kvq {
namespace {

constexpr int kPT = 128;    // threads
constexpr int kPRows = 8;   // rows of a CTA
constexpr int kPTile = 32;  // tokens of a tile
constexpr float kLog2eP = 1.4426950408889634f;

__global__ void __launch_bounds__(kPT) query_plain_kernel(KvqView v, QueryArgs a, int row_blocks) {
  __shared__ float qs[kPRows][kMaxHeadDim];
  __shared__ float kv[kPTile][kMaxHeadDim + 1];
  __shared__ float ps[kPRows][kPTile];
  __shared__ float ms[kPRows], ls[kPRows], al[kPRows];
  __shared__ float w_hi[kMaxHeadDim / 2], w_lo[kMaxHeadDim / 2];
  __shared__ int ends[kPRows];
  __shared__ unsigned char okt[kPTile];
  const int rb = blockIdx.x % row_blocks, x = blockIdx.x / row_blocks, h = x % v.Hkv, b = x / v.Hkv;
  const int D = v.D, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = query_count(v, a, b), T = seq_tokens(v, b), nq = n_quantized(T, v.R);
  const int rows = min(kPRows, n * v.n_rep - rb * kPRows);
  if (rows <= 0) return;
  // element offset of row r: query i = row / n_rep, head h * n_rep + row % n_rep
  auto row_elem = [&](int r) {
    const int row = rb * kPRows + r, i = row / v.n_rep;
    return (((long long)b * a.n_q + i) * v.Hq + h * v.n_rep + row % v.n_rep) * D;
  };
  if (threadIdx.x < kPRows) {
    ends[threadIdx.x] =
        threadIdx.x < rows ? query_end(a, T, n, (rb * kPRows + threadIdx.x) / v.n_rep) : 0;
    ms[threadIdx.x] = -INFINITY;
    ls[threadIdx.x] = 0.f;
  }
  for (int e = threadIdx.x; e < kPRows * D; e += kPT) {
    const int r = e / D, c = e % D;
    qs[r][c] = r < rows ? load_src(a.q, row_elem(r) + c, v.src_bf16) * a.scale * kLog2eP : 0.f;
  }
  if (v.rope_pre)
    for (int i = threadIdx.x; i < D / 2; i += kPT) rope_split(v, i, &w_hi[i], &w_lo[i]);
  float o[kPRows][kMaxHeadDim / kPT];
#pragma unroll
  for (int r = 0; r < kPRows; ++r)
#pragma unroll
    for (int j = 0; j < kMaxHeadDim / kPT; ++j) o[r][j] = 0.f;
  __syncthreads();
  int end = 0;
  for (int r = 0; r < kPRows; ++r) end = max(end, ends[r]);
  for (int t0 = 0; t0 < end; t0 += kPTile) {
    const int nt = min(kPTile, end - t0);
    if (threadIdx.x < kPTile) okt[threadIdx.x] = 1;
    __syncthreads();
    for (int e = threadIdx.x; e < nt * D; e += kPT) {
      const int tt = e / D, c = e % D;
      bool ok = true;
      kv[tt][c] = cache_key(v, b, h, t0 + tt, c, nq, &ok);
      if (!ok) okt[tt] = 0;  // every writer writes the same
    }
    __syncthreads();
    if (v.rope_pre) {
      for (int e = threadIdx.x; e < nt * (D / 2); e += kPT) {
        const int tt = e / (D / 2), i = e % (D / 2);
        float sn, cs;
        sincospif(2.f * rope_turns(t0 + tt, w_hi[i], w_lo[i]), &sn, &cs);
        const float kx = kv[tt][2 * i], ky = kv[tt][2 * i + 1];
        kv[tt][2 * i] = kx * cs - ky * sn;
        kv[tt][2 * i + 1] = kx * sn + ky * cs;
      }
      __syncthreads();
    }
    for (int e = threadIdx.x; e < kPRows * kPTile; e += kPT) {
      const int r = e / kPTile, tt = e % kPTile;
      float s = -INFINITY;
      if (tt < nt && okt[tt] && t0 + tt < ends[r]) {
        s = 0.f;
        for (int c = 0; c < D; ++c) s = fmaf(qs[r][c], kv[tt][c], s);
      }
      ps[r][tt] = s;
    }
    __syncthreads();
    for (int r = warp; r < kPRows; r += kPT / 32) {
      const float s = ps[r][lane];
      float mx = s;
      for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
      const float m = fmaxf(ms[r], mx);
      const bool seen = lane < nt && okt[lane] && t0 + lane < ends[r];
      const float p = s == -INFINITY ? 0.f : exp2f(s - m);
      float sum = p;
      for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
      const float alpha = m == -INFINITY ? 1.f : exp2f(ms[r] - m);
      __syncwarp();
      ps[r][lane] = seen ? p : -1.f;
      if (lane == 0) {
        al[r] = alpha;
        ls[r] = ls[r] * alpha + sum;
        ms[r] = m;
      }
      __syncwarp();
    }
    for (int e = threadIdx.x; e < nt * D; e += kPT) kv[e / D][e % D] = cache_value(v, b, h, t0 + e / D, e % D, nq);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kPRows; ++r) {
      const float alpha = al[r];
#pragma unroll
      for (int j = 0; j < kMaxHeadDim / kPT; ++j) {
        const int c = threadIdx.x + j * kPT;
        if (c >= D) continue;
        float s = o[r][j] * alpha;
        for (int tt = 0; tt < nt; ++tt) {
          const float p = ps[r][tt];
          if (!(p < 0.f)) s = fmaf(p, kv[tt][c], s);  // a token that the row does not see adds nothing, whatever it holds
        }
        o[r][j] = s;
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < kPRows; ++r) {
    if (r >= rows) break;
    const float inv = ls[r] == 0.f ? 0.f : 1.f / ls[r];  // NaN stays
#pragma unroll
    for (int j = 0; j < kMaxHeadDim / kPT; ++j) {
      const int c = threadIdx.x + j * kPT;
      if (c >= D) continue;
      const float y = o[r][j] * inv;
      if (a.out_f32) {
        static_cast<float*>(a.out)[row_elem(r) + c] = y;
      } else {
        static_cast<__nv_bfloat16*>(a.out)[row_elem(r) + c] = __float2bfloat16_rn(y);
      }
    }
  }
}

kvq_status launch_query_plain(const KvqView& v, const QueryArgs& a, cudaStream_t st) {
  const long long row_blocks = ((long long)a.n_q * v.n_rep + kPRows - 1) / kPRows;
  const long long grid = row_blocks * v.Hkv * v.batch;
  if (grid > 0x7FFFFFFFLL) return KVQ_ERR_CAPACITY;
  query_plain_kernel<<<(unsigned)grid, kPT, 0, st>>>(v, a, (int)row_blocks);
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace

// The tensor-core kernels take bf16 sources over PER_BLOCK caches of one format whose keys are stored
// rotated (or need no rotation).  A batch beyond 4096 sequences exceeds their plan's shared memory.
bool query_tc_shape(const KvqView& v) {
  return v.kaxis == KVQ_PER_BLOCK && v.kfmt == v.vfmt && v.src_bf16 && !v.rope_pre && v.batch <= 4096;
}

bool query_tc_eligible(const KvqView& v) {
  return query_tc_shape(v) && (long long)v.n_pages * v.page_bytes / 128 < (1LL << 31) && tensor_map_encoder() != nullptr;
}

// A call is small if passes of 8 rows over the tokens that its block table could hold are 2.5 units of 64 tokens, or
// fewer, for each of the warps that such passes fill the GPU with.  The kernel of 8 rows is the shortest, and what a
// short call waits for is its instructions (passes of 8 against one of 24 or 32 rows, us, 8 kv-heads of 128: 20 rows
// over 512 tokens 10.6 and 14.9, over 4 x 2,000 18.6 and 22.3, 32 rows over 4,101 18.5 and 25.8; beyond the bound 20 rows
// over 16 x 1,000 29.1 and 27.0, 32 over 40,000 57 and 52).
bool few_small(const KvqView& v, int batch, long long rows, long long tokens) {
  if (rows > kFewSmallRows) return false;
  const double units = (double)batch * v.Hkv * (double)((rows + 7) / 8) * (double)tokens / 64.0;
  return units <= 2.5 * 12 * num_sms();
}

// Which of the two: the few-row kernel reads the cache once per 32 rows (16 at head_dim 256 or with fp32 output) at
// close to the memory's rate; the many-row kernel reads it once per 256 and multiplies at the tensor cores' rate, but
// a unit of its work starts and ends slowly.  So the former takes up to 32 rows, small calls, and up to 64 or 256
// rows over few tokens (few-row against many-row kernel, us: 40 rows over 8 heads x 2,992 tokens 15 and 29, 64 rows
// over 512 x 224 40 and 50, 112 rows over 5 x 4,502 22 and 36; beyond the bounds 36 rows over 128 x 4,096 97 and 84,
// 64 rows over 56 x 5,666 75 and 58, 264 rows over 216 x 128 55 and 32).  head_dim 256 and fp32 output exceed the
// many-row kernel's shared and tensor memory.
static bool takes_few(const KvqView& v, int batch, long long rows, int out_f32, long long tokens) {
  if (rows <= kFewPass || v.D > 128 || out_f32 || few_small(v, batch, rows, tokens)) return true;
  const double pairs = (double)batch * v.Hkv, passes = (double)((rows + kFewPass - 1) / kFewPass);
  const double products = (double)rows * pairs * (double)tokens * v.D;
  return passes <= 2 ? pairs <= 2048.0 && products <= 2147483648.0
                     : passes <= kFewPasses && pairs * passes <= 1024.0 && products <= 536870912.0;
}

// Decode calls (fp32 output) take as many runs as their records fit the fixed scratch array of
// kvq_decode_attention_noalloc with, so that both entry points run the same plan and the latter takes wide groups too;
// where pairs alone fill it, all.
int few_runs(const KvqView& v, int batch, long long rows, int out_f32) {
  if (!out_f32) return kFewUnits;
  const long long passes = rows < 16 * kFewPasses ? (rows + 15) / 16 : kFewPasses, most = rows < 16 ? rows : 16;
  const long long fit = (long long)((KVQ_NOALLOC_SCRATCH_BYTES - few_header_bytes(batch)) / (most * (v.D + 4) * sizeof(float))) -
                        (long long)batch * v.Hkv * passes;
  return fit < kFewLeast || fit > kFewUnits ? kFewUnits : (int)fit;
}

static size_t few_bytes(const KvqView& v, int batch, long long rows, int out_f32) {
  const long long pass = v.D > 128 || out_f32 ? 16 : kFewPass, pairs = (long long)batch * v.Hkv;
  const long long passes = rows < pass * kFewPasses ? (rows + pass - 1) / pass : kFewPasses;
  const long long runs = few_runs(v, batch, rows, out_f32);
  long long records = (runs + pairs * passes) * (rows < pass ? rows : pass);
  if (few_small(v, batch, rows, v.P)) {  // as it may be, with the narrowest table
    const long long by8 = (runs + pairs * ((rows + 7) / 8)) * (rows < 8 ? rows : 8);
    if (by8 > records) records = by8;
  }
  return few_header_bytes(batch) + (size_t)records * (v.D + 4) * sizeof(float);
}

// What a call of n_q queries needs.
size_t query_call_bytes(const KvqView& v, int batch, int n_q) {
  KvqView b = v;
  b.batch = batch;
  if (!query_tc_shape(b)) return 256;
  const long long rows = (long long)n_q * v.n_rep;
  const size_t few = takes_few(v, batch, rows, 0, v.P) ? few_bytes(v, batch, rows, 0) : 0;
  if (takes_few(v, batch, rows, 0, 1LL << 62)) return few;
  const size_t many = query_many_workspace_bytes(v, batch, n_q);
  return few > many ? few : many;
}

// What any call of at most n_q queries needs: the few-row kernel's records can take more than the many-row kernel's, and
// up to kFewSmallRows rows may be the former's.
size_t query_workspace_bytes(const KvqView& v, int batch, int n_q) {
  size_t most = query_call_bytes(v, batch, n_q);
  const int few = (kFewSmallRows + v.n_rep - 1) / v.n_rep;
  static_assert(kFewPass * kFewPasses <= kFewSmallRows, "the most rows of the few-row kernel");
  for (int n = 1; n < n_q && n <= few; ++n) {
    const size_t x = query_call_bytes(v, batch, n);
    if (x > most) most = x;
  }
  return most;
}

// A decode call's (fp32 output, in passes of 16 rows).
size_t decode_workspace_bytes(const KvqView& v, int batch) {
  KvqView b = v;
  b.batch = batch;
  return query_tc_shape(b) ? few_bytes(v, batch, v.n_rep, 1) : 256;
}

kvq_status launch_query(const KvqView& v, const QueryArgs& a, void* ws, cudaStream_t st) {
  const long long rows = (long long)a.n_q * v.n_rep;
  if (!query_tc_eligible(v) || rows >= (1LL << 30) || (long long)v.batch * v.Hkv * kFewPasses * kFewPass > 0x7FFFFFFFLL)
    return launch_query_plain(v, a, st);
  if (!takes_few(v, v.batch, rows, a.out_f32, (long long)v.max_pages * v.P)) return launch_query_many(v, a, ws, st);
  return v.kfmt == KVQ_INT8 ? launch_query_few_i8(v, a, ws, st)
         : v.kfmt == KVQ_FP8_E4M3 ? launch_query_few_e4(v, a, ws, st)
                                  : launch_query_few_e5(v, a, ws, st);
}

}  // namespace kvq
