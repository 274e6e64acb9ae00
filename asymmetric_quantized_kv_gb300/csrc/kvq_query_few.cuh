// Attention of few rows (query token x query head) per kv-head over a PER_BLOCK cache:
// decode steps, drafts and short calls, bf16 sources, head_dim 64, 128 or 256.  The kernel
// takes 8, 16, 24 or 32 rows a pass (16 at head_dim 256); more rows take several passes, side
// by side in one launch.
//
// Mathematics, for a 16-token tile (it lies in one block of the cache, so one key scale ks
// and one value scale vs = 2^e f, f in [1, 2)): with code matrices C_k, C_v,
//   x = (q . C_k) (ks scale log2 e),   p = 2^(x + e - M),
//   l += p 2^-e,   o += (p f) C_v,   out = o / l,
// M a running maximum of x + e.  The value scale's exponent rides in the softmax's, so
// the products that enter the tensor cores stay near 1 whatever the scales are; M is
// raised only when a tile exceeds it by 2^8 (p f then stays below 2^9, inside f16).
// The operands are exact: every code is an f16 number, and a bf16 query row is one after
// scaling by a power of two (elements more than 2^25 below the row's largest drop bits).
// p f is rounded to f16 once (bf16 output: 2^-11 against the output's own 2^-8), or split
// in two f16 terms for fp32 output.
//
// What bounds it: reading the codes.  A warp owns a unit (sequence, chunk, kv-head) and
// streams 16-token tiles of keys and values through its own 3-stage ring, filled by 2-D
// TMA copies of the pool seen as rows of 128 bytes with the 128-byte swizzle, so warps
// never wait for one another.  Keys are the M operand of m16n8k16 (16 tokens x 8 rows),
// values, transposed on the way from shared memory, that of the second product (16
// channels x 8 rows); with more rows a converted operand serves up to four products.  p
// crosses from one layout to the other with movmatrix.  The window's tokens (bf16) take the
// same path from registers, each scaled by a power of two of its own: a shared one would let
// a large token take bits from tokens whose queries do not see it.  All work lies in one row
// that is cut into equal runs, one a warp or up to four; a second kernel merges a row's
// records.
//
// Measured (8 kv-heads of 128): 8 x 131,072 tokens with 8 rows 354 us, 6.1 TB/s (89% of the
// measured copy bandwidth); 64 sequences of 1,024 to 65,536 tokens, 1.10M in all, with 4
// rows 368 us, 6.1 TB/s; 16 drafts of 5 tokens, 20 rows, 46 us, 1.9 TB/s, bound by the warps' issue (two a
// scheduler at 255 registers); 1 x 4,101 tokens 11 us, bound by latency: 2.5 us to start
// and plan, 6 for a unit, mostly instructions that no cache holds yet, 2.5 for the merge.
#pragma once

#include <math.h>

#include "kvq_code.cuh"
#include "kvq_ptx.cuh"
#include "kvq_query.cuh"
#include "kvq_tmap.h"

namespace kvq {
namespace {

using namespace ptx;

constexpr int kTile = 16;
constexpr int kFWarps = 4;
constexpr int kFThreads = kFWarps * 32;
constexpr int kFStages = 3;
constexpr int kRounds = 4;          // units per warp at most
constexpr int kUnitTokens = 512;    // a warp takes several units only if they are this long
constexpr int kMinUnit = 64;        // tokens of the smallest chunk
constexpr float kLazy = 8.f;
constexpr float kMinit = -3e38f;  // below any logit

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}

// ---- plan: a sequence's work is its places (of 16 tokens, or 16 << sh where their number would pass 31 bits),
// for each of `heads` pairs of a kv-head and a pass of its rows.  All pairs' places lie in one row, cut into runs
// of the same length, a warp's work each; a pair that is cut leaves a record per run, which the merge joins.
// Where a warp gets one run, pairs are padded to whole runs if runs up to a quarter longer allow that (no warp
// then starts two units: 16 drafts of 5 tokens take 46 us, not 47.5); else a pair has kUnitCost places before its
// own, for its unit's start, and runs cross pairs: the warps' work is then even (64 sequences of 1,024 to 65,536
// tokens take 387 us, not 407; 128 of 466 tokens with 24 rows fill the warps once, not twice).
struct FewPlan {
  unsigned run;  // places of a run
  int runs, aligned, pad;
};
constexpr unsigned kUnitCost = 3;

__device__ __forceinline__ unsigned few_units(int T, int sh) { return ((unsigned)T + (kTile << sh) - 1) >> (4 + sh); }
__device__ __forceinline__ unsigned few_places(const FewPlan& p, unsigned n) {
  if (n == 0) return 0;
  return p.aligned ? (n + p.run - 1) / p.run * p.run : n + kUnitCost;
}

// One warp; pref: B + 1 ints of shared memory, the places before a sequence.  workers: warps of the grid; max_runs: the
// call's, one a warp at least.  Lanes over the sequences, whose lengths are read once (a decode step's time is a chain of
// such latencies).
__device__ inline void few_plan(const KvqView& v, int heads, int sh, int workers, int max_runs, unsigned* pref, FewPlan* plan) {
  const int B = v.batch, lane = threadIdx.x & 31;
  unsigned sum = 0, some = 0;
#pragma unroll 1
  for (int b = lane; b < B; b += 32) {
    const unsigned n = few_units(seq_tokens(v, b), sh);
    pref[b] = n;
    sum += n;
    some += n > 0;
  }
  const unsigned work = __reduce_add_sync(0xffffffffu, sum) * heads;
  const unsigned rounds = min(max(work / workers / (unsigned)max(1, kUnitTokens >> (4 + sh)), 1u),
                              (unsigned)min(kRounds, max(1, max_runs / workers)));
  const unsigned most = min(rounds * (unsigned)workers, (unsigned)max_runs);
  FewPlan p;
  p.run = max((work + most - 1) / most, (unsigned)(kMinUnit / kTile));
  p.aligned = rounds == 1;
  const unsigned longest = p.run + p.run / 4;
  unsigned runs = 0;
#pragma unroll 1
  while (p.aligned) {
    runs = 0;
#pragma unroll 1
    for (int b = lane; b < B; b += 32) runs += (pref[b] + p.run - 1) / p.run;
    runs = __reduce_add_sync(0xffffffffu, runs) * heads;
    if (runs <= most) break;
    p.run += p.run / 16 + 1;
    p.aligned = p.run <= longest;
  }
  if (!p.aligned) {
    const unsigned places = work + __reduce_add_sync(0xffffffffu, some) * heads * kUnitCost;
    p.run = max((places + most - 1) / most, 1u);
    runs = (places + p.run - 1) / p.run;
  }
  p.runs = (int)runs;
  p.pad = 0;
  unsigned before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int b = b0 + lane;
    const unsigned x = b < B ? few_places(p, pref[b]) * heads : 0;
    unsigned incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (b < B) pref[b] = before + incl - x;
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) {
    pref[B] = before;
    *plan = p;
  }
}

// Whether the ring's phase ended within kWaitPolls tries, each of which suspends for some time.
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitPolls; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}

// Rows of a pass: 8 NB.  The query operand stays in registers up to 32 of them, else in shared memory.
template <int D, int NB>
constexpr bool query_in_smem() { return NB * (D / 16) > 16; }

// CTAs an SM: with 128, 168 or 255 registers a thread.
template <int D, int NB>
constexpr int few_ctas() { return D == 64 && NB == 1 ? 4 : D * NB <= 128 ? 3 : 2; }

template <int D, int NB>
struct __align__(1024) FewSmem {
  uint8_t kv[kFWarps][kFStages][2][kTile * D];
  uint2 bq[query_in_smem<D, NB>() ? kFWarps : 1][query_in_smem<D, NB>() ? NB : 1][D / 16][32];
  uint64_t bar[kFWarps][kFStages];
  int valid[kFWarps][kFStages];
};

// Byte o of a 1024-byte aligned tile under the 128-byte swizzle.
__device__ __forceinline__ uint32_t swz(uint32_t o) { return o ^ (((o >> 7) & 7u) << 4); }

// Rows of a 16-token value tile with a code that is not finite are zeroed, and the first such token noted.
template <int D>
__device__ __forceinline__ void drop_not_finite(uint8_t* vt, int lane, FiniteTest test, int tok, int& bad_from) {
  const uint32_t at = (lane >> 1) * D + (lane & 1) * (D / 2);  // half a row a lane
  uint32_t carries = 0u;
#pragma unroll 1
  for (int c = 0; c < D / 2; c += 16) {
    const uint4 x = *reinterpret_cast<const uint4*>(vt + swz(at + c));
    carries |= test.carry(x.x) | test.carry(x.y) | test.carry(x.z) | test.carry(x.w);
  }
  const uint32_t bad = __ballot_sync(0xffffffffu, test.fails(carries));
  if (bad) {
    bad_from = min(bad_from, tok + (__ffs(bad) - 1) / 2);
    if ((bad >> (lane & ~1)) & 3u) {
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 16) *reinterpret_cast<uint4*>(vt + swz(at + c)) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async();  // the slot's next copy comes after these
    __syncwarp();
  }
}

// The same for the second product's words of four window rows (tokens 2t, 2t + 1, 2t + 8, 2t + 9 of the tile).
template <int W>
__device__ __forceinline__ void drop_not_finite(uint32_t (&wv)[4][W], int tok, int& bad_from) {
  constexpr FiniteTest test = kFiniteBf16x2;
  const int t = threadIdx.x & 3;
  uint32_t bad = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t carries = 0u;
#pragma unroll
    for (int c = 0; c < W; ++c) carries |= test.carry(wv[j][c]);
    if (test.fails(carries)) bad |= 1u << (2 * t + (j & 1) + 8 * (j >> 1));
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (bad) {
    bad_from = min(bad_from, tok + __ffs(bad) - 1);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if ((bad >> (2 * t + (j & 1) + 8 * (j >> 1))) & 1u)
#pragma unroll
        for (int c = 0; c < W; ++c) wv[j][c] = 0u;
  }
}

template <int F, int D, int NB, bool kF32>
__global__ void __launch_bounds__(kFThreads, few_ctas<D, NB>())
    query_few_kernel(KvqView v, QueryArgs a, int row_base, int passes, int sh, int max_runs, float* ws, int dynamic,
                     const __grid_constant__ CUtensorMap tmap) {
  constexpr int NS = D / 16;      // steps of the first product, and channel tiles of the second
  constexpr int LC = D / 4;       // channels a lane holds of a key row
  constexpr int GC = D / 8;       // channels a lane holds of a value row
  constexpr int KB = kTile * D;   // bytes of a tile
  extern __shared__ unsigned char dyn_raw[];
  unsigned char* dyn = dyn_raw + ((1024 - (smem_u32(dyn_raw) & 1023)) & 1023);
  FewSmem<D, NB>& sm = *reinterpret_cast<FewSmem<D, NB>*>(dyn);
  unsigned* pref = reinterpret_cast<unsigned*>(dyn + sizeof(FewSmem<D, NB>));
  __shared__ FewPlan s_plan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int workers = gridDim.x * kFWarps, heads = v.Hkv * passes;
  if (warp == 0) few_plan(v, heads, sh, workers, max_runs, pref, &s_plan);
  __syncthreads();
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) *reinterpret_cast<FewPlan*>(ws) = s_plan;
    unsigned* hd = reinterpret_cast<unsigned*>(reinterpret_cast<char*>(ws) + sizeof(FewPlan));
#pragma unroll 1
    for (int b = threadIdx.x; b <= v.batch; b += kFThreads) hd[b] = pref[b];
  }
  grid_dep_launch();
  if (lane == 0) {
    for (int s = 0; s < kFStages; ++s) mbar_init(&sm.bar[warp][s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  const FewPlan plan = s_plan;
  const int rows_max = min(8 * NB, a.n_q * v.n_rep - row_base);
  unsigned* counter = reinterpret_cast<unsigned*>(reinterpret_cast<char*>(ws) + few_counter_offset(v.batch));
  float* part = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + few_header_bytes(v.batch));
  int lstage = 0, cstage = 0;
  uint32_t cphase = 0, n_loaded = 0, n_consumed = 0;
  bool stalled = false;

  int run = blockIdx.x * kFWarps + warp;
  unsigned pos = 0, stop = 0, nxt = 0;
  while (true) {
    if (pos >= stop) {
      if (stop) run = dynamic ? workers + (int)__shfl_sync(0xffffffffu, nxt, 0) : run + workers;
      if (run >= plan.runs) break;
      if (dynamic && lane == 0) nxt = atomicAdd(counter, 1u);  // the next run, known by the time this one ends
      pos = run * plan.run;
      stop = min(pos + plan.run, pref[v.batch]);
    }
    int lo = 0, hi = v.batch - 1;  // largest b with pref[b] <= pos (sequences without places share a value)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pref[mid] <= pos) lo = mid; else hi = mid - 1;
    }
    const int b = lo, T = seq_tokens(v, b);
    const unsigned units = few_units(T, sh), skip = plan.aligned ? 0 : kUnitCost;
    const unsigned places = (pref[b + 1] - pref[b]) / heads, off = pos - pref[b], hp = off / places, at = off - hp * places;
    const unsigned here = min(places - at, stop - pos);
    const unsigned j0 = max(at, skip) - skip, j1 = min(units, max(at + here, skip) - skip);  // its share of the pair
    pos += here;
    if (j0 >= j1) continue;
    int h = hp, row0 = row_base;
    if (passes > 1) {
      h = (int)hp / passes;
      row0 += ((int)hp - h * passes) * 8 * NB;
    }
    const int nq = n_quantized(T, v.R), n = query_count(v, a, b), rows = n * v.n_rep - row0;
    // no token that the pass's last row does not see (the call's last row sees them all)
    const int seen = rows <= 0 ? 0 : rows <= 8 * NB ? T : query_end(a, T, n, (row0 + 8 * NB - 1) / v.n_rep);
    // Tiles behind this hold tokens that some rows do not see.  A weight of zero would not keep such a row from a value
    // that is not finite; so there those values are left out, and the rows that see one get NaN for their sum.
    const int all_see = rows > 0 ? query_end(a, T, n, row0 / v.n_rep) : T;
    int bad_from = 0x7fffffff;
    const int t0 = (int)(j0 << (4 + sh));
    const int t1 = max(t0, (int)min(min((unsigned)T, few_units(seen, 0) * kTile), j1 << (4 + sh)));
    const int tq = min(t1, nq);                                // tiles before tq come from the pages
    const int qtiles = tq > t0 ? (tq - t0) / kTile : 0;        // nq and t0 are multiples of 16
    const int tiles = (t1 - t0 + kTile - 1) / kTile;
    const int32_t* bt = v.block_table + (long long)b * v.max_pages;
    const long long head_off = (long long)h * v.head_bytes;

    // ---- the ring: lane 0 walks page and slot; the next page's id is read a tile ahead
    int pg = t0 / v.P, slot = t0 % v.P, pid = 0, pid_next = 0;
    auto issue = [&]() {
      const int stage = lstage;
      if (++lstage == kFStages) lstage = 0;
      ++n_loaded;
      uint64_t* bar = &sm.bar[warp][stage];
      const bool ok = pid >= 0 && pid < v.n_pages;
      sm.valid[warp][stage] = ok;
      if (!ok) {
        atomicOr(v.status, KVQ_DEV_BAD_PAGE);
        mbar_arrive(bar);
      } else {
        const long long byte0 = (long long)pid * v.page_bytes + head_off + (long long)slot * D;
        const int yk = (int)(byte0 >> 7), yv = yk + (v.off_vc >> 7);
        mbar_arrive_expect_tx(bar, 2 * KB);
        const uint64_t pol = l2_evict_first();
        tma_load_2d_hint(sm.kv[warp][stage][0], &tmap, 0, yk, bar, pol);
        tma_load_2d_hint(sm.kv[warp][stage][1], &tmap, 0, yv, bar, pol);
      }
      slot += kTile;
      if (slot >= v.P) {
        slot = 0;
        ++pg;
        pid = pid_next;
        pid_next = pg + 1 < v.max_pages ? bt[pg + 1] : -1;
      }
    };
    if (lane == 0 && !stalled && qtiles > 0) {
      pid = bt[pg];
      pid_next = pg + 1 < v.max_pages ? bt[pg + 1] : -1;
      fence_proxy_async();
      for (int i = 0; i < min(kFStages, qtiles); ++i) issue();
    }
    // ---- block scales: lane j holds those of block blk0 + j of the unit
    float ks_l = 0.f, vs_l = 0.f;
    bool sok_l = true;
    int blk0 = t0 / v.kgroup, blk = 0, left = (v.kgroup - (t0 - blk0 * v.kgroup)) / kTile;  // tiles left of block blk0 + blk
    auto load_scales = [&]() {
      const int g0 = (blk0 + lane) * v.kgroup;
      ks_l = vs_l = 0.f;
      sok_l = true;
      if (g0 < tq) {
        const int p = bt[g0 / v.P];
        sok_l = p >= 0 && p < v.n_pages;
        if (sok_l) {
          const uint8_t* hb = v.pages + (long long)p * v.page_bytes + head_off;
          const int s = (g0 % v.P) / v.kgroup;
          ks_l = load_meta(hb + v.off_km, s, v.meta16);
          vs_l = load_meta(hb + v.off_vm, s, v.meta16);
        } else {
          atomicOr(v.status, KVQ_DEV_BAD_PAGE);
        }
      }
    };
    if (qtiles > 0) load_scales();

    // ---- queries: column g is row g; lane (g, t) holds its channels t LC .. t LC + LC - 1, brought into
    // f16 by the row's power of two
    constexpr bool kQS = query_in_smem<D, NB>();
    uint32_t bq[kQS ? 1 : NB][NS][2];
    float fct[NB][2];  // this lane's logits are those of rows 2t, 2t + 1 of each block: their factor,
    int end[NB][2];    // and the tokens they see
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      uint32_t u[LC / 2];
#pragma unroll
      for (int i = 0; i < LC / 2; ++i) u[i] = 0u;
      if (8 * nb + g < rows) {
        const int row = row0 + 8 * nb + g;
        const long long qi = (((long long)b * a.n_q + row / v.n_rep) * v.Hq + h * v.n_rep + row % v.n_rep) * D + t * LC;
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + qi);
#pragma unroll
        for (int i = 0; i < LC / 8; ++i) {
          const uint4 x = p[i];
          u[4 * i] = x.x; u[4 * i + 1] = x.y; u[4 * i + 2] = x.z; u[4 * i + 3] = x.w;
        }
      }
      uint32_t m2 = 0u;
#pragma unroll
      for (int i = 0; i < LC / 2; ++i) m2 = bf16x2_absmax(m2, u[i]);
      uint32_t top = max(m2 & 0xffffu, m2 >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      float down, up;
      norm_factors(top, down, up);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const uint32_t x = bf16x2_scaled(u[2 * s], down), y = bf16x2_scaled(u[2 * s + 1], down);
        if constexpr (kQS) {
          sm.bq[warp][nb][s][lane] = make_uint2(x, y);
        } else {
          bq[nb][s][0] = x;
          bq[nb][s][1] = y;
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nb + 2 * t + e;
        fct[nb][e] = __shfl_sync(0xffffffffu, up, 8 * t + 4 * e) * a.scale * 1.4426950408889634f;
        end[nb][e] = r < rows ? query_end(a, T, n, (row0 + r) / v.n_rep) : 0;
      }
    }
    __syncwarp();
    auto query = [&](int nb, int s) -> uint2 {
      if constexpr (kQS) return sm.bq[warp][nb][s][lane];
      else return make_uint2(bq[nb][s][0], bq[nb][s][1]);
    };

    float O[NB][NS][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int m = 0; m < NS; ++m) O[nb][m][0] = O[nb][m][1] = O[nb][m][2] = O[nb][m][3] = 0.f;
    float m_run[NB][2], l_run[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m_run[nb][0] = m_run[nb][1] = kMinit;
      l_run[nb][0] = l_run[nb][1] = 0.f;
    }

    // logits of the tile at token tok (acc: token g / g + 8 x row 2t / 2t + 1) -> B operands of the second
    // product; scale of the keys, and of the values as 2^e f, of tokens g (kf0, e0) and g + 8
    auto softmax = [&](const float (&acc)[NB][4], int tok, float kf0, float kf1, int e0, int e1, float f, uint32_t (&ph)[NB][2],
                       uint32_t (&pl)[NB][2]) {
      const float fe0 = (float)e0, fe1 = (float)e1, ie0 = pow2i(-e0), ie1 = pow2i(-e1);
      float x[NB][2][2];  // [block][token g / g + 8][row]
      bool need = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          x[nb][0][r] = tok + g < end[nb][r] ? fmaf(acc[nb][r], kf0 * fct[nb][r], fe0) : -INFINITY;
          x[nb][1][r] = tok + g + 8 < end[nb][r] ? fmaf(acc[nb][2 + r], kf1 * fct[nb][r], fe1) : -INFINITY;
          need = need || fmaxf(x[nb][0][r], x[nb][1][r]) > m_run[nb][r] + kLazy;
        }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float mx = fmaxf(x[nb][0][r], x[nb][1][r]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mn = fmaxf(m_run[nb][r], mx), al = ex2(m_run[nb][r] - mn);
            m_run[nb][r] = mn;
            l_run[nb][r] *= al;
#pragma unroll
            for (int m = 0; m < NS; ++m) {  // columns 2t, 2t + 1 of the outputs are the same rows
              O[nb][m][r] *= al;
              O[nb][m][2 + r] *= al;
            }
          }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float p[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          p[0][r] = ex2(x[nb][0][r] - m_run[nb][r]);
          p[1][r] = ex2(x[nb][1][r] - m_run[nb][r]);
          l_run[nb][r] = e0 == e1 ? fmaf(p[0][r] + p[1][r], ie0, l_run[nb][r])
                                  : fmaf(p[0][r], ie0, fmaf(p[1][r], ie1, l_run[nb][r]));
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if constexpr (kF32) {
            uint32_t hi2, lo2;
            split_hi_lo(p[k][0] * f, p[k][1] * f, hi2, lo2);
            ph[nb][k] = movmatrix(hi2);
            pl[nb][k] = movmatrix(lo2);
          } else {
            ph[nb][k] = movmatrix(pack_f16x2(p[k][0] * f, p[k][1] * f));
          }
        }
      }
    };

    for (int i = 0; i < qtiles; ++i) {
      const int tok = t0 + i * kTile, stage = cstage;
      bool valid = false;
      if (!stalled) {
        if (!ring_wait(&sm.bar[warp][stage], cphase)) {
          atomicOr(v.status, KVQ_DEV_TIMEOUT);
          stalled = true;
        } else {
          valid = sm.valid[warp][stage] != 0;
        }
      }
      if (++cstage == kFStages) {
        cstage = 0;
        cphase ^= 1u;
      }
      ++n_consumed;
      const float kf = __shfl_sync(0xffffffffu, ks_l, blk);
      float vf = __shfl_sync(0xffffffffu, vs_l, blk);
      valid = valid && __shfl_sync(0xffffffffu, (int)sok_l, blk);
      if (--left == 0) {
        left = v.kgroup / kTile;
        if (++blk == 32) {
          blk0 += 32;
          blk = 0;
          load_scales();
        }
      }
      if (__all_sync(0xffffffffu, valid)) {  // a tile without its page, or its scales, takes no weight
        const uint8_t* kt = sm.kv[warp][stage][0];
        const uint8_t* vt = sm.kv[warp][stage][1];
        if (__builtin_expect(tok + kTile > all_see, 0)) {
          if constexpr (F != kI8)
            drop_not_finite<D>(sm.kv[warp][stage][1], lane, F == kE4 ? kFiniteE4 : kFiniteE5, tok, bad_from);
          if (!(vf < INFINITY)) {
            bad_from = min(bad_from, tok);
            vf = 0.f;
          }
        }
        float acc[NB][4], odd[4] = {0.f, 0.f, 0.f, 0.f};  // one block: two chains of half the length
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[nb][0] = acc[nb][1] = acc[nb][2] = acc[nb][3] = 0.f;
#pragma unroll
        for (int c = 0; c < LC / 16; ++c) {
          const uint4 k0 = *reinterpret_cast<const uint4*>(kt + swz(g * D + t * LC + 16 * c));
          const uint4 k1 = *reinterpret_cast<const uint4*>(kt + swz((g + 8) * D + t * LC + 16 * c));
          const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t a0, a1, a2, a3;
            codes_to_f16<F>(w0[j], a0, a2);
            codes_to_f16<F>(w1[j], a1, a3);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              const uint2 b2 = query(nb, 4 * c + j);
              mma_16816(NB == 1 && (j & 1) ? odd : acc[nb], a0, a1, a2, a3, b2.x, b2.y);
            }
          }
        }
        if constexpr (NB == 1) {
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) acc[0][i4] += odd[i4];
        }
        const int e = vf == 0.f ? kZeroExp : min(126, max(kMinExp, exponent_of(vf)));
        const float f = vf * pow2i(-e);  // in [1, 2), or less below 2^kMinExp
        uint32_t ph[NB][2], pl[NB][2];
        softmax(acc, tok, kf, kf, e, e, f, ph, pl);
        // ---- second product: rows g / g + 8 of channel tile m = channels g GC + 2m / + 1,
        //      k-slots = tokens 2t, 2t + 1, 2t + 8, 2t + 9
        constexpr int W = GC / 4;  // words of a value row a lane holds
        uint32_t wv[4][W];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 2 * t + (j & 1) + 8 * (j >> 1);
          if constexpr (W == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(vt + swz(r * D + g * GC));
            wv[j][0] = x.x;
            wv[j][1] = x.y;
          } else {
#pragma unroll
            for (int c = 0; c < W / 4; ++c) {
              const uint4 x = *reinterpret_cast<const uint4*>(vt + swz(r * D + g * GC + 16 * c));
              wv[j][4 * c] = x.x; wv[j][4 * c + 1] = x.y; wv[j][4 * c + 2] = x.z; wv[j][4 * c + 3] = x.w;
            }
          }
        }
#pragma unroll
        for (int m = 0; m < NS; ++m) {
          // bytes 2 (m % 2), 2 (m % 2) + 1 of word m / 2 of two tokens: (even channel: both, odd channel: both)
          const uint32_t sel = (m & 1) ? 0x7362u : 0x5140u;
          uint32_t a0, a1, a2, a3;
          codes_to_f16<F>(prmt(wv[0][m >> 1], wv[1][m >> 1], sel), a0, a1);
          codes_to_f16<F>(prmt(wv[2][m >> 1], wv[3][m >> 1], sel), a2, a3);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma_16816(O[nb][m], a0, a1, a2, a3, ph[nb][0], ph[nb][1]);
            if constexpr (kF32) mma_16816(O[nb][m], a0, a1, a2, a3, pl[nb][0], pl[nb][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0 && i + kFStages < qtiles && !stalled) {
        fence_proxy_async();
        issue();
      }
    }

    // ---- the window's tokens: bf16 rows, a power of two per token in place of the scales
    for (int i = qtiles; i < tiles; ++i) {
      const int tok = t0 + i * kTile;
      const uint16_t* kw = static_cast<const uint16_t*>(v.k_win) + (((long long)b * v.R + (tok - nq)) * v.Hkv + h) * D;
      const uint16_t* vw = static_cast<const uint16_t*>(v.v_win) + (((long long)b * v.R + (tok - nq)) * v.Hkv + h) * D;
      const long long pitch = (long long)v.Hkv * D;
      const uint4 z4 = make_uint4(0u, 0u, 0u, 0u);
      float acc[NB][4], kf0, kf1;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) acc[nb][0] = acc[nb][1] = acc[nb][2] = acc[nb][3] = 0.f;
      {
        uint32_t x0[LC / 2], x1[LC / 2], m0 = 0u, m1 = 0u;
#pragma unroll
        for (int c = 0; c < LC / 8; ++c) {
          const uint4 y0 = tok + g < t1 ? *reinterpret_cast<const uint4*>(kw + g * pitch + t * LC + 8 * c) : z4;
          const uint4 y1 = tok + g + 8 < t1 ? *reinterpret_cast<const uint4*>(kw + (g + 8) * pitch + t * LC + 8 * c) : z4;
          x0[4 * c] = y0.x; x0[4 * c + 1] = y0.y; x0[4 * c + 2] = y0.z; x0[4 * c + 3] = y0.w;
          x1[4 * c] = y1.x; x1[4 * c + 1] = y1.y; x1[4 * c + 2] = y1.z; x1[4 * c + 3] = y1.w;
        }
#pragma unroll
        for (int c = 0; c < LC / 2; ++c) {
          m0 = bf16x2_finite_max(m0, x0[c]);
          m1 = bf16x2_finite_max(m1, x1[c]);
        }
        m0 = finite_top(m0);
        m1 = finite_top(m1);
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {  // over the four lanes of a row
          m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, o));
          m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, o));
        }
        float down0, down1;
        norm_factors(m0, down0, kf0);
        norm_factors(m1, down1, kf1);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const uint32_t a0 = bf16x2_scaled(x0[2 * s], down0), a1 = bf16x2_scaled(x1[2 * s], down1);
          const uint32_t a2 = bf16x2_scaled(x0[2 * s + 1], down0), a3 = bf16x2_scaled(x1[2 * s + 1], down1);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const uint2 b2 = query(nb, s);
            mma_16816(acc[nb], a0, a1, a2, a3, b2.x, b2.y);
          }
        }
      }
      constexpr int W = GC / 2;  // bf16 pairs of a value row a lane holds
      uint32_t wv[4][W], exps = 0u;  // exponents of the four rows, a byte each
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 2 * t + (j & 1) + 8 * (j >> 1);
#pragma unroll
        for (int c = 0; c < W / 4; ++c) {
          const uint4 x = tok + r < t1 ? *reinterpret_cast<const uint4*>(vw + r * pitch + g * GC + 8 * c) : z4;
          wv[j][4 * c] = x.x; wv[j][4 * c + 1] = x.y; wv[j][4 * c + 2] = x.z; wv[j][4 * c + 3] = x.w;
        }
        uint32_t m2 = 0u;
#pragma unroll
        for (int c = 0; c < W; ++c) m2 = bf16x2_finite_max(m2, wv[j][c]);
        m2 = finite_top(m2);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) m2 = max(m2, __shfl_xor_sync(0xffffffffu, m2, o));  // over the row's eight lanes
        exps |= (uint32_t)(value_exponent(m2) & 0xff) << (8 * j);
      }
      if (__builtin_expect(tok + kTile > all_see, 0)) drop_not_finite(wv, tok, bad_from);
      const uint32_t mine = __shfl_sync(0xffffffffu, exps, g >> 1) >> (8 * (g & 1));  // of tokens g, g + 8
      uint32_t ph[NB][2], pl[NB][2];
      softmax(acc, tok, kf0, kf1, (int8_t)mine, (int8_t)(mine >> 16), 1.f, ph, pl);
      float down[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) down[j] = pow2i(-(int8_t)(exps >> (8 * j)));
#pragma unroll
      for (int m = 0; m < NS; ++m) {  // channels g GC + 2m, + 1 are pair m of each row
        const uint32_t y0 = bf16x2_scaled(wv[0][m], down[0]), y1 = bf16x2_scaled(wv[1][m], down[1]);
        const uint32_t y2 = bf16x2_scaled(wv[2][m], down[2]), y3 = bf16x2_scaled(wv[3][m], down[3]);
        const uint32_t a0 = prmt(y0, y1, 0x5410u), a1 = prmt(y0, y1, 0x7632u);
        const uint32_t a2 = prmt(y2, y3, 0x5410u), a3 = prmt(y2, y3, 0x7632u);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          mma_16816(O[nb][m], a0, a1, a2, a3, ph[nb][0], ph[nb][1]);
          if constexpr (kF32) mma_16816(O[nb][m], a0, a1, a2, a3, pl[nb][0], pl[nb][1]);
        }
      }
    }

    // ---- the unit's records
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l_run[nb][r] += __shfl_xor_sync(0xffffffffu, l_run[nb][r], o);
        const int row = 8 * nb + 2 * t + r;
        if (row < rows) {
          float* rec = part + ((long long)(run + b * heads + (int)hp) * rows_max + row) * (D + 4);
          if (g == 0) {
            rec[0] = m_run[nb][r];
            rec[1] = end[nb][r] > bad_from ? __int_as_float(0x7fffffff) : l_run[nb][r];
          }
#pragma unroll
          for (int m = 0; m < NS; ++m)
            *reinterpret_cast<float2*>(rec + 4 + g * GC + 2 * m) = make_float2(O[nb][m][r], O[nb][m][2 + r]);
        }
      }
    __syncwarp();
  }
  if (lane == 0) {  // copies issued and not consumed (a stalled ring): wait for them, bounded, before leaving
    while (n_consumed < n_loaded) {
      ring_wait(&sm.bar[warp][cstage], cphase);
      if (++cstage == kFStages) {
        cstage = 0;
        cphase ^= 1u;
      }
      ++n_consumed;
    }
  }
}

// Rows that are merged.  Up to one an SM: a CTA of 16 warps each, the warps over every sixteenth record, lanes over
// channel pairs or quads, merged through shared memory (32 rows of 65 records: a decode step of 4,101 tokens takes
// 11.3 us so, 12.5 with 4 warps, 18.4 with a warp a row).  More: 4 warps a row (2,560 rows of 9 records: 45 us with
// the products, 74 with 16 warps, 51 with a warp a row).  Many, with few records each: a warp a row (24,576 rows:
// 49 us with the products, 76 with 4 warps a row).
constexpr long long kSoloRows = 4096;
constexpr int kSoloWarps = 4;
template <int D, bool kF32, int kMWarps>
__global__ void __launch_bounds__(kMWarps * 32)
    few_merge_kernel(KvqView v, QueryArgs a, int row_base, int passes, int sh, int rows_max, int solo, const float* ws) {
  constexpr int PER = D / 32;  // channels per lane: 2, 4 or 8
  __shared__ float o_s[kMWarps][D];
  __shared__ float m_s[kMWarps], l_s[kMWarps];
  const int heads = v.Hkv * passes;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned idx = solo ? blockIdx.x * kMWarps + warp : blockIdx.x;
  const int r = idx % rows_max, x = idx / rows_max, hp = x % heads, b = x / heads;
  int h = hp, row = row_base + r;
  if (passes > 1) {
    h = hp / passes;
    row += (hp - h * passes) * rows_max;
  }
  const int i = row / v.n_rep, hq = h * v.n_rep + (row - i * v.n_rep);
  const bool some = b < v.batch && i < query_count(v, a, b);
  const unsigned units = some ? few_units(seq_tokens(v, b), sh) : 0;
  grid_dep_wait();  // every CTA: where no row has a query, the end of this grid still follows the first kernel's
  if (!some) return;
  const FewPlan plan = *reinterpret_cast<const FewPlan*>(ws);
  const unsigned* pref =
      reinterpret_cast<const unsigned*>(reinterpret_cast<const char*>(ws) + sizeof(FewPlan));
  const unsigned first = pref[b] + hp * few_places(plan, units) + (plan.aligned ? 0 : kUnitCost);
  const int run0 = (int)(first / plan.run), nc = units ? (int)((first + units - 1) / plan.run) - run0 + 1 : 0;
  const long long stride = (long long)rows_max * (D + 4);
  const float* rec = reinterpret_cast<const float*>(reinterpret_cast<const char*>(ws) + few_header_bytes(v.batch)) +
                     ((long long)(run0 + b * heads + hp) * rows_max + r) * (D + 4);
  float m = kMinit, l = 0.f, o[PER];
#pragma unroll
  for (int c = 0; c < PER; ++c) o[c] = 0.f;
  constexpr int kBatch = kMWarps > 4 ? 8 : 4;
  const int stepk = solo ? 1 : kMWarps;
#pragma unroll 1
  for (int k0 = solo ? 0 : warp; k0 < nc; k0 += stepk * kBatch) {
    float rm[kBatch], rl[kBatch], y[kBatch][PER];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int k = k0 + j * stepk;
      rm[j] = kMinit;
      rl[j] = 0.f;
#pragma unroll
      for (int c = 0; c < PER; ++c) y[j][c] = 0.f;
      if (k < nc) {
        const float* rk = rec + (long long)k * stride;
        const float2 ml = *reinterpret_cast<const float2*>(rk);
        rm[j] = ml.x;
        rl[j] = ml.y;
#pragma unroll
        for (int c = 0; c < PER; c += 2) {
          const float2 z = *reinterpret_cast<const float2*>(rk + 4 + lane * PER + c);
          y[j][c] = z.x;
          y[j][c + 1] = z.y;
        }
      }
    }
    float mn = m;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) mn = fmaxf(mn, rm[j]);
    const float al = exp2f(m - mn);
    l *= al;
#pragma unroll
    for (int c = 0; c < PER; ++c) o[c] *= al;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const float w = exp2f(rm[j] - mn);
      l = fmaf(rl[j], w, l);
#pragma unroll
      for (int c = 0; c < PER; ++c) o[c] = fmaf(y[j][c], w, o[c]);
    }
    m = mn;
  }
  const long long out0 = (((long long)b * a.n_q + i) * v.Hq + hq) * D;
  if (solo) {
    const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN stays
#pragma unroll
    for (int c = 0; c < PER; c += 2) {
      const long long at = out0 + lane * PER + c;
      if (kF32) {
        static_cast<float*>(a.out)[at] = o[c] * inv;
        static_cast<float*>(a.out)[at + 1] = o[c + 1] * inv;
      } else {
        *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + at) =
            __floats2bfloat162_rn(o[c] * inv, o[c + 1] * inv);
      }
    }
    return;
  }
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
#pragma unroll
  for (int c = 0; c < PER; ++c) o_s[warp][lane * PER + c] = o[c];
  __syncthreads();
  float M = kMinit, L = 0.f;
#pragma unroll
  for (int w = 0; w < kMWarps; ++w) M = fmaxf(M, m_s[w]);
#pragma unroll
  for (int w = 0; w < kMWarps; ++w) L = fmaf(l_s[w], exp2f(m_s[w] - M), L);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  for (int c = threadIdx.x; c < D; c += kMWarps * 32) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kMWarps; ++w) s = fmaf(o_s[w][c], exp2f(m_s[w] - M), s);
    s *= inv;
    if (kF32) {
      static_cast<float*>(a.out)[out0 + c] = s;
    } else {
      static_cast<__nv_bfloat16*>(a.out)[out0 + c] = __float2bfloat16_rn(s);
    }
  }
}

template <int F, int D, int NB, bool kF32>
kvq_status launch_few_t(const KvqView& v, const QueryArgs& a, int row0, int passes, float* ws, const CUtensorMap& tmap,
                        cudaStream_t st) {
  constexpr int kMaxBatch = 4096;  // the plan's prefix in shared memory (query_tc_shape)
  constexpr int kNB = NB - 1, kDi = D == 64 ? 0 : D == 128 ? 1 : 2;
  const auto kern = query_few_kernel<F, D, NB, kF32>;
  const size_t smem = sizeof(FewSmem<D, NB>) + 1024 + sizeof(int) * (v.batch + 1);
  int occ = 0;
  const kvq_status so = occupancy_once(kSlotQueryFew + ((F * 3 + kDi) * 4 + kNB) * 2 + (kF32 ? 1 : 0), kern, kFThreads,
                                       sizeof(FewSmem<D, NB>) + 1024 + sizeof(int) * 65,
                                       sizeof(FewSmem<D, NB>) + 1024 + sizeof(int) * (kMaxBatch + 1), &occ);
  if (so != KVQ_OK) return so;
  int grid = num_sms() * occ;
  const int max_runs = few_runs(v, v.batch, (long long)a.n_q * v.n_rep, a.out_f32);
  if (grid > max_runs / kFWarps) grid = max_runs / kFWarps;
  // warps take their next unit from a counter where one may come (workers run at unequal speed);
  // a call too small for that saves the counter's clearing
  const long long pairs = (long long)v.batch * v.Hkv * passes;
  int sh = 0;
  while (pairs * (((long long)v.max_pages * v.P >> (4 + sh)) + kUnitCost + 1) > (1LL << 30)) ++sh;
  const long long most = pairs * v.max_pages * v.P;
  const int dynamic = most > (long long)grid * kFWarps * kUnitTokens;
  if (dynamic && cudaMemsetAsync(reinterpret_cast<char*>(ws) + few_counter_offset(v.batch), 0, 8, st) != cudaSuccess)
    return KVQ_ERR_CUDA;
  kern<<<grid, kFThreads, smem, st>>>(v, a, row0, passes, sh, max_runs, ws, dynamic, tmap);
  if (cudaGetLastError() != cudaSuccess) return KVQ_ERR_CUDA;
  const long long rows = (long long)a.n_q * v.n_rep - row0;
  const int rows_max = (int)(rows < 8 * NB ? rows : 8 * NB);
  const long long merged = pairs * rows_max;
  const int solo = merged >= kSoloRows, wide = merged <= num_sms();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(solo ? (merged + kSoloWarps - 1) / kSoloWarps : merged));
  cfg.blockDim = dim3((wide ? 16 : kSoloWarps) * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto merge = wide ? few_merge_kernel<D, kF32, 16> : few_merge_kernel<D, kF32, kSoloWarps>;
  return cudaLaunchKernelEx(&cfg, merge, v, a, row0, passes, sh, rows_max, solo, (const float*)ws) == cudaSuccess
             ? KVQ_OK
             : KVQ_ERR_CUDA;
}

// Rows in passes of 32 (16 at head_dim 256, or with fp32 output, whose second product doubles), up to kFewPasses of
// them in a launch, side by side, as blocks of the smallest size that holds them all; in a small call in passes of 8.
template <int F, int D, bool kF32>
kvq_status launch_few_rows(const KvqView& v, const QueryArgs& a, float* ws, const CUtensorMap& tmap, cudaStream_t st) {
  constexpr int kBlocks = D <= 128 && !kF32 ? 4 : 2;
  const long long rows = (long long)a.n_q * v.n_rep;
  if (few_small(v, v.batch, rows, (long long)v.max_pages * v.P))
    return launch_few_t<F, D, 1, kF32>(v, a, 0, (int)(rows + 7) / 8, ws, tmap, st);
  for (long long r = 0; r < rows; r += 8 * kBlocks * kFewPasses) {
    const int now = (int)(rows - r < 8 * kBlocks * kFewPasses ? rows - r : 8 * kBlocks * kFewPasses);
    const int passes = (now + 8 * kBlocks - 1) / (8 * kBlocks), nb = (now + 8 * passes - 1) / (8 * passes);
    const kvq_status s = nb == 1   ? launch_few_t<F, D, 1, kF32>(v, a, (int)r, passes, ws, tmap, st)
                         : nb == 2 ? launch_few_t<F, D, 2, kF32>(v, a, (int)r, passes, ws, tmap, st)
                         : nb == 3 ? launch_few_t<F, D, kBlocks == 4 ? 3 : 2, kF32>(v, a, (int)r, passes, ws, tmap, st)
                                   : launch_few_t<F, D, kBlocks, kF32>(v, a, (int)r, passes, ws, tmap, st);
    if (s != KVQ_OK) return s;
  }
  return KVQ_OK;
}

template <int F>
kvq_status launch_few_format(const KvqView& v, const QueryArgs& a, void* ws, cudaStream_t st) {
  CUtensorMap tmap;  // the pool as rows of 128 bytes, read in tiles of 16 tokens
  const cuuint64_t dims[2] = {128, (cuuint64_t)((long long)v.n_pages * v.page_bytes / 128)};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {128, (cuuint32_t)(kTile * v.D / 128)};
  const cuuint32_t estr[2] = {1, 1};
  if (tensor_map_encoder()(&tmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, v.pages, dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return KVQ_ERR_CUDA;
  float* w = static_cast<float*>(ws);
  if (a.out_f32) {
    if (v.D == 64) return launch_few_rows<F, 64, true>(v, a, w, tmap, st);
    if (v.D == 128) return launch_few_rows<F, 128, true>(v, a, w, tmap, st);
    return launch_few_rows<F, 256, true>(v, a, w, tmap, st);
  }
  if (v.D == 64) return launch_few_rows<F, 64, false>(v, a, w, tmap, st);
  if (v.D == 128) return launch_few_rows<F, 128, false>(v, a, w, tmap, st);
  return launch_few_rows<F, 256, false>(v, a, w, tmap, st);
}

}  // namespace
}  // namespace kvq
