// Attention of more than 32 rows (query token x query head) per kv-head over a PER_BLOCK
// cache: prompts and their chunks, longer drafts, cross attention; bf16 sources, head_dim
// 64 or 128.
//
// Mathematics, for a tile of 128 tokens whose 16-token pieces carry a key scale ks and a
// value scale vs: with code matrices C_k, C_v,
//   x = (q . C_k) (ks scale log2 e) + log2 vs,   p = 2^(x - M),
//   l += p / vs,   o += p C_v,   out = o / l,
// M a running maximum of x, raised when a tile exceeds it by 2^8.  The scales cost the
// softmax nothing (one multiply-add per element, as without them) and p stays an f16 number
// whatever they are.  Codes are exact in f16, and a bf16 query row is after scaling by a
// power of two; p is rounded to f16 once (2^-11 against the output's own 2^-8).
//
// What bounds it: the tensor cores and the softmax's exponentials for many rows, the codes'
// traffic for few.  One persistent CTA per SM of 23 warps, each with one task:
//   20     copies the tiles' codes into shared memory (bulk copies, a page each) and reads
//          the scales, two tiles ahead;
//   16-19  turn codes (and the window's bf16 rows) into f16 tiles with the 128-byte swizzle;
//   21, 22 issue the products of a stream each: S = Q K^T from shared memory, O += P V with
//          P in tensor memory;
//   0-7, 8-15  two streams of 128 rows: two threads own a row, half of its columns each,
//          read S from tensor memory, write P over it and rescale O.
// The two streams' products alternate, so that one runs while the other's softmax does.
// With more than 128 rows a unit is 256 rows, one half a stream, over the same tiles;
// with fewer the streams take every other tile of one half and are joined at the end.
//
// A 16-token piece of the window has one power of two for its keys and one for its values, as long as its tokens lie
// within 2^12 of one another.  Where they may not, a shared one would take bits from the smaller tokens, and so let a
// token change the outputs of queries that do not see it: each token then has its own, in a table of the workspace that
// the softmax reads.  It comes to know of it by an infinite scale, which sends the tile the way of a new maximum.
//
// Work split: units (sequence, kv-head, 256 or 128 rows) laid end to end as tiles; every CTA
// takes an equal run of them, whatever the lengths are, so that all SMs finish together.
// A unit cut by such a boundary leaves fp32 partial records, which a second kernel merges.
//
// Measured, 32 query heads on 8 kv-heads of 128: a causal prompt of 8,192 tokens takes 485 us, 1.1 PFLOP/s (58% of the
// measured matrix rate); 4 x 1,000 queries over 30,011 tokens 1.61 ms, 1.22 PFLOP/s (62%).  A tile of 256 rows and
// 128 tokens takes about 3,500 cycles, 2,048 of them products; the rest is handshakes that the two streams overlap only
// in part.  A unit's start and end take the time of 5 tiles, which bounds calls of short units: 16 x 448 queries on 16
// heads of 64 over up to 1,500 tokens take 84 us, 0.15 PFLOP/s.  (Two percent either way is where the code lies in the
// instruction caches: changes to parts that a call does not run move its time by as much.)
#include <math.h>

#include "kvq_code.cuh"
#include "kvq_query.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

using namespace ptx;

constexpr int kRows = 128;    // rows of a stream
constexpr int kTok = 128;     // tokens of a tile
constexpr int kPieces = kTok / 16;
constexpr int kSoftWarps = 16;           // 8 a stream: 4 warps reach the 128 rows, twice, for half the columns each
constexpr int kConv0 = kSoftWarps, kConvWarps = 4, kLoadWarp = kConv0 + kConvWarps, kMmaWarp = kLoadWarp + 1;
constexpr int kMThreads = (kMmaWarp + 2) * 32;
constexpr int kBarStream = 1, kBarJoin = 3;  // named barriers: of the streams (and the next), of both
constexpr int kSlots = 8;     // tiles whose scales are kept
constexpr int kFarSlots = 4;  // tiles whose tokens' exponents are kept (the converters are two ahead of the softmax at most)
constexpr int kFarSpan = 12;  // exponents that a piece's tokens may span with one power of two (2^-21 of a token's largest lost)
constexpr int kSegs = 8;      // segments that are told of
constexpr float kLazyM = 256.f;  // a piece's weights may sum to this before the maximum is raised
constexpr float kMinitM = -3e38f;  // below any logit
constexpr float kWideM = 1048576.f;  // x - M is one multiply-add, exact, where M is an x that was rounded: up to this, by 2^-4 at most

// A CTA's partial records: that of its first unit and that of its last, where they are cut.
struct RecHeader {
  int used;            // the record holds a cut unit's partial
  int b, h, qt;        // the unit
  int begins, ends;    // its first / last tile is in it
  int pad[2];
};

// Shared memory (D the head_dim): f16 tiles of Q (one per stream), K and V (two stages each), then the raw
// codes of one tile of keys and of values, then the small things.
template <int D>
struct Lay {
  static constexpr int kTileB = 128 * D * 2;
  static constexpr int kRawB = 128 * D;
  static constexpr int kQ = 0, kK = 2 * kTileB, kV = kK + 2 * kTileB, kRawK = kV + 2 * kTileB, kRawV = kRawK + kRawB;
  static constexpr int kMisc = kRawV + kRawB;
  // Raw stage: one with 256 rows, two with 128, whose second Q tile is free
  static __device__ __forceinline__ int raw_k(int stage) { return stage ? kQ + kTileB : kRawK; }
  static __device__ __forceinline__ int raw_v(int stage) { return stage ? kQ + kTileB + kRawB : kRawV; }
};

// A CTA's tiles of one unit, as the copying warp tells the others (who then need no plan of their own).
struct Seg {
  int b, h, qt;
  int T, nq, n, rows;  // of sequence b
  int j0, j1;          // tiles (none: the run is empty)
  int ends;            // j1 is the unit's last
  int i, r;            // the unit's first row: query and head in the group
  int last;            // nothing follows
  int pad[3];
};

struct Misc {
  // of each piece: key scale, log2 of the value scale (-inf: it has no tokens to see), 1 / value scale
  float4 scale[kSlots][kPieces];
  uint32_t skip_k[kSlots];      // pieces to fill with zeros; from bit 8: pieces whose tokens have exponents of their own
  uint32_t skip_v[kSlots];
  uint64_t raw_k_full[2], raw_v_full[2], raw_k_empty[2], raw_v_empty[2];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2], q_full[2], turn[2];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  Seg seg[kSegs];
  int bad_from[kSegs];          // of a segment: first token whose value is not finite, among those that some rows do not see
  float row_x[2][kRows];        // exchange between the two threads of a row
  uint32_t tmem;
  int abort;
};

// ---- units

struct Walk {  // one unit, and the CTA's place in it
  int b, h, qt;
  int T, n, rows, nqt;  // of sequence b
  int tiles;            // of the unit
};

// Out of line, like everything that a tile's loop does not run: the tasks' loops share the SM's instruction
// caches, and the kernel's inlined form (250 KB) missed them all the time.
static __device__ __noinline__ int unit_tiles(int causal, int n_rep, int T, int n, int rows, int qt, int RT) {
  const int last = min(rows, (qt + 1) * RT) - 1;
  const int end = causal ? max(0, T - n + last / n_rep + 1) : T;
  return max(1, (end + kTok - 1) / kTok);
}

static __device__ __noinline__ void load_sequence(const KvqView& v, const QueryArgs& a, int RT, Walk& w) {
  w.T = seq_tokens(v, w.b);
  w.n = query_count(v, a, w.b);
  w.rows = w.n * v.n_rep;
  w.nqt = (w.rows + RT - 1) / RT;
}

static __device__ __noinline__ void next_unit(const KvqView& v, const QueryArgs& a, int RT, Walk& w) {
  if (++w.qt == w.nqt) {
    w.qt = 0;
    if (++w.h == v.Hkv) {
      w.h = 0;
      do {
        ++w.b;
        load_sequence(v, a, RT, w);
      } while (w.nqt == 0);  // units remain, so a sequence with rows follows
    }
  }
  w.tiles = unit_tiles(a.causal, v.n_rep, w.T, w.n, w.rows, w.qt, RT);
}

// A tile on its way through the copying warp: this lane's share.
struct Pending {
  bool some;          // (whole warp) there is a tile
  bool good, scaled;  // this lane's page of codes is there; its piece's scales were read
  int t0, t1;         // the tile's tokens that come from pages
  int p0, p1;         // tokens of this lane's page in it
  int row0;           // the page's slot of token p0
  int gp, gslot;      // page of this lane's piece's scales, and their slot
  uint32_t missing;   // pieces whose page is missing
  long long page;     // byte of the page's head block
  long long head_off;
  float ks, vs;

  __device__ __forceinline__ void look_up(const KvqView& v, const Walk& w, int nq, int j, int lane) {
    const int32_t* bt = v.block_table + (long long)w.b * v.max_pages;
    t0 = j * kTok;
    t1 = min(t0 + kTok, nq);
    const int pg = t0 / v.P + lane;
    p0 = (int)max((long long)t0, min((long long)t1, (long long)pg * v.P));
    p1 = (int)min((long long)t1, ((long long)pg + 1) * v.P);
    row0 = (int)(p0 - (long long)pg * v.P);
    head_off = (long long)w.h * v.head_bytes;
    page = p0 < p1 ? bt[pg] : -1;  // the id, until read_scales
    gp = -1;
    gslot = 0;
    const int t = t0 + 16 * lane;
    if (lane < kPieces && t < t1) {
      const int g0 = t / v.kgroup * v.kgroup, q = g0 / v.P;
      gp = bt[q];
      gslot = (g0 - q * v.P) / v.kgroup;
    }
  }
  __device__ __forceinline__ void read_scales(const KvqView& v, int D, int lane) {
    const bool has = p0 < p1;
    good = has && page >= 0 && page < v.n_pages;
    missing = has && !good ? ((1u << ((p1 - t0) / 16)) - 1u) & ~((1u << ((p0 - t0) / 16)) - 1u) : 0u;
    missing = __reduce_or_sync(0xffffffffu, missing);
    page = (good ? page : 0) * v.page_bytes + head_off;
    scaled = gp >= 0 && gp < v.n_pages;
    ks = vs = 0.f;
    if (scaled) {
      const uint8_t* hb = v.pages + gp * v.page_bytes + head_off;
      ks = load_meta(hb + v.off_km, gslot, v.meta16);
      vs = load_meta(hb + v.off_vm, gslot, v.meta16);
    }
  }
};

__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {  // without an arrival
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// A CTA's run over the units.  A unit counts its tiles and kUnitCost more, for what its start and end cost
// (queries in, outputs out, and products and softmax without each other); these stand before its tiles.
constexpr int kUnitCost = 5;
struct Run {
  Walk w;
  unsigned long long left;  // of the run, from place p of unit w on
  int p;
  int j0, j1;               // the unit's tiles in the run (may be none)
  __device__ __forceinline__ void open() {
    const int n = (int)min((unsigned long long)(w.tiles + kUnitCost - p), left);
    j0 = max(0, p - kUnitCost);
    j1 = max(0, p + n - kUnitCost);
  }
  // To the next unit with tiles; false at the run's end.
  __device__ __noinline__ bool next(const KvqView& v, const QueryArgs& a, int RT) {
    do {
      const unsigned long long n = min((unsigned long long)(w.tiles + kUnitCost - p), left);
      left -= n;
      if (left == 0) return false;
      p = 0;
      next_unit(v, a, RT, w);
      open();
    } while (j0 == j1);
    return true;
  }
  // Whether no unit with tiles follows this one: a next one's first kUnitCost places have none.
  __device__ __forceinline__ bool last() const {
    return left - min((unsigned long long)(w.tiles + kUnitCost - p), left) <= kUnitCost;
  }
};

static __device__ __noinline__ unsigned long long divide(unsigned long long a, unsigned long long b) { return a / b; }

// This CTA's run (one warp; wb: a number per sequence in shared memory).  False: none.
static __device__ __noinline__ bool plan_run(const KvqView& v, const QueryArgs& a, int RT, unsigned long long* wb, Run& run) {
  const int lane = threadIdx.x & 31;
  auto sum64 = [](unsigned long long x) {
#pragma unroll 1
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  };
  unsigned long long total = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < v.batch; b0 += 32) {  // places of a kv-head of each sequence
    const int b = b0 + lane;
    const int T = b < v.batch ? seq_tokens(v, b) : 0, n = b < v.batch ? query_count(v, a, b) : 0, rows = n * v.n_rep;
    const int nqt = (rows + RT - 1) / RT;
    unsigned long long s = 0;
    if (__reduce_max_sync(0xffffffffu, nqt) <= 4) {
#pragma unroll 1
      for (int qt = 0; qt < nqt; ++qt) s += unit_tiles(a.causal, v.n_rep, T, n, rows, qt, RT) + kUnitCost;
    } else {  // long ones: the lanes over a sequence's units
#pragma unroll 1
      for (int k = 0; k < min(32, v.batch - b0); ++k) {
        const int Tk = __shfl_sync(0xffffffffu, T, k), nk = __shfl_sync(0xffffffffu, n, k);
        const int rk = __shfl_sync(0xffffffffu, rows, k), qk = __shfl_sync(0xffffffffu, nqt, k);
        unsigned long long x = 0;
#pragma unroll 1
        for (int qt = lane; qt < qk; qt += 32) x += unit_tiles(a.causal, v.n_rep, Tk, nk, rk, qt, RT) + kUnitCost;
        x = sum64(x);
        if (lane == k) s = x;
      }
    }
    if (b < v.batch) wb[b] = s;
    total += s;
  }
  __syncwarp();  // wb is read by other lanes than wrote it
  total = sum64(total) * v.Hkv;
  // no CTA between two others is left without a place: the merge walks from one to the next
  const unsigned long long runs = min((unsigned long long)gridDim.x, total), me = blockIdx.x;
  if (me >= runs) return false;
  const unsigned long long each = divide(total, runs), more = total - each * runs;  // `more` runs get one place more
  unsigned long long left = each * me + min(me, more);
  run.left = each + (me < more ? 1 : 0);
  Walk& w = run.w;
  w.b = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < v.batch; b0 += 32) {  // the sequence that holds the first place
    const unsigned long long x = b0 + lane < v.batch ? wb[b0 + lane] * v.Hkv : 0ull;
    unsigned long long incl = x;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, incl > left);
    if (hit) {
      const int k = __ffs(hit) - 1;
      w.b = b0 + k;
      left -= __shfl_sync(0xffffffffu, incl - x, k);
      break;
    }
    left -= __shfl_sync(0xffffffffu, incl, 31);
  }
  load_sequence(v, a, RT, w);
  w.h = (int)divide(left, wb[w.b]);
  left -= (unsigned long long)w.h * wb[w.b];
  w.qt = 0;
#pragma unroll 1
  for (int q0 = 0; q0 < w.nqt; q0 += 32) {
    const unsigned x = q0 + lane < w.nqt ? unit_tiles(a.causal, v.n_rep, w.T, w.n, w.rows, q0 + lane, RT) + kUnitCost : 0;
    unsigned incl = x;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, incl > left);
    if (hit) {
      const int k = __ffs(hit) - 1;
      w.qt = q0 + k;
      left -= __shfl_sync(0xffffffffu, incl - x, k);
      break;
    }
    left -= __shfl_sync(0xffffffffu, incl, 31);
  }
  w.tiles = unit_tiles(a.causal, v.n_rep, w.T, w.n, w.rows, w.qt, RT);
  run.p = (int)left;
  run.open();
  return run.j0 < run.j1 || run.next(v, a, RT);  // a run may lie in what stands before the tiles
}

// Bounded wait of a task; after a wait that gave up nothing more is waited for.
struct Waiter {
  Misc& m;
  int32_t* status;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
#pragma unroll 1
    for (uint32_t i = 0; i < kWaitPolls; ++i) {
      if (mbar_try_wait(bar, parity)) return true;
      if (*reinterpret_cast<volatile int*>(&m.abort)) return false;
    }
    *reinterpret_cast<volatile int*>(&m.abort) = 1;
    atomicOr(status, KVQ_DEV_TIMEOUT);
    return false;
  }
};

// Byte offset of 16-byte chunk c (of 8 f16) of row r in a tile of 128-row panels of 64 channels.
__device__ __forceinline__ uint32_t tile_chunk(int r, int c) {
  return (uint32_t)((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__host__ __device__ inline size_t many_rec_bytes(int D, int RT) { return (size_t)RT * (D + 4) * sizeof(float); }
// The workspace: the CTAs' record headers, their tables of exponents, their records.
__host__ __device__ inline size_t many_far_bytes() { return (size_t)kFarSlots * kTok * sizeof(int2); }  // of a CTA
__host__ __device__ inline size_t many_far_offset(int grid) { return ((size_t)grid * 2 * sizeof(RecHeader) + 255) / 256 * 256; }
__host__ __device__ inline size_t many_header_bytes(int grid) { return many_far_offset(grid) + (size_t)grid * many_far_bytes(); }
// Table of a tile's exponents.
__device__ __forceinline__ int2* far_table(unsigned char* ws, uint32_t it) {
  return reinterpret_cast<int2*>(ws + many_far_offset(gridDim.x) + blockIdx.x * many_far_bytes()) + it % kFarSlots * kTok;
}

// ---- converter: K pieces of 16 tokens of a raw tile, 4 pieces apart, -> f16 (whole warp).  A lane takes 8 codes
// of a row, one 16-byte chunk of the tile: eight lanes' loads and stores then meet no bank twice.
template <int F, int D, int K>
__device__ __forceinline__ void convert_n(const uint8_t* raw, uint8_t* dst, int piece, int lane) {
  constexpr int CPR = D / 8;          // chunks per row
  constexpr int RPI = 32 / CPR;       // rows per pass: 2 or 4
  constexpr int N = 16 / RPI;
  const int r0 = 16 * piece + lane / CPR, c = lane % CPR;
  const uint8_t* src = raw + r0 * D + 8 * c;
  uint2 x[K][N];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) x[k][i] = *reinterpret_cast<const uint2*>(src + (64 * k + i * RPI) * D);
  uint8_t* at[8 / RPI];  // rows 8 apart share their swizzle
#pragma unroll
  for (int i = 0; i < 8 / RPI; ++i) at[i] = dst + tile_chunk(r0 + i * RPI, c);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint32_t f[4];
      codes_to_f16<F>(x[k][i].x, f[0], f[1]);
      codes_to_f16<F>(x[k][i].y, f[2], f[3]);
      *reinterpret_cast<uint4*>(at[i % (8 / RPI)] + 64 * k * 128 + i / (8 / RPI) * 1024) = make_uint4(f[0], f[1], f[2], f[3]);
    }
}
template <int F, int D>
__device__ __noinline__ void convert_piece(const uint8_t* raw, uint8_t* dst, int piece, int lane) {
  convert_n<F, D, 1>(raw, dst, piece, lane);
}
// Both pieces of a warp, their loads in flight together.
template <int F, int D>
__device__ __forceinline__ void convert_pieces(const uint8_t* raw, uint8_t* dst, int piece, int lane) {
  static_assert(kPieces == 2 * kConvWarps && kConvWarps == 4, "two pieces a warp, 64 rows apart");
  convert_n<F, D, 2>(raw, dst, piece, lane);
}
template <int D>
__device__ __noinline__ void zero_piece(uint8_t* dst, int piece, int lane) {
#pragma unroll 1
  for (int i = lane; i < 16 * (D / 8); i += 32)
    *reinterpret_cast<uint4*>(dst + tile_chunk(16 * piece + i / (D / 8), i % (D / 8))) = make_uint4(0u, 0u, 0u, 0u);
}
// Window rows of a piece of 16 tokens from tok on, those before T (the last one in place of those behind, so that loads
// need no branch and are in flight together).  A lane has the same chunk of every RPI-th row.
template <int D>
struct WindowRows {
  static constexpr int CPR = D / 8, RPI = 32 / CPR, N = 16 / RPI;
  const uint16_t* src;
  long long pitch;
  int r0, n;
  __device__ __forceinline__ WindowRows(const void* win, const KvqView& v, int b, int h, int tok, int T, int nq, int lane)
      : pitch((long long)v.Hkv * D), r0(lane / CPR), n(T - tok) {
    src = static_cast<const uint16_t*>(win) + (((long long)b * v.R + (tok - nq)) * v.Hkv + h) * D + 8 * (lane % CPR);
  }
  __device__ __forceinline__ uint4 load(int i) const {
    return *reinterpret_cast<const uint4*>(src + min(r0 + i * RPI, n - 1) * pitch);
  }
  __device__ __forceinline__ bool has(int i) const { return r0 + i * RPI < n; }
};
// Loops over them are short code, with four loads in flight: what a unit's few window pieces wait for is instructions
// that no cache holds.

// Whether two of the rows lie further apart than one power of two serves (top: the largest magnitude).
template <int D>
__device__ __noinline__ bool rows_apart(const WindowRows<D> w, uint32_t top) {
  bool apart = false;
#pragma unroll 1
  for (int i = 0; i < w.N; ++i) {
    uint32_t m = chunk_top(w.load(i));
#pragma unroll
    for (int o = w.CPR / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    apart = apart || (m && value_exponent(m) < value_exponent(top) - kFarSpan);  // zeros go with any
  }
  return __any_sync(0xffffffffu, apart);
}
// The rows scaled by 2^-k with k their common exponent (zeros behind the last).  write == false: only the exponent.
// kFarBit is added to it where rows are too far apart for that.
constexpr int kFarBit = 1024;
template <int D>
__device__ __noinline__ int window_piece(const void* win, const KvqView& v, int b, int h, int tok, int T, int nq, uint8_t* dst,
                                            int piece, int lane, bool write) {
  const WindowRows<D> w(win, v, b, h, tok, T, nq, lane);
  uint32_t top = 0u, low = 0x7fff7fffu;
#pragma unroll 1
  for (int i = 0; i < w.N; i += 4) {
    uint4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = w.load(i + j);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t m = bf16x2_finite_max(bf16x2_finite_max(bf16x2_finite_max(bf16x2_finite_max(0u, x[j].x), x[j].y), x[j].z), x[j].w);
      top = bf16x2_absmax(top, m);
      low = bf16x2_min(low, m);  // of some of a row: no more than the row's largest
    }
  }
  top = finite_top(__reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16)));
  low = __reduce_min_sync(0xffffffffu, min(low & 0xffffu, low >> 16));
  const int k = value_exponent(top);
  if (write) {
    const float down = pow2i(-k);
#pragma unroll 1
    for (int i = 0; i < w.N; i += 4) {
      uint4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = w.load(i + j);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!w.has(i + j)) x[j] = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(dst + tile_chunk(16 * piece + w.r0 + (i + j) * w.RPI, lane % w.CPR)) =
            make_uint4(bf16x2_scaled(x[j].x, down), bf16x2_scaled(x[j].y, down), bf16x2_scaled(x[j].z, down),
                       bf16x2_scaled(x[j].w, down));
      }
    }
  }
  const bool near = low > 0x80u && value_exponent(low - 0x80u) >= k - kFarSpan;
  return k + (top && !near && rows_apart<D>(w, top) ? kFarBit : 0);
}
// The same with a power of two for each row, whose exponents go to exps, two ints apart.  Seldom called.
template <int D>
__device__ __noinline__ void far_piece(const void* win, const KvqView& v, int b, int h, int tok, int T, int nq, uint8_t* dst,
                                       int piece, int lane, bool write, int* exps) {
  const WindowRows<D> w(win, v, b, h, tok, T, nq, lane);
#pragma unroll 1
  for (int i = 0; i < w.N; ++i) {
    const int r = w.r0 + i * w.RPI, c = lane % w.CPR;
    const uint4 x = w.has(i) ? w.load(i) : make_uint4(0u, 0u, 0u, 0u);
    uint32_t top = chunk_top(x);
#pragma unroll
    for (int o = w.CPR / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int k = value_exponent(top);
    const float down = pow2i(-k);
    if (c == 0) exps[2 * r] = k;
    if (write)
      *reinterpret_cast<uint4*>(dst + tile_chunk(16 * piece + r, c)) =
          make_uint4(bf16x2_scaled(x.x, down), bf16x2_scaled(x.y, down), bf16x2_scaled(x.z, down), bf16x2_scaled(x.w, down));
  }
}

// Such a piece's keys, exponents and scale, and its values.
template <int D>
__device__ __noinline__ void far_keys(const KvqView& v, Misc& mi, const Seg& g, unsigned char* ws, uint32_t it, int tok, int piece,
                                      uint8_t* dst) {
  const int lane = threadIdx.x & 31, slot = it % kSlots;
  int* tab = reinterpret_cast<int*>(far_table(ws, it) + 16 * piece);
  far_piece<D>(v.k_win, v, g.b, g.h, tok, g.T, g.nq, dst, piece, lane, true, tab);
  far_piece<D>(v.v_win, v, g.b, g.h, tok, g.T, g.nq, dst, piece, lane, false, tab + 1);
  if (lane == 0) {
    atomicOr(&mi.skip_k[slot], 1u << (8 + piece));
    mi.scale[slot][piece] = make_float4(0.f, INFINITY, 0.f, 0.f);
  }
}
template <int D>
__device__ __noinline__ void far_values(const KvqView& v, const Seg& g, unsigned char* ws, uint32_t it, int tok, int piece, uint8_t* dst) {
  far_piece<D>(v.v_win, v, g.b, g.h, tok, g.T, g.nq, dst, piece, threadIdx.x & 31, true,
               reinterpret_cast<int*>(far_table(ws, it) + 16 * piece) + 1);
}

// A weight of zero would not keep a row from a value that is not finite.  So in tiles that some of the unit's rows do
// not see whole, such tokens' rows of a piece are zeroed, and the first noted: rows that see it get NaN for their sum.
template <int D>
__device__ __noinline__ void drop_not_finite(uint8_t* dst, int piece, int lane, int tok, int* bad_from) {
  constexpr int CPR = D / 8;
  __syncwarp();
  constexpr FiniteTest test = kFiniteF16x2;
  uint32_t carries = 0u;
#pragma unroll
  for (int r0 = 0; r0 < 16; r0 += 32 / CPR) {
    const uint4 x = *reinterpret_cast<const uint4*>(dst + tile_chunk(16 * piece + r0 + lane / CPR, lane % CPR));
    carries |= test.carry(x.x) | test.carry(x.y) | test.carry(x.z) | test.carry(x.w);
  }
  if (!__any_sync(0xffffffffu, test.fails(carries))) return;
#pragma unroll 1
  for (int r0 = 0; r0 < 16; r0 += 32 / CPR) {
    const int r = r0 + lane / CPR;
    uint4* at = reinterpret_cast<uint4*>(dst + tile_chunk(16 * piece + r, lane % CPR));
    const uint4 x = *at;
    const bool bad = test.fails(test.carry(x.x) | test.carry(x.y) | test.carry(x.z) | test.carry(x.w));
    const uint32_t mine = __ballot_sync(0xffffffffu, bad) >> (lane / CPR * CPR) & ((1u << CPR) - 1u);
    if (mine) {
      *at = make_uint4(0u, 0u, 0u, 0u);
      if (lane % CPR == 0) atomicMin(bad_from, tok + r);
    }
  }
}

// Place of a row in q and out: rows follow one another head by head within a query, then to the next query's
// heads of the same kv-head.
struct RowAt {
  long long e;
  int row, r;  // of the sequence and kv-head; its head in the group
  __device__ __forceinline__ void start(const KvqView& v, const QueryArgs& a, const Seg& g, int RT, int off, int D) {
    const int x = g.r + off, q = x / v.n_rep;
    row = g.qt * RT + off;
    r = x - q * v.n_rep;
    e = (((long long)g.b * a.n_q + g.i + q) * v.Hq + g.h * v.n_rep + r) * D;
  }
  __device__ __forceinline__ void step(const KvqView& v, int n, int D) {
    row += n;
    r += n;
    e += n * D;
#pragma unroll 1
    while (r >= v.n_rep) {
      r -= v.n_rep;
      e += (v.Hq - v.n_rep) * D;
    }
  }
};

// Arrive once per warp on a barrier that hands shared memory written here to the tensor cores.
__device__ __forceinline__ void hand_over(uint64_t* bar, int lane) {
  fence_proxy_async();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// ---- softmax of half a row: 64 of a tile's logits, from column tS; columns from lim on are masked.
// Loops are short: the tasks' code together has to stay in the instruction caches.

// Largest x.
template <bool kMasked>
__device__ __noinline__ float half_max(uint32_t tS, const float4* sc, float fct, int lim) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t r[32];
    tc::tmem_ld32(tS + 32 * c, r);
    tc::wait_ld(r);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (!kMasked || 32 * c + 16 * h + e < lim) m[e & 3] = fmaxf(m[e & 3], __uint_as_float(r[16 * h + e]));
      // an all-masked piece times a zero scale is NaN, which fmaxf passes over
      const float4 k = sc[2 * c + h];
      mx = fmaxf(mx, fmaf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), k.x * fct, k.y));
    }
  }
  return mx;
}

// Weights 2^(x - M) as f16 pairs in pk, to go over the first 32 of the columns they come from; returns the
// sum of weight / value scale, and in top the largest sum of a piece's weights (above 2^8 when M lags).
template <bool kMasked>
__device__ __forceinline__ float half_weights(uint32_t tS, const float4* sc, float fct, float M, int lim, uint32_t (&pk)[32],
                                              float& top) {
  float l = 0.f;
  top = 0.f;
  uint32_t r[2][16];
  tc::tmem_ld16(tS, r[0]);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    tc::wait_ld(r[c & 1]);
    if (c < 3) tc::tmem_ld16(tS + 16 * c + 16, r[(c + 1) & 1]);
    const float4 k = sc[c];
    const float cc = k.x * fct, bb = k.y - M;
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float2 x = fma2(make_float2(__uint_as_float(r[c & 1][2 * e]), __uint_as_float(r[c & 1][2 * e + 1])), make_float2(cc, cc),
                      make_float2(bb, bb));
      if (kMasked) {
        if (16 * c + 2 * e >= lim) x.x = -INFINITY;
        if (16 * c + 2 * e + 1 >= lim) x.y = -INFINITY;
      }
      const float2 p = make_float2(ex2(x.x), ex2(x.y));
      sum = add2(sum, p);
      pk[8 * c + e] = pack_f16x2(p.x, p.y);
    }
    const float piece = sum.x + sum.y;
    top = fmaxf(top, piece);
    l = fmaf(piece, k.z, l);
  }
  return l;
}

// The same two steps for a tile with pieces (the bits of far) whose tokens have exponents of their own, in tab (of the
// keys, of the values), or with logits whose rounding is not small: the largest x, which takes the place of the logits, and then the weights, written over the first
// 32 of the columns they come from; returns the sum of weight / value scale.  Seldom called.
static __device__ __noinline__ float far_max(uint32_t tS, const Misc& mi, unsigned char* ws, uint32_t it, float fct, int lim) {
  const int hf = (threadIdx.x >> 7) & 1, slot = it % kSlots;
  const float4* sc = mi.scale[slot] + 4 * hf;
  const int2* tab = far_table(ws, it) + 64 * hf;
  const uint32_t far = mi.skip_k[slot] >> (8 + 4 * hf);
  float mx = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[16];
    tc::tmem_ld16(tS + 16 * c, r);
    tc::wait_ld(r);
    const float4 k = sc[c];
    const bool own = (far >> c) & 1u;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int2 t = own ? tab[16 * c + e] : make_int2(0, 0);
      const float kx = (own ? pow2i(t.x) : k.x) * fct, ky = own ? (float)t.y : k.y;
      const float x = 16 * c + e < lim ? fmaf(__uint_as_float(r[e]), kx, ky) : -INFINITY;
      mx = fmaxf(mx, x);
      r[e] = __float_as_uint(x);
    }
    tc::tmem_st16(tS + 16 * c, r);
  }
  tc::wait_st();
  return mx;
}
static __device__ __noinline__ float far_weights(uint32_t tS, const Misc& mi, unsigned char* ws, uint32_t it, float M) {
  const int hf = (threadIdx.x >> 7) & 1, slot = it % kSlots;
  const float4* sc = mi.scale[slot] + 4 * hf;
  const int2* tab = far_table(ws, it) + 64 * hf;
  const uint32_t far = mi.skip_k[slot] >> (8 + 4 * hf);
  float l = 0.f;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[16], pk[8];
    tc::tmem_ld16(tS + 16 * c, r);
    tc::wait_ld(r);
    const float z = sc[c].z;
    const bool own = (far >> c) & 1u;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float p = ex2(__uint_as_float(r[e]) - M);
      l = fmaf(p, own ? pow2i(-tab[16 * c + e].y) : z, l);
      r[e] = __float_as_uint(p);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) pk[e] = pack_f16x2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
    tc::tmem_st8(tS + 8 * c, pk);
  }
  tc::wait_st();
  return l;
}

// Barrier of kThreads threads that also says whether any of them asks.
template <int kThreads>
__device__ __forceinline__ bool any_of(int bar, bool ask) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.or.pred q, %1, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(bar), "r"((uint32_t)ask), "n"(kThreads)
      : "memory");
  return r != 0;
}

template <int F, int D>
__global__ void __launch_bounds__(kMThreads, 1) query_many_kernel(KvqView v, QueryArgs a, unsigned char* ws, int RT) {
  using L = Lay<D>;
  extern __shared__ __align__(1024) unsigned char sm[];  // the swizzle's atoms
  Misc& mi = *reinterpret_cast<Misc*>(sm + L::kMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool two = RT == 2 * kRows;  // a stream per half of the unit; else both over one half
  grid_dep_launch();

  RecHeader* hdr = reinterpret_cast<RecHeader*>(ws) + 2 * blockIdx.x;
  if (threadIdx.x < 2) hdr[threadIdx.x].used = 0;
  if (threadIdx.x == 0) mi.abort = 0;
  Run run;
  bool some = false;
  if (warp == kLoadWarp) some = plan_run(v, a, RT, reinterpret_cast<unsigned long long*>(sm), run);
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&mi.tmem, 512);
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&mi.raw_k_full[i], 1);
        mbar_init(&mi.raw_v_full[i], 1);
        mbar_init(&mi.raw_k_empty[i], kConvWarps);
        mbar_init(&mi.raw_v_empty[i], kConvWarps);
        mbar_init(&mi.k_full[i], kConvWarps);
        mbar_init(&mi.k_empty[i], two ? 2 : 1);  // each stream that multiplies by the tile
        mbar_init(&mi.v_full[i], kConvWarps);
        mbar_init(&mi.v_empty[i], two ? 2 : 1);
        mbar_init(&mi.s_full[i], 1);
        mbar_init(&mi.turn[i], 1);
        mbar_init(&mi.p_full[i], 8);
        mbar_init(&mi.o_full[i], 1);
        mbar_init(&mi.q_full[i], 8);
      }
      for (int i = 0; i < kSegs; ++i) {
        mbar_init(&mi.seg_full[i], 1);
        mbar_init(&mi.seg_empty[i], kSoftWarps + kConvWarps + 2);
      }
      fence_mbar_init();
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = mi.tmem;
  const Waiter wait{mi, v.status};

  // The next segment (every warp but the copying one), read whole.  Its place is given back when the warp reads and
  // writes it no more: the softmax warps read bad_from at the segment's end.
  uint32_t nseg = 0;
  auto segment = [&](Seg& g) -> bool {
    const uint32_t k = nseg % kSegs;
    const bool ok = wait(&mi.seg_full[k], (nseg / kSegs) & 1);
    g = mi.seg[k];
    ++nseg;
    return __all_sync(0xffffffffu, ok);
  };
  auto leave_segment = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&mi.seg_empty[(nseg - 1) % kSegs]);
  };

  if (warp == kLoadWarp) {
    // Tiles pass through three steps, one tile apart, so that no load's latency is waited for: page ids
    // (lane i: the tile's i-th page, and the page of piece i's scales), then scales, then the copies.
    Pending p2, p1, p0;
    p1.some = p0.some = false;
    const Walk& w = run.w;
    bool ok = true;
    uint32_t it = 0;  // tiles copied
    int nq = 0, j = 0;
    auto tell = [&]() {
      const uint32_t k = nseg % kSegs;
      ok = ok && __all_sync(0xffffffffu, wait(&mi.seg_empty[k], ((nseg / kSegs) & 1) ^ 1));
      ++nseg;
      nq = n_quantized(w.T, v.R);
      j = run.j0;
      if (lane == 0) {
        const int i = w.qt * RT / v.n_rep;
        mi.bad_from[k] = 0x7fffffff;
        mi.seg[k] = Seg{w.b, w.h, w.qt, w.T, nq, w.n, w.rows, run.j0, run.j1, run.j1 == w.tiles,
                        i, w.qt * RT - i * v.n_rep, run.last(), {0, 0, 0}};
        mbar_arrive(&mi.seg_full[k]);
      }
      __syncwarp();
    };
    if (some) {
      tell();
    } else if (lane == 0) {
      mi.seg[0] = Seg{};
      mi.seg[0].last = 1;
      mbar_arrive(&mi.seg_full[0]);
    }
    bool todo = some;  // tiles not yet looked up: j of the run's unit
    for (;;) {
      p2.some = todo;
      if (todo) {
        p2.look_up(v, w, nq, j, lane);
        if (++j == run.j1) {
          todo = run.next(v, a, RT);
          if (todo) tell();
          if (!ok) break;
        }
      }
      if (p1.some) p1.read_scales(v, D, lane);
      if (p0.some) {
        const int slot = it % kSlots, rs = two ? 0 : it & 1;  // raw stage and its phase
        const uint32_t rp = two ? it & 1 : (it >> 1) & 1;
        const uint32_t bytes = p0.good ? (uint32_t)(p0.p1 - p0.p0) * D : 0u;
        const uint32_t sum = __reduce_add_sync(0xffffffffu, bytes);
        const uint8_t* src = v.pages + p0.page + (long long)p0.row0 * D;
        ok = __all_sync(0xffffffffu, wait(&mi.raw_k_empty[rs], rp ^ 1));
        if (!ok) break;
        if (lane == 0 && sum) mbar_expect_tx(&mi.raw_k_full[rs], sum);
        __syncwarp();
        if (bytes) bulk_g2s(sm + L::raw_k(rs) + (p0.p0 - p0.t0) * D, src, bytes, &mi.raw_k_full[rs]);
        float4 sc = make_float4(0.f, -INFINITY, 0.f, 0.f);
        bool drop_v = false;
        uint32_t bad = p0.missing;
        if (lane < kPieces && p0.t0 + 16 * lane < p0.t1) {
          if (p0.scaled && !((bad >> lane) & 1u)) {
            drop_v = p0.vs < pow2i(kMinExp);  // values below 2^-91: read as 0
            // (the third is finite for a scale of NaN too: rows that do not see the piece multiply it by 0)
            sc = make_float4(p0.ks, drop_v ? (float)kZeroExp : __log2f(p0.vs), drop_v ? pow2i(-kZeroExp) : p0.vs > 0.f ? __frcp_rn(p0.vs) : 0.f, 0.f);
          } else {
            bad |= 1u << lane;
          }
        }
        bad = __reduce_or_sync(0xffffffffu, bad);
        const uint32_t dv = __ballot_sync(0xffffffffu, drop_v);
        if (lane < kPieces) mi.scale[slot][lane] = sc;
        if (lane == 0) {
          mi.skip_k[slot] = bad;
          mi.skip_v[slot] = bad | dv;
          if (bad) atomicOr(v.status, KVQ_DEV_BAD_PAGE);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&mi.raw_k_full[rs]);
        ok = __all_sync(0xffffffffu, wait(&mi.raw_v_empty[rs], rp ^ 1));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&mi.raw_v_full[rs], sum);
        __syncwarp();
        if (bytes) bulk_g2s(sm + L::raw_v(rs) + (p0.p0 - p0.t0) * D, src + v.off_vc, bytes, &mi.raw_v_full[rs]);
        ++it;
      } else if (!p1.some && !p2.some) {
        break;
      }
      p0 = p1;
      p1 = p2;
    }
  } else if (warp >= kConv0 && warp < kConv0 + kConvWarps) {
    uint32_t it = 0;
    bool ok = true;
    Seg w;
    do {
      if (!(ok = segment(w))) break;
      for (int j = w.j0; j < w.j1; ++j, ++it) {
        const int t0 = j * kTok, slot = it % kSlots, st = it & 1;
        const uint32_t ph = (it >> 1) & 1, rp = two ? it & 1 : ph;
        const int rs = two ? 0 : st;
        uint8_t* kd = sm + L::kK + st * L::kTileB;
        uint8_t* vd = sm + L::kV + st * L::kTileB;
        ok = __all_sync(0xffffffffu, wait(&mi.raw_k_full[rs], rp) && wait(&mi.k_empty[st], ph ^ 1));
        if (!ok) break;  // the warp as one: what follows has barriers of the warp
        const uint32_t skip_k = mi.skip_k[slot], skip_v = mi.skip_v[slot];
        const bool plain = t0 + kTok <= w.nq;  // every piece is a page's
        if (plain && skip_k == 0) {
          convert_pieces<F, D>(sm + L::raw_k(rs), kd, warp - kConv0, lane);
        } else
#pragma unroll 1
        for (int i = 0; i < kPieces / kConvWarps; ++i) {
          const int piece = (warp - kConv0) + i * kConvWarps, tok = t0 + 16 * piece;
          if (tok >= w.T || ((skip_k >> piece) & 1u)) {
            zero_piece<D>(kd, piece, lane);
          } else if (tok < w.nq) {
            convert_piece<F, D>(sm + L::raw_k(rs), kd, piece, lane);
          } else {
            const int kk = window_piece<D>(v.k_win, v, w.b, w.h, tok, w.T, w.nq, kd, piece, lane, true);
            const int kv = window_piece<D>(v.v_win, v, w.b, w.h, tok, w.T, w.nq, vd, piece, lane, false);
            if (max(kk, kv) >= kFarBit / 2) {
              far_keys<D>(v, mi, mi.seg[(nseg - 1) % kSegs], ws, it, tok, piece, kd);
            } else if (lane == 0) {
              mi.scale[slot][piece] = make_float4(pow2i(kk), (float)kv, pow2i(-kv), 0.f);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&mi.raw_k_empty[rs]);
        hand_over(&mi.k_full[st], lane);
        ok = __all_sync(0xffffffffu, wait(&mi.raw_v_full[rs], rp) && wait(&mi.v_empty[st], ph ^ 1));
        if (!ok) break;
        const bool whole = t0 + kTok <= query_end(a, w.T, w.n, w.i);  // every row of the unit sees the tile
        if (plain && skip_v == 0) {
          convert_pieces<F, D>(sm + L::raw_v(rs), vd, warp - kConv0, lane);
        } else
#pragma unroll 1
        for (int i = 0; i < kPieces / kConvWarps; ++i) {
          const int piece = (warp - kConv0) + i * kConvWarps, tok = t0 + 16 * piece;
          if (tok >= w.T || (tok < w.nq && ((skip_v >> piece) & 1u))) {
            zero_piece<D>(vd, piece, lane);
          } else if (tok < w.nq) {
            convert_piece<F, D>(sm + L::raw_v(rs), vd, piece, lane);
          } else if ((mi.skip_k[slot] >> (8 + piece)) & 1u) {
            far_values<D>(v, mi.seg[(nseg - 1) % kSegs], ws, it, tok, piece, vd);
          } else {
            window_piece<D>(v.v_win, v, w.b, w.h, tok, w.T, w.nq, vd, piece, lane, true);
          }
        }
        if (!whole && !(plain && F == kI8)) {
#pragma unroll 1
          for (int piece = warp - kConv0; piece < kPieces; piece += kConvWarps)
            drop_not_finite<D>(vd, piece, lane, t0 + 16 * piece, &mi.bad_from[(nseg - 1) % kSegs]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&mi.raw_v_empty[rs]);
        hand_over(&mi.v_full[st], lane);
      }
      leave_segment();
    } while (ok && !w.last);
  } else if (warp >= kMmaWarp) {
    // A warp a stream, so that one's waits do not hold up the other's products (issuing blocks until the
    // products before are nearly done).  The whole warp walks the steps with values it knows to be uniform,
    // and one elected lane issues: the descriptors then stay in uniform registers (issued from a divergent
    // lane, a product cost 160 cycles).
    constexpr uint32_t id_s = tc::f16_idesc(128, 128, false), id_o = tc::f16_idesc(128, D, true);
    constexpr uint32_t kPanel = 128 * 128;
    const int s = __shfl_sync(0xffffffffu, warp - kMmaWarp, 0), by = two ? 1 : 2;
    const uint64_t dq = tc::smem_desc(smem_u32(sm + L::kQ + (two ? s : 0) * L::kTileB), 16);
    const uint64_t dk = tc::smem_desc(smem_u32(sm + L::kK), 16), dv = tc::smem_desc(smem_u32(sm + L::kV), kPanel);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0) + 128 * s;
    const uint32_t to = __shfl_sync(0xffffffffu, tmem, 0) + 256 + D * s;
    const bool elected = tc::elect_one();
    uint32_t it0 = 0, np = 0, turns = 0;  // tiles before this segment; phases of the weights; turns
    bool ok = true;
    Seg w;
    do {
      if (!segment(w) || w.j0 == w.j1) break;
      leave_segment();
      const int nt = __shfl_sync(0xffffffffu, w.j1 - w.j0, 0);
      const int i0 = two ? 0 : s;  // the stream's tiles: i0, i0 + by, ...
      ok = __all_sync(0xffffffffu, wait(&mi.q_full[two ? s : 0], (nseg - 1) & 1));
      // step i: P V of tile i (not at first), then S of tile i + by, which takes P's place
#pragma unroll 1
      for (int i = i0 - by; i < nt && ok; i += by) {
        const uint32_t it = it0 + i, nx = it + by;
        const bool now = i >= i0, more = i + by < nt;
        const uint64_t b = dv + (it & 1) * (L::kTileB >> 4), k = dk + (nx & 1) * (L::kTileB >> 4);
        // what is ready early is waited for first, the weights last
        if (more) ok = wait(&mi.k_full[nx & 1], (nx >> 1) & 1);
        if (now) ok = ok && wait(&mi.v_full[it & 1], (it >> 1) & 1);
        // The streams issue in turn (256 rows): one's softmax then runs beside the other's products.  Left to
        // themselves they fall into step, and products and softmax alternate (4100 cycles a tile, not 3300).
        if (two) ok = ok && wait(&mi.turn[s], (turns++ & 1) ^ (s ^ 1));
        ok = __all_sync(0xffffffffu, ok);
        if (now) ok = ok && wait(&mi.p_full[s], np++ & 1);
        tc::fence_after();
        if (elected && ok) {
          if (now) {
#pragma unroll
            for (int x = 0; x < kTok / 16; ++x)
              tc::mma_ts(to, tm + 8 * x + (x < 4 ? 0 : 32), b + x * (2048 >> 4), id_o, i > i0 || x > 0);
            tc::commit(&mi.v_empty[it & 1]);
          }
          if (more) {
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
              const uint32_t off = ((x >> 2) * kPanel + (x & 3) * 32) >> 4;
              tc::mma_ss(tm, dq + off, k + off, id_s, x > 0);
            }
            tc::commit(&mi.s_full[s]);
            tc::commit(&mi.k_empty[nx & 1]);
          } else if (now) {
            tc::commit(&mi.o_full[s]);
          }
          if (two) mbar_arrive(&mi.turn[s ^ 1]);
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      it0 += nt;
    } while (ok && !w.last);
  } else {  // ---- softmax streams: warp = 8 stream + 4 half + quarter of the rows
    const int s = __shfl_sync(0xffffffffu, warp >> 3, 0), hf = (warp >> 2) & 1, row_l = threadIdx.x & (kRows - 1);
    const uint32_t lane_off = (uint32_t)(warp & 3) << 21;  // 32 lanes a warp, in the address's upper half
    constexpr int kOutC = D / 2;                           // channels of this thread's output
    const uint32_t tS = tmem + lane_off + 128 * s + 64 * hf, tO = tmem + lane_off + 256 + D * s + kOutC * hf;
    float* rx = &mi.row_x[s][row_l];
    uint32_t ns = 0, it0 = 0, no = 0;
    bool ok = true;
    // Query rows come, and outputs leave, 16 rows a warp with the lanes along them.
    constexpr int CPR = D / 8, RPP = 32 / CPR, NP = 16 / RPP;  // chunks a row, rows a pass, passes
    const int r0 = (warp & 7) * 16 + lane / CPR, c8 = lane % CPR;
    uint8_t* const qd = sm + L::kQ + (two ? s : 0) * L::kTileB;
    Seg w;
    do {
      // (threads that share barriers give up together: with 128 rows both streams, which are joined at the end)
      ok = segment(w);
      if ((two ? any_of<2 * kRows>(kBarStream + s, !ok) : any_of<4 * kRows>(kBarJoin, !ok)) || w.j0 == w.j1) break;
      const int j0 = w.j0, nt = w.j1 - w.j0;
      const int off = two ? s * kRows : 0;                     // the stream's first row in the unit
      const bool live = w.qt * RT + off + row_l < w.rows;
      const int qi = w.i + (w.r + off + row_l) / v.n_rep;
      // ---- the stream's query rows into f16, K-major; rows past the last are zeros.  Each row's power of two goes
      // to its threads.
      RowAt at;  // row r0
      at.start(v, a, w, RT, off + r0, D);
      {
        RowAt k = at;
        if (it0 > 0) named_bar_sync(kBarStream + s, 2 * kRows);  // the last segment's rows have left the tile
#pragma unroll 1
        for (int i0 = 0; i0 < NP; i0 += 4) {
          uint4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (k.row < w.rows) x[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + k.e + 8 * c8);
            k.step(v, RPP, D);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t m2 = bf16x2_absmax(bf16x2_absmax(bf16x2_absmax(bf16x2_absmax(0u, x[i].x), x[i].y), x[i].z), x[i].w);
            uint32_t top = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
            for (int o = CPR / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            float down, up;
            norm_factors(top, down, up);
            const int r = r0 + (i0 + i) * RPP;
            if (c8 == 0) mi.row_x[s][r] = up;
            if (two || s == 0)
              *reinterpret_cast<uint4*>(qd + tile_chunk(r, c8)) =
                  make_uint4(bf16x2_scaled(x[i].x, down), bf16x2_scaled(x[i].y, down), bf16x2_scaled(x[i].z, down),
                             bf16x2_scaled(x[i].w, down));
          }
        }
        if (two || s == 0) hand_over(&mi.q_full[s], lane);
        named_bar_sync(kBarStream + s, 2 * kRows);
      }
      const float fct = *rx * a.scale * 1.4426950408889634f;
      const int end = live ? query_end(a, w.T, w.n, qi) : 0x3FFFFFFF;  // rows past the last: never masked, never written
      const int warp_end = __reduce_min_sync(0xffffffffu, end);
      float M = kMinitM, l = 0.f;
      bool any = false;  // this stream has had a tile of this segment
      bool wide = false;  // its maxima are too large for that: every tile then goes the way of far ones
      for (int i = two ? 0 : s; i < nt; i += two ? 1 : 2) {
        const int t0 = (j0 + i) * kTok + 64 * hf, slot = (it0 + i) % kSlots;
        ok = wait(&mi.s_full[s], ns & 1);
        ++ns;
        tc::fence_after();
        const float4* sc = mi.scale[slot] + 4 * hf;
        const int lim = end - t0;
        const bool masked = t0 + 64 > warp_end;
        // With the standing maximum first: it holds for nearly every tile.  The weights stay in registers
        // until both halves of every row have agreed to it.
        uint32_t pk[32];
        float top = INFINITY, sum = 0.f;  // nothing stands before the first tile
        if (any) sum = masked ? half_weights<true>(tS, sc, fct, M, lim, pk, top) : half_weights<false>(tS, sc, fct, M, lim, pk, top);
        // (a stream whose wait gave up stops as one: the barrier carries that too)
        if (any_of<2 * kRows>(kBarStream + s, top > kLazyM || wide || !ok)) {
          if (any_of<2 * kRows>(kBarStream + s, !ok)) {
            ok = false;
            break;
          }
          const uint32_t far = mi.skip_k[slot] >> 8;  // the same for the whole stream
          const float mx = far ? far_max(tS, mi, ws, it0 + i, fct, lim)
                           : masked ? half_max<true>(tS, sc, fct, lim) : half_max<false>(tS, sc, fct, lim);
          if (hf) *rx = mx;
          named_bar_sync(kBarStream + s, 2 * kRows);
          float mn = M;
          if (!hf) {
            mn = fmaxf(M, fmaxf(mx, *rx));
            *rx = mn;
          }
          wide = any_of<2 * kRows>(kBarStream + s, !hf && fabsf(mn) > kWideM && mn > kMinitM);
          if (hf) mn = *rx;
          const float al = ex2(M - mn);
          M = mn;
          l *= al;
          if (any) {
#pragma unroll 1
            for (int c = 0; c < kOutC; c += 16) {
              uint32_t r[16];
              tc::tmem_ld16(tO + c, r);
              tc::wait_ld(r);
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * al);
              tc::tmem_st16(tO + c, r);
            }
          }
          if (wide && !far) far_max(tS, mi, ws, it0 + i, fct, lim);
          if (far || wide) {
            sum = far_weights(tS, mi, ws, it0 + i, M);
            tc::tmem_ld32(tS, pk);
            tc::wait_ld(pk);
          } else {
            sum = masked ? half_weights<true>(tS, sc, fct, M, lim, pk, top) : half_weights<false>(tS, sc, fct, M, lim, pk, top);
          }
        }
        any = true;
        l += sum;
        tc::tmem_st32(tS, pk);
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&mi.p_full[s]);
      }
      // ---- the segment's output
      if (ok && any) {
        ok = wait(&mi.o_full[s], no & 1);
        ++no;
        tc::fence_after();
      }
      ok = !any_of<2 * kRows>(kBarStream + s, !ok);
      if (hf) *rx = l;
      named_bar_sync(kBarStream + s, 2 * kRows);
      if (!hf) {
        l += *rx;
        *rx = l;
      }
      named_bar_sync(kBarStream + s, 2 * kRows);
      if (hf) l = *rx;
      if (!two) {
        // stream 1's (M, l, O) to stream 0, O through the Q tile (its products are done), 16 channels a thread at
        // a time
        float* ex = reinterpret_cast<float*>(sm + L::kQ) + hf * (16 * kRows);
        float* ml = mi.row_x[0];
        ok = !any_of<4 * kRows>(kBarJoin, !ok);  // both streams' sums have been read
        if (s == 1 && !hf) {
          ml[row_l] = any ? M : kMinitM;
          ml[kRows + row_l] = any ? l : 0.f;
        }
        named_bar_sync(kBarJoin, 4 * kRows);
        float a0 = 1.f, a1 = 0.f;
        if (s == 0) {
          const float M1 = ml[row_l], l1 = ml[kRows + row_l], mn = fmaxf(M, M1);
          a0 = ex2(M - mn);
          a1 = ex2(M1 - mn);
          M = mn;
          l = l * a0 + l1 * a1;
        }
        if (nt > 1) {
#pragma unroll 1
          for (int c = 0; c < kOutC; c += 16) {
            uint32_t r[16];
            tc::tmem_ld16(tO + c, r);
            tc::wait_ld(r);
            if (s == 1) {
#pragma unroll
              for (int e = 0; e < 16; ++e) ex[e * kRows + row_l] = __uint_as_float(r[e]);
            }
            named_bar_sync(kBarJoin, 4 * kRows);
            if (s == 0) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                r[e] = __float_as_uint(__uint_as_float(r[e]) * a0 + ex[e * kRows + row_l] * a1);
              tc::tmem_st16(tO + c, r);
              tc::wait_st();
            }
            named_bar_sync(kBarJoin, 4 * kRows);
          }
        } else {
          named_bar_sync(kBarJoin, 4 * kRows);  // stream 0 has read the statistics
        }
      }
      const bool begins = j0 == 0, ends = w.ends;
      if (ok && (two || s == 0)) {
        const bool first = it0 == 0;
        const bool whole = begins && ends;
        if (end > mi.bad_from[(nseg - 1) % kSegs]) l = __int_as_float(0x7fffffff);
        const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN stays
        const int rs = (two ? s * kRows : 0) + row_l;
        float* rec = reinterpret_cast<float*>(ws + many_header_bytes(gridDim.x) +
                                              (2ull * blockIdx.x + (first ? 0 : 1)) * many_rec_bytes(D, RT)) +
                     (long long)rs * (D + 4);
        if (!whole) {
          if (threadIdx.x == 0) hdr[first ? 0 : 1] = RecHeader{1, w.b, w.h, w.qt, begins, ends, {0, 0}};
          if (live && !hf) *reinterpret_cast<float4*>(rec) = make_float4(M, l, 0.f, 0.f);
        }
        // a whole unit's rows leave through the Q tile (its products are done), lanes along the rows
#pragma unroll 1
        for (int c = 0; c < kOutC; c += 16) {
          uint32_t r[16];
          __syncwarp();
          tc::tmem_ld16(tO + c, r);
          tc::wait_ld(r);
          if (whole) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t y[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 z = __floats2bfloat162_rn(__uint_as_float(r[8 * e + 2 * k]) * inv,
                                                               __uint_as_float(r[8 * e + 2 * k + 1]) * inv);
                y[k] = *reinterpret_cast<const uint32_t*>(&z);
              }
              *reinterpret_cast<uint4*>(qd + tile_chunk(row_l, (kOutC * hf + c) / 8 + e)) = make_uint4(y[0], y[1], y[2], y[3]);
            }
          } else if (live) {
            uint4* op = reinterpret_cast<uint4*>(rec + 4 + kOutC * hf + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) op[e] = make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
          }
        }
        if (whole) {
          named_bar_sync(kBarStream + s, 2 * kRows);
#pragma unroll 1
          for (int i = 0; i < NP; ++i) {
            if (at.row < w.rows)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at.e + 8 * c8) =
                  *reinterpret_cast<const uint4*>(qd + tile_chunk(r0 + i * RPP, c8));
            at.step(v, RPP, D);
          }
        }
      }
      tc::fence_before();
      leave_segment();
      it0 += nt;
    } while (ok && !w.last);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (mi.abort) {  // a wait gave up: copies and products in flight end (microseconds) before the memory is released
#pragma unroll 1
    for (int i = 0; i < 4096; ++i) __nanosleep(250);
    __syncthreads();
  }
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// Merge of the cut units: the blocks of CTA x take the unit whose first tile is in a record of x and whose
// last is not, a warp a row; its records are x's and the first ones of the CTAs that follow.
constexpr int kMergeRows = 16;
template <int D>
__global__ void __launch_bounds__(kMergeRows * 32) many_merge_kernel(KvqView v, QueryArgs a, const unsigned char* ws, int RT, int grid) {
  constexpr int PER = D / 32;
  const int per = RT / kMergeRows, x = blockIdx.x / per, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rs = blockIdx.x % per * kMergeRows + warp;
  grid_dep_wait();
  const RecHeader* hdr = reinterpret_cast<const RecHeader*>(ws);
  int at = -1;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const RecHeader& r = hdr[2 * x + k];
    if (r.used && r.begins && !r.ends) at = 2 * x + k;
  }
  if (at < 0) return;
  const RecHeader u = hdr[at];
  const int row = u.qt * RT + rs;
  if (row >= query_count(v, a, u.b) * v.n_rep) return;
  float m = kMinitM, l = 0.f, o[PER];
#pragma unroll
  for (int c = 0; c < PER; ++c) o[c] = 0.f;
  for (int k = at;;) {
    const float* rec =
        reinterpret_cast<const float*>(ws + many_header_bytes(grid) + (unsigned long long)k * many_rec_bytes(D, RT)) + (long long)rs * (D + 4);
    const float2 ml = *reinterpret_cast<const float2*>(rec);
    float y[PER];
#pragma unroll
    for (int c = 0; c < PER; c += 2) {
      const float2 z = *reinterpret_cast<const float2*>(rec + 4 + lane * PER + c);
      y[c] = z.x;
      y[c + 1] = z.y;
    }
    const float mn = fmaxf(m, ml.x), a0 = exp2f(m - mn), a1 = exp2f(ml.x - mn);
    m = mn;
    l = l * a0 + ml.y * a1;
#pragma unroll
    for (int c = 0; c < PER; ++c) o[c] = o[c] * a0 + y[c] * a1;
    if (hdr[k].ends) break;
    k = (k / 2 + 1) * 2;  // the next CTA's first record
    if (k >= 2 * grid || !hdr[k].used) break;  // a run that gave up
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const long long e = (((long long)u.b * a.n_q + row / v.n_rep) * v.Hq + u.h * v.n_rep + row % v.n_rep) * D + lane * PER;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + e);
#pragma unroll
  for (int c = 0; c < PER; c += 2) {
    const __nv_bfloat162 z = __floats2bfloat162_rn(o[c] * inv, o[c + 1] * inv);
    out[c / 2] = *reinterpret_cast<const uint32_t*>(&z);
  }
}

template <int F, int D>
kvq_status launch_many_t(const KvqView& v, const QueryArgs& a, unsigned char* ws, cudaStream_t st) {
  const int RT = (long long)a.n_q * v.n_rep > kRows ? 2 * kRows : kRows;
  const auto kern = query_many_kernel<F, D>;
  // at least what keeps a second CTA off the SM: each takes all of its tensor memory
  constexpr size_t need = Lay<D>::kMisc + sizeof(Misc), smem = need > 120 * 1024 ? need : 120 * 1024;
  static_assert(smem <= 232448, "shared memory of an SM");
  const kvq_status ss = ensure_dynamic_smem(kSlotQueryTc + F * 2 + (D == 64 ? 0 : 1), kern, smem);
  if (ss != KVQ_OK) return ss == KVQ_ERR_CAPACITY ? KVQ_ERR_CUDA : ss;
  int grid = num_sms();
  if (grid > kManyGrid) grid = kManyGrid;
  kern<<<grid, kMThreads, smem, st>>>(v, a, ws, RT);
  if (cudaGetLastError() != cudaSuccess) return KVQ_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid * (RT / kMergeRows));
  cfg.blockDim = dim3(kMergeRows * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, many_merge_kernel<D>, v, a, (const unsigned char*)ws, RT, grid) == cudaSuccess ? KVQ_OK
                                                                                                               : KVQ_ERR_CUDA;
}

}  // namespace

size_t query_many_workspace_bytes(const KvqView& v, int batch, int n_q) {
  const int RT = (long long)n_q * v.n_rep > kRows ? 2 * kRows : kRows;
  return many_header_bytes(kManyGrid) + 2ull * kManyGrid * many_rec_bytes(v.D, RT);
}

kvq_status launch_query_many(const KvqView& v, const QueryArgs& a, void* ws, cudaStream_t st) {
  unsigned char* w = static_cast<unsigned char*>(ws);
  switch (fmt_index(v.kfmt) * 2 + (v.D == 128)) {
    case 0: return launch_many_t<kI8, 64>(v, a, w, st);
    case 1: return launch_many_t<kI8, 128>(v, a, w, st);
    case 2: return launch_many_t<kE4, 64>(v, a, w, st);
    case 3: return launch_many_t<kE4, 128>(v, a, w, st);
    case 4: return launch_many_t<kE5, 64>(v, a, w, st);
    default: return launch_many_t<kE5, 128>(v, a, w, st);
  }
}

}  // namespace kvq
