// Append to a PER_BLOCK cache (8-bit codes, one scale per block of G tokens and
// kv-head), with or without the position rotation, and the rotation of the queries
// that come with the keys.
//
// Mathematics (include/kvq.h gives the exact roundings): rotated keys and the values
// go to the residual window; a window that fills is cut into blocks of G tokens x D
// channels, s = max|x| * (1 / qmax) over the block, code = x / s rounded.
//
// What bounds it: memory for prompts (each row is read once and written once, 16
// bytes a thread and access), launch latency for decode steps.  A thread owns items of
// 16 channels of one row: two 8-channel pieces that hold both channels of 8 rotation
// pairs (adjacent pieces for interleaved pairs, half the rotated width apart for
// halves), so a rotation never leaves the thread and its cosines and sines are two
// contiguous runs of 8.  A CTA keeps a whole block's keys and values in registers
// between the maximum and the rounding, where they fit (64 bf16 tokens of 128 channels);
// larger blocks are read twice, the second
// time from L2.
//
// Decode steps take one launch: a cluster per sequence, its CTAs over the kv-heads, the
// CTA that reads a head's window also overwriting it, and the length advanced behind a
// cluster barrier that follows every CTA's read of it.  Prompts take two: blocks and
// queries over the whole GPU, then (a programmatic dependent) the window rows and lengths.
//
// Measured (8 kv-heads of 128): 8 prompts of 4,096 tokens with 64 query heads take 230 us, 5.6 TB/s (82% of the
// measured copy bandwidth); a decode step of 64 sequences 5.5 us, 9 where a window fills.
#include "kvq_host.h"
#include "kvq_internal.cuh"
#include "kvq_ptx.cuh"
#include "kvq_rope.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kCh = 16;  // channels per item

// 16 channels as two 8-channel pieces, in the source dtype.
template <bool BF16>
struct Item;
template <>
struct Item<true> {
  uint4 lo, hi;
  __device__ __forceinline__ void load(const void* row, int cl, int ch) {
    const uint16_t* p = static_cast<const uint16_t*>(row);
    lo = *reinterpret_cast<const uint4*>(p + cl);
    hi = *reinterpret_cast<const uint4*>(p + ch);
  }
  __device__ __forceinline__ void store(void* row, int cl, int ch) const {
    uint16_t* p = static_cast<uint16_t*>(row);
    *reinterpret_cast<uint4*>(p + cl) = lo;
    *reinterpret_cast<uint4*>(p + ch) = hi;
  }
  __device__ __forceinline__ void zero() { lo = hi = make_uint4(0u, 0u, 0u, 0u); }
  static __device__ __forceinline__ void unpack8(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
  }
  __device__ __forceinline__ void get(float (&x)[kCh]) const {
    unpack8(lo, x);
    unpack8(hi, x + 8);
  }
  __device__ __forceinline__ void set(const float (&x)[kCh]) {  // rounds to nearest even
    lo = pack8(x);
    hi = pack8(x + 8);
  }
};
template <>
struct Item<false> {
  float4 lo[2], hi[2];
  __device__ __forceinline__ void load(const void* row, int cl, int ch) {
    const float* p = static_cast<const float*>(row);
    lo[0] = *reinterpret_cast<const float4*>(p + cl);
    lo[1] = *reinterpret_cast<const float4*>(p + cl + 4);
    hi[0] = *reinterpret_cast<const float4*>(p + ch);
    hi[1] = *reinterpret_cast<const float4*>(p + ch + 4);
  }
  __device__ __forceinline__ void store(void* row, int cl, int ch) const {
    float* p = static_cast<float*>(row);
    *reinterpret_cast<float4*>(p + cl) = lo[0];
    *reinterpret_cast<float4*>(p + cl + 4) = lo[1];
    *reinterpret_cast<float4*>(p + ch) = hi[0];
    *reinterpret_cast<float4*>(p + ch + 4) = hi[1];
  }
  __device__ __forceinline__ void zero() { lo[0] = lo[1] = hi[0] = hi[1] = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&x)[kCh]) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      x[4 * j] = lo[j].x; x[4 * j + 1] = lo[j].y; x[4 * j + 2] = lo[j].z; x[4 * j + 3] = lo[j].w;
      x[8 + 4 * j] = hi[j].x; x[9 + 4 * j] = hi[j].y; x[10 + 4 * j] = hi[j].z; x[11 + 4 * j] = hi[j].w;
    }
  }
  __device__ __forceinline__ void set(const float (&x)[kCh]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      lo[j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
      hi[j] = make_float4(x[8 + 4 * j], x[9 + 4 * j], x[10 + 4 * j], x[11 + 4 * j]);
    }
  }
};

// Items a thread holds of each of keys and values: 32 packed registers in all, so that four CTAs share an SM
// (a batch's decode step is then resident at once, and a prompt's loads cover the memory's latency).
template <bool BF16>
constexpr int items_held() { return BF16 ? 2 : 1; }

// Channels of item p of a row: its two pieces.
__device__ __forceinline__ void item_channels(const RopeView& r, int p, int& cl, int& ch) {
  const bool split = r.cs != nullptr && r.halves && p < r.rot / kCh;
  cl = split ? 8 * p : kCh * p;
  ch = split ? r.rot / 2 + 8 * p : kCh * p + 8;
}

struct Angles {
  float c[8], s[8];
  __device__ __forceinline__ void load(const RopeView& r, int pos, int p) {
    const float* row = r.cs + (long long)pos * r.rot + 8 * p;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float4 a = *reinterpret_cast<const float4*>(row + 4 * j);
      const float4 b = *reinterpret_cast<const float4*>(row + r.rot / 2 + 4 * j);
      c[4 * j] = a.x; c[4 * j + 1] = a.y; c[4 * j + 2] = a.z; c[4 * j + 3] = a.w;
      s[4 * j] = b.x; s[4 * j + 1] = b.y; s[4 * j + 2] = b.z; s[4 * j + 3] = b.w;
    }
  }
};

// Rotate a rotated item's 8 pairs and round them to the source dtype.
template <bool BF16>
__device__ __forceinline__ void rotate(Item<BF16>& it, const Angles& a, bool halves) {
  float x[kCh], y[kCh];
  it.get(x);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float u = halves ? x[i] : x[2 * i], w = halves ? x[8 + i] : x[2 * i + 1];
    const float f = rope_first(u, w, a.c[i], a.s[i]), g = rope_second(u, w, a.c[i], a.s[i]);
    if (halves) {
      y[i] = f;
      y[8 + i] = g;
    } else {
      y[2 * i] = f;
      y[2 * i + 1] = g;
    }
  }
  it.set(y);
}

// One call, as its kernels see it.
struct BlockAppend {
  RopeView r;
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  long long qs, ks, vs;  // elements between rows
  int n_new, rotate_keys;
  const int32_t* n_per_seq;
};

// Sequence b's length before the call and its number of new rows; false: nothing to do
// (*bad: because it does not fit).
__device__ __forceinline__ bool sequence_step(const KvqView& v, const BlockAppend& a, int b, int& T0, int& n, bool* bad) {
  T0 = v.seq_lens[b];
  n = a.n_per_seq ? a.n_per_seq[b] : a.n_new;
  *bad = false;
  if (n <= 0) return false;
  const long long end = (long long)T0 + n;
  if (T0 < 0 || n > a.n_new || end > (long long)v.max_pages * v.P || (a.r.cs && end > a.r.positions)) {
    *bad = true;
    return false;
  }
  return true;
}

template <bool BF16>
__device__ __forceinline__ const void* row_at(const void* base, long long elem) {
  return static_cast<const char*>(base) + elem * (BF16 ? 2 : 4);
}
template <bool BF16>
__device__ __forceinline__ void* row_at(void* base, long long elem) {
  return static_cast<char*>(base) + elem * (BF16 ? 2 : 4);
}

// Item p of token t's key (KEY) or value, rotated where it is new.
template <bool BF16, bool KEY>
__device__ __forceinline__ void load_item(const KvqView& v, const BlockAppend& a, int b, int h, int T0, int wbase, int t,
                                          int p, Item<BF16>& it) {
  int cl, ch;
  item_channels(a.r, p, cl, ch);
  if (t < T0) {  // in the window, rotated when it came
    const long long w = (((long long)b * v.R + (t - wbase)) * v.Hkv + h) * v.D;
    it.load(row_at<BF16>(KEY ? v.k_win : v.v_win, w), cl, ch);
  } else {
    const long long i = ((long long)b * a.n_new + (t - T0)) * (KEY ? a.ks : a.vs) + (long long)h * v.D;
    it.load(row_at<BF16>(KEY ? a.k : a.v, i), cl, ch);
    if (KEY && a.rotate_keys && p < a.r.rot / kCh) {
      Angles g;
      g.load(a.r, t, p);
      rotate<BF16>(it, g, a.r.halves);
    }
  }
}

// Largest magnitude of an item, as bits: ordered like the magnitudes, infinities and then NaN above them (a maximum of
// floats would pass over NaN).
template <bool BF16>
__device__ __forceinline__ uint32_t item_absmax(const Item<BF16>& it) {
  float x[kCh];
  it.get(x);
  uint32_t m[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < kCh; ++i) m[i & 3] = max(m[i & 3], __float_as_uint(x[i]) & 0x7fffffffu);
  return max(max(m[0], m[1]), max(m[2], m[3]));
}

// Two FP8 bytes (a in the low one): nearest, ties to even, saturating.
template <bool E5M2>
__device__ __forceinline__ uint32_t fp8x2(float a, float b) {
  uint16_t r;
  if constexpr (E5M2) {
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(b), "f"(a));
  } else {
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(b), "f"(a));
  }
  return r;
}

// The codes of 8 channels, from r = fl32(1 / s) instead of a division each.
// INT8: rint(fl32(x * r)) equals rint(fl32(x / s)) unless a half-integer lies between them; products within
// 2^-20 |q| of one (over five times the distance of the two quotients) and values that are not finite take the
// IEEE division.  FP8: the quotient lies between q (1 - 2^-20) and q (1 + 2^-20), and rounding is monotone: where
// both ends give the same byte it is the quotient's, elsewhere the division decides.  (r is exact enough only
// while 1 / s is a normal number: smaller or larger scales divide.)  Scales of 0 and NaN give codes 0.
template <int F>  // 0 INT8, 1 E4M3, 2 E5M2
__device__ __forceinline__ uint2 codes8(const float* x, float s, float r) {
  uint32_t w[2] = {0u, 0u};
  if constexpr (F == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = __fmul_rn(x[i], r);
      float c = rintf(q);
      if (!(fabsf(__fsub_rn(fabsf(__fsub_rn(q, c)), 0.5f)) > __fmul_rn(9.5367431640625e-07f, fabsf(q))))
        c = rintf(__fdiv_rn(x[i], s));
      const uint32_t u = !(s > 0.f) ? 0u : static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(c, -127.f), 127.f))) & 0xFFu;
      w[i >> 2] |= u << (8 * (i & 3));
    }
  } else {
    constexpr float kLo = 1.f - 9.5367431640625e-07f, kHi = 1.f + 9.5367431640625e-07f;
    const bool near = s > 7.888609052210118e-31f && s < 1.2676506002282294e+30f;  // 2^-100 .. 2^100
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float a = __fmul_rn(x[i], r), b = __fmul_rn(x[i + 1], r);
      uint32_t u = fp8x2<F == 2>(__fmul_rn(a, kLo), __fmul_rn(b, kLo));
      if (!near || u != fp8x2<F == 2>(__fmul_rn(a, kHi), __fmul_rn(b, kHi)))
        u = !(s > 0.f) ? 0u : fp8x2<F == 2>(__fdiv_rn(x[i], s), __fdiv_rn(x[i + 1], s));
      w[i >> 2] |= u << (8 * (i & 2));
    }
  }
  return make_uint2(w[0], w[1]);
}

// The 16 codes of an item.  Out of line: a launch runs this code a few times from cold instruction caches, so
// one copy for every item of keys and values costs less than the calls.
template <bool BF16>
__device__ __noinline__ uint4 item_codes(Item<BF16> it, float s, float r, int fmt) {
  float x[kCh];
  it.get(x);
  uint2 a, b;
  if (fmt == KVQ_FP8_E4M3) {
    a = codes8<1>(x, s, r);
    b = codes8<1>(x + 8, s, r);
  } else if (fmt == KVQ_FP8_E5M2) {
    a = codes8<2>(x, s, r);
    b = codes8<2>(x + 8, s, r);
  } else {
    a = codes8<0>(x, s, r);
    b = codes8<0>(x + 8, s, r);
  }
  return make_uint4(a.x, a.y, b.x, b.y);
}

template <bool BF16>
__device__ __forceinline__ void store_codes(uint8_t* row, int cl, int ch, const Item<BF16>& it, float s, float r, int fmt) {
  const uint4 c = item_codes<BF16>(it, s, r, fmt);
  *reinterpret_cast<uint2*>(row + cl) = make_uint2(c.x, c.y);
  *reinterpret_cast<uint2*>(row + ch) = make_uint2(c.z, c.w);
}

// Scale of a block whose largest magnitude has the bits m; NaN where an element is not finite.
__device__ __forceinline__ float block_scale_of(uint32_t m, float rqmax, int meta16) {
  const float s = __fmul_rn(__uint_as_float(m), rqmax);
  return m >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : meta16 ? f16_up(s) : s;
}

__device__ __forceinline__ float block_rqmax(int fmt) {  // the fp32 numbers nearest to 1 / qmax
  return fmt == KVQ_FP8_E4M3 ? 1.f / 448.f : fmt == KVQ_FP8_E5M2 ? 1.f / 57344.f : 1.f / 127.f;
}

struct FoldSmem {
  uint32_t mk[kThreads / 32], mv[kThreads / 32];  // of either kernel's warps
};

// Quantize block [t0, t0 + G) of one head.  Whole CTA; ends with a barrier, so the window
// rows it read may be overwritten.
template <bool BF16, int NT>
__device__ void fold_block(const KvqView& v, const BlockAppend& a, FoldSmem& sm, int b, int h, int T0, int wbase, int t0) {
  constexpr int N = items_held<BF16>();
  const int np = v.D / kCh, lp = __ffs(np) - 1, G = v.kgroup, items = G << lp;
  const bool held = items <= N * NT;
  Item<BF16> k[N], w[N];
  uint32_t mk = 0u, mv = 0u;
  for (int base = 0; base < items; base += N * NT) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = base + j * NT + threadIdx.x;
      k[j].zero();
      w[j].zero();
      if (e < items) {
        load_item<BF16, true>(v, a, b, h, T0, wbase, t0 + (e >> lp), e & (np - 1), k[j]);
        load_item<BF16, false>(v, a, b, h, T0, wbase, t0 + (e >> lp), e & (np - 1), w[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      mk = max(mk, item_absmax<BF16>(k[j]));
      mv = max(mv, item_absmax<BF16>(w[j]));
    }
  }
  mk = __reduce_max_sync(0xffffffffu, mk);
  mv = __reduce_max_sync(0xffffffffu, mv);
  if ((threadIdx.x & 31) == 0) {
    sm.mk[threadIdx.x >> 5] = mk;
    sm.mv[threadIdx.x >> 5] = mv;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    mk = max(mk, sm.mk[i]);
    mv = max(mv, sm.mv[i]);
  }
  const float ks = block_scale_of(mk, block_rqmax(v.kfmt), v.meta16), vs = block_scale_of(mv, block_rqmax(v.vfmt), v.meta16);
  const float kr = ks > 0.f ? __frcp_rn(ks) : 0.f, vr = vs > 0.f ? __frcp_rn(vs) : 0.f;
  if (threadIdx.x == 0) {
    uint8_t* page = page_of(v, b, t0);
    if (page) {
      uint8_t* hb = page + (long long)h * v.head_bytes;
      const int slot = (t0 % v.P) / G;
      store_meta(hb + v.off_km, slot, ks, v.meta16);
      store_meta(hb + v.off_vm, slot, vs, v.meta16);
    }
  }
  for (int base = 0; base < items; base += N * NT) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = base + j * NT + threadIdx.x;
      if (e >= items) continue;
      const int t = t0 + (e >> lp), p = e & (np - 1);
      if (!held) {
        load_item<BF16, true>(v, a, b, h, T0, wbase, t, p, k[j]);
        load_item<BF16, false>(v, a, b, h, T0, wbase, t, p, w[j]);
      }
      uint8_t* page = page_of(v, b, t);
      if (!page) continue;
      uint8_t* hb = page + (long long)h * v.head_bytes + (long long)(t % v.P) * v.D;
      int cl, ch;
      item_channels(a.r, p, cl, ch);
      store_codes<BF16>(hb, cl, ch, k[j], ks, kr, v.kfmt);
      store_codes<BF16>(hb + v.off_vc, cl, ch, w[j], vs, vr, v.vfmt);
    }
  }
  __syncthreads();
}

// The new rows that stay in the window, tokens [max(T1 / R * R, T0), T1) of heads [h0, h1): thread `at` of `n`.
template <bool BF16>
__device__ __forceinline__ void write_window(const KvqView& v, const BlockAppend& a, int b, int h0, int h1, int T0, int T1, int at,
                                             int n) {
  const int base = T1 / v.R * v.R, first = max(base, T0);
  const int np = v.D / kCh, lp = __ffs(np) - 1, per = (h1 - h0) << lp;  // items of a token
#pragma unroll 1
  for (int e = at; e < (T1 - first) * per; e += n) {
    const int t = first + e / per, h = h0 + (e % per >> lp), p = e & (np - 1);
    Item<BF16> k, w;
    load_item<BF16, true>(v, a, b, h, T0, base, t, p, k);
    load_item<BF16, false>(v, a, b, h, T0, base, t, p, w);
    const long long o = (((long long)b * v.R + (t - base)) * v.Hkv + h) * v.D;
    int cl, ch;
    item_channels(a.r, p, cl, ch);
    k.store(row_at<BF16>(v.k_win, o), cl, ch);
    w.store(row_at<BF16>(v.v_win, o), cl, ch);
  }
}

// Queries [i0, i1) of sequence b, heads [h0, h1): a thread takes one item of a group of HG heads
// of a token, so that its cosines and sines are read once a group.
template <bool BF16, int NT, int HG>
__device__ __forceinline__ void rotate_queries(const KvqView& v, const BlockAppend& a, int b, int T0, int i0, int i1,
                                               int h0, int h1) {
  const int np = v.D / kCh, lp = __ffs(np) - 1;
  const int p = threadIdx.x & (np - 1), slot = threadIdx.x >> lp, slots = NT >> lp;
  const int groups = (h1 - h0 + HG - 1) / HG;
  const bool rot = p < a.r.rot / kCh;
  int cl, ch;
  item_channels(a.r, p, cl, ch);
  for (int e = slot; e < (i1 - i0) * groups; e += slots) {
    const int i = i0 + e / groups, hq = h0 + e % groups * HG;
    const long long tok = (long long)b * a.n_new + i;
    Item<BF16> x[HG];
#pragma unroll
    for (int j = 0; j < HG; ++j)
      if (hq + j < h1) x[j].load(row_at<BF16>(a.q, tok * a.qs + (long long)(hq + j) * v.D), cl, ch);
    if (rot) {
      Angles g;
      g.load(a.r, T0 + i, p);
#pragma unroll
      for (int j = 0; j < HG; ++j)
        if (hq + j < h1) rotate<BF16>(x[j], g, a.r.halves);
    }
#pragma unroll
    for (int j = 0; j < HG; ++j)
      if (hq + j < h1) x[j].store(row_at<BF16>(a.q_out, (tok * v.Hq + hq + j) * v.D), cl, ch);
  }
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }

// A cluster of `ranks` CTAs per sequence.  whole: the blocks and queries too (a decode step);
// otherwise only the window rows and the length, behind the grid that did the rest.
template <bool BF16>
__global__ void __launch_bounds__(kThreads, 4) block_step_kernel(KvqView v, BlockAppend a, int ranks, int whole) {
  __shared__ FoldSmem sm;
  if (!whole) ptx::grid_dep_wait();
  const int b = blockIdx.x / ranks, rank = blockIdx.x % ranks;
  int T0, n;
  bool bad;
  const bool live = sequence_step(v, a, b, T0, n, &bad);
  cluster_arrive();  // this CTA has read the length
  if (whole && bad && rank == 0 && threadIdx.x == 0) atomicOr(v.status, KVQ_DEV_OVERFLOW);
  if (live) {
    const int T1 = T0 + n;
    if (whole && a.q) {
      const int per = (v.Hq + ranks - 1) / ranks;
      rotate_queries<BF16, kThreads, 1>(v, a, b, T0, 0, n, min(v.Hq, rank * per), min(v.Hq, rank * per + per));
    }
    if (whole && T1 / v.R > T0 / v.R) {  // n <= R: one window fills at most
      const int wbase = T0 / v.R * v.R;
      for (int h = rank; h < v.Hkv; h += ranks) {
        for (int t = wbase; t < wbase + v.R; t += v.kgroup) fold_block<BF16, kThreads>(v, a, sm, b, h, T0, wbase, t);
        write_window<BF16>(v, a, b, h, h + 1, T0, T1, threadIdx.x, kThreads);  // after this head's rows were read
      }
    } else {
      write_window<BF16>(v, a, b, 0, v.Hkv, T0, T1, rank * kThreads + threadIdx.x, ranks * kThreads);
    }
  }
  cluster_wait();
  if (live && rank == 0 && threadIdx.x == 0) v.seq_lens[b] = T0 + n;
}

// Heads a thread takes of a token in a prompt.  8 prompts of 4,096 tokens with 64 query heads take 230 us with 2, 238
// with 4, 340 with 8 (fewer threads with loads in flight), 272 with 1 (the angles are loaded again).
constexpr int kQHeads = 2;

// Blocks and queries of a prompt: CTAs [0, nfold) take one (sequence, block, head) each, the
// rest q_tok tokens of a sequence's queries.
template <bool BF16>
__global__ void __launch_bounds__(kThreads, 4) block_prompt_kernel(KvqView v, BlockAppend a, unsigned nfold, int blocks, int q_tok,
                                                                int q_units) {
  __shared__ FoldSmem sm;
  ptx::grid_dep_launch();
  const unsigned u = blockIdx.x;
  int T0, n;
  bool bad;
  if (u < nfold) {
    const int h = u % v.Hkv, x = u / v.Hkv, j = x % blocks, b = x / blocks;
    const bool live = sequence_step(v, a, b, T0, n, &bad);
    if (bad && j == 0 && h == 0 && threadIdx.x == 0) atomicOr(v.status, KVQ_DEV_OVERFLOW);
    if (!live) return;
    const int wbase = T0 / v.R * v.R, t = wbase + j * v.kgroup;
    if (t < (T0 + n) / v.R * v.R) fold_block<BF16, kThreads>(v, a, sm, b, h, T0, wbase, t);
  } else {
    const unsigned x = u - nfold;
    const int b = x / q_units, i0 = x % q_units * q_tok;
    if (!sequence_step(v, a, b, T0, n, &bad)) return;
    if (i0 < n) rotate_queries<BF16, kThreads, kQHeads>(v, a, b, T0, i0, min(n, i0 + q_tok), 0, v.Hq);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) rope_query_kernel(KvqView v, BlockAppend a, int q_tok, int q_units) {
  const int b = blockIdx.x / q_units, i0 = blockIdx.x % q_units * q_tok;
  int T0, n;
  bool bad;
  if (!sequence_step(v, a, b, T0, n, &bad) || i0 >= n) return;
  rotate_queries<BF16, kThreads, 1>(v, a, b, T0, i0, min(n, i0 + q_tok), 0, v.Hq);
}

// Tokens of queries a CTA takes: about two passes of its threads over groups of kQHeads heads.
int query_tokens(const KvqView& v) {
  const int slots = kThreads / (v.D / kCh), groups = (v.Hq + kQHeads - 1) / kQHeads;
  const int t = 2 * slots / groups;
  return t < 1 ? 1 : t;
}

constexpr int kRanks = 8;  // CTAs per cluster (the portable limit)

// Whether a call takes the one-launch kernel.  Where no window fills it is ahead to 48 rows and beyond (16 sequences, 32
// query heads on 8 of 128, R = 64, us, against the two launches: 32 rows 8.3 and 12.0); where one does, a head's
// blocks take one CTA turns and it falls behind from 17 rows on (12.8 and 11.9, 32 rows 14.3 and 12.3).  So it
// takes up to 16 rows, and up to 32 if at most every other call of that size fills a window.
bool one_launch(const KvqView& v, int n) { return n <= v.R && (n <= 16 || (n <= 32 && 2 * n <= v.R)); }

template <bool BF16>
kvq_status launch_block_t(const KvqView& v, const BlockAppend& a, cudaStream_t st) {
  const bool step = one_launch(v, a.n_new);
  const int ranks = kRanks;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((long long)v.batch * ranks > 0x7FFFFFFFLL) return KVQ_ERR_CAPACITY;
  if (!step) {
    const long long blocks = ((long long)a.n_new + v.R - 1) / v.R * (v.R / v.kgroup);
    const int q_tok = query_tokens(v);
    const long long q_units = a.q ? ((long long)a.n_new + q_tok - 1) / q_tok : 0;
    const long long nfold = blocks * v.Hkv * v.batch, total = nfold + q_units * v.batch;
    if (total > 0x7FFFFFFFLL) return KVQ_ERR_CAPACITY;
    block_prompt_kernel<BF16><<<(unsigned)total, kThreads, 0, st>>>(v, a, (unsigned)nfold, (int)blocks, q_tok,
                                                                    q_units ? (int)q_units : 1);
    if (cudaGetLastError() != cudaSuccess) return KVQ_ERR_CUDA;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
  }
  cfg.gridDim = dim3((unsigned)v.batch * ranks);
  return cudaLaunchKernelEx(&cfg, block_step_kernel<BF16>, v, a, ranks, step ? 1 : 0) == cudaSuccess ? KVQ_OK
                                                                                                     : KVQ_ERR_CUDA;
}

}  // namespace

kvq_status launch_block_append(const KvqView& v, const RopeView& r, const void* q, const void* k_new,
                               const void* v_new, long long qs, long long ks, long long vs, int n_new,
                               const int32_t* n_new_per_seq, void* q_out, cudaStream_t st) {
  const BlockAppend a{r, q, k_new, v_new, q_out, qs, ks, vs, n_new, r.cs != nullptr && !v.rope_pre, n_new_per_seq};
  return v.src_bf16 ? launch_block_t<true>(v, a, st) : launch_block_t<false>(v, a, st);
}

kvq_status launch_rope_queries(const KvqView& v, const RopeView& r, const void* q, long long qs, int n_new,
                               const int32_t* n_new_per_seq, void* q_out, cudaStream_t st) {
  const BlockAppend a{r, q, nullptr, nullptr, q_out, qs, 0, 0, n_new, 0, n_new_per_seq};
  const int q_tok = query_tokens(v);
  const long long q_units = ((long long)n_new + q_tok - 1) / q_tok, total = q_units * v.batch;
  if (total > 0x7FFFFFFFLL) return KVQ_ERR_CAPACITY;
  if (v.src_bf16) {
    rope_query_kernel<true><<<(unsigned)total, kThreads, 0, st>>>(v, a, q_tok, (int)q_units);
  } else {
    rope_query_kernel<false><<<(unsigned)total, kThreads, 0, st>>>(v, a, q_tok, (int)q_units);
  }
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace kvq
