// One stored key or value, dequantized by the rules of include/kvq.h: the plain
// per-element reading of a cache that kvq_dequantize and the plain attention kernel
// share.  Every axis, format and the window; a missing page reads as 0.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

// Scale slot of PER_CHANNEL / PER_BLOCK group g0 / G inside its page (the page of token g0).
__device__ __forceinline__ int group_slot(int g0, int P, int G) { return (g0 % P) / G; }

// Scale of the PER_BLOCK block that holds token t of sequence b (0, and *ok cleared, when its page is missing).
// off_meta: v.off_km or v.off_vm.
__device__ __forceinline__ float block_scale(const KvqView& v, int b, int h, int t, int off_meta, bool* ok) {
  const int g0 = t / v.kgroup * v.kgroup;  // keys and values share one group
  const uint8_t* page = page_of(v, b, g0);
  if (!page) {
    *ok = false;
    return 0.f;
  }
  return load_meta(page + (long long)h * v.head_bytes + off_meta, group_slot(g0, v.P, v.kgroup), v.meta16);
}

// Value of an 8-bit code byte of a PER_BLOCK tensor, before its scale (exact).
__device__ __forceinline__ float block_code_value(unsigned u, int fmt) {
  return is_fp8(fmt) ? fp8_to_float(u, fmt) : static_cast<float>(static_cast<int8_t>(u));
}

// Channel c of the key of token t < T (nq = n_quantized(T, R)) of sequence b, kv-head h.
// *ok is cleared when its page is missing, or the page that holds its group's scale.
__device__ inline float cache_key(const KvqView& v, int b, int h, int t, int c, int nq, bool* ok) {
  if (t >= nq) return load_src(v.k_win, (((long long)b * v.R + (t - nq)) * v.Hkv + h) * v.D + c, v.src_bf16);
  const uint8_t* page = page_of(v, b, t);
  if (!page) {
    *ok = false;
    return 0.f;
  }
  const uint8_t* hb = page + (long long)h * v.head_bytes;
  const int slot = t % v.P;
  const unsigned ku = get_code(hb + (long long)slot * v.krow, c, v.kbits);
  if (v.kaxis == KVQ_PER_BLOCK) return __fmul_rn(block_code_value(ku, v.kfmt), block_scale(v, b, h, t, v.off_km, ok));
  if (is_fp8(v.kfmt)) return __fmul_rn(fp8_to_float(ku, v.kfmt), v.k_scale[h]);
  if (v.kaxis == KVQ_PER_TENSOR) return dequant_sym(signed_code(ku, v.kbits, KVQ_SYM_ABSMAX), v.k_scale[h]);
  const uint8_t* meta;
  float s, mn = 0.f;
  if (v.kaxis == KVQ_PER_TOKEN) {
    meta = hb + v.off_km + (long long)slot * v.k_ng * v.k_nmeta * v.mb;
    const int grp = c / v.kgroup;
    s = load_meta(meta, grp, v.meta16);
    if (v.k_nmeta == 2) mn = load_meta(meta, v.k_ng + grp, v.meta16);
  } else {
    const int g0 = (t / v.kgroup) * v.kgroup;
    const uint8_t* gp = page_of(v, b, g0);
    if (!gp) *ok = false;
    meta = gp ? gp + (long long)h * v.head_bytes + v.off_km +
                    (long long)group_slot(g0, v.P, v.kgroup) * v.D * v.k_nmeta * v.mb
              : nullptr;
    s = meta ? load_meta(meta, c, v.meta16) : 0.f;
    if (meta && v.k_nmeta == 2) mn = load_meta(meta, v.D + c, v.meta16);
  }
  const int code = signed_code(ku, v.kbits, v.kmode);
  return v.kmode == KVQ_ASYM_MINMAX ? dequant_asym(code, s, mn) : dequant_sym(code, s);
}

// Channel c of the value of the same token.
__device__ inline float cache_value(const KvqView& v, int b, int h, int t, int c, int nq) {
  if (t >= nq) return load_src(v.v_win, (((long long)b * v.R + (t - nq)) * v.Hkv + h) * v.D + c, v.src_bf16);
  const uint8_t* page = page_of(v, b, t);
  if (!page) return 0.f;
  const uint8_t* hb = page + (long long)h * v.head_bytes;
  const int slot = t % v.P;
  const unsigned vu = get_code(hb + v.off_vc + (long long)slot * v.vrow, c, v.vbits);
  if (v.vaxis == KVQ_PER_BLOCK) {
    bool ok;  // as its key's
    return __fmul_rn(block_code_value(vu, v.vfmt), block_scale(v, b, h, t, v.off_vm, &ok));
  }
  if (is_fp8(v.vfmt)) return __fmul_rn(fp8_to_float(vu, v.vfmt), v.v_scale[h]);
  if (v.vaxis == KVQ_PER_TENSOR) return dequant_sym(signed_code(vu, v.vbits, KVQ_SYM_ABSMAX), v.v_scale[h]);
  const uint8_t* meta = hb + v.off_vm + (long long)slot * v.v_ng * v.v_nmeta * v.mb;
  const int grp = c / v.vgroup;
  const int code = signed_code(vu, v.vbits, v.vmode);
  const float s = load_meta(meta, grp, v.meta16);
  return v.vmode == KVQ_ASYM_MINMAX ? dequant_asym(code, s, load_meta(meta, v.v_ng + grp, v.meta16))
                                    : dequant_sym(code, s);
}

}  // namespace kvq
