"""Block-scaled 8-bit caches, rotated append and query attention without a GPU: the
oracle's new steps against hand-worked values and independent formulas, the library's
layout arithmetic against the oracle's, and every refusal of the new entry points
(arguments are checked before anything is launched)."""
import ctypes

import numpy as np
import pytest

from oracle import kvq_oracle as O

BLK, S = O.PER_BLOCK, O.SYM


@pytest.fixture(scope="module")
def K():
    import __graft_entry__
    __graft_entry__.build()
    import asymmetric_quantized_kv_gb300 as K
    return K


# ------------------------------------------------------------------------------ oracle

def test_block_quantizer_by_hand():
    x = np.zeros((32, 64))
    x[3, 7] = -254.0          # block 0: scale 2
    x[5, 1] = 3.0             # 1.5 -> 2 (ties to even)
    x[6, 2] = 5.0             # 2.5 -> 2
    c, s, _ = O._quant_block(x, O.QSpec(O.INT8, S, BLK, 16))
    assert s.tolist() == [2.0, 0.0]
    assert (c[3, 7], c[5, 1], c[6, 2]) == (-127, 2, 2) and not c[16:].any()
    x[20, 0] = 896.0          # block 1 in E4M3: scale 2, byte of 448
    x[21, 0] = 17.0           # 8.5: between 8 and 9, ties to the even mantissa (8)
    c, s, _ = O._quant_block(x, O.QSpec(O.FP8_E4M3, S, BLK, 16))
    assert s[1] == 2.0 and c[20, 0] == 0x7E and c[21, 0] == 0x50
    d = O._dequant_block(c, s, O.QSpec(O.FP8_E4M3, S, BLK, 16))
    assert d[20, 0] == 896.0 and d[21, 0] == 16.0


@pytest.mark.parametrize("fmt,step", [(O.INT8, None), (O.FP8_E4M3, 2.0 ** -4), (O.FP8_E5M2, 2.0 ** -3)])
@pytest.mark.parametrize("m16", [False, True])
def test_block_quantizer_error_bound(fmt, step, m16):
    x = O.bf16(np.random.default_rng(3).standard_normal((96, 64)) * 3)
    spec = O.QSpec(fmt, S, BLK, 32)
    c, s, _ = O._quant_block(x, spec, m16)
    err = np.abs(O._dequant_block(c, s, spec) - x).reshape(3, -1)
    xa = np.abs(x).reshape(3, -1)
    # INT8: half a scale; FP8: half a step relative, or half the subnormal step times the scale.
    # fl32(x/s) and the product are each off by 2^-24 of themselves, so of |x| and of at most
    # |x| + s/2: together under 2^-22 |x| (where |x| < s/2 the code is 0 and the error is |x|)
    sub = {O.FP8_E4M3: 2.0 ** -10, O.FP8_E5M2: 2.0 ** -17}.get(fmt)
    lim = s[:, None] / 2 if fmt == O.INT8 else np.maximum(xa * step, sub * s[:, None])
    assert np.all(err <= lim + 2.0 ** -22 * xa)


def test_block_stream_equals_token_at_a_time():
    cfg = O.Config(4, 2, 64, O.QSpec(O.INT8, S, BLK, 16), O.QSpec(O.FP8_E4M3, S, BLK, 16), 32, 16)
    g = np.random.default_rng(0)
    K_, V_ = O.fl32(g.standard_normal((2, 101, 64)))
    a = O.quantize_stream(cfg, K_, V_)
    m = O.StreamCache(cfg)
    for i in range(0, 101, 7):
        m.append(K_[i:i + 7], V_[i:i + 7])
    b = m.state()
    assert a.n_q == 96 and b.n_q == 96
    for f in ("kc", "ks", "vc", "vs", "k_win", "v_win"):
        assert np.array_equal(getattr(a, f), getattr(b, f)), f


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("rot", [16, 64])
def test_rope_rows_against_complex_numbers(halves, rot):
    g = np.random.default_rng(1)
    x = O.fl32(g.standard_normal((9, 64)))
    pos = g.integers(0, 50, 9)
    ang = np.arange(50)[:, None] * 1e4 ** (-2 * np.arange(rot // 2) / rot)
    table = O.fl32(np.concatenate([np.cos(ang), np.sin(ang)], 1))
    y = O.rope_rows(x, pos, table, rot, halves)
    half = rot // 2
    z = x[:, :half] + 1j * x[:, half:rot] if halves else x[:, 0:rot:2] + 1j * x[:, 1:rot:2]
    z = z * np.exp(1j * ang[pos])
    got = y[:, :half] + 1j * y[:, half:rot] if halves else y[:, 0:rot:2] + 1j * y[:, 1:rot:2]
    # three fp32 roundings a channel (two products, a sum) and the table's: 2^-22 of the pair's size
    assert np.all(np.abs(got - z) <= 2.0 ** -22 * (np.abs(z) + 1e-30))
    assert np.array_equal(y[:, rot:], x[:, rot:])
    assert np.array_equal(O.rope_rows(x, pos, table, rot, halves, O.BF16), O.bf16(y))


def test_bf16_rounding():
    import torch
    x = np.random.default_rng(2).standard_normal(4096).astype(np.float32) * 7
    assert np.array_equal(O.bf16(x), torch.from_numpy(x).to(torch.bfloat16).double().numpy())


def test_query_attention_reduces_to_attention():
    g = np.random.default_rng(4)
    q, K_, V_ = g.standard_normal((5, 3, 16)), g.standard_normal((7, 16)), g.standard_normal((7, 16))
    full, size = O.query_attention(q, K_, V_, False)
    caus, _ = O.query_attention(q, K_, V_, True)
    for i in range(5):
        assert np.allclose(full[i], O.attention(q[i], K_, V_), rtol=1e-13, atol=1e-13)
        assert np.allclose(caus[i], O.attention(q[i], K_[:3 + i], V_[:3 + i]), rtol=1e-13, atol=1e-13)
    assert np.all(size >= np.abs(full) - 1e-12)
    more, _ = O.query_attention(g.standard_normal((9, 3, 16)), K_, V_, True)  # more queries than tokens
    assert not more[:2].any() and more[2].any()


# ------------------------------------------------------------------- layout and validation

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P,G", [(16, 16), (16, 64), (64, 64), (64, 32), (256, 64), (128, 16)])
@pytest.mark.parametrize("meta", [O.F32, O.F16])
def test_block_layout_agrees_with_oracle(K, D, P, G, meta):
    for kf in (O.INT8, O.FP8_E4M3):
        for vf in (O.INT8, O.FP8_E5M2):
            cfg = O.Config(8, 2, D, O.QSpec(kf, S, BLK, G), O.QSpec(vf, S, BLK, G), 2 * G, P, meta_dtype=meta)
            c = K.kvq_config(8, 2, D, K.kvq_qspec(kf, 0, BLK, G), K.kvq_qspec(vf, 0, BLK, G), 2 * G, P, 0, 1e4, 1, meta)
            assert K.kvq_validate(c) == 0
            L = O.layout(cfg)
            assert K.kvq_page_bytes(c) == L["page"] and K.kvq_head_block_bytes(c) == L["head"]
            assert K.kvq_head_block_offsets(c) == [L["kc"], L["vc"], L["vm"], L["km"]]
            assert L["head"] % 128 == 0 and L["head"] >= 2 * P * D + 2 * max(1, P // G) * (2 if meta else 4)


def _cfg(K, **kw):
    base = dict(num_q_heads=32, num_kv_heads=8, head_dim=128, k=K.kvq_qspec(9, 0, 3, 64), v=K.kvq_qspec(9, 0, 3, 64),
                residual=64, page_size=64, rope_pre=0, rope_theta=1e4, src_dtype=1)
    base.update(kw)
    return K.kvq_config(**base)


def test_block_validation(K):
    E, U, q = K.KVQ_ERR_INVALID_ARG, K.KVQ_ERR_UNSUPPORTED, K.kvq_qspec
    ok = lambda **kw: K.kvq_validate(_cfg(K, **kw))
    assert ok() == 0 and ok(residual=128) == 0
    assert ok(k=q(8, 0, 3, 64), v=q(10, 0, 3, 64)) == 0
    assert ok(k=q(4, 0, 3, 64), v=q(4, 0, 3, 64)) == U       # 8-bit formats only
    assert ok(k=q(8, 1, 3, 64)) == U                         # symmetric only
    assert ok(v=q(9, 0, 0, 0)) == U                          # keys and values together
    assert ok(k=q(8, 0, 2, 64)) == U
    assert ok(v=q(9, 0, 3, 32)) == U                         # one group
    assert ok(k=q(9, 0, 3, 40), v=q(9, 0, 3, 40)) == E and ok(k=q(9, 0, 3, 0), v=q(9, 0, 3, 0)) == E
    assert ok(residual=0) == E and ok(residual=96) == E
    assert ok(k=q(9, 0, 3, 48), v=q(9, 0, 3, 48), residual=48) == E   # pages of 64 do not hold whole blocks
    assert ok(k=q(9, 0, 4, 64)) == E


def _cache(K, cfg, **kw):
    f = dict(pages=4096, block_table=4096, seq_lens=4096, k_win=4096, v_win=4096, k_scale=4096, v_scale=4096, batch=2,
             max_pages_per_seq=4, n_pages=8, status=4096, rope_table=None, rope_positions=0)
    f.update(kw)
    return K.kvq_cache(*[f[n] for n, _ in K.kvq_cache._fields_])


def test_rope_append_refusals(K):
    """Made-up device addresses: each call is refused before anything reads them."""
    E = K.KVQ_ERR_INVALID_ARG

    def call(cfg=None, cache=None, rope=(4096, 256, 128, 1), q=4096, k=4096, v=4096, qs=0, ks=0, vs=0, n=1, qo=8192):
        cfg = cfg or _cfg(K)
        cache = cache or _cache(K, cfg)
        r = K.kvq_rope(*rope) if rope else None
        return K.binding.LIB.kvq_rope_append(ctypes.byref(cfg), ctypes.byref(cache), ctypes.byref(r) if r else None, q, k,
                                             v, qs, ks, vs, n, None, qo, None)
    assert call(n=0) == 0
    assert call(rope=None) == E
    for rope in [(None, 256, 128, 1), (4100, 256, 128, 1), (4096, 0, 128, 1), (4096, 256, 8, 1), (4096, 256, 24, 1),
                 (4096, 256, 144, 1), (4096, 256, 128, 2)]:
        assert call(rope=rope) == E, rope
    assert call(n=-1) == E and call(n=4 * 64 + 1) == K.KVQ_ERR_CAPACITY
    assert call(k=None) == E and call(v=None) == E and call(qo=None) == E
    assert call(q=4098) == E and call(k=4104) == E and call(v=4097) == E and call(qo=8200) == E
    assert call(qs=32 * 128 - 8) == E and call(ks=8 * 128 - 8) == E and call(vs=-1024) == E  # less than a row
    assert call(qs=32 * 128 + 4) == E                                                        # not 16 bytes
    assert call(q=8192, qo=8192, qs=48 * 128) == E                                           # in place: dense only
    assert call(cfg=_cfg(K, residual=0)) == E
    assert call(cache=_cache(K, None, k_win=None)) == E and call(cache=_cache(K, None, v_win=4104)) == E
    assert call(cache=_cache(K, None, batch=0)) == E


def test_block_quantize_append_refuses_misaligned_rows(K):
    cfg = _cfg(K)
    cache = _cache(K, cfg)
    f = K.binding.LIB.kvq_quantize_append
    for k, v in ((4098, 4096), (4096, 4104)):
        assert f(ctypes.byref(cfg), ctypes.byref(cache), k, v, 1, None, None) == K.KVQ_ERR_INVALID_ARG


def test_query_attention_refusals(K):
    E = K.KVQ_ERR_INVALID_ARG

    def call(cfg=None, cache=None, q=4096, n=3, mask=1, out=8192, scale=0.0, ws=4096, nbytes=None):
        cfg = cfg or _cfg(K)
        cache = cache or _cache(K, cfg)
        if nbytes is None:
            nbytes = K.kvq_query_workspace_bytes(cfg, 2, max(n, 1))
        return K.binding.LIB.kvq_query_attention(ctypes.byref(cfg), ctypes.byref(cache), q, n, None, mask, out, scale, ws,
                                                 nbytes, None)
    assert call(n=0) == 0
    assert call(n=-1) == E and call(n=(1 << 24) + 1, nbytes=1 << 62) == K.KVQ_ERR_CAPACITY
    assert call(mask=2) == E and call(mask=-1) == E
    assert call(q=None) == E and call(out=None) == E and call(q=4098) == E and call(out=8200) == E
    assert call(scale=-1.0) == E and call(scale=float("nan")) == E and call(scale=float("inf")) == E
    W = K.KVQ_ERR_WORKSPACE
    assert call(ws=None) == W and call(ws=4096 + 16) == W
    assert call(nbytes=K.kvq_query_workspace_bytes(_cfg(K), 2, 3) - 1) == W
    assert call(cfg=_cfg(K, head_dim=96)) == K.KVQ_ERR_UNSUPPORTED
    assert call(cache=_cache(K, None, status=None)) == E
    assert K.kvq_query_workspace_bytes(_cfg(K), 0, 1) == 0 and K.kvq_query_workspace_bytes(_cfg(K), 1, 0) == 0
    assert K.kvq_query_workspace_bytes(_cfg(K, head_dim=96), 1, 1) == 0


# ------------------------------------------------------------------ the cache object's checks

def _object(K, batch=4, heads=2, D=64):
    """A cache object with what its checks of arguments read, and no device."""
    c = K.PagedKVCache.__new__(K.PagedKVCache)
    c.batch, c._D, c._H, c._Hq, c._src = batch, D, heads, 3 * heads, K.src_torch_dtype(_cfg(K))
    c._beside = lambda name, t: None
    return c


def test_broadcast_rows_are_refused(K):
    """A row stride of 0 (or below a row) would be read as dense rows, past the end of the tensor's storage."""
    import torch
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    c, one = _object(K), _object(K, batch=1)
    for obj, x in ((c, z(1, 1, 2, 64).expand(4, 1, 2, 64)),      # a decode step, one row for all sequences
                   (one, z(1, 1, 2, 64).expand(1, 9, 2, 64)),    # a prompt, one row for all tokens
                   (c, z(1, 1, 2, 64).expand(4, 9, 2, 64)),
                   (c, z(4, 1, 2, 64).expand(4, 9, 2, 64)),
                   (c, z(1, 9, 2, 64).expand(4, 9, 2, 64)),
                   (c, z(4, 9, 1, 64).expand(4, 9, 2, 64)),
                   (c, z(4, 9, 2, 1).expand(4, 9, 2, 64)),
                   (one, z(20 * 64).as_strided((1, 9, 2, 64), (9 * 64, 64, 64, 1)))):
        n = x.shape[1]
        with pytest.raises(ValueError, match="evenly spaced"):
            obj._rows("k_new", x, n, 2)
        fine = torch.zeros_like(x, memory_format=torch.contiguous_format)
        for k, v in ((x, fine), (fine, x)):
            with pytest.raises(ValueError, match="evenly spaced"):
                obj.append(k, v)
    assert c._rows("k", z(4, 9, 2, 64), 9, 2) == 128
    assert c._rows("k", z(4, 9, 8, 64)[:, :, 3:5], 9, 2) == 512
    assert c._rows("k", z(4, 1, 8, 64)[:, :, 3:5], 1, 2) == 512
    assert one._rows("k", z(1, 9, 8, 64)[:, ::3, 3:5], 3, 2) == 3 * 512
    assert one._rows("k", z(1, 1, 2, 64), 1, 2) == 128
    assert c._rows("k", z(4, 0, 8, 64)[:, :, 3:5], 0, 2) >= 0
    # kvq_quantize_append takes dense rows alone
    for k, v in ((z(4, 9, 8, 64)[:, :, :2], z(4, 9, 2, 64)), (z(4, 9, 2, 64), z(4, 9, 8, 64)[:, :, :2]),
                 (z(4, 9, 2, 64), z(4, 8, 2, 64)), (z(4, 9, 2, 64).float(), z(4, 9, 2, 64)), (z(3, 9, 2, 64), z(3, 9, 2, 64))):
        with pytest.raises(ValueError):
            c.append(k, v)


@pytest.mark.parametrize("fmt", [O.INT8, O.FP8_E4M3, O.FP8_E5M2])
@pytest.mark.parametrize("m16", [False, True])
def test_block_quantizer_of_values_that_are_not_finite(fmt, m16):
    x = np.random.default_rng(5).standard_normal((64, 64))
    spec = O.QSpec(fmt, S, BLK, 16)
    want, ws, _ = O._quant_block(x, spec, m16)
    for bad in (np.nan, np.inf, -np.inf):
        y = x.copy()
        y[20, 3], y[63, 63] = bad, bad
        c, s, _ = O._quant_block(y, spec, m16)
        assert np.isnan(s).tolist() == [False, True, False, True] and s[0] == ws[0] and s[2] == ws[2]
        assert not c[16:32].any() and not c[48:].any()
        assert np.array_equal(c[:16], want[:16]) and np.array_equal(c[32:48], want[32:48])
        assert np.isnan(O._dequant_block(c, s, spec)).reshape(4, -1).all(1).tolist() == [False, True, False, True]


@pytest.mark.parametrize("batch", [1, 3, 64, 600])
@pytest.mark.parametrize("D,Hq,H", [(128, 32, 8), (64, 16, 16), (256, 8, 2), (128, 7, 1), (128, 64, 1)])
def test_workspace_of_more_queries_serves_fewer(K, D, Hq, H, batch):
    """The size is for calls of at most n_q queries, whichever kernel they take."""
    cfg = _cfg(K, num_q_heads=Hq, num_kv_heads=H, head_dim=D)
    sizes = [K.kvq_query_workspace_bytes(cfg, batch, n) for n in list(range(1, 300)) + [1000, 10000, 1 << 20]]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_tables_and_buffers_off_the_device_are_refused(K):
    """Host memory never reaches a kernel: the rotation's table, and the buffers of a cache."""
    import torch
    c = _object(K)
    del c._beside
    c._index, c._device = 0, torch.device("cuda:0")
    k = torch.zeros(4, 1, 2, 64, dtype=torch.bfloat16)
    rope = K.make_rope(torch.zeros(32, 64), 64)
    with pytest.raises(ValueError, match="cos_sin must be on the cache's device"):
        c.append_rope(rope, None, k, k)
    cfg = _cfg(K)
    buffers = dict(pages=torch.zeros(K.kvq_page_bytes(cfg), dtype=torch.uint8), block_table=torch.zeros(1, 1, dtype=torch.int32),
                   seq_lens=torch.zeros(1, dtype=torch.int32))
    buffers["k_win"], buffers["v_win"] = (torch.zeros(1, 64, 8, 128, dtype=torch.bfloat16) for _ in range(2))
    with pytest.raises(ValueError, match="CUDA"):
        K.PagedKVCache.over(cfg, **buffers)


def test_broadcast_block_table_is_laid_out(K):
    """A table that is a broadcast view (all sequences over the same pages) is copied to whole rows."""
    import torch
    spec = (K.KVQ_FP8_E4M3, 0, K.KVQ_PER_BLOCK, 64)
    cfg = K.make_config(8, 2, 64, spec, spec, 64, 64, src_dtype=K.KVQ_BF16)
    table = torch.tensor([[1, 0, 2]], dtype=torch.int32).expand(4, 3)
    c = K.PagedKVCache(cfg, 4, 3, n_pages=3, block_table=table, device="cpu")
    assert c.block_table.is_contiguous() and c.block_table.tolist() == [[1, 0, 2]] * 4


@pytest.mark.parametrize("D,Hq,H,batch", [(128, 16, 1, 1), (128, 9, 1, 1), (128, 64, 8, 200), (256, 8, 1, 1), (256, 32, 2, 300),
                                          (128, 128, 1, 64), (64, 64, 8, 1000), (256, 128, 8, 20)])
def test_decode_workspaces_fit_the_library_s_own(K, D, Hq, H, batch):
    """kvq_decode_attention_noalloc takes wide groups: their calls are cut into fewer runs."""
    cfg = _cfg(K, num_q_heads=Hq, num_kv_heads=H, head_dim=D)
    assert 0 < K.kvq_workspace_bytes(cfg, batch, 4096) <= K.KVQ_NOALLOC_SCRATCH_BYTES
