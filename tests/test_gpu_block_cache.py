"""Block-scaled 8-bit caches, rotated append and query attention on the GPU against the
oracle.  Bit-exact: page bytes, windows, lengths, rotated queries, kvq_dequantize.
Attention: against 64 bits on the dequantized cache, element by element.

Tolerance of an output x (bf16 sources): the final rounding is off by at most
2^-8 |x|.  The weights enter the tensor cores in f16, each off by at most 2^-11 of
itself, so the sum by 2^-11 A with A = sum p |v| / sum p; a weight below 2^-14, a
subnormal f16, is off by at most 2^-25 instead, in units in which the running maximum's
weight is 1 and the sum of the weights therefore at least 1: together at most 2^-25
sum |v| over the tokens (a channel whose heavier tokens hold zeros has no larger term).
The logits are fp32 sums of exact products, off
by under 2^-22 sum |q k| scale, which for these streams (sum |q k| scale < 2^10) is
2^-12 relative on a weight, at most 2^-11 A on the output after normalisation.
fp32 sources (plain kernel): the final rounding 2^-24 |x|, the logits' fp32 sum of D
products (at most D 2^-24 sum |q k| scale, under 2^-9 on a weight for the outlier
channels here; measured sums err far less), so 2^-10 A covers both.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import kvq_oracle as O  # noqa: E402

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from kvq_testlib import Case, torch_src  # noqa: E402

S, BLK = O.SYM, O.PER_BLOCK
I8, E4, E5 = O.INT8, O.FP8_E4M3, O.FP8_E5M2


def cfg_of(Hq, H, D, kf, vf, G, R, P, **kw):
    return O.Config(Hq, H, D, O.QSpec(kf, S, BLK, G), O.QSpec(vf, S, BLK, G), R, P, 0, 1e4, kw.pop("src", O.BF16), **kw)


# name: (config, sequence lengths)
CASES = {
    "e4m3_p64": (cfg_of(32, 8, 128, E4, E4, 64, 64, 64), [0, 1, 63, 64, 65, 300, 1000]),
    "int8_p16": (cfg_of(8, 2, 128, I8, I8, 64, 64, 16), [1, 64, 130, 700, 2100]),
    "e5m2_p256": (cfg_of(16, 2, 128, E5, E5, 64, 128, 256), [127, 128, 129, 900]),
    "mixed_formats": (cfg_of(8, 2, 128, E4, I8, 32, 64, 64), [5, 64, 333]),
    "g16_p16": (cfg_of(4, 4, 128, I8, I8, 16, 16, 16), [3, 16, 17, 250]),
    "g128_p32": (cfg_of(8, 1, 128, E4, E4, 128, 256, 32), [255, 256, 700]),
    "d64": (cfg_of(16, 16, 64, E4, E4, 64, 64, 64), [5, 64, 200, 1500]),
    "d64_int8_nrep4": (cfg_of(8, 2, 64, I8, I8, 32, 64, 16), [1, 31, 64, 500]),
    "d256": (cfg_of(8, 2, 256, E4, E4, 64, 64, 64), [7, 64, 260]),
    "d256_int8": (cfg_of(4, 4, 256, I8, I8, 32, 32, 32), [32, 100]),
    "nrep7": (cfg_of(14, 2, 128, E4, E4, 64, 64, 64), [65, 400]),
    "nrep16": (cfg_of(16, 1, 128, I8, I8, 64, 64, 64), [65, 400]),
    "nrep40": (cfg_of(40, 1, 64, E5, E5, 64, 64, 64), [100, 64]),
    "meta16": (cfg_of(8, 2, 128, E4, E4, 64, 64, 64, meta_dtype=O.F16), [1, 64, 300]),
    "meta16_int8_p16": (cfg_of(8, 8, 64, I8, I8, 32, 32, 16, meta_dtype=O.F16), [40, 33, 0]),
    "f32": (cfg_of(8, 2, 128, E4, E4, 64, 64, 64, src=O.F32), [1, 64, 130]),
    "f32_int8_d64": (cfg_of(4, 4, 64, I8, I8, 16, 48, 16, src=O.F32), [47, 48, 100]),
    "p48_g16": (cfg_of(8, 2, 128, E4, E4, 16, 48, 48), [47, 48, 49, 500]),     # pages that end inside a tile
    "p80_g16_d64": (cfg_of(12, 4, 64, I8, I8, 16, 32, 80), [79, 80, 161, 640]),
    "p48_g48": (cfg_of(8, 2, 128, I8, I8, 48, 96, 48), [95, 96, 300]),         # blocks that end inside a tile
    "p96_g48_d64": (cfg_of(4, 4, 64, E5, E5, 48, 48, 96), [100, 480]),
    "group_512": (cfg_of(8, 2, 128, I8, I8, 512, 512, 64), [511, 512, 1300]),  # more than registers hold
}


@pytest.fixture(scope="module", params=sorted(CASES))
def case(request):
    cfg, lens = CASES[request.param]
    c = Case(cfg, lens, seed=100 + sorted(CASES).index(request.param))
    c.name = request.param
    return c


def test_pages_bit_exact(case):
    case.check_pages()


def test_lengths_and_window(case):
    case.check_lengths_and_window()


def test_dequantize_bit_exact(case):
    case.check_dequantize()


def test_decode_attention(case):
    import asymmetric_quantized_kv_gb300 as K
    assert case.cache.decode_kernel() == K.KVQ_KERNEL_BLOCK8
    case.check_attention()
    case.check_attention(scale=0.05)


def check_queries(case, n, causal, per_seq=None, scale=0.0, seed=7, q=None):
    """kvq_query_attention of n queries a sequence against the oracle; rows past a sequence's count keep
    what they held."""
    cfg = case.cfg
    Bn, D = len(case.lens), cfg.head_dim
    g = np.random.default_rng(seed)
    if q is None:
        q = g.standard_normal((Bn, n, cfg.num_q_heads, D)).astype(np.float32)
        q = O.bf16(q).astype(np.float32) if cfg.src_dtype == O.BF16 else q
    counts = [n] * Bn if per_seq is None else list(per_seq)
    tq = torch_src(q, cfg)
    for b, c in enumerate(counts):  # rows that are not to be read
        tq[b, c:] = float("nan")
    out = torch.full_like(tq, 7.25)
    per = None if per_seq is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    case.cache.query_attention(tq, causal=causal, n_q_per_seq=per, out=out, softmax_scale=scale)
    got = out.double().cpu().numpy()
    half = 2.0 ** -8 if cfg.src_dtype == O.BF16 else 2.0 ** -24
    worst = 0.0
    for b in range(Bn):
        assert np.all(got[b, counts[b]:] == 7.25)
        for h in range(cfg.num_kv_heads):
            Kd, Vd = O.dequantize_stream(cfg, case.states[b][h], case.k_scale[h], case.v_scale[h])
            if cfg.rope_pre:
                Kd = O.rope(Kd, np.arange(Kd.shape[0]), cfg.rope_theta)
            heads = slice(h * cfg.n_rep, (h + 1) * cfg.n_rep)
            ref, size = O.query_attention(q[b, :counts[b], heads].astype(np.float64), Kd, Vd, causal, scale or None)
            err = np.abs(got[b, :counts[b], heads] - ref)
            lim = half * np.abs(ref) + 2.0 ** -10 * size + 2.0 ** -25 * np.abs(Vd).sum(0)
            assert np.all(err <= lim), (case.name, b, h, float((err - lim).max()))
            worst = max(worst, float(np.max(err / np.maximum(size, 1e-30), initial=0)))
    assert int(case.cache.status.item()) == 0
    return worst


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [1, 2, 5, 33])
def test_query_attention(case, n, causal):
    check_queries(case, n, causal)


def test_query_attention_ragged_counts(case):
    Bn = len(case.lens)
    check_queries(case, 9, True, [(3 * b) % 10 for b in range(Bn)])
    check_queries(case, 9, False, [9 - (4 * b) % 10 for b in range(Bn)], scale=0.03)


@pytest.mark.parametrize("name,n", [("e4m3_p64", 129), ("int8_p16", 300), ("d64", 257), ("nrep40", 64), ("nrep7", 100)])
def test_query_attention_many_rows(name, n):
    """Several row tiles, cut ones among them; more queries than some sequences have tokens."""
    cfg, lens = CASES[name]
    c = Case(cfg, lens, seed=3)
    c.name = name
    check_queries(c, n, True)
    check_queries(c, n, False, [n - 17 * (b % 3) for b in range(len(lens))])


# ------------------------------------------------------------------------ other caches

OTHER = {
    "rope_pre_i8i4": (O.Config(32, 8, 128, O.QSpec(O.INT8, S, O.PER_CHANNEL, 64), O.QSpec(O.INT4, O.ASYM, O.PER_TOKEN, 0),
                               64, 16, 1, 5e5, O.BF16), [1, 64, 200]),
    "kivi2": (O.Config(8, 2, 128, O.QSpec(O.INT2, O.ASYM, O.PER_CHANNEL, 32), O.QSpec(O.INT2, O.ASYM, O.PER_TOKEN, 32),
                       128, 64, 0, 1e4, O.BF16), [5, 128, 300]),
    "fp8_static": (O.Config(16, 2, 128, O.QSpec(E4, S, O.PER_TENSOR), O.QSpec(E4, S, O.PER_TENSOR), 0, 16, 0, 1e4, O.F32),
                   [1, 17, 130]),
    "int8_token_d256": (O.Config(2, 2, 256, O.QSpec(I8, S, O.PER_TOKEN, 64), O.QSpec(I8, O.ASYM, O.PER_TOKEN, 128), 32, 32,
                                 0, 1e4, O.BF16, meta_dtype=O.F16), [31, 32, 90]),
    "int4_channel_r512": (O.Config(8, 1, 64, O.QSpec(O.INT4, O.ASYM, O.PER_CHANNEL, 512),
                                   O.QSpec(O.INT4, O.ASYM, O.PER_TOKEN, 0), 512, 512, 0, 1e4, O.F32), [512, 700]),
    "block_rope_pre": (O.Config(8, 2, 128, O.QSpec(E4, S, BLK, 64), O.QSpec(E4, S, BLK, 64), 64, 64, 1, 1e4, O.BF16),
                       [1, 64, 200]),
}


@pytest.mark.parametrize("name", sorted(OTHER))
def test_query_attention_of_every_axis(name):
    cfg, lens = OTHER[name]
    c = Case(cfg, lens, seed=11)
    c.name = name
    for n, causal in ((1, True), (3, True), (4, False)):
        check_queries(c, n, causal)


# ------------------------------------------------------------------------ rotated append

def rope_setup(positions, rot, theta=1e4):
    ang = np.arange(positions)[:, None] * theta ** (-2 * np.arange(rot // 2) / rot)
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    return table, torch.from_numpy(table).cuda()


def rotated_case(cfg, lens, rot, halves, chunks, seed=0, fused=True, positions=None):
    """Fill an empty cache through append_rope in the given chunk sizes; returns a Case-like object
    whose oracle streams hold the oracle's rotated keys."""
    import asymmetric_quantized_kv_gb300 as K
    Bn, H, Hq, D = len(lens), cfg.num_kv_heads, cfg.num_q_heads, cfg.head_dim
    c = Case.__new__(Case)
    base = Case(cfg, [0] * Bn, seed=seed, extra_pages=-(-max(max(lens), max(chunks)) // cfg.page_size) + 1)
    c.__dict__.update(base.__dict__)
    c.lens, c.name = list(lens), "rotated"
    g = np.random.default_rng(seed)
    rnd = (lambda x: O.bf16(x)) if cfg.src_dtype == O.BF16 else (lambda x: O.fl32(x))
    x = rnd(g.standard_normal((Bn, max(lens), Hq + 2 * H, D))).astype(np.float32)
    x[:, :, Hq:Hq + H, 3::29] *= 8
    table, tt = rope_setup(positions or c.maxp * cfg.page_size, rot)
    rope = K.make_rope(tt, rot, K.KVQ_ROPE_HALVES if halves else K.KVQ_ROPE_INTERLEAVED)
    if O.is_fp8(cfg.k.fmt) and cfg.k.axis == O.PER_TENSOR:
        c.k_scale, c.v_scale = [0.25] * H, [0.125] * H
        c.cache.k_scale.fill_(0.25)
        c.cache.v_scale.fill_(0.125)
    done, qs = [0] * Bn, []
    step = 0
    while any(done[b] < lens[b] for b in range(Bn)):
        n = chunks[step % len(chunks)]
        step += 1
        take = [min(n - (b % 2 if n > 2 else 0), lens[b] - done[b]) for b in range(Bn)]
        rows = np.zeros((Bn, n, Hq + 2 * H, D), np.float32)
        for b in range(Bn):
            rows[b, :take[b]] = x[b, done[b]:done[b] + take[b]]
        t = torch_src(rows, cfg)
        for b in range(Bn):
            t[b, take[b]:] = float("nan")  # rows past a sequence's count are not read
        q, k, v = t[:, :, :Hq], t[:, :, Hq:Hq + H], t[:, :, Hq + H:]
        if not fused:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        out = torch.full((Bn, n, Hq, D), 3.5, dtype=t.dtype, device="cuda")
        c.cache.append_rope(rope, q, k, v, torch.tensor(take, dtype=torch.int32, device="cuda"), q_out=out)
        got = out.double().cpu().numpy()
        for b in range(Bn):
            assert np.all(got[b, take[b]:] == 3.5)
            pos = np.arange(done[b], done[b] + take[b])
            for h in range(Hq):
                want = O.rope_rows(rows[b, :take[b], h], pos, table, rot, halves, cfg.src_dtype)
                assert np.array_equal(got[b, :take[b], h], want), (b, h, step)
            done[b] += take[b]
    torch.cuda.synchronize()
    assert int(c.cache.status.item()) == 0
    c.K = [[(x[b, :lens[b], Hq + h].astype(np.float64) if cfg.rope_pre else
             O.rope_rows(x[b, :lens[b], Hq + h], np.arange(lens[b]), table, rot, halves, cfg.src_dtype))
            for h in range(H)] for b in range(Bn)]
    c.V = [[x[b, :lens[b], Hq + H + h].astype(np.float64) for h in range(H)] for b in range(Bn)]
    c.states = [[O.quantize_stream(cfg, c.K[b][h], c.V[b][h], c.k_scale[h], c.v_scale[h]) for h in range(H)]
                for b in range(Bn)]
    return c


ROT = {  # name: (config, rot, halves, chunk sizes)
    "one_by_one": (cfg_of(4, 2, 128, E4, E4, 32, 32, 16), 128, True, [1]),
    "steps_and_prompts": (cfg_of(8, 2, 128, I8, I8, 64, 64, 64), 128, False, [3, 50, 1, 200]),
    "prompt": (cfg_of(8, 2, 128, E4, E4, 64, 128, 64), 64, True, [400]),
    "small_steps_d64": (cfg_of(6, 3, 64, E5, E5, 16, 32, 16), 16, True, [7, 16, 17]),
    "d256": (cfg_of(4, 2, 256, I8, E4, 32, 64, 64), 256, False, [5, 90]),
    "one_head": (cfg_of(3, 1, 128, E4, E4, 64, 64, 256), 96, False, [2, 70]),
    "many_heads": (cfg_of(24, 12, 64, E4, E4, 64, 64, 64), 64, True, [1, 66]),
    "f32": (cfg_of(4, 2, 128, E4, E4, 32, 64, 32, src=O.F32), 128, True, [4, 40, 1]),
    "p48_g16": (cfg_of(8, 2, 128, E4, E4, 16, 48, 48), 128, True, [40, 1, 90]),
    "p48_g48": (cfg_of(4, 2, 128, I8, I8, 48, 96, 48), 32, False, [3, 100]),
    "meta16": (cfg_of(4, 2, 128, I8, I8, 32, 64, 32, meta_dtype=O.F16), 32, False, [1, 33]),
    "group_512": (cfg_of(4, 2, 128, I8, I8, 512, 512, 64), 128, True, [300]),
    "other_kivi2": (OTHER["kivi2"][0], 128, True, [1, 100, 30]),
    "other_fp8_static": (OTHER["fp8_static"][0], 64, False, [1, 70]),
    "other_r512": (OTHER["int4_channel_r512"][0], 64, True, [600]),
    "other_token_d256": (OTHER["int8_token_d256"][0], 256, True, [9, 40]),
    "rope_pre": (OTHER["rope_pre_i8i4"][0], 128, False, [1, 90]),
    "block_rope_pre": (OTHER["block_rope_pre"][0], 128, False, [1, 90]),
}


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("name", sorted(ROT))
def test_rope_append_bit_exact(name, fused):
    cfg, rot, halves, chunks = ROT[name]
    big = cfg.residual >= 512
    lens = [600, 520] if big else ([70, 33, 1] if name == "one_by_one" else [200, 131, 64, 1])
    c = rotated_case(cfg, lens, rot, halves, chunks, seed=len(name), fused=fused)
    c.check_pages()
    c.check_lengths_and_window()
    c.check_dequantize()


def test_rotation_in_place_and_without_queries():
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(8, 2, 128, E4, E4, 64, 64, 64)
    table, tt = rope_setup(256, 128)
    rope = K.make_rope(tt, 128, K.KVQ_ROPE_HALVES)
    for n in (3, 40):
        a, b = (Case(cfg, [0, 0], seed=1, extra_pages=3).cache for _ in range(2))
        g = torch.Generator(device="cuda").manual_seed(n)
        q = torch.randn(2, n, 8, 128, generator=g, device="cuda").bfloat16()
        k, v = (torch.randn(2, n, 2, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
        want = a.append_rope(rope, q, k, v)
        mine = q.clone()
        assert b.append_rope(rope, mine, k, v, q_out=mine) is mine
        assert torch.equal(mine, want)
        assert b.append_rope(rope, None, k, v) is None
        a.append_rope(rope, None, k, v)
        assert torch.equal(a.pages, b.pages) and torch.equal(a.k_win, b.k_win) and a.seq_lens.tolist() == [2 * n] * 2


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("axis", ["block", "other"])
def test_rope_append_that_does_not_fit(n, axis):
    """A sequence that would pass its pages, or the table, is left as it was and reported."""
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(4, 2, 128, E4, E4, 32, 32, 16) if axis == "block" else O.Config(
        4, 2, 128, O.QSpec(I8, S, O.PER_CHANNEL, 32), O.QSpec(I8, S, O.PER_TOKEN, 0), 32, 32, 0, 1e4, O.BF16)
    for positions, full in ((512, 1), (90, 0)):
        c = Case(cfg, [10, 60], seed=2, extra_pages=0)   # 64 tokens fit
        if full == 0:
            c = Case(cfg, [10, 60], seed=2, extra_pages=10)
        start = [10, 64 - n + 1] if full else [10, 90 - n + 1]
        c.cache.seq_lens.copy_(torch.tensor(start, dtype=torch.int32))
        _, tt = rope_setup(positions, 128)
        rope = K.make_rope(tt, 128)
        pages, win = c.cache.pages.clone(), c.cache.k_win.clone()
        q = torch.randn(2, n, 4, 128, device="cuda").bfloat16()
        k, v = (torch.randn(2, n, 2, 128, device="cuda").bfloat16() for _ in range(2))
        out = torch.full_like(q, 2.0)
        c.cache.append_rope(rope, q, k, v, q_out=out)
        assert int(c.cache.status.item()) == K.KVQ_DEV_OVERFLOW
        assert c.cache.seq_lens.tolist() == [10 + n, start[1]]
        assert torch.equal(c.cache.k_win[1], win[1]) and bool((out[1] == 2.0).all())
        own = c.cache.page_view()[c.block_table[1]]
        assert torch.equal(own, pages.view_as(c.cache.page_view())[c.block_table[1]])


# ------------------------------------------------------------------------ used together

def test_prompt_drafts_and_steps_together():
    """A prompt in two chunks, drafted tokens, a rejected draft (the lengths set back), single steps:
    each append followed by its attention, against the oracle."""
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(8, 2, 128, E4, E4, 32, 64, 32)
    Bn, H, Hq, D = 2, 2, 8, 128
    table, tt = rope_setup(512, D)
    rope = K.make_rope(tt, D, K.KVQ_ROPE_HALVES)
    cache = Case(cfg, [0] * Bn, seed=1, extra_pages=12).cache
    g = np.random.default_rng(8)
    Ks, Vs = [np.zeros((0, H, D))] * Bn, [np.zeros((0, H, D))] * Bn
    for n, keep in ((100, 100), (37, 37), (5, 3), (1, 1), (5, 5), (1, 1), (50, 50), (1, 1)):
        x = O.bf16(g.standard_normal((Bn, n, Hq + 2 * H, D))).astype(np.float32)
        t = torch_src(x, cfg)
        q = cache.append_rope(rope, t[:, :, :Hq], t[:, :, Hq:Hq + H], t[:, :, Hq + H:])
        out = cache.query_attention(q).double().cpu().numpy()
        T0 = Ks[0].shape[0]
        pos = np.arange(T0, T0 + n)
        rot = lambda y: O.rope_rows(y, pos, table, D, True, O.BF16)
        for b in range(Bn):
            Ks[b] = np.concatenate([Ks[b], np.stack([rot(x[b, :, Hq + h]) for h in range(H)], 1)])
            Vs[b] = np.concatenate([Vs[b], x[b, :, Hq + H:].astype(np.float64)])
            for h in range(H):
                st = O.quantize_stream(cfg, Ks[b][:, h], Vs[b][:, h])
                Kd, Vd = O.dequantize_stream(cfg, st)
                qq = np.stack([rot(x[b, :, r]) for r in range(4 * h, 4 * h + 4)], 1)
                ref, size = O.query_attention(qq, Kd, Vd, True)
                err = np.abs(out[b, :, 4 * h:4 * h + 4] - ref)
                lim = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * size + 2.0 ** -25 * np.abs(Vd).sum(0)
                assert np.all(err <= lim), (n, b, h)
        if keep < n:  # no window filled since, so its rows are all still there
            assert T0 // 64 == (T0 + n) // 64
            cache.seq_lens.sub_(n - keep)
            Ks, Vs = [y[:T0 + keep] for y in Ks], [y[:T0 + keep] for y in Vs]
    assert int(cache.status.item()) == 0


def test_cross_attention_of_two_batches_over_shared_pages():
    """Two decoder batches over one encoder cache, whose block table names the same pages twice."""
    import asymmetric_quantized_kv_gb300 as K
    cfg, _ = CASES["d64"]
    c = Case(cfg, [192, 128], seed=4)   # whole windows: everything is in the pages
    twice = K.PagedKVCache.over(c.c_cfg, c.cache.pages, c.cache.block_table.repeat(2, 1), c.cache.seq_lens.repeat(2),
                                c.cache.k_win.repeat(2, 1, 1, 1), c.cache.v_win.repeat(2, 1, 1, 1))
    q = torch.randn(4, 21, 16, 64, device="cuda").bfloat16()
    both = twice.query_attention(q, causal=False)
    assert torch.equal(both[:2], c.cache.query_attention(q[:2].contiguous(), causal=False))
    assert torch.equal(both[2:], c.cache.query_attention(q[2:].contiguous(), causal=False))


@pytest.mark.parametrize("n", [1, 3, 40])
def test_graph_replays_step_by_step(n):
    """Append and attention captured once and replayed advance the cache as eager calls do, bit for bit."""
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(8, 2, 128, E4, E4, 32, 32, 32)
    _, tt = rope_setup(512, 128)
    rope = K.make_rope(tt, 128)
    eager, graph, warm = (Case(cfg, [30, 7], seed=6, extra_pages=8).cache for _ in range(3))
    x = torch.randn(2, n, 12, 128, device="cuda").bfloat16()
    qo, out = torch.empty(2, n, 8, 128, device="cuda").bfloat16(), torch.empty(2, n, 8, 128, device="cuda").bfloat16()

    def step(cache, qo, out):
        cache.append_rope(rope, x[:, :, :8], x[:, :, 8:10], x[:, :, 10:], q_out=qo)
        cache.query_attention(qo, out=out)
    step(warm, qo.clone(), out.clone())
    graph.query_attention(qo.zero_(), out=out)  # its workspace, before the capture
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step(graph, qo, out)
    for i in range(4):
        x.copy_(torch.randn(2, n, 12, 128, device="cuda"))
        gr.replay()
        qe, oe = torch.empty_like(qo), torch.empty_like(out)
        step(eager, qe, oe)
        assert torch.equal(qe, qo) and torch.equal(oe, out), i
        assert torch.equal(eager.pages, graph.pages) and torch.equal(eager.seq_lens, graph.seq_lens)
    assert int(graph.status.item()) == 0


def test_bad_counts_and_pages():
    """Counts outside [0, n] and block-table entries outside the pool are reported, never followed."""
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(8, 2, 128, E4, E4, 64, 64, 64)
    for n in (2, 40):
        c = Case(cfg, [300, 300, 300], seed=9)
        q = torch.randn(3, n, 8, 128, device="cuda").bfloat16()
        want = c.cache.query_attention(q)
        out = torch.full_like(q, 5.0)
        c.cache.query_attention(q, n_q_per_seq=torch.tensor([n, -1, n + 1], dtype=torch.int32, device="cuda"), out=out)
        assert int(c.cache.status.item()) == K.KVQ_DEV_BAD_LENGTH
        assert torch.equal(out[0], want[0]) and bool((out[1:] == 5.0).all())
        c.cache.status.zero_()
        c.cache.block_table[1, 1] = 1 << 20
        c.cache.block_table[2, 2] = -5
        got = c.cache.query_attention(q)
        assert int(c.cache.status.item()) == K.KVQ_DEV_BAD_PAGE
        assert torch.equal(got[0], want[0]) and bool(torch.isfinite(got).all())


def test_binding_refusals():
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(8, 2, 128, E4, E4, 64, 64, 64)
    c = Case(cfg, [10, 20], seed=1).cache
    q = torch.zeros(2, 3, 8, 128, device="cuda").bfloat16()
    kv = torch.zeros(2, 3, 2, 128, device="cuda").bfloat16()
    rope = K.make_rope(rope_setup(256, 128)[1], 128)
    bad = [lambda: c.query_attention(q.float()), lambda: c.query_attention(q[:1]), lambda: c.query_attention(q[:, :, :4]),
           lambda: c.query_attention(q.transpose(0, 1).contiguous().transpose(0, 1)), lambda: c.query_attention(q.cpu()),
           lambda: c.query_attention(q, out=q.float()),
           lambda: c.query_attention(q, n_q_per_seq=torch.zeros(2, dtype=torch.int64, device="cuda")),
           lambda: c.append_rope(rope, q, kv[:, :2], kv), lambda: c.append_rope(rope, q.float(), kv, kv),
           lambda: c.append_rope(rope, q, kv.transpose(0, 1).contiguous().transpose(0, 1), kv),
           lambda: c.append_rope(rope, q, kv, kv, q_out=q.float()),
           lambda: c.append_rope(rope, q, kv, kv, torch.zeros(3, dtype=torch.int32, device="cuda")),
           lambda: K.make_rope(torch.zeros(8, 64, device="cuda"), 128),
           lambda: K.PagedKVCache.over(c.cfg, c.pages[:-1], c.block_table, c.seq_lens, c.k_win, c.v_win),
           lambda: K.PagedKVCache.over(c.cfg, c.pages, c.block_table, c.seq_lens, None, c.v_win),
           lambda: K.PagedKVCache.over(c.cfg, c.pages, c.block_table.long(), c.seq_lens, c.k_win, c.v_win)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("not refused:", i)
    assert c.seq_lens.tolist() == [10, 20]


# --------------------------------------------------------------- what must not be read, or lies far

SOILED = ["e4m3_p64", "int8_p16", "e5m2_p256", "d64", "nrep16", "d256", "f32", "p48_g16"]


@pytest.mark.parametrize("name", SOILED)
def test_what_lies_behind_a_sequence_is_not_read(name):
    """NaN bytes in unused pages and slots, NaN and infinities in unused window rows, page ids of no page behind
    each sequence's last: the outputs are those of a clean cache, bit for bit, in every kernel."""
    cfg, lens = CASES[name]
    c = Case(cfg, lens, seed=21)
    c.name = name
    n_pages, P = c.cache.n_pages, cfg.page_size
    calls = [(1, True), (5, True), (5, False), (48, True), (48, False)]
    q = {n: torch_src(O.bf16(np.random.default_rng(n).standard_normal((len(lens), n, cfg.num_q_heads, cfg.head_dim))), cfg)
         for n in (1, 5, 48)}
    clean = [c.cache.query_attention(q[n], causal=k) for n, k in calls] + [c.cache.attention(q[1][:, 0].contiguous())]
    pages, defined = c.oracle_pages()
    soiled = c.cache.page_view().cpu().numpy().copy()
    soiled[~defined] = 0xFF
    c.cache.page_view().copy_(torch.from_numpy(soiled))
    for b, T in enumerate(lens):
        r = T % cfg.residual
        c.cache.k_win[b, r:] = float("nan")
        c.cache.v_win[b, r:] = float("inf")
        used = -(-(T - r) // P)
        c.cache.block_table[b, used:] = torch.tensor([n_pages + 7, -3] * c.maxp, dtype=torch.int32)[:c.maxp - used].cuda()
    again = [c.cache.query_attention(q[n], causal=k) for n, k in calls] + [c.cache.attention(q[1][:, 0].contiguous())]
    for (n, k), a, b in zip(calls + [("decode", 0)], clean, again):
        assert torch.equal(a, b), (n, k)
    assert int(c.cache.status.item()) == 0


def test_pool_beyond_four_gigabytes():
    """The same cache at the start of a small pool and at the end of one of 5 GB."""
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(16, 4, 128, E4, E4, 64, 64, 64)
    _, tt = rope_setup(1024, 128)
    rope = K.make_rope(tt, 128, K.KVQ_ROPE_HALVES)
    small = Case(cfg, [0, 0], seed=1, extra_pages=12, permute_pages=False).cache
    n_pages = 5 * (1 << 30) // small.page_bytes
    far = K.PagedKVCache.over(small.cfg, torch.empty(n_pages * small.page_bytes, dtype=torch.uint8, device="cuda"),
                              small.block_table + (n_pages - small.n_pages), small.seq_lens.clone(), small.k_win.clone(),
                              small.v_win.clone())
    for n in (400, 1, 60, 1):
        x = torch.randn(2, n, 24, 128, device="cuda").bfloat16()
        outs = []
        for cache in (small, far):
            q = cache.append_rope(rope, x[:, :, :16], x[:, :, 16:20], x[:, :, 20:])
            outs.append((q, cache.query_attention(q), cache.query_attention(q[:, :1].contiguous(), causal=False),
                         cache.attention(q[:, 0].contiguous())))
        assert all(torch.equal(a, b) for a, b in zip(*outs)), n
        assert bool(torch.isfinite(outs[1][1]).all())
    used = far.page_view()[n_pages - small.n_pages:]
    nq = 462 // 64 * 64
    for b in range(2):
        rows = small.block_table[b, :nq // 64].long()
        assert torch.equal(used[rows], small.page_view()[rows])
    assert int(small.status.item()) == 0 and int(far.status.item()) == 0


def test_another_stream():
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(8, 2, 128, E4, E4, 64, 64, 64)
    _, tt = rope_setup(512, 128)
    rope = K.make_rope(tt, 128)
    a, b = (Case(cfg, [100, 70], seed=6, extra_pages=4).cache for _ in range(2))
    x = torch.randn(2, 70, 12, 128, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qa = a.append_rope(rope, x[:, :, :8], x[:, :, 8:10], x[:, :, 10:])
    oa = a.query_attention(qa)
    qb, ob = torch.empty_like(qa), torch.empty_like(oa)
    b.append_rope(rope, x[:, :, :8], x[:, :, 8:10], x[:, :, 10:], q_out=qb, stream=side)
    b.query_attention(qb, out=ob, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(qa, qb) and torch.equal(oa, ob) and torch.equal(a.pages, b.pages)


def test_decode_without_a_workspace():
    import asymmetric_quantized_kv_gb300 as K
    cfg, lens = CASES["int8_p16"]
    c = Case(cfg, lens, seed=3)
    q = torch_src(c.queries(), cfg)
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    K.kvq_decode_attention_noalloc(c.c_cfg, c.cache.c, q, out, 0.0)
    assert torch.equal(out, c.cache.attention(q))


def test_append_to_a_missing_page():
    """Rows and scales of a block-table entry outside the pool are not written anywhere; the rest is."""
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(8, 2, 128, E4, E4, 32, 64, 32)
    for n in (1, 130):
        c = Case(cfg, [127, 127], seed=5, extra_pages=8)
        good = Case(cfg, [127, 127], seed=5, extra_pages=8)
        c.cache.block_table[1, 3] = c.cache.n_pages + 5   # tokens 96 .. 127
        k, v = (torch.randn(2, n, 2, 128, device="cuda").bfloat16() for _ in range(2))
        for x in (c, good):
            x.cache.append(k, v)
        assert int(c.cache.status.item()) == K.KVQ_DEV_BAD_PAGE
        assert c.cache.seq_lens.tolist() == [127 + n] * 2
        keep = torch.ones(c.cache.n_pages, dtype=torch.bool)
        keep[int(c.block_table[1, 3])] = False
        assert torch.equal(c.cache.page_view()[keep.cuda()], good.cache.page_view()[keep.cuda()])
        assert torch.equal(c.cache.k_win, good.cache.k_win)


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -20, 2.0 ** 30, 2.0 ** 90])
def test_values_of_any_magnitude(scale):
    """Value blocks whose scales differ by far, and all of them far from 1: the weights carry the scale's exponent."""
    cfg = cfg_of(8, 2, 128, E4, E4, 64, 64, 64)
    g = np.random.default_rng(4)
    lens = [300, 200]
    Ks = [[O.bf16(g.standard_normal((T, 128))) for _ in range(2)] for T in lens]
    Vs = [[O.bf16(g.standard_normal((T, 128)) * scale * np.where((np.arange(T) // 64) % 2, 2.0 ** -12, 1.0)[:, None])
           for _ in range(2)] for T in lens]
    c = Case(cfg, lens, seed=1, streams=(Ks, Vs))
    c.name = "magnitude"
    for n in (1, 7, 40):
        check_queries(c, n, True)
        check_queries(c, n, False)
    c.check_attention()


def test_zero_keys_values_and_queries():
    cfg = cfg_of(8, 2, 128, E4, E4, 64, 64, 64)
    z = [[np.zeros((T, 128)) for _ in range(2)] for T in (130, 64)]
    c = Case(cfg, [130, 64], seed=1, streams=(z, z))
    c.name = "zeros"
    for n in (1, 40):
        check_queries(c, n, True)
        q = torch.zeros(2, n, 8, 128, device="cuda").bfloat16()
        assert not bool(c.cache.query_attention(q).any())


def test_logits_far_apart():
    """Each tile's logits far above the last's (and then far below): the running maximum moves in every tile."""
    cfg = cfg_of(8, 2, 128, I8, I8, 16, 16, 64)
    T = 640
    up = np.arange(T) / 20.0
    for ramp in (up, up[::-1].copy(), np.where(np.arange(T) == 500, 60.0, 0.0)):
        K_ = np.zeros((T, 128))
        K_[:, 0] = ramp
        Ks = [[O.bf16(K_), O.bf16(-K_)]]
        Vs = [[O.bf16(np.random.default_rng(h).standard_normal((T, 128))) for h in range(2)]]
        c = Case(cfg, [T], seed=1, streams=(Ks, Vs))
        c.name = "ramp"
        for n in (2, 40, 80):
            q = np.zeros((1, n, 8, 128), np.float32)
            q[..., 0] = 24.0
            check_queries(c, n, True, q=q)
            check_queries(c, n, False, q=q)


# ------------------------------------------------- wide block tables: more rows than 32 then take the other kernel

def widened(c, tokens):
    """A view of Case c whose block table could hold `tokens` a sequence (no page behind those in use)."""
    import asymmetric_quantized_kv_gb300 as K
    w = object.__new__(Case)
    w.__dict__.update(c.__dict__)
    table = torch.full((len(c.lens), -(-tokens // c.cfg.page_size)), -1, dtype=torch.int32, device="cuda")
    table[:, :c.cache.block_table.shape[1]] = c.cache.block_table
    w.cache = K.PagedKVCache.over(c.c_cfg, c.cache.pages, table, c.cache.seq_lens, c.cache.k_win, c.cache.v_win)
    return w


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [9, 33, 64, 150])
def test_query_attention_wide_table(case, n, causal):
    check_queries(widened(case, 1 << 21), n, causal)


@pytest.mark.parametrize("name", SOILED)
def test_what_lies_behind_a_sequence_is_not_read_wide_table(name):
    cfg, lens = CASES[name]
    c = Case(cfg, lens, seed=22)
    c.name = name
    q = torch_src(O.bf16(np.random.default_rng(3).standard_normal((len(lens), 70, cfg.num_q_heads, cfg.head_dim))), cfg)
    clean = [widened(c, 1 << 21).cache.query_attention(q, causal=k) for k in (True, False)]
    _, defined = c.oracle_pages()
    soiled = c.cache.page_view().cpu().numpy().copy()
    soiled[~defined] = 0xFF
    c.cache.page_view().copy_(torch.from_numpy(soiled))
    for b, T in enumerate(lens):
        c.cache.k_win[b, T % cfg.residual:] = float("nan")
        c.cache.v_win[b, T % cfg.residual:] = float("inf")
    again = [widened(c, 1 << 21).cache.query_attention(q, causal=k) for k in (True, False)]
    assert all(torch.equal(a, b) for a, b in zip(clean, again))


@pytest.mark.parametrize("n", [1, 5])
def test_table_whose_work_passes_31_bits(n):
    """Tokens that the table could hold x heads / 16 beyond 2^30: the split counts in larger places."""
    cfg, lens = CASES["e4m3_p64"]
    c = Case(cfg, lens, seed=2)
    c.name = "e4m3_p64"
    w = widened(c, 400_000_000)
    check_queries(w, n, True)
    check_queries(w, n, False)


@pytest.mark.parametrize("Bn,T,n", [(40, 466, 12), (64, 100, 3), (9, 700, 16), (150, 33, 5), (33, 1200, 8)])
def test_runs_that_cross_sequences(Bn, T, n):
    """Batches whose pairs do not divide evenly among the warps, with sequences of no and of one token between."""
    cfg = cfg_of(16, 8, 64, E4, E4, 64, 64, 64)
    lens = [T - (b % 5) for b in range(Bn)]
    lens[1], lens[Bn // 2] = 0, 1
    c = Case(cfg, lens, seed=8)
    c.name = "runs"
    check_queries(c, n, True, [(7 * b) % (n + 1) for b in range(Bn)])
    check_queries(c, n, False)


def test_passes_of_one_launch():
    """Rows of several passes in one launch and of several launches: head_dim 256 takes 16 a pass, 128 a launch."""
    cfg, lens = CASES["d256"]
    c = Case(cfg, lens, seed=5)
    c.name = "d256"
    for n in (4, 7, 32, 33, 75):
        check_queries(c, n, True)
        check_queries(c, n, False, [n - (b * n) // 3 for b in range(len(lens))])


def test_decode_without_a_workspace_eight_heads_a_group():
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(64, 8, 128, E4, E4, 64, 64, 64)
    c = Case(cfg, [100, 700, 64, 5], seed=3)
    q = torch_src(c.queries(), cfg)
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    K.kvq_decode_attention_noalloc(c.c_cfg, c.cache.c, q, out, 0.0)
    assert torch.equal(out, c.cache.attention(q))


@pytest.mark.parametrize("cfg,rot,halves", [
    (cfg_of(8, 2, 128, E4, E4, 64, 64, 64), 128, True), (cfg_of(6, 3, 64, I8, I8, 32, 128, 32), 32, False),
    (cfg_of(4, 2, 256, E5, E5, 32, 64, 64), 256, True), (cfg_of(4, 2, 128, E4, E4, 32, 64, 32, src=O.F32), 128, True),
    (cfg_of(18, 9, 128, E4, E4, 64, 64, 16), 64, True)])
def test_rope_append_of_17_to_32_rows(cfg, rot, halves):
    """Chunks that fill a window, more than one of its rows behind it, and chunks that do not."""
    for fused in (True, False):
        c = rotated_case(cfg, [220, 131, 64, 20, 0], rot, halves, [20, 32, 31, 17], seed=rot, fused=fused)
        c.check_pages()
        c.check_lengths_and_window()
        c.check_dequantize()


# ----------------------------------------------------------- what a row does not see must not reach it

@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fmt", [E4, E5, I8])
@pytest.mark.parametrize("D,Hq,H,n", [(128, 8, 2, 5), (64, 16, 16, 21), (128, 16, 4, 70), (64, 4, 4, 300), (256, 8, 2, 9),
                                      (128, 2, 1, 140)])
def test_masked_tokens_that_are_not_finite(fmt, D, Hq, H, n, wide):
    """NaN and infinities in keys and values of tokens that only later queries see, in the window and in blocks
    (as codes, and as an infinite scale): the earlier queries' outputs stay (each is within 2^-8 |out| + 2^-10 sum p |v| of
    the exact one, |v| < 8, so two differ by 2^-7 |out| + 2^-6 at most); every row that sees a value of NaN is NaN."""
    cfg = cfg_of(Hq, H, D, fmt, fmt, 64, 64, 64)
    g, L = np.random.default_rng(5), O.layout(cfg)
    for T, first in ((500, 497), (500, 460 if n > 45 else 498), (448, 446),
                     (470 + n, (470 + n) // 64 * 64 - 20 if n > 30 else 470 + n - 2)):
        if T - n > first:
            continue
        Ks = [[O.bf16(g.standard_normal((T, D))) for _ in range(H)]]
        Vs = [[O.bf16(g.standard_normal((T, D))) for _ in range(H)]]
        c = Case(cfg, [T], seed=1, streams=(Ks, Vs))
        q = torch_src(O.bf16(g.standard_normal((1, n, Hq, D))), cfg)
        cache = (widened(c, 1 << 21) if wide else c).cache
        want = cache.query_attention(q)
        seen = first - (T - n)                   # queries [0, seen) see no token from `first` on
        nq = T // 64 * 64
        for bad in (float("nan"), float("inf"), -float("inf")):
            for b in range(max(first, nq), T):   # window rows
                cache.k_win[0, b - nq, :, 3] = bad
                cache.v_win[0, b - nq, :, D - 2] = bad
            if first < nq and fmt != I8:         # codes of the tokens of the last block that are not seen
                page = cache.page_view()[c.block_table[0, (nq - 1) // 64]]
                code = 0x7F if fmt == E4 else (0x7E if np.isnan(bad) else 0x7C)
                for h in range(H):
                    hb = page[h * L["head"]:]
                    for t in range(first, nq):
                        hb[L["kc"] + (t % 64) * D + 1] = code
                        hb[L["vc"] + (t % 64) * D + D - 1] = code
            got = cache.query_attention(q)
            assert torch.allclose(got[:, :seen].float(), want[:, :seen].float(), rtol=2.0 ** -7, atol=2.0 ** -6), (T, first, bad)
            assert bool(torch.isfinite(got[:, :seen]).all())
            if np.isnan(bad) and (first >= nq or fmt != I8):
                assert bool(torch.isnan(got[:, seen:, :, D - 2 if first >= nq else D - 1]).all())
        before = nq - 64 - (T - n)               # queries that see nothing of the last block
        if before > 0:
            page = cache.page_view()[c.block_table[0, (nq - 1) // 64]]
            for h in range(H):
                for at in (L["vm"], L["km"]):
                    page[h * L["head"] + at:h * L["head"] + at + 4] = torch.tensor([0, 0, 0x80, 0x7F], dtype=torch.uint8)
            got = cache.query_attention(q)
            assert torch.allclose(got[:, :before].float(), want[:, :before].float(), rtol=2.0 ** -7, atol=2.0 ** -6)
        assert int(cache.status.item()) == 0


@pytest.mark.parametrize("n", [1, 6, 40])
@pytest.mark.parametrize("Bn", [1000, 4096, 4097])
def test_large_batches(Bn, n):
    """Thousands of sequences over the same pages (4,097 exceed the split's table and take the plain kernel): every
    one within the bound of the exact output, empty ones zeros."""
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(4, 2, 64, E4, E4, 32, 32, 32)
    c = Case(cfg, [137], seed=3)
    lens = torch.full((Bn,), 137, dtype=torch.int32, device="cuda")
    lens[5::7] = 0
    many = K.PagedKVCache.over(c.c_cfg, c.cache.pages, c.cache.block_table.repeat(Bn, 1), lens,
                               c.cache.k_win.repeat(Bn, 1, 1, 1), c.cache.v_win.repeat(Bn, 1, 1, 1))
    q = torch_src(O.bf16(np.random.default_rng(n).standard_normal((1, n, 4, 64))), cfg)
    got = many.query_attention(q.repeat(Bn, 1, 1, 1)).double().cpu().numpy()
    assert not got[5::7].any()
    got = np.delete(got, np.s_[5::7], 0)
    qs = q.double().cpu().numpy()[0]
    for h in range(2):
        Kd, Vd = O.dequantize_stream(cfg, c.states[0][h], c.k_scale[h], c.v_scale[h])
        ref, size = O.query_attention(qs[:, 2 * h:2 * h + 2], Kd, Vd, True)
        lim = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * size + 2.0 ** -25 * np.abs(Vd).sum(0)
        assert np.all(np.abs(got[:, :, 2 * h:2 * h + 2] - ref) <= lim)
    assert int(many.status.item()) == 0


def test_nothing_to_do():
    """No new rows, no queries, no tokens."""
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(8, 2, 128, E4, E4, 64, 64, 64)
    c = Case(cfg, [0, 0], seed=1, extra_pages=2).cache
    rope = K.make_rope(rope_setup(256, 128)[1], 128)
    x = torch.zeros(2, 0, 12, 128, device="cuda").bfloat16()
    q = c.append_rope(rope, x[:, :, :8], x[:, :, 8:10], x[:, :, 10:])
    assert q.shape == (2, 0, 8, 128) and c.seq_lens.tolist() == [0, 0]
    assert c.query_attention(q).shape == (2, 0, 8, 128)
    for n in (1, 5, 40, 300):
        q = torch.ones(2, n, 8, 128, device="cuda").bfloat16()
        for causal in (True, False):
            assert not bool(c.query_attention(q, causal=causal).any())
    assert not bool(c.attention(torch.ones(2, 8, 128, device="cuda").bfloat16()).any())
    counts = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = torch.full((2, 5, 8, 128), 3.0, device="cuda").bfloat16()
    assert bool((c.query_attention(torch.ones_like(out), n_q_per_seq=counts, out=out) == 3.0).all())
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("n", [1, 6, 90])
def test_two_streams_at_once(n):
    """Two cache objects over the same pages, their calls interleaved on two streams: the results of one at a time."""
    import asymmetric_quantized_kv_gb300 as K
    cfg, lens = CASES["e4m3_p64"]
    c = Case(cfg, lens, seed=12)
    a, b = widened(c, 1 << 21).cache, widened(c, 1 << 21).cache
    qs = [torch_src(O.bf16(np.random.default_rng(i).standard_normal((len(lens), n, 32, 128))), cfg) for i in range(2)]
    want = [c.cache.query_attention(q, causal=False) if n <= 8 else a.query_attention(q, causal=False) for q in qs]
    b.query_attention(qs[1], causal=False)  # its workspace
    torch.cuda.synchronize()
    s0, s1 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [[torch.empty_like(q) for _ in range(10)] for q in qs]
    for i in range(10):
        a.query_attention(qs[0], causal=False, out=outs[0][i], stream=s0)
        b.query_attention(qs[1], causal=False, out=outs[1][i], stream=s1)
    torch.cuda.synchronize()
    for w, row in zip(want, outs):
        for o in row:
            assert torch.allclose(o.float(), w.float(), rtol=2.0 ** -7, atol=2.0 ** -6)
            assert torch.equal(o, row[0])
    assert int(c.cache.status.item()) == 0


@pytest.mark.parametrize("n", [40, 200])
def test_graph_of_many_rows(n):
    """Many-row attention captured once: replays follow the lengths on the device, as eager calls do, bit for bit."""
    cfg, _ = CASES["int8_p16"]
    c = Case(cfg, [1500, 700, 64], seed=13)
    cache = widened(c, 1 << 21).cache
    q = torch_src(O.bf16(np.random.default_rng(n).standard_normal((3, n, 8, 128))), cfg)
    out = torch.empty_like(q)
    cache.query_attention(q, out=out)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        cache.query_attention(q, out=out)
    for lens in ([1500, 700, 64], [1472, 0, 1], [64, 699, 64], [1, 1, 1]):
        cache.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7.0)
        gr.replay()
        assert torch.equal(out, cache.query_attention(q)), lens
    assert int(cache.status.item()) == 0


@pytest.mark.parametrize("n_rep,n,D", [(4, 10, 128), (5, 7, 64), (2, 64, 128), (4, 64, 128)])
def test_not_finite_in_hundreds_of_one_tile_units(n_rep, n, D):
    """A CTA of the many-row kernel has many units of one tile each in flight; what one notes of a value that is not
    finite stays until its outputs have left.  The last token's value is NaN in every other sequence: of those the last
    query alone is NaN, in all channels or in that one, and every other row is as without it."""
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(8 * n_rep, 8, D, E4, E4, 64, 64, 64)
    c = Case(cfg, [97], seed=3)
    Bn = 600
    many = K.PagedKVCache.over(c.c_cfg, c.cache.pages, c.cache.block_table.repeat(Bn, 1), c.cache.seq_lens.repeat(Bn),
                               c.cache.k_win.repeat(Bn, 1, 1, 1), c.cache.v_win.repeat(Bn, 1, 1, 1))
    wide = widened(c, 1 << 21).cache
    q = torch_src(O.bf16(np.random.default_rng(n).standard_normal((1, n, 8 * n_rep, D))), cfg)
    want = wide.query_attention(q)
    assert bool(torch.isfinite(want).all())
    many.v_win[::2, 96 - 64, :, 5] = float("nan")
    for _ in range(4):
        got = many.query_attention(q.repeat(Bn, 1, 1, 1))
        assert bool(torch.isnan(got[::2, n - 1, :, 5]).all())
        # each within 2^-8 |out| + 2^-10 sum p |v| of the exact output, |v| < 8
        for part, ref in ((got[::2, :n - 1], want[:, :n - 1]), (got[1::2], want)):
            assert torch.allclose(part.float(), ref.float().expand_as(part), rtol=2.0 ** -7, atol=2.0 ** -6)
    assert int(many.status.item()) == 0


def test_calls_without_queries_between_others():
    """Calls in which no sequence has a query write their plan to the same workspace as the calls around them."""
    cfg, lens = CASES["e4m3_p64"]
    c = Case(cfg, lens, seed=4)
    q = torch_src(O.bf16(np.random.default_rng(1).standard_normal((len(lens), 3, 32, 128))), cfg)
    none = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    cache = widened(c, 1 << 21).cache
    want, keep = cache.query_attention(q), torch.full_like(q, 7.0)
    outs = [torch.empty_like(q) for _ in range(40)]
    for o in outs:
        cache.query_attention(q, n_q_per_seq=none, out=keep)
        cache.query_attention(q, out=o)
        cache.query_attention(q, n_q_per_seq=none, out=keep)
    assert all(torch.equal(o, want) for o in outs) and bool((keep == 7.0).all())
    assert int(cache.status.item()) == 0


@pytest.mark.parametrize("kind", ["bf16", "f32", "mixed"])
def test_missing_page_of_a_blocks_scales(kind):
    """Blocks over several pages.  A missing page's tokens get no weight, and where it holds the block's scales the
    whole block gets none: on the tensor-core kernels (bf16) and on the plain one (fp32 sources, differing formats)."""
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(8, 2, 128, E4, I8 if kind == "mixed" else E4, 64, 64, 16, src=O.F32 if kind == "f32" else O.BF16)
    T = 300
    c = Case(cfg, [T], seed=6)
    c.cache.block_table[0, 4] = c.cache.n_pages + 3   # tokens 64 .. 79, and the scales of 64 .. 127
    c.cache.block_table[0, 9] = -1                    # tokens 144 .. 159 alone
    keep = np.ones(T, bool)
    keep[64:128] = keep[144:160] = False
    half = 2.0 ** -24 if kind == "f32" else 2.0 ** -8
    for n in (1, 6, 40):
        q = O.bf16(np.random.default_rng(n).standard_normal((1, n, 8, 128)))
        for cache in (c.cache, widened(c, 1 << 21).cache):
            got = cache.query_attention(torch_src(q, cfg), causal=False).double().cpu().numpy()
            assert int(c.cache.status.item()) | int(cache.status.item()) == K.KVQ_DEV_BAD_PAGE
            for h in range(2):
                Kd, Vd = O.dequantize_stream(cfg, c.states[0][h], c.k_scale[h], c.v_scale[h])
                ref, size = O.query_attention(q[0, :, 4 * h:4 * h + 4], Kd[keep], Vd[keep], False)
                lim = half * np.abs(ref) + 2.0 ** -10 * size + 2.0 ** -25 * np.abs(Vd).sum(0)
                assert np.all(np.abs(got[0, :, 4 * h:4 * h + 4] - ref) <= lim), (n, h)


@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("kind", [I8, E4, E5, "f32", "meta16"])
def test_not_finite_through_an_append(kind, bad):
    """A block that gets a value that is not finite reads as NaN, every other block as without it; queries that see a
    token of the block are NaN, those that do not are within the bound of the exact output: on the plain kernel (fp32
    sources), the few-row and the many-row one."""
    fmt = kind if kind in (I8, E4, E5) else I8
    cfg = cfg_of(8, 2, 128, fmt, fmt, 32, 64, 32, src=O.F32 if kind == "f32" else O.BF16,
                 meta_dtype=O.F16 if kind == "meta16" else O.F32)
    T, x, half = 300, float(bad), 2.0 ** -24 if kind == "f32" else 2.0 ** -8
    g = np.random.default_rng(3)
    rows = lambda: [[O.bf16(g.standard_normal((T, 128))) for _ in range(2)] for _ in range(3)]
    Ks, Vs = rows(), rows()
    Ks[0][1][250, 7] = x          # a key in tokens 224 .. 255: sequence 0, head 1
    Vs[1][0][131, 100] = x        # a value in tokens 128 .. 159: sequence 1, head 0
    Vs[2][1][290, 9] = x          # a value in the window: sequence 2, head 1
    c = Case(cfg, [T] * 3, seed=1, streams=(Ks, Vs))
    block = {(0, 1): (224, 256), (1, 0): (128, 160)}
    deq = []
    for b in range(3):
        k, v = (t.double().cpu().numpy() for t in c.cache.dequantize(b, 0, T))
        for h in range(2):
            Kd, Vd = O.dequantize_stream(cfg, c.states[b][h])
            np.testing.assert_array_equal(k[:, h], Kd)
            np.testing.assert_array_equal(v[:, h], Vd)
            deq.append((b, h, Kd, Vd))
            if (b, h) in block:
                lo, hi = block[b, h]
                assert np.isnan((Kd if b == 0 else Vd)[lo:hi]).all()
                assert np.isfinite(np.delete(Kd if b == 0 else Vd, np.s_[lo:hi], 0)).all()
    for n in (1, 5, 200):
        q = O.bf16(g.standard_normal((3, n, 8, 128)))
        for cache in (c.cache, widened(c, 1 << 21).cache):
            got = cache.query_attention(torch_src(q, cfg)).double().cpu().numpy()
            for b, h, Kd, Vd in deq:
                y, end = got[b, :, 4 * h:4 * h + 4], T - n + 1 + np.arange(n)
                first = block[b, h][0] if (b, h) in block else 290 if (b, h) == (2, 1) else T
                sees = end > first
                if (b, h) == (2, 1):
                    assert not np.isfinite(y[sees, :, 9]).any()
                else:
                    assert np.isnan(y[sees]).all(), (b, h, n)
                if not sees.all():
                    m = int((~sees).sum())
                    ref, size = O.query_attention(q[b, :m, 4 * h:4 * h + 4], Kd[:end[m - 1]], Vd[:end[m - 1]], True)
                    lim = half * np.abs(ref) + 2.0 ** -10 * size + 2.0 ** -25 * np.abs(Vd[:end[m - 1]]).sum(0)
                    assert np.all(np.abs(y[:m] - ref) <= lim), (b, h, n)
    assert int(c.cache.status.item()) == 0


def oracle_limits(cfg, state, q, h, causal=True):
    """Exact outputs of kv-head h's queries, and the bound of the file's head for each element."""
    Kd, Vd = O.dequantize_stream(cfg, state)
    heads = slice(h * cfg.n_rep, (h + 1) * cfg.n_rep)
    ref, size = O.query_attention(q[:, heads].astype(np.float64), Kd, Vd, causal)
    return ref, 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * size + 2.0 ** -25 * np.abs(Vd).sum(0)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D,Hq,H,n", [(128, 8, 2, 5), (64, 16, 16, 21), (128, 16, 4, 70), (64, 4, 4, 300), (256, 8, 2, 9),
                                      (128, 2, 1, 140)])
def test_window_tokens_far_apart(D, Hq, H, n, wide):
    """Finite keys and values of any size in the window.  Those of tokens that only later queries see leave the earlier
    ones within the bound of the exact output; rows 2^40 and 2^45 times the others leave every query within it (a logit
    2^40 times the others is off by more than they are large, but its weight is 0 or 1 whatever it is off by)."""
    cfg = cfg_of(Hq, H, D, E4, E4, 64, 64, 64)
    g, T = np.random.default_rng(6), 500          # 52 tokens in the window
    big = float(np.frombuffer(np.uint32(0x7F7F0000).tobytes(), np.float32)[0])   # the largest bf16
    q = O.bf16(g.standard_normal((1, n, Hq, D)))

    def outputs(Ks, Vs):
        c = Case(cfg, [T], seed=1, streams=([Ks], [Vs]))
        got = (widened(c, 1 << 21) if wide else c).cache.query_attention(torch_src(q, cfg)).double().cpu().numpy()[0]
        assert int(c.cache.status.item()) == 0
        return c, got

    def streams():
        return tuple([O.bf16(g.standard_normal((T, D))) for _ in range(H)] for _ in range(2))
    for large in (2.0 ** 40, big):
        for first in (T - 2, T - 20):
            if n <= T - first:
                continue
            Ks, Vs = streams()
            for X, ch in ((Ks, 3), (Vs, D - 2)):
                for x in X:
                    x[first:, ch] = np.where(np.arange(T - first) % 2, large, -large)
            c, got = outputs(Ks, Vs)
            m = n - (T - first)                   # queries that see none of them
            for h in range(H):
                st = O.quantize_stream(cfg, Ks[h][:first], Vs[h][:first])
                ref, lim = oracle_limits(cfg, st, q[0, :m], h)
                assert np.all(np.abs(got[:m, h * cfg.n_rep:(h + 1) * cfg.n_rep] - ref) <= lim), (large, first, h)
    for rows, which in (((470, 471), 0), ((475, 490), 1)):
        for at in ((rows[0],), rows):
            KV = streams()
            for x in KV[which]:
                for i, r in enumerate(at):
                    x[r] *= 2.0 ** (40 + 5 * i)
            c, got = outputs(*KV)
            for h in range(H):
                ref, lim = oracle_limits(cfg, c.states[0][h], q[0], h)
                assert np.all(np.abs(got[:, h * cfg.n_rep:(h + 1) * cfg.n_rep] - ref) <= lim), (which, at, h)
            c.check_attention()


@pytest.mark.parametrize("fmt", [E4, I8])
def test_heavy_tokens_without_values(fmt):
    """A token with most of the weight whose block's values are all zero (padding, a sink) leaves the others' weights
    their bits: they all have 2^-17.5 of its weight, so that a rounding would go the same way in all of them."""
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(4, 2, 64, fmt, fmt, 32, 32, 32)
    T, Bn = 970, 600                      # long runs: a warp's, and a unit's, hold the token and many others
    Ks, Vs = ([np.zeros((T, 64)) for _ in range(2)] for _ in range(2))
    for h in range(2):
        Ks[h][5, 0] = 1.0
        Vs[h][32:] = O.bf16(1.0 + np.random.default_rng(h).random((T - 32, 64)))
    c = Case(cfg, [T], seed=3, streams=([Ks], [Vs]))
    many = K.PagedKVCache.over(c.c_cfg, c.cache.pages, c.cache.block_table.repeat(Bn, 1), c.cache.seq_lens.repeat(Bn),
                               c.cache.k_win.repeat(Bn, 1, 1, 1), c.cache.v_win.repeat(Bn, 1, 1, 1))
    for n in (1, 6, 40):
        q = np.zeros((1, n, 4, 64))
        q[..., 0] = O.bf16(np.full((1, n, 4), 17.5 * np.log(2.0) * 8.0))
        got = many.query_attention(torch_src(q, cfg).repeat(Bn, 1, 1, 1), causal=False).double().cpu().numpy()
        for h in range(2):
            ref, lim = oracle_limits(cfg, c.states[0][h], q[0], h, False)
            assert np.all(np.abs(got[:, :, 2 * h:2 * h + 2] - ref) <= lim), (n, h)


def test_new_tensors_belong_to_the_stream_that_writes_them():
    """With a stream named, what a call allocates comes from that stream's pool, not from the current stream's, where
    the memory may still be in use."""
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(8, 2, 128, E4, E4, 64, 64, 64)
    _, tt = rope_setup(512, 128)
    rope = K.make_rope(tt, 128)
    cache = Case(cfg, [100, 70], seed=6, extra_pages=4).cache
    x = torch.randn(2, 5, 12, 128, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        q = cache.append_rope(rope, x[:, :, :8], x[:, :, 8:10], x[:, :, 10:], stream=stream)
        made = [q, cache.query_attention(q, stream=stream), cache.attention(q[:, 0].contiguous(), stream=stream),
                *cache.dequantize(0, 0, 90, stream=stream)]
        side.synchronize()
        made.append(cache.workspace)          # grown by the first query_attention
        where = [next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= t.data_ptr() < s["address"] + s["total_size"])
                 for t in made]
        assert where == [side.cuda_stream] * len(made)
    assert cache.query_attention(q, stream=0).data_ptr() != 0
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 0


def test_outgrown_workspaces_stay_below_the_one_in_use():
    cfg = cfg_of(2, 2, 128, E4, E4, 64, 64, 64)
    cache = Case(cfg, [100], seed=6).cache
    for n in range(1, 80):
        cache.query_attention(torch.zeros(1, n, 2, 128, device="cuda").bfloat16())
        assert sum(w.numel() for w in cache._outgrown) <= cache.workspace.numel()


def test_logits_far_below_zero():
    """Every logit below -10^31: the largest still has the weight 1."""
    cfg = cfg_of(8, 2, 128, E4, E4, 32, 32, 32)
    T = 330
    for heavy in (7, 328):                       # in a block, in the window
        Ks, Vs = ([O.bf16(np.random.default_rng(h).standard_normal((T, 128))) for h in range(2)] for _ in range(2))
        for x in Ks:
            x[:] = 0.0
            x[:, 0] = -2.0 ** 57
            x[heavy, 0] = -2.0 ** 56
        c = Case(cfg, [T], seed=3, streams=([Ks], [Vs]))
        for n in (1, 5, 70):
            q = np.zeros((1, n, 8, 128))
            q[..., 0] = 2.0 ** 50
            for cache in (c.cache, widened(c, 1 << 21).cache):
                got = cache.query_attention(torch_src(q, cfg), causal=False).double().cpu().numpy()[0]
                for h in range(2):
                    Kd, Vd = O.dequantize_stream(cfg, c.states[0][h])
                    assert np.all(np.abs(got[:, 4 * h:4 * h + 4] - Vd[heavy]) <= 2.0 ** -8 * np.abs(Vd[heavy])), (heavy, n, h)


@pytest.mark.parametrize("D,Hq,H,Bn", [(128, 16, 1, 2), (256, 32, 2, 5), (128, 64, 8, 100), (128, 128, 1, 3), (256, 16, 1, 1)])
def test_decode_without_a_workspace_wide_groups(D, Hq, H, Bn):
    """Calls whose records would not fit the fixed array with all runs: the same bits as with a workspace, and the
    oracle's outputs."""
    import asymmetric_quantized_kv_gb300 as K
    cfg = cfg_of(Hq, H, D, E4, E4, 64, 64, 64)
    c = Case(cfg, [3000 if b == 0 else 100 + 37 * b for b in range(Bn)], seed=3)
    q = torch_src(c.queries(), cfg)
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    K.kvq_decode_attention_noalloc(c.c_cfg, c.cache.c, q, out, 0.0)
    assert torch.equal(out, c.cache.attention(q))
    c.check_attention()


def odd_values(g, Ks, Vs, lens, R, D):
    """A few tokens, most of them in the window, with NaN, an infinity, zeros or a row far larger than the others."""
    for _ in range(int(g.integers(0, 4))):
        b, h = int(g.integers(0, len(lens))), int(g.integers(0, len(Ks[0])))
        if lens[b] == 0:
            continue
        t = int(g.integers(0, lens[b])) if g.random() < 0.3 else lens[b] - 1 - int(g.integers(0, min(lens[b], R)))
        X, kind = (Ks, Vs)[int(g.integers(0, 2))], int(g.integers(0, 4))
        if kind == 0:
            X[b][h][t, int(g.integers(0, D))] = np.nan
        elif kind == 1:
            X[b][h][t, int(g.integers(0, D))] = -np.inf
        elif kind == 2:
            X[b][h][t] = 0.0
        else:
            X[b][h][t] *= 2.0 ** (36 if X is Ks else 20)


@pytest.mark.parametrize("copies", [1, 120])
@pytest.mark.parametrize("first", range(0, 100, 20))
def test_random_calls_with_odd_values(first, copies):
    """Random shapes, formats, lengths and masks over tokens of any kind, alone and as many copies over shared pages
    (many units of every kernel's split): finite rows within the bound, with 2^-25 of the largest magnitude of each
    token's block (in the window, of the token) in place of the channel's, rows that see NaN not finite."""
    import asymmetric_quantized_kv_gb300 as K
    for seed in range(first, first + 20):
        g = np.random.default_rng(1000 * copies + seed)
        D, H, rep = int(g.choice([64, 128, 128, 256])), int(g.choice([1, 2, 3])), int(g.choice([1, 2, 4, 5, 8]))
        G, P, fmt = int(g.choice([16, 32, 64])), int(g.choice([16, 64, 128])), int(g.choice([E4, E5, I8]))
        R = G * int(g.choice([1, 2, 3]))
        n, causal = int(g.choice([1, 2, 5, 9, 17, 33, 70, 140])), bool(g.random() < 0.7)
        lens = [int(g.choice([int(g.integers(0, 130)), int(g.integers(0, 3 * R + 300))])) for _ in range(int(g.integers(1, 4)))]
        cfg = cfg_of(H * rep, H, D, fmt, fmt, G, R, P, meta_dtype=O.F16 if seed % 5 == 0 else O.F32)
        Ks, Vs = ([[O.bf16(g.standard_normal((T, D))) for _ in range(H)] for T in lens] for _ in range(2))
        odd_values(g, Ks, Vs, lens, R, D)
        with np.errstate(all="ignore"):
            c = Case(cfg, lens, seed=1, streams=(Ks, Vs))
        q = O.bf16(g.standard_normal((len(lens), n, H * rep, D)))
        m = c.cache
        caches = [m, widened(c, 1 << 21).cache] if copies == 1 else [K.PagedKVCache.over(
            c.c_cfg, m.pages, m.block_table.repeat(copies, 1), m.seq_lens.repeat(copies), m.k_win.repeat(copies, 1, 1, 1),
            m.v_win.repeat(copies, 1, 1, 1))]
        got = [x.query_attention(torch_src(q, cfg).repeat(copies, 1, 1, 1), causal=causal).double().cpu().numpy()
               .reshape(copies, *q.shape) for x in caches]
        got = np.concatenate(got)
        assert all(int(x.status.item()) == 0 for x in caches)
        for b, T in enumerate(lens):
            nq = T // R * R
            for h in range(H):
                Kd, Vd = O.dequantize_stream(cfg, c.states[b][h])
                a = np.abs(Vd).max(1, initial=0.0)
                a[:nq] = np.repeat(a[:nq].reshape(-1, G).max(1, initial=0.0), G)
                for i in range(n):
                    end = max(0, T - n + i + 1) if causal else T
                    y, k, v = got[:, b, i, h * rep:(h + 1) * rep], Kd[:end], Vd[:end]
                    if np.isfinite(k).all() and np.isfinite(v).all():
                        ref, size = O.query_attention(q[b, i:i + 1, h * rep:(h + 1) * rep], k, v, False)
                        lim = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * size + 2.0 ** -25 * a[:end].sum()
                        assert np.all(np.abs(y - ref[0]) <= lim[0]), (seed, b, h, i)
                    elif np.isnan(k).any():
                        assert np.isnan(y).all(), (seed, b, h, i)
                    elif np.isfinite(k).all():
                        assert not np.isfinite(y[..., np.isnan(v).any(0)]).any(), (seed, b, h, i)
