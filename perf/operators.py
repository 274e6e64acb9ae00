"""Measured cases of three operators on a paged key/value cache held in 8 bits with one
scale for each (block of tokens, kv-head), and of the position rotation on the way in:

* append: new queries, keys and values as a fused projection leaves them; queries and keys
  are rotated to their positions, keys and values go into the residual window, and every
  window that fills is quantized into the pages (kvq_rope_append).
* attend: causal attention of each sequence's newest tokens over its cache: one token a
  sequence (a decode step), a few (checking a draft) or many (a prompt's chunk)
  (kvq_query_attention with the causal mask).
* cross: attention of decoder tokens over the cached states of an encoder, a sequence of
  another length, without a mask (kvq_query_attention without one).

With own = False, run() computes them from elementary torch operations in 32 bits; with
own = True, through the package.
"""
import math

import numpy as np
import torch

own = False

INT8, E4M3, E5M2 = 8, 9, 10            # the package's names for the formats
QMAX = {INT8: 127.0, E4M3: 448.0, E5M2: 57344.0}
F8 = {E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}
THETA = 500000.0


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one new token for each of 64 running sequences, 32 query heads on 8 kv-heads: the append
        # of a decode step, where the call's latency counts
        dict(name="append_step_64", op="append", B=64, n=1, start=4101, ragged=True, Hq=32, Hkv=8, D=128, fmt=E4M3, G=64,
             R=64, P=64, rot=128, halves=True),
        # the prompts of 13 sequences of up to 701 tokens, added to caches of odd lengths; half of each
        # head rotated, interleaved pairs, blocks of 32 tokens in pages of 16
        dict(name="append_chunk_ragged", op="append", B=13, n=701, start=333, ragged=True, Hq=16, Hkv=4, D=128, fmt=INT8,
             G=32, R=128, P=16, rot=64, halves=False),
        # a whole batch of prompts at once, 64 query heads on 8 kv-heads
        dict(name="append_prompt_8x4096", op="append", B=8, n=4096, start=0, ragged=False, Hq=64, Hkv=8, D=128, fmt=E4M3,
             G=64, R=64, P=64, rot=128, halves=True),
        # one running sequence of 4,101 tokens: the smallest decode step
        dict(name="attend_step_1x4101", op="attend", B=1, n=1, T=4101, ragged=False, Hq=32, Hkv=8, D=128, fmt=E4M3, G=64,
             R=64, P=64),
        # the paged ragged layer of the benchmark: 64 sequences of 1,024 to 65,536 tokens
        dict(name="attend_step_ragged_64", op="attend", B=64, n=1, T=65536, ragged=True, Hq=32, Hkv=8, D=128, fmt=INT8,
             G=64, R=64, P=16),
        # the long-context layer of the benchmark: 8 sequences of 131,072 tokens, 64 query heads on 8
        dict(name="attend_step_8x131072", op="attend", B=8, n=1, T=131072, ragged=False, Hq=64, Hkv=8, D=128, fmt=E4M3,
             G=64, R=64, P=256),
        # five drafted tokens checked for each of 16 sequences of odd lengths
        dict(name="attend_draft_16x5", op="attend", B=16, n=5, T=9001, ragged=True, Hq=32, Hkv=8, D=128, fmt=E4M3, G=64,
             R=64, P=64),
        # a prompt taken in chunks: 512 more tokens for each of 4 sequences of 16,421 tokens
        dict(name="attend_chunk_4x512", op="attend", B=4, n=512, T=16421, ragged=False, Hq=32, Hkv=8, D=128, fmt=INT8,
             G=64, R=64, P=64),
        # a whole prompt of 8,192 tokens
        dict(name="attend_prompt_8192", op="attend", B=1, n=8192, T=8192, ragged=False, Hq=32, Hkv=8, D=128, fmt=E4M3,
             G=64, R=64, P=64),
        # a decoding step of 32 sequences over up to 1,500 encoder states, 16 heads of 64 without sharing
        dict(name="cross_step_32x1500", op="cross", B=32, n=1, T=1500, ragged=True, Hq=16, Hkv=16, D=64, fmt=E4M3, G=64,
             R=64, P=64),
        # the teacher-forced pass of the same: 448 decoder tokens a sequence
        dict(name="cross_pass_16x448", op="cross", B=16, n=448, T=1500, ragged=True, Hq=16, Hkv=16, D=64, fmt=E5M2, G=64,
             R=64, P=64),
        # 1,000 decoder tokens over the states of long documents
        dict(name="cross_long_4x1000", op="cross", B=4, n=1000, T=30011, ragged=False, Hq=32, Hkv=8, D=128, fmt=INT8,
             G=128, R=128, P=64),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm; every third one is a round one."""
    x = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, x if rng.random() < 0.67 else (x + 15) // 16 * 16))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "cross"])
    Hkv, rep = rng.choice([(8, 4), (8, 8), (4, 4), (8, 1), (16, 1), (2, 8), (8, 2), (4, 6), (5, 7)])
    G = rng.choice([32, 64, 64, 128])
    c = dict(op=op, Hq=Hkv * rep, Hkv=Hkv, D=rng.choice([64, 128, 128]), fmt=rng.choice([INT8, E4M3, E4M3, E5M2]), G=G,
             R=G * rng.choice([1, 1, 2]), P=rng.choice([16, 32, 64, 64, 128, 256]), ragged=rng.random() < 0.6)
    if op == "append":
        c["rot"] = c["D"] // rng.choice([1, 1, 2])
        c["halves"] = rng.random() < 0.5
        c["start"] = rng.choice([0, _log(rng, 1, 8000)])
        if rng.random() < 0.5:
            c["n"], c["B"] = rng.choice([1, 1, 1, 2, 5]), _log(rng, 1, 256)
        else:
            c["n"] = _log(rng, 16, 8192)
            c["B"] = _log(rng, 1, max(1, 32768 // c["n"]))
        while c["B"] > 1 and c["B"] * (c["start"] + c["n"]) * Hkv * c["D"] > 3e8:  # a pool of at most 600 MB
            c["B"] -= 1
        return c
    kind = rng.choice(["one", "one", "few", "many"])
    if kind == "one":
        c["n"], tokens = 1, _log(rng, 2000, 1 << 20)
    elif kind == "few":
        c["n"], tokens = rng.randint(2, 16), _log(rng, 2000, 1 << 18)
    else:
        c["n"], tokens = _log(rng, 33, 2048), _log(rng, 1000, 65536)
    c["T"] = _log(rng, 100, min(tokens, 131072 if kind == "one" else 32768))
    if op == "cross" and kind != "many":
        c["T"] = min(c["T"], 8000)
    c["B"] = max(1, min(tokens // c["T"], 128))
    if op == "attend":
        c["T"] = max(c["T"], c["n"])
    # no more work than the largest listed pass
    while c["B"] > 1 and (c["B"] * c["n"] * c["T"] * c["Hq"] * c["D"] > 2e11 or c["B"] * c["T"] * Hkv * c["D"] > 1e9):
        c["B"] -= 1
    return c


# ------------------------------------------------------- the cache: sizes and bytes of a page

def _geometry(case):
    """Byte offsets of a page's head block: key codes [P][D], value codes [P][D], value scales,
    key scales (one for each block of G tokens, in the page of the block's first token), each
    section on 16 bytes, the whole on 128."""
    P, D, G = case["P"], case["D"], case["G"]
    up = lambda n, m: (n + m - 1) // m * m
    vm = 2 * P * D
    km = up(vm + 4 * max(1, P // G), 16)
    return dict(vc=P * D, vm=vm, km=km, head=up(km + 4 * max(1, P // G), 128))


def _views(pages, case):
    """Codes [pages, heads, P, D] and scales [pages, heads, blocks] of keys and values, as views of the bytes."""
    g, P, D, H = _geometry(case), case["P"], case["D"], case["Hkv"]
    n = pages.shape[0]
    nb = max(1, P // case["G"])
    raw = pages.view(n, H, g["head"])
    f32 = pages.view(-1).view(torch.float32).view(n, H, g["head"] // 4)
    code = lambda o: raw[:, :, o:o + P * D].unflatten(2, (P, D))
    scale = lambda o: f32[:, :, o // 4:o // 4 + nb]
    return code(0), code(g["vc"]), scale(g["km"]), scale(g["vm"])


def _lengths(case, most, gen):
    """Tokens of each sequence: `most` each, or spread over a factor of up to 64 in their logarithm, the first one whole."""
    B = case["B"]
    if not case["ragged"] or most < 2:
        return np.full(B, most, np.int64)
    lo = max(1, most // 64)
    t = np.exp(gen.uniform(math.log(lo), math.log(most + 1), B)).astype(np.int64).clip(lo, most)
    t[0] = most
    return t


def _encode(y, fmt):
    """Bytes of y (already divided by its block's scale)."""
    if fmt == INT8:
        return y.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return y.clamp(-QMAX[fmt], QMAX[fmt]).to(F8[fmt]).view(torch.uint8)


def _decode(code, fmt):
    return code.view(torch.int8).float() if fmt == INT8 else code.view(F8[fmt]).float()


def _quantize(x, G, fmt):
    """x [B, n, H, D] float32, n a multiple of G -> bytes of the same shape and scales [B, n / G, H]."""
    B, n, H, D = x.shape
    x = x.view(B, n // G, G, H, D)
    s = x.abs().amax((2, 4)) / QMAX[fmt]
    d = s[:, :, None, :, None]
    y = torch.where(d > 0, x / d, torch.zeros((), device=x.device))
    return _encode(y, fmt).view(B, n, H, D), s


def _source(shape, gen, outliers):
    """Normal values as 16-bit projections give them; keys carry a few channels of larger magnitude."""
    x = torch.randn(shape, generator=gen, device="cuda")
    if outliers:
        x[..., 5::37] *= 12.0
    return x.to(torch.bfloat16)


def _fill(case, lens, gen, rng, n_pages, table):
    """A cache of those lengths: pages (and a spare one at the end), window, and its lengths."""
    B, H, D, P, G, R = (case[k] for k in ("B", "Hkv", "D", "P", "G", "R"))
    pages = torch.zeros(n_pages + 1, H * _geometry(case)["head"], dtype=torch.uint8, device="cuda")
    kc, vc, ks, vs = _views(pages, case)
    win = [torch.zeros(B, R, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    step = max(P, G)
    nq = torch.from_numpy(lens // R * R).cuda()
    rows = 1 << 15  # tokens of all sequences drawn at a time, so that the 32-bit values stay small
    span = max(step, rows // B // step * step)
    table64 = table.long()
    for t0 in range(0, int(lens.max()), span):
        n = min(span, -(-(int(lens.max()) - t0) // step) * step)
        t = torch.arange(t0, t0 + n, device="cuda")
        page = table64[:, (t // P).clamp(max=table.shape[1] - 1)]
        page = torch.where(t[None] < nq[:, None], page, n_pages)
        first = t[::G]
        for code, scale, w, k in ((kc, ks, win[0], True), (vc, vs, win[1], False)):
            x = _source((B, n, H, D), gen, k)
            c, s = _quantize(x.float(), G, case["fmt"])
            code[page, :, t % P] = c
            scale[page[:, ::G], :, (first % P) // G] = s
    for w, k in zip(win, (True, False)):
        w.copy_(_source((B, R, H, D), gen, k))
    return pages, win


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    B, Hq, H, D, P, R = (case[k] for k in ("B", "Hq", "Hkv", "D", "P", "R"))
    app = case["op"] == "append"
    lens = _lengths(case, case["start"] if app else case["T"], rng)
    if not app:
        new = np.full(B, case["n"], np.int64)
        lens = np.maximum(lens, new) if case["op"] == "attend" else lens
    else:
        new = _lengths(case, case["n"], rng)
    need = -(-(lens + (new if app else 0)) // max(P, case["G"])) * max(1, case["G"] // P)  # pages of each sequence
    if app:  # the pool comes back whole, so its size goes by the case, not by the seed
        need[:] = -(-(case["start"] + case["n"]) // max(P, case["G"])) * max(1, case["G"] // P)
    most, n_pages = int(need.max()), int(need.sum())
    table = np.zeros((B, most), np.int32)
    table[np.arange(most)[None] < need[:, None]] = rng.permutation(n_pages)
    table = torch.from_numpy(table).cuda()
    pages, win = _fill(case, lens, gen, rng, n_pages, table)
    s = dict(case=case, pages=pages, k_win=win[0], v_win=win[1], table=table, n_pages=n_pages,
             lens0=torch.from_numpy(lens.astype(np.int32)).cuda(), n=torch.from_numpy(new.astype(np.int32)).cuda(),
             lens=torch.from_numpy(lens.astype(np.int32)).cuda())
    if app:
        # queries, keys and values side by side in each token's row, as one projection writes them
        x = _source((B, case["n"], Hq + 2 * H, D), gen, False)
        x[:, :, Hq:Hq + H, 5::37] *= 12.0
        s["qkv"] = x
        s["q"], s["k"], s["v"] = x[:, :, :Hq], x[:, :, Hq:Hq + H], x[:, :, Hq + H:]
        s["q_out"] = torch.zeros(B, case["n"], Hq, D, dtype=torch.bfloat16, device="cuda")
        i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
        a = torch.arange(most * P, dtype=torch.float64, device="cuda")[:, None] * THETA ** (-2 * i / case["rot"])
        s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float()
    else:
        s["q"] = _source((B, case["n"], Hq, D), gen, False)
    return s


# ------------------------------------------------------------------- the package's calls

def _handle(s):
    """The cache object of a serving program, over the buffers that prepare() made."""
    import asymmetric_quantized_kv_gb300 as K
    c = s["case"]
    spec = (c["fmt"], K.KVQ_SYM_ABSMAX, K.KVQ_PER_BLOCK, c["G"])
    cfg = K.make_config(c["Hq"], c["Hkv"], c["D"], spec, spec, c["R"], c["P"], src_dtype=K.KVQ_BF16)
    cache = K.PagedKVCache.over(cfg, s["pages"][:s["n_pages"]], s["table"], s["lens"], s["k_win"], s["v_win"])
    rope = None
    if c["op"] == "append":
        rope = K.make_rope(s["cos_sin"], c["rot"], K.KVQ_ROPE_HALVES if c["halves"] else K.KVQ_ROPE_INTERLEAVED)
    return cache, rope


def _run_own(s):
    c = s["case"]
    if "handle" not in s:
        s["handle"] = _handle(s)
    cache, rope = s["handle"]
    if c["op"] == "append":
        s["lens"].copy_(s["lens0"])  # the scheduler's lengths of this step's batch
        cache.append_rope(rope, s["q"], s["k"], s["v"], s["n"], q_out=s["q_out"])
        if "outputs" not in s:  # views of the buffers that the call writes: a program names them once
            s["outputs"] = _append_outputs(s)
        return s["outputs"]
    return cache.query_attention(s["q"], causal=c["op"] == "attend")


# ----------------------------------------------------------------------- the plain form

def _rotate(x, cos, sin, rot, halves):
    """x [B, n, H, D] float32; cos, sin [B, n, 1, rot / 2]."""
    y = x.clone()
    if halves:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    return y


def _append_outputs(s):
    c = s["case"]
    kc, vc, ks, vs = _views(s["pages"][:s["n_pages"]], c)
    kind = torch.int8 if c["fmt"] == INT8 else F8[c["fmt"]]
    return dict(q=s["q_out"], k_codes=kc.view(kind), v_codes=vc.view(kind), k_scales=ks, v_scales=vs, k_win=s["k_win"],
                v_win=s["v_win"], lens=s["lens"])


def _run_append(s):
    c = s["case"]
    B, P, G, R, n = c["B"], c["P"], c["G"], c["R"], c["n"]
    s["lens"].copy_(s["lens0"])
    T0, new = s["lens"].long(), s["n"].long()
    i = torch.arange(n, device="cuda")
    live = (i[None] < new[:, None])[..., None, None]
    cs = s["cos_sin"][(T0[:, None] + i[None]).clamp(max=s["cos_sin"].shape[0] - 1)][:, :, None]
    cos, sin = cs[..., :c["rot"] // 2], cs[..., c["rot"] // 2:]
    q = _rotate(s["q"].float(), cos, sin, c["rot"], c["halves"]).to(torch.bfloat16)
    s["q_out"].copy_(torch.where(live, q, s["q_out"]))
    k = _rotate(s["k"].float(), cos, sin, c["rot"], c["halves"]).to(torch.bfloat16)
    # each sequence's window rows, then its new rows, from the last block boundary on
    have = T0 % R
    base = T0 - have
    L = -(-(R - 1 + n) // R) * R
    j = torch.arange(L, device="cuda")
    old = (j[None] < have[:, None])[..., None, None]
    b = torch.arange(B, device="cuda")[:, None]
    fresh = (j[None] - have[:, None]).clamp(0, n - 1)
    full = (have + new) // R * R                      # rows that are quantized by this call
    kc, vc, ks, vs = _views(s["pages"], c)
    t = base[:, None] + j[None]
    page = s["table"].long()[b, (t // P).clamp(max=s["table"].shape[1] - 1)]
    page = torch.where(j[None] < full[:, None], page, s["n_pages"])
    at = torch.arange(R, device="cuda")
    tail = (have + new - full)[:, None] > at[None]
    for x, win, code, scale in ((k, s["k_win"], kc, ks), (s["v"], s["v_win"], vc, vs)):
        rows = torch.where(old, win[:, j.clamp(max=R - 1)], x[b, fresh])
        cd, sc = _quantize(rows.float(), G, c["fmt"])
        code[page, :, t % P] = cd
        scale[page[:, ::G], :, (t[:, ::G] % P) // G] = sc
        left = rows[b, (full[:, None] + at[None]).clamp(max=L - 1)]
        win.copy_(torch.where(tail[..., None, None], left, win))
    s["lens"].add_(s["n"])
    return _append_outputs(s)


def _tokens(s):
    """Keys and values [B, H, T, D] in 32 bits: the pages in the order of the table, with each
    sequence's window rows in their places."""
    c = s["case"]
    P, G, R = c["P"], c["G"], c["R"]
    table, T = s["table"].long(), s["lens"].long()
    kc, vc, ks, vs = _views(s["pages"], c)
    B, np_ = table.shape
    nq = T // R * R
    t = torch.arange(np_ * P, device="cuda")
    first = t // G * G                                 # the block's first token says where its scale is
    live = t[None] < nq[:, None]
    w = (t[None] - nq[:, None]).clamp(0, R - 1)
    b = torch.arange(B, device="cuda")[:, None]
    got = []
    for code, scale, win in ((kc, ks, s["k_win"]), (vc, vs, s["v_win"])):
        x = _decode(code[table], c["fmt"]).transpose(2, 3).flatten(1, 2)              # [B, T, H, D]
        x *= scale[table[:, first // P], :, ((first % P) // G)[None]][..., None]
        got.append(torch.where(live[..., None, None], x, win[b, w].float()).transpose(1, 2))
    return got


def _run_attend(s):
    c = s["case"]
    B, n, Hq, H, D = c["B"], c["n"], c["Hq"], c["Hkv"], c["D"]
    k, v = _tokens(s)
    q = s["q"].float().view(B, n, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, Hq // H * n, D)
    x = (q @ k.transpose(2, 3)).view(B, H, Hq // H, n, -1) / math.sqrt(D)
    t = torch.arange(k.shape[2], device="cuda")
    end = s["lens"].long()[:, None]                    # the first token that a query does not see
    if c["op"] == "attend":
        end = end - n + 1 + torch.arange(n, device="cuda")[None]
    x = x.masked_fill_((t >= end[..., None])[:, None, None], -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1)
    o = (x.view(B, H, Hq // H * n, -1) @ v).view(B, H, Hq // H, n, D) / total[..., None]
    return o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D).to(torch.bfloat16)


def run(s):
    if own:
        return _run_own(s)
    return _run_append(s) if s["case"]["op"] == "append" else _run_attend(s)


# ------------------------------------------------------------------------- work and truth

def work(case):
    """Each input read once and each output written once; sequences count with their mean length."""
    B, n, Hq, H, D = (case[k] for k in ("B", "n", "Hq", "Hkv", "D"))

    def mean(most):  # of _lengths(): uniform in the logarithm between most / 64 and most
        if not case["ragged"] or most < 2:
            return most
        lo = max(1, most // 64)
        return ((most - lo) / math.log(most / lo) * (B - 1) + most) / B if most > lo else most
    if case["op"] == "append":
        tok = B * mean(case["n"])
        row = 2 * D * (2 * Hq + 2 * H) + 2 * H * D + 4 * case["rot"]  # q, k, v in; q, codes out; the angle's row
        return dict(bytes=tok * row + tok * H * 8 / case["G"], flops=tok * ((Hq + H) * 3 * case["rot"] + 2 * H * D * 3))
    T = mean(case["T"])
    seen = T if case["op"] == "cross" else max(1.0, T - (n - 1) / 2)
    return dict(bytes=B * T * H * (2 * D + 8 / case["G"]) + 2 * 2 * B * n * Hq * D, flops=4.0 * B * n * seen * Hq * D)


def _table(fmt):
    """Value of every byte, from the format's fields."""
    v = np.arange(256)
    if fmt == INT8:
        return torch.from_numpy(np.where(v < 128, v, v - 256).astype(np.float64)).cuda()
    man, bias = (3, 7) if fmt == E4M3 else (2, 15)
    e, m = (v & 127) >> man, (v & ((1 << man) - 1)) / (1 << man)
    x = np.where(e == 0, m * 2.0 ** (1 - bias), (1 + m) * 2.0 ** (e - bias))
    return torch.from_numpy(np.where(v < 128, x, -x)).cuda()


def exact(case, seed):
    if case["op"] != "append" and 4.0 * case["B"] * case["n"] * case["T"] * case["Hq"] * case["D"] > 6e12:
        return None
    s = prepare(case, seed)
    B, n, Hq, H, D, P, G, R = (case[k] for k in ("B", "n", "Hq", "Hkv", "D", "P", "G", "R"))
    T, new = s["lens0"].tolist(), s["n"].tolist()
    if case["op"] == "append":
        rot, half = case["rot"], case["rot"] // 2

        def turned(x, b):  # pairs as complex numbers, turned by the table's angle
            cs = s["cos_sin"][T[b]:T[b] + new[b]].double()
            z = torch.complex(cs[:, None, :half].contiguous(), cs[:, None, half:].contiguous())
            y = x.double().clone()
            pairs = y[..., :rot].unflatten(-1, (2, half)).transpose(-1, -2) if case["halves"] else y[..., :rot].unflatten(-1, (half, 2))
            w = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
            y[..., :rot] = (w.transpose(-1, -2) if case["halves"] else w).flatten(-2)
            return y
        q = s["q_out"].double()
        win = [s["k_win"].double(), s["v_win"].double()]
        for b in range(B):
            q[b, :new[b]] = turned(s["q"][b, :new[b]], b)
            end, base = T[b] + new[b], (T[b] + new[b]) // R * R
            for w, x in zip(win, (turned(s["k"][b, :new[b]], b), s["v"][b, :new[b]].double())):
                t0 = max(base, T[b])
                w[b, t0 - base:end - base] = x[t0 - T[b]:]
        # codes and scales come after the keys' rounding to 16 bits, so they have no value of their own in 64
        return dict(q=q, k_codes=None, v_codes=None, k_scales=None, v_scales=None, k_win=win[0], v_win=win[1], lens=None)
    byte = _table(case["fmt"])
    kc, vc, ks, vs = _views(s["pages"], case)
    out = torch.zeros(B, n, Hq, D, dtype=torch.float64, device="cuda")
    for b in range(B):
        nq = T[b] // R * R
        t = torch.arange(nq, device="cuda")
        page, home = s["table"][b].long()[t // P], s["table"][b].long()[t // G * G // P]
        slot = t // G * G % P // G
        for h in range(H):
            k = torch.cat([byte[kc[page, h, t % P].long()] * ks[home, h, slot].double()[:, None], s["k_win"][b, :T[b] - nq, h].double()])
            v = torch.cat([byte[vc[page, h, t % P].long()] * vs[home, h, slot].double()[:, None], s["v_win"][b, :T[b] - nq, h].double()])
            for r in range(h * (Hq // H), (h + 1) * (Hq // H)):
                x = s["q"][b, :, r].double() @ k.T * D ** -0.5
                if case["op"] == "attend":
                    x += torch.full_like(x, -math.inf).triu(T[b] - n + 1)
                out[b, :, r] = torch.softmax(x, -1) @ v
    return out
