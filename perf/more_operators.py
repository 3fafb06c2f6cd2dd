"""Cases that measure the operators around the attention: the norm and rotation of queries and keys (qk_norm_rope), attention
with a window and first positions that stay visible (attn_decode_kv4_sinks, attn_prefill_sinks), and the decode step of a
batch that shares a prefix (attn_decode_kv4_prefix).

`run` computes a case in plain torch operations, in 32 bits (angles in 64), or, where `own` is set, by the library's
calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TYPE_ID = {"f32": 0, "f16": 1, "bf16": 2}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ---- cases -----------------------------------------------------------------------------------------------------

def listed():
    return [
        # one new token for each of 32 sequences, straight from the fp32 projections: latency
        dict(name="rope_step_f32", op="rope", type="f32", out="f32", H=32, Hkv=8, Dh=128, R=128, neighbours=False,
             base=10000.0, lens="ragged:32:1:4000:1", new=1),
        # the second chunk of two long prompts, a quarter of each head rotated, fp32 projections to 16-bit rows
        dict(name="rope_chunk_f32_bf16", op="rope", type="f32", out="bf16", H=16, Hkv=4, Dh=256, R=64, neighbours=True,
             base=500000.0, lens="120001,9777", new=2047),
        # a packed prompt of eight requests
        dict(name="rope_prompt_bf16", op="rope", type="bf16", out="bf16", H=32, Hkv=8, Dh=128, R=128, neighbours=False,
             base=10000.0, lens="ragged:8:500:8191:2", new=0),
        # the first tokens of a chat, far fewer than the window: latency
        dict(name="sinks_short_f32", op="decode", type="f32", H=32, Hkv=8, Dh=128, page=16, lens="17", Tq=1, window=1024,
             sinks=4),
        # 32 streaming chats, most of them longer than the window
        dict(name="sinks_chats_bf16", op="decode", type="bf16", H=32, Hkv=8, Dh=128, page=64, lens="ragged:32:1:20000:3",
             Tq=1, window=1024, sinks=4),
        # three tokens verified at once, a wide window and a system prompt that stays
        dict(name="sinks_verify_f16", op="decode", type="f16", H=16, Hkv=16, Dh=64, page=32, lens="ragged:24:1:60000:4",
             Tq=3, window=8192, sinks=100),
        # three tiny prompts: latency
        dict(name="sinks_prompt_tiny_f16", op="prefill", type="f16", H=8, Hkv=2, Dh=64, lens="5,1,329", lq="", window=128,
             sinks=3),
        # requests of ordinary length packed, the second chunk of two of them
        dict(name="sinks_packed_bf16", op="prefill", type="bf16", H=32, Hkv=8, Dh=128, lens="777,2048,1,3301,512,1999",
             lq="777,1024,1,1301,512,1999", window=512, sinks=4),
        # one long prompt
        dict(name="sinks_long_bf16", op="prefill", type="bf16", H=32, Hkv=8, Dh=128, lens="16384", lq="", window=4096,
             sinks=64),
        # four answers to one short question: latency
        dict(name="prefix_few_f32", op="prefix", type="f32", H=32, Hkv=8, Dh=128, page=16, prefix=300,
             tails="1,77,20,131", Tq=1),
        # 32 chats under one system prompt that ends inside a page
        dict(name="prefix_chats_bf16", op="prefix", type="bf16", H=32, Hkv=8, Dh=128, page=64, prefix=6001,
             tails="ragged:32:1:1500:5", Tq=1),
        # 48 questions about one book
        dict(name="prefix_book_f32", op="prefix", type="f32", H=64, Hkv=8, Dh=128, page=64, prefix=40001,
             tails="ragged:48:1:600:6", Tq=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "decode", "prefill", "prefix"])
    Dh, Hkv = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8, 16])
    page, B = rng.choice([16, 32, 64, 128, 256]), _log(rng, 1, 48)
    kind = rng.choice(["f32", "f16", "bf16"])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if op == "rope":
        hi = _log(rng, 2, max(2, min(32768, 100_000_000 // (B * (1 + G) * Hkv * Dh))))
        return dict(op=op, type=kind, out=kind if kind != "f32" else rng.choice(["f32", "f16", "bf16"]), H=G * Hkv,
                    Hkv=Hkv, Dh=Dh, R=rng.choice([16, Dh // 4, Dh // 2, Dh, Dh]), neighbours=rng.random() < 0.5,
                    base=rng.choice([10000.0, 500000.0, 1e6]), lens="ragged:%d:1:%d:%d" % (B, hi, rng.randrange(1 << 20)),
                    new=rng.choice([0, 0, 1, 2, 7]))
    if op == "decode":
        hi = _log(rng, 2, max(2, min(131072, 400_000_000 // (B * Hkv * Dh))))
        return dict(op=op, type=kind, H=G * Hkv, Hkv=Hkv, Dh=Dh, page=page,
                    lens="ragged:%d:1:%d:%d" % (B, hi, rng.randrange(1 << 20)), Tq=rng.choice([1, 1, 1, 2, 3, 5]),
                    window=_log(rng, 1, hi), sinks=rng.choice([1, 4, 16, _log(rng, 1, 500)]))
    if op == "prefill":
        kind, G, B = rng.choice(["f16", "bf16"]), rng.choice([1, 2, 3, 4, 8]), _log(rng, 1, 12)
        Hkv = rng.choice([1, 2, 4, 8])
        hi = _log(rng, 2, min(8192, int((8192 * 8192 * 32 * 128 / (B * G * Hkv * Dh)) ** 0.5)))
        lens = [rng.randint(1, hi) for _ in range(B)]
        lq = [n if rng.random() < 0.7 else rng.randint(1, n) for n in lens]
        return dict(op=op, type=kind, H=G * Hkv, Hkv=Hkv, Dh=Dh, lens=",".join(map(str, lens)),
                    lq=",".join(map(str, lq)), window=_log(rng, 1, hi), sinks=rng.choice([1, 4, 16, _log(rng, 1, 500)]))
    Tq = rng.choice([1, 1, 1, 2, 3, 5])
    most = 40000 * 48 * 64 * 128 // (B * Tq * G * Hkv * Dh)  # pairs of the largest listed case
    return dict(op=op, type=kind, H=G * Hkv, Hkv=Hkv, Dh=Dh, page=page,
                prefix=_log(rng, 1, max(1, min(65536, most // 2, 200_000_000 // (Hkv * Dh)))),
                tails="ragged:%d:1:%d:%d" % (B, _log(rng, 1, max(1, min(2000, most // 2, 100_000_000 // (B * Hkv * Dh)))),
                                             rng.randrange(1 << 20)), Tq=Tq)


def lens_of(text):
    """Lengths as a case gives them: a list, or ragged:count:least:most:seed."""
    if not text.startswith("ragged:"):
        return [int(n) for n in text.split(",")]
    count, lo, hi, seed = (int(n) for n in text.split(":")[1:])
    r = random.Random(seed)
    return [r.randint(lo, hi) for _ in range(count)]


def _news(case, lens):
    """New tokens of each sequence: all of it, or the last few."""
    return [min(case["new"], n) if case["new"] else n for n in lens]


def _visible(lq, lk, window, sinks):
    """Keys that lq queries at the end of lk keys see, in all."""
    pos = torch.arange(lk - lq, lk, dtype=torch.int64)
    seen = (pos + 1).clamp(min=0)
    if window:
        seen = seen.clamp(max=window) + (seen - window).clamp(min=0, max=sinks)
    return int(seen.sum())


def work(case):
    s, H, Hkv, Dh = SIZE[case["type"]], case["H"], case["Hkv"], case["Dh"]
    if case["op"] == "rope":
        n = sum(_news(case, lens_of(case["lens"]))) * (H + Hkv) * Dh
        return {"bytes": n * (s + SIZE[case["out"]]), "flops": 7 * n}
    if case["op"] == "prefill":
        lens = lens_of(case["lens"])
        lq = lens_of(case["lq"] or case["lens"])
        pairs = sum(_visible(a, b, case["window"], case["sinks"]) for a, b in zip(lq, lens))
        return {"bytes": s * Dh * (2 * sum(lq) * H + 2 * sum(lens) * Hkv), "flops": 4 * pairs * H * Dh}
    Tq = case["Tq"]
    if case["op"] == "decode":
        lens = lens_of(case["lens"])
        held = sum(min(n, case["window"] + Tq - 1 + case["sinks"]) for n in lens)
        pairs = sum(_visible(Tq, n, case["window"], case["sinks"]) for n in lens)
    else:
        lens = [case["prefix"] + n for n in lens_of(case["tails"])]
        held = case["prefix"] + sum(lens_of(case["tails"]))
        pairs = sum(_visible(Tq, n, 0, 0) for n in lens)
    return {"bytes": 2 * held * Hkv * Dh * 17 // 32 + len(lens) * Tq * H * Dh * (s + 4), "flops": 4 * pairs * H * Dh}


# ---- inputs ----------------------------------------------------------------------------------------------------

def _cumulative(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=DEV)


def _normal(g, n, heads, Dh, kind):
    """[n, heads, Dh]: normal, some channels of a head larger than others, as keys are."""
    x = torch.randn(n, heads, Dh, generator=g, device=DEV)
    return (x * (0.5 + 1.5 * torch.rand(heads, Dh, generator=g, device=DEV) ** 4)).to(TYPES[kind])


def _fill_cache(g, kv, page, Hkv, Dh):
    """A cache that holds something: normal values of every page, quantized a few pages at a time."""
    some = max(1, (1 << 24) // (page * Hkv * Dh))
    for p in range(0, kv.shape[0], some):
        m = min(some, kv.shape[0] - p)
        for which in (0, 1):
            codes, scale = _quantize(_normal(g, m * page, Hkv, Dh, "bf16").float())
            _place(kv[p:p + m], page, Dh, which, codes.view(m, page, Hkv, Dh), scale.view(m, page, Hkv, Dh // 32))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = dict(case, status=torch.zeros(1, dtype=torch.int32, device=DEV), scale=case["Dh"] ** -0.5)
    H, Hkv, Dh, kind = case["H"], case["Hkv"], case["Dh"], case["type"]
    if case["op"] == "prefix":
        lens = [case["prefix"] + n for n in lens_of(case["tails"])]
    else:
        lens = lens_of(case["lens"])
    st.update(lens_host=lens, B=len(lens), max_len=max(lens), lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    if case["op"] == "rope":
        news = _news(case, lens)
        # queries and keys are parts of one matrix, as a fused projection leaves them
        qkv = _normal(g, sum(news), H + 2 * Hkv, Dh, kind)
        st.update(cu=_cumulative(news), n=sum(news), q=qkv[:, :H], k=qkv[:, H:H + Hkv])
        for w in ("wq", "wk"):  # what a model has learned, near 1
            st[w] = 1 + 0.25 * torch.randn(Dh, generator=g, device=DEV)
        i = torch.arange(case["R"] // 2, dtype=torch.float64, device=DEV)
        st["freq"] = (case["base"] ** (-2 * i / case["R"])).float()
        return st
    if case["op"] == "prefill":
        lq = lens_of(case["lq"] or case["lens"])
        st.update(cu_q=_cumulative(lq), cu_k=_cumulative(lens), nq=sum(lq), nk=sum(lens), max_q=max(lq))
        st["q"] = _normal(g, st["nq"], H, Dh, kind)
        st["k"], st["v"] = _normal(g, st["nk"], 2 * Hkv, Dh, kind).split([Hkv, Hkv], dim=1)
        return st
    page, prefix = case["page"], case.get("prefix", 0)
    # pages in a random order: the prefix's, then each sequence's own, from the block that the prefix ends in
    skip = prefix // page
    need = [-(-prefix // page)] + [max(-(-n // page) - skip, 0) for n in lens]
    st["max_pages"], st["num_pages"] = skip + max(need[1:]), sum(need) + 3
    order = torch.randperm(st["num_pages"], generator=g, device=DEV).to(torch.int32)
    st["prefix_pages"] = order[:need[0]].contiguous()
    block = torch.arange(st["max_pages"], device=DEV)[None] - skip
    at = _cumulative(need)[1:-1].long()[:, None] + block
    # entries of the prefix and behind a sequence are never read
    st["pages"] = order[at.clamp(0, st["num_pages"] - 1)].contiguous()
    st["kv"] = torch.zeros(st["num_pages"], Hkv, page * Dh * 17 // 16, dtype=torch.uint8, device=DEV)
    _fill_cache(g, st["kv"], page, Hkv, Dh)
    st["q"] = _normal(g, st["B"] * case["Tq"], H, Dh, kind)
    return st


# ---- plain forms -----------------------------------------------------------------------------------------------

def _quantize(x):
    """Codes 0..15 and scale bytes of [..., Dh] fp32 in blocks of 32."""
    b = x.unflatten(-1, (-1, 32))
    m, e = torch.frexp(b.abs().amax(-1))  # |x| <= m * 2^e with m in [1/2, 1), and 6 = 3/4 * 2^3
    e = torch.where(m == 0, -120, e - 3 + (m > 0.75).int()).clamp(min=-120)
    a = torch.ldexp(b.abs(), -e[..., None])
    code = torch.where(a <= 2, torch.round(2 * a), torch.where(a <= 4, 2 + torch.round(a), 4 + torch.round(a / 2)))
    code = code.int() + 8 * torch.signbit(b).int()
    return code.flatten(-2).to(torch.uint8), (e + 127).to(torch.uint8)


def _views(kv, page, Dh, which):
    """Codes [pages, Hkv, ...] and scales of the keys (which = 0) or values (1), as views of the cache's bytes."""
    P, H, half, sc = kv.shape[0], kv.shape[1], page * Dh // 2, page * Dh // 32
    codes = kv[:, :, which * half:(which + 1) * half]
    scales = kv[:, :, 2 * half + which * sc:2 * half + (which + 1) * sc]
    if which == 0:
        return codes.view(P, H, page, Dh // 2), scales.view(P, H, page, Dh // 32)
    return codes.view(P, H, page // 4, Dh // 8, 4, 4), scales.view(P, H, page // 4, Dh // 32, 4)


def _place(kv, page, Dh, which, codes, scales):
    """Whole pages' codes [pages, page, Hkv, Dh] and scales into the cache's bytes."""
    c, s = _views(kv, page, Dh, which)
    pairs = codes.unflatten(-1, (-1, 2))
    data, sc = (pairs[..., 0] + 16 * pairs[..., 1]).transpose(1, 2), scales.transpose(1, 2)
    if which:  # four tokens side by side
        data = data.unflatten(2, (-1, 4)).unflatten(-1, (-1, 4)).transpose(3, 4)
        sc = sc.unflatten(2, (-1, 4)).transpose(3, 4)
    c.copy_(data)
    s.copy_(sc)


def _read(kv, page, Dh, which, pg, off):
    """fp32 values [..., Hkv, Dh] of the tokens at page pg, place off."""
    c, s = _views(kv, page, Dh, which)
    if which == 0:
        data, sc = c[pg, :, off], s[pg, :, off]
    else:
        data, sc = c[pg, :, off // 4, :, off % 4].flatten(-2), s[pg, :, off // 4, :, off % 4]
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=kv.device)
    code = torch.stack([data & 15, data >> 4], -1).flatten(-2)
    return table[code.int()].unflatten(-1, (-1, 32)).mul(torch.exp2(sc.float() - 127)[..., None]).flatten(-2)


def _softmax(s, seen):
    """Softmax over the last axis of what is seen; 0 where nothing is."""
    s = s.masked_fill(~seen, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=torch.finfo(s.dtype).min))
    return p / p.sum(-1, keepdim=True).clamp(min=torch.finfo(s.dtype).tiny)


def _seen(pos, j, window, sinks):
    """Which of the keys at j the query at pos sees, pos and j shaped alike but for the last axis of pos."""
    seen = j <= pos[..., None]
    return seen & ((j > pos[..., None] - window) | (j < sinks)) if window else seen


def _rotate(x, cos, sin, R, neighbours):
    """x [n, heads, Dh] by the angles of cos and sin [n, 1, R/2]."""
    y = x.clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if neighbours else (slice(0, R // 2), slice(R // 2, R))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _plain_rope(st):
    cu = st["cu"].long()
    tok = torch.arange(st["n"], device=DEV)
    seq = torch.searchsorted(cu, tok, right=True) - 1
    pos = st["lens"].long()[seq] - cu[seq + 1] + tok
    angle = (pos.double()[:, None] * st["freq"].double())[:, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    out = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        out.append(_rotate(x, cos, sin, st["R"], st["neighbours"]).to(TYPES[st["out"]]))
    return out


def _places(st, j):
    """Page and place of the positions j [B, n] of each sequence."""
    return st["pages"].long().gather(1, j // st["page"]), j % st["page"]


def _grouped_queries(st):
    """[B, Hkv, Tq * G, Dh] fp32."""
    B, Tq, H, Hkv, Dh = (st[n] for n in ("B", "Tq", "H", "Hkv", "Dh"))
    return st["q"].float().view(B, Tq, Hkv, H // Hkv, Dh).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, Dh)


def _ungrouped(st, y):
    B, Tq, H, Hkv, Dh = (st[n] for n in ("B", "Tq", "H", "Hkv", "Dh"))
    return y.view(B, Hkv, Tq, H // Hkv, Dh).permute(0, 2, 1, 3, 4).reshape(B * Tq, H, Dh)


def _plain_decode(st):
    B, Tq, H, Hkv, Dh, page = (st[n] for n in ("B", "Tq", "H", "Hkv", "Dh", "page"))
    lens = st["lens"].long()[:, None]
    # the first positions and the window's, which begins behind them
    first = (lens - Tq - st["window"] + 1).clamp(min=min(st["sinks"], st["max_len"]))
    head = torch.arange(min(st["sinks"], st["max_len"]), device=DEV).expand(B, -1)
    j = torch.cat([head, first + torch.arange(min(st["window"] + Tq - 1, st["max_len"]), device=DEV)], 1)
    pg, off = _places(st, torch.where(j < lens, j, 0))
    k, v = (_read(st["kv"], page, Dh, which, pg, off).transpose(1, 2).contiguous() for which in (0, 1))
    s = torch.matmul(_grouped_queries(st), k.transpose(2, 3).contiguous()) * st["scale"]
    pos = lens - Tq + torch.arange(Tq, device=DEV)
    seen = _seen(pos, j[:, None], st["window"], st["sinks"]).repeat_interleave(H // Hkv, 1)[:, None]
    return _ungrouped(st, torch.matmul(_softmax(s, seen), v))


def _padded(x, cu, lens, L):
    """Packed [n, heads, Dh] as fp32 [B, heads, L, Dh], and the mask [B, L] of what is there."""
    j = torch.arange(L, device=DEV)
    there = j < lens[:, None]
    at = torch.where(there, cu[:-1, None] + j, 0)
    return torch.where(there[:, :, None, None], x.float()[at], 0.0).transpose(1, 2).contiguous(), there


def _plain_prefill(st):
    H, Hkv, Dh, L, Lq = st["H"], st["Hkv"], st["Dh"], st["max_len"], st["max_q"]
    cq, ck = st["cu_q"].long(), st["cu_k"].long()
    nq, nk = cq[1:] - cq[:-1], ck[1:] - ck[:-1]
    q, there = _padded(st["q"], cq, nq, Lq)
    k, v = _padded(st["k"], ck, nk, L)[0], _padded(st["v"], ck, nk, L)[0]
    B = q.shape[0]
    q = q.view(B, Hkv, (H // Hkv) * Lq, Dh)
    s = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(st["scale"]).view(B, H, Lq, L)
    pos = (nk - nq)[:, None] + torch.arange(Lq, device=DEV)
    p = _softmax(s, _seen(pos, torch.arange(L, device=DEV), st["window"], st["sinks"])[:, None])
    del s
    y = torch.matmul(p.view(B, Hkv, -1, L), v).view(B, H, Lq, Dh)
    return y.transpose(1, 2)[there].to(st["q"].dtype)


def _plain_prefix(st):
    B, Tq, H, Hkv, Dh, page, P = (st[n] for n in ("B", "Tq", "H", "Hkv", "Dh", "page", "prefix"))
    lens, G = st["lens"].long()[:, None], H // Hkv
    # the prefix once for all queries, then each sequence's own positions
    j = torch.arange(P, device=DEV)
    pg = st["prefix_pages"].long()[j // page]
    kp, vp = (_read(st["kv"], page, Dh, which, pg, j % page).transpose(0, 1).contiguous() for which in (0, 1))
    jt = P + torch.arange(st["max_len"] - P, device=DEV).expand(B, -1)
    block = torch.where(jt < lens, jt, 0)
    pg, off = _places(st, block)
    kt, vt = (_read(st["kv"], page, Dh, which, torch.where(jt < lens, pg, 0), off).transpose(1, 2).contiguous()
              for which in (0, 1))
    q = _grouped_queries(st)
    rows = q.transpose(0, 1).reshape(Hkv, -1, Dh)
    sp = torch.matmul(rows, kp.transpose(1, 2).contiguous()).view(Hkv, B, Tq * G, P).transpose(0, 1)
    s = torch.cat([sp, torch.matmul(q, kt.transpose(2, 3).contiguous())], 3) * st["scale"]
    del sp
    pos = lens - Tq + torch.arange(Tq, device=DEV)
    seen = _seen(pos, torch.cat([j.expand(B, -1), jt], 1)[:, None], 0, 0).repeat_interleave(G, 1)[:, None]
    p = _softmax(s, seen)
    del s
    yp = torch.matmul(p[..., :P].transpose(0, 1).reshape(Hkv, -1, P), vp).view(Hkv, B, Tq * G, Dh).transpose(0, 1)
    return _ungrouped(st, yp + torch.matmul(p[..., P:].contiguous(), vt))


# ---- the library's calls ---------------------------------------------------------------------------------------

def _own_rope(st, qg):
    n, H, Hkv, Dh, q, k = (st[name] for name in ("n", "H", "Hkv", "Dh", "q", "k"))
    q_out = torch.empty(n, H, Dh, dtype=TYPES[st["out"]], device=DEV)
    k_out = torch.empty(n, Hkv, Dh, dtype=TYPES[st["out"]], device=DEV)
    qg.qk_norm_rope(TYPE_ID[st["type"]], q, q.stride(0), k, k.stride(0), n, st["cu"], st["lens"], st["B"], H, Hkv, Dh,
                    st["wq"], st["wk"], EPS, st["R"], qg.ROPE_NEIGHBOURS if st["neighbours"] else qg.ROPE_HALVES,
                    st["freq"], TYPE_ID[st["out"]], q_out, H * Dh, k_out, Hkv * Dh, st["status"])
    return [q_out, k_out]


def _own_cache(st):
    return st["pages"], st["max_pages"], st["page"], st["num_pages"], st["kv"]


def _own_workspace(st, nbytes):
    if "ws" not in st:  # a program keeps one for its largest call
        st["ws"], st["ws_bytes"] = torch.empty(nbytes(), dtype=torch.uint8, device=DEV), nbytes()
    return st["ws"], st["ws_bytes"]


def _own_decode(st, qg):
    B, Tq, H, Hkv, Dh, window, sinks = (st[n] for n in ("B", "Tq", "H", "Hkv", "Dh", "window", "sinks"))
    ws = _own_workspace(st, lambda: qg.attn_decode_sinks_workspace_bytes(B, Tq, H, Hkv, Dh, st["max_len"], window, sinks))
    y = torch.empty(B * Tq, H, Dh, dtype=torch.float32, device=DEV)
    qg.attn_decode_kv4_sinks(TYPE_ID[st["type"]], st["q"], H * Dh, st["lens"], B, Tq, H, Hkv, Dh, st["scale"], window,
                             sinks, st["max_len"], *_own_cache(st), y, *ws, st["status"])
    return y


def _own_prefill(st, qg):
    q, k, v = st["q"], st["k"], st["v"]
    y = torch.empty(st["nq"], st["H"], st["Dh"], dtype=q.dtype, device=DEV)
    qg.attn_prefill_sinks(TYPE_ID[st["type"]], q, q.stride(0), k, k.stride(0), v, v.stride(0), st["nq"], st["nk"],
                          st["cu_q"], st["cu_k"], st["B"], st["H"], st["Hkv"], st["Dh"], st["scale"], st["window"],
                          st["sinks"], y, st["status"])
    return y


def _own_prefix(st, qg):
    B, Tq, H, Hkv, Dh = (st[n] for n in ("B", "Tq", "H", "Hkv", "Dh"))
    ws = _own_workspace(st, lambda: qg.attn_decode_prefix_workspace_bytes(B, Tq, H, Hkv, Dh, st["max_len"], st["prefix"]))
    y = torch.empty(B * Tq, H, Dh, dtype=torch.float32, device=DEV)
    qg.attn_decode_kv4_prefix(TYPE_ID[st["type"]], st["q"], H * Dh, st["lens"], B, Tq, H, Hkv, Dh, st["scale"],
                              st["max_len"], st["prefix"], st["prefix_pages"], *_own_cache(st), y, *ws, st["status"])
    return y


def run(state):
    if own:
        import routed_moe_matvec_amd as qg
        return {"rope": _own_rope, "decode": _own_decode, "prefill": _own_prefill,
                "prefix": _own_prefix}[state["op"]](state, qg)
    return {"rope": _plain_rope, "decode": _plain_decode, "prefill": _plain_prefill,
            "prefix": _plain_prefix}[state["op"]](state)


# ---- the definition in 64 bits ---------------------------------------------------------------------------------

def _exact_cache(kv, page, Dh, which):
    """[pages, Hkv, page, Dh] in 64 bits, from the bytes and the layout's formulas."""
    t, c = torch.arange(page, device=DEV)[:, None], torch.arange(Dh, device=DEV)[None]
    if which == 0:
        at, sat = t * (Dh // 2) + c // 2, page * Dh + t * (Dh // 32) + c // 32
    else:
        at = page * Dh // 2 + ((t // 4) * (Dh // 8) + c // 8) * 16 + (t % 4) * 4 + (c % 8) // 2
        sat = page * Dh + page * Dh // 32 + ((t // 4) * (Dh // 32) + c // 32) * 4 + t % 4
    nib = (kv[:, :, at] >> (4 * (c % 2)).to(torch.uint8)) & 15
    mag = torch.tensor(E2M1, dtype=torch.float64, device=DEV)[(nib & 7).int()]
    return torch.where(nib >= 8, -mag, mag) * torch.exp2(kv[:, :, sat].double() - 127)


def _exact_attend(q, k, v, scale, window, sinks):
    """One sequence: q [Lq, H, Dh] at the end of k, v [Lk, Hkv, Dh]; a head and a few hundred queries at a time."""
    Lq, H, Dh = q.shape
    Lk, Hkv = k.shape[:2]
    y = torch.zeros(Lq, H, Dh, dtype=torch.float64, device=q.device)
    j = torch.arange(Lk, device=q.device)
    step = max(1, (1 << 27) // max(1, Lk))
    for h in range(H):
        kh, vh = k[:, h * Hkv // H].double().contiguous(), v[:, h * Hkv // H].double().contiguous()
        for i in range(0, Lq, step):
            pos = Lk - Lq + torch.arange(i, min(Lq, i + step), device=q.device)[:, None]
            seen = (j <= pos) & ((j > pos - (window or Lk + Lq)) | (j < sinks))
            s = scale * (q[i:i + step, h].double() @ kh.t().contiguous())
            s = torch.where(seen, s, -math.inf)
            w = torch.where(seen, torch.exp(s - s.amax(1, keepdim=True)), 0.0)
            z = w.sum(1, keepdim=True)
            y[i:i + step, h] = torch.where(z > 0, (w @ vh) / torch.where(z > 0, z, 1.0), 0.0)
    return y


def _exact_rope(st):
    """Each pair of channels as one complex number, turned by the token's angle."""
    pos = torch.cat([torch.arange(n - m, n, dtype=torch.float64, device=DEV)
                     for n, m in zip(st["lens_host"], (st["cu"][1:] - st["cu"][:-1]).tolist())])
    angle = (pos[:, None] * st["freq"].double())[:, None]
    turn, R = torch.polar(torch.ones_like(angle), angle), st["R"]
    out = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        x = x.double()
        u = w.double() * x / torch.sqrt(x.square().sum(-1, keepdim=True) / st["Dh"] + EPS)
        pairs = u[..., :R].unflatten(-1, (-1, 2) if st["neighbours"] else (2, -1))
        if not st["neighbours"]:
            pairs = pairs.transpose(-1, -2)
        turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        if not st["neighbours"]:
            turned = turned.transpose(-1, -2)
        out.append(torch.cat([turned.flatten(-2), u[..., R:]], -1))
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st)
    if case["op"] == "prefill":
        cq, ck = st["cu_q"].tolist(), st["cu_k"].tolist()
        return torch.cat([_exact_attend(st["q"][cq[b]:cq[b + 1]], st["k"][ck[b]:ck[b + 1]], st["v"][ck[b]:ck[b + 1]],
                                        st["scale"], st["window"], st["sinks"]) for b in range(st["B"])])
    out, page, Dh, Tq, P = [], case["page"], case["Dh"], case["Tq"], case.get("prefix", 0)

    def rows(ids, lo, hi):
        """Keys and values of the places lo..hi-1 of the pages ids."""
        held = st["kv"][ids.long()]
        return [_exact_cache(held, page, Dh, which).transpose(1, 2).flatten(0, 1)[lo:hi] for which in (0, 1)]

    shared = rows(st["prefix_pages"], 0, P) if P else None
    for b, n in enumerate(st["lens_host"]):
        k, v = rows(st["pages"][b, P // page:-(-n // page)], P % page, n - P // page * page)
        if P:
            k, v = torch.cat([shared[0], k]), torch.cat([shared[1], v])
        out.append(_exact_attend(st["q"][b * Tq:(b + 1) * Tq], k, v, st["scale"], case.get("window", 0),
                                 case.get("sinks", 0)))
    return torch.cat(out)
