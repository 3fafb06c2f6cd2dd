"""Cases that measure the attention operators: the paged FP4 key/value cache (kv4_append, kv4_gather), single-token
attention over it (attn_decode_kv4) and causal attention over packed prompts (attn_prefill).

`run` computes a case in plain torch operations, in 32 bits, or, where `own` is set, by the library's calls.
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


# ---- cases -----------------------------------------------------------------------------------------------------

def listed():
    return [
        # one new token for each of 32 sequences, straight from the fp32 projections: latency
        dict(name="append_step_f32", op="append", type="f32", Hkv=8, Dh=128, page=16, lens="ragged:32:1:4000:1", new=1),
        # a packed prompt of eight requests entering the cache
        dict(name="append_prompt_bf16", op="append", type="bf16", Hkv=8, Dh=128, page=64, lens="ragged:8:500:8191:2",
             new=0),
        # a short odd prefix of three requests, for the next chunk of their prompts
        dict(name="gather_chunk_f16", op="gather", type="f16", Hkv=2, Dh=64, page=32, lens="77,1,1310", new=0),
        # long prefixes of four requests
        dict(name="gather_long_bf16", op="gather", type="bf16", Hkv=8, Dh=128, page=64, lens="ragged:4:20001:32768:3",
             new=0),
        # the first tokens of one short chat: latency
        dict(name="decode_one_short_f32", op="decode", type="f32", H=32, Hkv=8, Dh=128, page=16, lens="17", Tq=1,
             window=0),
        # sixteen chats of ordinary length
        dict(name="decode_chats_bf16", op="decode", type="bf16", H=32, Hkv=8, Dh=128, page=64,
             lens="ragged:16:1:4096:4", Tq=1, window=0),
        # one request over a book
        dict(name="decode_book_f32", op="decode", type="f32", H=64, Hkv=8, Dh=128, page=64, lens="131001", Tq=1,
             window=0),
        # a full serving batch, grouped-projection width (32768 outputs: 128 heads of 256)
        dict(name="decode_batch_f32", op="decode", type="f32", H=128, Hkv=8, Dh=256, page=128,
             lens="ragged:32:3000:8192:5", Tq=1, window=0),
        # two tokens verified at once, one key head per query head, sliding window
        dict(name="decode_verify_window_f16", op="decode", type="f16", H=16, Hkv=16, Dh=64, page=32,
             lens="ragged:24:1:20000:6", Tq=2, window=4096),
        # three tiny prompts: latency
        dict(name="prefill_tiny_f16", op="prefill", type="f16", H=8, Hkv=2, Dh=64, lens="5,1,129", lq="", window=0),
        # requests of ordinary length packed, the second chunk of two of them
        dict(name="prefill_packed_bf16", op="prefill", type="bf16", H=32, Hkv=8, Dh=128,
             lens="777,2048,1,3301,512,1999", lq="777,1024,1,1301,512,1999", window=0),
        # one long prompt
        dict(name="prefill_long_bf16", op="prefill", type="bf16", H=32, Hkv=8, Dh=128, lens="16384", lq="", window=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "gather", "decode", "decode", "prefill", "prefill"])
    Dh, Hkv = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8, 16])
    page, B = rng.choice([16, 32, 64, 128, 256]), _log(rng, 1, 48)
    kind = rng.choice(["f32", "f16", "bf16"])
    if op in ("append", "gather"):
        hi = _log(rng, 2, max(2, min(32768, 100_000_000 // (B * Hkv * Dh))))
        return dict(op=op, type=kind, Hkv=Hkv, Dh=Dh, page=page,
                    lens="ragged:%d:1:%d:%d" % (B, hi, rng.randrange(1 << 20)),
                    new=rng.choice([0, 0, 1, 2, 7]) if op == "append" else 0)
    if op == "decode":
        G, Tq = rng.choice([1, 2, 3, 4, 5, 8, 16]), rng.choice([1, 1, 1, 2, 3, 5])
        hi = _log(rng, 2, max(2, min(131072, 400_000_000 // (B * Hkv * Dh))))
        return dict(op=op, type=kind, H=G * Hkv, Hkv=Hkv, Dh=Dh, page=page,
                    lens="ragged:%d:1:%d:%d" % (B, hi, rng.randrange(1 << 20)), Tq=Tq,
                    window=rng.choice([0, 0, 0, 1 + rng.randrange(hi)]))
    kind, G, B = rng.choice(["f16", "bf16"]), rng.choice([1, 2, 3, 4, 8]), _log(rng, 1, 12)
    Hkv = rng.choice([1, 2, 4, 8])
    hi = _log(rng, 2, min(8192, int((8192 * 8192 * 32 * 128 / (B * G * Hkv * Dh)) ** 0.5)))
    lens = [rng.randint(1, hi) for _ in range(B)]
    lq = [n if rng.random() < 0.7 else rng.randint(1, n) for n in lens]
    return dict(op=op, type=kind, H=G * Hkv, Hkv=Hkv, Dh=Dh, lens=",".join(map(str, lens)), lq=",".join(map(str, lq)),
                window=rng.choice([0, 0, 0, 1 + rng.randrange(hi)]))


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


def _visible(lq, lk, window):
    """Keys that lq queries at the end of lk keys see, in all."""
    pos = torch.arange(lk - lq, lk, dtype=torch.int64)
    seen = (pos + 1).clamp(min=0)
    return int((seen.clamp(max=window) if window else seen).sum())


def work(case):
    lens, s = lens_of(case["lens"]), SIZE[case["type"]]
    Hkv, Dh = case["Hkv"], case["Dh"]
    if case["op"] in ("append", "gather"):
        n = 2 * sum(_news(case, lens)) * Hkv * Dh
        return {"bytes": n * s + n * 17 // 32, "flops": 2 * n}
    H = case["H"]
    if case["op"] == "decode":
        Tq = case["Tq"]
        held = sum(min(n, case["window"] + Tq - 1) if case["window"] else n for n in lens)
        pairs = sum(_visible(Tq, n, case["window"]) for n in lens)
        return {"bytes": 2 * held * Hkv * Dh * 17 // 32 + len(lens) * Tq * H * Dh * (s + 4),
                "flops": 4 * pairs * H * Dh}
    lq = lens_of(case["lq"] or case["lens"])
    pairs = sum(_visible(a, b, case["window"]) for a, b in zip(lq, lens))
    return {"bytes": s * Dh * (2 * sum(lq) * H + 2 * sum(lens) * Hkv), "flops": 4 * pairs * H * Dh}


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


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    lens = lens_of(case["lens"])
    st = dict(case, lens_host=lens, B=len(lens), max_len=max(lens), status=torch.zeros(1, dtype=torch.int32, device=DEV),
              scale=case["Dh"] ** -0.5)
    Hkv, Dh, kind = case["Hkv"], case["Dh"], case["type"]
    if case["op"] == "prefill":
        lq = lens_of(case["lq"] or case["lens"])
        st.update(cu_q=_cumulative(lq), cu_k=_cumulative(lens), nq=sum(lq), nk=sum(lens), max_q=max(lq))
        # the three lie in one matrix where every token has a query, as a fused projection leaves them
        if lq == lens:
            qkv = _normal(g, st["nk"], case["H"] + 2 * Hkv, Dh, kind)
            st["q"], st["k"], st["v"] = qkv.split([case["H"], Hkv, Hkv], dim=1)
        else:
            st["q"] = _normal(g, st["nq"], case["H"], Dh, kind)
            st["k"], st["v"] = _normal(g, st["nk"], 2 * Hkv, Dh, kind).split([Hkv, Hkv], dim=1)
        return st
    page = case["page"]
    need = [-(-n // page) for n in lens]
    st["max_pages"], st["num_pages"] = max(need), sum(need) + 3
    order = torch.randperm(st["num_pages"], generator=g, device=DEV).to(torch.int32)
    start = (_cumulative(need)[:-1]).long()[:, None] + torch.arange(st["max_pages"], device=DEV)[None]
    st["pages"] = order[start.clamp(max=st["num_pages"] - 1)].contiguous()  # entries behind a sequence are never read
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["kv"] = torch.zeros(st["num_pages"], Hkv, page * Dh * 17 // 16, dtype=torch.uint8, device=DEV)
    if case["op"] == "append":
        news = _news(case, lens)
        st.update(cu=_cumulative(news), n=sum(news), k=_normal(g, sum(news), Hkv, Dh, kind),
                  v=_normal(g, sum(news), Hkv, Dh, kind))
        return st
    # a cache that holds something: normal values of every page, quantized a few pages at a time
    some = max(1, (1 << 24) // (page * Hkv * Dh))
    for p in range(0, st["num_pages"], some):
        m = min(some, st["num_pages"] - p)
        for which in (0, 1):
            codes, scale = _quantize(_normal(g, m * page, Hkv, Dh, "bf16").float())
            _place(st["kv"][p:p + m], page, Dh, which, codes.view(m, page, Hkv, Dh), scale.view(m, page, Hkv, Dh // 32))
    if case["op"] == "gather":
        news = _news(case, lens)
        st.update(cu=_cumulative(news), n=sum(news))
    else:
        st["q"] = _normal(g, st["B"] * case["Tq"], case["H"], Dh, kind)
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


def _write(kv, page, Dh, which, pg, off, codes, scales):
    """Tokens' codes [n, Hkv, Dh] and scales to page pg [n], place off [n]."""
    c, s = _views(kv, page, Dh, which)
    pairs = codes.unflatten(-1, (-1, 2))
    data = pairs[..., 0] + 16 * pairs[..., 1]
    if which == 0:
        c[pg, :, off], s[pg, :, off] = data, scales
    else:
        c[pg, :, off // 4, :, off % 4], s[pg, :, off // 4, :, off % 4] = data.unflatten(-1, (-1, 4)), scales


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


def _packed_places(st):
    """Sequence and position of each packed token, and its page and place in it."""
    cu = st["cu"].long()
    tok = torch.arange(st["n"], device=DEV)
    seq = torch.searchsorted(cu, tok, right=True) - 1
    pos = st["lens"].long()[seq] - cu[seq + 1] + tok
    return st["pages"][seq, pos // st["page"]].long(), pos % st["page"]


def _softmax(s, seen):
    """Softmax over the last axis of what is seen; 0 where nothing is."""
    s = s.masked_fill(~seen, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=torch.finfo(s.dtype).min))
    return p / p.sum(-1, keepdim=True).clamp(min=torch.finfo(s.dtype).tiny)


def _seen(pos, L, window):
    """[..., L]: which of the keys 0..L-1 the query at pos sees."""
    j = torch.arange(L, device=DEV)
    seen = j <= pos[..., None]
    return seen & (j > pos[..., None] - window) if window else seen


def _plain_append(st):
    pg, off = _packed_places(st)
    out = []
    for which, x in ((0, st["k"]), (1, st["v"])):
        _write(st["kv"], st["page"], st["Dh"], which, pg, off, *_quantize(x.float()))
        out.append(_read(st["kv"], st["page"], st["Dh"], which, pg, off).to(x.dtype))
    return out


def _plain_gather(st):
    pg, off = _packed_places(st)
    return [_read(st["kv"], st["page"], st["Dh"], which, pg, off).to(TYPES[st["type"]]) for which in (0, 1)]


def _plain_decode(st):
    B, Tq, H, Hkv, Dh, L, page = (st[n] for n in ("B", "Tq", "H", "Hkv", "Dh", "max_len", "page"))
    j = torch.arange(L, device=DEV)
    inside = j < st["lens"].long()[:, None]
    pg = torch.where(inside, st["pages"].long().gather(1, (j // page).expand(B, L)), 0)
    off = (j % page).expand(B, L)
    k, v = (_read(st["kv"], page, Dh, which, pg, off).transpose(1, 2).contiguous() for which in (0, 1))
    q = st["q"].float().view(B, Tq, Hkv, H // Hkv, Dh).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, Dh)
    s = torch.matmul(q, k.transpose(2, 3).contiguous()) * st["scale"]
    pos = st["lens"].long()[:, None] - Tq + torch.arange(Tq, device=DEV)
    seen = (_seen(pos, L, st["window"])).repeat_interleave(H // Hkv, 1)[:, None]
    y = torch.matmul(_softmax(s, seen), v)
    return y.view(B, Hkv, Tq, H // Hkv, Dh).permute(0, 2, 1, 3, 4).reshape(B * Tq, H, Dh)


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
    seen = _seen((nk - nq)[:, None] + torch.arange(Lq, device=DEV), L, st["window"])[:, None]
    p = _softmax(s, seen)
    del s
    y = torch.matmul(p.view(B, Hkv, -1, L), v).view(B, H, Lq, Dh)
    return y.transpose(1, 2)[there].to(st["q"].dtype)


# ---- the library's calls ---------------------------------------------------------------------------------------

def _own_cache(st):
    return st["pages"], st["max_pages"], st["page"], st["num_pages"], st["kv"]


def _own_gather(st, qg):
    t, Hkv, Dh = st["type"], st["Hkv"], st["Dh"]
    k, v = (torch.empty(st["n"], Hkv, Dh, dtype=TYPES[t], device=DEV) for _ in range(2))
    qg.kv4_gather(TYPE_ID[t], k, Hkv * Dh, v, Hkv * Dh, st["n"], st["cu"], st["lens"], st["B"], Hkv, Dh,
                  *_own_cache(st), st["status"])
    return [k, v]


def _own_append(st, qg):
    Hkv, Dh = st["Hkv"], st["Dh"]
    qg.kv4_append(TYPE_ID[st["type"]], st["k"], Hkv * Dh, st["v"], Hkv * Dh, st["n"], st["cu"], st["lens"], st["B"],
                  Hkv, Dh, *_own_cache(st), st["status"])
    return _own_gather(st, qg)


def _own_decode(st, qg):
    B, Tq, H, Hkv, Dh = (st[n] for n in ("B", "Tq", "H", "Hkv", "Dh"))
    if "ws" not in st:  # a program keeps one for its largest call
        st["ws_bytes"] = qg.attn_decode_workspace_bytes(B, Tq, H, Hkv, Dh, st["max_len"], st["window"])
        st["ws"] = torch.empty(st["ws_bytes"], dtype=torch.uint8, device=DEV)
    y = torch.empty(B * Tq, H, Dh, dtype=torch.float32, device=DEV)
    qg.attn_decode_kv4(TYPE_ID[st["type"]], st["q"], H * Dh, st["lens"], B, Tq, H, Hkv, Dh, st["scale"], st["window"],
                       st["max_len"], *_own_cache(st), y, st["ws"], st["ws_bytes"], st["status"])
    return y


def _own_prefill(st, qg):
    q, k, v = st["q"], st["k"], st["v"]
    y = torch.empty(st["nq"], st["H"], st["Dh"], dtype=q.dtype, device=DEV)
    qg.attn_prefill(TYPE_ID[st["type"]], q, q.stride(0), k, k.stride(0), v, v.stride(0), st["nq"], st["nk"],
                    st["cu_q"], st["cu_k"], st["B"], st["H"], st["Hkv"], st["Dh"], st["scale"], st["window"], y,
                    st["status"])
    return y


def run(state):
    if own:
        import routed_moe_matvec_amd as qg
        return {"append": _own_append, "gather": _own_gather, "decode": _own_decode,
                "prefill": _own_prefill}[state["op"]](state, qg)
    return {"append": _plain_append, "gather": _plain_gather, "decode": _plain_decode,
            "prefill": _plain_prefill}[state["op"]](state)


# ---- the definition in 64 bits ---------------------------------------------------------------------------------

def _exact_values(x):
    """What [..., 32k] stands for once held in 4 bits: the nearest of the sixteen values, the even code on a tie."""
    b = x.double().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    exps = torch.arange(-120, 128, dtype=torch.float64, device=x.device)
    e = exps[torch.searchsorted(6.0 * torch.exp2(exps), amax)]  # the least with amax <= 6 * 2^e
    a, vals = b.abs() / torch.exp2(e), torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(vals, a).clamp(1, 7)
    up, down = vals[hi] - a, a - vals[hi - 1]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
    return (torch.copysign(vals[code], b) * torch.exp2(e)).flatten(-2)


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


def _exact_attend(q, k, v, scale, window):
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
            seen = (j <= pos) & (j > pos - (window or Lk + Lq))
            s = scale * (q[i:i + step, h].double() @ kh.t().contiguous())
            s = torch.where(seen, s, -math.inf)
            top = s.amax(1, keepdim=True) if Lk else s.new_zeros(s.shape[0], 1)
            w = torch.where(seen, torch.exp(s - top), 0.0)
            z = w.sum(1, keepdim=True)
            y[i:i + step, h] = torch.where(z > 0, (w @ vh) / torch.where(z > 0, z, 1.0), 0.0)
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return [_exact_values(st["k"]), _exact_values(st["v"])]
    if case["op"] == "prefill":
        cq, ck = st["cu_q"].tolist(), st["cu_k"].tolist()
        return torch.cat([_exact_attend(st["q"][cq[b]:cq[b + 1]], st["k"][ck[b]:ck[b + 1]], st["v"][ck[b]:ck[b + 1]],
                                        st["scale"], st["window"]) for b in range(st["B"])])
    out, page, Dh = [], case["page"], case["Dh"]
    cu = st["cu"].tolist() if case["op"] == "gather" else None
    for b, n in enumerate(st["lens_host"]):
        held = st["kv"][st["pages"][b, :-(-n // page)].long()]
        k, v = (_exact_cache(held, page, Dh, which).transpose(1, 2).flatten(0, 1)[:n] for which in (0, 1))
        if cu is None:
            out.append(_exact_attend(st["q"][b * case["Tq"]:(b + 1) * case["Tq"]], k, v, st["scale"], case["window"]))
        else:
            m = cu[b + 1] - cu[b]
            out.append((k[n - m:], v[n - m:]))
    if cu is None:
        return torch.cat(out)
    return [torch.cat([o[0] for o in out]), torch.cat([o[1] for o in out])]
