"""Cases for measuring the operators of the attention half of a decoder layer:
rotary positions, appending keys and values to a paged cache with the rotation
on the way, and the attention of new tokens over that cache (one decoded token,
a few drafted ones, whole prompts).

With ``own`` false, run() computes an operator in its plain form (elementary
torch operations in f32; angles, rotations and what an 8-bit code hangs on in
f64); with ``own`` true it makes the library's calls.  exact() is the same
result from the definition in f64, written apart.

The cache.  A sequence's tokens lie in pages of `page` tokens; its row of the
page table names them.  Per page and head, in this order:
    f16    keys [page][dim], values [dim][page]
    Q8_0   keys  int8 codes [page][dim], then f16 scales [dim/32][page]
           values int8 codes [dim][page], then f16 scales [dim/32][page]
Keys and values have a pool each.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5
F16, Q8_0 = 1, 8
TAGS = {"f16": F16, "q8_0": Q8_0}


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # the queries of one decoded token of the 32-head, 128-wide layer (latency)
        dict(name="rope_decode", op="rope", N=1, H=32, D=128, rot=128, layout="half", far=8192, yarn=1.0),
        # a small odd batch far into a stretched context; two thirds of a head turn
        dict(name="rope_partial_far", op="rope", N=37, H=9, D=96, rot=64, layout="interleaved", far=131072, yarn=8.0),
        # eight 512-token prompts, queries and keys side by side: the streaming size
        dict(name="rope_prefill_many", op="rope", N=4096, H=40, D=128, rot=128, layout="half", far=8192, yarn=1.0),
        # one decoded token goes into the cache, its queries turned in the same call
        dict(name="append_decode", op="append", kv="f16", Hq=32, Hk=8, D=128, rot=128, layout="interleaved", page=64,
             seqs=1, new=1, ragged=False, lo=2000, hi=2000, norm=False),
        # drafted tokens of a few sequences of a 64-wide model that norms its heads, 8-bit cache
        dict(name="append_verify_q8", op="append", kv="q8_0", Hq=32, Hk=8, D=64, rot=64, layout="half", page=32,
             seqs=5, new=7, ragged=True, lo=9, hi=700, norm=True),
        # eight 512-token prompts into an empty cache
        dict(name="append_prefill_many", op="append", kv="f16", Hq=32, Hk=8, D=128, rot=128, layout="half", page=64,
             seqs=8, new=512, ragged=False, lo=512, hi=512, norm=False),
        # one decoded token with a short history (latency)
        dict(name="attn_decode_short", op="attn", kv="f16", Hq=32, Hk=8, D=128, page=64, seqs=1, new=1, ragged=False,
             lo=513, hi=513, causal=True, window=0, cap=0.0),
        # one decoded token at the end of a long context
        dict(name="attn_decode_long", op="attn", kv="f16", Hq=32, Hk=8, D=128, page=64, seqs=1, new=1, ragged=False,
             lo=131072, hi=131072, causal=True, window=0, cap=0.0),
        # a serving batch: 64 sequences of very different lengths
        dict(name="attn_decode_batch", op="attn", kv="f16", Hq=32, Hk=8, D=128, page=64, seqs=64, new=1, ragged=False,
             lo=1, hi=8192, causal=True, window=0, cap=0.0),
        # seven drafted tokens of eight sequences verified at once, 8-bit cache
        dict(name="attn_verify_q8", op="attn", kv="q8_0", Hq=32, Hk=8, D=128, page=32, seqs=8, new=7, ragged=False,
             lo=900, hi=4096, causal=True, window=0, cap=0.0),
        # a 512-token chunk of a long prompt
        dict(name="attn_prefill", op="attn", kv="f16", Hq=32, Hk=8, D=128, page=64, seqs=1, new=512, ragged=False,
             lo=8192, hi=8192, causal=True, window=0, cap=0.0),
        # ragged prompts of a 64-wide model with a sliding window, 8-bit cache
        dict(name="attn_prefill_q8_ragged", op="attn", kv="q8_0", Hq=24, Hk=8, D=64, page=16, seqs=5, new=777,
             ragged=True, lo=777, hi=2500, causal=True, window=1024, cap=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn"])
    D = rng.choice([64, 96, 128, 192, 256])
    rot = rng.choice([D, D, D // 2, D // 4])
    layout = rng.choice(["half", "interleaved"])
    if op == "rope":
        H = _log(rng, 1, 64)
        N = max(1, min(_log(rng, 1, 4096), 4096 * 40 * 128 // (H * D)))
        return dict(op=op, N=N, H=H, D=D, rot=rot, layout=layout, far=_log(rng, 100, 131072),
                    yarn=rng.choice([1.0, 1.0, 4.0, 8.0]))
    kv = rng.choice(["f16", "q8_0"])
    Hk = _log(rng, 1, 16)
    Hq = Hk * rng.choice([1, 2, 3, 4, 7, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    seqs, ragged = _log(rng, 1, 64), rng.random() < 0.5
    if op == "append":
        new = max(1, min(_log(rng, 1, 512), 8 * 512 * 48 * 128 // (seqs * (Hq + 2 * Hk) * D)))
        hi = new + min(_log(rng, 1, 2048), (1 << 25) // (seqs * Hk * D))
        return dict(op=op, kv=kv, Hq=Hq, Hk=Hk, D=D, rot=rot, layout=layout, page=page, seqs=seqs, new=new,
                    ragged=ragged, lo=new, hi=hi, norm=rng.random() < 0.5)
    # no more cache than the largest listed case reads, no more products than the prompt chunk
    new = rng.choice([1, 1, rng.randint(2, 16), _log(rng, 17, 1024)])
    seqs = min(seqs, 16) if new > 16 else seqs
    hi = max(1, min(_log(rng, 16, 32768), (1 << 28) // (seqs * Hk * D), 512 * 8192 * 32 * 128 // (seqs * new * Hq * D)))
    new = min(new, hi)
    return dict(op=op, kv=kv, Hq=Hq, Hk=Hk, D=D, page=page, seqs=seqs, new=new, ragged=ragged and new > 1,
                lo=rng.randint(new, hi), hi=hi, causal=rng.random() < 0.9, window=0, cap=rng.choice([0.0, 0.0, 30.0]))


def _spread(n, lo, hi):
    """n whole numbers of lo .. hi, unevenly spread, hi among them."""
    return [lo + int(round((hi - lo) * (((n - 1 - i) * 0.6180339887498949 + 1.0 - 1e-12) % 1.0))) for i in range(n)]


def _tokens(c):
    """Tokens of each sequence, the new ones included, and its new ones."""
    lens = _spread(c["seqs"], c["lo"], c["hi"])
    new = _spread(c["seqs"], 1, c["new"]) if c["ragged"] else [c["new"]] * c["seqs"]
    return lens, new


# ----------------------------------------------------------------- inputs ----
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _freqs(rot, yarn, base=500000.0, context=8192, fast=32.0, slow=1.0):
    """Frequency of every pair, f32; with yarn > 1 the slow ones are stretched."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot)
    if yarn > 1.0:
        at = [rot * math.log(context / (2.0 * math.pi * r)) / (2.0 * math.log(base)) for r in (fast, slow)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
        f = f * (1.0 - ramp) + f / yarn * ramp
    return f.float().cuda()


def _rec(c):
    """Bytes of one page of one head in a pool."""
    return c["page"] * c["D"] * 2 if c["kv"] == "f16" else c["page"] * c["D"] + c["page"] * c["D"] // 16


def _pool_views(c, pool, values):
    """(codes or f16 values, scales or None) of a pool, as views with [pages][heads] in front."""
    page, D, Hk, n = c["page"], c["D"], c["Hk"], c["page"] * c["D"]
    shape = (D, page) if values else (page, D)
    if c["kv"] == "f16":
        return pool.view(torch.float16).view(-1, Hk, *shape), None
    r = _rec(c)
    codes = pool.view(torch.int8).view(-1, Hk, r)[..., :n].unflatten(2, shape)
    return codes, pool.view(torch.float16).view(-1, Hk, r // 2)[..., n // 2:].unflatten(2, (D // 32, page))


def _fill(g, c, pages, values):
    """A pool with the keys (some dims large, as keys have) or values of earlier tokens."""
    pool = torch.empty(pages * c["Hk"] * _rec(c), device="cuda", dtype=torch.uint8)
    a, sc = _pool_views(c, pool, values)
    x = torch.randn(a.shape, generator=g, device="cuda", dtype=torch.float16)
    if not values:
        x[..., ::16] *= 2.0
    if sc is None:
        a.copy_(x)
    else:
        a.copy_((x * 40.0).round_().clamp_(-127.0, 127.0))
        sc.copy_(torch.rand(sc.shape, generator=g, device="cuda") * 0.02 + 0.015)
    return pool


def prepare(case, seed):
    g, c = _gen(seed), case
    if c["op"] == "rope":
        return dict(case=c, X=_randn(g, c["N"], c["H"] * c["D"]), freqs=_freqs(c["rot"], c["yarn"]),
                    mscale=1.0 if c["yarn"] == 1.0 else 0.1 * math.log(c["yarn"]) + 1.0,
                    pos=torch.randint(0, c["far"], (c["N"],), generator=g, device="cuda", dtype=torch.int32))
    lens, new = _tokens(c)
    page, seqs = c["page"], c["seqs"]
    need = [(n + page - 1) // page for n in lens]
    pages = sum(need)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table, at = torch.full((seqs, max(need)), -1, device="cuda", dtype=torch.int32), 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    rows = starts[-1]
    s = dict(case=c, pages=pages, max_pages=max(need), rows=rows, new=new, len_list=lens, start_list=starts,
             table=table, lens=torch.tensor(lens, device="cuda", dtype=torch.int32),
             starts=torch.tensor(starts, device="cuda", dtype=torch.int32) if c["ragged"] else None,
             k=_fill(g, c, pages, False), v=_fill(g, c, pages, True))
    if c["op"] == "attn":
        s["Q"] = 1.5 * _randn(g, rows, c["Hq"] * c["D"])
        return s
    # the projections of the new tokens, side by side as one product leaves them
    s["qkv"] = _randn(g, rows, (c["Hq"] + 2 * c["Hk"]) * c["D"])
    s["freqs"] = _freqs(c["rot"], 1.0)
    if c["norm"]:
        s["q_norm"], s["k_norm"] = 1.0 + 0.1 * _randn(g, c["D"]), 1.0 + 0.1 * _randn(g, c["D"])
    return s


# ------------------------------------------------------------ plain forms ----
def _turn(x, pos, freqs, rot, layout, mscale):
    """x [N][H][D] in f64, the first rot dims of each head turned; f32."""
    a = (pos.double().unsqueeze(1) * freqs.double()).unsqueeze(1)
    cos, sin = torch.cos(a) * mscale, torch.sin(a) * mscale
    y = x.clone()
    if layout == "half":
        u, w = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = u * cos - w * sin, u * sin + w * cos
    else:
        u, w = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = u * cos - w * sin, u * sin + w * cos
    return y.float()


def _plain_rope(s):
    c = s["case"]
    y = _turn(s["X"].view(c["N"], c["H"], c["D"]).double(), s["pos"], s["freqs"], c["rot"], c["layout"], s["mscale"])
    return y.view(c["N"], -1)


def _quantize(x):
    """f32 [..., D] -> int8 codes [..., D] and f16 scales [..., D/32]."""
    b = x.unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True) / 127.0
    inv = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    return torch.round(b * inv).clamp(-128, 127).to(torch.int8).flatten(-2), d.squeeze(-1).half()


def _values(c, pool, values):
    """The pool as the f32 values that it stands for (f16 pools as they are)."""
    a, sc = _pool_views(c, pool, values)
    if sc is None:
        return a
    sc = sc.float()
    return a * (sc.repeat_interleave(32, 2) if values else sc.transpose(2, 3).repeat_interleave(32, 3))


def _plain_append(s):
    c = s["case"]
    D, Hq, Hk, rows, page = c["D"], c["Hq"], c["Hk"], s["rows"], c["page"]
    qkv = s["qkv"].view(rows, Hq + 2 * Hk, D).double()
    qk, v = qkv[:, :Hq + Hk], qkv[:, Hq + Hk:].float()
    if c["norm"]:
        w = torch.cat([s["q_norm"].double().expand(Hq, D), s["k_norm"].double().expand(Hk, D)])
        qk = qk / torch.sqrt(qk.square().mean(2, keepdim=True) + EPS) * w
    starts = s["starts"] if s["starts"] is not None else torch.arange(c["seqs"] + 1, device="cuda") * c["new"]
    row = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(starts[1:].contiguous(), row, right=True)
    at = s["lens"][seq].long() - (starts[seq + 1] - row)
    qk = _turn(qk, at, s["freqs"], c["rot"], c["layout"], 1.0)
    q, k = qk[:, :Hq].reshape(rows, Hq * D), qk[:, Hq:]
    pg, off = s["table"][seq, at // page].long(), at % page
    (ka, ks), (va, vs) = _pool_views(c, s["k"], False), _pool_views(c, s["v"], True)
    if c["kv"] == "f16":
        ka[pg, :, off], va[pg, :, :, off] = k.half(), v.half()
        return {"q": q, "k": ka, "v": va}
    ka[pg, :, off], ks[pg, :, :, off] = _quantize(k)
    va[pg, :, :, off], vs[pg, :, :, off] = _quantize(v)
    return {"q": q, "k": _values(c, s["k"], False), "v": _values(c, s["v"], True)}


def _history(s, b, dtype):
    """Keys and values of sequence b: [heads][len][dim] each."""
    c = s["case"]
    n = s["len_list"][b]
    pg = s["table"][b, :(n + c["page"] - 1) // c["page"]].long()
    out = []
    for pool, values in ((s["k"], False), (s["v"], True)):
        a, sc = _pool_views(c, pool, values)
        a = a[pg].to(dtype)
        if sc is not None:
            w = sc[pg].to(dtype)
            a = a * (w.repeat_interleave(32, 2) if values else w.transpose(2, 3).repeat_interleave(32, 3))
        a = a.permute(1, 0, 3, 2) if values else a.transpose(0, 1)
        out.append(a.reshape(c["Hk"], -1, c["D"])[:, :n].contiguous())
    return out


def _hidden(c, n_new, n, t0, t1):
    """[t1-t0][n]: True where new token t0 + i may not look at key j; None if nowhere."""
    if not c["causal"] and not c["window"]:
        return None
    i = torch.arange(n - n_new + t0, n - n_new + t1, device="cuda").unsqueeze(1)
    j = torch.arange(n, device="cuda").unsqueeze(0)
    hide = j > i
    return hide | (j <= i - c["window"]) if c["window"] else hide


def _plain_attn(s):
    c = s["case"]
    D, Hq, Hk, G = c["D"], c["Hq"], c["Hk"], c["Hq"] // c["Hk"]
    out = torch.empty(s["rows"], Hq, D, device="cuda")
    for b in range(c["seqs"]):
        k, v = _history(s, b, torch.float32)
        t0, n_new, n = s["start_list"][b], s["new"][b], s["len_list"][b]
        q = s["Q"][t0:t0 + n_new].view(n_new, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * n_new, D)
        x = torch.bmm(q, k.transpose(1, 2)) * D ** -0.5
        if c["cap"]:
            x = c["cap"] * torch.tanh(x / c["cap"])
        hide = _hidden(c, n_new, n, 0, n_new)
        if hide is not None and n_new > 1:
            x.view(Hk, G, n_new, n).masked_fill_(hide, -math.inf)
        elif hide is not None and c["window"]:
            x.masked_fill_(hide, -math.inf)
        p = torch.exp(x - x.amax(2, keepdim=True))
        o = torch.bmm(p, v) / p.sum(2, keepdim=True)
        out[t0:t0 + n_new] = o.view(Hk, G, n_new, D).permute(2, 0, 1, 3).reshape(n_new, Hq, D)
    return out.view(s["rows"], Hq * D)


# ---------------------------------------------------- the library's calls ----
def _kept(s, name, make):
    """What the program keeps between calls (outputs, workspaces, descriptions)."""
    if name not in s:
        s[name] = make()
    return s[name]


def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, device="cuda", dtype=dtype)


def _layout(q, c):
    return q.QMM_ROPE_HALF if c["layout"] == "half" else q.QMM_ROPE_INTERLEAVED


def _own_rope(s):
    import gguf_block_quant_qmm_amd as q
    c = s["case"]
    y = _kept(s, "out", lambda: _empty(c["N"], c["H"] * c["D"]))
    q.qmm_rope(s["X"], c["N"], c["H"], c["D"], s["pos"], s["freqs"], c["rot"], y, layout=_layout(q, c),
               mscale=s["mscale"])
    return y


def _cache(q, s):
    c = s["case"]
    cache = _kept(s, "cache", lambda: q.KvCache(s["k"], s["v"], TAGS[c["kv"]], s["pages"], c["page"], c["Hk"], c["D"]))
    batch = _kept(s, "batch", lambda: q.KvBatch(s["table"], s["lens"], c["seqs"], s["max_pages"], c["new"], s["rows"],
                                                starts=s["starts"]))
    return cache, batch


def _own_append(s):
    import gguf_block_quant_qmm_amd as q
    c = s["case"]
    D, Hq, Hk = c["D"], c["Hq"], c["Hk"]
    cache, batch = _cache(q, s)
    out = _kept(s, "out", lambda: _empty(s["rows"], Hq * D))
    qkv, wide = s["qkv"], (Hq + 2 * Hk) * D
    q.qmm_kv_append(cache, batch, qkv[:, Hq * D:], qkv[:, (Hq + Hk) * D:], freqs=s["freqs"], rot=c["rot"],
                    layout=_layout(q, c), Q=qkv, q_heads=Hq, q_out=out, q_norm=s.get("q_norm"), k_norm=s.get("k_norm"),
                    eps=EPS, q_stride=wide, k_stride=wide, v_stride=wide)
    return {"q": out, "k": _values(c, s["k"], False), "v": _values(c, s["v"], True)}


def _own_attn(s):
    import gguf_block_quant_qmm_amd as q
    c = s["case"]
    cache, batch = _cache(q, s)
    out = _kept(s, "out", lambda: _empty(s["rows"], c["Hq"] * c["D"]))
    work = _kept(s, "work", lambda: _empty(q.attention_work_bytes(cache, batch, c["Hq"]), dtype=torch.uint8))
    q.qmm_attention(cache, batch, s["Q"], c["Hq"], out, scale=c["D"] ** -0.5, causal=c["causal"], window=c["window"],
                    softcap=c["cap"], work=work)
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "attn": _own_attn}[op](state)
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn}[op](state)


# ------------------------------------------------------------------- work ----
def work(case):
    c = case
    if c["op"] == "rope":
        n = c["N"] * c["H"]
        return {"bytes": 8 * n * c["D"] + 4 * c["N"] + 2 * c["rot"], "flops": 3 * n * c["rot"]}
    lens, new = _tokens(c)
    rows, D = sum(new), c["D"]
    each = 2.0 if c["kv"] == "f16" else 1.0625
    if c["op"] == "append":
        return {"bytes": 4 * rows * (2 * c["Hq"] + 2 * c["Hk"]) * D + 2 * each * rows * c["Hk"] * D,
                "flops": 3 * rows * (c["Hq"] + c["Hk"]) * c["rot"]}
    seen = pairs = 0
    for n, m in zip(lens, new):
        w = c["window"] or n
        if not c["causal"]:
            seen, pairs = seen + n, pairs + n * m
            continue
        seen += min(n, w + m - 1)
        pairs += sum(min(i + 1, w) for i in range(n - m, n))
    return {"bytes": 2 * each * seen * c["Hk"] * D + 8 * rows * c["Hq"] * D, "flops": 4 * pairs * c["Hq"] * D}


# ------------------------------------------------------------------ exact ----
def _spin(x, pos, s):
    """x [N][H][D] in f64 turned as complex numbers."""
    c, rot = s["case"], s["case"]["rot"]
    a = pos.double().view(-1, 1, 1) * s["freqs"].double().view(1, 1, -1)
    z = torch.polar(torch.full_like(a, s.get("mscale", 1.0)), a)
    part = x[..., :rot]
    if c["layout"] == "half":
        w = torch.complex(part[..., :rot // 2].contiguous(), part[..., rot // 2:].contiguous()) * z
        turned = torch.cat([w.real, w.imag], -1)
    else:
        w = torch.view_as_complex(part.reshape(*part.shape[:-1], rot // 2, 2).contiguous()) * z
        turned = torch.view_as_real(w).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _exact_append(s):
    c = s["case"]
    D, Hq, Hk, page = c["D"], c["Hq"], c["Hk"], c["page"]
    x = s["qkv"].double().view(s["rows"], -1, D)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    if c["norm"]:
        q = q * s["q_norm"].double() * ((q * q).sum(-1, keepdim=True) / D + EPS).rsqrt()
        k = k * s["k_norm"].double() * ((k * k).sum(-1, keepdim=True) / D + EPS).rsqrt()
    place = [(s["len_list"][b] - n + t, b) for b, n in enumerate(s["new"]) for t in range(n)]
    at = torch.tensor([p for p, _ in place], device="cuda")
    q, k = _spin(q, at, s), _spin(k, at, s)
    table = s["table"].tolist()
    pg = torch.tensor([table[b][p // page] for p, b in place], device="cuda")
    off = at % page

    def held(y):
        """What the cache stands for; the codes' definition rounds to f32 at each step."""
        if c["kv"] == "f16":
            return y.float().half().double()
        b = y.float().view(*y.shape[:-1], D // 32, 32)
        d = (b.double().abs().max(-1, keepdim=True).values / 127.0).float()
        inv = torch.where(d > 0, (1.0 / d.double()).float(), torch.zeros_like(d))
        return (torch.round((b.double() * inv.double()).float().double()) * d.half().double()).view(y.shape)

    kk, vv = _values(c, s["k"], False).double(), _values(c, s["v"], True).double()
    kk.permute(0, 2, 1, 3)[pg, off] = held(k)
    vv.permute(0, 3, 1, 2)[pg, off] = held(v)
    return {"q": q.reshape(s["rows"], -1), "k": kk, "v": vv}


def _exact_attn(s):
    c = s["case"]
    D, Hq, Hk = c["D"], c["Hq"], c["Hk"]
    out = torch.zeros(s["rows"], Hq, D, device="cuda", dtype=torch.float64)
    for b in range(c["seqs"]):
        k, v = _history(s, b, torch.float64)
        first, n_new, n = s["start_list"][b], s["new"][b], s["len_list"][b]
        for t0 in range(0, n_new, 128):
            t1 = min(n_new, t0 + 128)
            hide = _hidden(c, n_new, n, t0, t1)
            for h in range(Hq):
                q = s["Q"][first + t0:first + t1, h * D:(h + 1) * D].double()
                x = q @ k[h * Hk // Hq].t() / math.sqrt(D)
                x = c["cap"] * torch.tanh(x / c["cap"]) if c["cap"] else x
                x = x if hide is None else x.masked_fill(hide, -math.inf)
                out[first + t0:first + t1, h] = torch.softmax(x, 1) @ v[h * Hk // Hq]
    return out.view(s["rows"], Hq * D)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _spin(s["X"].double().view(case["N"], case["H"], case["D"]), s["pos"], s).reshape(case["N"], -1)
    return _exact_append(s) if case["op"] == "append" else _exact_attn(s)
