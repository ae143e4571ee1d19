"""Cases for measuring the operators of a sparse feed-forward block: the norms
around the block, the router, and the routed experts' products on GGUF
block-quantized weights.

With ``own`` false, run() computes an operator in its plain form (elementary
torch operations in f32, in f64 where a choice or a rounding border hangs on
the last bits); with ``own`` true it makes the library's calls.  exact() is
the same result from the definition in f64, with a decoder of its own.
"""
from __future__ import annotations

import math

import torch

own = False

Q4_0, Q4_1, Q8_0, Q4_K, Q5_K, Q6_K = 2, 3, 8, 12, 13, 14
TAGS = {"Q4_0": Q4_0, "Q4_1": Q4_1, "Q8_0": Q8_0, "Q4_K": Q4_K, "Q5_K": Q5_K, "Q6_K": Q6_K}
BLOCK = {Q4_0: (32, 18), Q4_1: (32, 20), Q8_0: (32, 34), Q4_K: (256, 144), Q5_K: (256, 176), Q6_K: (256, 210)}
EPS = 1e-5


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one decoded token of the 4096-wide model: the attention output joins
        # the residual and the next norm follows (latency)
        dict(name="norm_decode", op="norm", N=1, K=4096, post=False, gate="none", q8=False, scale=1.0),
        # an odd width and batch, a norm after the block and a gate per token
        dict(name="norm_odd", op="norm", N=37, K=4099, post=True, gate="token", q8=False, scale=0.22),
        # a 512-token prefill whose next product takes Q8_0 activations
        dict(name="norm_prefill_q8", op="norm", N=512, K=4096, post=True, gate="row", q8=True, scale=1.0),
        # eight 512-token prompts together: the streaming size
        dict(name="norm_prefill_many", op="norm", N=4096, K=4096, post=True, gate="row", q8=False, scale=0.22),
        # one decoded token, 64 experts, softmax scores
        dict(name="route_decode", op="route", N=1, E=64, T=8, scoring="softmax", bias=False, groups=1, keep=1, top=1,
             renorm=True, scale=1.0),
        # a long prefill, 256 experts in 8 groups, sigmoid scores with a balance bias
        dict(name="route_prefill_groups", op="route", N=4096, E=256, T=8, scoring="sigmoid", bias=True, groups=8,
             keep=4, top=2, renorm=True, scale=2.5),
        # one decoded token, two of eight wide experts
        dict(name="swiglu_decode", op="swiglu", dtype="Q4_0", E=8, M=14336, K=4096, N=1, T=2, pad=0),
        # a small ragged batch of a fine-grained model, some of its tokens padding
        dict(name="swiglu_ragged", op="swiglu", dtype="Q6_K", E=60, M=1408, K=2048, N=37, T=4, pad=5),
        # a full prefill dispatch over eight wide experts: the largest
        dict(name="swiglu_prefill", op="swiglu", dtype="Q4_K", E=8, M=14336, K=4096, N=512, T=2, pad=0),
        # one decoded token, the wide experts' way back
        dict(name="down_decode", op="down", dtype="Q6_K", E=8, M=4096, K=14336, N=1, T=2, pad=0, residual=True),
        # seven drafted tokens verified at once, eight of 64 experts each
        dict(name="down_verify", op="down", dtype="Q5_K", E=64, M=4096, K=1024, N=7, T=8, pad=0, residual=True),
        # a full prefill dispatch of the fine-grained model
        dict(name="down_prefill", op="down", dtype="Q8_0", E=64, M=4096, K=1024, N=512, T=8, pad=0, residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "swiglu", "down"])
    if op == "norm":
        q8 = rng.random() < 0.4
        K = _log(rng, 64, 16384)
        K = max(64, K // 32 * 32) if q8 else K
        N = min(_log(rng, 1, 4096), 4096 * 4096 // K)
        return dict(op=op, N=N, K=K, post=rng.random() < 0.5, gate=rng.choice(["none", "row", "token"]), q8=q8,
                    scale=rng.choice([1.0, 0.22]))
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * max(4, _log(rng, 8, 512) // groups)
        keep = rng.randint(1, groups)
        T = rng.randint(1, min(16, keep * (E // groups)))
        return dict(op=op, N=_log(rng, 1, 4096), E=E, T=T, scoring=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, keep=keep, top=rng.choice([1, 2]),
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))
    name = rng.choice(sorted(TAGS))
    bs = BLOCK[TAGS[name]][0]
    E, T, N = _log(rng, 4, 128), rng.randint(1, 8), _log(rng, 1, 512)
    T = min(T, E)
    K = max(bs, _log(rng, 256, 14336) // bs * bs)
    M = _log(rng, 64, 14336)
    # no more weights or products than the largest listed case
    M = max(1, min(M, 8 * 14336 * 4096 // (E * K), 512 * 2 * 14336 * 4096 // (N * T * K)))
    c = dict(op=op, dtype=name, E=E, M=M, K=K, N=N, T=T, pad=rng.randint(0, N // 4))
    if op == "down":
        c["residual"] = rng.random() < 0.5
    return c


# ----------------------------------------------------------------- inputs ----
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _uniform(g, lo, hi, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32) * (hi - lo) + lo


def _f16(v):
    return v.half().unsqueeze(-1).view(torch.uint8)


def _blob(g, tag, rows, K):
    """Random GGUF blocks of rows x K weights as a flat byte tensor."""
    bs, bb = BLOCK[tag]
    n = rows * (K // bs)
    raw = torch.randint(0, 256, (n, bb), generator=g, device="cuda", dtype=torch.uint8)
    if tag == Q4_0:
        raw[:, 0:2] = _f16(_uniform(g, 0.005, 0.05, n))
    elif tag == Q4_1:
        d = _uniform(g, 0.005, 0.05, n)
        raw[:, 0:2] = _f16(d)
        raw[:, 2:4] = _f16(-d * _uniform(g, 6.0, 9.0, n))
    elif tag == Q8_0:
        raw[:, 0:2] = _f16(_uniform(g, 0.002, 0.02, n))
    elif tag in (Q4_K, Q5_K):
        raw[:, 0:2] = _f16(_uniform(g, 5e-4, 2e-3, n))
        raw[:, 2:4] = _f16(_uniform(g, 5e-4, 2e-3, n))
    else:
        raw[:, 192:208] = torch.randint(-64, 64, (n, 16), generator=g, device="cuda", dtype=torch.int8).view(torch.uint8)
        raw[:, 208:210] = _f16(_uniform(g, 2e-4, 1e-3, n))
    return raw.reshape(-1)


def prepare(case, seed):
    g, c = _gen(seed), case
    if c["op"] == "norm":
        N, K = c["N"], c["K"]
        s = dict(case=c, block=3.0 * _randn(g, N, K), residual=_randn(g, N, K), w_pre=1.0 + 0.1 * _randn(g, K),
                 w_post=1.0 + 0.1 * _randn(g, K) if c["post"] else None,
                 gate={"none": lambda: None, "row": lambda: _uniform(g, 0.1, 1.0, K),
                       "token": lambda: _uniform(g, 0.1, 1.0, N, K)}[c["gate"]]())
        return s
    if c["op"] == "route":
        # logits of a trained router: a few experts stand out, and some are
        # liked by every token
        E = c["E"]
        return dict(case=c, logits=1.5 * _randn(g, c["N"], E) + 0.5 * _randn(g, E),
                    bias=0.05 * _randn(g, E) if c["bias"] else None)
    tag, E, M, K, N, T = TAGS[c["dtype"]], c["E"], c["M"], c["K"], c["N"], c["T"]
    pick = _randn(g, N, E) + 0.5 * _randn(g, E)
    score, ids = torch.topk(pick, T, dim=1)
    ids = ids.to(torch.int32)
    if c["pad"]:
        ids[N - c["pad"]:] = -1  # padding tokens go to no expert
    live = ids[ids >= 0]
    s = dict(case=c, ids=ids.contiguous(), most=int(torch.bincount(live.long(), minlength=E).max()) if live.numel() else 1)
    if c["op"] == "swiglu":
        s.update(gate=_blob(g, tag, E * M, K), up=_blob(g, tag, E * M, K), X=_randn(g, N, K))
    else:
        s.update(w=_blob(g, tag, E * M, K), weights=torch.softmax(score, dim=1).contiguous(), H=_randn(g, N, T, K),
                 residual=_randn(g, N, M) if c["residual"] else None)
    return s


# ------------------------------------------------------------ plain forms ----
def _half(raw, at):
    return raw[:, at:at + 2].contiguous().view(torch.float16).float()


def _six_bit(s):
    lo, mid, hi = s[:, 0:4], s[:, 4:8], s[:, 8:12]
    sc = torch.cat([lo & 63, (hi & 15) | ((lo >> 6) << 4)], 1)
    mn = torch.cat([mid & 63, (hi >> 4) | ((mid >> 6) << 4)], 1)
    return sc.float(), mn.float()


def _decode(raw, tag):
    """[blocks, bytes] -> [blocks, weights] in f32."""
    n = raw.shape[0]
    if tag == Q8_0:
        return raw[:, 2:].contiguous().view(torch.int8).float() * _half(raw, 0)
    if tag == Q4_0:
        return (torch.cat([raw[:, 2:] & 15, raw[:, 2:] >> 4], 1).float() - 8.0) * _half(raw, 0)
    if tag == Q4_1:
        return torch.cat([raw[:, 4:] & 15, raw[:, 4:] >> 4], 1).float() * _half(raw, 0) + _half(raw, 2)
    if tag == Q6_K:
        ql, qh = raw[:, 0:128].reshape(n, 2, 2, 32), raw[:, 128:192].reshape(n, 2, 1, 32)
        lo = torch.cat([ql & 15, ql >> 4], 2)  # [n, half, group, 32]
        hi = torch.cat([(qh >> k) & 3 for k in (0, 2, 4, 6)], 2)
        q = (lo | (hi << 4)).float() - 32.0
        sc = _half(raw, 208) * raw[:, 192:208].contiguous().view(torch.int8).float()
        return (q.reshape(n, 16, 16) * sc.unsqueeze(-1)).reshape(n, 256)
    sc, mn = _six_bit(raw[:, 4:16])
    qs = raw[:, 16 if tag == Q4_K else 48:].reshape(n, 4, 1, 32)
    q = torch.cat([qs & 15, qs >> 4], 2).reshape(n, 8, 32)
    if tag == Q5_K:
        bit = torch.arange(8, device=raw.device, dtype=torch.uint8).view(1, 8, 1)
        q = q | (((raw[:, 16:48].unsqueeze(1) >> bit) & 1) << 4)
    return (q.float() * (_half(raw, 0) * sc).unsqueeze(-1) - (_half(raw, 2) * mn).unsqueeze(-1)).reshape(n, 256)


def _slot_products(blobs, tag, E, M, K, ids, rows, most):
    """W[ids[s]] @ rows[s] for every slot s and blob; zero where the id is no expert."""
    bs, bb = BLOCK[tag]
    S, ok = ids.numel(), (ids >= 0) & (ids < E)
    if S < E:  # fewer slots than experts: only their weights are decoded
        at = ids.clamp(0, E - 1).long()
        out = [torch.bmm(_decode(b.view(E, -1)[at].reshape(-1, bb), tag).view(S, M, K), rows.unsqueeze(2)).squeeze(2)
               for b in blobs]
        return [torch.where(ok.unsqueeze(1), o, torch.zeros_like(o)) for o in out]
    # slots side by side per expert, `most` places each; place S is empty
    key = torch.where(ok, ids, torch.full_like(ids, E)).long()
    key, order = torch.sort(key, stable=True)
    start = torch.searchsorted(key, torch.arange(E + 1, device=key.device))
    rank = torch.arange(S, device=key.device) - start[key]
    place = torch.full(((E + 1) * most + S,), S, device=key.device, dtype=torch.long)
    place[torch.where(key < E, key * most + rank, E * most + torch.arange(S, device=key.device))] = order
    place = place[:E * most]
    packed = torch.cat([rows, rows.new_zeros(1, K)])[place].view(E, most, K)
    outs = []
    for b in blobs:
        o = rows.new_zeros(S + 1, M)
        o[place] = torch.bmm(packed, _decode(b.view(-1, bb), tag).view(E, M, K).transpose(1, 2)).view(E * most, M)
        outs.append(torch.where(ok.unsqueeze(1), o[:S], torch.zeros_like(o[:S])))
    return outs


def _plain_norm(s):
    c = s["case"]
    t = torch.float64 if c["q8"] else torch.float32  # codes next to a border hang on the last bits
    p = s["block"].to(t)
    if c["post"]:
        p = p / torch.sqrt(p.square().mean(1, keepdim=True) + EPS) * s["w_post"].to(t)
    if s["gate"] is not None:
        p = p * s["gate"].to(t)
    r = (s["residual"].to(t) + c["scale"] * p).float()
    h = r.to(t)
    h = (h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * s["w_pre"].to(t)).float()
    if not c["q8"]:
        return {"r": r, "h": h}
    v = h.view(c["N"], c["K"] // 32, 32)
    d = v.abs().amax(2, keepdim=True) / 127.0
    inv = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    codes = torch.round(v * inv).clamp(-128, 127)
    return {"r": r, "h8": (codes * d.half().float()).view(c["N"], c["K"])}


def _plain_route(s):
    c = s["case"]
    N, E, G = c["N"], c["E"], c["groups"]
    x = s["logits"].double()
    if c["scoring"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    choice = score if s["bias"] is None else score + s["bias"].double()
    if G > 1:
        best = torch.sort(choice.view(N, G, E // G), dim=2, descending=True).values[:, :, :c["top"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        open_ = torch.zeros(N, G, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        choice = torch.where(open_.unsqueeze(2), choice.view(N, G, E // G), torch.full((), -math.inf, device=x.device,
                                                                                       dtype=x.dtype)).view(N, E)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :c["T"]]
    w = torch.gather(score, 1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (w * c["scale"]).float()}


def _plain_swiglu(s):
    c = s["case"]
    N, T, M, K = c["N"], c["T"], c["M"], c["K"]
    rows = s["X"].unsqueeze(1).expand(N, T, K).reshape(N * T, K)
    g, u = _slot_products([s["gate"], s["up"]], TAGS[c["dtype"]], c["E"], M, K, s["ids"].view(-1), rows, s["most"])
    return (g / (1.0 + torch.exp(-g)) * u).view(N, T, M)


def _plain_down(s):
    c = s["case"]
    N, T, M, K = c["N"], c["T"], c["M"], c["K"]
    o, = _slot_products([s["w"]], TAGS[c["dtype"]], c["E"], M, K, s["ids"].view(-1), s["H"].view(N * T, K), s["most"])
    y = (o.view(N, T, M) * s["weights"].unsqueeze(2)).sum(1)
    return y if s["residual"] is None else y + s["residual"]


# ---------------------------------------------------- the library's calls ----
def _kept(s, name, make):
    """A buffer that the program keeps between calls (outputs, workspaces)."""
    if name not in s:
        s[name] = make()
    return s[name]


def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, device="cuda", dtype=dtype)


def _own_norm(s):
    import gguf_block_quant_qmm_amd as q
    c = s["case"]
    N, K = c["N"], c["K"]
    r = _kept(s, "out_r", lambda: _empty(N, K))
    if c["q8"]:
        scales = _kept(s, "out_scales", lambda: _empty(N, K // 32))
        quants = _kept(s, "out_quants", lambda: _empty(N, K, dtype=torch.int8))
        outs = dict(scales=scales, quants=quants)
    else:
        outs = dict(H=_kept(s, "out_h", lambda: _empty(N, K)))
    q.qmm_block_norm(s["residual"], N, K, residual_out=r, block=s["block"], w_post=s["w_post"], gate=s["gate"],
                     gate_stride=K if c["gate"] == "token" else 0, scale=c["scale"], w_pre=s["w_pre"], eps=EPS, **outs)
    if not c["q8"]:
        return {"r": r, "h": outs["H"]}
    return {"r": r, "h8": (quants.view(N, K // 32, 32) * scales.unsqueeze(2)).view(N, K)}


def _own_route(s):
    import gguf_block_quant_qmm_amd as q
    c = s["case"]
    ids = _kept(s, "out_ids", lambda: _empty(c["N"], c["T"], dtype=torch.int32))
    w = _kept(s, "out_w", lambda: _empty(c["N"], c["T"]))
    q.qmm_moe_route(s["logits"], c["N"], c["E"], c["T"], ids, w, bias=s["bias"],
                    scoring=q.QMM_ROUTE_SOFTMAX if c["scoring"] == "softmax" else q.QMM_ROUTE_SIGMOID,
                    groups=c["groups"], topk_groups=c["keep"], group_top=c["top"], renorm=c["renorm"], scale=c["scale"])
    return {"ids": ids, "weights": w}


def _own_swiglu(s):
    import gguf_block_quant_qmm_amd as q
    c = s["case"]
    dims = (TAGS[c["dtype"]], c["E"], c["M"], c["K"], c["N"], c["T"])
    out = _kept(s, "out", lambda: _empty(c["N"], c["T"], c["M"]))
    work = _kept(s, "work", lambda: _empty(q.moe_swiglu_work_bytes(*dims), dtype=torch.uint8))
    q.qmm_moe_swiglu(s["gate"], s["up"], *dims, s["ids"], s["X"], out, work=work)
    return out


def _own_down(s):
    import gguf_block_quant_qmm_amd as q
    c = s["case"]
    dims = (TAGS[c["dtype"]], c["E"], c["M"], c["K"], c["N"], c["T"])
    out = _kept(s, "out", lambda: _empty(c["N"], c["M"]))
    work = _kept(s, "work", lambda: _empty(q.moe_down_work_bytes(*dims), dtype=torch.uint8))
    q.qmm_moe_down(s["w"], *dims, s["ids"], s["weights"], s["H"], out, residual=s["residual"], work=work)
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "route": _own_route, "swiglu": _own_swiglu, "down": _own_down}[op](state)
    return {"norm": _plain_norm, "route": _plain_route, "swiglu": _plain_swiglu, "down": _plain_down}[op](state)


# ------------------------------------------------------------------- work ----
def work(case):
    c = case
    if c["op"] == "norm":
        n, K = c["N"] * c["K"], c["K"]
        read = 8 * n + 4 * K + (4 * K if c["post"] else 0) + {"none": 0, "row": 4 * K, "token": 4 * n}[c["gate"]]
        return {"bytes": read + 4 * n + (n + n // 8 if c["q8"] else 4 * n), "flops": 10 * n}
    if c["op"] == "route":
        return {"bytes": 4 * c["N"] * c["E"] + 8 * c["N"] * c["T"], "flops": 10 * c["N"] * c["E"]}
    bs, bb = BLOCK[TAGS[c["dtype"]]]
    E, M, K, N, T = c["E"], c["M"], c["K"], c["N"] - c["pad"], c["T"]
    touched = E * (1.0 - (1.0 - T / E) ** N)  # experts that some token goes to, on average
    one = touched * M * (K // bs) * bb
    if c["op"] == "swiglu":
        return {"bytes": 2 * one + 4 * N * K + 4 * c["N"] * T * M, "flops": 4 * N * T * M * K}
    return {"bytes": one + 4 * N * T * K + 4 * c["N"] * M * (2 if c["residual"] else 1), "flops": 2 * N * T * M * K}


# ------------------------------------------------------------------ exact ----
def _layout(tag):
    """Per weight j of a block: (byte, shift) of its low bits, (byte, shift) of
    its high bits or None, and the sub-block its scale belongs to."""
    where = []
    for j in range(BLOCK[tag][0]):
        if tag in (Q4_0, Q4_1):
            where.append((BLOCK[tag][1] - 16 + j % 16, 4 * (j // 16), None, 0, 0))
        elif tag == Q8_0:
            where.append((2 + j, 0, None, 0, 0))
        elif tag == Q6_K:
            half, grp, l = j // 128, j % 128 // 32, j % 32
            where.append((64 * half + 32 * (grp % 2) + l, 4 * (grp // 2), 128 + 32 * half + l, 2 * grp, j // 16))
        else:
            sub = j // 32
            base = 16 if tag == Q4_K else 48
            where.append((base + 32 * (sub // 2) + j % 32, 4 * (sub % 2), None if tag == Q4_K else 16 + j % 32, sub, sub))
    return where


def _weights64(raw, tag):
    """Blocks [n, bytes] decoded in f64 by the tables of _layout."""
    dev, where = raw.device, _layout(tag)
    col = [torch.tensor([w[k] if w[k] is not None else 0 for w in where], device=dev) for k in range(5)]
    low = raw.index_select(1, col[0])
    f16 = [raw[:, a].to(torch.int32) + 256 * raw[:, a + 1].to(torch.int32) for a in (0, 2, BLOCK[tag][1] - 2)]
    d = [v.to(torch.int16).view(torch.float16).double().unsqueeze(1) for v in f16]
    if tag == Q8_0:
        return d[0] * ((low.double() + 128.0) % 256.0 - 128.0)
    code = torch.bitwise_and(torch.bitwise_right_shift(low, col[1].to(torch.uint8)), 15).double()
    if where[0][2] is not None:
        top = torch.bitwise_right_shift(raw.index_select(1, col[2]), col[3].to(torch.uint8))
        code = code + 16.0 * torch.bitwise_and(top, 3 if tag == Q6_K else 1).double()
    if tag == Q4_0:
        return d[0] * (code - 8.0)
    if tag == Q4_1:
        return d[0] * code + d[1]
    if tag == Q6_K:
        sub = (raw[:, 192:208].double() + 128.0) % 256.0 - 128.0
        return d[2] * sub.index_select(1, col[4]) * (code - 32.0)
    packed = raw[:, 4:16].to(torch.int64)
    sc, mn = [], []
    for i in range(8):
        if i < 4:
            sc.append(packed[:, i] % 64)
            mn.append(packed[:, 4 + i] % 64)
        else:
            sc.append(packed[:, 4 + i] % 16 + 16 * (packed[:, i - 4] // 64))
            mn.append(packed[:, 4 + i] // 16 + 16 * (packed[:, i] // 64))
    sc, mn = torch.stack(sc, 1).double(), torch.stack(mn, 1).double()
    return d[0] * sc.index_select(1, col[4]) * code - d[1] * mn.index_select(1, col[4])


def _exact_products(blob, tag, E, M, K, ids, rows):
    out = torch.zeros(ids.numel(), M, device="cuda", dtype=torch.float64)
    for e in range(E):
        slots = torch.nonzero(ids == e).view(-1)
        if slots.numel():
            W = _weights64(blob.view(E, -1, BLOCK[tag][1])[e], tag).view(M, K)
            out[slots] = rows[slots].double() @ W.t()
    return out


def _exact_norm(s):
    c = s["case"]

    def unit(v, w):
        return v * w.double() / ((v * v).sum(1) / c["K"] + EPS).sqrt().unsqueeze(1)

    p = s["block"].double()
    p = unit(p, s["w_post"]) if c["post"] else p
    p = p * s["gate"].double() if s["gate"] is not None else p
    r = s["residual"].double() + c["scale"] * p
    h = unit(r.float().double(), s["w_pre"])
    if not c["q8"]:
        return {"r": r, "h": h}
    # the codes' definition rounds to f32 at each step: h, d = amax / 127, 1 / d, v * (1 / d)
    v = h.float().view(-1, 32)
    d = (v.double().abs().max(1, keepdim=True).values / 127.0).float()
    inv = (1.0 / d.double()).float()
    codes = torch.round((v.double() * inv.double()).float().double())
    return {"r": r, "h8": (codes * d.half().double()).view(c["N"], c["K"])}


def _exact_route(s):
    c = s["case"]
    x = s["logits"].double().cpu()
    b = None if s["bias"] is None else s["bias"].double().cpu()
    size = c["E"] // c["groups"]
    score = torch.sigmoid(x) if c["scoring"] == "sigmoid" else torch.softmax(x, 1)
    choice = score if b is None else score + b
    ids = torch.zeros(c["N"], c["T"], dtype=torch.int32)
    for n, row in enumerate(choice.tolist()):
        best = [sum(sorted(row[g * size:(g + 1) * size])[-c["top"]:]) for g in range(c["groups"])]
        keep = sorted(range(c["groups"]), key=lambda g: (-best[g], g))[:c["keep"]]
        some = sorted(e for g in keep for e in range(g * size, (g + 1) * size))
        ids[n] = torch.tensor(sorted(some, key=lambda e: (-row[e], e))[:c["T"]], dtype=torch.int32)
    w = score.gather(1, ids.long())
    w = w / w.sum(1, keepdim=True) if c["renorm"] else w
    return {"ids": ids, "weights": w * c["scale"]}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "norm":
        return _exact_norm(s)
    if c["op"] == "route":
        return _exact_route(s)
    tag, E, M, K, N, T = TAGS[c["dtype"]], c["E"], c["M"], c["K"], c["N"], c["T"]
    ids = s["ids"].view(-1)
    if c["op"] == "swiglu":
        rows = s["X"].repeat_interleave(T, 0)
        g = _exact_products(s["gate"], tag, E, M, K, ids, rows)
        return (g * torch.sigmoid(g) * _exact_products(s["up"], tag, E, M, K, ids, rows)).view(N, T, M)
    o = _exact_products(s["w"], tag, E, M, K, ids, s["H"].view(N * T, K)).view(N, T, M)
    y = torch.einsum("ntm,nt->nm", o, s["weights"].double())
    return y if s["residual"] is None else y + s["residual"].double()
