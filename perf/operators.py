"""What the 4-bit KV cache and the scoring head are measured on.

Three groups of calls, as a serving loop makes them:

``cache``  K and V rows are quantised into a 4-bit cache as they are written (a decode step's one
           row a lane, a batch of prompts) and, ``write`` false, read back as fp16 rows.  Where a
           case writes, the written rows are read back too, so the values they stand for come out.
``attend`` the queries of one decode step (or of a few consecutive tokens a lane) attend over the
           4-bit cache; with ``append`` the step's own K and V rows are written first.
``score``  log probabilities of given tokens under the tied embedding, the entropy of each row's
           distribution and its most probable alternatives, from final-norm outputs.

The cache's format: each K or V row of one (token, head) holds head_dim values in groups of 32;
a group has a scale and a zero point, both fp16, and 4-bit codes c, and its values are
zero + c * scale.  zero is the group's least value, scale its range / 15 rounded towards zero.
"""
import math

import torch

own = False

GROUP = 32
DEV = "cuda"


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of eight lanes: the new token's row of each lane
        dict(name="cache_step", op="cache", write=True, lanes=8, heads=16, hd=128, ctx=2112, rows="one", fill=2048),
        # five prompts of the small block's shape, lengths ragged, one of them empty
        dict(name="cache_ragged", op="cache", write=True, lanes=5, heads=4, hd=64, ctx=640, rows="ragged", fill=513),
        # eight long prompts written at once
        dict(name="cache_prompts", op="cache", write=True, lanes=8, heads=16, hd=128, ctx=2112, rows="full", fill=2048),
        # a cached prefix read back for one lane
        dict(name="read_prefix", op="cache", write=False, lanes=1, heads=16, hd=128, ctx=384, rows="full", fill=256),
        # every lane's prefix read back, ragged
        dict(name="read_lanes", op="cache", write=False, lanes=8, heads=16, hd=128, ctx=4096, rows="ragged", fill=4000),
        # batch 1 at the context of a short chat
        dict(name="attend_short", op="attend", lanes=1, heads=16, q_heads=16, hd=128, ctx=384, n_q=1, window=0, append=True),
        # the long-context batch: eight lanes of about 2048 positions
        dict(name="attend_batch", op="attend", lanes=8, heads=16, q_heads=16, hd=128, ctx=2112, n_q=1, window=0, append=True),
        # five drafted tokens verified at once, shared heads, a sliding window, head_dim 64
        dict(name="attend_verify", op="attend", lanes=3, heads=4, q_heads=12, hd=64, ctx=5000, n_q=5, window=1500, append=False),
        # two very long contexts with shared heads
        dict(name="attend_long", op="attend", lanes=2, heads=8, q_heads=32, hd=128, ctx=65536, n_q=1, window=0, append=False),
        # one step's token: its probability and alternatives
        dict(name="score_step", op="score", n=1, vocab=50257, d=2048, k=5),
        # a prompt of ordinary length
        dict(name="score_prompt", op="score", n=128, vocab=50257, d=2048, k=8),
        # a batch of texts scored at once, an odd number of rows
        dict(name="score_texts", op="score", n=1021, vocab=50257, d=2048, k=3),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache", "attend", "attend", "score"])
    if op == "score":
        return dict(op="score", n=_log_int(rng, 1, 1021), vocab=_log_int(rng, 1000, 50257),
                    d=rng.choice([256, 512, 1024, 2048]), k=rng.randint(0, 16))
    hd = rng.choice([64, 128])
    if op == "cache":
        lanes = rng.randint(1, 8)
        heads = rng.choice([1, 3, 4, 8, 16])
        ctx = _log_int(rng, 16, 2112)
        return dict(op="cache", write=rng.random() < 0.6, lanes=lanes, heads=heads, hd=hd, ctx=ctx,
                    rows=rng.choice(["one", "ragged", "full"]), fill=rng.randint(1, ctx))
    heads = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    lanes = _log_int(rng, 1, 8)
    ctx = _log_int(rng, 16, 65536 * 16 // (lanes * heads) if lanes * heads > 16 else 65536)
    return dict(op="attend", lanes=lanes, heads=heads, q_heads=heads * group, hd=hd, ctx=ctx,
                n_q=rng.choice([1, 1, 1, 2, 3, 5, 8]), window=rng.choice([0, 0, 0, _log_int(rng, 1, ctx)]),
                append=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _quantise(x):
    """x fp16 [..., hd] -> codes (int64 [..., hd], 0..15), scale and zero (fp16 [..., hd / 32]).

    The decisions are made in fp32, step by step as the format defines them."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP).float()
    lo, hi = g.amin(-1), g.amax(-1)
    q = (hi - lo) / 15.0
    scale = q.half()
    # towards zero: one step down where rounding to nearest went up
    up = scale.float() > q
    scale = torch.where(up, (scale.view(torch.int16) - up.to(torch.int16)).view(torch.float16), scale)
    s = scale.float()
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    codes = torch.round((g - lo[..., None]) * inv[..., None]).clamp(0, 15)
    return codes.reshape(x.shape).long(), scale, lo.half()


def _pack(codes):
    """codes [..., hd] -> int32 words [..., hd / 8], element 8j + i in bits 4i of word j."""
    w = codes.reshape(*codes.shape[:-1], codes.shape[-1] // 8, 8) << (4 * torch.arange(8, device=codes.device))
    w = w.sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _params(scale, zero):
    return torch.stack((scale, zero), -1)


def _unpack(words):
    c = (words[..., None] >> (4 * torch.arange(8, device=words.device, dtype=torch.int32))) & 15
    return c.reshape(*words.shape[:-1], words.shape[-1] * 8)


def _kv_rows(shape, gen):
    """K- or V-like rows: N(0, 1) with a few channels that stand off the others."""
    off = torch.randn(shape[-2:], device=DEV, generator=gen)
    off = torch.where(off.abs() > 1.8, off * 2.0, torch.zeros_like(off))
    return (torch.randn(shape, device=DEV, generator=gen) + off).half()


def _empty_cache(case):
    n, h, c, hd = case["lanes"], case["heads"], case["ctx"], case["hd"]
    return (torch.zeros(n, h, c, hd // 8, dtype=torch.int32, device=DEV),
            torch.zeros(n, h, c, hd // GROUP, 2, dtype=torch.float16, device=DEV))


def _filled(case, gen):
    """One tensor's cache (codes, params) with every position written."""
    codes, params = _empty_cache(case)
    for b in range(case["lanes"]):
        c, s, z = _quantise(_kv_rows((case["ctx"], case["heads"], case["hd"]), gen).transpose(0, 1))
        codes[b], params[b] = _pack(c), _params(s, z)
    return codes, params


def _ragged(case):
    """The lengths of a ragged batch's lanes (the seed decides their order): spread up to the fill, one of them 0."""
    most, lanes = min(case["fill"], case["ctx"]), case["lanes"]
    lens = [max(1, most * ((7 * i + 10) % 11 + 1) // 11) for i in range(lanes)]
    return lens if lanes == 1 else lens[:-1] + [0]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    pick = torch.Generator()
    pick.manual_seed(seed)
    st = dict(case)
    if case["op"] == "score":
        n, d, v = case["n"], case["d"], case["vocab"]
        E = (torch.randn(v, d, device=DEV, generator=gen) * 0.02).half()
        y = torch.randn(n, d, device=DEV, generator=gen)
        # rows lean towards a token by varying amounts: flat distributions to peaked ones
        lean = torch.randint(0, v, (n,), device=DEV, generator=gen)
        w = E[lean].float()
        y += torch.rand(n, 1, device=DEV, generator=gen) * 15.0 * w / w.norm(dim=1, keepdim=True)
        targets = torch.where(torch.rand(n, device=DEV, generator=gen) < 0.7, lean,
                              torch.randint(0, v, (n,), device=DEV, generator=gen))
        # a padded row has no token
        targets = torch.where(torch.rand(n, device=DEV, generator=gen) < 0.03, torch.full_like(targets, -1), targets)
        st.update(E=E, y=y, targets=targets.int())
        return st
    lanes, heads, hd, ctx = case["lanes"], case["heads"], case["hd"], case["ctx"]
    if case["op"] == "cache":
        most = min(case["fill"], ctx)
        if case["rows"] == "one":
            lens = [1] * lanes
        elif case["rows"] == "full":
            lens = [most] * lanes
        else:
            lens = [_ragged(case)[i] for i in torch.randperm(lanes, generator=pick).tolist()]
        pos = [int(torch.randint(0, ctx - v + 1, (1,), generator=pick)) for v in lens]
        n = sum(lens)
        cu = [0]
        for v in lens:
            cu.append(cu[-1] + v)
        st.update(n=n, lens=lens, pos=torch.tensor(pos, dtype=torch.int32, device=DEV),
                  cu=torch.tensor(cu, dtype=torch.int32, device=DEV))
        st["lane_of"] = torch.repeat_interleave(torch.arange(lanes, device=DEV), torch.tensor(lens, device=DEV))
        if case["write"]:
            # slices of a fused projection's rows [q | k | v], as a block has them
            st["qkv"] = _kv_rows((n, 3 * heads, hd), gen).reshape(n, 3 * heads * hd)
            st["kc"], st["kp"] = _empty_cache(case)
            st["vc"], st["vp"] = _empty_cache(case)
        else:
            st["kc"], st["kp"] = _filled(case, gen)
            st["vc"], st["vp"] = _filled(case, gen)
        return st
    n_q, qh = case["n_q"], case["q_heads"]
    st["kc"], st["kp"] = _filled(case, gen)
    st["vc"], st["vp"] = _filled(case, gen)
    least = max(1, ctx - ctx // 4)
    lens = torch.randint(least, ctx + 1, (lanes,), generator=pick)
    lens[0] = ctx
    st["lens"] = lens.to(torch.int32).to(DEV)
    st["q"] = torch.randn(lanes * n_q, qh * hd, device=DEV, generator=gen).half()
    if case["append"]:
        m = min(n_q, least)
        st["rows"] = m
        st["kv"] = _kv_rows((lanes * m, 2 * heads, hd), gen).reshape(lanes * m, 2 * heads * hd)
        st["pos"] = st["lens"] - m
    return st


# ------------------------------------------------------------------ the calls

def _values(codes, params):
    """The cache's values in fp32: zero + code * scale."""
    c = _unpack(codes).float()
    c = c.reshape(*c.shape[:-1], c.shape[-1] // GROUP, GROUP)
    p = params.float()
    return (p[..., 1:] + c * p[..., :1]).reshape(*c.shape[:-2], c.shape[-2] * GROUP)


def _where(st, pos, lane_of, n):
    """Each row's (lane, position) of a packed batch of rows."""
    at = torch.arange(n, device=DEV) - st["cu"][lane_of].long()
    return lane_of, pos[lane_of].long() + at


def _plain_write(st, x, codes, params, lane, at):
    c, s, z = _quantise(x)
    codes[lane, :, at] = _pack(c)
    params[lane, :, at] = _params(s, z)


def run(st):
    if own:
        import weight_shared_looped_b200 as tl
    if st["op"] == "score":
        E, y, targets, k, n = st["E"], st["y"], st["targets"], st["k"], st["n"]
        if own:
            logp = torch.empty(n, dtype=torch.float32, device=DEV)
            entropy = torch.empty(n, dtype=torch.float32, device=DEV)
            ids = torch.empty(n, k, dtype=torch.int32, device=DEV)
            top = torch.empty(n, k, dtype=torch.float32, device=DEV)
            work_bytes = tl.tl_score_head_workspace_bytes(n, st["vocab"], st["d"], k)
            space = torch.empty(work_bytes, dtype=torch.uint8, device=DEV)
            tl.tl_score_head(E, y, targets, logp, entropy, ids, top, space)
            return {"logp": logp, "entropy": entropy, "ids": ids, "top": top}
        logits = y @ E.float().t()
        best = logits.amax(1, keepdim=True)
        e = torch.exp(logits - best)
        total = e.sum(1, keepdim=True)
        lse = best + torch.log(total)
        entropy = (torch.log(total) - (e * (logits - best)).sum(1, keepdim=True) / total)[:, 0]
        t = targets.long()
        lp = logits.gather(1, t.clamp(min=0)[:, None])[:, 0] - lse[:, 0]
        logp = torch.where(t >= 0, lp, torch.zeros_like(lp))
        # the order of near-equal logits is decided in 64 bits, ties go to the lowest id
        few = min(st["vocab"], k + 8)
        cand = logits.topk(few, 1).indices.sort(1).values
        z = (E[cand.reshape(-1)].double().reshape(n, few, -1) * y.double()[:, None]).sum(-1)
        order = z.sort(dim=1, descending=True, stable=True).indices[:, :k]
        top = (z.gather(1, order) - lse.double()).float()
        return {"logp": logp, "entropy": entropy, "ids": cand.gather(1, order).int(), "top": top}
    heads, hd = st["heads"], st["hd"]
    if st["op"] == "cache":
        n, w = st["n"], heads * hd
        if own:
            if st["write"]:
                tl.tl_kv_write_int4(st["qkv"][:, w:2 * w], st["qkv"][:, 2 * w:], st["kc"], st["kp"], st["vc"], st["vp"],
                                    st["pos"], st["cu"])
            k = torch.empty(n, w, dtype=torch.float16, device=DEV)
            v = torch.empty(n, w, dtype=torch.float16, device=DEV)
            tl.tl_kv_read_int4(st["kc"], st["kp"], st["vc"], st["vp"], st["pos"], k, v, st["cu"])
            return {"k": k, "v": v}
        lane, at = _where(st, st["pos"], st["lane_of"], n)
        if st["write"]:
            _plain_write(st, st["qkv"][:, w:2 * w].reshape(n, heads, hd), st["kc"], st["kp"], lane, at)
            _plain_write(st, st["qkv"][:, 2 * w:].reshape(n, heads, hd), st["vc"], st["vp"], lane, at)
        k = _values(st["kc"][lane, :, at], st["kp"][lane, :, at])
        v = _values(st["vc"][lane, :, at], st["vp"][lane, :, at])
        return {"k": k.half().reshape(n, w), "v": v.half().reshape(n, w)}
    lanes, n_q, qh, ctx = st["lanes"], st["n_q"], st["q_heads"], st["ctx"]
    if own:
        if st["append"]:
            w = heads * hd
            tl.tl_kv_write_int4(st["kv"][:, :w], st["kv"][:, w:], st["kc"], st["kp"], st["vc"], st["vp"], st["pos"])
        out = torch.empty(lanes * n_q, qh * hd, dtype=torch.float16, device=DEV)
        tl.tl_attention_int4(st["q"], st["kc"], st["kp"], st["vc"], st["vp"], st["lens"], out, n_q=n_q, window=st["window"])
        return out
    if st["append"]:
        m, w = st["rows"], heads * hd
        lane = torch.arange(lanes, device=DEV).repeat_interleave(m)
        at = (st["pos"].long()[:, None] + torch.arange(m, device=DEV)).reshape(-1)
        kv = st["kv"].reshape(lanes * m, 2, heads, hd)
        _plain_write(st, kv[:, 0], st["kc"], st["kp"], lane, at)
        _plain_write(st, kv[:, 1], st["vc"], st["vp"], lane, at)
    K, V = _values(st["kc"], st["kp"]), _values(st["vc"], st["vp"])
    q = st["q"].float().reshape(lanes, n_q, heads, qh // heads, hd).permute(0, 2, 3, 1, 4).reshape(lanes, heads, -1, hd)
    s = (q @ K.transpose(2, 3)).reshape(lanes, heads, qh // heads, n_q, ctx) / math.sqrt(hd)
    me = st["lens"].long()[:, None] - n_q + torch.arange(n_q, device=DEV)
    j = torch.arange(ctx, device=DEV)
    seen = j <= me[..., None]
    if st["window"] > 0:
        seen &= j > me[..., None] - st["window"]
    seen = seen[:, None, None]
    s = s.masked_fill(~seen, -math.inf)
    best = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(best == -math.inf, torch.zeros_like(best), best))
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, torch.zeros_like(e))
    o = (p.reshape(lanes, heads, -1, ctx) @ V).reshape(lanes, heads, qh // heads, n_q, hd)
    return o.permute(0, 3, 1, 2, 4).reshape(lanes * n_q, qh * hd).half()


# ------------------------------------------------------------------ what cannot be done without

def work(case):
    if case["op"] == "score":
        n, v, d, k = case["n"], case["vocab"], case["d"], case["k"]
        return {"bytes": 2 * v * d + 4 * n * d + 4 * n * (3 + 2 * k), "flops": 2 * n * v * d}
    heads, hd = case["heads"], case["hd"]
    row = 2 * heads * (hd // 2 + hd // GROUP * 4)      # a token's codes and parameters, K and V
    plain = 2 * heads * hd * 2                         # and its fp16 rows
    if case["op"] == "cache":
        n = sum(_ragged(case)) if case["rows"] == "ragged" else case["lanes"] * (1 if case["rows"] == "one" else case["fill"])
        # written: rows in, cache out, rows out again; read: cache in, rows out
        return {"bytes": n * (2 * plain + row) if case["write"] else n * (plain + row), "flops": 4 * n * heads * hd}
    lanes, ctx, n_q, qh = case["lanes"], case["ctx"], case["n_q"], case["q_heads"]
    keys = ctx if lanes == 1 else ctx - ctx // 8
    if case["window"] > 0:
        keys = min(keys, case["window"] + n_q - 1)
    extra = lanes * n_q * (plain + row) if case["append"] else 0
    return {"bytes": lanes * keys * row + 4 * lanes * n_q * qh * hd + extra,
            "flops": 4 * lanes * n_q * qh * hd * keys}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_group(x):
    """One tensor's rows through the format: x fp16 [..., hd] -> the values (64 bits) it is held as."""
    g = x.double().unflatten(-1, (-1, GROUP))
    lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
    step = ((hi - lo).float() / 15.0).double()
    # the fp16 value next below (or at) step: 11 significant bits, at least 2^-24
    ulp = torch.exp2(torch.floor(torch.log2(step.clamp(min=2.0 ** -14))) - 10)
    step = torch.floor(step / ulp) * ulp
    inv = torch.where(step > 0, (1.0 / step).float(), torch.zeros_like(step, dtype=torch.float32))
    code = torch.round(((g - lo).float() * inv).double()).clamp(0, 15)
    return (lo + code * step).flatten(-2)


def _exact_cache(codes, params):
    at = 4 * torch.arange(8, device=codes.device)
    c = (codes.long().unsqueeze(-1) >> at & 15).flatten(-2).unflatten(-1, (-1, GROUP)).double()
    s, z = params.double().unbind(-1)
    return (z.unsqueeze(-1) + c * s.unsqueeze(-1)).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "score":
        E, y, k = st["E"].double(), st["y"].double(), case["k"]
        out = {"logp": [], "entropy": [], "ids": [], "top": []}
        for r0 in range(0, case["n"], 128):
            z = y[r0:r0 + 128] @ E.t()
            lp = z - torch.logsumexp(z, 1, keepdim=True)
            t = st["targets"][r0:r0 + 128].long()
            got = lp.gather(1, t.clamp(min=0).unsqueeze(1)).squeeze(1)
            out["logp"].append(torch.where(t < 0, 0.0, got))
            out["entropy"].append(-(lp.exp() * lp).sum(1))
            ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
            out["ids"].append(ids.int())
            out["top"].append(lp.gather(1, ids))
        return {name: torch.cat(v) for name, v in out.items()}
    heads, hd = case["heads"], case["hd"]
    if case["op"] == "cache":
        n = st["n"]
        if case["write"]:
            rows = st["qkv"].reshape(n, 3, heads, hd)
            return {"k": _exact_group(rows[:, 1]).reshape(n, -1), "v": _exact_group(rows[:, 2]).reshape(n, -1)}
        got = {"k": [], "v": []}
        for b, m in enumerate(st["lens"]):
            p = int(st["pos"][b])
            got["k"].append(_exact_cache(st["kc"][b, :, p:p + m], st["kp"][b, :, p:p + m]).transpose(0, 1).reshape(m, heads * hd))
            got["v"].append(_exact_cache(st["vc"][b, :, p:p + m], st["vp"][b, :, p:p + m]).transpose(0, 1).reshape(m, heads * hd))
        return {name: torch.cat(v) for name, v in got.items()}
    lanes, n_q, qh = case["lanes"], case["n_q"], case["q_heads"]
    out = torch.zeros(lanes, n_q, heads, qh // heads, hd, dtype=torch.float64, device=DEV)
    q = st["q"].double().reshape(lanes, n_q, heads, qh // heads, hd)
    for b in range(lanes):
        length = int(st["lens"][b])
        K, V = _exact_cache(st["kc"][b], st["kp"][b]), _exact_cache(st["vc"][b], st["vp"][b])
        if case["append"]:
            m = st["rows"]
            kv = _exact_group(st["kv"].reshape(lanes, m, 2, heads, hd)[b])
            K[:, length - m:length], V[:, length - m:length] = kv[:, 0].transpose(0, 1), kv[:, 1].transpose(0, 1)
        for i in range(n_q):
            last = length - n_q + i
            first = max(0, last - case["window"] + 1) if case["window"] > 0 else 0
            if last < 0:
                continue
            ks, vs = K[:, first:last + 1], V[:, first:last + 1]
            p = torch.softmax(torch.einsum("hgd,hjd->hgj", q[b, i], ks) / hd ** 0.5, -1)
            out[b, i] = torch.einsum("hgj,hjd->hgd", p, vs)
    return out.reshape(lanes * n_q, qh * hd)
