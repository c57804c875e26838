"""Measured cases of the cache-bounding operators around the absorbed MLA decode.

Four operators: decode over a sliding window with sink tokens (``window_decode``), the
attention weight that every cached token has received (``attention_mass``), eviction by that
weight (``evict_select`` and ``cache_compact``) and the verification of drafted tokens
(``verify_drafts``). ``run`` computes them in a plain form with elementary torch operations,
or, where ``own`` is true, through the package's entry points.
"""
import math

import torch

own = False

R, DR, BLOCK = 512, 64, 64   # latent and RoPE width and block size of the paged cache


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # window decode: the fp32 cache at the smallest call, one short sequence pair: latency
        dict(name="window_f32_tiny", op="window", dtype="f32", B=2, Sq=1, H=4, r=16, dr=8, block=64, L=64, ragged=False,
             window=24, sinks=4, causal=False, dist="unit"),
        # a LLaMA-2-7B-shaped converted model (32 heads), a short window and a few sinks
        dict(name="window_bf16_h32", op="window", dtype="bf16", B=16, Sq=1, H=32, r=R, dr=DR, block=BLOCK, L=8192,
             ragged=False, window=1024, sinks=4, causal=False, dist="half"),
        # the large decode batch (128 heads, 32K context), a 4K window: the largest call
        dict(name="window_bf16_h128", op="window", dtype="bf16", B=64, Sq=1, H=128, r=R, dr=DR, block=BLOCK, L=32768,
             ragged=False, window=4096, sinks=64, causal=False, dist="latent"),
        # ragged lengths and two causal query tokens per sequence (multi-token prediction)
        dict(name="window_bf16_mtp", op="window", dtype="bf16", B=96, Sq=2, H=128, r=R, dr=DR, block=BLOCK, L=16384,
             ragged=True, window=1500, sinks=4, causal=True, dist="latent"),
        # the 8-bit cache with per-token scales
        dict(name="window_fp8_h128", op="window", dtype="e4m3", B=32, Sq=1, H=128, r=R, dr=DR, block=BLOCK, L=65536,
             ragged=False, window=2048, sinks=4, causal=False, dist="unit"),
        # attention weight: one short sequence (latency), the large bf16 batch, the 8-bit cache
        dict(name="mass_bf16_one", op="mass", dtype="bf16", B=1, Sq=1, H=128, r=R, dr=DR, block=BLOCK, L=777,
             ragged=False, causal=False, dist="unit"),
        dict(name="mass_bf16_h128", op="mass", dtype="bf16", B=64, Sq=1, H=128, r=R, dr=DR, block=BLOCK, L=8192,
             ragged=False, causal=False, dist="unit"),
        dict(name="mass_fp8_ragged", op="mass", dtype="e4m3", B=48, Sq=1, H=128, r=R, dr=DR, block=BLOCK, L=16384,
             ragged=True, causal=False, dist="unit"),
        # eviction: one sequence just over its budget, and a large batch cut to half its length
        dict(name="evict_bf16_one", op="evict", dtype="bf16", B=1, r=R, dr=DR, block=BLOCK, L=1100, ragged=False,
             budget=512, sinks=4, recent=128),
        dict(name="evict_bf16_b64", op="evict", dtype="bf16", B=64, r=R, dr=DR, block=BLOCK, L=8192, ragged=True,
             budget=2048, sinks=4, recent=512),
        # verification: one sequence with one drafted token, and a batch with three
        dict(name="verify_one", op="verify", dtype="f32", B=1, K=1, V=32000, accept=0.5),
        dict(name="verify_b128", op="verify", dtype="f32", B=128, K=3, V=128000, accept=0.7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "mass", "evict", "verify"])
    if op == "verify":
        V = _log(rng, 500, 150000)
        B = min(_log(rng, 1, 128), max(1, 16_000_000 // V))
        return dict(op=op, dtype=rng.choice(["f32", "f32", "bf16"]), B=B, K=rng.randint(1, 5 if V < 80000 else 3), V=V,
                    accept=rng.choice([0.3, 0.6, 0.9]))
    if op == "evict":
        L = _log(rng, 20, 16384)
        budget = max(2, int(L * rng.uniform(0.1, 0.8)))
        sinks = rng.randint(0, min(64, budget // 2))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "e4m3", "f32"]), B=min(_log(rng, 1, 64), max(1, 400_000 // L)),
                    r=R, dr=DR, block=BLOCK, L=L, ragged=rng.random() < 0.5, budget=budget, sinks=sinks,
                    recent=rng.randint(0, budget - sinks))
    dtype = rng.choice(["bf16", "bf16", "bf16", "e4m3", "f32"])
    Sq = rng.choice([1, 1, 2, 3])
    c = dict(op=op, dtype=dtype, Sq=Sq, causal=Sq > 1, ragged=rng.random() < 0.5)
    if dtype == "f32":   # the generic widths
        c.update(r=rng.choice([16, 48, 64, 128]), dr=rng.choice([0, 8, 16]), block=rng.choice([16, 32, 64]),
                 H=rng.randint(1, 16), L=_log(rng, 1, 4096), dist="unit")
        c.update(B=min(_log(rng, 1, 32), max(1, 16384 // c["L"])))
    else:
        c.update(r=R, dr=DR, block=BLOCK, H=rng.choice([8, 16, 20, 32, 48, 64, 96, 128]),
                 L=_log(rng, 1, 32768 if op == "window" else 16384), dist=rng.choice(["unit", "half"]))
        c.update(B=min(_log(rng, 1, 64), max(1, (500_000 if op == "window" else 200_000) // c["L"])))
    if op == "window":
        c.update(window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 33, 64, 130]))
    return c


# ------------------------------------------------------------------------------- inputs
def _blocks(c):
    return (c["L"] + c["block"] - 1) // c["block"]


def _lens(c, g, dev):
    if not c["ragged"]:
        return torch.full((c["B"],), c["L"], dtype=torch.int32, device=dev)
    u = torch.rand(c["B"], generator=g, device=dev, dtype=torch.float64)
    lo = max(1.0, c["L"] / 16)
    return (lo * (c["L"] / lo) ** u).floor().clamp(1, c["L"]).to(torch.int32)


def _normal(g, dev, *shape, std=1.0):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std


def _cache(c, g, dev, blocks):
    """kv_cache, k_rope_cache, kv_scale of `blocks` blocks (the last two None for f32 and bf16)."""
    r, dr, bs = c["r"], c["dr"], c["block"]
    std = {"half": 0.5, "latent": 1.0 / math.sqrt(r)}.get(c.get("dist"), 1.0)
    gain = torch.ones(r + dr, device=dev)
    if c.get("dist") == "latent":   # a few strong channels, as latents have
        gain[torch.randperm(r, generator=g, device=dev)[: max(1, r // 100)]] = 8.0
    if c["dtype"] == "e4m3":
        lat = _normal(g, dev, blocks, bs, r, std=std)
        scale = lat.abs().amax(-1) / 448.0
        codes = (lat / scale.unsqueeze(-1)).to(torch.float8_e4m3fn)
        return codes, _normal(g, dev, blocks, bs, dr, std=std).to(torch.bfloat16), scale
    out = torch.empty(blocks, bs, r + dr, device=dev, dtype=torch.float32 if c["dtype"] == "f32" else torch.bfloat16)
    for i in range(0, blocks, 4096):   # in pieces: the fp32 random numbers of a large pool need room
        n = min(4096, blocks - i)
        out[i:i + n] = _normal(g, dev, n, bs, r + dr, std=std) * gain
    return out, None, None


def _lse(s):
    """The log-sum-exp of every query row, as the decode before this step left it, with the scores in 64 bits."""
    c, outs = s["case"], []
    for b in range(c["B"]):
        n = int(s["lens_host"][b])
        lat, key = _rows(s, s["table"][b, torch.arange(n, device=s["table"].device) // c["block"]].long() * c["block"]
                         + torch.arange(n, device=s["table"].device) % c["block"], torch.float32)
        q = torch.cat([s["q_lat"][b], s["q_rope"][b]], -1).reshape(c["Sq"] * c["H"], -1).float()
        x = (q @ torch.cat([lat, key], -1).T).double() * s["scale"]
        if c["causal"]:
            seen = n - c["Sq"] + 1 + torch.arange(c["Sq"], device=x.device).repeat_interleave(c["H"])
            x = x.masked_fill(torch.arange(n, device=x.device)[None] >= seen[:, None], float("-inf"))
        outs.append(torch.logsumexp(x, -1).float())
    return torch.stack(outs).reshape(c["B"], c["Sq"], c["H"])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    if c["op"] == "verify":
        B, K, V = c["B"], c["K"], c["V"]
        dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
        # the draft model's distribution near the target's, so that a share of the drafts is accepted
        logits = _normal(g, dev, B, K + 1, V, std=3.0)
        s["target"] = torch.softmax(logits, -1).to(dt)
        near = logits[:, :K] + _normal(g, dev, B, K, V, std=2.0 * (1.0 - c["accept"]))
        s["draft"] = torch.softmax(near, -1).to(dt)
        s["tokens"] = (near - torch.log(-torch.log(torch.rand(B, K, V, generator=g, device=dev).clamp(1e-9, 1 - 1e-7)))
                       ).argmax(-1).to(torch.int32)   # one token drawn from each draft distribution
        s["u"] = torch.rand(B, K, generator=g, device=dev)
        s["v"] = torch.rand(B, generator=g, device=dev)
        s["seq_lens"] = torch.randint(K + 1, 32768, (B,), generator=g, device=dev, dtype=torch.int32)
        return s
    nb = _blocks(c)
    s["lens"] = _lens(c, g, dev)
    s["lens_host"] = s["lens"].tolist()
    if c["op"] == "evict":
        nd = (c["budget"] + c["block"] - 1) // c["block"]
        pool = c["B"] * (nb + nd)
        perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
        s["table"] = perm[: c["B"] * nb].reshape(c["B"], nb).contiguous()
        s["dst"] = perm[c["B"] * nb:].reshape(c["B"], nd).contiguous()
        s["kv"], s["kr"], s["ks"] = _cache(c, g, dev, pool)
        # weights as they pile up: a few tokens hold most of it
        s["mass"] = torch.exp(_normal(g, dev, c["B"], nb * c["block"], std=2.0))
        s["mass_out"] = torch.zeros(c["B"], nd * c["block"], device=dev)
        return s
    pool = c["B"] * nb
    s["table"] = torch.randperm(pool, generator=g, device=dev).to(torch.int32).reshape(c["B"], nb).contiguous()
    s["kv"], s["kr"], s["ks"] = _cache(c, g, dev, pool)
    qt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    qstd = 0.5 if c["dist"] == "half" else 1.0
    s["q_lat"] = _normal(g, dev, c["B"], c["Sq"], c["H"], c["r"], std=qstd).to(qt)
    s["q_rope"] = _normal(g, dev, c["B"], c["Sq"], c["H"], c["dr"], std=qstd).to(qt)
    s["scale"] = 1.0 / math.sqrt(192.0 if c["r"] == R else c["r"] + c["dr"])
    if c["op"] == "mass":
        s["lse"] = _lse(s)
        S = nb * c["block"]
        s["mass_in"] = torch.rand(c["B"], S, generator=g, device=dev)
        s["mass"] = torch.zeros(c["B"], S, device=dev)
    return s


# ------------------------------------------------------------------------------- plain forms
def _rows(s, slot, dtype=torch.float32):
    """Latents and RoPE keys of the cache rows `slot`, as numbers."""
    c = s["case"]
    if c["dtype"] == "e4m3":
        lat = s["kv"].reshape(-1, c["r"])[slot].to(dtype) * s["ks"].reshape(-1)[slot].to(dtype).unsqueeze(-1)
        return lat, s["kr"].reshape(-1, c["dr"])[slot].to(dtype)
    x = s["kv"].reshape(-1, c["r"] + c["dr"])[slot].to(dtype)
    return x[..., : c["r"]], x[..., c["r"]:]


def _slots(s, pos):
    """Physical rows of the positions `pos` [B, n] through the block table."""
    bs = s["case"]["block"]
    return s["table"].gather(1, pos // bs).long() * bs + pos % bs


def _seen(s, dev):
    """Tokens that each query row sees: [B, rows, 1]."""
    c = s["case"]
    n = s["lens"].long()[:, None].expand(-1, c["Sq"] * c["H"])
    if c["causal"]:
        n = n - c["Sq"] + 1 + torch.arange(c["Sq"] * c["H"], device=dev)[None] // c["H"]
    return n.unsqueeze(-1)


def _plain_window(s):
    c = s["case"]
    dev, L, T = s["lens"].device, s["lens"].long()[:, None], _blocks(c) * c["block"]
    first = L - c["Sq"] + 1 if c["causal"] else L
    lo = (first - c["window"]).clamp(min=min(c["sinks"], T))   # the windows of all query rows, behind the sinks
    near = lo + torch.arange(min(c["window"] + c["Sq"], T), device=dev)[None]
    far = torch.arange(min(c["sinks"], T), device=dev)[None].expand(c["B"], -1)
    pos = torch.cat([far, near], 1)
    lat, key = _rows(s, _slots(s, pos.clamp(max=T - 1)))
    q = torch.cat([s["q_lat"], s["q_rope"]], -1).reshape(c["B"], c["Sq"] * c["H"], -1).float()
    x = q @ torch.cat([lat, key], -1).transpose(1, 2) * s["scale"]
    n, t = _seen(s, dev), pos[:, None]
    see = (t < n) & (t < L[:, None]) & ((t < c["sinks"]) | (t >= n - c["window"]))
    x = x.masked_fill(~see, float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.masked_fill(m == float("-inf"), 0.0))
    z = p.sum(-1, keepdim=True)
    out = (p @ lat) / z.masked_fill(z == 0, 1.0)
    lse = (m + torch.log(z)).squeeze(-1)
    return {"out": out.to(s["q_lat"].dtype).reshape(s["q_lat"].shape), "lse": lse.reshape(s["q_lat"].shape[:3])}


def _plain_mass(s):
    c = s["case"]
    dev, S = s["lens"].device, s["mass"].shape[1]
    t = torch.arange(S, device=dev)[None].expand(c["B"], -1)
    lat, key = _rows(s, _slots(s, t))
    q = torch.cat([s["q_lat"], s["q_rope"]], -1).reshape(c["B"], c["Sq"] * c["H"], -1).float()
    x = q @ torch.cat([lat, key], -1).transpose(1, 2)
    w = torch.exp(x * s["scale"] - s["lse"].reshape(c["B"], -1, 1))
    w = w.masked_fill(t[:, None] >= _seen(s, dev), 0.0).sum(1)
    s["mass"].copy_(torch.where(t < s["lens"][:, None], s["mass_in"] + w, s["mass"]))
    return {"mass": s["mass"]}


def _plain_evict(s):
    c = s["case"]
    dev, bs = s["lens"].device, c["block"]
    S, L = s["mass"].shape[1], s["lens"].long()[:, None]
    t = torch.arange(S, device=dev)[None].expand(c["B"], -1)
    safe = (t < c["sinks"]) | (t >= L - c["recent"])
    rank = s["mass"].masked_fill(safe, float("inf")).masked_fill(t >= L, float("-inf"))
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, : c["budget"]]
    j = torch.arange(order.shape[1], device=dev)[None]
    count = L.clamp(max=c["budget"])
    kept = order.masked_fill(j >= count, S).sort(1).values
    full = torch.full((c["B"], c["budget"]), -1, dtype=torch.int32, device=dev)
    full[:, : kept.shape[1]] = kept.masked_fill(j >= count, -1).to(torch.int32)
    dst = s["dst"].gather(1, (j // bs).expand(c["B"], -1)).long() * bs + j % bs
    src = torch.where(j < count, _slots(s, kept.clamp(max=S - 1)), dst)   # an entry past the count stays as it is
    for x in (s["kv"], s["kr"], s["ks"]):
        if x is not None:
            x = x.reshape(-1, x.shape[-1]) if x.dim() == 3 else x.reshape(-1)
            x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
            x[dst] = x[src]
    out = s["mass_out"].zero_()
    out[:, : kept.shape[1]] = s["mass"].gather(1, kept.clamp(max=S - 1)).masked_fill(j >= count, 0.0)
    return {"kv": s["kv"], "kr": s["kr"], "ks": s["ks"], "indices": full, "counts": count.squeeze(1).to(torch.int32),
            "mass": out}


def _plain_verify(s):
    c = s["case"]
    B, K = c["B"], c["K"]
    tok = s["tokens"].long()
    p = s["target"][:, :K].gather(2, tok.unsqueeze(-1)).squeeze(-1).double()
    q = s["draft"].gather(2, tok.unsqueeze(-1)).squeeze(-1).double()
    n = (s["u"].double() * q < p).long().cumprod(1).sum(1)   # drafts accepted before the first refusal
    row = n[:, None, None].expand(-1, 1, c["V"])
    pr = s["target"].gather(1, row).squeeze(1).double()
    qr = s["draft"].gather(1, row.clamp(max=K - 1)).squeeze(1).double().masked_fill((n == K)[:, None], 0.0)
    w = (pr - qr).clamp(min=0.0)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, pr)
    cum = w.cumsum(1)
    got = (cum <= s["v"].double()[:, None] * cum[:, -1:]).sum(1)
    j = torch.arange(K + 1, device=tok.device)[None]
    drafts = torch.cat([tok, tok.new_zeros(B, 1)], 1)
    out = torch.where(j < n[:, None], drafts, torch.where(j == n[:, None], got[:, None], -1))
    return {"tokens": out.to(torch.int32), "accepted": n.to(torch.int32), "seq_lens": (s["seq_lens"] - K + n).to(torch.int32)}


# ------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s)
    return {"window": _plain_window, "mass": _plain_mass, "evict": _plain_evict, "verify": _plain_verify}[op](s)


def _own(s):
    import head_latent_attention_split_b200 as mla
    c = s["case"]
    if c["op"] == "window":
        out, lse = mla.window_decode(s["q_lat"], s["q_rope"], s["kv"], s["table"], s["lens"], s["scale"], c["window"],
                                     sinks=c["sinks"], causal=c["causal"], k_rope_cache=s["kr"], kv_scale=s["ks"])
        return {"out": out, "lse": lse}
    if c["op"] == "mass":
        mla.attention_mass(s["q_lat"], s["q_rope"], s["kv"], s["table"], s["lens"], s["lse"], s["scale"], s["mass"],
                           mass_in=s["mass_in"], causal=c["causal"], k_rope_cache=s["kr"], kv_scale=s["ks"])
        return {"mass": s["mass"]}
    if c["op"] == "evict":
        indices, counts = mla.evict_select(s["mass"], s["lens"], c["budget"], sinks=c["sinks"], recent=c["recent"])
        mla.cache_compact(s["kv"], s["table"], s["dst"], indices, counts, k_rope_cache=s["kr"], kv_scale=s["ks"],
                          mass=s["mass"], mass_out=s["mass_out"])
        return {"kv": s["kv"], "kr": s["kr"], "ks": s["ks"], "indices": indices, "counts": counts, "mass": s["mass_out"]}
    tokens, accepted, seq_lens = mla.verify_drafts(s["target"], s["draft"], s["tokens"], s["u"], s["v"],
                                                   seq_lens=s["seq_lens"])
    return {"tokens": tokens, "accepted": accepted, "seq_lens": seq_lens}


# ------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """From the definitions, one sequence (and query token) at a time, in 64 bits."""
    c, s = dict(case), prepare(case, seed)
    if c["op"] == "verify":
        return None   # whole numbers only
    if c["op"] == "evict":
        mass = s["mass"].double().cpu()
        rows = torch.zeros(s["mass_out"].shape, dtype=torch.float64)
        for b, n in enumerate(s["lens_host"]):
            tail = range(max(0, n - c["recent"]), n)
            keep = set(range(min(n, c["sinks"]))) | set(tail)
            if n <= c["budget"]:
                keep = set(range(n))
            left = mass[b, :n].tolist()
            for t in sorted((t for t in range(n) if t not in keep), key=lambda t: (-left[t], t)):
                if len(keep) >= c["budget"]:
                    break
                keep.add(t)
            rows[b, : len(keep)] = mass[b, sorted(keep)]
        return {"kv": None, "kr": None, "ks": None, "indices": None, "counts": None, "mass": rows}
    if c["B"] * c["L"] * c["Sq"] * c["H"] > 8 * 10 ** 8:
        return None
    outs, lses, mass = [], [], s["mass"].double() if c["op"] == "mass" else None
    for b, n in enumerate(s["lens_host"]):
        t = torch.arange(n, device=s["table"].device)
        lat, key = _rows(s, s["table"][b].long()[t // c["block"]] * c["block"] + t % c["block"], torch.float64)
        got = torch.zeros(n, dtype=torch.float64, device=t.device)
        for i in range(c["Sq"]):
            last = n - c["Sq"] + i if c["causal"] else n - 1
            x = (s["q_lat"][b, i].double() @ lat.T + s["q_rope"][b, i].double() @ key.T) * s["scale"]
            if c["op"] == "mass":
                got += torch.where(t <= last, torch.exp(x - s["lse"][b, i].double()[:, None]), 0.0).sum(0)
                continue
            hidden = (t > last) | ((t >= c["sinks"]) & (t <= last - c["window"]))
            lse = torch.logsumexp(x.masked_fill(hidden, float("-inf")), 1)
            w = torch.where(hidden | torch.isinf(lse)[:, None], 0.0, torch.exp(x - lse[:, None]))
            outs.append(w @ lat)
            lses.append(lse)
        if c["op"] == "mass":
            mass[b, :n] = s["mass_in"][b, :n].double() + got
    if c["op"] == "mass":
        return {"mass": mass}
    shape = (c["B"], c["Sq"], c["H"])
    return {"out": torch.stack(outs).reshape(*shape, c["r"]), "lse": torch.stack(lses).reshape(shape)}


# ------------------------------------------------------------------------------- work
def work(case):
    """Bytes read and written once, and the products' operations, of one pass (for ragged lengths: of their mean)."""
    c = case
    if c["op"] == "verify":
        e = 4 if c["dtype"] == "f32" else 2
        return {"bytes": c["B"] * (2 * c["V"] * e + c["K"] * (8 + 2 * e) + (c["K"] + 1) * 4 + 16), "flops": c["B"] * c["V"] * 3}
    L = c["L"] * (15 / 16) / math.log(16) if c["ragged"] and c["L"] > 16 else c["L"]
    row = {"f32": 4 * (c["r"] + c["dr"]), "bf16": 2 * (c["r"] + c["dr"]), "e4m3": c["r"] + 2 * c["dr"] + 4}[c["dtype"]]
    if c["op"] == "evict":
        kept = min(L, c["budget"])
        return {"bytes": c["B"] * (4 * L + kept * (2 * row + 4 + 8)), "flops": c["B"] * L}
    rows, e = c["Sq"] * c["H"], 4 if c["dtype"] == "f32" else 2
    if c["op"] == "window":
        near = min(c["window"] + (c["Sq"] - 1 if c["causal"] else 0), L)
        seen = min(L, near + c["sinks"])
        per = min(L, c["window"] + c["sinks"])
        return {"bytes": c["B"] * (seen * row + rows * ((2 * c["r"] + c["dr"]) * e + 4)),
                "flops": 2 * c["B"] * rows * per * (2 * c["r"] + c["dr"])}
    return {"bytes": c["B"] * (L * (row + 8) + rows * ((c["r"] + c["dr"]) * e + 4)),
            "flops": 2 * c["B"] * rows * L * (c["r"] + c["dr"])}
