"""Plain 64-bit references of the operators that bound a generation's cache and work, with error bounds.

Each function walks the definition one sequence (and query row) at a time in float64 and returns
the values with a bound on how far a kernel that rounds as documented may be from them: half a
step of every type a value is rounded to, and n half steps of fp32 for a sum of n products.
"""
import numpy as np
import torch

import workloads as W

U32, U16, UBF = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8   # half steps of fp32, fp16 and bf16, relative


def to64(a, dtype):
    if a is None:
        return None
    if dtype == W.BF16:
        return torch.from_numpy(W.bf16_bits_to_f32(a)).double()
    return torch.from_numpy(np.ascontiguousarray(a)).double()


def rows_of(inp, b, n):
    """Latents [n, r] and RoPE keys [n, d_r] of the first n tokens of sequence b, float64."""
    w = inp["workload"]
    t = np.arange(n)
    slot = inp["block_table"][b, t // w.block_size].astype(np.int64) * w.block_size + t % w.block_size
    if w.cache_dtype == W.E4M3:
        codes = torch.from_numpy(inp["kv_cache"].reshape(-1, w.r)[slot]).view(torch.float8_e4m3fn).double()
        return (codes * to64(inp["kv_scale"].reshape(-1)[slot], W.F32)[:, None],
                to64(inp["k_rope_cache"].reshape(-1, w.d_r)[slot], W.BF16))
    x = to64(inp["kv_cache"].reshape(-1, w.r + w.d_r)[slot], w.cache_dtype)
    return x[:, :w.r], x[:, w.r:]


def scales_of(inp, b, n):
    """fp8 cache: the scales of the first n tokens of sequence b, float64."""
    w = inp["workload"]
    t = np.arange(n)
    slot = inp["block_table"][b, t // w.block_size].astype(np.int64) * w.block_size + t % w.block_size
    return to64(inp["kv_scale"].reshape(-1)[slot], W.F32)


def tokens_of_row(w, L, s):
    return max(L - w.Sq + 1 + s if w.causal else L, 0)


def seen(w, L, s, window=None, sinks=0):
    """Truth values over the L tokens: which ones query row s sees."""
    n = tokens_of_row(w, L, s)
    t = torch.arange(L)
    see = t < n
    return see if window is None else see & ((t >= n - window) | (t < sinks))


def window(inp, win, sinks):
    """(out, lse, bound of out, bound of lse) of the decode over window and sinks."""
    w = inp["workload"]
    q, qr = to64(inp["q_lat"], w.q_dtype), to64(inp["q_rope"], w.q_dtype)
    out = torch.zeros(w.B, w.Sq, w.H, w.r, dtype=torch.float64)
    lse = torch.full((w.B, w.Sq, w.H), -np.inf, dtype=torch.float64)
    bo, bl = torch.zeros_like(out), torch.zeros_like(lse)
    D = w.r + w.d_r
    for b, L in enumerate(int(x) for x in inp["seq_lens"]):
        for s in range(w.Sq):
            see = seen(w, L, s, win, sinks)
            if not bool(see.any()):
                continue
            c, k = (x[see] for x in rows_of(inp, b, L))
            x = (q[b, s] @ c.T + qr[b, s] @ k.T) * w.scale
            mag = (q[b, s].abs() @ c.abs().T + qr[b, s].abs() @ k.abs().T) * abs(w.scale)
            lse[b, s] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[b, s][:, None])
            out[b, s] = p @ c
            ac = p @ c.abs()
            # a score: D products summed in fp32, and the scale's own rounding; 2^x to 2 units in the
            # last place; an fp8 key's RoPE part is held as two bf16 terms (2^-16)
            ds = (D + 4) * U32 * mag.amax(1) + 2.0 ** -21
            if w.cache_dtype == W.E4M3:   # ... or the query as two e4m3 terms, see mass()
                ds = ds + 2.0 ** -16 * mag.amax(1) + 2.0 ** -16 * abs(w.scale) * torch.maximum(
                    q[b, s].abs().amax(1), qr[b, s].abs().amax(1)) * c.abs().sum(1).amax()
            n = x.shape[1]
            bl[b, s] = ds + (n + 8) * U32 + 4 * U32 * lse[b, s].abs()
            # out: the weights' errors, their rounding for the second product, its sum in fp32, and the
            # output's rounding. The weights go in as bf16; with an fp8 cache as weight * scale s, in two
            # e4m3 terms: 2^-4 of what the first leaves, which is 2^-4 again (or in fp16: 2^-11). At
            # e4m3's smallest step 2^-9 each term may lose half of it, 2^-9 per token and code of at most
            # 448, where the largest weight * s is at least 2^4 (its logarithm t is the softmax's maximum).
            up = {W.F32: 0.0, W.BF16: UBF, W.E4M3: 2.0 ** -8}[w.cache_dtype]
            bo[b, s] = ac * (2 * ds[:, None] + up + (n + 8) * U32)
            if w.cache_dtype == W.E4M3:
                t = x + torch.log(scales_of(inp, b, L)[see].clamp(min=2.0 ** -64))
                z = torch.exp(x - t.amax(1, keepdim=True)).sum(1, keepdim=True)
                bo[b, s] += 2.0 ** -9 * 448 / 16 * n / z
                # (the kernel that keeps them in fp16: its smallest step, 2^-24)
                z = torch.exp(x - x.amax(1, keepdim=True)).sum(1, keepdim=True)
                bo[b, s] += 2.0 ** -25 * 448 * n / z
            if w.out_dtype == W.BF16:
                bo[b, s] += UBF * out[b, s].abs()
    return out, lse, bo, bl


def mass(inp, lse, mass_in):
    """(mass, bound) of the attention weight; lse [B, Sq, H] and mass_in [B, S] float64 (S columns)."""
    w = inp["workload"]
    q, qr = to64(inp["q_lat"], w.q_dtype), to64(inp["q_rope"], w.q_dtype)
    res, bound = mass_in.clone(), torch.zeros_like(mass_in)
    for b, L in enumerate(int(x) for x in inp["seq_lens"]):
        if L == 0:
            continue
        c, k = rows_of(inp, b, L)
        for s in range(w.Sq):
            see = seen(w, L, s)
            x = (q[b, s] @ c.T + qr[b, s] @ k.T) * w.scale
            mag = (q[b, s].abs() @ c.abs().T + qr[b, s].abs() @ k.abs().T) * abs(w.scale)
            ds = (w.r + w.d_r + 4) * U32 * mag + 2.0 ** -21 + 4 * U32 * lse[b, s][:, None].abs()
            if w.cache_dtype == W.E4M3:   # a query value split in two e4m3 terms, the row's largest at 128 or more
                # and e4m3's smallest step 2^-9, of which each term may lose half: 2^-9 / 128
                ds = ds + 2.0 ** -16 * abs(w.scale) * q[b, s].abs().amax(1)[:, None] * c.abs().sum(1)[None]
            wt = torch.where(see[None], torch.exp(x - lse[b, s][:, None]), 0.0)
            res[b, :L] += wt.sum(0)
            bound[b, :L] += torch.where(see[None], wt * ds * 1.01, 0.0).sum(0)
        bound[b, :L] += (w.Sq * w.H + 4) * U32 * res[b, :L]
    return res, bound


def evict(mass, lens, budget, sinks, recent):
    """(indices [B, budget], counts [B]) by a sort of the candidates."""
    idx = np.full((len(lens), budget), -1, np.int32)
    cnt = np.zeros(len(lens), np.int32)
    for b, L in enumerate(int(x) for x in lens):
        keep = list(range(L))
        if L > budget:
            mid = range(sinks, L - recent)
            v = {t: (np.inf if np.isnan(mass[b, t]) else float(mass[b, t])) for t in mid}
            best = sorted(mid, key=lambda t: (not np.isnan(mass[b, t]), -v[t], t))[:budget - sinks - recent]
            keep = sorted(list(range(sinks)) + best + list(range(L - recent, L)))
        idx[b, :len(keep)] = keep
        cnt[b] = len(keep)
    return idx, cnt


def verify(target, draft, tokens, u, v, lens=None):
    """(tokens [B, K + 1], accepted [B]) from the definition in float64; -1 rows for unusable input."""
    B, K1, V = target.shape
    out, acc = np.full((B, K1), -1, np.int32), np.zeros(B, np.int32)
    t64 = target.astype(np.float64)
    d64 = None if draft is None else draft.astype(np.float64)
    for b in range(B):
        n = nd = K1 - 1 if lens is None else int(lens[b])
        bad = not 0 <= nd < K1
        for i in range(0 if bad else nd):
            x = int(tokens[b, i])
            if not 0 <= x < V:
                bad = True
                break
            q = 1.0 if d64 is None else d64[b, i, x]
            if not np.float64(u[b, i]) * q < t64[b, i, x]:
                n = i
                break
        if bad:
            acc[b] = -1
            continue
        p = t64[b, n]
        w = p
        if n < nd:
            q = d64[b, n] if d64 is not None else (np.arange(V) == tokens[b, n]).astype(np.float64)
            w = p - q
            if d64 is None:
                w = np.where(np.arange(V) == tokens[b, n], 0.0, p)
        with np.errstate(invalid="ignore"):
            w = np.where(w > 0, w, 0.0)
            if n < nd and w.sum() == 0:
                w = np.where(p > 0, p, 0.0)
        total = w.sum()
        if not (total > 0 and np.isfinite(total)):
            acc[b] = -1
            continue
        uu = float(v[b])
        uu = 1 - 2.0 ** -24 if uu >= 1 else uu if uu >= 0 else 0.0
        cum = np.cumsum(w)
        t = int(np.searchsorted(cum, uu * cum[-1], side="right"))
        out[b, :n] = tokens[b, :n]
        out[b, n] = min(t, int(np.nonzero(w)[0][-1]))
        acc[b] = n
    return out, acc
