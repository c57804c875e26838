"""A generation with a bounded cache, every operator in its place: drafted tokens are appended, decoded (whole
cache and window), verified; refused ones leave; the attention weight piles up and the cache is cut by it,
into other blocks of the pool. Every step is compared with a float64 walk over plain lists of tokens."""
from __future__ import annotations

import numpy as np
import pytest

import bounded_ref as R
import workloads as W

pytestmark = pytest.mark.gpu

r, d_r, bs = 512, 64, 64


class Plain:
    """One sequence: its tokens' latents and keys (float64 of what the cache stores) and weights."""

    def __init__(self):
        self.c, self.k, self.mass = np.zeros((0, r)), np.zeros((0, d_r)), np.zeros(0)

    def append(self, c, k):
        self.c, self.k = np.concatenate([self.c, c]), np.concatenate([self.k, k])
        self.mass = np.concatenate([self.mass, np.zeros(len(c))])

    def keep(self, idx):
        self.c, self.k, self.mass = self.c[idx], self.k[idx], self.mass[idx]


def attend(q, qr, c, k, scale, see):
    """(out, lse, weights, bound of a score) of one query row block [H, .] over the tokens `see`."""
    x = (q @ c.T + qr @ k.T) * scale
    ds = (r + d_r + 4) * R.U32 * ((np.abs(q) @ np.abs(c).T + np.abs(qr) @ np.abs(k).T) * scale).max() + 2.0 ** -21
    x = np.where(see, x, -np.inf)
    m = x.max(1, keepdims=True)
    z = np.exp(x - m).sum(1, keepdims=True)
    return np.exp(x - m) / z @ c, (m + np.log(z))[:, 0], np.exp(x - m) / z, ds


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_drafts_windows_weights_and_eviction_together(fp8):
    import torch
    import head_latent_attention_split_b200 as mla
    rng = np.random.default_rng(7 + fp8)
    B, H, K, V, budget, sinks, recent, win, scale = 3, 16, 2, 500, 72, 2, 20, 50, 0.07
    mb, pool = 4, 3 * 4 * 2
    dev = "cuda"
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    # the pool starts as NaN: nothing that was not appended may be looked at
    if fp8:
        kv = torch.full((pool, bs, r), 0x7F, dtype=torch.uint8, device=dev)
        kr = torch.full((pool, bs, d_r), float("nan"), dtype=torch.bfloat16, device=dev)
        ks = torch.full((pool, bs), float("nan"), device=dev)
    else:
        kv, kr, ks = torch.full((pool, bs, r + d_r), float("nan"), dtype=torch.bfloat16, device=dev), None, None
    perm = rng.permutation(pool).astype(np.int32)
    table, free = torch.tensor(perm[:12].reshape(B, mb), device=dev), torch.tensor(perm[12:].reshape(B, mb), device=dev)
    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    mass = torch.zeros(B, mb * bs, device=dev)
    plain = [Plain() for _ in range(B)]
    evictions = 0
    for step in range(20):
        # a prompt first, then a committed token and K drafts per sequence
        n = 60 if step == 0 else K + 1
        c = torch.tensor(rng.normal(size=(B, n, r)) * 0.5, device=dev).bfloat16()
        k = torch.tensor(rng.normal(size=(B, n, d_r)) * 0.5, device=dev).bfloat16()
        lens = lens + n
        mla.cache_append(c, k, kv, table, lens, k_rope_cache=kr, kv_scale=ks)
        stored = f64(c)
        if fp8:   # what the append stores, by its definition
            codes, s = W.quantize_e4m3_per_token(c.float().cpu().numpy())
            stored = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy() * s.astype(np.float64)[..., None]
        for b in range(B):
            plain[b].append(stored[b], f64(k)[b])
        Sq = min(n, K + 1)
        q = torch.tensor(rng.normal(size=(B, Sq, H, r)), device=dev).bfloat16()
        qr = torch.tensor(rng.normal(size=(B, Sq, H, d_r)), device=dev).bfloat16()
        kw = dict(causal=True, k_rope_cache=kr, kv_scale=ks)
        out, lse = mla.decode(q, qr, kv, table, lens, scale, **kw)
        wout, wlse = mla.window_decode(q, qr, kv, table, lens, scale, win, sinks=sinks, **kw)
        mla.attention_mass(q, qr, kv, table, lens, lse, scale, mass, mass_in=mass, **kw)
        target = torch.softmax(torch.tensor(rng.normal(size=(B, K + 1, V)) * 2, device=dev).float(), -1)
        draft = torch.softmax(torch.log(target[:, :K]) + torch.tensor(rng.normal(size=(B, K, V)), device=dev).float(), -1)
        toks = torch.multinomial(draft.reshape(B * K, V), 1, generator=torch.Generator(dev).manual_seed(step)).reshape(B, K).int()
        u, v = torch.tensor(rng.random((B, K), np.float32), device=dev), torch.tensor(rng.random(B, np.float32), device=dev)
        if step > 0:
            tokens, accepted, new_lens = mla.verify_drafts(target, draft, toks, u, v, seq_lens=lens)
        assert mla.device_status() == 0

        old = lens.tolist()
        for b in range(B):
            p = plain[b]
            added = np.zeros(old[b])
            err = np.zeros(old[b])
            for s in range(Sq):
                t = np.arange(old[b])
                m = old[b] - Sq + 1 + s
                qb, qrb = f64(q[b, s]), f64(qr[b, s])
                for got, got_l, see in ((out, lse, t < m), (wout, wlse, (t < m) & ((t >= m - win) | (t < sinks)))):
                    o, l, w, ds = attend(qb, qrb, p.c, p.k, scale, see[None])
                    # weights' errors and their rounding (bf16, fp16 or two e4m3 terms: 2^-8 at most, and for
                    # these near-equal scales 2^-9 * 448 / 16 per 120 of the largest term), the output's
                    ds += 2.0 ** -15 * scale * 576 * 5 * fp8
                    tol = (2 * ds + 2.0 ** -8 + 2.0 ** -8 * fp8) * (w @ np.abs(p.c)) + 2.0 ** -8 * np.abs(o) + 1e-3 * fp8
                    assert (np.abs(f64(got[b, s]) - o) <= tol).all(), (step, b, s)
                    assert (np.abs(f64(got_l[b, s]) - l) <= ds + 1e-5).all(), (step, b, s)
                    if got is out:
                        added += w.sum(0)
                        err += w.sum(0) * 2 * ds
            p.mass = p.mass + added
            assert (np.abs(f64(mass[b, :old[b]]) - p.mass) <= (step + 1) * (err + 1e-5 * (1 + p.mass))).all(), (step, b)
            assert bool((mass[b, old[b]:] == 0).all())
        if step > 0:
            ref_t, ref_a = R.verify(*(x.cpu().numpy() for x in (target, draft, toks, u, v)))
            np.testing.assert_array_equal(tokens.cpu().numpy(), ref_t)
            np.testing.assert_array_equal(accepted.cpu().numpy(), ref_a)
            np.testing.assert_array_equal(new_lens.cpu().numpy(), np.array(old) - K + ref_a)
            # the refused drafts leave: their positions' weight with them
            mass.masked_fill_(torch.arange(mb * bs, device=dev)[None] >= new_lens[:, None], 0.0)
            lens = new_lens
            for b, n in enumerate(lens.tolist()):
                plain[b].keep(np.arange(n))
        if int(lens.max()) > budget:
            evictions += 1
            idx, cnt = mla.evict_select(mass, lens, budget - 16, sinks=sinks, recent=recent)
            fresh = torch.empty_like(mass)
            mla.cache_compact(kv, table, free, idx, cnt, k_rope_cache=kr, kv_scale=ks, mass=mass, mass_out=fresh)
            assert mla.device_status() == 0
            ref_i, ref_c = R.evict(mass.cpu().numpy(), lens.cpu().numpy(), budget - 16, sinks, recent)
            np.testing.assert_array_equal(idx.cpu().numpy(), ref_i)
            np.testing.assert_array_equal(cnt.cpu().numpy(), ref_c)
            # the kept tokens attended in place give what the compacted cache gives
            if not fp8:
                q1, qr1 = q[:, :1].contiguous(), qr[:, :1].contiguous()
                a = mla.sparse_decode(q1, qr1, kv, table, idx, cnt, scale)
                b2 = mla.decode(q1, qr1, kv, free, cnt, scale)
                assert float((a[0].float() - b2[0].float()).abs().max()) <= 2.0 ** -6 * float(b2[0].float().abs().max())
            table, free = free, table
            lens, mass = cnt, fresh
            for b in range(B):
                plain[b].keep(ref_i[b, :ref_c[b]])
    assert evictions >= 2


def test_two_calls_at_once_on_two_streams():
    import torch
    import head_latent_attention_split_b200 as mla
    ws = [W.WORKLOADS[3].with_(B=6, seq_lens=(700, 65, 1300, 900, 2000, 31), spare_blocks=1), W.WORKLOADS[4].with_(B=4, seq_lens=(900, 2100, 65, 1500))]
    T = [W.to_torch(W.make_inputs(w)) for w in ws]

    def chain(i, stream=None):
        t, w = T[i], ws[i]
        a = (t["q_lat"], t["q_rope"], t["kv_cache"], t["block_table"], t["seq_lens"])
        kw = dict(causal=w.causal, k_rope_cache=t["k_rope_cache"], kv_scale=t["kv_scale"], stream=stream)
        out, lse = mla.window_decode(*a, w.scale, 600, sinks=4, **kw)
        full = mla.decode(*a, w.scale, w.causal, t["k_rope_cache"], t["kv_scale"], stream=stream)[1] if stream is None else lse
        mass = torch.zeros(w.B, 2200, device="cuda") if stream is None else None
        return out, lse, full, mass
    ref = [chain(0), chain(1)]
    masses = [mla.attention_mass(*(T[i][k] for k in ("q_lat", "q_rope", "kv_cache", "block_table", "seq_lens")), ref[i][2],
                                 ws[i].scale, ref[i][3], causal=ws[i].causal, k_rope_cache=T[i]["k_rope_cache"],
                                 kv_scale=T[i]["kv_scale"]) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            out, lse, _, _ = chain(i, s)
            with torch.cuda.stream(s):
                m = torch.zeros(ws[i].B, 2200, device="cuda")
            mla.attention_mass(*(T[i][k] for k in ("q_lat", "q_rope", "kv_cache", "block_table", "seq_lens")), ref[i][2],
                               ws[i].scale, m, causal=ws[i].causal, k_rope_cache=T[i]["k_rope_cache"],
                               kv_scale=T[i]["kv_scale"], stream=s)
            got[i].append((out, lse, m))
    torch.cuda.synchronize()
    assert mla.device_status() == 0
    for i in range(2):
        for out, lse, m in got[i]:
            assert torch.equal(out, ref[i][0]) and torch.equal(lse, ref[i][1]) and torch.equal(m, masses[i])
