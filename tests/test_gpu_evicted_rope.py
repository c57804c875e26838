"""A generation step behind an eviction with rotated RoPE keys: the kept keys hold the rotations of the positions they
had, so the next token's key has to be rotated for its position in the whole sequence, not in what is left."""
from __future__ import annotations

import math

import pytest

import bounded_ref as R

pytestmark = pytest.mark.gpu

r, d_r, bs, H, BASE, SCALE = 512, 64, 64, 16, 10000.0, 1.0 / math.sqrt(192.0)


def rotated(k, pos):
    """RoPE of pairs (2i, 2i + 1) by pos * BASE^(-2i / d_r), in float64."""
    import torch
    th = pos.double()[..., None] * BASE ** (-torch.arange(0, d_r, 2, device=k.device, dtype=torch.float64) / d_r)
    x, y = k.double()[..., 0::2], k.double()[..., 1::2]
    return torch.stack([x * th.cos() - y * th.sin(), x * th.sin() + y * th.cos()], -1).flatten(-2)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_the_token_behind_an_eviction_keeps_its_position(fp8):
    import torch
    import head_latent_attention_split_b200 as mla
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    B, n0, budget = 2, 300, 130
    nb = B * (6 + 3)
    perm = torch.randperm(nb, generator=g, device="cuda").int()
    table, dst = perm[:B * 6].reshape(B, 6).contiguous(), perm[B * 6:].reshape(B, 3).contiguous()
    if fp8:
        kv = torch.zeros(nb, bs, r, dtype=torch.uint8, device="cuda")
        kr, ks = torch.zeros(nb, bs, d_r, dtype=torch.bfloat16, device="cuda"), torch.zeros(nb, bs, device="cuda")
    else:
        kv, kr, ks = torch.zeros(nb, bs, r + d_r, dtype=torch.bfloat16, device="cuda"), None, None
    side = dict(k_rope_cache=kr, kv_scale=ks)
    lens = torch.tensor([n0, n0 - 17], dtype=torch.int32, device="cuda")
    c0, k0 = rnd(B, n0, r), rnd(B, n0, d_r)
    for b in range(B):   # (prompts of unlike lengths, one call each; positions from the lengths)
        n = int(lens[b])
        mla.cache_append(c0[b:b + 1, :n].contiguous(), k0[b:b + 1, :n].contiguous(), kv, table[b:b + 1].contiguous(),
                         lens[b:b + 1], rope=True, rope_base=BASE, **side)
    mass = torch.rand(B, 384, generator=g, device="cuda")
    idx, cnt = mla.evict_select(mass, lens, budget, sinks=4, recent=40)
    mla.cache_compact(kv, table, dst, idx, cnt, **side)

    # the next token: slot cnt of the cut cache, position lens of the sequence. Its key comes rotated, rope=False.
    c1, k1 = rnd(B, 1, r), rnd(B, 1, d_r)
    now = cnt + 1
    mla.cache_append(c1, rotated(k1, lens[:, None]).float().bfloat16(), kv, dst, now, rope=False, **side)
    q, qr = rnd(B, 1, H, r), rnd(B, 1, H, d_r)
    out, lse = mla.decode(q, qr, kv, dst, now, SCALE, k_rope_cache=kr, kv_scale=ks)
    wout, wlse = mla.window_decode(q, qr, kv, dst, now, SCALE, 64, sinks=4, **side)
    torch.cuda.synchronize()
    assert mla.device_status() == 0
    for b in range(B):
        keep = idx[b, :int(cnt[b])].long()
        c = torch.cat([c0[b, keep], c1[b]]).double()
        k = rotated(torch.cat([k0[b, keep], k1[b]]), torch.cat([keep, lens[b:b + 1].long()])).float().bfloat16().double()
        # a rotated key may round to the other neighbour (one unit, 2^-7 of a value of up to 2 sqrt(2) amax);
        # an fp8 latent is off by half a step, 2^-4, or where it is subnormal by 2^-10 of amax / 448
        dc = c.abs() * 2.0 ** -4 + c.abs().amax(1, keepdim=True) / 448 * 2.0 ** -10 if fp8 else 0 * c
        x = (q[b, 0].double() @ c.T + qr[b, 0].double() @ k.T) * SCALE
        ds = (q[b, 0].double().abs() @ dc.T + qr[b, 0].double().abs() @ k.abs().T * 2.0 ** -7) * SCALE + 1e-4
        t = torch.arange(len(c), device="cuda")
        for got, got_l, see in ((out, lse, t >= 0), (wout, wlse, (t < 4) | (t >= len(c) - 64))):
            l64 = torch.logsumexp(x[:, see], 1)
            e = ds[:, see].amax(1)
            p = torch.exp(x[:, see] - l64[:, None])
            assert bool(((got_l[b, 0].double() - l64).abs() <= e + 1e-5).all())
            o = p @ c[see]
            tol = (p @ c[see].abs()) * (torch.expm1(2 * e)[:, None] + 2.0 ** -8 + 2.0 ** -7 * fp8) + p @ dc[see] + R.UBF * o.abs()
            tol = tol + fp8 * (2.0 ** -8 + 2.0 ** -9) * c[see].abs().amax(0)
            assert bool(((got[b, 0].double() - o).abs() <= tol).all())
    # (the same bits that the append stores for this position where nothing was evicted)
    full = lens + 1
    mla.cache_append(c1, k1, kv, table, full, rope=True, rope_base=BASE, **side)
    torch.cuda.synchronize()
    for b in range(B):
        at = lambda tb, p: (int(tb[b, p // bs]), p % bs)  # noqa: E731
        keys = kr if fp8 else kv[..., r:]
        was, cut = keys[at(table, int(lens[b]))], keys[at(dst, int(cnt[b]))]
        assert bool((was.view(torch.int16).int() - cut.view(torch.int16).int()).abs().le(1).all())
    assert mla.device_status() == 0
