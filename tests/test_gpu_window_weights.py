"""The window decode where a few tokens hold most of the softmax: every weight has to reach the output, however
small it is beside the largest and however many there are. Scores are set through the RoPE part (the
e4m3 cache's latents carry the values), so that they are exact products."""
from __future__ import annotations

import math

import pytest

import bounded_ref as R

pytestmark = pytest.mark.gpu

r, d_r, bs, SCALE = 512, 64, 64, 1.0 / 16
# A weight w = p s_t goes into the second product as two 8-bit terms. They hold it to 2^-8 of itself, or, below e4m3's
# normal range, to 2^-14, in units where one token of every 8 x 128 such ones weighs 2^4, and one of any other 128
# weighs 2^2. So all the small ones together miss this part of the row's sum of w at most:
FLOOR = 8 * 128 * 2.0 ** -14 / 2 ** 4 + 128 * 2.0 ** -14 / 2 ** 2


def build(n, levels, heads, Sq=1, seed=0, amp=None, cut=0):
    """One sequence of n tokens whose natural-log score for head h, query token s is levels[h](t) (float64
    [n] -> rounded as the operands are). amp: the tokens' latent magnitudes. Returns the call's tensors."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    nb = (n + bs - 1) // bs
    # the tail's latents share a mean, so that its weight shows in the output; the first token's differ
    lat = torch.randn(r, generator=g, device=dev) + 0.3 * torch.randn(nb * bs, r, generator=g, device=dev)
    lat[0] = torch.randn(r, generator=g, device=dev)
    if amp is not None:
        lat *= amp[:, None]
    scale = (lat.abs().amax(1) / 448).float()
    codes = (lat / scale[:, None].clamp(min=1e-30)).to(torch.float8_e4m3fn)
    # head h reads channels 2h, 2h + 1 of the keys: a level as two bf16 terms
    key = torch.zeros(nb * bs, d_r, device=dev, dtype=torch.bfloat16)
    q = torch.zeros(1, Sq, heads, d_r, device=dev, dtype=torch.bfloat16)
    for i, f in enumerate(levels):
        x = (f(torch.arange(nb * bs, device=dev, dtype=torch.float64)) / SCALE / 16).float()
        hi = x.bfloat16()
        key[:, 2 * i], key[:, 2 * i + 1] = hi, (x - hi.float()).bfloat16()
    for h in range(heads):
        i = h % len(levels)
        q[:, :, h, 2 * i:2 * i + 2] = 16.0
    perm = torch.randperm(nb + 3, generator=g, device=dev)[:nb].to(torch.int32)
    kv = torch.full((nb + 3, bs, r), 0x7F, dtype=torch.uint8, device=dev)
    kr = torch.full((nb + 3, bs, d_r), float("nan"), dtype=torch.bfloat16, device=dev)
    ks = torch.full((nb + 3, bs), float("nan"), device=dev)
    kv[perm.long()] = codes.view(torch.uint8).reshape(nb, bs, r)
    kr[perm.long()] = key.reshape(nb, bs, d_r)
    ks[perm.long()] = scale.reshape(nb, bs)
    return dict(q_lat=torch.zeros(1, Sq, heads, r, device=dev, dtype=torch.bfloat16), q_rope=q, kv=kv, kr=kr, ks=ks,
                table=perm[None].contiguous(), lens=torch.tensor([n], dtype=torch.int32, device=dev), n=n,
                c=codes.double() * scale.double()[:, None], k=key.double(), s=scale.double())


def check(t, win, sinks, causal=False, l2=None, **kw):
    import torch
    import head_latent_attention_split_b200 as mla
    n, (Sq, H) = t["n"], t["q_rope"].shape[1:3]
    out, lse = mla.window_decode(t["q_lat"], t["q_rope"], t["kv"], t["table"], t["lens"], SCALE, win, sinks=sinks, causal=causal,
                                 k_rope_cache=t["kr"], kv_scale=t["ks"], out_dtype=0, **kw)
    torch.cuda.synchronize()
    assert mla.device_status() == 0
    pos, worst = torch.arange(n, device="cuda"), 0.0
    for s in range(Sq):
        end = n - Sq + 1 + s if causal else n
        see = (pos < end) & ((pos >= end - win) | (pos < sinks))
        c, k = t["c"][:n][see], t["k"][:n][see]
        x = t["q_rope"][0, s].double() @ k.T * SCALE
        ref_l = torch.logsumexp(x, 1)
        p = torch.exp(x - ref_l[:, None])
        ds = (r + d_r + 4) * R.U32 * x.abs().amax(1) + 2.0 ** -21     # (as bounded_ref.window)
        m = c.shape[0]
        # what the small ones miss is a weight of theirs, on codes of any of them: sum w times the channel's largest
        sc = t["s"][:n][see]
        tol = (p @ c.abs()) * (2 * ds[:, None] + 2.0 ** -8 + (m + 8) * R.U32) + FLOOR * (p @ sc)[:, None] * (
            c / sc[:, None]).abs().amax(0)
        err = (out[0, s].double() - p @ c).abs()
        worst = max(worst, float((err / tol).max()))
        # over a tail of one mean that is 2^-8 of the tail's vector and of the sink's, each of about sqrt(r) and
        # nearly orthogonal: 2^-8 sqrt(2) of the output at the most where both weigh the same
        if l2 is not None:
            assert float((err.norm(dim=1) / (p @ c).norm(dim=1)).max()) <= l2
        assert bool(((lse[0, s].double() - ref_l).abs() <= ds + (m + 8) * R.U32 + 4 * R.U32 * ref_l.abs()).all())
    assert worst <= 1.0, f"off by {worst:.3g} bounds"


def sink(log_odds):
    """The first token's score over a flat tail."""
    return lambda t: (t == 0).double() * log_odds


def noisy(log_odds, sigma, seed):
    import torch

    def f(t):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64) * sigma
        x[0] = log_odds + sigma * sigma / 2
        return x
    return f


@pytest.mark.parametrize("n", [2052, 4100, 16388, 65540])
@pytest.mark.parametrize("workers", [0, 1])
def test_a_sink_over_a_long_tail(n, workers):
    """The sink holds 0.5, 0.9 and 0.99 of the softmax over a flat and over a noisy tail; and scores it by
    9 to 11 above each of them."""
    odds = [math.log(a / (1 - a) * n) for a in (0.5, 0.9, 0.99)]
    levels = [sink(x) for x in odds] + [noisy(x, s, 3) for x in odds[:2] for s in (0.5, 1.7)]
    levels += [sink(x) for x in (9.0, 9.5, 10.0, 11.0)] + [lambda t: 0 * t]
    check(build(n, levels, len(levels)), n - 4, 4, l2=1e-2, num_workers=workers)


@pytest.mark.parametrize("heads,Sq,workers", [(8, 1, 0), (128, 1, 0), (80, 2, 0), (16, 2, 3)])
def test_a_sink_before_a_window(heads, Sq, workers):
    n, win = 20000, 8000
    levels = [sink(math.log(win)), sink(math.log(9 * win)), noisy(math.log(win), 1.0, 5), noisy(0.0, 1.7, 6)]
    check(build(n, levels, heads, Sq), win, 4, causal=Sq > 1, l2=1e-2, num_workers=workers)


@pytest.mark.parametrize("workers", [0, 1, 5])
def test_scores_that_fall_rise_and_swing(workers):
    """Levels that make the weights' reference go down, up, down by more than it may, and both in turn; the weight
    stands in the first, the last or the middle tokens."""
    n = 64 * 90 + 17
    tile = lambda t: (t // 64)  # noqa: E731
    levels = [lambda t: -0.7 * tile(t), lambda t: 0.7 * tile(t), lambda t: -0.03 * tile(t), lambda t: 0.05 * tile(t),
              lambda t: -4.0 * (tile(t) // 12), lambda t: 4.0 * (tile(t) // 12), lambda t: 5.0 * ((tile(t) // 20) % 2),
              lambda t: -30.0 * (t > 0), lambda t: -12.0 * (tile(t) % 18 > 0), lambda t: 9.0 * (t == 3000) - 2.0 * (t > 4000),
              lambda t: -15.0 * ((t > 100) & (t < 5000)), lambda t: 3.0 * ((t * 7919) % 131 == 0)]
    check(build(n, [(lambda t, f=f: f(t).double()) for f in levels], len(levels)), n, 0, num_workers=workers)


def test_a_sink_among_tokens_of_unlike_magnitudes():
    """Token scales over six octaves: the weights that the second product takes hold the token's scale."""
    import torch
    n = 6000
    g = torch.Generator(device="cuda").manual_seed(9)
    amp = torch.exp2(-6 * torch.rand(6016, generator=g, device="cuda"))
    levels = [sink(math.log(n)), sink(math.log(9 * n)), noisy(math.log(n), 1.0, 2), noisy(0.0, 0.5, 2)]
    check(build(n, levels, 16, amp=amp), n, 0)
    check(build(n, levels, 16, amp=amp * 2.0 ** -12), 3000, 1)


@pytest.mark.parametrize("back", [0.0, 2.0, 3.0, 4.0])
@pytest.mark.parametrize("workers", [1, 0])
def test_one_rows_turn_leaves_its_neighbours_large_weights(back, workers):
    """Rows beside one another: one of a sink over a flat tail, the others low too but for one pair of tiles, each
    another one, where their scores come back to the first token's level (and `back` above it)."""
    n = 64 * 50
    pair = lambda t: t // 128  # noqa: E731
    levels = [sink(14.0)] + [(lambda t, j=j: (14.0 + back * (t > 0)) * ((t == 0) | (pair(t) == j)).double()) for j in range(1, 21)]
    check(build(n, levels, 32), n, 0, num_workers=workers)
    levels = [noisy(14.0, 0.3, 4)] + [(lambda t, j=j: (14.0 + back * (t > 0)) * ((t == 0) | (t == 128 * j + 77)).double()
                                       - 9.0 * (pair(t) % 3 == 1)) for j in range(4, 24)]
    check(build(n, levels, 21, Sq=2), n, 0, causal=True, num_workers=workers)
