"""E4M3 cache on the tensor cores: the query as two 8-bit terms must keep its small channels beside a large one, and
its latent part beside a large RoPE part. The large channels meet zeros in the cache, so that the scores are
the small ones' alone."""
from __future__ import annotations

import pytest

import bounded_ref as R

pytestmark = pytest.mark.gpu

r, d_r, bs, SCALE = 512, 64, 64, 1.0 / 16
USED = 4   # latent channels whose products are not zero


def build(n, H, Sq, big_lat, big_rope, small, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, nb = "cuda", (n + bs - 1) // bs
    ch = torch.randperm(r, generator=g, device=dev)
    use, outlier = ch[:USED], ch[USED]
    codes = torch.randint(0, 0x7F, (nb * bs, r), generator=g, device=dev, dtype=torch.uint8)   # up to 448
    codes |= torch.randint(0, 2, codes.shape, generator=g, device=dev, dtype=torch.uint8) << 7
    codes[:, outlier] = 0
    scale = 0.25 * (1 + torch.rand(nb * bs, generator=g, device=dev))
    key = torch.randn(nb * bs, d_r, generator=g, device=dev).bfloat16()
    key[:, 5] = 0
    q = torch.zeros(1, Sq, H, r, device=dev)
    v = torch.exp2(-8 * torch.rand(Sq, H, USED, generator=g, device=dev)) * small   # eight octaves below `small`
    q[0, :, :, use] = v * (2 * torch.randint(0, 2, v.shape, generator=g, device=dev) - 1)
    q[..., outlier] = big_lat
    qr = torch.randn(1, Sq, H, d_r, generator=g, device=dev)
    qr[..., 5] = big_rope
    perm = torch.randperm(nb, generator=g, device=dev).to(torch.int32)
    at = lambda x, *s: torch.empty(nb, bs, *s, dtype=x.dtype, device=dev).index_copy_(0, perm.long(), x.reshape(nb, bs, *s))  # noqa: E731
    return dict(q=q.bfloat16(), qr=qr.bfloat16(), kv=at(codes, r), kr=at(key, d_r), ks=at(scale), table=perm[None].contiguous(),
                lens=torch.tensor([n], dtype=torch.int32, device=dev), n=n,
                c=codes.view(torch.float8_e4m3fn).double() * scale.double()[:, None], k=key.double())


def scores(t, s):
    """Scores of query token s in float64, and how far the kernel's may be: the fp32 sum of D products, and a split
    query value's error, 2^-21 of the latent part's largest magnitude, in every channel that has one."""
    q, qr, c, k = t["q"][0, s].double(), t["qr"][0, s].double(), t["c"][:t["n"]], t["k"][:t["n"]]
    x = (q @ c.T + qr @ k.T) * SCALE
    mag = (q.abs() @ c.abs().T + qr.abs() @ k.abs().T) * SCALE
    held = 2.0 ** -21 * q.abs().amax(1)[:, None] * ((q != 0).double() @ c.abs().T) * SCALE
    return x, (r + d_r + 4) * R.U32 * mag + 2.0 ** -21 + held


SIZES = [(1000.0, 1.0, 1.0), (1.0, 3000.0, 1.0), (2.0 ** 20, 2.0 ** -20, 1.0), (2.0 ** -40, 1.0, 2.0 ** -6), (1.0, 2.0 ** 30, 0.5),
         (0.0, 2.0 ** 60, 0.5)]


@pytest.mark.parametrize("H,Sq", [(8, 1), (128, 1), (80, 2)])
@pytest.mark.parametrize("big_lat,big_rope,small", SIZES)
def test_window_decode_keeps_small_query_channels(H, Sq, big_lat, big_rope, small):
    import torch
    import head_latent_attention_split_b200 as mla
    t = build(300, H, Sq, big_lat, big_rope, small, seed=H)
    _, lse = mla.window_decode(t["q"], t["qr"], t["kv"], t["table"], t["lens"], SCALE, 300, causal=Sq > 1, k_rope_cache=t["kr"],
                               kv_scale=t["ks"])
    torch.cuda.synchronize()
    assert mla.device_status() == 0
    for s in range(Sq):
        x, ds = scores(t, s)
        m = t["n"] - Sq + 1 + s
        ref = torch.logsumexp(x[:, :m], 1)
        tol = ds[:, :m].amax(1) + (m + 8) * R.U32 + 4 * R.U32 * ref.abs()
        err = (lse[0, s].double() - ref).abs()
        assert bool((err <= tol).all()), f"off by {float((err / tol).max()):.3g} bounds"


@pytest.mark.parametrize("H,Sq", [(8, 1), (128, 1), (80, 2)])
@pytest.mark.parametrize("big_lat,big_rope,small", SIZES)
def test_attention_mass_keeps_small_query_channels(H, Sq, big_lat, big_rope, small):
    import torch
    import head_latent_attention_split_b200 as mla
    t = build(300, H, Sq, big_lat, big_rope, small, seed=H)
    n, want, tol = t["n"], 0.0, 0.0
    lse = torch.empty(1, Sq, H, device="cuda")
    for s in range(Sq):
        x, ds = scores(t, s)
        see = torch.arange(n, device="cuda") < n - Sq + 1 + s
        lse[0, s] = torch.logsumexp(x[:, see], 1).float()
        l64 = lse[0, s].double()[:, None]
        w = torch.where(see, torch.exp(x - l64), 0.0)
        want = want + w.sum(0)
        tol = tol + (w * torch.expm1(ds + 4 * R.U32 * l64.abs())).sum(0)
    tol = tol + (Sq * H + 4) * R.U32 * want
    mass = torch.zeros(1, n, device="cuda")
    mla.attention_mass(t["q"], t["qr"], t["kv"], t["table"], t["lens"], lse, SCALE, mass, causal=Sq > 1, k_rope_cache=t["kr"],
                       kv_scale=t["ks"])
    torch.cuda.synchronize()
    assert mla.device_status() == 0
    err = (mass[0].double() - want).abs()
    assert bool((err <= tol).all()), f"off by {float((err / tol).max()):.3g} bounds"
