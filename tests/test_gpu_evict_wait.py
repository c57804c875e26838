"""The compaction's copy when its waits run out: what it leaves, and that it says so."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_an_expired_wait_leaves_whole_rows_and_says_so(fp8):
    import torch
    import head_latent_attention_split_b200 as mla
    g = torch.Generator(device="cuda").manual_seed(4)
    B, bs, mb, n = 40, 64, 8, 4 * 64 - 9
    kv = torch.randn(2 * B * mb, bs, 512 if fp8 else 576, generator=g, device="cuda").bfloat16()
    kr = ks = None
    if fp8:
        kv = kv.to(torch.float8_e4m3fn).view(torch.uint8)
        kr = torch.randn(2 * B * mb, bs, 64, generator=g, device="cuda").bfloat16()
        ks = torch.rand(2 * B * mb, bs, generator=g, device="cuda")
    perm = torch.randperm(2 * B * mb, generator=g, device="cuda").int()
    bt, dt = perm[:B * mb].reshape(B, mb).contiguous(), perm[B * mb:].reshape(B, mb).contiguous()
    idx = torch.stack([torch.randperm(mb * bs, generator=g, device="cuda")[:n].sort().values for _ in range(B)]).int()
    cnt = torch.full((B,), n, dtype=torch.int32, device="cuda")
    t, j = idx.long(), torch.arange(n, device="cuda")
    src = (bt.gather(1, t // bs).long() * bs + t % bs).reshape(-1)
    dst = (dt[:, j // bs].long() * bs + j % bs).reshape(-1)
    planes = [x for x in (kv, kr) if x is not None]
    start = [x.clone() for x in planes]
    flat = lambda x: x.reshape(2 * B * mb * bs, -1).view(torch.uint8)  # noqa: E731
    expired = 0
    for limit in [1] * 8 + [0]:   # 0: the default limit again
        for x, s in zip(planes, start):
            x.copy_(s)
        torch.cuda.synchronize()
        mla.set_wait_timeout_ns(limit)
        try:
            mla.cache_compact(kv, bt, dt, idx, cnt, k_rope_cache=kr, kv_scale=ks)
            torch.cuda.synchronize()
        finally:
            mla.set_wait_timeout_ns(0)
        st = mla.device_status()
        assert st in ((0, 8) if limit else (0,)) and mla.device_status() == 0
        expired += st == 8
        for x, s in zip(planes, start):
            got, old = flat(x), flat(s)
            new = (got[dst] == old[src]).all(1)
            kept = (got[dst] == old[dst]).all(1)
            assert bool((new | kept).all())                      # a row has moved whole, or not at all
            assert bool(new.all()) if st == 0 else bool(kept.any())   # and the status tells which
            other = torch.ones(got.shape[0], dtype=torch.bool, device="cuda")
            other[dst] = False
            assert torch.equal(got[other], old[other])           # sources, and slots behind the lists
    assert expired > 0
