"""GPU checks of the eviction: the choice of the tokens that stay (bit for bit) and their copy."""
from __future__ import annotations

import numpy as np
import pytest

import bounded_ref as R
import workloads as W

pytestmark = pytest.mark.gpu


def select(mass, lens, budget, sinks, recent):
    import torch
    import head_latent_attention_split_b200 as mla
    idx, cnt = mla.evict_select(torch.from_numpy(mass).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), budget,
                                sinks=sinks, recent=recent)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), cnt.cpu().numpy(), mla.device_status()


def masses(kind, B, S, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "lognormal":
        return np.exp(2 * rng.standard_normal((B, S))).astype(np.float32)
    if kind == "ties":
        return rng.integers(0, 4, (B, S)).astype(np.float32)
    if kind == "equal":
        return np.full((B, S), 3.5, np.float32)
    if kind == "signed":
        x = rng.standard_normal((B, S)).astype(np.float32)
        x[:, ::3] = 0.0
        x[:, 1::6] = -0.0
        return x
    x = rng.standard_normal((B, S)).astype(np.float32)   # special values
    x[:, ::5] = np.inf
    x[:, 1::7] = -np.inf
    x[:, 2::11] = np.nan
    x[:, 3::13] = -np.nan
    x[:, 4::9] = np.float32(1e-42)
    return x


@pytest.mark.parametrize("kind", ["lognormal", "ties", "equal", "signed", "special"])
@pytest.mark.parametrize("S,lens,budget,sinks,recent", [
    (100, (0, 1, 7, 8, 9, 100), 8, 2, 3),
    (1001, (1001, 500, 64, 999), 64, 4, 16),
    (1001, (1001, 500, 64, 999), 64, 64, 0),      # nothing to choose
    (1001, (1001, 333), 1, 0, 0),
    (1001, (1001, 1000), 1000, 0, 0),
    (16384, (16384, 16383, 5000), 2048, 4, 512),
    (16385, (16385, 16384, 100), 777, 1, 1),      # a cluster of two CTAs
    (70003, (70003, 65537, 20000), 5001, 33, 70),
])
def test_select_matches_a_sort(kind, S, lens, budget, sinks, recent):
    mass = masses(kind, len(lens), S, seed=S + budget)
    for b, L in enumerate(lens):
        mass[b, L:] = np.nan   # past the length: not looked at
    idx, cnt, st = select(mass, lens, budget, sinks, recent)
    ref_i, ref_c = R.evict(mass, lens, budget, sinks, recent)
    assert st == 0
    np.testing.assert_array_equal(cnt, ref_c)
    np.testing.assert_array_equal(idx, ref_i)


@pytest.mark.parametrize("kind", ["lognormal", "ties", "special"])
@pytest.mark.parametrize("S", [4095, 4096, 4097, 8191, 8192, 8193])
def test_select_around_the_rows_that_change_the_keys_per_thread(kind, S):
    lens = (S, S - 1, S - 5, 1025)
    mass = masses(kind, len(lens), S, seed=S)
    idx, cnt, st = select(mass, lens, 1024, 3, 200)
    ref_i, ref_c = R.evict(mass, lens, 1024, 3, 200)
    assert st == 0 and np.array_equal(idx, ref_i) and np.array_equal(cnt, ref_c)


def test_select_rows_longer_than_a_cluster_holds():
    S = 8 * 16384 * 2 + 77
    mass = masses("ties", 2, S, 3) + masses("lognormal", 2, S, 4).round(1)
    lens = (S, S - 16400)
    idx, cnt, st = select(mass, lens, 3000, 4, 100)
    ref_i, ref_c = R.evict(mass, lens, 3000, 4, 100)
    assert st == 0 and np.array_equal(idx, ref_i) and np.array_equal(cnt, ref_c)


def test_select_bad_length():
    mass = masses("lognormal", 3, 200)
    idx, cnt, st = select(mass, (100, 201, -1), 50, 0, 0)
    assert st == 7 and cnt.tolist() == [50, 0, 0] and (idx[1:] == -1).all()
    np.testing.assert_array_equal(idx[0], R.evict(mass[:1], (100,), 50, 0, 0)[0][0])


def pool(dtype, nb, bs, r, d_r, seed):
    import torch
    rng = np.random.default_rng(seed)
    dev = "cuda"
    if dtype == W.E4M3:
        return (torch.from_numpy(rng.integers(0, 256, (nb, bs, r), dtype=np.uint8)).to(dev),
                torch.from_numpy(rng.integers(0, 1 << 15, (nb, bs, d_r)).astype(np.int16)).view(torch.bfloat16).to(dev),
                torch.from_numpy(rng.standard_normal((nb, bs)).astype(np.float32)).to(dev))
    x = rng.standard_normal((nb, bs, r + d_r)).astype(np.float32)
    x = torch.from_numpy(x).to(dev)
    return (x.bfloat16() if dtype == W.BF16 else x), None, None


@pytest.mark.parametrize("dtype,bs,r,d_r", [(W.BF16, 64, 512, 64), (W.E4M3, 64, 512, 64), (W.F32, 32, 16, 8),
                                            (W.BF16, 16, 18, 0), (W.BF16, 8, 5, 4), (W.E4M3, 16, 7, 3), (W.F32, 5, 3, 0)])
@pytest.mark.parametrize("with_mass", [True, False])
def test_compact_copies_the_listed_rows_and_nothing_else(dtype, bs, r, d_r, with_mass):
    import torch
    import head_latent_attention_split_b200 as mla
    lens, budget = [5 * bs + 3, 2, 0, 7 * bs, 40], 2 * bs + 1
    B, mb, db = len(lens), 7 + 40 // bs, 4
    nb = B * (mb + db) + 3
    rng = np.random.default_rng(bs + r)
    perm = rng.permutation(nb).astype(np.int32)
    bt, dt = perm[:B * mb].reshape(B, mb).copy(), perm[B * mb:B * (mb + db)].reshape(B, db).copy()
    mass = masses("lognormal", B, mb * bs, 1)
    idx, cnt = R.evict(mass, lens, budget, 1, min(3, budget - 1))
    kv, kr, ks = pool(dtype, nb, bs, r, d_r, 2)
    before = [x.clone() if x is not None else None for x in (kv, kr, ks)]
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    m_in, m_out = (dev(mass), torch.full((B, budget + 9), 5.0, device="cuda")) if with_mass else (None, None)
    mla.cache_compact(kv, dev(bt), dev(dt), dev(idx), dev(cnt), k_rope_cache=kr, kv_scale=ks, mass=m_in, mass_out=m_out)
    torch.cuda.synchronize()
    assert mla.device_status() == 0
    for x, old in zip((kv, kr, ks), before):
        if x is None:
            continue
        want = old.reshape(nb * bs, -1).clone()
        for b in range(B):
            for j in range(int(cnt[b])):
                t = int(idx[b, j])
                want[int(dt[b, j // bs]) * bs + j % bs] = old.reshape(nb * bs, -1)[int(bt[b, t // bs]) * bs + t % bs]
        bits = lambda y: y.contiguous().view(torch.uint8)  # noqa: E731
        assert torch.equal(bits(x.reshape(nb * bs, -1)), bits(want))
    if with_mass:
        want = np.zeros((B, budget + 9), np.float32)
        for b in range(B):
            want[b, :cnt[b]] = mass[b, idx[b, :cnt[b]]]
        np.testing.assert_array_equal(m_out.cpu().numpy(), want)


def test_compact_flags_bad_entries_and_skips_them():
    import torch
    import head_latent_attention_split_b200 as mla
    bs, nb = 16, 12
    kv = torch.arange(nb * bs * 8, dtype=torch.float32, device="cuda").reshape(nb, bs, 8)
    old = kv.clone()
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    bt, dt = i([[0, 1], [2, -1], [3, 4], [5, 6]]), i([[7], [8], [99], [10]])
    idx = i([[0, 17, 32, -1], [3, 16, 20, 5], [0, 1, 2, 3], [2, 2, 9, 31]])
    mass = torch.arange(4 * 32, dtype=torch.float32, device="cuda").reshape(4, 32)
    out = torch.empty(4, 4, device="cuda")
    mla.cache_compact(kv, bt, dt, idx, i([3, 4, 2, 5]), mass=mass, mass_out=out)
    torch.cuda.synchronize()
    assert mla.device_status() in (6, 7)
    want = old.clone()
    want[7, 0], want[7, 1] = old[0, 0], old[1, 1]                    # entry 2 is past the table
    want[8, 0], want[8, 3] = old[2, 3], old[2, 5]                    # entries 1, 2 map to block -1
    want[10, 0], want[10, 1], want[10, 2], want[10, 3] = old[5, 2], old[5, 2], old[5, 9], old[6, 15]   # twice is fine
    assert torch.equal(kv, want)
    got = out.cpu().numpy()
    assert got[0, :2].tolist() == [0, 17] and np.isnan(got[0, 2]) and got[0, 3] == 0
    assert np.isnan(got[1, 1:3]).all() and got[1, [0, 3]].tolist() == [35, 37]
    assert np.isnan(got[2, :2]).all() and (got[2, 2:] == 0).all()
    assert got[3].tolist() == [98, 98, 105, 127]


def test_front_end_refuses_tensors_that_do_not_fit():
    import torch
    import head_latent_attention_split_b200 as mla
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    for bad in (dict(mass=f(2, 64).half()), dict(mass=f(64, 2).T), dict(seq_lens=i(3)), dict(seq_lens=f(2))):
        a = dict(mass=f(2, 64), seq_lens=i(2), **{})
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            mla.evict_select(a["mass"], a["seq_lens"], 8)
    for budget, sinks, recent in ((0, 0, 0), (8, 9, 0), (8, 4, 5), (8, -1, 0)):
        with pytest.raises(mla.MlaError):
            mla.evict_select(f(2, 64), i(2), budget, sinks=sinks, recent=recent)
    kv, bt, dt, idx, cnt = f(4, 16, 24), i(2, 1), i(2, 1), i(2, 16), i(2)
    with pytest.raises(mla.MlaError):
        mla.cache_compact(kv, bt, bt, idx, cnt)                 # one table for both sides
    with pytest.raises(mla.MlaError):
        mla.cache_compact(kv, bt, dt, i(2, 17), cnt)            # more entries than slots
    with pytest.raises(mla.MlaError):
        mla.cache_compact(kv, bt, dt, idx, cnt, mass=f(2, 16))  # mass without mass_out
    with pytest.raises((TypeError, ValueError)):
        mla.cache_compact(kv, bt, dt, idx, cnt.long())
    torch.cuda.synchronize()
    assert mla.device_status() == 0


def test_an_expired_wait_ends_cleanly():
    import torch
    import head_latent_attention_split_b200 as mla
    B, bs, n = 40, 64, 40
    kv = torch.randn(2 * B * 8, bs, 576, device="cuda").bfloat16()
    old = kv.clone()
    i32 = lambda x: x.to(torch.int32).cuda()  # noqa: E731
    bt, dt = i32(torch.arange(B * 8).reshape(B, 8)), i32(torch.arange(B * 8, 2 * B * 8).reshape(B, 8))
    idx, cnt = i32(torch.arange(0, 8 * bs, 2)[None].expand(B, -1)).contiguous(), i32(torch.full((B,), 4 * bs))
    mla.set_wait_timeout_ns(1)
    try:
        mla.cache_compact(kv, bt, dt, idx, cnt)
        torch.cuda.synchronize()
    finally:
        mla.set_wait_timeout_ns(0)
    assert mla.device_status() in (0, 8) and mla.device_status() == 0
    assert torch.equal(kv[:B * 8], old[:B * 8])          # the sources are never written
    mla.cache_compact(kv, bt, dt, idx, cnt)
    torch.cuda.synchronize()
    assert mla.device_status() == 0
    rows = lambda x: x.reshape(B, 8 * bs, 576)  # noqa: E731
    assert torch.equal(rows(kv[B * 8:])[:, :4 * bs], rows(kv[:B * 8])[:, ::2][:, :4 * bs])
    assert torch.equal(rows(kv[B * 8:])[:, 4 * bs:], rows(old[B * 8:])[:, 4 * bs:])


def test_select_and_compact_in_a_graph():
    import torch
    import head_latent_attention_split_b200 as mla
    B, S, bs, budget = 3, 640, 64, 200
    kv = torch.randn(B * 10 + B * 4, bs, 576, device="cuda").bfloat16()
    perm = torch.randperm(B * 14, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    bt, dt = perm[:B * 10].reshape(B, 10).contiguous(), perm[B * 10:].reshape(B, 4).contiguous()
    mass, lens = torch.rand(B, S, device="cuda"), torch.tensor([640, 100, 333], dtype=torch.int32, device="cuda")
    idx, cnt = torch.empty(B, budget, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    out = torch.empty(B, 256, device="cuda")

    def step():
        mla.evict_select(mass, lens, budget, sinks=4, recent=50, indices=idx, counts=cnt)
        mla.cache_compact(kv, bt, dt, idx, cnt, mass=mass, mass_out=out)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    mass.copy_(torch.rand(B, S, generator=torch.Generator().manual_seed(2)))
    lens.copy_(torch.tensor([200, 640, 201], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert mla.device_status() == 0
    ref_i, ref_c = R.evict(mass.cpu().numpy(), lens.cpu().numpy(), budget, 4, 50)
    np.testing.assert_array_equal(idx.cpu().numpy(), ref_i)
    np.testing.assert_array_equal(cnt.cpu().numpy(), ref_c)
    flat = kv.reshape(-1, 576)
    for b in range(B):
        t = torch.from_numpy(ref_i[b, :ref_c[b]].astype(np.int64)).cuda()
        j = torch.arange(ref_c[b], device="cuda")
        assert torch.equal(flat[dt[b, j // bs].long() * bs + j % bs], flat[bt[b, t // bs].long() * bs + t % bs])
        assert torch.equal(out[b, :ref_c[b]], mass[b, t]) and bool((out[b, ref_c[b]:] == 0).all())


@pytest.mark.parametrize("bad", [dict(budget=2 ** 32 + 8), dict(sinks=2 ** 32), dict(recent=-2 ** 32 + 2)])
def test_select_numbers_beyond_32_bits_are_refused_not_cut(bad):
    import torch
    import head_latent_attention_split_b200 as mla
    mass, lens = torch.ones(2, 40, device="cuda"), torch.tensor([40, 30], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="32 bits"):
        mla.evict_select(mass, lens, **{**dict(budget=8, sinks=1, recent=2), **bad})


def test_back_to_back_selections_and_copies_see_each_others_writes():
    import torch
    import head_latent_attention_split_b200 as mla
    g = torch.Generator(device="cuda").manual_seed(5)
    B, S, bs, budget = 40, 1000, 64, 300
    mb, db = 16, 5
    perm = torch.randperm(B * (mb + db), generator=g, device="cuda").int()
    bt, dt = perm[:B * mb].reshape(B, mb).contiguous(), perm[B * mb:].reshape(B, db).contiguous()
    kv = torch.empty(B * (mb + db), bs, 576, dtype=torch.bfloat16, device="cuda")
    idx, cnt = torch.empty(B, budget, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    out, lens = torch.empty(B, budget, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    j = torch.arange(budget, device="cuda")
    for i in range(40):   # nothing waits on the host in between; every buffer is used again
        kv.normal_(generator=g)
        mass = torch.rand(B, S, generator=g, device="cuda")
        lens.random_(200, S + 1, generator=g)
        mla.evict_select(mass, lens, budget, 4, 50, indices=idx, counts=cnt)
        mla.cache_compact(kv, bt, dt, idx, cnt, mass=mass, mass_out=out)
        t = idx.long().clamp(min=0)
        src = (bt.gather(1, t // bs).long() * bs + t % bs)
        dst = dt[:, j // bs].long() * bs + j % bs
        live = j < cnt[:, None]
        flat = kv.view(-1, 576)
        wrong += ((flat[src] != flat[dst]).any(-1) & live).sum() + ((out != mass.gather(1, t)) & live).sum()
        wrong += (cnt != lens.clamp(max=budget)).sum() + ((idx >= 0) != live).sum()
    assert int(wrong) == 0 and mla.device_status() == 0
