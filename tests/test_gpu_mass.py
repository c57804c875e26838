"""GPU parity of the attention weight per cached token, both kernels and all storage types."""
from __future__ import annotations

import numpy as np
import pytest

import bounded_ref as R
import workloads as W

pytestmark = pytest.mark.gpu

F32 = W.WORKLOADS[0].with_(contiguous=False, spare_blocks=2)
BF16 = W.WORKLOADS[2].with_(spare_blocks=2, c_std=0.3)
MTP = W.WORKLOADS[3].with_(spare_blocks=2, c_std=0.3)
FP8 = W.WORKLOADS[4].with_(spare_blocks=2)


def setup(w, extra=5):
    """Inputs, the lse that a decode leaves (fp32) and the earlier weights (S columns, some past every length)."""
    import torch
    inp = W.make_inputs(w)
    S = max(int(x) for x in inp["seq_lens"]) + extra
    lse = R.window(inp, 1 << 30, 0)[1].float()
    g = torch.Generator().manual_seed(w.seed + 5)
    return inp, lse, torch.rand(w.B, S, generator=g)


def run(inp, lse, mass_in, mass, **kw):
    import torch
    import head_latent_attention_split_b200 as mla
    t, w = W.to_torch(inp), inp["workload"]
    mla.attention_mass(t["q_lat"], t["q_rope"], t["kv_cache"], t["block_table"], t["seq_lens"], lse.cuda(), w.scale, mass,
                       mass_in=mass_in, causal=w.causal, k_rope_cache=t["k_rope_cache"], kv_scale=t["kv_scale"], **kw)
    torch.cuda.synchronize()
    return mla.device_status()


def check(inp, lse, mass_in, got, before):
    ref, bound = R.mass(inp, lse.double(), mass_in.double())
    got = got.double().cpu()
    for b, L in enumerate(int(x) for x in inp["seq_lens"]):
        d = (got[b, :L] - ref[b, :L]).abs()
        assert bool(d.le(bound[b, :L]).all()), f"sequence {b}: {(d / bound[b, :L]).max():.3g} bounds"
        assert bool((got[b, L:] == before).all())   # entries past the length are left alone


CASES = [
    (F32.with_(B=4, seq_lens=(0, 1, 64, 200)), "auto", 0),
    (F32.with_(B=3, Sq=2, H=5, causal=True, seq_lens=(1, 70, 333), block_size=16, r=50, d_r=6, scale=0.2), "auto", 0),
    (F32.with_(B=2, seq_lens=(40, 100), d_r=0, scale=-0.3), "auto", 0),
    (BF16.with_(B=3, seq_lens=(1, 63, 300), H=12), "simt", 0),
    (FP8.with_(B=2, seq_lens=(90, 130), H=9), "simt", 0),
    (BF16.with_(B=5, seq_lens=(1, 64, 700, 0, 129)), "auto", 0),
    (BF16.with_(B=3, seq_lens=(1000, 65, 2111)), "auto", 2),
    (BF16.with_(B=3, seq_lens=(900, 65, 333), H=20), "auto", 0),
    (BF16.with_(B=2, seq_lens=(500, 127), H=1), "auto", 1),
    (MTP.with_(B=5, seq_lens=(1, 2, 700, 65, 1300)), "auto", 0),
    (MTP.with_(B=3, Sq=3, H=48, seq_lens=(2, 700, 129)), "auto", 3),
    (BF16.with_(B=2, Sq=70, H=16, causal=True, seq_lens=(70, 257)), "auto", 0),
    (FP8.with_(B=4, seq_lens=(1, 63, 1000, 450)), "auto", 0),
    (FP8.with_(B=3, Sq=2, H=80, causal=True, seq_lens=(1, 700, 129)), "auto", 4),
    (FP8.with_(B=2, seq_lens=(300, 500), zero_every=7, tiny_every=5), "auto", 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0].name}-S{c[0].Sq}H{c[0].H}-{c[1]}-W{c[2]}")
def test_attention_mass_matches_the_definition(case):
    import torch
    w, kernel, workers = case
    inp, lse, mass_in = setup(w)
    mass = torch.full(mass_in.shape, -7.0, device="cuda")
    assert run(inp, lse, mass_in.cuda(), mass, kernel=kernel, num_workers=workers) == 0
    check(inp, lse, mass_in, mass, -7.0)


@pytest.mark.parametrize("w", [F32.with_(B=2, seq_lens=(64, 200)), BF16.with_(B=2, seq_lens=(300, 64)),
                               MTP.with_(B=2, seq_lens=(2, 200)), FP8.with_(B=2, seq_lens=(300, 64))],
                         ids=lambda w: w.name)
def test_in_place_without_earlier_weights_and_twice(w):
    import torch
    inp, lse, mass_in = setup(w)
    zero = torch.zeros_like(mass_in)
    fresh = torch.zeros_like(mass_in).cuda()
    assert run(inp, lse, None, fresh) == 0
    check(inp, lse, zero, fresh, 0.0)
    again = torch.zeros_like(mass_in).cuda()
    assert run(inp, lse, None, again) == 0
    assert torch.equal(fresh, again)
    place = mass_in.cuda()
    assert run(inp, lse, place, place) == 0
    other = mass_in.cuda()
    assert run(inp, lse, mass_in.cuda(), other) == 0
    assert torch.equal(place, other)


def test_the_decodes_own_lse_gives_one_per_row():
    import torch
    import head_latent_attention_split_b200 as mla
    for w in (BF16.with_(B=3, seq_lens=(700, 1, 1300)), MTP.with_(B=2, seq_lens=(65, 1500)),
              FP8.with_(B=2, seq_lens=(900, 130)), F32.with_(B=2, seq_lens=(64, 200))):
        t = W.to_torch(W.make_inputs(w))
        a = (t["q_lat"], t["q_rope"], t["kv_cache"], t["block_table"], t["seq_lens"])
        kw = dict(causal=w.causal, k_rope_cache=t["k_rope_cache"], kv_scale=t["kv_scale"])
        _, lse = mla.decode(*a, w.scale, **kw)
        mass = mla.attention_mass(*a, lse, w.scale, torch.zeros(w.B, 1500, device="cuda"), **kw)
        got = mass.double().sum(1).cpu()
        # two fp32 score paths (2 x 600 half steps of a magnitude below 100) on every weight
        assert bool(((got - w.Sq * w.H).abs() < w.Sq * w.H * 2 * 600 * R.U32 * 100).all()), got


@pytest.mark.parametrize("w,kernel", [(F32, "auto"), (BF16, "simt"), (BF16, "auto"), (FP8, "auto")],
                         ids=["f32", "bf16-simt", "bf16", "fp8"])
def test_bad_lengths_and_blocks(w, kernel):
    import torch
    w = w.with_(B=4, seq_lens=(300, 400, 200, 130))
    inp, lse, mass_in = setup(w)
    bad = dict(inp, block_table=inp["block_table"].copy(), seq_lens=inp["seq_lens"].copy())
    bad["block_table"][1, 2] = inp["num_blocks"] + 3
    bad["seq_lens"][2] = mass_in.shape[1] + 1
    mass = torch.full(mass_in.shape, -7.0, device="cuda")
    assert run(bad, lse, mass_in.cuda(), mass, kernel=kernel) in (6, 7)
    got = mass.cpu()
    lo, hi = 2 * w.block_size, 3 * w.block_size
    assert bool(got[1, lo:hi].isnan().all()) and not bool(got[1, :lo].isnan().any()) and not bool(got[1, hi:].isnan().any())
    assert bool((got[2] == -7.0).all())
    ref, bound = R.mass(inp, lse.double(), mass_in.double())
    for b, L in ((0, 300), (3, 130)):
        assert bool((got[b, :L].double() - ref[b, :L]).abs().le(bound[b, :L]).all())


def test_graph_replay_and_other_stream():
    import torch
    import head_latent_attention_split_b200 as mla
    w = BF16.with_(B=3, seq_lens=(700, 65, 1300))
    inp, lse, mass_in = setup(w)
    t = W.to_torch(inp)
    l, mi, mass = lse.cuda(), mass_in.cuda(), torch.full(mass_in.shape, -7.0, device="cuda")

    def step(**kw):
        mla.attention_mass(t["q_lat"], t["q_rope"], t["kv_cache"], t["block_table"], t["seq_lens"], l, w.scale, mass,
                           mass_in=mi, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(stream=side)
    side.synchronize()
    check(inp, lse, mass_in, mass, -7.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    mi.mul_(2.0)
    t["seq_lens"].copy_(torch.tensor([690, 1, 1290], dtype=torch.int32))
    mass.fill_(-7.0)
    g.replay()
    torch.cuda.synchronize()
    # the lse of the longer lengths stays a valid input
    check(dict(inp, seq_lens=np.array([690, 1, 1290], np.int32)), lse, mass_in * 2, mass, -7.0)
    assert mla.device_status() == 0


@pytest.mark.parametrize("w", [BF16, MTP, FP8], ids=["bf16", "two-groups", "fp8"])
def test_an_expired_wait_ends_cleanly(w):
    import torch
    import head_latent_attention_split_b200 as mla
    w = w.with_(B=3, seq_lens=(900, 300, 1500))
    inp, lse, mass_in = setup(w)
    mass = torch.full(mass_in.shape, -7.0, device="cuda")
    mla.set_wait_timeout_ns(200)
    try:
        st = run(inp, lse, mass_in.cuda(), mass)
    finally:
        mla.set_wait_timeout_ns(0)
    assert st == 8 and mla.device_status() == 0
    assert bool(mass.isnan().any())
    mass.fill_(-7.0)
    assert run(inp, lse, mass_in.cuda(), mass) == 0
    check(inp, lse, mass_in, mass, -7.0)


def test_a_large_batch_of_short_and_empty_sequences():
    import torch
    rng = np.random.default_rng(4)
    lens = tuple(int(x) for x in rng.integers(0, 300, 200))
    for w in (BF16.with_(B=200, H=4, seq_lens=lens), FP8.with_(B=200, H=4, seq_lens=lens), F32.with_(B=200, seq_lens=lens)):
        inp, lse, mass_in = setup(w)
        mass = torch.full(mass_in.shape, -7.0, device="cuda")
        assert run(inp, lse, mass_in.cuda(), mass) == 0
        check(inp, lse, mass_in, mass, -7.0)


def test_front_end_refuses_tensors_that_do_not_fit():
    import torch
    import head_latent_attention_split_b200 as mla
    w = BF16.with_(B=2, seq_lens=(70, 130), H=16)
    t = W.to_torch(W.make_inputs(w))
    good = dict(q_lat=t["q_lat"], q_rope=t["q_rope"], kv_cache=t["kv_cache"], block_table=t["block_table"],
                seq_lens=t["seq_lens"], lse=torch.zeros(2, 1, 16, device="cuda"), softmax_scale=w.scale,
                mass=torch.zeros(2, 130, device="cuda"))
    mla.attention_mass(**good)
    for bad in (dict(lse=torch.zeros(2, 16, device="cuda")), dict(mass=torch.zeros(3, 130, device="cuda")),
                dict(mass=torch.zeros(130, 2, device="cuda").T), dict(mass_in=torch.zeros(2, 131, device="cuda")),
                dict(mass=torch.zeros(2, 130, device="cuda").double()), dict(q_rope=None), dict(seq_lens=t["seq_lens"].long())):
        with pytest.raises((TypeError, ValueError)):
            mla.attention_mass(**{**good, **bad})
    with pytest.raises(mla.MlaError):
        mla.attention_mass(**{**good, "kernel": "tc_pair"})
    torch.cuda.synchronize()
    assert mla.device_status() == 0
