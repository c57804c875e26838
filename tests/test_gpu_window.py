"""GPU parity of the decode over a sliding window and sink tokens, all kernels and storage types."""
from __future__ import annotations

import numpy as np
import pytest

import bounded_ref as R
import workloads as W

pytestmark = pytest.mark.gpu

F32 = W.WORKLOADS[0].with_(contiguous=False, spare_blocks=2)
BF16 = W.WORKLOADS[2].with_(spare_blocks=2)
MTP = W.WORKLOADS[3].with_(spare_blocks=2)
FP8 = W.WORKLOADS[4].with_(spare_blocks=2)


def hide(inp, win, sinks):
    """Tokens that no query row sees become NaN in the cache, and the blocks that hold none but those
    lose their id: neither may be looked at."""
    w = inp["workload"]
    inp = dict(inp, block_table=inp["block_table"].copy())
    for k in ("kv_cache", "k_rope_cache", "kv_scale"):
        inp[k] = None if inp[k] is None else inp[k].copy()
    for b, L in enumerate(int(x) for x in inp["seq_lens"]):
        see = np.zeros(L, bool)
        for s in range(w.Sq):
            see |= R.seen(w, L, s, win, sinks).numpy()
        for i in range((L + w.block_size - 1) // w.block_size):
            lo, hi = i * w.block_size, min(L, (i + 1) * w.block_size)
            blk = inp["block_table"][b, i]
            gone = np.nonzero(~see[lo:hi])[0]
            if w.cache_dtype == W.E4M3:
                inp["kv_cache"][blk, gone] = W.E4M3_NAN
                inp["k_rope_cache"][blk, gone] = W.BF16_NAN
                inp["kv_scale"][blk, gone] = np.nan
            else:
                inp["kv_cache"][blk, gone] = np.nan if w.cache_dtype == W.F32 else W.BF16_NAN
            # a window's first row may see nothing of a block between the sinks and the window
            if gone.size == hi - lo and sinks <= lo and hi <= L - (w.Sq - 1 if w.causal else 0) - win:
                inp["block_table"][b, i] = -1
    return inp


def run(inp, win, sinks, **kw):
    import torch
    import head_latent_attention_split_b200 as mla
    t, w = W.to_torch(inp), inp["workload"]
    out, lse = mla.window_decode(t["q_lat"], t["q_rope"], t["kv_cache"], t["block_table"], t["seq_lens"], w.scale, win,
                                 sinks=sinks, causal=w.causal, k_rope_cache=t["k_rope_cache"], kv_scale=t["kv_scale"],
                                 **kw)
    torch.cuda.synchronize()
    return out, lse, mla.device_status()


def close(out, lse, ref, what=""):
    o, l, bo, bl = ref
    o1, l1 = out.double().cpu(), lse.double().cpu()
    assert bool((o1 - o).abs().le(bo).all()), f"{what}: out off by {((o1 - o).abs() / bo.clamp(min=1e-300)).max():.3g} bounds"
    inf = l.isinf()
    assert bool((l1.isinf() == inf).all()) and bool((l1[inf] == l[inf]).all())
    assert bool((l1[~inf] - l[~inf]).abs().le(bl[~inf]).all()), f"{what}: lse off by {(l1 - l)[~inf].abs().max():.3g}"


CASES = [
    # (workload, kernel, window, sinks, workers)
    (F32.with_(B=4, seq_lens=(0, 1, 64, 200)), "auto", 24, 4, 0),
    (F32.with_(B=3, seq_lens=(65, 300, 130), block_size=16, r=48, d_r=0, scale=0.2), "auto", 33, 17, 5),
    (F32.with_(B=2, Sq=3, H=5, causal=True, seq_lens=(2, 150), block_size=32), "auto", 1, 0, 0),
    (BF16.with_(B=3, seq_lens=(1, 63, 700)), "simt", 100, 3, 0),
    (BF16.with_(B=5, seq_lens=(1, 64, 700, 0, 129)), "auto", 1, 0, 0),
    (BF16.with_(B=4, seq_lens=(1000, 64, 2111, 640)), "auto", 128, 64, 0),
    (BF16.with_(B=4, seq_lens=(1000, 64, 2111, 640)), "auto", 100, 5, 3),
    (BF16.with_(B=3, seq_lens=(900, 65, 333), H=20), "auto", 70, 200, 1),
    (BF16.with_(B=3, seq_lens=(900, 65, 333), H=8, out_dtype=W.F32), "auto", 64, 0, 0),
    (BF16.with_(B=3, seq_lens=(900, 190, 333)), "tcgen05", 100, 5, 0),
    (MTP.with_(B=5, seq_lens=(1, 2, 700, 65, 1300)), "auto", 127, 4, 0),
    (MTP.with_(B=4, Sq=3, H=48, seq_lens=(2, 700, 66, 1300)), "auto", 1, 1, 7),
    (MTP.with_(B=3, seq_lens=(1, 400, 129)), "tcgen05", 65, 2, 0),
    (FP8.with_(B=4, seq_lens=(1, 63, 1000, 450)), "auto", 100, 4, 0),
    (FP8.with_(B=3, Sq=2, H=32, causal=True, seq_lens=(1, 700, 129)), "auto", 64, 70, 5),
    (FP8.with_(B=2, seq_lens=(300, 90)), "simt", 40, 2, 0),
    (FP8.with_(B=4, seq_lens=(1, 63, 1000, 450)), "tcgen05", 100, 4, 0),
    (FP8.with_(B=3, Sq=2, H=80, causal=True, seq_lens=(2, 1500, 129)), "tc_pair", 700, 70, 3),
    (FP8.with_(B=2, seq_lens=(300, 500), zero_every=7, tiny_every=5), "auto", 200, 3, 0),
    (FP8.with_(B=2, seq_lens=(300, 500), tiny_every=2, tiny_exp=-18, out_dtype=W.F32), "auto", 200, 3, 2),
    (FP8.with_(B=2, seq_lens=(300, 500), zero_every=1), "auto", 200, 3, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0].name}-S{c[0].Sq}H{c[0].H}-{c[1]}-w{c[2]}s{c[3]}W{c[4]}")
def test_window_decode_matches_the_definition(case):
    import torch
    w, kernel, win, sinks, workers = case
    inp = W.make_inputs(w)
    ref = R.window(inp, win, sinks)
    od = W.F32 if w.out_dtype == W.F32 else None
    out, lse, st = run(hide(inp, win, sinks), win, sinks, kernel=kernel, num_workers=workers, out_dtype=od)
    assert st == 0
    assert out.dtype == (torch.float32 if w.out_dtype == W.F32 else torch.bfloat16)
    close(out, lse, ref)


@pytest.mark.parametrize("w", [F32.with_(B=3, seq_lens=(1, 64, 200)), BF16.with_(B=3, seq_lens=(1, 640, 1300)),
                               MTP.with_(B=3, seq_lens=(1, 700, 65)), FP8.with_(B=2, seq_lens=(65, 800))],
                         ids=lambda w: w.name)
def test_a_window_over_everything_is_the_decode(w):
    import torch
    import head_latent_attention_split_b200 as mla
    inp = W.make_inputs(w)
    t = W.to_torch(inp)
    ref = mla.decode(t["q_lat"], t["q_rope"], t["kv_cache"], t["block_table"], t["seq_lens"], w.scale, w.causal,
                     t["k_rope_cache"], t["kv_scale"])
    for win, sinks in ((int(max(inp["seq_lens"])), 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1)):
        # (an e4m3 cache's decode runs the channel-split kernel, its window decode the split-role one)
        out, lse, st = run(inp, win, sinks, kernel="tcgen05" if w.cache_dtype == W.E4M3 else "auto")
        assert st == 0 and torch.equal(out, ref[0]) and torch.equal(lse, ref[1]), (win, sinks)


def test_runs_are_identical_and_match_under_any_worker_count():
    import torch
    w = BF16.with_(B=4, seq_lens=(1500, 64, 2111, 640))
    inp = W.make_inputs(w)
    ref = R.window(inp, 600, 4)
    for workers in (0, 1, 2, 5, 74):
        a, b = run(inp, 600, 4, num_workers=workers), run(inp, 600, 4, num_workers=workers)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        close(a[0], a[1], ref, f"W={workers}")


@pytest.mark.parametrize("w,kernel", [(F32, "auto"), (BF16, "auto"), (BF16, "tcgen05"), (FP8, "auto")],
                         ids=["f32", "bf16", "bf16-tcgen05", "fp8"])
def test_bad_lengths_and_visible_bad_blocks_poison_their_sequence_only(w, kernel):
    w = w.with_(B=4, seq_lens=(300, 400, 500, 130))
    inp = W.make_inputs(w)
    ref = R.window(inp, 100, 4)
    bad = dict(inp, block_table=inp["block_table"].copy(), seq_lens=inp["seq_lens"].copy())
    bad["block_table"][1, (400 - 100) // w.block_size] = inp["num_blocks"]   # a block of the window
    bad["seq_lens"][2] = -3
    out, lse, st = run(bad, 100, 4, kernel=kernel)
    assert st in (6, 7)
    for b in (1, 2):
        assert bool(out[b].isnan().all()) and bool(lse[b].isnan().all())
    for b in (0, 3):
        close(out[b], lse[b], tuple(x[b] for x in ref))


def test_graph_replay_other_stream_and_given_buffers():
    import torch
    import head_latent_attention_split_b200 as mla
    w = MTP.with_(B=3, seq_lens=(700, 65, 1300))
    inp = W.make_inputs(w)
    t = W.to_torch(inp)
    p = mla.params_for(t["q_lat"], t["q_rope"], t["kv_cache"], t["block_table"], w.scale, w.causal)
    ws = torch.empty(mla.workspace_size(p), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(t["q_lat"]), torch.empty(t["q_lat"].shape[:3], device="cuda")

    def step(**kw):
        return mla.window_decode(t["q_lat"], t["q_rope"], t["kv_cache"], t["block_table"], t["seq_lens"], w.scale, 200,
                                 sinks=4, causal=True, **kw)
    ref = R.window(inp, 200, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    with torch.cuda.stream(side):
        step(out=out, lse=lse, workspace=ws)
    side.synchronize()
    close(*got, ref)
    close(out, lse, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(out=out, lse=lse, workspace=ws)
    # new queries and lengths in place, then a replay
    w2 = w.with_(seed=77, seq_lens=(1290, 640, 3))
    inp2 = dict(W.make_inputs(w2.with_(seq_lens=w.seq_lens)))
    inp2["seq_lens"] = np.array((690, 33, 1290), np.int32)
    t2 = W.to_torch(inp2)
    for k in ("q_lat", "q_rope", "kv_cache", "block_table", "seq_lens"):
        t[k].copy_(t2[k])
    out.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    close(out, lse, R.window(inp2, 200, 4))
    assert mla.device_status() == 0


def test_front_end_refuses_tensors_that_do_not_fit():
    import torch
    import head_latent_attention_split_b200 as mla
    w = BF16.with_(B=2, seq_lens=(70, 130), H=16)
    t = W.to_torch(W.make_inputs(w))
    args = [t[k] for k in ("q_lat", "q_rope", "kv_cache", "block_table", "seq_lens")]

    def call(i=None, x=None, **kw):
        a = list(args)
        if i is not None:
            a[i] = x
        return mla.window_decode(*a, w.scale, kw.pop("window", 8), **kw)
    call()
    for i, x, err in ((0, args[0].float(), TypeError), (1, args[1][:, :, :8], ValueError),
                      (2, args[2].transpose(0, 1), ValueError), (2, args[2][:, :, :512].contiguous(), ValueError),
                      (3, args[3].long(), TypeError), (4, args[4][:1], ValueError), (4, args[4].cpu(), ValueError),
                      (0, args[0][..., ::2], ValueError)):
        with pytest.raises(err):
            call(i, x)
    with pytest.raises(ValueError):
        call(kv_scale=torch.zeros(2, 64, device="cuda"))
    with pytest.raises(mla.MlaError):
        call(window=0)
    with pytest.raises(mla.MlaError):
        call(sinks=-1)
    with pytest.raises(TypeError):
        call(out=torch.empty(args[0].shape, device="cuda"))
    torch.cuda.synchronize()
    assert mla.device_status() == 0


@pytest.mark.parametrize("w,kernel", [(BF16, "tc_pair"), (BF16, "tcgen05"), (FP8, "tc_pair"), (FP8, "tcgen05")],
                         ids=["bf16-pair", "bf16-tcgen05", "fp8-pair", "fp8-tcgen05"])
def test_an_expired_wait_ends_cleanly(w, kernel):
    import torch
    import head_latent_attention_split_b200 as mla
    w = w.with_(B=3, seq_lens=(900, 300, 1500))
    inp = W.make_inputs(w)
    ref = R.window(inp, 600, 4)
    mla.set_wait_timeout_ns(200)
    try:
        out, lse, st = run(inp, 600, 4, kernel=kernel)
    finally:
        mla.set_wait_timeout_ns(0)
    assert st == 8 and mla.device_status() == 0
    nan = lse.isnan()
    assert bool(nan.any()) and bool(out[nan].isnan().all())
    out, lse, st = run(inp, 600, 4, kernel=kernel)
    assert st == 0
    close(out, lse, ref)


def test_buffers_are_not_written_past_their_ends():
    import torch
    import head_latent_attention_split_b200 as mla
    for w, win in ((MTP.with_(B=3, H=20, seq_lens=(700, 65, 1300)), 300), (FP8.with_(B=3, H=40, seq_lens=(700, 0, 1300)), 600),
                   (F32.with_(B=3, seq_lens=(100, 0, 64)), 30)):
        inp = W.make_inputs(w)
        t = W.to_torch(inp)
        p = mla.params_for(t["q_lat"], t["q_rope"], t["kv_cache"], t["block_table"], w.scale, w.causal)
        need, n, guard = mla.workspace_size(p), t["q_lat"].numel(), 4096
        ob = torch.full((n + 2 * guard,), 7.0, dtype=t["q_lat"].dtype, device="cuda")
        lb = torch.full((n // w.r + 2 * guard,), 7.0, device="cuda")
        wb = torch.full((need + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
        out, lse = ob[guard:guard + n].view(t["q_lat"].shape), lb[guard:guard + n // w.r].view(t["q_lat"].shape[:3])
        mla.window_decode(t["q_lat"], t["q_rope"], t["kv_cache"], t["block_table"], t["seq_lens"], w.scale, win, sinks=2,
                          causal=w.causal, k_rope_cache=t["k_rope_cache"], kv_scale=t["kv_scale"], out=out, lse=lse,
                          workspace=wb[guard:guard + need])
        torch.cuda.synchronize()
        assert mla.device_status() == 0
        for buf, v in ((ob, 7.0), (lb, 7.0), (wb, 0xA5)):
            assert bool((buf[:guard] == v).all()) and bool((buf[-guard:] == v).all())
        close(out, lse, R.window(inp, win, 2))


def test_a_large_batch_of_short_and_empty_sequences():
    rng = np.random.default_rng(3)
    lens = tuple(int(x) for x in rng.integers(0, 400, 300))
    for w in (BF16.with_(B=300, H=4, seq_lens=lens), FP8.with_(B=300, H=4, seq_lens=lens), F32.with_(B=300, seq_lens=lens)):
        inp = W.make_inputs(w)
        out, lse, st = run(hide(inp, 90, 3), 90, 3)
        assert st == 0
        close(out, lse, R.window(inp, 90, 3))


# Every way to cut the tile lists among the workers: evenly, whole sequences (one or more per worker) and parts of
# a sequence, with more parts than a short or empty sequence has tiles.
@pytest.mark.parametrize("w", [BF16.with_(B=4, seq_lens=(0, 3000, 2500, 70)), MTP.with_(B=3, seq_lens=(2600, 1, 1900)),
                               FP8.with_(B=3, seq_lens=(2700, 130, 2200)), BF16.with_(B=2, H=24, seq_lens=(2200, 2600))],
                         ids=["bf16", "two-row-groups", "fp8", "few-rows"])
@pytest.mark.parametrize("win,sinks", [(1700, 70), (90, 1)])
def test_every_cut_of_the_tile_lists(w, win, sinks):
    inp = W.make_inputs(w)
    ref, hidden = R.window(inp, win, sinks), hide(inp, win, sinks)
    for workers in (0, 1, 3, 8, 13, 30, 37):
        out, lse, st = run(hidden, win, sinks, num_workers=workers)
        assert st == 0
        close(out, lse, ref, f"W={workers}")


def test_a_bad_block_in_one_part_poisons_the_whole_sequence():
    w = BF16.with_(B=2, seq_lens=(2600, 2700))
    inp = W.make_inputs(w)
    ref = R.window(inp, 2000, 4)
    for tile in (0, 12, 24, 40):   # the sinks' block, and blocks of different parts of the window
        bad = dict(inp, block_table=inp["block_table"].copy())
        bad["block_table"][1, tile] = inp["num_blocks"]
        out, lse, st = run(bad, 2000, 4)
        assert st == 6   # MLA_ERR_BAD_BLOCK_ID
        assert bool(out[1].isnan().all()) and bool(lse[1].isnan().all())
        close(out[:1], lse[:1], tuple(x[:1] for x in ref), f"tile {tile}")


def test_a_large_batch_with_one_long_window():
    w = BF16.with_(B=80, H=32, seq_lens=(6000,) + tuple(1 + 7 * i for i in range(79)))   # an even cut, many rows to merge
    inp = W.make_inputs(w)
    out, lse, st = run(hide(inp, 5500, 3), 5500, 3)
    assert st == 0
    close(out, lse, R.window(inp, 5500, 3))
