"""CPU-only checks of the window decode, attention weight, eviction and draft verification: their
refusals (nothing is launched, no pointer is followed) and the references that the GPU tests use."""
import math

import numpy as np
import pytest

import oracle
import workloads as W
import bounded_ref as R

FAKE = 1 << 20   # a 256-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def m():
    from head_latent_attention_split_b200 import build as B
    B.build()
    import head_latent_attention_split_b200 as mod
    return mod


# ----------------------------------------------------------------------------- refusals, C ABI
DECODE = dict(B=2, Sq=1, H=4, r=16, d_r=8, block_size=64, num_blocks=2, max_blocks_per_seq=1, q_dtype=0, cache_dtype=0,
              out_dtype=0, causal=False, softmax_scale=0.2, num_workers=3, kernel="simt")
DECODE_PTRS = dict(q_lat=FAKE, q_rope=FAKE, kv_cache=FAKE, k_rope_cache=None, kv_scale=None, block_table=FAKE,
                   seq_lens=FAKE)


def _split(base, kw):
    ptrs = {k: kw.pop(k, v) for k, v in base.items()}
    return ptrs, kw


def _window(m, **kw):
    ptrs, kw = _split(dict(DECODE_PTRS, out=FAKE, lse=FAKE, workspace=FAKE, workspace_bytes=1 << 30), dict(kw))
    win, sinks = kw.pop("window", 16), kw.pop("sinks", 2)
    p = m.make_params(**{**DECODE, **kw})
    return m.mla_window_decode(p, win, sinks, stream=0, check=False, **ptrs)


@pytest.mark.parametrize("bad,code", [
    (dict(window=0), 1), (dict(window=-5), 1), (dict(sinks=-1), 1), (dict(Sq=0), 1), (dict(q_lat=None), 1),
    (dict(q_rope=None), 1), (dict(lse=None), 1), (dict(kv_scale=FAKE), 1), (dict(workspace=None), 1),
    (dict(softmax_scale=float("nan")), 1), (dict(r=2048), 2), (dict(kernel="tc_pair"), 2), (dict(out=FAKE + 2), 3),
    (dict(workspace=FAKE + 16), 3), (dict(workspace_bytes=16), 4), (dict(B=0, q_lat=None), 0)])
def test_window_decode_refusals(m, bad, code):
    assert _window(m, **bad) == code


@pytest.mark.parametrize("call", [lambda m: _window(m, window=2 ** 32 + 16), lambda m: _window(m, sinks=2 ** 32),
                                  lambda m: _mass(m, max_seq_len=2 ** 32 + 64)])
def test_numbers_beyond_32_bits_are_refused_not_cut(m, call):
    with pytest.raises(ValueError, match="32 bits"):
        call(m)


def _mass(m, **kw):
    ptrs, kw = _split(dict(DECODE_PTRS, lse=FAKE, mass_in=None, mass=FAKE), dict(kw))
    S = kw.pop("max_seq_len", 64)
    p = m.make_params(**{**DECODE, **kw})
    return m.mla_attention_mass(p, S, stream=0, check=False, **ptrs)


@pytest.mark.parametrize("bad,code", [
    (dict(max_seq_len=-1), 1), (dict(H=0), 1), (dict(q_lat=None), 1), (dict(lse=None), 1), (dict(mass=None), 1),
    (dict(kv_cache=None), 1), (dict(q_rope=None), 1), (dict(kv_scale=FAKE), 1),
    (dict(q_dtype=1, cache_dtype=2, out_dtype=1), 1), (dict(kernel="tc_pair"), 2), (dict(kernel="tcgen05"), 2),
    (dict(r=1280, d_r=8), 2), (dict(num_workers=1 << 20), 2), (dict(Sq=1 << 14, H=1 << 11), 2), (dict(mass=FAKE + 2), 3),
    (dict(lse=FAKE + 1), 3), (dict(B=0, mass=None), 0), (dict(max_seq_len=0, mass=None), 0)])
def test_attention_mass_refusals(m, bad, code):
    assert _mass(m, **bad) == code


def _evict(m, **kw):
    ptrs, kw = _split(dict(mass=FAKE, seq_lens=FAKE, indices=FAKE, counts=FAKE), dict(kw))
    f = dict(batch=2, max_seq_len=100, budget=10, sinks=2, recent=3, reserved=0)
    return m.mla_evict_select(m.EvictParams(**{**f, **kw}), stream=0, check=False, **ptrs)


@pytest.mark.parametrize("bad,code", [
    (dict(batch=-1), 1), (dict(budget=0), 1), (dict(sinks=-1), 1), (dict(recent=-1), 1), (dict(sinks=8), 1),
    (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1, budget=2 ** 31 - 1), 1), (dict(max_seq_len=-1), 1),
    (dict(reserved=1), 1), (dict(mass=None), 1), (dict(indices=None), 1), (dict(max_seq_len=(1 << 30) + 1), 2),
    (dict(counts=FAKE + 2), 3), (dict(batch=0, mass=None), 0)])
def test_evict_select_refusals(m, bad, code):
    assert _evict(m, **bad) == code


def _compact(m, **kw):
    ptrs, kw = _split(dict(kv_cache=FAKE, k_rope_cache=None, kv_scale=None, block_table=FAKE, dst_block_table=FAKE * 2,
                           indices=FAKE, counts=FAKE, mass=None, mass_out=None), dict(kw))
    f = dict(batch=2, kv_rank=16, rope_dim=8, block_size=64, num_blocks=8, max_blocks_per_seq=3, dst_max_blocks=1,
             cache_dtype=1, list_stride=64, mass_stride=192, mass_out_stride=64, reserved=0)
    return m.mla_cache_compact(m.CompactParams(**{**f, **kw}), stream=0, check=False, **ptrs)


@pytest.mark.parametrize("bad,code", [
    (dict(batch=-1), 1), (dict(kv_rank=0), 1), (dict(block_size=0), 1), (dict(num_blocks=0), 1),
    (dict(cache_dtype=3), 1), (dict(list_stride=0), 1), (dict(list_stride=65), 1), (dict(mass=FAKE), 1),
    (dict(mass_out=FAKE), 1), (dict(mass=FAKE, mass_out=FAKE, mass_out_stride=63), 1),
    (dict(mass=FAKE, mass_out=FAKE, mass_stride=0), 1), (dict(kv_cache=None), 1), (dict(counts=None), 1),
    (dict(kv_scale=FAKE), 1), (dict(cache_dtype=2), 1), (dict(cache_dtype=2, kv_scale=FAKE), 1), (dict(reserved=7), 1),
    (dict(dst_block_table=FAKE), 1),   # the tables may not be one: the destination blocks have to be free
    (dict(max_blocks_per_seq=1 << 30), 2), (dict(indices=FAKE + 2), 3), (dict(kv_cache=FAKE + 1), 3),
    (dict(batch=0, kv_cache=None), 0)])
def test_cache_compact_refusals(m, bad, code):
    assert _compact(m, **bad) == code


def _verify(m, **kw):
    ptrs, kw = _split(dict(target=FAKE, draft=FAKE, draft_tokens=FAKE, draft_lens=None, accept_u=FAKE, sample_u=FAKE,
                           seq_lens=None, tokens=FAKE, accepted=FAKE, new_seq_lens=None), dict(kw))
    f = dict(batch=2, max_drafts=3, vocab=1000, prob_dtype=0, reserved=0)
    return m.mla_verify_drafts(m.VerifyParams(**{**f, **kw}), stream=0, check=False, **ptrs)


@pytest.mark.parametrize("bad,code", [
    (dict(batch=-1), 1), (dict(max_drafts=-1), 1), (dict(vocab=0), 1), (dict(prob_dtype=2), 1), (dict(reserved=1), 1),
    (dict(target=None), 1), (dict(draft_tokens=None), 1), (dict(accept_u=None), 1), (dict(sample_u=None), 1),
    (dict(tokens=None), 1), (dict(accepted=None), 1), (dict(seq_lens=FAKE), 1), (dict(new_seq_lens=FAKE), 1),
    (dict(vocab=1 << 24), 2), (dict(target=FAKE + 2), 3), (dict(draft=FAKE + 1, prob_dtype=1), 3),
    (dict(tokens=FAKE + 2), 3), (dict(batch=0, target=None), 0)])
def test_verify_drafts_refusals(m, bad, code):
    assert _verify(m, **bad) == code


def test_torch_front_end_refuses_host_tensors(m):
    import torch
    f, i = torch.zeros, lambda *s: torch.zeros(*s, dtype=torch.int32)
    q, qr, kv, bt, sl = f(1, 1, 2, 16), f(1, 1, 2, 8), f(2, 64, 24), i(1, 2), i(1)
    with pytest.raises(ValueError, match="CUDA"):
        m.window_decode(q, qr, kv, bt, sl, 0.1, 8)
    with pytest.raises(ValueError, match="CUDA"):
        m.attention_mass(q, qr, kv, bt, sl, f(1, 1, 2), 0.1, f(1, 128))
    with pytest.raises(ValueError, match="CUDA"):
        m.evict_select(f(1, 128), sl, 8)
    with pytest.raises(ValueError, match="CUDA"):
        m.cache_compact(kv, bt, i(1, 1), i(1, 8), i(1))
    with pytest.raises(ValueError, match="CUDA"):
        m.verify_drafts(f(1, 2, 8), f(1, 1, 8), i(1, 1), f(1, 1), f(1))


# ----------------------------------------------------------------------------- the references
def test_window_reference_equals_the_oracle_when_nothing_is_hidden():
    w = W.WORKLOADS[0].with_(B=3, Sq=2, causal=True, seq_lens=(1, 70, 129), contiguous=False)
    inp = W.make_inputs(w)
    ref_o, ref_l = oracle.decode_inputs(inp)
    for win, sinks in ((129, 0), (1 << 20, 3), (1, 129)):
        out, lse, _, _ = R.window(inp, win, sinks)
        np.testing.assert_allclose(out.numpy(), ref_o, atol=1e-12)
        np.testing.assert_allclose(lse.numpy(), ref_l, atol=1e-12)


def test_window_reference_equals_the_oracles_list_decode():
    w = W.WORKLOADS[0].with_(B=1, seq_lens=(200,))
    inp = W.make_inputs(w)
    out, lse, _, _ = R.window(inp, 20, 5)
    c, k = R.rows_of(inp, 0, 200)
    keep = list(range(5)) + list(range(180, 200))
    x = (R.to64(inp["q_lat"], W.F32)[0, 0] @ c[keep].T + R.to64(inp["q_rope"], W.F32)[0, 0] @ k[keep].T) * w.scale
    p = x.softmax(1)
    np.testing.assert_allclose(out[0, 0].numpy(), (p @ c[keep]).numpy(), atol=1e-13)
    np.testing.assert_allclose(lse[0, 0].numpy(), x.logsumexp(1).numpy(), atol=1e-13)


def test_mass_reference_adds_one_per_row():
    import torch
    w = W.WORKLOADS[0].with_(B=2, Sq=2, causal=True, seq_lens=(130, 1))
    inp = W.make_inputs(w)
    _, lse, _, _ = R.window(inp, 1 << 20, 0)
    mass, _ = R.mass(inp, lse, torch.zeros(2, 130, dtype=torch.float64))
    # the second sequence's first row sees nothing
    np.testing.assert_allclose(mass.sum(1).numpy(), [2 * w.H, w.H], atol=1e-12)


def test_evict_reference_keeps_the_heaviest():
    mass = np.array([[5, 1, 9, 9, 2, 9, 0, 3]], np.float32)
    idx, cnt = R.evict(mass, [8], 5, 1, 1)
    assert cnt[0] == 5 and idx[0].tolist() == [0, 2, 3, 5, 7]
    idx, cnt = R.evict(mass, [8], 4, 1, 1)      # a tie at 9: the lower positions
    assert idx[0].tolist() == [0, 2, 3, 7]
    idx, cnt = R.evict(mass, [3], 4, 1, 1)
    assert cnt[0] == 3 and idx[0].tolist() == [0, 1, 2, -1]


def test_verify_reference_samples_the_target():
    # speculative sampling leaves the target's distribution: first token over many draws, V = 3
    rng = np.random.default_rng(0)
    n, p, q = 40000, np.array([0.5, 0.2, 0.3], np.float32), np.array([0.2, 0.5, 0.3], np.float32)
    tok = rng.choice(3, size=(n, 1), p=q.astype(np.float64) / q.astype(np.float64).sum()).astype(np.int32)
    out, acc = R.verify(np.broadcast_to(p, (n, 2, 3)), np.broadcast_to(q, (n, 1, 3)), tok,
                        rng.random((n, 1), np.float32), rng.random(n, np.float32))
    freq = np.bincount(out[:, 0], minlength=3) / n
    # 5 standard deviations of a frequency: 5 sqrt(1/4 / 40000) = 0.0125
    assert np.abs(freq - p).max() < 5 * math.sqrt(0.25 / n)
