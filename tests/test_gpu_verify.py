"""GPU checks of the draft verification: every accepted count and token equals the definition's."""
from __future__ import annotations

import numpy as np
import pytest

import bounded_ref as R

pytestmark = pytest.mark.gpu


def problem(B, K, V, seed, near=0.5, sharp=3.0, bf16=False):
    rng = np.random.default_rng(seed)

    def soft(x):
        e = np.exp(x - x.max(-1, keepdims=True))
        return (e / e.sum(-1, keepdims=True)).astype(np.float32)
    lt = sharp * rng.standard_normal((B, K + 1, V)).astype(np.float32)
    ld = lt[:, :K] + near * rng.standard_normal((B, K, V)).astype(np.float32)
    target, draft = soft(lt), soft(ld)
    if bf16:   # rounded to nearest by torch
        import torch
        target, draft = (torch.from_numpy(x).bfloat16().float().numpy() for x in (target, draft))
    tok = np.zeros((B, K), np.int32)
    for b in range(B):
        for i in range(K):
            c = np.cumsum(draft[b, i].astype(np.float64))
            tok[b, i] = np.searchsorted(c, rng.random() * c[-1], side="right")
    return target, draft, tok, rng.random((B, K), np.float32), rng.random(B, np.float32)


def run(target, draft, tok, u, v, bf16=False, lens=None, seq_lens=None):
    import torch
    import head_latent_attention_split_b200 as mla
    dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    pt, pd = dev(target), dev(draft)
    if bf16:
        pt, pd = pt.bfloat16(), None if pd is None else pd.bfloat16()
    got = mla.verify_drafts(pt, pd, dev(tok), dev(u), dev(v), draft_lens=dev(lens), seq_lens=dev(seq_lens))
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in got], mla.device_status()


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,K,V", [(1, 1, 1), (3, 2, 5), (7, 1, 513), (5, 4, 4096), (4, 3, 4097), (6, 2, 32000),
                                   (3, 5, 50257), (9, 3, 128000), (2, 40, 1000)])
def test_matches_the_definition(B, K, V, bf16):
    for seed, near in ((1, 0.1), (2, 1.0), (3, 3.0)):
        p = problem(B, K, V, seed * 100 + V, near, bf16=bf16)
        (tok, acc), st = run(*p, bf16=bf16)
        ref_t, ref_a = R.verify(*p)
        assert st == 0
        np.testing.assert_array_equal(acc, ref_a)
        np.testing.assert_array_equal(tok, ref_t)


def test_drafts_without_probabilities_lengths_and_cache_lengths():
    target, draft, tok, u, v = problem(12, 4, 3000, 5, sharp=6.0)
    tok[:, 0] = target[:, 0].argmax(-1)
    lens = np.array([0, 1, 2, 3, 4, 4, 3, 2, 1, 0, 4, 4], np.int32)
    seq = np.arange(100, 112).astype(np.int32)
    for d in (draft, None):
        (t, a, n), st = run(target, d, tok, u, v, lens=lens, seq_lens=seq)
        ref_t, ref_a = R.verify(target, d, tok, u, v, lens)
        assert st == 0 and np.array_equal(t, ref_t) and np.array_equal(a, ref_a)
        np.testing.assert_array_equal(n, seq - lens + ref_a)


def test_no_drafts_is_plain_sampling():
    target, _, _, _, v = problem(20, 0, 700, 6)
    (t, a), st = run(target, None, np.zeros((20, 0), np.int32), np.zeros((20, 0), np.float32), v)
    ref_t, _ = R.verify(target, None, np.zeros((20, 0), np.int32), np.zeros((20, 0), np.float32), v)
    assert st == 0 and (a == 0).all() and np.array_equal(t, ref_t)


def test_edges_of_the_random_numbers_and_the_residual():
    V = 1000
    target, draft, tok, u, v = problem(8, 2, V, 7)
    u[0], v[0] = 0.0, 0.0
    u[1], v[1] = 1 - 2.0 ** -24, 1 - 2.0 ** -24
    u[2, 0], v[2] = np.nan, 1.0             # refused; the last token with a weight
    u[3, 0], v[3] = np.nan, -1.0            # refused; the first
    v[4] = np.nan
    draft[5] = target[5, :2]                # equal distributions: any u below 1 accepts
    u[6, 0] = 2.0
    draft[6, 0] = target[6, 0]              # refused although equal: the residual is 0, the target's row is drawn from
    target[7, 0, tok[7, 0]] = 0.0           # refused at once, the draft's token has no weight left
    u[7, 0] = 0.0
    p = (target, draft, tok, u, v)
    (t, a), st = run(*p)
    ref_t, ref_a = R.verify(*p)
    assert st == 0 and a[5] == 2 and a[6] == 0 and a[7] == 0
    np.testing.assert_array_equal(a, ref_a)
    np.testing.assert_array_equal(t, ref_t)


def test_rows_that_are_not_needed_may_hold_anything():
    target, draft, tok, u, v = problem(6, 3, 2000, 8)
    u[:, 1] = np.nan                    # the second draft is refused wherever the first is not (2 q < p can hold)
    target[:, 2:], draft[:, 2:], tok[:, 2] = np.nan, np.nan, -5
    (t, a), st = run(target, draft, tok, u, v)
    ref_t, ref_a = R.verify(target, draft, tok, u, v)
    assert st == 0 and np.array_equal(t, ref_t) and np.array_equal(a, ref_a)


def test_unusable_input_is_flagged_for_its_sequence_only():
    V = 300
    for i in range(6):
        target, draft, tok, u, v = problem(4, 2, V, 9)
        u[1] = 0.0 if i != 2 else np.nan
        lens = np.full(4, 2, np.int32)
        seq = np.array([50, 60, 70, 80], np.int32)
        if i == 0:
            tok[1, 0] = V
        elif i == 1:
            tok[1, 1] = -1
        elif i == 2:
            target[1, 0], draft[1, 0] = np.inf, 0.1
        elif i == 3:
            target[1, 2] = 0.0
        elif i == 4:
            lens[1] = 3
        else:
            lens[1] = -1
        (t, a, n), st = run(target, draft, tok, u, v, lens=lens, seq_lens=seq)
        ref_t, ref_a = R.verify(target, draft, tok, u, v, lens)
        assert st == 9, i
        assert ref_a[1] == -1
        np.testing.assert_array_equal(a, ref_a)
        np.testing.assert_array_equal(t, ref_t)
        assert n[1] == (60 if i >= 4 else 58)


def test_graph_replay_in_place_lengths_and_other_stream():
    import torch
    import head_latent_attention_split_b200 as mla
    p = problem(5, 2, 4000, 10)
    d = [torch.from_numpy(x).cuda() for x in p]
    seq = torch.arange(50, 55, dtype=torch.int32, device="cuda")
    toks, acc = torch.empty(5, 3, dtype=torch.int32, device="cuda"), torch.empty(5, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t, a = mla.verify_drafts(*d, stream=side)
    side.synchronize()
    ref = R.verify(*p)
    assert np.array_equal(t.cpu().numpy(), ref[0]) and np.array_equal(a.cpu().numpy(), ref[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.verify_drafts(*d, seq_lens=seq, new_seq_lens=seq, tokens=toks, accepted=acc)
    q = problem(5, 2, 4000, 11)
    for x, y in zip(d, q):
        x.copy_(torch.from_numpy(y))
    g.replay()
    torch.cuda.synchronize()
    ref = R.verify(*q)
    assert np.array_equal(toks.cpu().numpy(), ref[0]) and np.array_equal(acc.cpu().numpy(), ref[1])
    np.testing.assert_array_equal(seq.cpu().numpy(), np.arange(50, 55) - 2 + ref[1])
    assert mla.device_status() == 0


def test_front_end_refuses_tensors_that_do_not_fit():
    import torch
    import head_latent_attention_split_b200 as mla
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    good = dict(target_probs=f(2, 3, 16), draft_probs=f(2, 2, 16), draft_tokens=i(2, 2), accept_u=f(2, 2), sample_u=f(2))
    for bad in (dict(target_probs=f(2, 3, 16).half()), dict(draft_probs=f(2, 3, 16)), dict(draft_probs=f(2, 2, 16).bfloat16()),
                dict(draft_tokens=i(2, 2).long()), dict(accept_u=f(2, 3)), dict(sample_u=f(3)), dict(draft_lens=f(2)),
                dict(new_seq_lens=i(2)), dict(target_probs=f(2, 16, 3).transpose(1, 2)), dict(sample_u=torch.zeros(2))):
        with pytest.raises((TypeError, ValueError)):
            mla.verify_drafts(**{**good, **bad})
    torch.cuda.synchronize()
    assert mla.device_status() == 0
