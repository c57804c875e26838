"""CPU-only: calls of the bounded-cache operators whose buffers overlap, or whose numbers leave the range that the
kernels index in, are refused before anything is launched."""
import pytest

from test_bounded_host import FAKE, _compact, _evict, _mass, m  # noqa: F401

F = 4   # bytes of a weight


# mass [2, 192] and mass_out [2, 64]: one buffer for both, a first or last element in common
@pytest.mark.parametrize("out", [FAKE, FAKE + 191 * F, FAKE + (2 * 192 - 1) * F, FAKE - (2 * 64 - 1) * F])
def test_compact_refuses_weights_that_it_would_read_and_write(m, out):  # noqa: F811
    assert _compact(m, mass=FAKE, mass_out=out) == 1


# ... side by side (the call is refused for its list's alignment, checked later, and not before)
@pytest.mark.parametrize("out", [FAKE + 2 * 192 * F, FAKE - 2 * 64 * F])
def test_compact_takes_weights_side_by_side(m, out):  # noqa: F811
    assert _compact(m, mass=FAKE, mass_out=out, indices=FAKE + 2) == 3


# A row of more than 2^30 entries: the kernels' 32-bit loop counters would pass 2^31 and come back negative.
BIG = (1 << 30) + 1


@pytest.mark.parametrize("budget", [BIG, 2 ** 31 - 1])
def test_select_refuses_a_budget_that_its_counters_cannot_pass(m, budget):  # noqa: F811
    assert _evict(m, budget=budget) == 2


@pytest.mark.parametrize("bad", [dict(list_stride=BIG, dst_max_blocks=1 << 25, mass=None, mass_out=None), dict(mass_out_stride=BIG),
                                 dict(mass_out_stride=2 ** 31 - 1), dict(mass_stride=BIG)])
def test_compact_refuses_rows_that_its_counters_cannot_pass(m, bad):  # noqa: F811
    out = FAKE + (1 << 40)
    assert _compact(m, **{**dict(mass=FAKE, mass_out=out), **bad}) == 2


# mass_in may be mass itself; half on top of it, one row's sums would be another's start
@pytest.mark.parametrize("mass_in,code", [(FAKE + F, 1), (FAKE - F, 1), (FAKE + (2 * 64 - 1) * F, 1),
                                          (FAKE + 2 * 64 * F, 3), (FAKE, 3), (None, 3)])
def test_attention_mass_refuses_a_start_that_overlaps_its_result(m, mass_in, code):  # noqa: F811
    assert _mass(m, mass_in=mass_in, lse=FAKE + 2) == code   # (3: taken so far, refused for lse's alignment)


def test_workspace_size_answers_for_the_calls_that_the_decode_takes(m):  # noqa: F811
    # the decode has no split-role kernel for an e4m3 cache, so there is no size for it either
    shape = dict(B=2, Sq=1, H=128, r=512, d_r=64, block_size=64, num_blocks=2, max_blocks_per_seq=1, q_dtype=1, out_dtype=1,
                 causal=False, softmax_scale=0.2, num_workers=74)
    p = m.make_params(**shape, cache_dtype=2, kernel="tc_pair")
    with pytest.raises(m.MlaError) as e:
        m.workspace_size(p)
    assert e.value.status == 2
    # the window decode, which has one, is sized as by the decode's kernel and takes exactly that
    from head_latent_attention_split_b200 import api
    need = api._window_workspace(p)
    assert need == m.workspace_size(m.make_params(**shape, cache_dtype=2, kernel="tcgen05")) and p.kernel == m.KERNELS["tc_pair"]
    ptrs = dict(q_lat=FAKE, q_rope=FAKE, kv_cache=FAKE, k_rope_cache=FAKE, kv_scale=FAKE, block_table=FAKE, seq_lens=FAKE,
                out=FAKE + 8, lse=FAKE, workspace=FAKE)
    call = lambda n: m.mla_window_decode(p, 16, 2, stream=0, check=False, workspace_bytes=n, **ptrs)  # noqa: E731
    assert call(need - 1) == 4 and call(need) == 3   # too small; enough, and then refused for out's alignment
