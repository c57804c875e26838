"""GPU check of the draw at the ends of sample_u's range, against tokens written out by hand."""
import pytest

pytestmark = pytest.mark.gpu

# sample_u outside [0, 1 - 2^-24] acts as the nearer end: the draw is the lowest t whose running sum exceeds
# u times the total, so weights at the end that add up to less than 2^-24 of it are not drawn by any u.
ROWS = [
    # (weights, u, token)
    ([1.0, 1e-9], 1.0, 0), ([1.0, 1e-9], 1 - 2.0 ** -24, 0), ([1.0, 1e-9], 7.5, 0), ([1.0, 1e-9], float("inf"), 0),
    ([1.0, 2.0 ** -20], 1.0, 1), ([1.0, 2.0 ** -20], 1 - 2.0 ** -24, 1), ([0.0, 0.25, 0.75, 0.0], 1.0, 2),
    ([0.0, 0.25, 0.75, 0.0], 0.0, 1), ([0.0, 0.25, 0.75, 0.0], -3.0, 1), ([0.0, 0.25, 0.75, 0.0], float("nan"), 1),
    ([0.0, 0.25, 0.75, 0.0], float("-inf"), 1), ([0.0, 0.25, 0.75, 0.0], 0.25, 2), ([0.0, 0.25, 0.75, 0.0], 0.25 - 2.0 ** -26, 1),
]


@pytest.mark.parametrize("V", [4, 5000])
@pytest.mark.parametrize("w,u,token", ROWS)
def test_the_draw_at_the_ends_of_its_range(w, u, token, V):
    import torch
    import head_latent_attention_split_b200 as mla
    p = torch.zeros(1, 1, V, device="cuda")
    p[0, 0, V - len(w):] = torch.tensor(w)
    none = torch.zeros(1, 0, device="cuda")
    t, a = mla.verify_drafts(p, None, none.int(), none, torch.tensor([u], device="cuda"))
    torch.cuda.synchronize()
    assert mla.device_status() == 0 and a.tolist() == [0] and t.tolist() == [[V - len(w) + token]]
