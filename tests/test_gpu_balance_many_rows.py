"""GPU tests of the router losses' sums over very many rows: their error may not
grow with the number of rows.

Bars, u = 2^-24.  Rows of equal logits 0: every exponential is 1, their sum E,
both exact, so a probability is the rounded 1/E (u).  A sum of positive terms adds
at most u per addition: 64 in a run of rows, 64 runs to a wavefront at most (a
wavefront has T / 4096 rows), 16 wavefronts in 9, 256 chunks in 32 + 8.  In all
(1 + 64 + 64 + 9 + 40 + 2) u = 180 u for prob_sum; the balance loss, a product and
a sum of E terms in 64 bits, adds its own rounding.
lse = log(E), whose logarithm is good to 4 u; its square, summed in 64 bits, to 8 u
and the last rounding: 10 u.
"""
import numpy as np
import pytest
import torch

from parity import need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("T", [(1 << 20) + 77, (1 << 24) - 1])
@pytest.mark.parametrize("E", [5, 21, 37, 64])
def test_equal_rows(T, E):
    import bit_expert_ffn_top_amd as bf
    dev = need_gpu()
    lg = torch.zeros((T, E), device=dev)
    ix = (torch.arange(T, device=dev, dtype=torch.int32) % E).view(T, 1)
    f = bf.route_balance(lg, ix)
    assert int(f.n_tokens) == T
    assert torch.equal(f.counts[0], torch.bincount(ix.flatten(), minlength=E).int())
    p = f.prob_sum.double().cpu().numpy()[0]
    assert np.abs(p / (T / E) - 1).max() <= 180 * U
    assert abs(float(f.balance) - 1) <= 182 * U             # E / (k T^2) sum_e count_e T/E = 1
    assert abs(float(f.z) / np.log(E) ** 2 - 1) <= 10 * U


def test_half_of_the_rows_masked_and_two_sequences():
    """The rows that take part are what is counted, not the rows passed over."""
    import bit_expert_ffn_top_amd as bf
    dev = need_gpu()
    T, E = (1 << 24) - 1, 21
    cut = 5_000_003
    lg = torch.zeros((T, E), device=dev)
    ix = torch.zeros((T, 1), dtype=torch.int32, device=dev)
    mask = (torch.arange(T, device=dev) % 3 != 0)
    f = bf.route_balance(lg, ix, torch.tensor([0, cut, T], dtype=torch.int32, device=dev), mask)
    n = np.array([int(mask[:cut].sum()), int(mask[cut:].sum())])
    assert np.array_equal(f.n_tokens.cpu().numpy(), n)
    p = f.prob_sum.double().cpu().numpy()
    assert np.abs(p / (n[:, None] / E) - 1).max() <= 180 * U
    assert np.abs(f.z.double().cpu().numpy() / np.log(E) ** 2 - 1).max() <= 10 * U


def test_mean_of_squares_that_add_up_past_fp32():
    """Every lse is 1.5e19: the squares (2.25e38) have a mean that fp32 holds, and a
    sum that it does not."""
    import bit_expert_ffn_top_amd as bf
    dev = need_gpu()
    for T in (8, 300):
        lg = torch.full((T, 4), 1.5e19, device=dev)
        f = bf.route_balance(lg, torch.zeros((T, 1), dtype=torch.int32, device=dev))
        want = float(np.float32(1.5e19)) ** 2      # log(4) is below a step of lse
        assert abs(float(f.z) / want - 1) <= 2 * U
