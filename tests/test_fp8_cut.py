"""CPU: what the cut of the E4M3 matrix instructions comes to, by its definition."""
import pytest
import torch

import fp8_cut
import fp8_ref as R


def test_cut_by_hand():
    def one(values, others):
        s, _ = fp8_cut.cut_groups(torch.tensor([values], dtype=torch.float64), torch.tensor([others], dtype=torch.float64))
        return s.flatten().tolist()
    big = [256.0] + [0.0] * 7
    for other, kept in ((8.0, 8.0), (4.0, 0.0), (-4.0, 0.0), (12.0, 8.0), (-12.0, -8.0)):  # 2^16: what is below 2^3 goes
        assert one([256.0, other, 0, 0, 0, 0, 0, 0], [256.0, 1.0, 0, 0, 0, 0, 0, 0]) == [65536.0 + kept]
    assert one(big + [2.0 ** -6] + [0.0] * 7, big + [0.5] + [0.0] * 7) == [65536.0, 2.0 ** -7]  # groups do not meet
    assert one([1.75] * 8, [1.75] * 8) == [8 * 1.75 * 1.75]  # like exponents lose nothing


@pytest.mark.parametrize("least", [0.0, 1.0])
def test_cut_of_random_values(least):
    """Some 1.5e-5 of a result, whatever the length of the sum, without a bias.  A product has eight significant bits, so one
    loses nothing until it is 2^-7 of the largest's binade: without the smallest values (below 1 of 112) less is cut."""
    g = torch.Generator().manual_seed(1)
    for K in (128, 1024, 4096):
        A, B = ((torch.randn((64, K), generator=g) * 112).clamp(-448, 448) for _ in range(2))
        A, B = (torch.where(t.abs() < least, 0, t).to(torch.float8_e4m3fn) for t in (A, B))
        cut, _, exact = fp8_cut.product(A, torch.ones((R.blocks(K), 64)), B, torch.ones((1, R.blocks(K))))
        assert (0.0 if least else 1.3e-5) < (cut - exact).norm() / exact.norm() < 1.7e-5
        assert (cut - exact).mean().abs() < 1e-6 * exact.std()
