"""Renormalised weights of sigmoids that 32 bits do not hold, beside ones that they do: still ratios of the scores.

Bound: of each exponential, by its argument's rounding, (|x| + 4) 2^-24 relative with |x| <= 110; a sum of k <= 8 positive
terms, a sum with 1 and two divisions by 2^-24 each: 2 (114) + 16 units of 2^-24, and 2^-126 where results are subnormal."""
import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("best", [30.0, 3.0, 0.0, -3.0, -20.0, -29.0, -29.9, -30.1, -45.0])
def test_ratios_of_far_sigmoids(best):
    x = torch.full((4, 32), -400.0)
    for t in range(4):
        x[t, 3:11] = best - torch.tensor([0.0, 0.5, 9.0, 40.0, 58.0, 66.0, 71.0, 80.0]) * (1 + 0.02 * t)
    e, w = binding.route_experts(x.cuda(), 8, "sigmoid")
    assert e.cpu().tolist() == [list(range(3, 11))] * 4
    s = x[:, 3:11].double()
    log = torch.minimum(s, torch.zeros_like(s)) - torch.log1p(torch.exp(-s.abs()))
    want = torch.softmax(log, -1)
    assert ((w.double().cpu() - want).abs() <= 244 * 2.0**-24 * want + 2.0**-126).all()
