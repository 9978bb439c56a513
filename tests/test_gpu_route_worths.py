"""Groups of experts whose worths 32 bits do not tell apart, as their two best keys are far larger than the sum of both."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_route_ties import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [1e2, 1e4, 1e5, 1e6])
@pytest.mark.parametrize("groups,E", [(2, 16), (8, 64), (8, 256)])
def test_keys_that_cancel(groups, E, size, scoring):
    """One expert of every group forced by its bias, the others masked by one: a worth is near 1, its terms near `size`."""
    g = torch.Generator().manual_seed(int(size))
    x = torch.randn(20000, E, generator=g)
    bias = torch.full((E,), -size)
    bias[::E // groups] = size
    check(x, 2, scoring, bias, groups=groups, top_groups=max(1, groups // 2))


def test_worths_without_bound():
    """Biases whose sum 32 bits do not hold: as in 64 bits, in which they swallow the scores alike wherever they are computed."""
    big = torch.finfo(torch.float32).max
    x = torch.randn(300, 32, generator=torch.Generator().manual_seed(1))
    for values in ((big, big, 0.0, 0.0), (big, -big, 1.0, -1.0), (-big, -big, 0.0, -big)):
        bias = torch.tensor(values).repeat(8)
        bias[8:16] *= 0.5
        for best in (1, 2):
            for top in (1, 2, 3):
                check(x, 3, "sigmoid", bias, every_row=True, groups=4, top_groups=top, group_best=best)
