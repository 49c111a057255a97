"""The router on both sides of its one-launch form's border (128 ids, times the
rounds in which 16 waves take the tokens), and the sort over so few ids that
most of its waves have none."""
import numpy as np
import pytest

from test_moe_gpu import _check_route

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,top", [(1, 64), (2, 64), (3, 42), (3, 43), (16, 8), (16, 9), (17, 3), (17, 4), (32, 2), (32, 3),
                                   (33, 1), (42, 1), (43, 1), (129, 1), (5, 64), (256, 1), (257, 1), (64, 4)])
@pytest.mark.parametrize("experts", [64, 129, 1000])
def test_route_at_the_one_launch_border(n, top, experts):
    rng = np.random.default_rng([997, n, top, experts])
    logits = rng.integers(-40, 40, (n, experts)).astype(np.float32) / 4      # ties
    logits[rng.random((n, experts)) < 0.1] = -np.inf
    logits[n // 2] = -np.inf                                                 # a token without experts
    _check_route(logits, top, normalize=bool((n + top) % 2), scale=1.5)
