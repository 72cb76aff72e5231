"""Keys and values that are not finite, written to 4-bit caches: every byte (tests/test_gpu_kv4.py's plain form)."""
import pytest
import torch

from tests._gpu_util import require_gpu
from tests.test_gpu_kv4 import _fill_case, _rand

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("n_pairs,norm,inter", [(0, False, False), (32, False, False), (20, False, True), (64, False, True), (0, True, False)])
def test_infinities(n_pairs, norm, inter):
    """An infinity is written as 7 d of the largest scale, with its sign; what lies past that as well. (A head that is normed or
    turned with one has numbers of no value: only values there.)"""
    M, H, D = 40, 2, 128
    x = _rand((M, 2 * H, D), 17, 40.0)
    at = slice(None) if not norm and n_pairs == 0 else slice(H, None)
    y = x[:, at]
    y[3, 0, 5], y[3, 0, 6], y[4, 1, 127], y[5, 0, 0] = INF, -INF, INF, -INF
    y[6, 0, ::2], y[6, 0, 1::2] = INF, -INF
    y[7, 0, 33], y[7, 1, 64], y[8, 0, 1] = 3.4e38, -3.4e38, 3361.0
    y[9, 1] = INF
    _fill_case(M, 3, H, D, 16, 2, n_pairs, norm=norm, inter=inter, x=x)
