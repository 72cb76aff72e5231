"""The calls on 4-bit caches at the ends of what they take: lengths next to the most rows a table may have."""
import math

import pytest
import torch

from quant_int8_quantized_gb300 import mq
from tests import _kv4_ref as R
from tests._gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("rows,back", [(1024, 0), (1024, 700), (16, 5)])
def test_attention_at_the_most_rows(rows, back):
    """Places of pages are looked up ahead of the tile, past what 32 signed bits count. All entries name one page, so the result
    is that page's (the last `back` rows' share of it is below 2^-21), the sum of weights as many times as large."""
    H, D, width = 1, 64, (2 ** 31 - 256) // rows
    one = R.random_cache(1, 1, rows, H, D, 5, spare=0)
    cache = mq.KV4(one.pages, torch.zeros((1, width), dtype=torch.int32, device="cuda"), rows, H, D)
    n = width * rows - back
    q = torch.randn((1, 1, 2, D), generator=torch.Generator("cuda").manual_seed(6), device="cuda").half()
    out, lse = torch.full((1, 1, 2, D), float("nan"), device="cuda"), torch.zeros((1, 1, 2), device="cuda")
    mq.mq_attn_kv4(q, cache, torch.tensor([n], dtype=torch.int32, device="cuda"), out, lse=lse)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == mq.MQ_OK
    k, v = (x[0, :, 0] for x in R.unpack(one.pages, rows, H, D))
    # A warp adds up some 2^31 / (32 * 16 * SMs) steps of 32 keys in 32 bits, one rounding (of a step of the sum at most) for each
    # half of a step, and four for each of its lanes' weights
    steps = n / (32 * 16 * torch.cuda.get_device_properties(0).multi_processor_count)
    off = steps * (2 * 2.0 ** -23 + 4 * 2.0 ** -24) + 2.0 ** -10
    for h in range(2):
        s = k @ q[0, 0, h].double() * D ** -0.5
        p = torch.softmax(s, 0)
        assert bool(((out[0, 0, h].double() - p @ v).abs() <= off * (p @ v.abs())).all())
        assert abs(float(lse[0, 0, h]) - float(torch.logsumexp(s, 0)) - math.log(n / rows)) <= off
