"""Calls on another stream than the current one, with memory that the binding allocates for them: what the current
stream allocates and fills right afterwards must not meet it."""
import pytest
import torch

from quant_int8_quantized_gb300 import mq
from tests._gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _rand(shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").half()


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("T,scores", [(1, False), (1, True), (600, False)])
def test_attention_with_a_workspace_of_its_own(T, scores, raw):
    B, Hq, Hkv, D, P, cap = 3, 8, 2, 128, 700, 900
    q, own = _rand((B, T, Hq, D), 1), mq.KV(_rand((B, cap, Hkv, D), 2), _rand((B, cap, Hkv, D), 3))
    pre = mq.KV(_rand((1, P, Hkv, D), 4), _rand((1, P, Hkv, D), 5))
    n = torch.tensor([900, 650, 777], dtype=torch.int32, device="cuda")
    score = torch.zeros((B, Hkv, cap), device="cuda") if scores else None
    so = [torch.zeros_like(score) for _ in range(2)] if scores else [None, None]
    want = torch.empty((B, T, Hq, D), device="cuda")
    mq.mq_attn_prefix(q, pre, own, n, want, score=score, score_out=so[0], ws=mq.attn_workspace(B, T, Hq, Hkv, D, P, cap, scores))
    size = mq.mq_attn_ws_bytes(B, T, Hq, Hkv, D, P, cap, scores)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(10):
        out = torch.zeros_like(want)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(2000000)              # about a ms: the kernels run after what follows here
        mq.mq_attn_prefix(q, pre, own, n, out, score=score, score_out=so[1], stream=side.cuda_stream if raw else side)
        other = [torch.full((size,), i, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(out, want) and (not scores or torch.equal(so[0], so[1]))
        assert all(bool((x == i).all()) for x in other)
    assert mq.mq_device_status() == mq.MQ_OK
