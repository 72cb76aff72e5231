"""Shapes that users run and the other tests leave out: prompts of heads 96 and 256 wide, few queries of many
sequences (or many query heads to a key head) on a long prefix, eviction in place over many rounds. The library as it is;
sampled sequences and queries against plain 64-bit forms."""
import pytest
import torch

from quant_int8_quantized_gb300 import mq
from tests import _attn_ref as R
from tests._gpu_util import require_gpu
from tests.test_gpu_heads import _evict_case

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _rand(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _run(B, T, Hq, Hkv, D, P, cap, lens, dtype, out_dtype, sequences, only, scores=False):
    q, k, v = _rand((B, T, Hq, D), dtype, 1, 1.5), _rand((B, cap, Hkv, D), dtype, 2), _rand((B, cap, Hkv, D), dtype, 3)
    pk, pv = (_rand((1, P, Hkv, D), dtype, 4 + i) for i in range(2)) if P else (None, None)
    for b, n in enumerate(lens):
        k[b, n:], v[b, n:] = float("nan"), float("nan")
    out, lse = torch.empty((B, T, Hq, D), dtype=out_dtype, device="cuda"), torch.empty((B, T, Hq), device="cuda")
    mq.mq_attn_prefix(q, mq.KV(pk, pv) if P else None, mq.KV(k, v), torch.tensor(lens, dtype=torch.int32, device="cuda"), out, lse=lse)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == mq.MQ_OK
    for b in sequences:
        want, bound = R.attention(q[b:b + 1], pk[0] if P else None, pv[0] if P else None, k[b:b + 1], v[b:b + 1], lens[b:b + 1],
                                  D ** -0.5, out_dtype, only=only)
        assert bool(((out[b:b + 1, only].double() - want[0][:, only]).abs() <= bound[0][:, only]).all()), f"out of {b}"
        same = lse[b:b + 1, only].double() == want[1][:, only]            # (-infinity where nothing is seen)
        assert bool((same | ((lse[b:b + 1, only].double() - want[1][:, only]).abs() <= bound[1][:, only])).all()), f"lse of {b}"


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("dtype,out_dtype", [(F16, F16), (BF16, F32)])
def test_prompts_of_every_width(D, dtype, out_dtype):
    T, lens = 1200, [1500, 1203, 900]
    _run(3, T, 8, 2, D, 333, 1500, lens, dtype, out_dtype, [0, 1, 2], [0, 15, 16, 127, 299, 300, 301, 600, T - 1])


@pytest.mark.parametrize("B,T,Hq,Hkv,P,cap", [(64, 5, 28, 4, 4001, 700), (64, 4, 40, 8, 3000, 1000), (64, 1, 40, 1, 9000, 2048),
                                              (40, 8, 32, 2, 700, 900), (64, 3, 64, 8, 5000, 1500), (130, 1, 32, 1, 2500, 1111)])
@pytest.mark.parametrize("D", [64, 128])
def test_few_queries_of_many_sequences_on_a_long_prefix(B, T, Hq, Hkv, P, cap, D):
    """17 to 128 query rows a sequence and key head; lengths from none to all, below T among them."""
    lens = [[0, 1, T - 1, T, cap, cap - 1][b % 6] if b < 12 else (b * 97) % (cap + 1) for b in range(B)]
    _run(B, T, Hq, Hkv, D, P, cap, lens, F16, F32, [0, 1, 2, 3, 4, 5, B // 2, B - 1], list(range(T)))


@pytest.mark.parametrize("score_in_place", [False, True])
@pytest.mark.parametrize("head_major", [False, True])
def test_eviction_in_place_over_many_rounds(head_major, score_in_place):
    _evict_case(3, 4, 128, 9000, [9000, 7777, 4100], 4100, 333, in_place=True, head_major=head_major, score_in_place=score_in_place, dtype=BF16)
    _evict_case(2, 8, 256, 3001, [3001, 2999], 1500, 100, in_place=True, head_major=head_major, score_in_place=score_in_place, kind="ties")
