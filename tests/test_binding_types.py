"""What the binding's attention and rotation calls say to arguments that are no tensors. No GPU: tensors without storage."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from quant_int8_quantized_gb300 import mq

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")


@pytest.mark.parametrize("out", [None, [0.0], 7])
def test_attention_output(out):
    with FakeTensorMode():
        q = torch.empty((2, 1, 4, 64), dtype=torch.float16, device="cuda")
        own, n = mq.KV.empty(2, 10, 2, 64), torch.empty(2, dtype=torch.int32, device="cuda")
        with pytest.raises(TypeError, match="out must be a torch.Tensor"):
            mq.mq_attn_prefix(q, None, own, n, out)


@pytest.mark.parametrize("what", ["q", "k", "v"])
def test_rotation_inputs(what):
    with FakeTensorMode():
        args = dict(q=None, k=None, v=None) | {what: [[1.0]]}
        with pytest.raises(TypeError, match=f"{what} must be a torch.Tensor"):
            mq.mq_qk_norm_rope(**args, q_out=None, cache=mq.KV.empty(1, 4, 2, 64))
