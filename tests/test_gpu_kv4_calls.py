"""Calls of the 4-bit KV cache that the header and the binding allow, on streams and buffers
other than the plain ones."""
import pytest
import torch

from tests import test_gpu_kv4 as T

pytestmark = pytest.mark.gpu
R = T.R                                                  # the fixture


@pytest.mark.parametrize("counts", [[5, 20], None])
def test_outputs_belong_to_the_stream_of_the_call(R, counts):
    """The current stream is busy for some milliseconds: what it did to a call's output
    afterwards (zeroing it) would be seen."""
    kv4, _ = T.make(R, "bf16", 64, 2, 2, [100, 60], max_queries=40)
    Q = T.rand((2, 20, 4, 64), 3, "bf16").cuda()
    c = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    want, d_want, r_want = kv4.prefill(Q, c), kv4.decode(Q[:, 0].contiguous()), kv4.read(3, 50)
    q = Q[:, 0].contiguous()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)                        # about 10 ms
    out, d_out, r_out = kv4.prefill(Q, c, stream=s), kv4.decode(q, stream=s), kv4.read(3, 50, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(d_out, d_want)
    assert all(torch.equal(x, y) for x, y in zip(r_out, r_want))
    if counts:
        assert (out[0, 5:] == 0).all() and (out[0, :5] != 0).any() and (out[1] != 0).any()
