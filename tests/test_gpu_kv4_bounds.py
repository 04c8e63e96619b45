"""The bounds-checked build (librecsa_bounds.so) on the 4-bit KV cache: every slot that is
written or read, the rows that eviction moves, the tiles, parts and output rows of the attention
kernels are range-checked on the device.  Small cases through that build finish with status OK
and give the normal build's results, bit for bit."""
import pytest
import torch

from tests import test_gpu_kv4 as T
from tests.test_gpu_debug_bounds import libs  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def run(R, dtype, d, Hkv, G, lengths, n, cap, mq, huge):
    """Build, append, chunk with weights, decode with weights, evict, chunk again, read."""
    B = len(lengths)
    L = max(lengths)
    k, v = T.keys((B, Hkv, L, d), 1, dtype), T.rand((B, Hkv, L, d), 2, dtype)
    if huge:
        v[0, 0, 1] *= 2.0 ** 40
    cfg = R.Config(head_dim=d, n_q_heads=G * Hkv, n_kv_heads=Hkv, dtype=dtype)
    kv4 = R.RecsaKV4(cfg, cap, B, max_queries=mq)
    kv4.recsa_kv4_build(k.cuda(), v.cuda(), lengths)
    new = T.keys((B, Hkv, n, d), 3, dtype).cuda()
    counts = torch.tensor([n - b % n for b in range(B)], dtype=torch.int32, device="cuda")
    kv4.recsa_kv4_append(new, new, counts)
    Q = T.rand((B, n, G * Hkv, d), 4, dtype).cuda()
    outs = [kv4.prefill(Q, counts, accumulate_rows=n)]
    outs.append(kv4.decode(Q[:, 0].contiguous(), accumulate=True))
    kv4.recsa_kv4_evict(max(n, L // 2), 2, 5)
    outs += [kv4.weights().clone(), kv4.positions().clone()]
    outs.append(kv4.prefill(Q, accumulate_rows=1))
    outs += [*kv4.read(0, cap), kv4.weights().clone(), kv4.lengths().clone()]
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK
    return outs


@pytest.mark.parametrize("dtype,d,Hkv,G,lengths,n,cap,mq,huge", [
    ("bf16", 128, 2, 4, [300, 70, 33], 20, 400, 60, False), ("bf16", 64, 3, 1, [1, 200], 7, 210, 14, False),
    ("f32", 64, 2, 8, [129, 5], 12, 150, 10, False), ("bf16", 128, 1, 8, [900], 300, 1200, 300, False),
    ("bf16", 128, 2, 2, [8000, 100], 40, 8100, 80, False), ("bf16", 64, 2, 4, [150, 60], 16, 200, 32, True),
    ("f32", 128, 2, 1, [64] * 9, 3, 70, 27, False)])
def test_the_same_results_and_no_index_out_of_range(libs, dtype, d, Hkv, G, lengths, n, cap, mq, huge):  # noqa: F811
    R, checked = libs
    for a, b in zip(run(R, dtype, d, Hkv, G, lengths, n, cap, mq, huge),
                    run(checked, dtype, d, Hkv, G, lengths, n, cap, mq, huge)):
        assert torch.equal(torch.nan_to_num(a.float(), nan=7.0), torch.nan_to_num(b.float(), nan=7.0))
