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


@pytest.mark.parametrize("dtype,d,G,n", [("bf16", 128, 4, 40), ("bf16", 64, 2, 3), ("f32", 64, 4, 9), ("f32", 128, 1, 1)])
def test_rows_in_place(R, dtype, d, G, n):
    """out = q is right without weights, over cut and whole units; with weights a second launch
    would read the overwritten queries, and the call is refused, as any partial overlap is."""
    B, Hkv = 2, 2
    kv4, _ = T.make(R, dtype, d, Hkv, G, [900, 64], max_queries=B * max(n // 2, 1))
    Q = T.rand((B, n, G * Hkv, d), 5, dtype).cuda()
    want = kv4.prefill(Q)
    X = Q.clone()
    kv4.recsa_kv4_prefill_chunk(X, X)
    assert torch.equal(X, want)
    q = Q[:, 0].contiguous()
    want, x = kv4.decode(q), q.clone()
    kv4.recsa_kv4_decode(x, x)
    assert torch.equal(x, want)
    flat = torch.zeros(q.numel() + 64, dtype=q.dtype, device="cuda")
    a, b = (flat[i:i + q.numel()].view_as(q) for i in (0, 64))
    for args, kw in [((q, q), dict(accumulate=True)), ((a, b), {}), ((b, a), {})]:
        with pytest.raises(R.RecsaError) as e:
            kv4.recsa_kv4_decode(*args, **kw)
        assert e.value.status == R.RECSA_E_INVAL
    flat = torch.zeros(Q.numel() + 64, dtype=q.dtype, device="cuda")
    a, b = (flat[i:i + Q.numel()].view_as(Q) for i in (0, 64))
    for args, kw in [((Q, Q), dict(accumulate_rows=1)), ((a, b), {}), ((b, a), {})]:
        with pytest.raises(R.RecsaError) as e:
            kv4.recsa_kv4_prefill_chunk(*args, **kw)
        assert e.value.status == R.RECSA_E_INVAL
    assert (kv4.weights() == 0).all()


@pytest.mark.parametrize("lengths", [[7], [1]])
def test_strides_of_dims_of_one_element_do_not_matter(R, lengths):
    """k alone and v a part of a larger tensor, one sequence and one KV head: the same rows."""
    d, L = 64, lengths[0]
    cfg = R.Config(head_dim=d, n_q_heads=2, n_kv_heads=1, dtype="bf16")
    k = T.keys((1, 1, L, d), 1, "bf16").cuda()
    big = T.rand((3, 2, L, d), 2, "bf16").cuda()
    v = big[1:2, 1:2]
    assert k.stride() != v.stride()
    kv4, same = R.RecsaKV4(cfg, 16, 1), R.RecsaKV4(cfg, 16, 1)
    kv4.recsa_kv4_build(k, v, lengths)
    same.recsa_kv4_build(k, v.clone(memory_format=torch.contiguous_format), lengths)
    assert all(torch.equal(a, b) for a, b in zip(kv4.read(0, L), same.read(0, L)))
    with pytest.raises(ValueError):
        kv4.recsa_kv4_build(k.expand(1, 1, L, d), T.rand((1, 1, L, 2 * d), 3, "bf16").cuda()[..., :d], [2])


def test_append_up_to_the_last_position(R):
    """2^31 - 1 tokens a sequence in all: the last positions are used, one more is refused and
    leaves the sequence as it was, and a build starts anew."""
    kv4, _ = T.make(R, "f32", 64, 1, 1, [4, 4], cap=12)
    seen = kv4._table(kv4.workspace, kv4.info.tokens_seen, (2,), torch.int64)
    seen[0] = 2 ** 31 - 1 - 3                            # as after as many appends and evictions
    k = T.rand((2, 1, 3, 64), 1, "f32").cuda()
    kv4.recsa_kv4_append(k, k)
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK
    assert kv4.positions()[0, 0, 4:7].tolist() == [2 ** 31 - 4, 2 ** 31 - 3, 2 ** 31 - 2]
    q = T.rand((2, 1, 1, 64), 2, "f32").cuda()
    both = kv4.prefill(q)
    assert torch.equal(both[0, 0], kv4.decode(q[:, 0].contiguous())[0])
    kv4.recsa_kv4_append(k[:, :, :1].contiguous(), k[:, :, :1].contiguous())
    assert kv4.recsa_kv4_get_status() == R.RECSA_E_CAPACITY
    assert kv4.lengths().tolist() == [7, 8] and seen.tolist() == [2 ** 31 - 1, 8]
    kv4.recsa_kv4_build(k, k, [3, 3])
    kv4.recsa_kv4_append(k, k)
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK and seen.tolist() == [6, 6]


@pytest.mark.parametrize("dtype,d,G,n", [("bf16", 128, 4, 40), ("bf16", 64, 2, 3), ("f32", 64, 4, 9)])
def test_a_chunk_without_rows(R, dtype, d, G, n):
    """Counts of zero for every sequence: nothing is read, written or recorded."""
    kv4, _ = T.make(R, dtype, d, 2, G, [90, 0], max_queries=2 * n)
    Q = T.rand((2, n, 2 * G, d), 1, dtype).cuda()
    out = torch.full_like(Q, 3.0)
    kv4.recsa_kv4_prefill_chunk(Q, out, torch.zeros(2, dtype=torch.int32, device="cuda"), accumulate_rows=n)
    assert (out == 3.0).all() and (kv4.weights() == 0).all()
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype,d,G,n", [("bf16", 128, 4, 40), ("bf16", 64, 2, 3), ("f32", 64, 4, 9), ("f32", 128, 1, 5)])
def test_a_query_that_is_no_number_reaches_its_own_row_only(R, dtype, d, G, n, bad):
    kv4, _ = T.make(R, dtype, d, 2, G, [300, 77], max_queries=2 * n)
    Q = T.rand((2, n, 2 * G, d), 1, dtype).cuda()
    want, q = kv4.prefill(Q), Q[:, 0].contiguous()
    d_want = kv4.decode(q)
    X = Q.clone()
    X[1, n // 2, 1, 3] = bad
    out = kv4.prefill(X)
    assert torch.isnan(out[1, n // 2, 1]).all()
    out[1, n // 2, 1] = want[1, n // 2, 1]
    assert torch.equal(out, want)
    x = q.clone()
    x[0, 0, 5] = bad
    out = kv4.decode(x)
    assert torch.isnan(out[0, 0]).all()
    out[0, 0] = d_want[0, 0]
    assert torch.equal(out, d_want)


def test_many_heads_of_a_short_cache(R):
    """20000 units of 5 tokens: every call, against the oracle at a few of them."""
    B, Hkv, G, d, n = 4, 5000, 2, 64, 5
    k, v = T.keys((B, Hkv, 5, d), 1, "bf16"), T.rand((B, Hkv, 5, d), 2, "bf16")
    cfg = R.Config(head_dim=d, n_q_heads=G * Hkv, n_kv_heads=Hkv, dtype="bf16")
    kv4 = R.RecsaKV4(cfg, 8, B, max_queries=B * n)
    kv4.recsa_kv4_build(k.cuda(), v.cuda(), [5, 5, 4, 5])
    kv4.recsa_kv4_append(k[:, :, :1].contiguous().cuda(), v[:, :, :1].contiguous().cuda())
    Q = T.rand((B, n, G * Hkv, d), 3, "bf16")
    out = kv4.prefill(Q.cuda(), accumulate_rows=n)
    dec = kv4.decode(Q[:, 0].contiguous().cuda(), accumulate=True)
    w = kv4.weights()[:, :, :6].double().sum(-1)
    assert (w - (n + 1) * G).abs().max() <= 2.0 ** -17 * (n + 1) * G
    kept = kv4.weights().clone()
    kv4.recsa_kv4_evict(4, 1, 1)
    for b, h in [(0, 0), (1, 4999), (2, 2500), (3, 17), (3, 4999)]:
        u = T.O.Unit(d)
        L = 4 if b == 2 else 5
        u.append(T.np64(k[b, h, :L]), T.np64(v[b, h, :L]))
        u.append(T.np64(k[b, h, :1]), T.np64(v[b, h, :1]))
        for i in range(n):
            qs = T.np64(Q[b, i, h * G:(h + 1) * G])
            floor = T.bound_of(u, qs, "bf16", True)[1]
            T.check_rows(out[b, i, h * G:(h + 1) * G], u.attend(qs, u.seen - n + i), floor, "bf16", (b, h, i))
        qs = T.np64(Q[b, 0, h * G:(h + 1) * G])
        T.check_rows(dec[b, h * G:(h + 1) * G], u.attend(qs, u.seen), T.bound_of(u, qs, "bf16")[1], "bf16", (b, h))
        u.w = T.np64(kept[b, h, :L + 1])
        u.evict(4, 1, 1)
        assert kv4.positions()[b, h, :4].tolist() == u.pos.tolist(), (b, h)
    assert kv4.lengths().tolist() == [4] * 4 and kv4.recsa_kv4_get_status() == R.RECSA_OK


@pytest.mark.parametrize("B,Hkv,L,cap,budget", [
    (16, 8, 7000, 7100, 6000), (2, 3, 7000, 7100, 6999), (64, 16, 3000, 45000, 1500), (5, 8, 20000, 20001, 4097),
    (64, 8, 9000, 50000, 8999)])
def test_evict_of_many_and_few_units(R, B, Hkv, L, cap, budget):
    """One CTA a unit and a cluster, by the units and the capacity; ragged lengths, many ties."""
    first, recent = 5, 100
    lengths = [L - 37 * (b % 5) for b in range(B)]
    cfg = R.Config(head_dim=64, n_q_heads=Hkv, n_kv_heads=Hkv, dtype="bf16")
    kv4 = R.RecsaKV4(cfg, cap, B)
    x = torch.zeros(1, 1, L, 64, dtype=torch.bfloat16, device="cuda").expand(B, Hkv, L, 64)
    kv4.recsa_kv4_build(x, x, lengths)
    g = torch.Generator(device="cuda").manual_seed(1)
    w = (torch.rand(B, Hkv, L, generator=g, device="cuda") * 500).floor()
    at, Ls = torch.arange(L, device="cuda"), torch.tensor(lengths, device="cuda")[:, None]
    there = at < Ls
    w = torch.where(there[:, None], w, 0.0)
    kv4.weights()[:, :, :L] = w
    kv4.recsa_kv4_evict(budget, first, recent)
    safe = (at < first) | (at >= Ls - recent)
    key = torch.where(safe[:, None], torch.inf, w)
    key = torch.where(there[:, None], key, -1.0)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    kept = torch.zeros(B, Hkv, L, dtype=torch.bool, device="cuda").scatter_(2, order, True)
    pos = kv4.positions()
    for b in range(B):
        if lengths[b] <= budget:
            assert torch.equal(pos[b, :, :lengths[b]], at[:lengths[b]].int().expand(Hkv, -1))
            continue
        for h in range(0, Hkv, 3):
            want = torch.arange(budget, device="cuda")
            want[~kept[b, h, :budget]] = at[budget:][kept[b, h, budget:]]
            assert torch.equal(pos[b, h, :budget].long(), want), (b, h)
            assert torch.equal(kv4.weights()[b, h, :budget], w[b, h, want])
    assert kv4.lengths().tolist() == [min(x, budget) for x in lengths]
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK
