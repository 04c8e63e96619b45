"""Attention over the 4-bit KV cache where keys and values span many magnitudes: a huge token
that no row gives weight to, that a row does not see, or that was evicted; groups of dims of
unequal size; a heavy token of tiny value before a long faint background.

Tolerances, from the arithmetic, of one output dim of one row with probabilities p_t:
  * probabilities: off by twice a score's error (relative), 16 * 2^-24 * S with S = 2 * scale *
    sum |q| |K_t| over the tokens that have weight, plus 2^-20 for exp2 and the sums: times
    sum p |V|.
  * P' (probability times step, 2^-11; fp32 tensors 2^-21) meets codes of at most 8 in
    magnitude: times 8 sum p s.  Below fp16's normal numbers it is off by 2^-25 where the
    largest of the row and group is at least 2^8: N tokens add at most N * 2^-33 of the
    largest p s, times 8 (fp32 tensors: the low part is scaled by 2^11, 2^-44).
  * on the tensor cores K and V enter as fp16 (2^-11; S then adds 2^-12 * S) and P too.
  * the output is rounded to its type."""
import numpy as np
import pytest
import torch

from oracle import kv4_oracle as O
from tests import test_gpu_kv4 as T

pytestmark = pytest.mark.gpu
R = T.R                                                  # the fixture


def floor_of(u, s, q, at, dtype, tc):
    """Tolerance [d] of one row q [d] at position `at`, beside the output's own rounding."""
    p = u.probabilities(q, at)
    heavy = p > 2.0 ** -60
    S = 2 * u.scale * (np.abs(u.k[heavy]) @ np.abs(q)).max()
    delta = 16 * 2.0 ** -24 * S + (2.0 ** -12 * S if tc else 0)
    pv = p[heavy] @ np.abs(u.v[heavy])
    steps = (p[:, None] * s).repeat(32, 1)
    floor = (2 * delta + 2.0 ** -20) * pv + T.PROB[dtype] * 8 * steps.sum(0)
    floor += 8 * len(p) * 2.0 ** (-33 if dtype == "bf16" else -44) * steps.max(0)
    return floor + (2 * 2.0 ** -11 * pv if tc else 0)


def run(R, dtype, d, k, v, Q, n, lengths=None, prepare=None):
    """One KV head: k, v [L][d], Q [n][G][d]; n = 0: a decode of Q[0].  Compares all rows."""
    L, G = len(k), Q.shape[1]
    k, v, Q = (x.to(T.DT[dtype]) for x in (k, v, Q))
    cfg = R.Config(head_dim=d, n_q_heads=G, n_kv_heads=1, dtype=dtype)
    kv4 = R.RecsaKV4(cfg, L, 1, max_queries=max(n, 1))
    kv4.recsa_kv4_build(k.cuda()[None, None], v.cuda()[None, None], [L])
    u = O.Unit(d)
    u.append(T.np64(k), T.np64(v))
    s = O.quantize(T.np64(v))[1]
    if prepare:
        s = prepare(kv4, u, s)
    if n == 0:
        out = kv4.decode(Q[:1].cuda().contiguous())[0][None]
    else:
        out = kv4.prefill(Q[None].cuda())[0]
    tc = T.on_tensor_cores(dtype, n * G)
    out = T.np64(out)
    for i in range(max(n, 1)):
        at = u.seen - max(n, 1) + i
        for g in range(G):
            q = T.np64(Q[i, g])
            want = u.attend(q[None], at)[0]
            tol = T.HALF[dtype] * np.abs(want) * 1.01 + floor_of(u, s, q, at, dtype, tc) + 1e-40
            err = np.abs(out[i, g] - want)
            assert (err <= tol).all(), (i, g, (err / tol).max(), out[i, g][err > tol][:4], want[err > tol][:4])
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK


def normal(L, d, n, G, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(L, d, generator=g), torch.randn(L, d, generator=g),
            torch.randn(max(n, 1), G, d, generator=g))


# (dtype, d, n, G): decode, chunks of few rows, chunks of fp32, chunks on the tensor cores
FORMS = [("bf16", 128, 0, 4), ("bf16", 64, 0, 8), ("f32", 64, 0, 2), ("f32", 128, 0, 8), ("bf16", 128, 4, 2),
         ("bf16", 64, 8, 1), ("f32", 128, 5, 1), ("f32", 64, 30, 4), ("bf16", 128, 5, 4), ("bf16", 64, 70, 2)]


@pytest.mark.parametrize("big", [2.0 ** 12, 2.0 ** 40, 2.0 ** 90])
@pytest.mark.parametrize("dtype,d,n,G", FORMS)
def test_a_huge_value_without_weight(R, dtype, d, n, G, big):
    """Its key points away from every query: p = exp(-60 or less)."""
    k, v, Q = normal(300, d, n, G, 1)
    Q[..., 0] = 6.0
    k[:, 0] = 0
    k[17, 0] = -40.0 * d ** 0.5
    v[17] *= big
    run(R, dtype, d, k, v, Q, n)


@pytest.mark.parametrize("big", [2.0 ** 12, 2.0 ** 40])
@pytest.mark.parametrize("dtype,d,n,G", [f for f in FORMS if f[2]])
def test_a_huge_token_that_some_rows_do_not_see(R, dtype, d, n, G, big):
    L = 200
    k, v, Q = normal(L, d, n, G, 2)
    v[L - 2] *= big
    run(R, dtype, d, k, v, Q, n)


@pytest.mark.parametrize("dtype,d,n,G", FORMS)
def test_a_huge_token_that_was_evicted(R, dtype, d, n, G):
    L = 260
    k, v, Q = normal(L, d, n, G, 3)
    k[100] *= 2.0 ** 40
    v[100] *= 2.0 ** 40

    def evict(kv4, u, s):
        u.w = np.ones(L)
        u.w[[100, 7]] = 0.0
        kv4.weights()[0, 0, :L] = torch.from_numpy(u.w).float().cuda()
        kv4.recsa_kv4_evict(L - 2, 0, 20)
        before = u.pos.copy()
        u.evict(L - 2, 0, 20)
        return s[[list(before).index(p) for p in u.pos]]

    run(R, dtype, d, k, v, Q, n, prepare=evict)


@pytest.mark.parametrize("big", [2.0 ** 12, 2.0 ** 40, 2.0 ** 90])
@pytest.mark.parametrize("dtype,d,n,G", FORMS)
def test_groups_of_unequal_size(R, dtype, d, n, G, big):
    """The dims of one group are larger than the others', in all tokens: every group's outputs
    are right by their own size."""
    k, v, Q = normal(300, d, n, G, 4)
    v[:, 32:64] *= big
    run(R, dtype, d, k, v, Q, n)


@pytest.mark.parametrize("tiny", [2.0 ** -20, 2.0 ** -60])
@pytest.mark.parametrize("dtype,d,n,G", FORMS)
def test_a_few_tokens_are_smaller(R, dtype, d, n, G, tiny):
    """Rows whose weight lies on tokens of tiny value, among others that have none."""
    k, v, Q = normal(300, d, n, G, 5)
    Q[..., 0] = 6.0
    k[:, 0] = -40.0 * d ** 0.5
    k[40:45, 0] = 0
    v[40:45] *= tiny
    run(R, dtype, d, k, v, Q, n)


@pytest.mark.parametrize("dtype,d,n,G", [f for f in FORMS if f[2] < 10])
def test_a_heavy_token_of_tiny_value_before_a_faint_background(R, dtype, d, n, G):
    """One token takes nearly all weight and has almost no value; 40000 others share 2^-5 of it
    and make the output; one value is 2^12 times the others' and has no weight."""
    L = 40000
    k, v, Q = normal(L, d, n, G, 6)
    k *= 0.02
    Q[..., 0] = 8.0
    k[:, 0] = -20.0 * 0.6931 * d ** 0.5 / 8
    k[0, 0] = 0.0
    k[9, 0] = -60.0 * d ** 0.5
    v[0] *= 2.0 ** -20
    v[1:] += 0.5
    v[9] *= 2.0 ** 12
    run(R, dtype, d, k, v, Q, n)


def test_wide_sequences_among_others(R):
    """A batch of four: huge values in one sequence from the start, in another by an append; a
    captured chunk with weights, replayed after the append and after a rebuild without them."""
    B, Hkv, G, d, n, L = 4, 2, 4, 128, 6, 200
    lengths = [200, 90, 150, 64]
    k, v = T.keys((B, Hkv, L, d), 1, "bf16"), T.rand((B, Hkv, L, d), 2, "bf16")
    k2, v2 = T.keys((B, Hkv, 3, d), 3, "bf16"), T.rand((B, Hkv, 3, d), 4, "bf16")
    plain = (k.clone(), v.clone())
    v[1, 1, 3] *= 2.0 ** 50
    k2[2, 0, 1, 5] = 2.0 ** 40
    Q = T.rand((B, n, G * Hkv, d), 5, "bf16")
    Q[2, :, :, 5] = -1.0                                 # no row gives the huge key weight
    cfg = R.Config(head_dim=d, n_q_heads=G * Hkv, n_kv_heads=Hkv, dtype="bf16")
    kv4 = R.RecsaKV4(cfg, L + 3, B, max_queries=B * n)
    Qc = Q.cuda()
    out = torch.empty_like(Qc)
    kv4.recsa_kv4_build(k.cuda(), v.cuda(), lengths)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            kv4.recsa_kv4_prefill_chunk(Qc, out, accumulate_rows=2)

    def check(units):
        kv4.weights().zero_()
        out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        w = T.np64(kv4.weights())
        for b, row in enumerate(units):
            for h, u in enumerate(row):
                u.w[:] = 0
                for i in range(n):
                    at = u.seen - n + i
                    qs = T.np64(Q[b, i, h * G:(h + 1) * G])
                    want = u.attend(qs, at, accumulate=i >= n - 2)
                    for x in range(G):
                        floor = floor_of(u, u.steps, qs[x], at, "bf16", True)
                        err = np.abs(T.np64(out[b, i, h * G + x]) - want[x])
                        assert (err <= T.HALF["bf16"] * np.abs(want[x]) * 1.01 + floor).all(), (b, h, i, x)
                assert abs(w[b, h].sum() - 2 * G) <= 2.0 ** -17 * 2 * G
                assert np.abs(w[b, h, :len(u.w)] - u.w).max() <= 2.0 ** -9

    def fresh(k, v):
        units = [[O.Unit(d) for _ in range(Hkv)] for _ in range(B)]
        for b in range(B):
            for h in range(Hkv):
                u, x = units[b][h], T.np64(v[b, h, :lengths[b]])
                u.append(T.np64(k[b, h, :lengths[b]]), x)
                u.steps = O.quantize(x)[1]
        return units

    units = fresh(k, v)
    check(units)
    kv4.recsa_kv4_append(k2.cuda(), v2.cuda())
    for b in range(B):
        for h in range(Hkv):
            u = units[b][h]
            u.append(T.np64(k2[b, h]), T.np64(v2[b, h]))
            u.steps = np.concatenate([u.steps, O.quantize(T.np64(v2[b, h]))[1]])
    check(units)
    kv4.recsa_kv4_build(plain[0].cuda(), plain[1].cuda(), lengths)
    check(fresh(*plain))
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK


@pytest.mark.parametrize("d,G,n,L", [(64, 8, 0, 2_000_001), (64, 8, 16, 500_000), (128, 4, 24, 300_003)])
def test_fp32_sums_over_a_long_cache_do_not_drift(R, d, G, n, L):
    """Nearly flat softmax over many tokens: the output is a small mean of values of both signs, so
    a sum that rounds one way shows (2e-5 to 2e-4 of the output, in norm, with the products' own
    accumulators).  Errors that differ from token to token shrink as the output does: scores
    16 * 2^-24 * 4, exp2 2^-22 and P' 2^-22, together below 2^-19; a lane's m additions to nearest
    add 2^-24 sqrt(m), m <= 2000 (2^-18.5): 2^-18 in norm.  The oracle takes the cache's values as
    they are read back (exact in fp32, tested beside this file)."""
    k, v, Q = normal(L, d, n, G, 8)
    cfg = R.Config(head_dim=d, n_q_heads=G, n_kv_heads=1, dtype="f32")
    kv4 = R.RecsaKV4(cfg, L, 1, max_queries=max(n, 1))
    kv4.recsa_kv4_build(k.cuda()[None, None], v.cuda()[None, None], [L])
    out = kv4.prefill(Q[None].cuda())[0] if n else kv4.decode(Q.cuda())
    K, V = (x[0, 0].double() for x in kv4.read(0, L))
    at = torch.arange(L, device="cuda")
    off = size = 0.0
    for i in range(max(n, 1)):
        s = Q[i].cuda().double() @ K.T / d ** 0.5
        want = torch.softmax(s.masked_fill(at > L - max(n, 1) + i, -float("inf")), -1) @ V
        off += float((out[i].double() - want).square().sum())
        size += float(want.square().sum())
    assert off ** 0.5 <= 2.0 ** -18 * size ** 0.5, (off / size) ** 0.5


def test_bf16_sums_over_a_long_cache_do_not_drift(R):
    """512 units of 262144 tokens (one pair of tensors read by all: strides of 0), nearly flat
    softmax: beside the outputs' own rounding, P' may be off by 2^-11 independently."""
    B, Hkv, G, d, L = 64, 8, 1, 64, 262144
    k, v, Q = normal(L, d, 0, B * Hkv * G, 9)
    k, v, Q = k.bfloat16().cuda(), v.bfloat16().cuda(), Q[0].bfloat16().view(B, Hkv * G, d).cuda()
    cfg = R.Config(head_dim=d, n_q_heads=G * Hkv, n_kv_heads=Hkv, dtype="bf16")
    kv4 = R.RecsaKV4(cfg, L, B)
    kv4.recsa_kv4_build(k.expand(B, Hkv, L, d), v.expand(B, Hkv, L, d), [L] * B)
    out = kv4.decode(Q).double()
    u = O.Unit(d)
    u.append(T.np64(k), T.np64(v))
    K, V = torch.from_numpy(u.k).cuda(), torch.from_numpy(u.v).cuda()
    want = torch.softmax(Q.double().view(-1, d) @ K.T / d ** 0.5, -1) @ V
    want = want.view_as(out)
    own = (want.bfloat16().double() - want).norm()
    assert (out - want).norm() <= (own.square() + (2.0 ** -11 * want.norm()).square()).sqrt()
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK


@pytest.mark.parametrize("Hkv,G,n,L,mean", [(64, 2, 70, 1_000_000, 0.0), (148, 1, 12, 300_001, 0.3), (200, 1, 130, 70_000, 0.0)])
def test_chunk_sums_over_a_long_cache_do_not_drift(R, Hkv, G, n, L, mean):
    """Units that lie nearly whole in a CTA (one pair of tensors read by all: strides of 0).  The
    products' accumulators may lose half a step, 2^-25, a product, over the 2048 products of 256
    tiles; the outputs' own rounding is unbiased (its mean over 2000 and more outputs is below
    2^-8 / 3 / 45).  So the outputs' scale is within 2^-13 of the exact one."""
    d = 64
    k, v, Q = normal(L, d, n, Hkv * G, 10)
    k, v, Q = k.bfloat16().cuda(), (v + mean).bfloat16().cuda(), Q.bfloat16().cuda()
    cfg = R.Config(head_dim=d, n_q_heads=G * Hkv, n_kv_heads=Hkv, dtype="bf16")
    kv4 = R.RecsaKV4(cfg, L, 1, max_queries=n)
    kv4.recsa_kv4_build(k.expand(1, Hkv, L, d), v.expand(1, Hkv, L, d), [L])
    out = kv4.prefill(Q[None])[0].double()
    u = O.Unit(d)
    u.append(T.np64(k), T.np64(v))
    K, V = torch.from_numpy(u.k).cuda(), torch.from_numpy(u.v).cuda()
    at = torch.arange(L, device="cuda")[None] <= L - n + torch.arange(n, device="cuda")[:, None]
    dot = square = off = own = 0.0
    for h in (0, Hkv // 2, Hkv - 1):
        s = (Q[:, h * G].double() @ K.T / d ** 0.5).masked_fill(~at, -float("inf"))
        want, got = torch.softmax(s, -1) @ V, out[:, h * G]
        dot += float((got * want).sum())
        square += float(want.square().sum())
        off += float((got - want).square().sum())
        own += float((want.bfloat16().double() - want).square().sum())
    assert abs(dot / square - 1) <= 2.0 ** -13, dot / square - 1
    # K, V and P as fp16 are off by 2^-11 each, independently
    assert off <= own + 3 * 2.0 ** -22 * square, ((off / square) ** 0.5, (own / square) ** 0.5)
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK
