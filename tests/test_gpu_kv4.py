"""The 4-bit KV cache on the GPU against the fp64 oracle.

Tolerances, from the arithmetic.  A score is a sum of at most 16 fp32 roundings of terms
bounded by S = scale * sum |q| (|lo| + 15 s), so it is off by at most 16 * 2^-24 * S, and a
probability by twice that (relative), plus 2^-21 for exp2 and the sums.  P' (probability
times step) is rounded to fp16 (2^-11; fp32 tensors: twice 11 bits, 2^-21) and meets codes of
at most 8 in magnitude, so an output adds that times 8 s.  The output is rounded to its type:
half a step, 2^-8 (bf16) or 2^-24 of it.

bf16 chunks of more than 8 rows a KV head (`tc`): K and V enter the products as fp16, half a
step is 2^-11 of each value.  A score is then off by at most 2^-11 * scale * sum |q| |K|, and
S above is at least twice that sum; P and V are each off by 2^-11, so an output by
2 * 2^-11 * max |V| more.  These errors are independent from token to token and dim to dim,
so beside that bound the whole output's error, in norm, is within the bf16 rounding's."""
import numpy as np
import pytest
import torch

from oracle import kv4_oracle as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
PROB = {"bf16": 2.0 ** -11, "f32": 2.0 ** -21}


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import long_context_recsa_b200.recsa as R
    return R


def rand(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(DT[dtype])


def keys(shape, seed, dtype):
    """Keys with unequal channels and offsets."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g)
    x = x * torch.exp(0.5 * torch.randn(shape[-1], generator=g)) + torch.randn(shape[-1], generator=g)
    return x.to(DT[dtype])


def np64(x):
    return x.detach().cpu().double().numpy()


def make(R, dtype, d, Hkv, G, lengths, seed=0, cap=None, max_queries=None, extra=0):
    """A built cache and the oracle's units."""
    B = len(lengths)
    T = max(max(lengths), 1)
    cap = cap or T + extra
    k, v = keys((B, Hkv, T, d), seed + 1, dtype), rand((B, Hkv, T, d), seed + 2, dtype)
    cfg = R.Config(head_dim=d, n_q_heads=G * Hkv, n_kv_heads=Hkv, dtype=dtype)
    kv4 = R.RecsaKV4(cfg, cap, B, max_queries=max_queries)
    kv4.recsa_kv4_build(k.cuda(), v.cuda(), lengths)
    units = [[O.Unit(d) for _ in range(Hkv)] for _ in range(B)]
    for b in range(B):
        for h in range(Hkv):
            units[b][h].append(np64(k[b, h, :lengths[b]]), np64(v[b, h, :lengths[b]]))
    return kv4, units


def on_tensor_cores(dtype, rows):
    return dtype == "bf16" and rows > 8


def bound_of(u, q, dtype, tc=False):
    """(score error, tolerance floor of an output) of one unit and query rows q [G][d]."""
    if len(u.k) == 0:
        return 0.0, 0.0
    big = np.abs(u.k).max(0) * 2 + 1e-30
    S = u.scale * (np.abs(q) @ big).max()
    delta = 16 * 2.0 ** -24 * S
    if tc:
        delta += 2.0 ** -12 * S
        return delta, (2 * delta + 2.0 ** -10) * np.abs(u.v).max()
    g = u.v.reshape(len(u.v), -1, 32)
    step8 = 8.0 / 15.0 * 1.01 * (g.max(-1) - g.min(-1)).max()
    return delta, PROB[dtype] * step8 + (2 * delta + 2.0 ** -21) * np.abs(u.v).max()


def check_rows(out, want, floor, dtype, what):
    err = np.abs(np64(out) - want)
    tol = HALF[dtype] * np.abs(want) * 1.01 + floor
    assert (err <= tol).all(), f"{what}: {err.max()} at tolerance {tol.flat[err.argmax()]}"


def check_decode(kv4, units, q, out, dtype, G):
    for b, row in enumerate(units):
        for h, u in enumerate(row):
            qs = np64(q[b, h * G:(h + 1) * G])
            want = u.attend(qs, u.seen - 1)
            check_rows(out[b, h * G:(h + 1) * G], want, bound_of(u, qs, dtype)[1], dtype, (b, h))


def check_weights(kv4, units, dtype, rows, q_all, tc=False):
    w = np64(kv4.weights())
    for b, row in enumerate(units):
        for h, u in enumerate(row):
            delta = bound_of(u, q_all[b, h], dtype, tc)[0]
            err = np.abs(w[b, h, :len(u.w)] - u.w)
            assert (err <= (2 * delta + 2.0 ** -19) * np.abs(u.w) + 1e-30).all(), (b, h, err.max())
            assert (w[b, h, len(u.w):] == 0).all()


# ------------------------------------------------------------------------- writing -----
def check_values(kv4, units, dtype):
    n = max(max(len(u.k) for row in units for u in row), 1)
    k, v = kv4.read(0, n)
    lens = kv4.lengths().tolist()
    for b, row in enumerate(units):
        for h, u in enumerate(row):
            L = len(u.k)
            assert lens[b] == L
            for got, want in ((k, u.k), (v, u.v)):
                # values are short sums: exact in fp32, then rounded once
                w = torch.from_numpy(want).float().to(DT[dtype])
                assert torch.equal(torch.nan_to_num(got[b, h, :L].cpu(), nan=7e7),
                                   torch.nan_to_num(w, nan=7e7)), (b, h)
                assert (got[b, h, L:] == 0).all()
            assert kv4.positions()[b, h, :L].cpu().tolist() == u.pos.tolist()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,Hkv,lengths", [(64, 1, [1]), (64, 3, [0, 33, 5]), (128, 2, [129, 64, 0, 1]),
                                           (128, 1, [1000])])
def test_build_values(R, dtype, d, Hkv, lengths):
    kv4, units = make(R, dtype, d, Hkv, 2, lengths)
    check_values(kv4, units, dtype)
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_special_groups(R, dtype):
    """Ties, constants, signs, tiny and huge values, infinities and NaN."""
    d = 128
    x = torch.zeros(16, d)
    x[0] = 3.0
    x[1] = torch.arange(d) % 32 * 0.5 - 4                # many exact ties of code + 1/2
    x[2] = torch.arange(d) % 31 * 1.0
    x[3] = -x[2]
    x[4] = torch.linspace(1e-38, 3e-38, d)
    x[5] = torch.linspace(-3e38, 3e38, d)
    x[6] = 100 + torch.linspace(-1, 1, d)
    x[7] = torch.randn(d, generator=torch.Generator().manual_seed(3))
    x[8] = x[7]; x[8, 40] = float("inf")
    x[9] = x[7]; x[9, 40] = float("nan"); x[9, 100] = -float("inf")
    x[10] = torch.linspace(-1e-40, 1e-40, d)             # subnormal
    x[11, ::2] = -0.0
    x[12] = torch.linspace(1, 1.0001, d)
    x[13] = 2.0 ** torch.arange(-64.0, 64.0)
    x[14] = torch.linspace(-1, 15 * 0.37 - 1, d)
    x = x.to(DT[dtype])
    cfg = R.Config(head_dim=d, n_q_heads=1, n_kv_heads=1, dtype=dtype)
    kv4 = R.RecsaKV4(cfg, 16, 1)
    kv4.recsa_kv4_build(x.cuda()[None, None], x.flip(0).contiguous().cuda()[None, None], [16])
    u = O.Unit(d)
    u.append(np64(x), np64(x.flip(0)))
    k, v = kv4.read(0, 16)
    for got, want in ((k, u.k), (v, u.v)):
        got, want = got[0, 0].cpu(), torch.from_numpy(want).float().to(DT[dtype])
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_build_from_a_strided_cache_and_again(R, dtype, d):
    B, Hkv, T = 2, 2, 50
    big = keys((B, T + 9, Hkv, 2 * d), 5, dtype).cuda()  # [b][t][h][.., d of it]
    k = big[:, :, :, :d].permute(0, 2, 1, 3)
    v = big[:, :, :, d:].permute(0, 2, 1, 3)
    cfg = R.Config(head_dim=d, n_q_heads=2, n_kv_heads=Hkv, dtype=dtype)
    kv4 = R.RecsaKV4(cfg, 70, B)
    kv4.recsa_kv4_build(k, v, [50, 41])
    kv4.weights()[0, 0, :50] = 3.0
    kv4.recsa_kv4_build(k, v, [20, 7])                   # shorter: the rest is cleared
    units = [[O.Unit(d) for _ in range(Hkv)] for _ in range(B)]
    for b, L in enumerate([20, 7]):
        for h in range(Hkv):
            units[b][h].append(np64(k[b, h, :L]), np64(v[b, h, :L]))
    check_values(kv4, units, dtype)
    assert (kv4.weights() == 0).all() and (kv4.positions()[:, :, 20:] == 0).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 128), ("bf16", 64)])
def test_append_with_counts(R, dtype, d):
    kv4, units = make(R, dtype, d, 2, 1, [5, 0, 30], cap=60)
    for step, (n, counts) in enumerate([(1, None), (7, [7, 0, 3]), (40, [1, 40, 0]), (3, None)]):
        k, v = keys((3, 2, n, d), 50 + step, dtype), rand((3, 2, n, d), 60 + step, dtype)
        c = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
        kv4.recsa_kv4_append(k.cuda(), v.cuda(), c)
        for b in range(3):
            m = n if counts is None else counts[b]
            for h in range(2):
                units[b][h].append(np64(k[b, h, :m]), np64(v[b, h, :m]))
        check_values(kv4, units, dtype)
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK


def test_append_past_the_capacity_and_bad_counts(R):
    kv4, units = make(R, "f32", 64, 1, 1, [5, 9], cap=10)
    k = keys((2, 1, 3, 64), 1, "f32").cuda()
    kv4.recsa_kv4_append(k, k)                           # fits the first sequence only
    assert kv4.recsa_kv4_get_status() == R.RECSA_E_CAPACITY
    units[0][0].append(np64(k[0, 0]), np64(k[0, 0]))
    check_values(kv4, units, "f32")
    bad = torch.tensor([4, -1], dtype=torch.int32, device="cuda")
    kv4.recsa_kv4_append(k, k, bad)
    assert kv4.recsa_kv4_get_status() == R.RECSA_E_DEVICE
    check_values(kv4, units, "f32")
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK
    with pytest.raises(R.RecsaError) as e:
        kv4.recsa_kv4_append(torch.zeros(2, 1, 11, 64, device="cuda"), torch.zeros(2, 1, 11, 64, device="cuda"))
    assert e.value.status == R.RECSA_E_CAPACITY


# ------------------------------------------------------------------------- decode ------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,Hkv,G,lengths", [
    (64, 1, 1, [1]), (128, 1, 8, [16, 17]), (128, 2, 4, [0, 31, 33, 200]), (64, 2, 8, [5, 1000]),
    (64, 3, 2, [95, 96, 97, 0, 1]), (128, 1, 2, [2500]), (64, 1, 4, [777])])
def test_decode(R, dtype, d, Hkv, G, lengths):
    kv4, units = make(R, dtype, d, Hkv, G, lengths)
    q = rand((len(lengths), G * Hkv, d), 9, dtype)
    out = kv4.decode(q.cuda())
    check_decode(kv4, units, q, out, dtype, G)
    assert torch.equal(out, kv4.decode(q.cuda()))        # the same bits each time
    assert (kv4.weights() == 0).all()
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK


@pytest.mark.parametrize("dtype,d,G", [("bf16", 128, 4), ("f32", 64, 8), ("f32", 128, 2), ("bf16", 64, 1)])
def test_decode_accumulates(R, dtype, d, G):
    Hkv, lengths = 2, [300, 0, 37]
    kv4, units = make(R, dtype, d, Hkv, G, lengths)
    for step in range(2):
        q = rand((3, G * Hkv, d), 20 + step, dtype, 1.5)
        out = kv4.decode(q.cuda(), accumulate=True)
        check_decode(kv4, units, q, out, dtype, G)
        for b in range(3):
            for h in range(Hkv):
                units[b][h].attend(np64(q[b, h * G:(h + 1) * G]), 10 ** 6, accumulate=True)
    check_weights(kv4, units, dtype, 2, np64(q).reshape(3, Hkv, G, d))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_over_many_splits_and_large_logits(R, dtype):
    """One unit over the whole grid; one sharp query, one flat, one zero."""
    d, L = 128, 50021
    k, v = keys((1, 1, L, d), 3, dtype), rand((1, 1, L, d), 4, dtype)
    q = rand((1, 4, d), 5, dtype)
    q[0, 0] = (k[0, 0, 31337].float() * 8).to(DT[dtype])
    q[0, 1] *= 0.01
    q[0, 2] = 0
    cfg = R.Config(head_dim=d, n_q_heads=4, n_kv_heads=1, dtype=dtype)
    kv4 = R.RecsaKV4(cfg, L, 1)
    kv4.recsa_kv4_build(k.cuda(), v.cuda(), [L])
    out = kv4.decode(q.cuda(), accumulate=True)
    u = O.Unit(d)
    u.append(np64(k[0, 0]), np64(v[0, 0]))
    for i in range(4):
        qs = np64(q[0, i:i + 1])
        check_rows(out[0, i:i + 1], u.attend(qs, L, True), bound_of(u, qs, dtype)[1], dtype, i)
    check_weights(kv4, [[u]], dtype, 1, np64(q).reshape(1, 1, 4, d))


def test_values_of_unequal_magnitude(R):
    """Tokens whose values differ by 2^40: the small ones count where the large have no weight."""
    d, L = 64, 64
    k = torch.zeros(1, 1, L, d)
    k[0, 0, 0] = -40.0
    v = rand((1, 1, L, d), 1, "f32")
    v[0, 0, 0] *= 2.0 ** 20
    v[0, 0, 1:] *= 2.0 ** -4
    cfg = R.Config(head_dim=d, n_q_heads=1, n_kv_heads=1, dtype="f32")
    kv4 = R.RecsaKV4(cfg, L, 1)
    kv4.recsa_kv4_build(k.cuda(), v.cuda(), [L])
    q = torch.ones(1, 1, d)
    out = np64(kv4.decode(q.cuda())[0])
    u = O.Unit(d)
    u.append(np64(k[0, 0]), np64(v[0, 0]))
    want = u.attend(np64(q[0]), L)
    assert np.abs(out - want).max() <= 2e-6 * np.abs(u.v[1:]).max()


# ------------------------------------------------------------------------- chunks ------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,Hkv,G,lengths,n,counts,mq", [
    (64, 1, 1, [5], 5, None, None), (128, 2, 4, [40, 33], 3, None, None),
    (128, 1, 8, [100, 9, 64], 9, [9, 0, 4], 5 * 3), (64, 2, 2, [200, 77], 50, [50, 13], 2 * 50),
    (64, 1, 4, [0, 130], 7, [0, 7], 2 * 7), (128, 1, 2, [150], 150, None, 64), (64, 1, 1, [1], 1, None, 1),
    (128, 2, 4, [129, 500], 33, None, 2 * 33), (128, 1, 1, [1030], 300, None, 300), (64, 1, 8, [400], 70, None, 40),
    (64, 2, 1, [128, 127, 9], 9, [9, 0, 5], 3 * 9), (128, 1, 4, [260], 260, None, 260)])
def test_chunk(R, dtype, d, Hkv, G, lengths, n, counts, mq):
    B = len(lengths)
    kv4, units = make(R, dtype, d, Hkv, G, lengths, max_queries=mq)
    Q = rand((B, n, G * Hkv, d), 31, dtype)
    c = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    O_ = torch.full((B, n, G * Hkv, d), 5.0, dtype=DT[dtype], device="cuda")
    acc = max(1, n // 3)
    wave = min(n, (mq or B) // B)
    tc = on_tensor_cores(dtype, wave * G)
    kv4.recsa_kv4_prefill_chunk(Q.cuda(), O_, c, accumulate_rows=acc)
    off = size = 0.0
    for b in range(B):
        m = n if counts is None else counts[b]
        assert (O_[b, m:] == 5.0).all()                  # rows behind are left as they were
        for i in range(m):
            at = lengths[b] - m + i
            for h in range(Hkv):
                u = units[b][h]
                qs = np64(Q[b, i, h * G:(h + 1) * G])
                want = u.attend(qs, at, accumulate=i >= m - acc)
                got = O_[b, i, h * G:(h + 1) * G]
                check_rows(got, want, bound_of(u, qs, dtype, tc)[1], dtype, (b, i, h))
                off += ((np64(got) - want) ** 2).sum()
                size += (want ** 2).sum()
    assert off ** 0.5 <= HALF[dtype] * size ** 0.5 + (0 if dtype == "bf16" else 2.0 ** -20 * size ** 0.5)
    q_all = np64(Q).reshape(B, n, Hkv, G, d).transpose(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)
    check_weights(kv4, units, dtype, acc, q_all, tc)
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK


def test_chunk_refuses_more_rows_than_tokens(R):
    kv4, units = make(R, "bf16", 64, 1, 2, [3, 20])
    Q = rand((2, 5, 2, 64), 1, "bf16").cuda()
    O_ = torch.full_like(Q, 9.0)
    kv4.recsa_kv4_prefill_chunk(Q, O_, accumulate_rows=2)
    assert kv4.recsa_kv4_get_status() == R.RECSA_E_DEVICE
    assert (O_[0] == 9.0).all() and (O_[1] != 9.0).any()  # the other sequence's rows are right
    want = units[1][0].attend(np64(Q[1, 4]), 19)
    check_rows(O_[1, 4], want, bound_of(units[1][0], np64(Q[1, 4]), "bf16")[1], "bf16", "row")
    big = R.RecsaKV4(kv4.cfg, 20, 2, max_queries=10)     # the same on the tensor cores
    big.recsa_kv4_append(rand((2, 1, 3, 64), 2, "bf16").cuda(), rand((2, 1, 3, 64), 3, "bf16").cuda())
    O_.fill_(9.0)
    big.recsa_kv4_prefill_chunk(Q, O_)
    assert big.recsa_kv4_get_status() == R.RECSA_E_DEVICE and (O_ == 9.0).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64), ("bf16", 64)])
def test_nan_tokens_reach_only_the_rows_that_see_them(R, dtype, d):
    n, L = 20, 70
    k, v = keys((1, 1, L, d), 1, dtype), rand((1, 1, L, d), 2, dtype)
    v[0, 0, 60, 3] = float("nan")                        # position 60: rows 0..9 do not see it
    k[0, 0, 66, 40] = float("inf")                       # position 66: rows 0..15 do not
    cfg = R.Config(head_dim=d, n_q_heads=2, n_kv_heads=1, dtype=dtype)
    kv4 = R.RecsaKV4(cfg, L + 30, 1, max_queries=n)
    kv4.recsa_kv4_build(k.cuda(), v.cuda(), [L])
    Q = rand((1, n, 2, d), 3, dtype)
    out = np64(kv4.prefill(Q.cuda())[0])
    assert np.isfinite(out[:10]).all()
    assert np.isnan(out[10:16, :, :32]).all() and np.isfinite(out[10:16, :, 32:]).all()
    assert np.isnan(out[16:]).all()
    k2, v2 = k.clone(), v.clone()
    k2[0, 0, 60:], v2[0, 0, 60:] = 0, 0
    kv4.recsa_kv4_build(k2.cuda(), v2.cuda(), [L])
    assert np.array_equal(out[:10], np64(kv4.prefill(Q.cuda())[0, :10]))
    # rows past the length may hold anything: shrink, and the NaN rows are out of it
    kv4.recsa_kv4_build(k.cuda(), v.cuda(), [L])
    kv4.recsa_kv4_build(k.cuda(), v.cuda(), [59])
    assert torch.isfinite(kv4.decode(Q[:, 0].contiguous().cuda())).all()


@pytest.mark.parametrize("big", [1.0, 2.0 ** 10, 2.0 ** 28])
@pytest.mark.parametrize("n,G", [(5, 1), (20, 2), (70, 4)])
def test_chunk_of_large_and_growing_logits(R, n, G, big):
    """Scores that rise along the cache, so that the running reference moves in every tile, up
    to 2^35.  Five neighbouring keys are equal, in every rounding; the next five score 2 * big
    less.  With big = 1 the general bound holds.  With the larger ones all weight of a row lies
    on the newest keys it sees that are equal (exp(-2048) = 0), whatever the keys' rounding;
    P and V are off by 2^-11 each."""
    d, L = 64, 600
    k = torch.zeros(1, 1, L, d)
    k[0, 0, :, 0] = torch.arange(L).float() // 5 - 60    # |k| <= 60: 8 bits; lo = s = exact or 0
    v = rand((1, 1, L, d), 4, "bf16").float()
    Q = torch.zeros(1, n, G, d)
    Q[..., 0] = 16.0 * big                               # score = 2 big k
    cfg = R.Config(head_dim=d, n_q_heads=G, n_kv_heads=1, dtype="bf16")
    kv4 = R.RecsaKV4(cfg, L, 1, max_queries=n)
    kv4.recsa_kv4_build(k.bfloat16().cuda(), v.bfloat16().cuda(), [L])
    u = O.Unit(d)
    u.append(np64(k.bfloat16()[0, 0]), np64(v.bfloat16()[0, 0]))
    out = np64(kv4.prefill(Q.bfloat16().cuda())[0])
    for i in range(n):
        qs = np64(Q[0, i, :1])
        want = u.attend(qs, L - n + i)
        tc = on_tensor_cores("bf16", n * G)
        floor = bound_of(u, qs, "bf16", tc)[1] if big == 1 else 2.0 ** -10 * np.abs(u.v).max()
        check_rows(torch.from_numpy(out[i]), np.repeat(want, G, 0), floor, "bf16", i)
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK


# ------------------------------------------------------------------------- eviction ----
def set_weights(kv4, units, seed, ties=False):
    g = torch.Generator().manual_seed(seed)
    for b, row in enumerate(units):
        for h, u in enumerate(row):
            w = torch.rand(len(u.w), generator=g)
            if ties:
                w = (w * 4).floor()
            u.w = w.double().numpy().copy()
            kv4.weights()[b, h, :len(u.w)] = w.cuda()


def check_evicted(kv4, units, dtype):
    check_values(kv4, units, dtype)
    for b, row in enumerate(units):
        for h, u in enumerate(row):
            w = kv4.weights()[b, h].cpu().double().numpy()
            assert np.array_equal(np.nan_to_num(w[:len(u.w)], nan=-9), np.nan_to_num(u.w, nan=-9))
            assert (w[len(u.w):] == 0).all() and (kv4.positions()[b, h, len(u.w):] == 0).all()


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("dtype,d,lengths,budget,first,recent", [
    ("bf16", 128, [100, 30, 31], 30, 4, 8), ("f32", 64, [2000, 0, 1999], 1000, 0, 0),
    ("bf16", 64, [5000], 64, 32, 32), ("f32", 128, [3, 1, 2], 1, 1, 0), ("bf16", 128, [1500, 9], 1499, 0, 700),
    ("f32", 64, [1025], 1, 0, 1), ("bf16", 64, [9000, 7000, 50], 4000, 16, 100), ("f32", 64, [6500], 6400, 0, 0),
    ("bf16", 128, [8193], 17, 3, 9)])
def test_evict(R, dtype, d, lengths, budget, first, recent, ties):
    kv4, units = make(R, dtype, d, 2, 1, lengths, extra=8)
    set_weights(kv4, units, 4, ties)
    kv4.recsa_kv4_evict(budget, first, recent)
    for row in units:
        for u in row:
            u.evict(budget, first, recent)
    check_evicted(kv4, units, dtype)
    q = rand((len(lengths), 2, d), 8, dtype)
    check_decode(kv4, units, q, kv4.decode(q.cuda()), dtype, 1)
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK


def test_evict_short_length_in_a_large_cache(R):
    """Most CTAs of the cluster own no slot."""
    kv4, units = make(R, "f32", 64, 2, 1, [100, 129, 1], cap=20000)
    set_weights(kv4, units, 5)
    kv4.recsa_kv4_evict(50, 3, 7)
    for row in units:
        for u in row:
            u.evict(50, 3, 7)
    check_evicted(kv4, units, "f32")


def test_evict_past_the_keys_that_shared_memory_holds(R):
    L, budget = 400_000, 150_000
    cfg = R.Config(head_dim=64, n_q_heads=1, n_kv_heads=1, dtype="bf16")
    kv4 = R.RecsaKV4(cfg, L + 7, 1)
    g = torch.Generator().manual_seed(1)
    x = torch.zeros(1, 1, L, 64, dtype=torch.bfloat16, device="cuda")
    kv4.recsa_kv4_build(x, x, [L])
    w = (torch.rand(L, generator=g) * 1000).floor()      # many ties
    kv4.weights()[0, 0, :L] = w.cuda()
    kv4.recsa_kv4_evict(budget, 5, 1000)
    safe = torch.zeros(L, dtype=torch.bool)
    safe[:5] = safe[L - 1000:] = True
    key = torch.where(safe, torch.tensor(float("inf")), w)
    keep = torch.sort(key, descending=True, stable=True).indices[:budget]
    kept = torch.zeros(L, dtype=torch.bool)
    kept[keep] = True
    want = torch.arange(budget)
    want[~kept[:budget]] = torch.arange(budget, L)[kept[budget:]]
    assert torch.equal(kv4.positions()[0, 0, :budget].cpu().long(), want)
    assert torch.equal(kv4.weights()[0, 0, :budget].cpu(), w[want])
    assert (kv4.weights()[0, 0, budget:] == 0).all() and kv4.lengths().tolist() == [budget]


def test_evict_orders_odd_weights(R):
    """NaN lowest, then -inf, negative, the two zeros alike, inf."""
    kv4, units = make(R, "f32", 64, 1, 1, [12])
    w = [float("nan"), -float("inf"), -1.0, -0.0, 0.0, 1e-45, 1.0, float("inf"), float("nan"), 0.0, -0.0, 2.0]
    for budget in (11, 10, 9, 8, 7, 6, 5, 4, 3, 2, 1):
        kv4, units = make(R, "f32", 64, 1, 1, [12])
        units[0][0].w = np.array(w)
        kv4.weights()[0, 0, :12] = torch.tensor(w)
        kv4.recsa_kv4_evict(budget)
        units[0][0].evict(budget, 0, 0)
        assert kv4.positions()[0, 0, :budget].cpu().tolist() == units[0][0].pos.tolist(), budget


def test_evict_refusals(R):
    kv4, _ = make(R, "f32", 64, 1, 1, [12])
    for args in [(0, 0, 0), (-3, 0, 0), (5, -1, 0), (5, 0, -1), (5, 3, 3), (5, 6, 0), (5, 2 ** 62, 2 ** 62)]:
        with pytest.raises(R.RecsaError) as e:
            kv4.recsa_kv4_evict(*args)
        assert e.value.status == R.RECSA_E_INVAL


# ------------------------------------------------------------------------- together ----
@pytest.mark.parametrize("dtype,d,G", [("bf16", 128, 4), ("f32", 64, 8), ("f32", 128, 1)])
def test_a_bounded_cache_in_use(R, dtype, d, G):
    """A prompt in two chunks, its newest rows' weights, eviction, decode steps that append,
    attend with weights and evict, and a chunk over the evicted cache (slots out of order)."""
    B, Hkv, cap, budget = 2, 2, 260, 90
    cfg = R.Config(head_dim=d, n_q_heads=G * Hkv, n_kv_heads=Hkv, dtype=dtype)
    kv4 = R.RecsaKV4(cfg, cap, B, max_queries=2 * 64)
    units = [[O.Unit(d) for _ in range(Hkv)] for _ in range(B)]

    def append(n, seed, counts=None):
        k, v = keys((B, Hkv, n, d), seed, dtype), rand((B, Hkv, n, d), seed + 1, dtype)
        c = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
        kv4.recsa_kv4_append(k.cuda(), v.cuda(), c)
        for b in range(B):
            m = n if counts is None else counts[b]
            for h in range(Hkv):
                units[b][h].append(np64(k[b, h, :m]), np64(v[b, h, :m]))
        return c

    def chunk(n, seed, counts=None, acc=0):
        Q = rand((B, n, G * Hkv, d), seed, dtype)
        c = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
        out = kv4.prefill(Q.cuda(), c, accumulate_rows=acc)
        for b in range(B):
            m = n if counts is None else counts[b]
            for i in range(m):
                for h in range(Hkv):
                    u = units[b][h]
                    qs = np64(Q[b, i, h * G:(h + 1) * G])
                    want = u.attend(qs, u.seen - m + i, accumulate=i >= m - acc)
                    tc = on_tensor_cores(dtype, min(n, 64) * G)
                    check_rows(out[b, i, h * G:(h + 1) * G], want, bound_of(u, qs, dtype, tc)[1], dtype, (b, i, h))

    def evict():
        # near-equal weights may rank either way: take the library's own weights
        w = kv4.weights().cpu().double().numpy()
        for b in range(B):
            for h in range(Hkv):
                u = units[b][h]
                assert np.abs(w[b, h, :len(u.w)] - u.w).max() <= 1e-4
                u.w = w[b, h, :len(u.w)].copy()
                u.evict(budget, 4, 16)
        kv4.recsa_kv4_evict(budget, 4, 16)
        check_evicted(kv4, units, dtype)

    append(70, 100)
    chunk(70, 110)
    append(50, 120, [50, 31])
    chunk(50, 130, [50, 31], acc=12)
    evict()
    for step in range(4):
        append(1, 140 + 10 * step)
        q = rand((B, G * Hkv, d), 145 + 10 * step, dtype)
        out = kv4.decode(q.cuda(), accumulate=True)
        check_decode(kv4, units, q, out, dtype, G)
        for b in range(B):
            for h in range(Hkv):
                units[b][h].attend(np64(q[b, h * G:(h + 1) * G]), 10 ** 6, accumulate=True)
        evict()
    append(20, 200)
    evict()                                              # between append and attend: rows out of order
    chunk(16, 210, acc=3)
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK


def test_captured_step_replays(R):
    """append + decode + evict captured once and replayed gives what eager steps give."""
    d, B, Hkv, G = 128, 2, 2, 4
    ks = [keys((B, Hkv, 1, d), 300 + i, "bf16").cuda() for i in range(6)]
    qs = [rand((B, G * Hkv, d), 320 + i, "bf16").cuda() for i in range(6)]

    def fresh():
        return make(R, "bf16", d, Hkv, G, [64, 50], cap=80)[0]

    def step(kv4, k, q, out):
        kv4.recsa_kv4_append(k, k)
        kv4.recsa_kv4_decode(q, out, accumulate=True)
        kv4.recsa_kv4_evict(60, 2, 8)

    eager = fresh()
    outs = []
    for k, q in zip(ks, qs):
        o = torch.empty_like(q)
        step(eager, k, q, o)
        outs.append(o)
    kv4 = fresh()
    k, q, o = ks[0].clone(), qs[0].clone(), torch.empty_like(qs[0])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(kv4, k, q, o)
    for i in range(6):
        k.copy_(ks[i])
        q.copy_(qs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, outs[i]), i
    assert torch.equal(kv4.positions(), eager.positions())
    assert torch.equal(kv4.weights(), eager.weights())
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK


@pytest.mark.parametrize("G,n", [(4, 40), (2, 3)])
def test_captured_chunk_replays_after_eager_calls(R, G, n):
    """A chunk with weights, captured while an eager chunk of the same handle came before and
    comes between replays; the tensor-core form and the other."""
    d, B, Hkv = 128, 2, 2
    kv4, _ = make(R, "bf16", d, Hkv, G, [300, 90], max_queries=B * n)
    Qs = [rand((B, n, G * Hkv, d), 70 + i, "bf16").cuda() for i in range(3)]
    want = [kv4.prefill(q) for q in Qs]
    kv4.prefill(Qs[0], accumulate_rows=2)
    once = kv4.weights().clone()
    Q, O_ = Qs[0].clone(), torch.empty_like(Qs[0])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            kv4.recsa_kv4_prefill_chunk(Q, O_, accumulate_rows=2)
    for i in range(3):
        Q.copy_(Qs[i])
        kv4.weights().zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(O_, want[i]), i
        assert i > 0 or torch.equal(kv4.weights(), once)
        assert torch.equal(kv4.prefill(Qs[2]), want[2])
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK


def test_two_chunks_on_two_streams(R):
    """Two caches' tensor-core chunks at once (each takes an SM's whole TMEM)."""
    n, G = 40, 4
    a, _ = make(R, "bf16", 128, 2, G, [900, 64], max_queries=2 * n)
    b, _ = make(R, "bf16", 64, 2, G, [500, 1200], max_queries=2 * n)
    qa, qb = rand((2, n, 8, 128), 1, "bf16").cuda(), rand((2, n, 8, 64), 2, "bf16").cuda()
    want_a, want_b = a.prefill(qa), b.prefill(qb)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = [torch.empty_like(qa) for _ in range(10)], [torch.empty_like(qb) for _ in range(10)]
    for i in range(10):
        a.recsa_kv4_prefill_chunk(qa, oa[i], stream=s1)
        b.recsa_kv4_prefill_chunk(qb, ob[i], stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want_a) for x in oa) and all(torch.equal(x, want_b) for x in ob)
    assert a.recsa_kv4_get_status() == R.RECSA_OK and b.recsa_kv4_get_status() == R.RECSA_OK


def test_two_caches_on_two_streams(R):
    """Handles do not share state: concurrent steps on two streams equal serial ones."""
    a, ua = make(R, "bf16", 128, 2, 4, [900, 33])
    b, ub = make(R, "f32", 64, 4, 2, [500, 1200])
    qa, qb = rand((2, 8, 128), 1, "bf16").cuda(), rand((2, 8, 64), 2, "f32").cuda()
    want_a, want_b = a.decode(qa), b.decode(qb)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = [torch.empty_like(qa) for _ in range(10)], [torch.empty_like(qb) for _ in range(10)]
    for i in range(10):
        a.recsa_kv4_decode(qa, oa[i], stream=s1)
        b.recsa_kv4_decode(qb, ob[i], stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want_a) for x in oa) and all(torch.equal(x, want_b) for x in ob)


def test_binding_refuses_wrong_tensors(R):
    kv4, _ = make(R, "bf16", 64, 2, 2, [9, 4], cap=20)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (q.float(), q[:1], q[:, :2], q.cpu(), q.transpose(0, 1), torch.zeros(2, 4, 128).cuda().bfloat16()[..., ::2]):
        with pytest.raises(ValueError):
            kv4.recsa_kv4_decode(bad, q)
        with pytest.raises(ValueError):
            kv4.recsa_kv4_decode(q, bad)
    k = torch.zeros(2, 2, 9, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        kv4.recsa_kv4_build(k, k, [10, 4])               # more rows than given
    with pytest.raises(ValueError):
        kv4.recsa_kv4_build(k, k.transpose(0, 1).contiguous().transpose(0, 1), [9, 4])
    with pytest.raises(R.RecsaError):
        kv4.recsa_kv4_build(k, k, [-1, 4])
    with pytest.raises(ValueError):
        kv4.recsa_kv4_append(k, k, torch.tensor([1, 1], device="cuda"))      # int64 counts
    for flat in (k[0], k[0, 0, 0]):
        with pytest.raises(ValueError):
            kv4.recsa_kv4_append(flat, flat)
        with pytest.raises(ValueError):
            kv4.recsa_kv4_prefill_chunk(flat, flat.clone())
    with pytest.raises(R.RecsaError):
        kv4.recsa_kv4_append(k[:, :, :0], k[:, :, :0])   # no rows
    with pytest.raises(R.RecsaError):
        kv4.read(15, 6)                                  # past the capacity
    with pytest.raises(R.RecsaError):
        kv4.recsa_kv4_prefill_chunk(q[:, None], q[:, None].clone(), accumulate_rows=-1)
