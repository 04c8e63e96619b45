"""Accumulated weights of the 4-bit KV cache where units share CTAs, and where the softmax
sums of a chunk's own kernel are inexact.

Tolerances, from the arithmetic.  Weights come from scores and sums of one and the same
evaluation (a first launch forms maxima and sums, a second the probabilities), so a unit's
weights add up to the number of rows that count times the group's heads whatever the
scores' own error: exp2 2^-22 relative twice and at most a hundred roundings of 2^-24 (the
additions of a lane over its tokens and over the blocks of rows), together below 2^-17.  Against the oracle a probability is also off by twice the
score's error: 16 * 2^-24 * S with S = scale * sum |q| * 2 max |K| (bound_of() of the tests
beside this file, without its term for keys rounded to fp16: the weights' scores are formed
from the codes)."""
import numpy as np
import pytest
import torch

from oracle import kv4_oracle as O
from tests import test_gpu_kv4 as T

pytestmark = pytest.mark.gpu
R = T.R                                                  # the fixture

SUM = 2.0 ** -17


def accumulate(units, Q, G, n, counts, lengths, acc):
    """The oracle's weights of a chunk's newest rows."""
    for b, row in enumerate(units):
        m = n if counts is None else counts[b]
        for i in range(max(0, m - acc), m):
            for h, u in enumerate(row):
                u.attend(T.np64(Q[b, i, h * G:(h + 1) * G]), lengths[b] - m + i, accumulate=True)


def check(kv4, units, Q, G, n, counts, acc, skip=()):
    w = T.np64(kv4.weights())
    for b, row in enumerate(units):
        m = n if counts is None else counts[b]
        for h, u in enumerate(row):
            if (b, h) in skip:
                continue
            got = w[b, h, :len(u.w)]
            rows = min(acc, m) * G
            assert abs(got.sum() - rows) <= SUM * rows, (b, h, got.sum(), rows)
            if rows == 0:
                continue
            qs = T.np64(Q[b, m - min(acc, m):m, h * G:(h + 1) * G]).reshape(-1, Q.shape[-1])
            delta = T.bound_of(u, qs, "bf16")[0]
            err = np.abs(got - u.w)
            assert (err <= (2 * delta + SUM) * np.abs(u.w) + 1e-30).all(), (b, h, (err / u.w).max())


# (lengths, KV heads, heads a group, d, rows, counts, rows that count): several units begin in
# one CTA of the weights' launches, the last of them often cut by the next CTA
SHARED = [
    ([70] * 4, 8, 4, 128, 4, None, 4), ([90] * 2, 2, 4, 128, 3, None, 3), ([40] * 1, 8, 4, 64, 4, None, 4),
    ([33, 64, 65, 96, 40], 3, 8, 64, 5, [5, 1, 0, 4, 2], 2), ([150] * 64, 16, 2, 64, 5, None, 5),
    ([2000, 60, 60, 70], 2, 4, 128, 8, None, 8), ([300, 10, 500, 9, 9, 31], 4, 1, 128, 9, None, 3),
    ([70, 70], 2, 8, 64, 40, [40, 17], 24)]


@pytest.mark.parametrize("lengths,Hkv,G,d,n,counts,acc", SHARED)
def test_weights_of_units_that_share_a_cta(R, lengths, Hkv, G, d, n, counts, acc):
    B = len(lengths)
    kv4, units = T.make(R, "bf16", d, Hkv, G, lengths, seed=11, max_queries=B * n)
    Q = T.rand((B, n, G * Hkv, d), 41, "bf16", 2.0)
    c = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    kv4.prefill(Q.cuda(), c, accumulate_rows=acc)
    accumulate(units, Q, G, n, counts, lengths, acc)
    check(kv4, units, Q, G, n, counts, acc)
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK


@pytest.mark.parametrize("Hkv,L,G,n", [(8, 40, 4, 4), (8, 70, 2, 6)])
def test_a_nan_key_reaches_its_own_unit_only(R, Hkv, L, G, n):
    d, bad = 128, 3
    k, v = T.keys((1, Hkv, L, d), 1, "bf16"), T.rand((1, Hkv, L, d), 2, "bf16")
    k[0, bad, 5, 40] = float("nan")
    cfg = R.Config(head_dim=d, n_q_heads=G * Hkv, n_kv_heads=Hkv, dtype="bf16")
    kv4 = R.RecsaKV4(cfg, L, 1, max_queries=n)
    kv4.recsa_kv4_build(k.cuda(), v.cuda(), [L])
    Q = T.rand((1, n, G * Hkv, d), 3, "bf16")
    kv4.prefill(Q.cuda(), accumulate_rows=n)
    units = [[O.Unit(d) for _ in range(Hkv)]]
    for h, u in enumerate(units[0]):
        u.append(T.np64(k[0, h]), T.np64(v[0, h]))
    k2 = [u for h, u in enumerate(units[0]) if h != bad]
    accumulate([k2], torch.cat([Q[:, :, h * G:(h + 1) * G] for h in range(Hkv) if h != bad], 2), G, n, None, [L], n)
    check(kv4, units, Q, G, n, None, n, skip={(0, bad)})
    assert torch.isnan(kv4.weights()[0, bad, 5])


@pytest.mark.parametrize("dtype,d,G,n,acc,mq", [
    ("bf16", 128, 4, 40, 40, None), ("bf16", 64, 2, 300, 200, None), ("bf16", 128, 4, 2, 2, None), ("f32", 64, 4, 20, 9, None),
    ("bf16", 128, 1, 33, 33, 22)])
@pytest.mark.parametrize("big", [1.0, 30.0, 2.0 ** 20])
def test_weights_add_up_whatever_the_scores(R, dtype, d, G, n, acc, mq, big):
    """Scores of tens, thousands and 2^30: a unit's weights add up all the same, in a chunk and
    after a decode, over units that are cut and units that are not."""
    lengths, Hkv = [700, 130], 2
    n = min(n, 130)
    acc = min(acc, n)
    kv4, units = T.make(R, dtype, d, Hkv, G, lengths, seed=21, max_queries=mq or 2 * n)
    Q = T.rand((2, n, G * Hkv, d), 51, dtype, 4.0 * big)
    kv4.prefill(Q.cuda(), accumulate_rows=acc)
    rows = acc * G
    for step in range(2):
        w = T.np64(kv4.weights())
        assert np.isfinite(w).all() and (w >= 0).all()
        assert (np.abs(w.sum(-1) - rows) <= SUM * rows).all(), (step, w.sum(-1), rows)
        if step == 0:
            kv4.decode(Q[:, 0].contiguous().cuda(), accumulate=True)
            rows += G
    assert kv4.recsa_kv4_get_status() == R.RECSA_OK


@pytest.mark.parametrize("dtype,d,G", [("bf16", 128, 4), ("f32", 64, 8), ("bf16", 64, 8)])
def test_weights_of_a_chunk_over_an_evicted_cache(R, dtype, d, G):
    """Slots out of order, units of a few tiles: weights after eviction and a chunk."""
    B, Hkv, L, n = 3, 2, 150, 16
    kv4, units = T.make(R, dtype, d, Hkv, G, [L, 120, 96], seed=31, max_queries=B * n)
    T.set_weights(kv4, units, 6)
    kv4.recsa_kv4_evict(90, 3, 20)
    for row in units:
        for u in row:
            u.evict(90, 3, 20)
    T.check_evicted(kv4, units, dtype)
    kv4.weights().zero_()
    Q = T.rand((B, n, G * Hkv, d), 61, dtype)
    kv4.prefill(Q.cuda(), accumulate_rows=3)
    for b, row in enumerate(units):
        for h, u in enumerate(row):
            u.w[:] = 0
            for i in range(n - 3, n):
                u.attend(T.np64(Q[b, i, h * G:(h + 1) * G]), u.seen - n + i, accumulate=True)
    check(kv4, units, Q, G, n, None, 3)
