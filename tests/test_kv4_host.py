"""The 4-bit KV cache without a GPU: the oracle against closed forms, sizes, and every
refusal that is made on the host before anything touches the device."""
import ctypes

import numpy as np
import pytest

from oracle import kv4_oracle as O


@pytest.fixture(scope="module")
def R():
    from long_context_recsa_b200 import build
    build.build()
    import long_context_recsa_b200.recsa as R
    return R


def cfg_of(R, **kw):
    return R.Config(**{**dict(head_dim=64, n_q_heads=4, n_kv_heads=2, dtype="bf16"), **kw})


# --- the oracle ------------------------------------------------------------------------
def test_oracle_whole_steps_are_exact():
    x = np.arange(32.0)[None] % 16 * 0.25 - 1.5         # lo = -1.5, s = 0.25, all on the grid
    codes, s, lo = O.quantize(x)
    assert lo[0, 0] == -1.5 and s[0, 0] == 0.25
    assert np.array_equal(codes[0, 0], np.arange(32) % 16)
    assert np.array_equal(O.value(x), x)


def test_oracle_constant_and_bad_groups():
    x = np.full((1, 64), 3.0)
    assert np.array_equal(O.value(x), x)                # s = 0
    x[0, 40] = np.inf
    y = O.value(x)
    assert np.array_equal(y[0, :32], x[0, :32]) and np.isnan(y[0, 32:]).all()


def test_oracle_rounds_offset_down_and_step_up():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 128)) * np.exp(rng.standard_normal((200, 1)) * 3)
    codes, s, lo = O.quantize(x)
    g = x.reshape(200, 4, 32)
    assert (lo <= g.min(-1)).all() and (lo + 15 * s >= g.max(-1)).all()
    # the error of a value is at most half a step
    assert (np.abs(O.value(x).reshape(g.shape) - g) <= 0.5 * s[..., None] * (1 + 1e-12)).all()
    # both are bf16: 8 significant bits
    for y in (s, lo):
        m, _ = np.frexp(y)
        assert np.array_equal(m * 256, np.rint(m * 256))


def test_oracle_evict_order():
    u = O.Unit(64)
    u.append(np.zeros((8, 64)), np.zeros((8, 64)))
    u.w = np.array([0.0, 5, 1, 1, 9, np.nan, 1, 0])
    u.evict(5, 1, 1)                                    # 0 and 7 are safe; 4, 1, then tie 2 of {2, 3, 6}
    # free slot 3 takes slot 7 (the only kept one past the budget)
    assert u.pos.tolist() == [0, 1, 2, 7, 4]


# --- sizes and refusals ------------------------------------------------------------------
def test_sizes(R):
    cb, wb = R.recsa_kv4_query_sizes(cfg_of(R, head_dim=128, n_q_heads=32, n_kv_heads=8), 524288, 4, 4)
    assert cb == 4 * 8 * 524288 * (160 + 8)             # 5/8 of bf16's 256 a row, and two words
    one, _ = R.recsa_kv4_query_sizes(cfg_of(R), 1, 1, 1)
    assert one == 2 * 128 * (2 * 32 + 2 * 8 + 8)        # rows go by 128


@pytest.mark.parametrize("kw,cap,B,Q,want", [
    (dict(head_dim=96), 10, 1, 1, 2), (dict(head_dim=256), 10, 1, 1, 2),
    (dict(n_q_heads=6), 10, 1, 1, 2), (dict(n_q_heads=32, n_kv_heads=2), 10, 1, 1, 2),
    (dict(n_q_heads=5), 10, 1, 1, 1), (dict(n_kv_heads=0), 10, 1, 1, 1),
    (dict(scale=-1.0), 10, 1, 1, 1), (dict(scale=float("nan")), 10, 1, 1, 1),
    (dict(), 0, 1, 1, 1), (dict(), 10, 0, 1, 1), (dict(), 10, 65, 65, 1), (dict(), 10, 4, 3, 1),
    (dict(), (1 << 30) + 1, 1, 1, 2), (dict(n_q_heads=8192, n_kv_heads=8192), 10, 8, 8, 2),
])
def test_sizes_refuse(R, kw, cap, B, Q, want):
    with pytest.raises(R.RecsaError) as e:
        R.recsa_kv4_query_sizes(cfg_of(R, **kw), cap, B, Q)
    assert e.value.status == want


def test_init_refuses_before_any_cuda_call(R):
    lib, c = R.lib, cfg_of(R).to_c()
    cb, wb = R.recsa_kv4_query_sizes(cfg_of(R), 100, 1, 1)
    h = ctypes.c_void_p()
    fake, off = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 16)
    for cache, ws, n, m, want in [(None, fake, cb, wb, R.RECSA_E_INVAL), (fake, None, cb, wb, R.RECSA_E_INVAL),
                                  (off, fake, cb, wb, R.RECSA_E_INVAL), (fake, off, cb, wb, R.RECSA_E_INVAL),
                                  (fake, fake, cb - 1, wb, R.RECSA_E_CAPACITY),
                                  (fake, fake, cb, wb - 1, R.RECSA_E_CAPACITY)]:
        assert lib.recsa_kv4_init(ctypes.byref(c), 100, 1, 1, cache, n, ws, m, None,
                                  ctypes.byref(h)) == want
        assert not h.value
    assert lib.recsa_kv4_init(ctypes.byref(c), 100, 1, 1, fake, cb, fake, wb, None, None) == R.RECSA_E_INVAL


def test_null_handles_refuse(R):
    lib = R.lib
    for name, args in [("recsa_kv4_build", (None,) * 6), ("recsa_kv4_append", (None, None, None, 1, None, None)),
                       ("recsa_kv4_decode", (None, None, None, 0, None)),
                       ("recsa_kv4_prefill_chunk", (None, None, 1, None, None, 0, None)),
                       ("recsa_kv4_evict", (None, 1, 0, 0, None)),
                       ("recsa_kv4_read", (None, 0, 1, None, None, None)),
                       ("recsa_kv4_get_status", (None, None)), ("recsa_kv4_info", (None, None)),
                       ("recsa_kv4_free", (None,))]:
        assert getattr(lib, name)(*args) == R.RECSA_E_INVAL, name


def test_a_handle_that_outlives_the_module_is_dropped_quietly(R, monkeypatch):
    """At the interpreter's end a module's names may be None before the last handle goes."""
    kv4 = R.RecsaKV4.__new__(R.RecsaKV4)
    kv4.handle = ctypes.c_void_p(1)
    monkeypatch.setattr(R, "lib", None)
    kv4.__del__()
    kv4.handle = None
