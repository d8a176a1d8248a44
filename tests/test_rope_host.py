"""The rotary table (CPU): phase steps against their formulas in exact and decimal
arithmetic, and the refusals of oscar_rope and RotaryEmbedding, none of which reach a GPU."""
import ctypes
import decimal
import math

import pytest

from int2_rotated_kv_rotate_gb300 import _native as N
from int2_rotated_kv_rotate_gb300 import build, rotary

DEC = decimal.Context(prec=50)
TWO_PI = decimal.Decimal("6.28318530717958647692528676655900576839433879875021164194989")


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def config(**kw):
    base = dict(rotary_dim=128, scaling=N.OSCAR_ROPE_UNSCALED, base=1e6, factor=1.0, low=1.0, high=4.0,
                original_context=32768.0)
    base.update(kw)
    return N.oscar_rope_config(*[base[f] for f, _ in N.oscar_rope_config._fields_])


def frequency(base, R, i):
    return DEC.power(DEC.create_decimal(base), DEC.divide(DEC.create_decimal(-2 * i), DEC.create_decimal(R)))


def expected(cfg):
    """Turns a position of every pair, in 50 digits."""
    R, D = cfg.rotary_dim, decimal.Decimal
    out = []
    for i in range(R // 2):
        f = frequency(cfg.base, R, i)
        keep = D(1)
        if cfg.scaling == N.OSCAR_ROPE_LINEAR:
            keep = D(0)
        elif cfg.scaling == N.OSCAR_ROPE_BANDS:
            n = DEC.divide(DEC.multiply(D(cfg.original_context), f), TWO_PI)
            keep = min(max(DEC.divide(n - D(cfg.low), D(cfg.high) - D(cfg.low)), D(0)), D(1))
        elif cfg.scaling == N.OSCAR_ROPE_YARN:
            x = [R * math.log(cfg.original_context / (2 * math.pi * n)) / (2 * math.log(cfg.base))
                 for n in (cfg.high, cfg.low)]
            a = min(max(math.floor(x[0]), 0), R - 1)
            b = min(max(math.ceil(x[1]), 0), R - 1)
            keep = 1 - min(max(DEC.divide(D(i - a), D(max(b - a, 0.001))), D(0)), D(1))
        if cfg.scaling != N.OSCAR_ROPE_UNSCALED:
            f = DEC.divide(f, D(cfg.factor)) * (1 - keep) + f * keep
        out.append(DEC.divide(f, TWO_PI) % 1)
    return out


@pytest.mark.parametrize("kw", [
    dict(), dict(base=10000.0, rotary_dim=64), dict(rotary_dim=2), dict(rotary_dim=18, base=500000.0),
    dict(rotary_dim=512), dict(scaling=N.OSCAR_ROPE_LINEAR, factor=8.0), dict(scaling=N.OSCAR_ROPE_LINEAR, factor=0.03),
    dict(scaling=N.OSCAR_ROPE_BANDS, factor=8.0), dict(scaling=N.OSCAR_ROPE_BANDS, factor=2.0, base=10000.0, low=2.0),
    dict(scaling=N.OSCAR_ROPE_YARN, factor=4.0, high=32.0), dict(scaling=N.OSCAR_ROPE_YARN, factor=1.0, high=32.0),
    dict(scaling=N.OSCAR_ROPE_YARN, factor=16.0, high=32.0, original_context=16.0)])
def test_steps_follow_the_formula(kw):
    cfg = config(**kw)
    steps, magnitude = N.oscar_rope_steps(cfg)
    # a handful of fp64 operations, each within 2^-53 of its value (pow within 2^-52): under
    # 16 * 2^-53 of the unreduced turns, plus one unit of the fixed point
    for got, want in zip(steps, expected(cfg)):
        turns = float(want) if cfg.factor >= 1 else float(want) + 1.0 / (cfg.factor * 2 * math.pi)
        err = abs(decimal.Decimal(got) / (1 << 64) - want)
        err = min(err, 1 - err)
        assert err <= decimal.Decimal(turns * 2.0**-49 + 2.0**-64)
    if cfg.scaling == N.OSCAR_ROPE_YARN:
        assert abs(magnitude - (0.1 * math.log(cfg.factor) + 1.0)) <= 2.0**-24 * magnitude
    else:
        assert magnitude == 1.0


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=-2), dict(rotary_dim=514), dict(base=1.0), dict(base=0.5),
    dict(base=math.inf), dict(base=math.nan), dict(scaling=4), dict(scaling=-1),
    dict(scaling=N.OSCAR_ROPE_LINEAR, factor=0.0), dict(scaling=N.OSCAR_ROPE_LINEAR, factor=math.nan),
    dict(scaling=N.OSCAR_ROPE_YARN, factor=0.5), dict(scaling=N.OSCAR_ROPE_BANDS, low=4.0, high=4.0),
    dict(scaling=N.OSCAR_ROPE_BANDS, low=0.0), dict(scaling=N.OSCAR_ROPE_YARN, original_context=0.0),
    dict(scaling=N.OSCAR_ROPE_YARN, high=math.inf)])
def test_bad_configurations_are_refused(kw):
    cfg = config(**kw)
    steps = (ctypes.c_uint64 * 1024)()
    m = ctypes.c_float()
    assert N.lib().oscar_rope_steps(ctypes.byref(cfg), steps, ctypes.byref(m)) == 1
    assert N.lib().oscar_last_error()


def call(n=1, rows=4, head_dim=128, rotary_dim=128, dtype=0, flags=0, steps=0x1000, positions=0x2000, **kw):
    t = dict(in_=0x10000, out=0x90000, n_heads=8, in_row=1024, in_head=128, out_row=1024, out_head=128)
    t.update(kw)
    arr = (N.oscar_rope_tensor * 2)(*[N.oscar_rope_tensor(*[t[f] for f, _ in N.oscar_rope_tensor._fields_])] * 2)
    return N.lib().oscar_rope(arr, n, steps, head_dim, rotary_dim, 1.0, dtype, flags, positions, rows, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), 1), (dict(n=3), 1), (dict(rotary_dim=130), 1), (dict(rotary_dim=5), 1), (dict(head_dim=514), 1),
    (dict(dtype=3), 2), (dict(flags=8), 1), (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(n_heads=0), 1),
    (dict(in_=None), 1), (dict(out=None), 1), (dict(out_row=1000), 1), (dict(out_head=64), 1), (dict(in_row=-1024), 1),
    (dict(out=0x10000, out_row=2048), 1), (dict(in_=0x10001), 1), (dict(dtype=2, out=0x90002), 1),
    (dict(steps=None), 1), (dict(steps=0x1004), 1), (dict(positions=None), 1),
    (dict(flags=N.OSCAR_ROPE_POSITIONS64, positions=0x2004), 1)])
def test_bad_calls_are_refused_before_the_gpu(kw, status):
    assert call(**kw) == status
    assert N.lib().oscar_last_error() and N.oscar_last_launch_count() == 0


def test_no_rows_launch_nothing():
    assert call(rows=0, in_=None, out=None, steps=None, positions=None) == 0
    assert N.oscar_last_launch_count() == 0


def test_constructor_refusals():
    for kw in (dict(head_dim=64, rotary_dim=128), dict(rotary_dim=0), dict(head_dim=1024),
               dict(scaling=dict(type="dynamic", factor=2.0)), dict(scaling=dict(factor=2.0)),
               dict(scaling=dict(type="linear", factor=2.0, slope=1.0))):
        with pytest.raises(ValueError):
            rotary.RotaryEmbedding(device="cpu", **kw)
    with pytest.raises(N.OscarError):
        rotary.RotaryEmbedding(device="cpu", rotary_dim=7)
    with pytest.raises(N.OscarError):
        rotary.RotaryEmbedding(device="cpu", scaling=dict(type="yarn", factor=4.0))  # no original_context
