"""V of any size over an fp8 cache for calls of up to four tokens (the decode kernel's several-token form, one, two and
two times two n-tiles of query rows), as the calls of more tokens have it: scales of 2^-60 .. 2^60, tokens
of very different size in one page, rows of zeros. Against the fp64 oracle, with the bar of the tcgen05 route's
tests (P times the scale's mantissa is rounded once to fp16 here, V not at all, so it has room)."""
import numpy as np
import pytest

from test_gpu_fp8_zero_rows import check, scaled, set_rows
from test_oracle_multi import Multi

pytestmark = pytest.mark.gpu

# (Hq, Hkv, T): 8, 16 and 32 query rows per KV head, and one row
FORMS = [(16, 2, 1), (4, 2, 4), (16, 2, 2), (16, 2, 4), (3, 3, 1), (32, 2, 2)]


def case(seed, Hq, Hkv, T):
    lens = [16, 40, 290, T, 0]
    return Multi(seed, Hq, Hkv, lens, [min(L, T - b % 2 if T > 1 else 1) for b, L in enumerate(lens)], T)


@pytest.mark.parametrize("Hq,Hkv,T", FORMS)
@pytest.mark.parametrize("power", [-50, -30, -20, -12, 0, 9, 14, 30, 55])
def test_values_far_from_one(Hq, Hkv, T, power):
    m = case(2500 + T + Hq, Hq, Hkv, T)
    m.c.hist_v[...] = scaled(m.c.hist_v, power)
    m.v_new[...] = scaled(m.v_new, power)
    check(m)
    check(m, window=19, sinks=False)


@pytest.mark.parametrize("Hq,Hkv,T", FORMS)
def test_tokens_of_every_size_side_by_side(Hq, Hkv, T):
    """The V rows of a sequence span 2^-40 .. 2^40."""
    m = case(2600 + T + Hq, Hq, Hkv, T)
    rng = np.random.default_rng(T)
    for b in range(m.c.B):
        for p in range(int(m.lens[b])):
            row = m.c.hist_v[b, p] if p < m.base[b] else m.v_new[b, p - m.base[b]]
            row[...] = scaled(row, int(rng.integers(-40, 41)))
    check(m)
    check(m, sinks=False)


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (16, 2)])
def test_a_later_token_far_larger_than_those_before(Hq, Hkv):
    """The last new token's V is 2^40 times the others': rows before it do not attend it, and keep their digits."""
    m = Multi(2700 + Hq, Hq, Hkv, [9, 60], [4, 4], 4)
    m.v_new[:, 3] = scaled(m.v_new[:, 3], 40)
    check(m)


@pytest.mark.parametrize("Hq,Hkv,T", FORMS)
@pytest.mark.parametrize("power", [-12, -24, 12])
def test_zero_values_beside_others(Hq, Hkv, T, power):
    m = case(2800 + T + Hq, Hq, Hkv, T)
    m.c.hist_v[...] = scaled(m.c.hist_v, power)
    m.v_new[...] = scaled(m.v_new, power)
    set_rows(m, "v", lambda b: range(3 + b, 300, 5), 0)
    set_rows(m, "v", lambda b: range(128, 176), 0x8000)
    set_rows(m, "k", lambda b: range(6 + b, 300, 9), 0)
    check(m)
    check(m, window=33, sinks=False)


@pytest.mark.parametrize("Hq,Hkv,T", FORMS)
def test_rows_of_scale_one_that_are_not_zeros(Hq, Hkv, T):
    m = case(2900 + T + Hq, Hq, Hkv, T)
    for x in (m.c.hist_v, m.v_new):
        x[..., 17] = 0x43E0                                     # 448: scale 1, the other elements' codes often 0
    set_rows(m, "v", lambda b: range(2 + b, 300, 7), 0)
    check(m)


@pytest.mark.parametrize("Hq,Hkv,T", FORMS)
def test_only_zeros(Hq, Hkv, T):
    m = case(2950 + T + Hq, Hq, Hkv, T)
    set_rows(m, "v", lambda b: range(0, 300), 0)
    check(m)
    check(m, sinks=False)


def test_split_sequences_of_very_small_and_large_values():
    """Partials of many warps and CTAs, whose maxima and denominators lie 2^80 apart."""
    m = Multi(2990, 16, 2, [6000, 20], [4, 4], 4)
    m.c.hist_v[:, :2000] = scaled(m.c.hist_v[:, :2000], -40)
    m.c.hist_v[:, 4000:] = scaled(m.c.hist_v[:, 4000:], 40)
    set_rows(m, "v", lambda b: range(2500, 3500), 0)
    check(m)
    check(m, sinks=False)
    check(m, window=3000)


@pytest.mark.parametrize("T", [1, 4, 16, 150])
@pytest.mark.parametrize("power", [-50, 66])
@pytest.mark.parametrize("zeros", [False, True])
def test_the_ends_of_the_range_on_both_routes(T, power, zeros):
    """Scales of about 2^-59 to 2^-57, and up to 2^60."""
    m = Multi(5000 + T, 16, 2, [T, T + 40, T + 700], [T] * 3, T)
    m.c.hist_v[...] = scaled(m.c.hist_v, power)
    m.v_new[...] = scaled(m.v_new, power)
    if zeros:
        set_rows(m, "v", lambda b: range(3, 900, 5), 0)
        set_rows(m, "v", lambda b: range(32, 96), 0)
    check(m)
    check(m, window=50, sinks=False)
