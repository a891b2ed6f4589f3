"""decode_attn_paged_tree_int8 over the whole range of its inputs: queries of any size, rows and elements of very
different sizes beside each other, V scales of keys that other rows see or that hardly weigh anything.

Bound on the fp32 output, u = 2^-24; as tests/tree_int8_reference.py, a relative error e_j of weight j moves the output by
at most sum_j p_j |V_j| e_j + |out| sum_j p_j e_j, with these terms besides or in another form:
  - a query row is taken by a power of two to a largest element of at least 2^-4 and rounded to fp16, whose smallest
    step is 2^-24: an element is off by at most half of that, 2^-25 / 2^-4 = 8 u of the row's largest, and the score by
    8 u max |q| scale sum_d |K_jd|;
  - a row's exponentials are taken relative to a reference r at which its largest contribution p_j vs_j lies in [2^6, 2^15),
    V scales (in units F, a power of two) below 2^-80 counting as that: |x - r| in base 2 is at most the distance
    from the row's maximum plus 15 + L, L = max(|log2 vs F|, 80 for a scale of 0) <= 84. Arguments and joins round there
    twice each: 4 u (15 + L), with L from the keys that the row sees, relative to the prefix's largest scale, which F
    brings to [8, 16);
  - a key's weight times its V scale is an fp16 pair hi + lo with an absolute step of 2^-24, half of it lost, beside a
    largest contribution of at least 2^6: 2^-31 127 max_j p_j |vs_j| a key that the row sees, whatever others see.
"""
import math

import numpy as np
import pytest

import paged_gqa_decode_head_gb300 as pg
import tree_int8_reference as ref
import tree_reference as bf16_ref
from paged_gqa_decode_head_gb300 import inputs
from test_gpu_tree_int8 import SCALE, Case
from tree_reference import U

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_flags():
    pg.device_error_flags(clear=True)
    yield
    assert pg.device_error_flags() == 0


def reference(c):
    """(out, bound) [B, M, Hq, 128] float64; rows i >= n_b, and those with a query that is no number, stay NaN."""
    out, bound = np.full(c.q.shape, np.nan), np.full(c.q.shape, np.nan)
    g = c.Hq // c.Hkv
    for b in range(c.B):
        T, n = int(c.lens[b]), c.n[b]
        prefix = T - n
        ks, vs = (ref.rows_of(x, c.table[b], T, c.P).astype(np.float64) for x in (c.ks, c.vs))
        K, V = (ref.rows_of(x, c.table[b], T, c.P).astype(np.float64) for x in (c.k8, c.v8))
        kpos = np.concatenate([np.arange(prefix), c.positions[b][:n]]).astype(np.float64)
        for i in range(n):
            seen = np.nonzero([j < prefix or int(c.masks[b][i]) >> (j - prefix) & 1 for j in range(T)])[0]
            for h in range(c.Hq):
                kv, qv = h // g, bf16_ref.widen(c.q[b, i, h])
                if not np.isfinite(qv).all():
                    continue
                size = np.abs(vs[kv, seen])
                k, v = K[kv, seen] * ks[kv, seen, None], V[kv, seen] * vs[kv, seen, None]
                x = c.scale * (k @ qv)
                e = abs(c.scale) * U * (256 * (np.abs(k) @ np.abs(qv)) + 8 * np.abs(qv).max() * np.abs(k).sum(1))
                e += 4 * U * np.abs(x)
                if c.softcap > 0:
                    x = c.softcap * np.tanh(x / c.softcap)
                    e += 8 * U * np.abs(x)
                if c.slopes is not None:
                    sl = float(c.slopes[h])
                    bias = sl * (kpos[seen] - (kpos[seen].min() if sl < 0 else kpos[seen].max()))
                    e += 2 * U * (np.abs(bias) + abs(sl) * 64 + np.abs(x))
                    x = x + bias
                unit = np.abs(vs[kv, :prefix]).max(initial=0.0) or 8.0
                spread = max(min(84.0, abs(math.log2(s / unit))) if s > 0 else 84.0 for s in size)
                e += 4 * U * (np.abs(x) + abs(x.max())) + 9 * U + 2.0 ** -21 + 4 * U * (15 + spread)
                e += 2 * (128 + T / 128 + 64) * U
                p = np.exp(x - x.max())
                p /= p.sum()
                o = p @ v
                out[b, i, h] = o
                bound[b, i, h] = ((p * e) @ np.abs(v) + np.abs(o) * (p @ e) +
                                  len(seen) * 2.0 ** -31 * 127 * (p * size).max())
    return out, bound


def check(c):
    of, ob = c.run()
    out, bound = reference(c)
    known = np.isfinite(out)
    assert np.isfinite(of[known]).all()
    over = np.abs(of - out)[known] - (bound + 2.0 ** -24 * np.abs(out))[known]
    assert (over <= 0).all(), (float(over.max()), float(np.nanmax(np.abs(of - out))))
    over = np.abs(ob - out)[known] - (bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(out))[known]
    assert (over <= 0).all(), float(over.max())
    return of


def scaled(bits, factor):
    return inputs.f32_to_bf16_bits((bf16_ref.widen(bits) * factor).astype(np.float32))


SLOPES = [-0.25, 0.5, 0.01, -1.0, 0.0, 2.0, 0.125, 0.3]
# rows per KV head: 6, 12, 24, 56 and 128 (two groups of rows)
SHAPES = [(3, 2), (12, 1), (12, 2), (28, 2), (64, 2)]


# ------------------------------------------------------------------ queries
@pytest.mark.parametrize("power", [-126, -100, -40, -24, -20, -16, -8, 4, 12, 40, 100, 124])
@pytest.mark.parametrize("M,g", SHAPES)
def test_queries_of_any_size(power, M, g):
    """Queries 2^power times as large and scores 2^-power times: the same attention."""
    c = Case(3000 + M, [300, M + 3], M, Hq=2 * g, Hkv=2)
    c.q, c.scale = scaled(c.q, 2.0 ** power), SCALE * 2.0 ** -power
    check(c)


@pytest.mark.parametrize("power,scale_power", [(13, 116), (13, 97), (60, 66), (-100, -20), (-60, -58), (-126, 10)])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("M,g", [(3, 2), (12, 2), (64, 2)])
def test_queries_and_scales_at_the_ends_of_their_range(power, scale_power, softcap, M, g):
    """The score is of usual size, products of two of its three factors are not; a key without a K row among them."""
    c = Case(3050 + M, [300, M + 3], M, Hq=2 * g, Hkv=2, softcap=softcap)
    c.q, c.scale = scaled(c.q, 2.0 ** power), SCALE * 2.0 ** scale_power
    c.ks = np.float32(c.ks.astype(np.float64) * 2.0 ** -(power + scale_power))
    c.k8[at(c, 0, 5)], c.ks[at(c, 0, 5)] = 0, 0
    check(c)


@pytest.mark.parametrize("power", [-60, -20, 20])
@pytest.mark.parametrize("softcap,biased", [(20.0, False), (0.0, True), (20.0, True)])
@pytest.mark.parametrize("M,g", [(3, 2), (12, 2), (64, 2)])
def test_queries_of_any_size_capped_and_biased(power, softcap, biased, M, g):
    c = Case(3100 + M, [300, M + 3], M, Hq=2 * g, Hkv=2, softcap=softcap, slopes=SLOPES[:2 * g] if biased else None)
    c.q, c.scale = scaled(c.q, 2.0 ** power), SCALE * 2.0 ** -power
    check(c)


@pytest.mark.parametrize("softcap,biased", [(0.0, False), (20.0, False), (0.0, True), (20.0, True)])
@pytest.mark.parametrize("M,g", SHAPES)
def test_rows_of_very_different_sizes(M, g, softcap, biased):
    """Heads and tokens whose queries differ by up to 2^48 in one call; the smallest decide nothing, the largest all."""
    c = Case(3200 + M, [300, M + 3], M, Hq=2 * g, Hkv=2, softcap=softcap, slopes=SLOPES[:2 * g] if biased else None)
    gen = np.random.default_rng(M + g)
    c.q = scaled(c.q, 2.0 ** gen.choice([-24.0, 0.0, 3.0, 24.0], (c.B, M, 2 * g, 1)))
    check(c)
    c.q[0, 0], c.scale = 0, SCALE * 2.0 ** 24  # a row of zeros among them
    check(c)


@pytest.mark.parametrize("softcap,biased", [(0.0, False), (20.0, True)])
@pytest.mark.parametrize("M,g", [(8, 2), (33, 2)])
def test_rows_of_very_different_sizes_over_long_runs(M, g, softcap, biased):
    """The same with many tiles and segments in every CTA, some segments' rows alike."""
    c = Case(3250 + M, [9000, 300, 12000, 40], M, Hq=4 * g, Hkv=4, softcap=softcap, slopes=SLOPES[:4 * g] if biased else None)
    gen = np.random.default_rng(M + g)
    c.q[1:] = scaled(c.q[1:], 2.0 ** gen.choice([-20.0, 0.0, 20.0], (3, M, 4 * g, 1)))
    check(c)


@pytest.mark.parametrize("M,g", [(3, 2), (12, 2), (64, 2)])
def test_elements_of_very_different_sizes(M, g):
    """A large element that meets zeros in K: the small ones make the scores."""
    for power in (10, 20, 30):
        c = Case(3300 + M, [300, M + 3], M, Hq=2 * g, Hkv=2)
        c.k8[..., 17] = 0
        x = bf16_ref.widen(c.q)
        x[..., 17] = 2.0 ** power
        c.q = inputs.f32_to_bf16_bits(x.astype(np.float32))
        check(c)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("M,g", [(3, 2), (12, 2), (64, 2)])
def test_a_query_that_is_no_number_stays_alone(bad, M, g):
    c = Case(3400 + M, [300, M + 3], M, Hq=2 * g, Hkv=2)
    x = bf16_ref.widen(c.q)
    x[0, 1, 0, 5], x[1, M - 1, 2 * g - 1, 100] = bad, bad
    c.q = inputs.f32_to_bf16_bits(x.astype(np.float32))
    of = check(c)
    assert np.isnan(of[0, 1, 0]).all() and np.isnan(of[1, M - 1, 2 * g - 1]).all()


# ------------------------------------------------------------------ V scales
def at(c, b, j):
    return c.table[b, j // c.P], slice(None), j % c.P


def blind_masks(M, j):
    """Drafted token j is seen by itself and by odd tokens behind it only."""
    masks = []
    for i in range(M):
        m = (2 << i) - 1
        masks.append(m & ~(1 << j) if i != j and i % 2 == 0 else m)
    return masks


@pytest.mark.parametrize("power", [12, 24, 60, 120])
@pytest.mark.parametrize("M,g", SHAPES)
def test_a_large_value_scale_of_a_key_that_others_see(power, M, g):
    """One drafted token's V scale is 2^power times the others': rows that do not see it keep all of their bits."""
    for T in (M, M + 40, 700):
        c = Case(3500 + M, [T], M, Hq=2 * g, Hkv=2, masks=[blind_masks(M, 1)])
        c.vs[at(c, 0, T - M + 1)] *= np.float32(2.0 ** power)
        check(c)


@pytest.mark.parametrize("M,g", [(3, 2), (12, 2), (64, 2)])
def test_large_value_scales_that_others_see_over_long_runs(M, g):
    """The same with several tiles in every CTA, and V scales of the prefix between 2^-8 and 2^8."""
    c = Case(3550 + M, [5000] * 8, M, Hq=2 * g, Hkv=2, masks=[blind_masks(M, 1)] * 8)
    gen = np.random.default_rng(M)
    for b in range(8):
        for j in range(5000):
            c.vs[at(c, b, j)] *= np.float32(2.0 ** gen.integers(-8, 9))
        c.vs[at(c, b, 5000 - M + 1)] *= np.float32(2.0 ** (10 * b))
    check(c)


@pytest.mark.parametrize("lower", [5.0, 12.0, 25.0, 60.0])
@pytest.mark.parametrize("T", [700, 9000])
def test_a_large_value_scale_of_a_key_that_hardly_weighs(lower, T):
    """A key whose V scale is 2^24 times the others' and whose score lies `lower` (base 2) below all of them."""
    c = Case(3600, [T], 2, Hq=2, Hkv=2)
    c.q[0, 1] = c.q[0, 0]
    c.k8[...] = np.random.default_rng(1).integers(-3, 4, c.k8.shape)
    for h in range(2):
        q = bf16_ref.widen(c.q[0, 0, h])
        c.k8[at(c, 0, 40)[0], h, 40 % c.P] = np.rint(-127 * q / np.abs(q).max())
        x = SCALE * (ref.rows_of(c.k8, c.table[0], T, c.P)[h].astype(np.float64) *
                     ref.rows_of(c.ks, c.table[0], T, c.P)[h, :, None].astype(np.float64)) @ q
        page, off = c.table[0, 40 // c.P], 40 % c.P
        c.ks[page, h, off] *= np.float32((lower * math.log(2) - np.median(x)) / -x[40])
    c.vs[at(c, 0, 40)] *= np.float32(2.0 ** 24)
    check(c)


@pytest.mark.parametrize("weigh", [8.0, 20.0, 30.0])
@pytest.mark.parametrize("value", [0.0, 2.0 ** -40, 2.0 ** -12, 1.0])
@pytest.mark.parametrize("B,M", [(1, 1), (1, 40), (12, 1), (12, 12), (8, 40)])
def test_a_first_key_that_takes_the_weight(weigh, value, B, M):
    """The first key's score lies `weigh` (nats) above the others, its V row is nothing or small: the output is the rest's,
    each with a weight of e^-weigh. In a batch a CTA has many tiles."""
    c = Case(3700, [6000] * B, M, Hq=2, Hkv=2)
    c.q[:, :] = c.q[:, :1]
    for b in range(B):
        page = c.table[b, 0]
        for h in range(2):
            q = bf16_ref.widen(c.q[b, 0, h])
            c.k8[page, h, 0] = np.rint(127 * q / np.abs(q).max())
            c.ks[page, h, 0] = weigh / (SCALE * (c.k8[page, h, 0].astype(np.float64) @ q))
        c.vs[page, :, 0] *= np.float32(value)
    check(c)


@pytest.mark.parametrize("power", [-70, -30, 30, 70])
@pytest.mark.parametrize("M,g", [(3, 2), (12, 2), (64, 2)])
def test_value_scales_of_any_size(power, M, g):
    """All V scales small or large, and those of a drafted token of its own size besides."""
    c = Case(3800 + M, [300, M + 200], M, Hq=2 * g, Hkv=2, masks=[blind_masks(M, 1)] * 2)
    c.vs *= np.float32(2.0 ** power)
    c.vs[at(c, 0, 300 - M + 1)] *= np.float32(2.0 ** 20)
    c.vs[at(c, 1, 200 + 1)] *= np.float32(2.0 ** -20)
    check(c)


@pytest.mark.parametrize("M,g", [(2, 2), (24, 1), (64, 1), (50, 2)])
def test_value_scales_that_grow_past_the_first_unit(M, g):
    """From the last tile, whose keys come first, to the first one V scales grow by 2^110."""
    c = Case(3900, [128 * 6] * 20, M, Hq=8 * g, Hkv=8)
    for b in range(20):
        for j in range(128 * 6):
            c.vs[at(c, b, j)] *= np.float32(2.0 ** (50 - 22 * (j // 128)))
    check(c)


@pytest.mark.parametrize("powers", [(-100, -100), (-60, 60), (100, 100)])
@pytest.mark.parametrize("M,g", [(3, 2), (33, 1), (64, 2)])
def test_rows_that_have_no_key_in_common(M, g, powers):
    """Every drafted token sees itself alone, each with a V scale of its own size: the output is its V row."""
    c = Case(3950, [M], M, Hq=2 * g, Hkv=2, masks=[[1 << i for i in range(M)]])
    for j in range(M):
        c.vs[at(c, 0, j)] *= np.float32(2.0 ** (powers[0] + (powers[1] - powers[0]) * j / M))
    check(c)
