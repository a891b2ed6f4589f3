"""decode_attn_paged_tree_int8 over the whole range of its inputs: queries of any size, rows and elements of very
different sizes beside each other.

Bound on the fp32 output, u = 2^-24; as tests/tree_int8_reference.py, a relative error e_j of weight j moves the output by
at most sum_j p_j |V_j| e_j + |out| sum_j p_j e_j, with this term besides:
  - a query row is taken by a power of two to a largest element of at least 2^-4 and rounded to fp16, whose smallest
    step is 2^-24: an element is off by at most half of that, 2^-25 / 2^-4 = 8 u of the row's largest, and the score by
    8 u max |q| scale sum_d |K_jd|.
"""
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
                e += 4 * U * (np.abs(x) + abs(x.max())) + 9 * U + 2.0 ** -21
                e += 2 * (128 + T / 128 + 64) * U
                p = np.exp(x - x.max())
                p /= p.sum()
                o = p @ v
                out[b, i, h] = o
                bound[b, i, h] = ((p * e) @ np.abs(v) + np.abs(o) * (p @ e) +
                                  T * 2.0 ** -28 * 127 * size.max())
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
