"""CPU checks of drafted-tree decoding: what the entry points refuse before touching the GPU, and the
reference's closed forms. No compute call is made here."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_gqa_decode_head_gb300 as pg
import tree_reference as ref
from paged_gqa_decode_head_gb300 import binding, inputs
from paged_gqa_decode_head_gb300 import build as libbuild

BASE = 0x10000000  # a well aligned address that is never dereferenced
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return binding.load_library()


def attention(lib, **kw):
    a = dict(q=BASE, k=BASE, v=BASE, bt=BASE, ctx=BASE, mask=BASE, pos=BASE, dl=None, slopes=None, B=1, M=8, Hq=16,
             Hkv=8, D=128, P=16, max_pages=4, num_pages=4, scale=0.1, cap=0.0, of=BASE, ob=None, ws=None, wsb=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.decode_attn_paged_tree(a["q"], a["k"], a["v"], a["bt"], a["ctx"], a["mask"], a["pos"], a["dl"],
                                      a["slopes"], a["B"], a["M"], a["Hq"], a["Hkv"], a["D"], a["P"], a["max_pages"],
                                      a["num_pages"], F(a["scale"]), F(a["cap"]), a["of"], a["ob"], a["ws"], a["wsb"],
                                      None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=64), -2), (dict(Hq=12), -2), (dict(Hq=72), -2), (dict(P=8), -2), (dict(P=48), -2), (dict(P=512), -2),
    (dict(B=-1), -1), (dict(B=65536), -2), (dict(M=0), -1), (dict(M=65), -1), (dict(scale=math.nan), -1),
    (dict(scale=math.inf), -1), (dict(cap=-1.0), -1), (dict(cap=math.nan), -1), (dict(cap=math.inf), -1),
    (dict(P=256, max_pages=(1 << 22) + 1), -2), (dict(B=60000, P=256, max_pages=1 << 22), -2),
    (dict(B=65535, M=64, Hq=8192, Hkv=1024), -2), (dict(Hq=70000, Hkv=70000), -2),
    (dict(max_pages=-1), -1), (dict(num_pages=-1), -1), (dict(num_pages=0), -1), (dict(num_pages=2 ** 26), -2),
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(bt=None), -1), (dict(ctx=None), -1),
    (dict(mask=None), -1), (dict(of=None), -1), (dict(slopes=BASE, pos=None), -1),
    (dict(q=BASE + 2), -3), (dict(k=BASE + 8), -3), (dict(v=BASE + 8), -3), (dict(of=BASE + 4), -3),
    (dict(ob=BASE + 8), -3), (dict(mask=BASE + 4), -3), (dict(bt=BASE + 2), -3), (dict(ctx=BASE + 1), -3),
    (dict(pos=BASE + 2), -3), (dict(dl=BASE + 2), -3), (dict(slopes=BASE + 2), -3), (dict(ws=BASE + 8), -3),
])
def test_attention_refuses(lib, kw, status):
    assert attention(lib, **kw) == status
    assert lib.pgqa_last_error()


def test_attention_of_no_sequences_is_a_no_op(lib):
    assert attention(lib, B=0, q=None, k=None, v=None, of=None) == 0


def prologue(lib, axes=None, **kw):
    a = dict(q=BASE, k=BASE, v=BASE, gq=BASE, gk=BASE, pos=BASE, n_axes=3, ctx=BASE, nl=None, bt=BASE, kc=BASE, vc=BASE,
             qo=BASE, B=1, M=8, Hq=16, Hkv=8, D=128, P=16, max_pages=4, num_pages=4, theta=1e6, eps=1e-6)
    assert set(kw) <= set(a)
    a.update(kw)
    axes = bytes(64) if axes is None else axes or None
    return lib.qk_norm_rope_append_axes(a["q"], a["k"], a["v"], a["gq"], a["gk"], a["pos"], a["n_axes"], axes, a["ctx"],
                                        a["nl"], a["bt"], a["kc"], a["vc"], a["qo"], a["B"], a["M"], a["Hq"], a["Hkv"],
                                        a["D"], a["P"], a["max_pages"], a["num_pages"], F(a["theta"]), F(a["eps"]), None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), -2), (dict(Hq=12), -2), (dict(P=24), -2), (dict(B=-1), -1), (dict(M=0), -1), (dict(M=-3), -1),
    (dict(B=65535, M=1 << 15), -2), (dict(n_axes=0), -2), (dict(n_axes=5), -2), (dict(theta=0.0), -1),
    (dict(theta=math.nan), -1), (dict(eps=-1.0), -1), (dict(axes=b""), -1), (dict(axes=bytes(63) + b"\x03"), -1),
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(gq=None), -1), (dict(gk=None), -1),
    (dict(pos=None), -1), (dict(ctx=None), -1), (dict(bt=None), -1), (dict(kc=None), -1), (dict(vc=None), -1),
    (dict(qo=None), -1), (dict(q=BASE + 8), -3), (dict(kc=BASE + 2), -3), (dict(pos=BASE + 2), -3),
    (dict(nl=BASE + 2), -3), (dict(ctx=BASE + 2), -3),
])
def test_prologue_refuses(lib, kw, status):
    assert prologue(lib, **kw) == status
    assert lib.pgqa_last_error()


def commit(lib, ks=(BASE,), vs=(BASE + 4096,), ts=(BASE,), **kw):
    far = BASE + (1 << 20)
    a = dict(n=len(ks or ()), ctx=BASE, dl=None, path=BASE, plen=BASE, out=far, B=2, M=8, A=4, Hkv=8, D=128, P=16, max_pages=4,
             num_pages=4)
    assert set(kw) <= set(a)
    a.update(kw)
    arr = lambda x: None if x is None else (ctypes.c_void_p * max(1, len(x)))(*x)  # noqa: E731
    return lib.kv_cache_commit_path(arr(ks), arr(vs), arr(ts), a["n"], a["ctx"], a["dl"], a["path"], a["plen"], a["out"],
                                    a["B"], a["M"], a["A"], a["Hkv"], a["D"], a["P"], a["max_pages"], a["num_pages"],
                                    None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=64), -2), (dict(P=8), -2), (dict(B=-1), -1), (dict(M=0), -1), (dict(M=65), -1), (dict(A=0), -1),
    (dict(A=9), -1), (dict(n=0), -2), (dict(n=129), -2), (dict(Hkv=0), -1), (dict(Hkv=70000), -2), (dict(ks=None, n=1), -1),
    (dict(ctx=None), -1), (dict(path=None), -1), (dict(plen=None), -1), (dict(out=None), -1),
    (dict(ks=(None,)), -1), (dict(vs=(None,)), -1), (dict(ts=(None,)), -1), (dict(ks=(BASE + 8,)), -3),
    (dict(ts=(BASE + 2,)), -3), (dict(out=BASE + 4), -1), (dict(out=BASE - 4), -1), (dict(path=BASE + 2), -3),
    (dict(ks=(BASE, BASE), vs=(BASE + 256, BASE + 512), ts=(BASE, BASE)), -1),
])
def test_commit_refuses(lib, kw, status):
    assert commit(lib, **kw) == status
    assert lib.pgqa_last_error()


@pytest.mark.parametrize("ks,vs", [((BASE, BASE + 512), (BASE + 256, BASE)), ((BASE, BASE + 256), (BASE + 256, BASE + 512))])
def test_commit_refuses_a_cache_that_is_k_of_one_layer_and_v_of_another(lib, ks, vs):
    assert commit(lib, ks=ks, vs=vs, ts=(BASE, BASE)) == -1
    assert lib.pgqa_last_error()


def test_commit_of_no_sequences_is_a_no_op(lib):
    assert commit(lib, B=0, ctx=None, path=None, plen=None, out=None) == 0


def test_workspace_of_bad_sizes_is_zero(lib):
    assert pg.decode_attn_tree_workspace_size(1, 0, 16, 8, 128, 16, 4) == 0
    assert pg.decode_attn_tree_workspace_size(1, 8, 12, 8, 128, 16, 4) == 0
    assert pg.decode_attn_tree_workspace_size(-1, 8, 16, 8, 128, 16, 4) == 0


# ------------------------------------------------------------------ the reference itself
def test_reference_of_equal_scores_is_the_mean():
    kv = inputs.paged_kv(1, [20], Hkv=1, page_size=16)
    q = np.zeros((1, 2, 1, 128), np.uint16)
    out, _ = ref.attention(q, kv.k_cache, kv.v_cache, kv.block_table, kv.context_lens, [[1, 3]], 1.0)
    V = ref.widen(ref.gather(kv.v_cache, kv.block_table[0], 20, 16))[0]
    np.testing.assert_allclose(out[0, 0, 0], V[:19].mean(0), rtol=1e-12)
    np.testing.assert_allclose(out[0, 1, 0], V.mean(0), rtol=1e-12)


def test_reference_bias_of_two_keys():
    """Zero scores, slope s, distances 0 and -1: weights 1 / (1 + e^-s) and the rest."""
    kv = inputs.paged_kv(2, [2], Hkv=1, page_size=16)
    q = np.zeros((1, 1, 1, 128), np.uint16)
    out, _ = ref.attention(q, kv.k_cache, kv.v_cache, kv.block_table, kv.context_lens, [[1]], 1.0, None,
                           np.array([[1]]), [0.7])
    V = ref.widen(ref.gather(kv.v_cache, kv.block_table[0], 2, 16))[0]
    w = 1 / (1 + math.exp(-0.7))
    np.testing.assert_allclose(out[0, 0, 0], w * V[1] + (1 - w) * V[0], rtol=1e-12)


def test_reference_rotation_keeps_relative_positions():
    """<R_p q, R_s k> depends on p - s on every axis."""
    gen = np.random.default_rng(3)
    x = inputs.normal_bf16(gen, (2, 128))
    one = inputs.f32_to_bf16_bits(np.ones(128, np.float32))
    axes = [0] * 16 + [1] * 24 + [2] * 24
    at = lambda v, p: ref.rotate(v, one, np.array(p), axes, 1e4, 1e-6)  # noqa: E731
    a = at(x[0], [5, 9, 30]) @ at(x[1], [3, 2, 7])
    b = at(x[0], [105, 59, 1030]) @ at(x[1], [103, 52, 1007])
    assert abs(a - b) < 1e-9


@pytest.mark.parametrize("make", [list, tuple, bytes, bytearray, np.array, lambda x: np.array(x, np.int32),
                                  lambda x: np.array(x, np.uint8), torch.tensor,
                                  lambda x: torch.tensor(x, dtype=torch.int32), iter])
def test_axes_of_any_sequence(make):
    """Axis numbers are taken one by one, whatever holds them."""
    axes = [0] * 16 + [1] * 24 + [2] * 24
    assert binding._axis_bytes(make(axes)) == bytes(axes)


@pytest.mark.parametrize("axes", [[0] * 63, [0] * 65, 64, "0" * 64, np.zeros(16, np.int32), np.zeros(8, np.int64),
                                  torch.zeros(16, dtype=torch.int32), [-1] * 64, [256] * 64, [0.0] * 64,
                                  np.zeros((64, 1), np.int32), None])
def test_axes_that_are_no_64_numbers_are_refused(axes):
    """Among them arrays of 64 bytes of memory that hold fewer numbers."""
    with pytest.raises((TypeError, ValueError)):
        binding._axis_bytes(axes)
