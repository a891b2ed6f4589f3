"""CPU checks of drafted-tree decoding over an INT8 cache and of the verification: what the entry points refuse before
touching the GPU, and the references' closed forms. No compute call is made here."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_gqa_decode_head_gb300 as pg
import tree_int8_reference as ref
import tree_reference as bf16_ref
from paged_gqa_decode_head_gb300 import binding, inputs
from paged_gqa_decode_head_gb300 import build as libbuild

BASE = 0x10000000  # a well aligned address that is never dereferenced
F, LL = ctypes.c_float, ctypes.c_longlong


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return binding.load_library()


def attention(lib, **kw):
    a = dict(q=BASE, k=BASE, v=BASE, ks=BASE, vs=BASE, bt=BASE, ctx=BASE, mask=BASE, pos=BASE, dl=None, slopes=None, B=1,
             M=8, Hq=16, Hkv=8, D=128, P=16, max_pages=4, num_pages=4, scale=0.1, cap=0.0, of=BASE, ob=None, ws=None, wsb=0)
    assert set(kw) <= set(a)
    a.update(kw)
    a["scale"], a["cap"] = F(a["scale"]), F(a["cap"])
    return lib.decode_attn_paged_tree_int8(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=64), -2), (dict(Hq=12), -2), (dict(Hq=72), -2), (dict(P=8), -2), (dict(P=48), -2), (dict(P=512), -2),
    (dict(B=-1), -1), (dict(B=65536), -2), (dict(M=0), -1), (dict(M=65), -1), (dict(scale=math.nan), -1),
    (dict(scale=math.inf), -1), (dict(cap=-1.0), -1), (dict(cap=math.nan), -1), (dict(cap=math.inf), -1),
    (dict(P=256, max_pages=(1 << 22) + 1), -2), (dict(B=60000, P=256, max_pages=1 << 22), -2),
    (dict(B=65535, M=64, Hq=8192, Hkv=1024), -2), (dict(Hq=70000, Hkv=70000), -2),
    (dict(max_pages=-1), -1), (dict(num_pages=-1), -1), (dict(num_pages=0), -1), (dict(num_pages=2 ** 26), -2),
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(ks=None), -1), (dict(vs=None), -1),
    (dict(bt=None), -1), (dict(ctx=None), -1), (dict(mask=None), -1), (dict(of=None), -1),
    (dict(slopes=BASE, pos=None), -1), (dict(q=BASE + 2), -3), (dict(k=BASE + 8), -3), (dict(v=BASE + 8), -3),
    (dict(ks=BASE + 4), -3), (dict(vs=BASE + 4), -3), (dict(of=BASE + 4), -3), (dict(ob=BASE + 8), -3),
    (dict(mask=BASE + 4), -3), (dict(bt=BASE + 2), -3), (dict(ctx=BASE + 1), -3), (dict(pos=BASE + 2), -3),
    (dict(dl=BASE + 2), -3), (dict(slopes=BASE + 2), -3), (dict(ws=BASE + 8), -3),
])
def test_attention_refuses(lib, kw, status):
    assert attention(lib, **kw) == status
    assert lib.pgqa_last_error()


def test_attention_of_no_sequences_is_a_no_op(lib):
    assert attention(lib, B=0, q=None, k=None, ks=None, of=None) == 0


def prologue(lib, axes=None, **kw):
    a = dict(q=BASE, k=BASE, v=BASE, gq=BASE, gk=BASE, pos=BASE, n_axes=3, axes=None, ctx=BASE, nl=None, bt=BASE, kc=BASE,
             vc=BASE, ks=BASE, vs=BASE, qo=BASE, B=1, M=8, Hq=16, Hkv=8, D=128, P=16, max_pages=4, num_pages=4, theta=1e6,
             eps=1e-6)
    assert set(kw) <= set(a)
    a.update(kw)
    a["axes"] = bytes(64) if axes is None else axes or None
    a["theta"], a["eps"] = F(a["theta"]), F(a["eps"])
    return lib.qk_norm_rope_append_axes_int8(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), -2), (dict(Hq=12), -2), (dict(P=24), -2), (dict(B=-1), -1), (dict(M=0), -1), (dict(M=-3), -1),
    (dict(B=65535, M=1 << 15), -2), (dict(n_axes=0), -2), (dict(n_axes=5), -2), (dict(theta=0.0), -1),
    (dict(theta=math.nan), -1), (dict(eps=-1.0), -1), (dict(axes=b""), -1), (dict(axes=bytes(63) + b"\x03"), -1),
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(gq=None), -1), (dict(gk=None), -1),
    (dict(pos=None), -1), (dict(ctx=None), -1), (dict(bt=None), -1), (dict(kc=None), -1), (dict(vc=None), -1),
    (dict(ks=None), -1), (dict(vs=None), -1), (dict(qo=None), -1), (dict(q=BASE + 8), -3), (dict(kc=BASE + 2), -3),
    (dict(vs=BASE + 8), -3), (dict(pos=BASE + 2), -3), (dict(nl=BASE + 2), -3), (dict(ctx=BASE + 2), -3),
])
def test_prologue_refuses(lib, kw, status):
    assert prologue(lib, **kw) == status
    assert lib.pgqa_last_error()


def read(lib, **kw):
    a = dict(k=BASE, v=BASE, ks=BASE, vs=BASE, bt=BASE, ctx=BASE, first=None, ko=BASE, vo=BASE, B=1, N=8, Hkv=8, D=128, P=16,
             max_pages=4, num_pages=4)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kv_cache_read_int8(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=64), -2), (dict(P=8), -2), (dict(B=-1), -1), (dict(B=70000), -2), (dict(N=-1), -1), (dict(Hkv=0), -1),
    (dict(Hkv=70000), -2), (dict(k=None), -1), (dict(vs=None), -1), (dict(ctx=None), -1), (dict(ko=None), -1),
    (dict(k=BASE + 8), -3), (dict(ks=BASE + 4), -3), (dict(vo=BASE + 2), -3), (dict(first=BASE + 2), -3),
])
def test_read_refuses(lib, kw, status):
    assert read(lib, **kw) == status
    assert lib.pgqa_last_error()


def test_read_of_nothing_is_a_no_op(lib):
    assert read(lib, B=0, k=None) == 0 and read(lib, N=0, ko=None, vo=None) == 0


def commit(lib, ks=(BASE,), vs=(BASE + 4096,), kss=(BASE + 8192,), vss=(BASE + 12288,), ts=(BASE,), **kw):
    far = BASE + (1 << 20)
    a = dict(n=len(ks or ()), ctx=BASE, dl=None, path=BASE, plen=BASE, out=far, B=2, M=8, A=4, Hkv=8, D=128, P=16,
             max_pages=4, num_pages=4)
    assert set(kw) <= set(a)
    a.update(kw)
    arr = lambda x: None if x is None else (ctypes.c_void_p * max(1, len(x)))(*x)  # noqa: E731
    return lib.kv_cache_commit_path_int8(arr(ks), arr(vs), arr(kss), arr(vss), arr(ts), *a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=64), -2), (dict(P=8), -2), (dict(B=-1), -1), (dict(M=0), -1), (dict(M=65), -1), (dict(A=0), -1),
    (dict(A=9), -1), (dict(n=0), -2), (dict(n=129), -2), (dict(Hkv=0), -1), (dict(ks=None, n=1), -1), (dict(kss=None), -1),
    (dict(vss=None), -1), (dict(ctx=None), -1), (dict(out=None), -1), (dict(kss=(None,)), -1), (dict(vs=(None,)), -1),
    (dict(ks=(BASE + 8,)), -3), (dict(vss=(BASE + 4,)), -3), (dict(ts=(BASE + 2,)), -3), (dict(out=BASE + 4), -1),
    (dict(ks=(BASE, BASE + 256), vs=(BASE + 512, BASE + 768), kss=(BASE, BASE), vss=(BASE + 16, BASE + 32),
          ts=(BASE, BASE)), -1),
])
def test_commit_refuses(lib, kw, status):
    assert commit(lib, **kw) == status
    assert lib.pgqa_last_error()


def verify(lib, **kw):
    a = dict(target=BASE, draft=BASE, f32=0, ts=1000, ds=1000, tokens=BASE, parents=BASE, dl=None, temps=BASE, u=BASE,
             noise=BASE, B=2, M=8, A=8, V=1000, path=BASE, plen=BASE, new=BASE, logp=BASE, ws=None, wsb=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.verify_drafted_tree(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), -1), (dict(B=65536), -2), (dict(M=0), -1), (dict(M=65), -1), (dict(A=0), -1), (dict(A=9), -1),
    (dict(V=0), -1), (dict(V=(1 << 24) + 1, ts=1 << 25, ds=1 << 25), -2), (dict(ts=999), -1), (dict(ds=999), -1),
    (dict(ts=(1 << 32) + 1), -2), (dict(target=None), -1), (dict(tokens=None), -1), (dict(parents=None), -1),
    (dict(temps=None), -1), (dict(u=None), -1), (dict(noise=None), -1), (dict(path=None), -1), (dict(plen=None), -1),
    (dict(new=None), -1), (dict(target=BASE + 2), -3), (dict(draft=BASE + 8), -3), (dict(noise=BASE + 4), -3),
    (dict(tokens=BASE + 2), -3), (dict(logp=BASE + 2), -3), (dict(dl=BASE + 1), -3),
])
def test_verification_refuses(lib, kw, status):
    assert verify(lib, **kw) == status
    assert lib.pgqa_last_error()


def test_verification_of_no_sequences_is_a_no_op(lib):
    assert verify(lib, B=0, target=None, path=None) == 0


def test_workspaces_of_bad_sizes_are_zero(lib):
    assert pg.decode_attn_tree_int8_workspace_size(1, 0, 16, 8, 128, 16, 4) == 0
    assert pg.decode_attn_tree_int8_workspace_size(1, 8, 12, 8, 128, 16, 4) == 0
    assert pg.verify_drafted_tree_workspace_size(-1, 8, 100) == 0
    assert pg.verify_drafted_tree_workspace_size(1, 65, 100) == 0


@pytest.mark.parametrize("shape,strides,ok", [((2, 3, 8), (24, 8, 1), 8), ((2, 3, 8), (30, 10, 1), 10), ((1, 3, 8), (7, 10, 1), 10),
                                             ((2, 1, 8), (12, 3, 1), 12), ((2, 3, 8), (31, 10, 1), None),
                                             ((2, 3, 8), (24, 8, 2), None), ((2, 3, 8), (21, 7, 1), None)])
def test_row_strides_of_logits(shape, strides, ok):
    t = torch.as_strided(torch.zeros(200), shape, strides)
    if ok is None:
        with pytest.raises(ValueError):
            binding._logit_rows(t, torch.float32, shape, "t", -1)
    else:
        assert binding._logit_rows(t, torch.float32, shape, "t", -1) == (t.data_ptr(), ok)


# ------------------------------------------------------------------ the references themselves
def test_reference_attention_is_the_bf16_one_for_scales_that_are_powers_of_two():
    """Codes times a power of two are bf16 numbers: the bf16 reference of those rows gives the same result."""
    kv = inputs.paged_kv(5, [40, 9], Hkv=2, page_size=16)
    gen = np.random.default_rng(5)
    k8, v8 = (gen.integers(-127, 128, kv.k_cache.shape).astype(np.int8) for _ in range(2))
    ks, vs = (2.0 ** gen.integers(-9, -4, kv.k_cache.shape[:3]).astype(np.float32) for _ in range(2))
    bits = lambda c, s: inputs.f32_to_bf16_bits(c.astype(np.float32) * s[..., None])  # noqa: E731
    q = inputs.normal_bf16(gen, (2, 3, 4, 128))
    args = dict(positions=np.array([[37, 38, 38], [6, 7, 8]]), slopes=np.array([0.5, -0.25, 0.0, 1.0]), softcap=4.0)
    masks = [[1, 3, 5], [1, 2, 7]]
    a, _ = ref.attention(q, k8, v8, ks, vs, kv.block_table, [40, 9], masks, 0.1, [3, 3], **args)
    b, _ = bf16_ref.attention(q, bits(k8, ks), bits(v8, vs), kv.block_table, [40, 9], masks, 0.1, None, **args)
    np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-14)


def test_reference_quantization_is_the_oracles():
    import oracle

    oracle.build()
    bits = inputs.normal_bf16(np.random.default_rng(6), (50, 128))
    bits[0], bits[1, 1:] = 0, 0
    codes, scales = oracle.quantize_rows_int8(bits)
    again, t = ref.quantize(bf16_ref.widen(bits).astype(np.float32))
    assert np.array_equal(codes, again) and np.array_equal(scales, t)


@pytest.mark.parametrize("draft", [False, True])
def test_reference_verification_keeps_the_targets_distribution(draft):
    """Exactly, by summing over what the random numbers decide: two siblings of one node, V = 3. P(new token = i) =
    P(first accepted) [t1 = i] + ... = p(i), for every order of drawn siblings weighted by its probability."""
    p = np.array([0.5, 0.2, 0.3])
    q = np.array([0.2, 0.7, 0.1])
    total = np.zeros(3)
    for t1 in range(3):
        for t2 in range(3):
            if t1 == t2:
                continue
            chance = q[t1] * q[t2] / (1 - q[t1]) if draft else 1 / 6
            args = (np.log(np.stack([p] * 3)), np.log(np.stack([q] * 3)) if draft else None, [0, t1, t2], [-1, 0, 0], 3, 1.0)
            left = chance
            grid = 4000  # u on a fine grid: the share of accepted u is the acceptance's probability
            for k, t in ((1, t1), (2, t2)):
                def took(x):
                    u = [0.0, 1.0, 1.0]
                    u[k] = x
                    return ref.verify(*args, np.array(u), np.ones(3), 3)[0] == [0, k]
                lo, hi = 0, grid
                while lo < hi:  # acceptance falls with u
                    mid = (lo + hi) // 2
                    lo, hi = (mid + 1, hi) if took(mid / grid) else (lo, mid)
                total[t] += left * lo / grid
                left *= 1 - lo / grid
            # what is left is drawn from the residual: its shares from races whose noise favours one token at a time
            rest = p.copy()
            if draft:
                r1 = np.maximum(rest - q, 0)
                r1[t1] = 0
                q2 = np.where(np.arange(3) == t1, 0, q)
                rest = r1 / r1.sum() if r1.sum() > 0 else r1
                rest = np.maximum(rest - q2 / q2.sum(), 0)
                rest[t2] = 0
            else:
                rest[[t1, t2]] = 0
            if rest.sum() > 0:
                total += left * rest / rest.sum()
            else:
                assert left < 1e-3
    np.testing.assert_allclose(total, p, atol=2e-3)
