"""Drafted-tree decoding over an INT8 cache on the GPU: the prologue that quantizes, the read back, attention of a
drafted tree, the commit of the accepted path, and steps of all of them with the verification between."""
import math

import numpy as np
import pytest
import torch

import oracle
import paged_gqa_decode_head_gb300 as pg
import tree_int8_reference as ref
import tree_reference as bf16_ref
from paged_gqa_decode_head_gb300 import binding, inputs
from paged_gqa_decode_head_gb300.runner import bf16_bits, to_device_bf16, to_device_i32

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)
THETA = 1e6
SENTINEL = 7.0


@pytest.fixture(autouse=True)
def _clean_flags():
    pg.device_error_flags(clear=True)
    yield


def mask_tensor(masks):
    a = np.array([[int(m) & (2 ** 64 - 1) for m in row] for row in masks], dtype=np.uint64)
    return torch.from_numpy(a.view(np.int64)).cuda()


def workspace(B, M, Hq, Hkv, P, max_pages):
    n = pg.decode_attn_tree_int8_workspace_size(B, M, Hq, Hkv, 128, P, max_pages)
    return torch.full((max(16, n),), 0xA5, dtype=torch.uint8, device="cuda")  # any contents


class Case:
    """Inputs of one attention call, on the host and on the GPU."""

    def __init__(self, seed, ctx, M, Hq=16, Hkv=8, P=16, draft_lens=None, masks=None, softcap=0.0, slopes=None, roots=1,
                 **kv_args):
        gen = inputs.generator(seed, 501)
        self.B, self.M, self.Hq, self.Hkv, self.P = len(ctx), M, Hq, Hkv, P
        kv = inputs.paged_kv(seed, ctx, Hkv=Hkv, page_size=P, **kv_args)
        self.table, self.lens, self.max_pages = kv.block_table, kv.context_lens, kv.max_pages
        finite = lambda bits: np.nan_to_num(bf16_ref.widen(bits), nan=1.0)  # noqa: E731
        self.k8, self.ks = ref.quantize(finite(kv.k_cache))
        self.v8, self.vs = ref.quantize(finite(kv.v_cache))
        for name in ("ks", "vs"):  # slots of nobody: anything in the scale
            unowned = np.isnan(bf16_ref.widen(kv.k_cache)).any(-1)
            getattr(self, name)[unowned] = np.nan
        self.q = inputs.normal_bf16(gen, (self.B, M, Hq, 128))
        self.n = list(draft_lens) if draft_lens is not None else [M] * self.B
        self.draft_lens = draft_lens
        trees = [bf16_ref.random_tree(gen, M, roots) for _ in range(self.B)]
        self.masks = masks if masks is not None else [t[0] for t in trees]
        self.positions = np.array([[ctx[b] - self.n[b] + d for d in trees[b][1]] for b in range(self.B)], np.int32)
        self.softcap, self.slopes, self.scale = softcap, None if slopes is None else np.asarray(slopes, np.float32), SCALE

    def upload(self):
        self.d = dict(q=to_device_bf16(self.q, "cuda"), k8=torch.from_numpy(self.k8).cuda(),
                      v8=torch.from_numpy(self.v8).cuda(), ks=torch.from_numpy(self.ks).cuda(),
                      vs=torch.from_numpy(self.vs).cuda(), bt=to_device_i32(self.table, "cuda"),
                      cl=to_device_i32(self.lens, "cuda"), mask=mask_tensor(self.masks),
                      pos=to_device_i32(self.positions, "cuda"),
                      dl=None if self.draft_lens is None else to_device_i32(np.array(self.draft_lens), "cuda"),
                      slopes=None if self.slopes is None else torch.from_numpy(self.slopes).cuda(),
                      ws=workspace(self.B, self.M, self.Hq, self.Hkv, self.P, self.max_pages),
                      of=torch.full(self.q.shape, SENTINEL, dtype=torch.float32, device="cuda"),
                      ob=torch.full(self.q.shape, SENTINEL, dtype=torch.bfloat16, device="cuda"))
        return self.d

    def launch(self, stream=None, f32=True, bf16=True):
        d = self.d
        pg.decode_attn_paged_tree_int8(d["q"], d["k8"], d["v8"], d["ks"], d["vs"], d["bt"], d["cl"], d["mask"], self.scale,
                                       positions=d["pos"], draft_lens=d["dl"], slopes=d["slopes"], softcap=self.softcap,
                                       out_f32=d["of"] if f32 else None, out_bf16=d["ob"] if bf16 else None,
                                       workspace=d["ws"], stream=stream)

    def results(self):
        torch.cuda.synchronize()
        return self.d["of"].cpu().numpy(), self.d["ob"].float().cpu().numpy()

    def run(self):
        self.upload()
        self.launch()
        return self.results()

    def reference(self, **kw):
        return ref.attention(self.q, self.k8, self.v8, self.ks, self.vs, self.table, self.lens, self.masks, self.scale,
                             self.n, self.positions, self.slopes, self.softcap, **kw)

    def check(self, flags=0, **kw):
        of, ob = self.run()
        check_outputs(of, ob, *self.reference(**kw), self.n)
        assert pg.device_error_flags() == flags
        return of


def check_outputs(of, ob, out, bound, n):
    for b in range(out.shape[0]):
        live = slice(0, n[b])
        assert np.isfinite(of[b, live]).all()
        over = np.abs(of[b, live] - out[b, live]) - (bound[b, live] + 2.0 ** -24 * np.abs(out[b, live]))
        assert (over <= 0).all(), (b, float(over.max()), float(np.abs(of[b, live] - out[b, live]).max()))
        # the bf16 output is the rounding of the fp32 one: half a step more
        over = np.abs(ob[b, live] - out[b, live]) - (bound[b, live] * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(out[b, live]))
        assert (over <= 0).all(), (b, float(over.max()))
        assert (of[b, n[b]:] == SENTINEL).all() and (ob[b, n[b]:] == SENTINEL).all()


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 130, 191, 255, 256, 257, 300, 513, 700])
def test_context_lengths(T):
    for M in (1, 2, 8, 17):
        if M <= T:
            Case(2000 + 37 * T + M, [T, T + 3], M).check()


@pytest.mark.parametrize("T", [64, 65, 128, 150, 192, 330])
def test_widest_trees(T):
    Case(2100 + T, [T, T + 1], 64, Hkv=2, Hq=4, roots=3).check()


@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("M", [1, 5, 33, 64])
def test_group_sizes(g, M):
    """Query rows per KV head from 1 to 512."""
    Case(2200 + 10 * g + M, [M + 140, M + 17], M, Hq=2 * g, Hkv=2).check()


@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
def test_page_sizes(P):
    Case(2300 + P, [3 * P + 5, 700, P, P + 1], 12, P=P).check()


@pytest.mark.parametrize("B,T", [(1, 4000), (3, 1500), (40, 260), (300, 40)])
def test_work_split(B, T):
    gen = inputs.generator(2400 + B, 5)
    ctx = [int(x) for x in gen.integers(8, T + 1, B)]
    ctx[0] = T
    Case(2400 + B, ctx, 8, Hq=4, Hkv=2).check()


@pytest.mark.parametrize("M,g", [(8, 1), (5, 3), (16, 2), (32, 2), (11, 8), (64, 3)])
def test_long_runs_of_tiles(M, g):
    """Several tiles in every CTA, segments behind each other, scores that rise along the keys."""
    c = Case(2450 + M, [12000, 900, 30000], M, Hq=4 * g, Hkv=4)
    for b in range(3):
        for page in range(-(-int(c.lens[b]) // 16)):
            c.ks[c.table[b, page]] *= np.float32(1 + 6 * (page // 40 % 5))
    c.check()


@pytest.mark.parametrize("M,g,P", [(33, 5, 16), (17, 8, 64), (50, 3, 256), (64, 8, 32)])
def test_row_groups_in_pairs(M, g, P):
    """More than 64 rows per KV head: two to eight groups of rows (three for the first three: the last pair lacks one),
    an absent draft, each output alone."""
    c = Case(2470 + M, [3000, 40, 900], M, Hq=2 * g, Hkv=2, P=P, draft_lens=[M, 0, M - 3])
    of = c.check()
    _, ob = c.results()
    c.upload()
    c.launch(f32=False)
    assert np.array_equal(c.results()[1], ob) and (c.d["of"] == SENTINEL).all()
    c.upload()
    c.launch(bf16=False)
    assert np.array_equal(c.results()[0], of) and (c.d["ob"] == SENTINEL).all()


def test_row_groups_in_pairs_over_long_runs():
    """Some 24 tiles a CTA: O leaves the tensor core on the way, a page lies outside the pool."""
    c = Case(2480, [60000], 33, Hq=20, Hkv=4)
    c.table[0, 1000] = -1
    c.check(flags=binding.DEVERR_BAD_PAGE, skip=lambda b, j: j // 16 == 1000)


def test_ragged_drafts_leave_other_rows_alone():
    Case(2500, [300, 1, 5, 16, 200, 129], 16, draft_lens=[0, 1, 5, 16, 9, 16]).check()


def test_absent_queries_may_hold_anything():
    c = Case(2505, [300, 140], 16, draft_lens=[5, 16], Hq=64)
    c.q[0, 5:] = 0x7FC0
    c.check()


def test_empty_sequence_beside_others():
    Case(2510, [0, 40, 0], 4, draft_lens=[0, 4, 0]).check()


def test_rows_that_see_nothing_are_zero():
    masks = [[0, 2, 0, 8, 1 << 40, 0xF, 0xF0, 1]]
    of = Case(2520, [6], 8, draft_lens=[6], masks=masks).check()
    assert (of[0, 0] == 0).all() and (of[0, 4] == 0).all()


def test_masks_need_not_be_trees():
    gen = inputs.generator(2530, 6)
    masks = [[int(gen.integers(0, 2 ** 63)) * 2 + int(gen.integers(0, 2)) for _ in range(64)] for _ in range(2)]
    masks[0][0], masks[0][1], masks[0][63] = 2 ** 64 - 1, 1 << 63, 1
    Case(2530, [64, 190], 64, Hq=4, Hkv=2, masks=masks).check()


@pytest.mark.parametrize("T", [40, 128, 135, 400])
def test_nonfinite_scales_reach_only_the_tokens_that_see_them(T):
    M = 16
    c = Case(2540 + T, [T], M, Hq=8, Hkv=4)
    bad = {3: np.nan, 7: np.inf, 12: -np.inf}
    ks, vs = c.ks.copy(), c.vs.copy()
    for j, x in bad.items():
        page, off = c.table[0, (T - M + j) // 16], (T - M + j) % 16
        c.vs[page, :, off] = x
        if j != 7:
            c.ks[page, :, off] = x
    of, _ = c.run()
    c.ks, c.vs = ks, vs
    out, bound = c.reference()
    sees = [[j for j in bad if c.masks[0][i] >> j & 1] for i in range(M)]
    assert any(sees) and not all(sees)
    for i in range(M):
        if not sees[i]:
            assert np.isfinite(of[0, i]).all()
            assert (np.abs(of[0, i] - out[0, i]) <= bound[0, i] + 2.0 ** -24 * np.abs(out[0, i])).all(), i
        else:
            assert not np.isfinite(of[0, i]).any()


@pytest.mark.parametrize("softcap", [1e-3, 0.5, 5.0, 30.0, 1e4, 3e38])
def test_capped_scores(softcap):
    c = Case(2600, [300, 77], 9, softcap=softcap)
    c.ks *= np.float32(6)
    c.check()


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("M", [1, 12, 40])
def test_distance_bias(M, softcap):
    slopes = [2.0 ** -(h / 2) * (-1 if h % 5 == 4 else 1) for h in range(16)]
    slopes[3] = 0.0
    Case(2610 + M, [900, 64, 333], M, slopes=slopes, softcap=softcap, roots=min(2, M)).check()


@pytest.mark.parametrize("far", [-2 ** 31, -70000, 10 ** 6, 2 ** 31 - 1])
def test_a_row_own_position_cancels(far):
    """Rows that see only the prefix: pos_i moves all of a row's scores alike."""
    c = Case(2620, [700], 4, slopes=[(-1) ** h * 2.0 ** -(h / 2) for h in range(16)], masks=[[0] * 4])
    c.positions[:] = far
    of, _ = c.run()
    c.positions[:] = 696
    out, bound = c.reference()
    assert (np.abs(of - out) <= bound + 2.0 ** -24 * np.abs(out)).all()


@pytest.mark.parametrize("T", [300, 12000])
def test_slopes_that_favour_the_first_keys(T):
    Case(2630 + T, [T], 3, Hq=4, Hkv=2, slopes=[-1.0, -0.01, -3.0, 0.5]).check()


@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_drafted_tokens_far_from_the_prefix(softcap):
    """Drafted tokens 10^9 past the prefix outweigh it, or are outweighed: the same as 5000 away."""
    c = Case(2640, [200, 90], 12, slopes=[(-1) ** h * (1 + h / 8) for h in range(16)], softcap=softcap)
    near = c.positions.copy()
    depth = near - np.array([[200 - 12], [90 - 12]])
    c.positions = (10 ** 9 + depth).astype(np.int32)
    of, _ = c.run()
    c.positions = (5000 + depth).astype(np.int32)
    out, bound = c.reference()
    assert (np.abs(of - out) <= bound + 2.0 ** -24 * np.abs(out)).all()


@pytest.mark.parametrize("T", [8, 60])
def test_steep_slopes_keep_scores_of_equal_positions_apart(T):
    """All drafted tokens 40 past the prefix, all seen: among them the scores decide, however steep the slope."""
    c = Case(2650 + T, [T], 8, Hq=4, Hkv=2, slopes=[1.0, 100.0, 1e5, 1e6], masks=[[255] * 8])
    c.positions[:] = T - 8 + 40
    c.check()


def test_peaked_scores_rescale_the_state():
    c = Case(2660, [900], 4, Hq=4, Hkv=2)
    f = np.linspace(0.0, 40.0, 900)
    for j in range(900):
        page, off = c.table[0, j // 16], j % 16
        for h in range(2):
            direction = bf16_ref.widen(c.q[0, 0, 2 * h])
            c.k8[page, h, off], c.ks[page, h, off] = ref.quantize(direction * (f[j] / np.linalg.norm(direction)))
    c.check()


@pytest.mark.parametrize("lo,hi", [(-30, 30), (-60, -40), (30, 60), (0, 12)])
def test_value_scales_over_many_magnitudes(lo, hi):
    """V rows whose scales grow, fall and jump by powers of two along the keys; zero rows among them."""
    for rising in (1, -1):
        c = Case(2670 + lo, [700, 260], 9, Hq=8, Hkv=4)
        gen = np.random.default_rng(abs(lo) + rising + 1)
        for b in range(2):
            for j in range(int(c.lens[b])):
                e = lo + (hi - lo) * (j if rising > 0 else int(c.lens[b]) - j) / int(c.lens[b]) + gen.normal()
                page, off = c.table[b, j // 16], j % 16
                c.vs[page, :, off] *= np.float32(2.0 ** round(e))
                if gen.random() < 0.05:
                    c.vs[page, :, off], c.v8[page, :, off] = 0, 0
        c.check()


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-30])
def test_scales(scale):
    c = Case(2680, [200], 6)
    c.scale = scale
    c.check()


def test_very_low_scores_are_still_a_softmax():
    c = Case(2690, [5], 1, Hq=2, Hkv=1)
    c.q[...] = inputs.f32_to_bf16_bits(np.full(c.q.shape, 1e4, np.float32))
    c.k8[...], c.ks[...], c.scale = -127, 1e28, 0.1
    of, _ = c.run()
    V = ref.rows_of(c.v8, c.table[0], 5, 16)[0].astype(np.float64) * ref.rows_of(c.vs, c.table[0], 5, 16)[0][:, None]
    np.testing.assert_allclose(of[0, 0, 0], V.mean(0), atol=1e-4)


def test_pages_outside_the_pool_are_skipped():
    c = Case(2700, [500, 100], 6)
    c.table[0, 3], c.table[0, 10], c.table[1, 6] = -1, c.k8.shape[0], 2 ** 31 - 1
    gone = {(0, 3), (0, 10), (1, 6)}
    c.check(flags=binding.DEVERR_BAD_PAGE, skip=lambda b, j: (b, j // 16) in gone)


def test_bad_lengths_give_zeros_and_a_flag():
    c = Case(2710, [60, 40, 50, 30, 20], 8, draft_lens=[8, 8, 8, 4, 2])
    c.lens[1] = 7                          # T < n
    c.lens[3] = c.max_pages * 16 + 1       # longer than the table
    c.lens[4] = -5
    c.draft_lens = c.n = [8, 8, 9, 4, -1]  # n > M, n < 0
    of, ob = c.run()
    assert pg.device_error_flags() == binding.DEVERR_BAD_CONTEXT
    assert (of[1:] == 0).all() and (ob[1:] == 0).all()
    out, bound = Case(2710, [60, 40, 50, 30, 20], 8, draft_lens=[8, 8, 8, 4, 2]).reference()
    assert (np.abs(of[0] - out[0]) <= bound[0] + 2.0 ** -24 * np.abs(out[0])).all()


def test_outputs_alone_and_together_agree():
    """Each output alone is within the bound; below a span's length they are the same bits."""
    c = Case(2730, [400], 7)
    of, ob = c.run()
    c.upload()
    c.launch(f32=False)
    _, only = c.results()
    assert np.array_equal(only, ob) and (c.d["of"] == SENTINEL).all()
    c.upload()
    c.launch(bf16=False)
    only, _ = c.results()
    assert np.array_equal(only, of) and (c.d["ob"] == SENTINEL).all()


def test_single_tokens_match_the_int8_decode():
    ctx = [40, 17, 600, 5000]
    c = Case(2740, ctx, 1, masks=[[1]] * 4)
    of, _ = c.run()
    d = c.d
    n = pg.decode_attn_int8_workspace_size(4, 16, 8, 128, 16, c.max_pages, 0)
    other = torch.empty_like(d["of"][:, 0])
    pg.decode_attn_paged_int8(d["q"][:, 0].contiguous(), d["k8"], d["v8"], d["ks"], d["vs"], d["bt"], d["cl"], SCALE,
                              out_f32=other, workspace=torch.zeros(max(16, n), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    out, _ = c.reference()
    # the single-token kernel's own bar is 2e-3 absolute; its fp16 pair holds it far inside
    assert np.abs(of[:, 0] - other.cpu().numpy()).max() < 1e-4


def test_repeated_calls_and_a_used_workspace_give_the_same_bits():
    c = Case(2750, [2000, 30, 700], 16)
    of, _ = c.run()
    other = Case(2751, [90], 16)
    other.upload()
    other.d["ws"] = c.d["ws"]
    other.launch()
    for _ in range(3):
        c.d["of"].fill_(SENTINEL)
        c.launch()
        assert np.array_equal(c.results()[0], of)


def test_two_streams_at_once_with_workspaces_of_their_own():
    a, b = Case(2760, [3000], 16), Case(2761, [2500, 800], 9)
    ra, rb = a.run()[0], b.run()[0]
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a.launch(stream=sa)
        b.launch(stream=sb)
    assert np.array_equal(a.results()[0], ra) and np.array_equal(b.results()[0], rb)


def test_captured_call_follows_lengths_masks_and_drafts():
    c = Case(2770, [700, 300], 16, draft_lens=[16, 16])
    c.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.launch()
    for ctx, n in (([650, 17], [3, 16]), ([30, 299], [16, 0]), ([700, 300], [16, 16])):
        c.lens[:] = ctx
        c.n = c.draft_lens = n
        c.positions[:] = np.array(ctx)[:, None] - np.array(n)[:, None] + np.arange(16)[None] % 5
        c.d["cl"].copy_(to_device_i32(c.lens, "cuda"))
        c.d["dl"].copy_(to_device_i32(np.array(n), "cuda"))
        c.d["pos"].copy_(to_device_i32(c.positions, "cuda"))
        c.d["of"].fill_(SENTINEL), c.d["ob"].fill_(SENTINEL)
        g.replay()
        of, ob = c.results()
        check_outputs(of, ob, *c.reference(), n)


def test_a_pool_past_32_bit_offsets():
    """Codes past 2^32 bytes in the pool."""
    P, Hkv, M, T = 256, 8, 5, 700
    c = Case(2780, [T], M, Hq=8, Hkv=Hkv, P=P)
    pages = (1 << 32) // (P * Hkv * 128) + 64
    c.upload()
    d = c.d
    big = [torch.zeros((pages, Hkv, P, 128), dtype=torch.int8, device="cuda") for _ in range(2)]
    big += [torch.zeros((pages, Hkv, P), device="cuda") for _ in range(2)]
    far = [pages - 1, pages - 9, pages - 2]
    for i, page in enumerate(far):
        for t, name in zip(big, ("k8", "v8", "ks", "vs")):
            t[page] = d[name][int(c.table[0, i])]
    d["k8"], d["v8"], d["ks"], d["vs"] = big
    d["bt"] = to_device_i32(np.array([far]), "cuda")
    c.launch()
    check_outputs(*c.results(), *c.reference(), c.n)


def test_one_long_context():
    Case(2790, [40000], 3, Hq=2, Hkv=1, softcap=30.0, slopes=[0.5, 0.001]).check()


@pytest.mark.parametrize("seed", range(24))
def test_random_calls(seed):
    gen = inputs.generator(2800 + seed, 7)
    pick = lambda *x: x[int(gen.integers(0, len(x)))]  # noqa: E731
    g, Hkv, P, M = pick(1, 2, 3, 5, 8), pick(1, 2, 3), pick(16, 32, 64, 128, 256), int(gen.integers(1, 65))
    B = int(gen.integers(1, 9))
    n = [int(gen.integers(0, M + 1)) for _ in range(B)]
    ctx = [x + int(pick(0, 1, gen.integers(0, 40), gen.integers(0, 700))) for x in n]
    slopes = [float(x) for x in gen.normal(0, 0.2, g * Hkv)] if gen.random() < 0.4 else None
    masks = None
    if gen.random() < 0.4:
        masks = [[int(gen.integers(0, 2 ** 62)) << int(gen.integers(0, 3)) for _ in range(M)] for _ in range(B)]
    Case(2800 + seed, ctx, M, Hq=g * Hkv, Hkv=Hkv, P=P, draft_lens=n, masks=masks, slopes=slopes,
         softcap=float(pick(0.0, 0.0, 8.0)), max_pages=max(1, -(-max(ctx) // P) + int(gen.integers(0, 5)))).check()


def test_more_sequences_than_threads():
    gen = inputs.generator(2830, 8)
    n = [int(gen.integers(0, 3)) for _ in range(900)]
    ctx = [x + (int(gen.integers(0, 300)) if x else 0) for x in n]
    Case(2830, ctx, 2, Hq=2, Hkv=1, draft_lens=n).check()


@pytest.mark.parametrize("B,M,Hq,Hkv,T", [(4, 2, 8, 8, 90000), (3, 40, 32, 8, 40000), (2, 16, 8, 4, 120000)])
def test_long_contexts_keep_fp32_outputs(B, M, Hq, Hkv, T):
    """Many tiles per CTA and stream, against the formula in 64 bits on the GPU: 2-norm within 2^-17 of the result. The
    weights' pair holds 2^-21 of each; the tensor core rounds its accumulators towards zero at each of a span's 128
    products of 16 keys, at most 2^-23 each, on average half: 2^-17."""
    P, gen = 64, torch.Generator(device="cuda").manual_seed(B)
    pages, g = -(-T // P), Hq // Hkv
    code = lambda: torch.randint(-127, 128, (B * pages, Hkv, P, 128), generator=gen, device="cuda", dtype=torch.int8)  # noqa: E731
    k8, v8 = code(), code()
    ks, vs = (torch.rand(B * pages, Hkv, P, generator=gen, device="cuda") / 40 + 0.005 for _ in range(2))
    table = torch.randperm(B * pages, generator=gen, device="cuda").int().view(B, pages)
    q = torch.randn(B, M, Hq, 128, generator=gen, device="cuda", dtype=torch.bfloat16)
    lens = torch.full((B,), T, dtype=torch.int32, device="cuda")
    masks = mask_tensor([[(1 << (i + 1)) - 1 for i in range(M)]] * B)
    out = torch.empty(B, M, Hq, 128, device="cuda")
    pg.decode_attn_paged_tree_int8(q, k8, v8, ks, vs, table, lens, masks, SCALE, out_f32=out,
                                   workspace=workspace(B, M, Hq, Hkv, P, pages))
    torch.cuda.synchronize()
    off = norm = 0.0
    for b in range(B):
        for h in range(Hkv):
            t = table[b].long()
            K = (k8[t, h].double() * ks[t, h].double()[..., None]).view(-1, 128)[:T]
            V = (v8[t, h].double() * vs[t, h].double()[..., None]).view(-1, 128)[:T]
            x = q[b, :, h * g:(h + 1) * g].double().reshape(-1, 128) @ K.t() * SCALE
            tail = torch.arange(M, device="cuda")
            hidden = (tail[None] > tail[:, None]).repeat_interleave(g, 0)
            x[:, T - M:] = x[:, T - M:].masked_fill(hidden, -math.inf)
            want = (torch.softmax(x, 1) @ V).view(M, g, 128)
            off += float((out[b, :, h * g:(h + 1) * g] - want).square().sum())
            norm += float(want.square().sum())
    assert math.sqrt(off / norm) < 2.0 ** -17
    assert pg.device_error_flags() == 0


def test_binding_refuses():
    c = Case(2850, [60], 8)
    d = c.upload()
    args = dict(q=d["q"], k_cache8=d["k8"], v_cache8=d["v8"], k_scale=d["ks"], v_scale=d["vs"], block_table=d["bt"],
                context_lens=d["cl"], tree_mask=d["mask"], scale=SCALE, out_f32=d["of"], workspace=d["ws"])
    pg.decode_attn_paged_tree_int8(**args)
    for name, bad in (("k_cache8", d["k8"].short()), ("v_cache8", d["v8"][:1]), ("k_scale", d["ks"].half()),
                      ("v_scale", d["vs"][..., :8]), ("q", d["q"].half()), ("tree_mask", d["mask"].int()),
                      ("out_f32", d["of"][:, :3]), ("k_scale", d["ks"].cpu()), ("slopes", d["ks"][0, 0, :3])):
        with pytest.raises((TypeError, ValueError)):
            pg.decode_attn_paged_tree_int8(**{**args, name: bad})
    if d["ws"].numel() > 16:
        with pytest.raises(pg.PgqaError):
            pg.decode_attn_paged_tree_int8(**{**args, "workspace": d["ws"][:16]})


# ------------------------------------------------------------------ prologue and read back
SECTIONS = [0] * 16 + [1] * 24 + [2] * 24


class Append:
    def __init__(self, seed, ctx, M, Hq=16, Hkv=8, P=16, new_lens=None, axes=SECTIONS, n_axes=3):
        gen = inputs.generator(seed, 601)
        B = len(ctx)
        kv = inputs.paged_kv(seed, ctx, Hkv=Hkv, page_size=P)
        self.table, self.lens = kv.block_table, kv.context_lens
        self.q, self.k, self.v = (inputs.normal_bf16(gen, (B, M, h, 128)) for h in (Hq, Hkv, Hkv))
        self.gq, self.gk = (inputs.uniform_bf16(gen, (128,), 0.5, 1.5) for _ in range(2))
        self.positions = gen.integers(0, 5000, (B, M, n_axes)).astype(np.int32)
        self.new_lens, self.n = new_lens, new_lens if new_lens is not None else [M] * B
        self.axes, self.M, self.P, self.Hkv = axes, M, P, Hkv
        self.pool = (kv.k_cache.shape[0], Hkv, P)

    def run(self, theta=THETA, eps=1e-6):
        """The INT8 prologue, and the bf16 one on caches of its own."""
        up = lambda x: to_device_bf16(x, "cuda")  # noqa: E731
        i32 = lambda x: to_device_i32(np.asarray(x), "cuda")  # noqa: E731
        nl = None if self.new_lens is None else i32(np.array(self.new_lens))
        given = (up(self.q), up(self.k), up(self.v), up(self.gq), up(self.gk), i32(self.positions), i32(self.lens),
                 i32(self.table))
        self.lens_d, self.table_d = given[6], given[7]
        self.k8, self.v8 = (torch.full((*self.pool, 128), 55, dtype=torch.int8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.full(self.pool, -3.0, device="cuda") for _ in range(2))
        self.q_out = torch.full(self.q.shape, SENTINEL, dtype=torch.bfloat16, device="cuda")
        pg.qk_norm_rope_append_axes_int8(*given, self.k8, self.v8, self.ks, self.vs, self.q_out, self.axes, theta, eps,
                                         new_lens=nl)
        flags = pg.device_error_flags(clear=True)
        self.kc, self.vc = (torch.full((*self.pool, 128), SENTINEL, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.q_bf16 = torch.full(self.q.shape, SENTINEL, dtype=torch.bfloat16, device="cuda")
        pg.qk_norm_rope_append_axes(*given, self.kc, self.vc, self.q_bf16, self.axes, theta, eps, new_lens=nl)
        torch.cuda.synchronize()
        assert pg.device_error_flags(clear=True) == flags
        return flags

    def check(self, flags=0, **kw):
        """The bytes are those of the quantized rows that the bf16 prologue appends (itself held to the formula), every
        other byte as it was."""
        assert self.run(**kw) == flags
        assert torch.equal(self.q_out, self.q_bf16)
        for rows, codes, scales in ((self.kc, self.k8, self.ks), (self.vc, self.v8, self.vs)):
            bits = bf16_bits(rows)
            written = (bits != bf16_bits(torch.tensor([SENTINEL]).bfloat16())[0]).any(-1)
            want, s = oracle.quantize_rows_int8(bits)
            again, t = ref.quantize(bf16_ref.widen(bits).astype(np.float32))
            assert np.array_equal(want, again) and np.array_equal(s, t)
            assert np.array_equal(codes.cpu().numpy(), np.where(written[..., None], want, 55))
            assert np.array_equal(scales.cpu().numpy(), np.where(written, s, np.float32(-3)))


@pytest.mark.parametrize("M", [1, 2, 7, 65, 300])
def test_prologue_lengths(M):
    Append(3000 + M, [M + 5, M, M + 300], M).check()


@pytest.mark.parametrize("Hq,Hkv,P", [(8, 8, 16), (24, 8, 64), (64, 8, 256), (4, 1, 32), (1, 1, 16), (5, 1, 128)])
def test_prologue_heads_and_pages(Hq, Hkv, P):
    Append(3010 + Hq, [P + 3, 9, 3 * P], 9, Hq=Hq, Hkv=Hkv, P=P).check()


@pytest.mark.parametrize("M,new_lens", [(460, None), (920, [920, 919, 0]), (1401, None), (2000, [3, 2000, 1999])])
def test_prologue_prompts(M, new_lens):
    """Token counts at which a block takes one, two and three tokens."""
    n = new_lens or [M] * 3
    Append(3020 + M, [x + 40 for x in n], M, new_lens=new_lens).check()


def test_prologue_ragged():
    Append(3030, [30, 12, 40, 7, 0], 12, new_lens=[0, 12, 5, 7, 0]).check()


def test_prologue_zero_tied_and_extreme_rows():
    """All-zero V rows have scale 0; halves between two codes go to the even one; the largest and smallest bf16."""
    c = Append(3040, [20], 8)
    c.v[0, 0] = 0
    c.k[0, 0] = 0
    c.v[0, 1] = inputs.f32_to_bf16_bits(np.tile(np.array([127.0, 0.5, 1.5, -2.5], np.float32), 32))
    c.v[0, 2] = 0x7F7F
    c.v[0, 3] = 0x0001
    c.v[0, 4, :, 1:] = 0
    c.v[0, 5] = inputs.f32_to_bf16_bits(np.linspace(-1e-38, 1e-38, 128, dtype=np.float32))
    c.check()


def test_prologue_flags():
    c = Append(3050, [60, 40, 50], 8, new_lens=[8, 9, 8])
    c.lens[2] = 7
    c.check(flags=binding.DEVERR_BAD_CONTEXT)
    c = Append(3051, [60, 40], 8)
    c.table[0, 3] = c.pool[0]
    c.check(flags=binding.DEVERR_BAD_PAGE)


@pytest.mark.parametrize("Hkv,P,N", [(1, 16, 5), (5, 64, 700), (8, 16, 33), (8, 256, 1), (70, 16, 9)])
def test_read_back(Hkv, P, N):
    """bf16(code scale), every bit; rows past a sequence's end and rows before `first` untouched."""
    ctx = [N + 3, max(1, N // 2), 0, 2 * P + 1]
    c = Case(3100 + N, ctx, 1, Hq=Hkv, Hkv=Hkv, P=P, draft_lens=[0] * 4)
    d = c.upload()
    for first in (None, [2, 0, 0, P - 1], [ctx[0], 5 * P, 0, 2 ** 31 - 1]):
        k, v = (torch.full((4, N, Hkv, 128), SENTINEL, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pg.kv_cache_read_int8(d["k8"], d["v8"], d["ks"], d["vs"], d["bt"], d["cl"], k, v,
                              first=None if first is None else to_device_i32(np.array(first), "cuda"))
        torch.cuda.synchronize()
        assert pg.device_error_flags() == 0
        for out, codes, scales in ((k, c.k8, c.ks), (v, c.v8, c.vs)):
            for b in range(4):
                f = 0 if first is None else first[b]
                T = ctx[b]
                have = max(0, min(N, T - f))
                assert (out[b, have:] == SENTINEL).all()
                if have:
                    x = ref.rows_of(codes, c.table[b], T, P).astype(np.float32) * ref.rows_of(scales, c.table[b], T, P)[..., None]
                    want = torch.from_numpy(x[:, f:f + have]).bfloat16().transpose(0, 1)
                    assert torch.equal(out[b, :have].cpu(), want)


def test_read_back_flags():
    c = Case(3150, [60, 40, 33], 1, draft_lens=[0] * 3)
    c.lens[0] = c.max_pages * 16 + 1
    c.table[2, 1] = -1
    d = c.upload()
    k, v = (torch.full((3, 40, 8, 128), SENTINEL, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pg.kv_cache_read_int8(d["k8"], d["v8"], d["ks"], d["vs"], d["bt"], d["cl"], k, v,
                          first=to_device_i32(np.array([0, -1, 0]), "cuda"))
    torch.cuda.synchronize()
    assert pg.device_error_flags() == binding.DEVERR_BAD_PAGE | binding.DEVERR_BAD_CONTEXT
    assert (k[:2] == SENTINEL).all() and (v[:2] == SENTINEL).all()
    assert (k[2, 16:32] == SENTINEL).all() and (k[2, :16] != SENTINEL).any() and (k[2, 32] != SENTINEL).any()


def test_append_then_read_back_on_another_stream_and_in_a_graph():
    c = Append(3160, [90, 40], 30)
    c.run()
    side = torch.cuda.Stream()
    k, v = (torch.zeros((2, 90, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    side.wait_stream(torch.cuda.current_stream())
    pg.kv_cache_read_int8(c.k8, c.v8, c.ks, c.vs, c.table_d, c.lens_d, k, v, stream=side)
    side.synchronize()
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pg.kv_cache_read_int8(c.k8, c.v8, c.ks, c.vs, c.table_d, c.lens_d, k2, v2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(k, k2) and torch.equal(v, v2)
    want = c.k8.float() * c.ks[..., None]
    page, off = int(c.table[0, 80 // 16]), 80 % 16
    assert torch.equal(k[0, 80], want[page, :, off].bfloat16())


# ------------------------------------------------------------------ commit
def commit_case(seed, L, ctx, n, M, paths, Hkv=8, P=16, keep=lambda b: True):
    """(layers' host arrays, expected, device arrays) of a commit."""
    gen = np.random.default_rng(seed)
    B, A = len(ctx), max(1, max(len(p) for p in paths))
    layers, dev = [], []
    for _ in range(L):
        kv = inputs.paged_kv(seed + len(layers), ctx, Hkv=Hkv, page_size=P)
        shape = kv.k_cache.shape
        host = [gen.integers(-128, 128, shape).astype(np.int8) for _ in range(2)]
        host += [gen.normal(size=shape[:3]).astype(np.float32) for _ in range(2)]
        layers.append((host, kv.block_table))
        dev.append(([torch.from_numpy(x.copy()).cuda() for x in host], to_device_i32(kv.block_table, "cuda")))
    expected = []
    for host, table in layers:
        new = [x.copy() for x in host]
        for b in range(B):
            if not keep(b):
                continue
            base = ctx[b] - n[b]
            for i, e in enumerate(paths[b]):
                s, t = base + e, base + i
                for x, y in zip(host, new):
                    y[table[b, t // P], :, t % P] = x[table[b, s // P], :, s % P]
        expected.append(new)
    path = np.full((B, A), -5, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    i32 = lambda x: to_device_i32(np.array(x), "cuda")  # noqa: E731
    args = dict(layers=pg.CacheLayersInt8(*[[d[0][k] for d in dev] for k in range(4)], [d[1] for d in dev]),
                context_lens=i32(ctx), path=i32(path), path_lens=i32([len(p) for p in paths]),
                context_lens_out=torch.zeros(B, dtype=torch.int32, device="cuda"), M=M, draft_lens=i32(n))
    return dev, expected, args


def check_commit(dev, expected, args, lens):
    pg.kv_cache_commit_path_int8(**args)
    torch.cuda.synchronize()
    assert args["context_lens_out"].tolist() == lens
    for (got, _), want in zip(dev, expected):
        for x, y in zip(got, want):
            assert np.array_equal(x.cpu().numpy(), y)


def test_commit_paths():
    n = [8, 8, 16, 16, 5]
    paths = [[], [0, 1, 2], [0, 3, 4, 9, 15], [15], [0, 2]]
    ctx = [30, 40, 100, 47, 33]
    check_commit(*commit_case(3200, 3, ctx, n, 16, paths), [c - m + len(p) for c, m, p in zip(ctx, n, paths)])
    assert pg.device_error_flags() == 0


def test_commit_long_paths_cross_chunks():
    paths = [list(range(1, 64)), [0] + list(range(2, 64)), list(range(0, 64, 2))]
    ctx = [64, 90, 200]
    check_commit(*commit_case(3210, 2, ctx, [64] * 3, 64, paths, Hkv=3), [c - 64 + len(p) for c, p in zip(ctx, paths)])


@pytest.mark.parametrize("L,B", [(1, 1), (28, 1), (2, 90), (128, 3)])
def test_commit_of_layers_and_sequences(L, B):
    gen = np.random.default_rng(L)
    n = [int(gen.integers(1, 13)) for _ in range(B)]
    paths = [sorted(gen.choice(m, int(gen.integers(0, m + 1)), replace=False).tolist()) for m in n]
    ctx = [m + int(gen.integers(0, 40)) for m in n]
    check_commit(*commit_case(3220 + L, L, ctx, n, 12, paths, Hkv=2), [c - m + len(p) for c, m, p in zip(ctx, n, paths)])


def test_commit_bad_paths_and_lengths_move_nothing():
    paths = [[0, 2, 2], [1, 0], [0, 8], [0, 1, 3], [0, 5]]
    ctx, n = [40, 40, 40, 40, 3], [8, 8, 8, 8, 4]
    check_commit(*commit_case(3230, 2, ctx, n, 8, paths, keep=lambda b: b == 3), [32, 32, 32, 35, 3])
    assert pg.device_error_flags() == binding.DEVERR_BAD_PATH | binding.DEVERR_BAD_CONTEXT


# ------------------------------------------------------------------ whole steps
def test_steps_match_token_by_token_decoding():
    """Prologue, tree attention, verification and commit over INT8 caches, three times and captured as one graph: the
    accepted path's outputs, and the committed codes and scales, are those of decoding its tokens one after another with
    qk_norm_rope_append_axes_int8 and single-token trees."""
    gen = np.random.default_rng(3300)
    B, M, Hq, Hkv, P, L, V = 3, 6, 8, 2, 16, 2, 50
    base = [37, 5, 64]
    max_pages, A = 12, 4
    table = torch.randperm(B * max_pages, generator=torch.Generator().manual_seed(1)).int().view(B, max_pages).cuda()
    gq, gk = (to_device_bf16(inputs.uniform_bf16(gen, (128,), 0.5, 1.5), "cuda") for _ in range(2))
    axes = [0] * 64
    embed = torch.from_numpy(gen.normal(size=(L, V, Hq + 2 * Hkv, 128))).to(torch.bfloat16).cuda()  # a token's heads

    def caches():
        c = []
        for _ in range(L):
            k8, v8 = (torch.zeros(B * max_pages, Hkv, P, 128, dtype=torch.int8, device="cuda") for _ in range(2))
            ks, vs = (torch.zeros(B * max_pages, Hkv, P, device="cuda") for _ in range(2))
            c.append((k8, v8, ks, vs))
        return c

    def heads(layer, tokens):
        x = embed[layer][tokens.long()]
        return x[..., :Hq, :].contiguous(), x[..., Hq:Hq + Hkv, :].contiguous(), x[..., Hq + Hkv:, :].contiguous()

    def append(c, layer, tokens, positions, lens):
        q, k, v = heads(layer, tokens)
        q_out = torch.empty_like(q)
        pg.qk_norm_rope_append_axes_int8(q, k, v, gq, gk, positions, lens, table, *c[layer], q_out, axes, THETA)
        return q_out

    tree, plain = caches(), caches()
    prompt = torch.from_numpy(gen.integers(0, V, (B, max(base)))).int().cuda()
    for b in range(B):  # prompts, with their own lengths
        for c in (tree, plain):
            for layer in range(L):
                lens = torch.zeros(B, dtype=torch.int32, device="cuda")
                lens[b] = base[b]
                new = lens.clone()
                q, k, v = heads(layer, prompt)
                pos = torch.arange(max(base), dtype=torch.int32, device="cuda")[None, :, None].expand(B, -1, 1).contiguous()
                pg.qk_norm_rope_append_axes_int8(q, k, v, gq, gk, pos, lens, table, *c[layer], torch.empty_like(q), axes,
                                                 THETA, new_lens=new)
    parents = torch.tensor([[-1, 0, 0, 1, 2, 4]] * B, dtype=torch.int32, device="cuda")
    depth = torch.tensor([0, 1, 1, 2, 2, 3], device="cuda")
    masks = mask_tensor([[1, 3, 5, 11, 21, 53]] * B)
    layers = pg.CacheLayersInt8(*[[c[k] for c in tree] for k in range(4)], [table] * L)
    state = dict(tokens=torch.from_numpy(gen.integers(0, V, (B, M))).int().cuda(),
                 target=torch.empty(B, M, V, device="cuda"), u=torch.empty(B, M, device="cuda"),
                 noise=torch.empty(B, V, device="cuda"), lens=torch.tensor(base, dtype=torch.int32, device="cuda"))
    out = [torch.zeros(B, M, Hq, 128, device="cuda") for _ in range(L)]
    ws = workspace(B, M, Hq, Hkv, P, max_pages)
    vws = torch.empty(max(16, pg.verify_drafted_tree_workspace_size(B, M, V)), dtype=torch.uint8, device="cuda")
    temps = torch.tensor([0.9, 0.0, 1.2], device="cuda")
    path, new_tokens = (torch.zeros(B, A, dtype=torch.int32, device="cuda") for _ in range(2))
    plens, lens_out = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    lens_in, positions = torch.zeros_like(plens), torch.zeros(B, M, 1, dtype=torch.int32, device="cuda")

    def step():
        torch.add(state["lens"], M, out=lens_in)
        positions.copy_((state["lens"][:, None] + depth[None])[..., None])
        for layer in range(L):
            q = append(tree, layer, state["tokens"], positions, lens_in)
            pg.decode_attn_paged_tree_int8(q, *tree[layer], table, lens_in, masks, SCALE, out_f32=out[layer], workspace=ws)
        pg.verify_drafted_tree(state["target"], state["tokens"], parents, temps, state["u"], state["noise"], path, plens,
                               new_tokens, workspace=vws)
        pg.kv_cache_commit_path_int8(layers, lens_in, path, plens, lens_out, M)
        state["lens"].copy_(lens_out)

    graph, lengths = None, list(base)
    accepted = 0
    for turn in range(3):
        state["target"].copy_(torch.from_numpy(gen.normal(0, 1.5, (B, M, V))))
        tokens = gen.integers(0, V, (B, M)).astype(np.int32)
        best = state["target"].argmax(-1).cpu().numpy()
        for b in range(B):  # drafts that the greedy sequence accepts too
            for i in range(1, M):
                if gen.random() < 0.7:
                    tokens[b, i] = best[b, int(parents[b, i])]
        state["tokens"].copy_(torch.from_numpy(tokens))
        state["u"].copy_(torch.from_numpy(gen.random((B, M)) * 0.3))
        state["noise"].copy_(torch.from_numpy(gen.exponential(size=(B, V)) + 1e-20))
        if turn == 1:
            before = [[x.clone() for x in c] for c in tree] + [state["lens"].clone()]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for c, saved in zip(tree, before):
                for x, y in zip(c, saved):
                    x.copy_(y)
            state["lens"].copy_(before[-1])
        graph.replay() if graph else step()
        torch.cuda.synchronize()
        t64 = state["target"].double().cpu().numpy()
        for b in range(B):
            want = ref.verify(t64[b], None, tokens[b].tolist(), parents[b].tolist(), M, float(temps[b]),
                              state["u"][b].double().cpu().numpy(), state["noise"][b].cpu().numpy(), A)
            assert want[3] > 1e-4 and path[b, :len(want[0])].tolist() == want[0] and int(plens[b]) == len(want[0])
            assert new_tokens[b, :len(want[1])].tolist() == want[1]
            # the same tokens one after another
            for i, node in enumerate(want[0]):
                lens = torch.zeros(B, dtype=torch.int32, device="cuda")
                lens[b] = lengths[b] + 1
                one = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
                one[b] = int(tokens[b, node])
                only = torch.zeros(B, dtype=torch.int32, device="cuda")
                only[b] = 1
                for layer in range(L):
                    q, k, v = heads(layer, one)
                    q_out, o = torch.empty_like(q), torch.empty(B, 1, Hq, 128, device="cuda")
                    pg.qk_norm_rope_append_axes_int8(q, k, v, gq, gk, (lens - 1)[:, None, None].contiguous(), lens, table,
                                                     *plain[layer], q_out, axes, THETA, new_lens=only)
                    pg.decode_attn_paged_tree_int8(q_out, *plain[layer], table, lens, mask_tensor([[1]] * B), SCALE,
                                                   draft_lens=only, out_f32=o,
                                                   workspace=workspace(B, 1, Hq, Hkv, P, max_pages))
                    # fp32 sums in another order over rows of N(0, 1): well under 1e-5
                    assert float((o[b, 0] - out[layer][b, node]).abs().max()) < 1e-5
                lengths[b] += 1
            assert int(state["lens"][b]) == lengths[b]
            accepted += len(want[0]) - 1
        for layer in range(L):
            for b in range(B):
                for x, y in zip(tree[layer], plain[layer]):
                    for s in range(lengths[b]):
                        page, off = int(table[b, s // P]), s % P
                        assert torch.equal(x[page, :, off], y[page, :, off])
    assert accepted >= 5
    assert pg.device_error_flags() == 0
