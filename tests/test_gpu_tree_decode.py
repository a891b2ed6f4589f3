"""Drafted-tree decoding on the GPU against 64-bit references: the prologue with several position axes,
attention of a drafted tree, the commit of the accepted path, and a verification step of all three."""
import math

import numpy as np
import pytest
import torch

import paged_gqa_decode_head_gb300 as pg
import tree_reference as ref
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


def mask_tensor(masks, device="cuda"):
    a = np.array([[int(m) & (2 ** 64 - 1) for m in row] for row in masks], dtype=np.uint64)
    return torch.from_numpy(a.view(np.int64)).to(device)


def workspace(B, M, Hq, Hkv, P, max_pages):
    n = pg.decode_attn_tree_workspace_size(B, M, Hq, Hkv, 128, P, max_pages)
    return torch.full((max(16, n),), 0xA5, dtype=torch.uint8, device="cuda")  # any contents


class Case:
    """Inputs of one attention call, on the host and on the GPU."""

    def __init__(self, seed, ctx, M, Hq=16, Hkv=8, P=16, draft_lens=None, masks=None, softcap=0.0, slopes=None,
                 roots=1, **kv_args):
        gen = inputs.generator(seed, 301)
        self.B, self.M, self.Hq, self.Hkv, self.P = len(ctx), M, Hq, Hkv, P
        self.kv = inputs.paged_kv(seed, ctx, Hkv=Hkv, page_size=P, **kv_args)
        self.q = inputs.normal_bf16(gen, (self.B, M, Hq, 128))
        self.n = list(draft_lens) if draft_lens is not None else [M] * self.B
        self.draft_lens = draft_lens
        trees = [ref.random_tree(gen, M, roots) for _ in range(self.B)]
        self.masks = masks if masks is not None else [t[0] for t in trees]
        self.positions = np.array([[ctx[b] - self.n[b] + d for d in trees[b][1]] for b in range(self.B)], np.int32)
        self.softcap, self.slopes = softcap, None if slopes is None else np.asarray(slopes, np.float32)
        self.scale = SCALE

    def upload(self):
        kv = self.kv
        self.d = dict(q=to_device_bf16(self.q, "cuda"), kc=to_device_bf16(kv.k_cache, "cuda"),
                      vc=to_device_bf16(kv.v_cache, "cuda"), bt=to_device_i32(kv.block_table, "cuda"),
                      cl=to_device_i32(kv.context_lens, "cuda"), mask=mask_tensor(self.masks),
                      pos=to_device_i32(self.positions, "cuda"),
                      dl=None if self.draft_lens is None else to_device_i32(np.array(self.draft_lens), "cuda"),
                      slopes=None if self.slopes is None else torch.from_numpy(self.slopes).cuda(),
                      ws=workspace(self.B, self.M, self.Hq, self.Hkv, self.P, kv.max_pages),
                      of=torch.full(self.q.shape, SENTINEL, dtype=torch.float32, device="cuda"),
                      ob=torch.full(self.q.shape, SENTINEL, dtype=torch.bfloat16, device="cuda"))
        return self.d

    def launch(self, stream=None, f32=True, bf16=True):
        d = self.d
        pg.decode_attn_paged_tree(d["q"], d["kc"], d["vc"], d["bt"], d["cl"], d["mask"], self.scale,
                                  positions=d["pos"], draft_lens=d["dl"], slopes=d["slopes"], softcap=self.softcap,
                                  out_f32=d["of"] if f32 else None, out_bf16=d["ob"] if bf16 else None,
                                  workspace=d["ws"], stream=stream)

    def run(self):
        self.upload()
        self.launch()
        torch.cuda.synchronize()
        return self.d["of"].cpu().numpy(), self.d["ob"].float().cpu().numpy()

    def reference(self, **kw):
        kv = self.kv
        return ref.attention(self.q, kv.k_cache, kv.v_cache, kv.block_table, kv.context_lens, self.masks, self.scale,
                             self.n, self.positions, self.slopes, self.softcap, **kw)

    def check(self, flags=0, **kw):
        of, ob = self.run()
        out, bound = self.reference(**kw)
        check_outputs(of, ob, out, bound, self.n)
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
    """One token up to several tiles, drafted tokens inside a page, a tile or across either's end."""
    for M in (1, 2, 8, 17):
        if M <= T:
            Case(1000 + 37 * T + M, [T, T + 3], M).check()


@pytest.mark.parametrize("T", [64, 65, 128, 150, 192, 330])
def test_widest_trees(T):
    Case(1100 + T, [T, T + 1], 64, Hkv=2, Hq=4, roots=3).check()


@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("M", [1, 5, 33, 64])
def test_group_sizes(g, M):
    """Query rows per KV head from 1 to 512: every number of row tiles, groups that do not divide a tile."""
    Case(1200 + 10 * g + M, [M + 140, M + 17], M, Hq=2 * g, Hkv=2).check()


@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
def test_page_sizes(P):
    Case(1300 + P, [3 * P + 5, 700, P, P + 1], 12, P=P).check()


@pytest.mark.parametrize("B,T", [(1, 4000), (3, 1500), (40, 260), (300, 40)])
def test_work_split(B, T):
    """One sequence over many SMs, many sequences per SM, ragged lengths."""
    gen = inputs.generator(1400 + B, 5)
    ctx = [int(x) for x in gen.integers(8, T + 1, B)]
    ctx[0] = T
    Case(1400 + B, ctx, 8, Hq=4, Hkv=2).check()


def test_ragged_drafts_leave_other_rows_alone():
    n = [0, 1, 5, 16, 9, 16]
    Case(1500, [300, 1, 5, 16, 200, 129], 16, draft_lens=n).check()


def test_empty_sequence_beside_others():
    """T = 0 with no drafted token: nothing to do, nothing written."""
    Case(1510, [0, 40, 0], 4, draft_lens=[0, 4, 0]).check()


def test_rows_that_see_nothing_are_zero():
    """No prefix and an empty mask; masks with only bits past n_b; beside rows that see something."""
    masks = [[0, 2, 0, 8, 1 << 40, 0xF, 0xF0, 1]]
    of = Case(1520, [6], 8, draft_lens=[6], masks=masks).check()
    assert (of[0, 0] == 0).all() and (of[0, 4] == 0).all()


def test_masks_need_not_be_trees():
    """Any bits: later tokens, not itself, all 64."""
    gen = inputs.generator(1530, 6)
    masks = [[int(gen.integers(0, 2 ** 63)) * 2 + int(gen.integers(0, 2)) for _ in range(64)] for _ in range(2)]
    masks[0][0], masks[0][1], masks[0][63] = 2 ** 64 - 1, 1 << 63, 1
    Case(1530, [64, 190], 64, Hq=4, Hkv=2, masks=masks).check()


@pytest.mark.parametrize("T", [40, 128, 135, 400])
def test_nonfinite_rows_reach_only_the_tokens_that_see_them(T):
    """K and V rows of drafted tokens with NaN and infinities: tokens whose masks leave them out get their
    result as if those rows held numbers; tokens that see one get what the formula gives, not finite."""
    M = 16
    c = Case(1540 + T, [T], M, Hq=8, Hkv=4)
    bad = {3: 0x7FC0, 7: 0x7F80, 12: 0xFF80}  # NaN, +inf, -inf
    masks = c.masks[0]
    kv = c.kv
    clean_k, clean_v = kv.k_cache.copy(), kv.v_cache.copy()
    for j, bits in bad.items():
        s = T - M + j
        page, off = kv.block_table[0, s // 16], s % 16
        kv.v_cache[page, :, off, 5] = bits
        kv.v_cache[page, :, off, 77] = bits
        if j != 7:
            kv.k_cache[page, :, off, 9] = bits
    of, ob = c.run()
    kv.k_cache, kv.v_cache = clean_k, clean_v
    out, bound = c.reference()
    sees = [[j for j in bad if masks[i] >> j & 1] for i in range(M)]
    assert any(sees) and not all(sees)
    for i in range(M):
        if not sees[i]:
            assert np.isfinite(of[0, i]).all()
            assert (np.abs(of[0, i] - out[0, i]) <= bound[0, i] + 2.0 ** -24 * np.abs(out[0, i])).all(), i
        elif sees[i] == [7]:  # +inf in V, a number in K: infinite where V is, numbers elsewhere
            assert (of[0, i, :, 5] == np.inf).all() and (of[0, i, :, 77] == np.inf).all()
            rest = [d for d in range(128) if d not in (5, 77)]
            assert (np.abs(of[0, i] - out[0, i])[:, rest] <= (bound[0, i] + 2.0 ** -24 * np.abs(out[0, i]))[:, rest]).all()
        else:
            assert not np.isfinite(of[0, i][:, [5, 77]]).any()


@pytest.mark.parametrize("softcap", [1e-3, 0.5, 5.0, 30.0, 1e4, 3e38])
def test_capped_scores(softcap):
    """Scores far past the cap, around it and far below it."""
    c = Case(1600, [300, 77], 9, softcap=softcap)
    c.kv.k_cache[...] = scaled(c.kv.k_cache, 6.0)
    c.check()


def scaled(bits, f):
    out = inputs.f32_to_bf16_bits((ref.widen(bits) * f).astype(np.float32)).reshape(bits.shape)
    return np.where((bits & 0x7FFF) > 0x7F80, bits, out).astype(np.uint16)


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("M", [1, 12])
def test_distance_bias(M, softcap):
    """Slopes of both signs and zero; drafted tokens at the positions that were given."""
    slopes = [2.0 ** -(h / 2) * (-1 if h % 5 == 4 else 1) for h in range(16)]
    slopes[3] = 0.0
    Case(1610 + M, [900, 64, 333], M, slopes=slopes, softcap=softcap, roots=min(2, M)).check()


def test_peaked_scores_rescale_the_state():
    """Scores that keep growing along the keys: the running maximum moves in every tile."""
    c = Case(1620, [900], 4, Hq=4, Hkv=2)
    T, P = 900, 16
    f = np.linspace(0.0, 40.0, T)
    for j in range(T):
        page, off = c.kv.block_table[0, j // P], j % P
        for h in range(2):
            direction = ref.widen(c.q[0, 0, 2 * h])
            row = direction * (f[j] / np.linalg.norm(direction))
            c.kv.k_cache[page, h, off] = inputs.f32_to_bf16_bits(row.astype(np.float32))
    c.check()


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-30])
def test_scales(scale):
    c = Case(1630, [200], 6)
    c.scale = scale
    c.check()


def test_very_low_scores_are_still_a_softmax():
    """All scores far below any start value of a running maximum: -1e35."""
    c = Case(1640, [5], 1, Hq=2, Hkv=1)
    c.q[...] = inputs.f32_to_bf16_bits(np.full(c.q.shape, 1e17, np.float32))
    c.kv.k_cache[...] = inputs.f32_to_bf16_bits(np.full(c.kv.k_cache.shape, -1e17, np.float32))
    c.scale = 0.1
    of, _ = c.run()
    V = ref.widen(ref.gather(c.kv.v_cache, c.kv.block_table[0], 5, 16))[0]
    np.testing.assert_allclose(of[0, 0, 0], V.mean(0), atol=1e-4)


def test_pages_outside_the_pool_are_skipped():
    c = Case(1700, [500, 100], 6)
    table = c.kv.block_table
    table[0, 3], table[0, 10], table[1, 6] = -1, c.kv.num_pages, 2 ** 31 - 1
    gone = {(0, 3), (0, 10), (1, 6)}
    c.check(flags=binding.DEVERR_BAD_PAGE, skip=lambda b, j: (b, j // 16) in gone)


def test_bad_lengths_give_zeros_and_a_flag():
    c = Case(1710, [60, 40, 50, 30], 8, draft_lens=[8, 8, 8, 4])
    c.kv.context_lens[1] = 7                                  # T < n
    c.kv.context_lens[3] = c.kv.max_pages * 16 + 1            # longer than the table
    c.draft_lens = c.n = [8, 8, 9, 4]                         # n > M
    of, ob = c.run()
    assert pg.device_error_flags() == binding.DEVERR_BAD_CONTEXT
    for b in (1, 2, 3):
        assert (of[b] == 0).all() and (ob[b] == 0).all()
    one = Case(1710, [60, 40, 50, 30], 8, draft_lens=[8, 8, 8, 4])
    out, bound = one.reference()
    assert (np.abs(of[0] - out[0]) <= bound[0] + 2.0 ** -24 * np.abs(out[0])).all()


def test_negative_lengths():
    c = Case(1720, [60, 40], 8, draft_lens=[8, 8])
    c.kv.context_lens[0] = -5
    c.draft_lens = c.n = [8, -1]
    of, _ = c.run()
    assert pg.device_error_flags() == binding.DEVERR_BAD_CONTEXT
    assert (of == 0).all()


def test_outputs_alone_and_together_agree():
    c = Case(1730, [400], 7)
    of, ob = c.run()
    c.upload()
    c.launch(f32=False)
    torch.cuda.synchronize()
    assert np.array_equal(c.d["ob"].float().cpu().numpy(), ob) and (c.d["of"] == SENTINEL).all()
    c.upload()
    c.launch(bf16=False)
    torch.cuda.synchronize()
    assert np.array_equal(c.d["of"].cpu().numpy(), of) and (c.d["ob"] == SENTINEL).all()


def test_chain_masks_match_the_multi_query_decode():
    """Causal masks: the same attention as decode_attn_paged_multi."""
    M, ctx = 4, [40, 17, 600]
    c = Case(1740, ctx, M, masks=[[(1 << (i + 1)) - 1 for i in range(M)]] * 3)
    of, _ = c.run()
    d = c.d
    n = pg.decode_attn_multi_workspace_size(3, M, 16, 8, 128, 16, c.kv.max_pages, 0)
    other = torch.empty_like(d["of"])
    pg.decode_attn_paged_multi(d["q"], d["kc"], d["vc"], d["bt"], d["cl"], SCALE, out_f32=other,
                               workspace=torch.zeros(max(16, n), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    out, bound = c.reference()
    assert (np.abs(of - other.cpu().numpy()) <= 2 * bound + 2.0 ** -23 * np.abs(out)).all()


def test_repeated_calls_and_a_used_workspace_give_the_same_bits():
    c = Case(1750, [2000, 30, 700], 16)
    of, _ = c.run()
    other = Case(1751, [90], 16)
    other.upload()
    other.d["ws"] = c.d["ws"]
    other.launch()
    for _ in range(3):
        c.d["of"].fill_(SENTINEL)
        c.launch()
        torch.cuda.synchronize()
        assert np.array_equal(c.d["of"].cpu().numpy(), of)


def test_two_streams_at_once_with_workspaces_of_their_own():
    a, b = Case(1760, [3000], 16), Case(1761, [2500, 800], 9)
    ra, rb = a.run()[0], b.run()[0]
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a.launch(stream=sa)
        b.launch(stream=sb)
    torch.cuda.synchronize()
    assert np.array_equal(a.d["of"].cpu().numpy(), ra) and np.array_equal(b.d["of"].cpu().numpy(), rb)


def test_captured_call_follows_lengths_masks_and_drafts():
    """A replay reads the lengths, masks, tables and drafted counts of its own time."""
    c = Case(1770, [700, 300], 16, draft_lens=[16, 16])
    c.upload()
    c.launch()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.launch()
    for ctx, n in (([650, 17], [3, 16]), ([30, 299], [16, 0]), ([700, 300], [16, 16])):
        c.kv.context_lens[:] = ctx
        c.n = c.draft_lens = n
        c.positions[:] = np.array(ctx)[:, None] - np.array(n)[:, None] + np.arange(16)[None] % 5
        c.d["cl"].copy_(to_device_i32(c.kv.context_lens, "cuda"))
        c.d["dl"].copy_(to_device_i32(np.array(n), "cuda"))
        c.d["pos"].copy_(to_device_i32(c.positions, "cuda"))
        c.d["of"].fill_(SENTINEL), c.d["ob"].fill_(SENTINEL)
        g.replay()
        torch.cuda.synchronize()
        # shorter contexts end inside pages whose later slots hold the old numbers: they are not seen
        out, bound = c.reference()
        check_outputs(c.d["of"].cpu().numpy(), c.d["ob"].float().cpu().numpy(), out, bound, n)


def test_a_pool_past_32_bit_offsets():
    """Pages whose elements lie past 2^31 (and bytes past 2^32) in the pool."""
    P, Hkv, M, T = 256, 8, 5, 700
    c = Case(1780, [T], M, Hq=8, Hkv=Hkv, P=P)
    pages = (1 << 31) // (P * Hkv * 128) + 64  # > 2^31 elements per cache
    c.upload()
    kc = torch.zeros((pages, Hkv, P, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    far = [pages - 1, pages - 9, pages - 2]
    for i, page in enumerate(far):
        kc[page] = c.d["kc"][int(c.kv.block_table[0, i])]
        vc[page] = c.d["vc"][int(c.kv.block_table[0, i])]
    c.d["kc"], c.d["vc"] = kc, vc
    c.d["bt"] = to_device_i32(np.array([far]), "cuda")
    c.launch()
    torch.cuda.synchronize()
    out, bound = c.reference()
    check_outputs(c.d["of"].cpu().numpy(), c.d["ob"].float().cpu().numpy(), out, bound, c.n)


def test_one_long_context():
    c = Case(1790, [40000], 3, Hq=2, Hkv=1, softcap=30.0, slopes=[0.5, 0.001])
    c.check()


@pytest.mark.parametrize("seed", range(24))
def test_random_calls(seed):
    """Sizes, lengths, heads, options and masks drawn together."""
    gen = inputs.generator(1800 + seed, 7)
    pick = lambda *x: x[int(gen.integers(0, len(x)))]  # noqa: E731
    g, Hkv, P, M = pick(1, 2, 3, 5, 8), pick(1, 2, 3), pick(16, 32, 64, 128, 256), int(gen.integers(1, 65))
    B = int(gen.integers(1, 9))
    n = [int(gen.integers(0, M + 1)) for _ in range(B)]
    ctx = [x + int(pick(0, 1, gen.integers(0, 40), gen.integers(0, 700))) for x in n]
    slopes = [float(x) for x in gen.normal(0, 0.2, g * Hkv)] if gen.random() < 0.4 else None
    masks = None
    if gen.random() < 0.4:
        masks = [[int(gen.integers(0, 2 ** 62)) << int(gen.integers(0, 3)) for _ in range(M)] for _ in range(B)]
    Case(1800 + seed, ctx, M, Hq=g * Hkv, Hkv=Hkv, P=P, draft_lens=n, masks=masks, slopes=slopes,
         softcap=float(pick(0.0, 0.0, 8.0)), max_pages=max(1, -(-max(ctx) // P) + int(gen.integers(0, 5)))).check()


def test_more_sequences_than_threads():
    """Several sequences per thread of the schedule's scan, empty ones among them."""
    gen = inputs.generator(1830, 8)
    n = [int(gen.integers(0, 3)) for _ in range(900)]
    ctx = [x + (int(gen.integers(0, 300)) if x else 0) for x in n]
    Case(1830, ctx, 2, Hq=2, Hkv=1, draft_lens=n).check()


@pytest.mark.parametrize("B,M,Hq,Hkv,T,rising", [(4, 2, 8, 8, 90000, False), (3, 40, 32, 8, 40000, False),
                                                 (2, 3, 4, 4, 120000, True)])
def test_long_contexts_keep_fp32_outputs(B, M, Hq, Hkv, T, rising):
    """Many tiles per CTA and stream, one and two row tiles, scores that rise along the keys; against the formula in
    64 bits on the GPU. The weights are within 2^-18 (hi + lo); the tensor core's accumulators lose at most one unit
    in the last place (2^-23) at each of the 256 products of a span, half of that on average: 2^-16."""
    P, g = 64, torch.Generator(device="cuda").manual_seed(B)
    pages = -(-T // P)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    kc, vc = rand(B * pages, Hkv, P, 128), rand(B * pages, Hkv, P, 128)
    q = rand(B, M, Hq, 128)
    bt = torch.randperm(B * pages, generator=g, device="cuda").to(torch.int32).view(B, pages)
    if rising:  # along the queries' mean direction, in steps that move the running reference now and then
        for b in range(B):
            d = q[b].float().view(M, Hkv, -1, 128).mean((0, 2))
            up = torch.linspace(0, 25, pages, device="cuda")[:, None, None, None] / 11.3
            kc[bt[b].long()] = (kc[bt[b].long()].float() + up * d[None, :, None]).bfloat16()
    lens = [T - 1000 * b for b in range(B)]
    of = torch.empty((B, M, Hq, 128), dtype=torch.float32, device="cuda")
    masks = [[(1 << (i + 1)) - 1 for i in range(M)]] * B
    pg.decode_attn_paged_tree(q, kc, vc, bt, to_device_i32(np.array(lens), "cuda"), mask_tensor(masks), SCALE,
                              out_f32=of, workspace=workspace(B, M, Hq, Hkv, P, pages))
    torch.cuda.synchronize()
    for b in range(B):
        n = lens[b]
        k = kc[bt[b].long()].transpose(0, 1).reshape(Hkv, -1, 128)[:, :n].double()
        v = vc[bt[b].long()].transpose(0, 1).reshape(Hkv, -1, 128)[:, :n].double()
        seen = torch.ones(M, n, dtype=torch.bool, device="cuda")
        seen[:, n - M:] = torch.tril(torch.ones(M, M, device="cuda")).bool()
        for h in range(Hq):
            x = (q[b, :, h].double() @ k[h // (Hq // Hkv)].t() * SCALE).masked_fill(~seen, -math.inf)
            want = torch.softmax(x, -1) @ v[h // (Hq // Hkv)]
            rel = ((of[b, :, h].double() - want).norm() / want.norm()).item()
            assert rel <= 2.0 ** -18 + 2.0 ** -16, (b, h, rel)
    assert pg.device_error_flags() == 0


@pytest.mark.parametrize("g,T", [(4, 3000), (8, 2000), (5, 1500)])
def test_wide_trees_over_many_pieces(g, T):
    """Two and more row tiles per KV head, every head split over several CTAs."""
    Case(1840 + g, [T], 64, Hq=g, Hkv=1).check()


@pytest.mark.parametrize("T", [64, 200, 1000])
def test_nonfinite_rows_with_two_row_tiles(T):
    M = 64
    c = Case(1850 + T, [T, T + 7], M, Hq=8, Hkv=2)
    kv = c.kv
    clean = kv.v_cache.copy()
    for b in range(2):
        s = int(kv.context_lens[b]) - M + 20
        kv.v_cache[kv.block_table[b, s // 16], :, s % 16, 3] = 0x7F80
    of, _ = c.run()
    kv.v_cache = clean
    out, bound = c.reference()
    for b in range(2):
        for i in range(M):
            if c.masks[b][i] >> 20 & 1:
                assert (of[b, i, :, 3] == np.inf).all()
            else:
                assert (np.abs(of[b, i] - out[b, i]) <= bound[b, i] + 2.0 ** -24 * np.abs(out[b, i])).all()


def test_binding_refuses():
    """Wrong dtype, shape, layout or device of a tensor: an error that names it, nothing launched."""
    c = Case(1860, [100], 8)
    d = c.upload()

    def call(**kw):
        a = dict(q=d["q"], kc=d["kc"], vc=d["vc"], bt=d["bt"], cl=d["cl"], mask=d["mask"], pos=d["pos"], dl=None,
                 slopes=None, of=d["of"], ws=d["ws"])
        a.update(kw)
        pg.decode_attn_paged_tree(a["q"], a["kc"], a["vc"], a["bt"], a["cl"], a["mask"], SCALE, positions=a["pos"],
                                  draft_lens=a["dl"], slopes=a["slopes"], out_f32=a["of"], workspace=a["ws"])

    bad = [("q", d["q"].half(), TypeError), ("kc", d["kc"].float(), TypeError), ("vc", d["vc"][:1], ValueError),
           ("kc", d["kc"].transpose(0, 2).contiguous().transpose(0, 2), ValueError), ("bt", d["bt"].long(), TypeError),
           ("cl", d["cl"].cpu(), ValueError), ("cl", d["cl"].repeat(2), ValueError),
           ("mask", d["mask"].int(), TypeError), ("mask", d["mask"][:, :4], ValueError),
           ("pos", d["pos"].reshape(-1), ValueError), ("dl", torch.zeros(2, dtype=torch.int32, device="cuda"), ValueError),
           ("slopes", torch.zeros(3, device="cuda"), ValueError), ("of", d["of"][..., :64], ValueError),
           ("of", d["of"].bfloat16(), TypeError), ("ws", d["ws"].float(), TypeError)]
    for name, value, error in bad:
        with pytest.raises(error):
            call(**{name: value})
    for ws in (None, d["ws"][:16]):
        with pytest.raises(binding.PgqaError) as e:
            call(ws=ws)
        assert e.value.status == -4
    torch.cuda.synchronize()
    assert (d["of"] == SENTINEL).all()
    p = prologue_case(1861, [20], 4, 3, SECTIONS)
    for axes in ([0] * 63, [3] * 64, 64, [300] * 64):
        with pytest.raises((ValueError, TypeError, binding.PgqaError)):
            run_prologue(dict(p, axes=axes))
    with pytest.raises(ValueError):
        pg.CacheLayers([d["kc"]], [d["vc"], d["vc"]], [d["bt"]])
    with pytest.raises(ValueError):
        pg.CacheLayers([d["kc"], d["kc"][:2]], [d["vc"], d["vc"]], [d["bt"], d["bt"]])
    layers = pg.CacheLayers([d["kc"]], [d["vc"]], [d["bt"]])
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    with pytest.raises(binding.PgqaError):  # in place
        pg.kv_cache_commit_path(layers, d["cl"], one.view(1, 1), one, d["cl"], 8)
    with pytest.raises(ValueError):
        pg.kv_cache_commit_path(layers, d["cl"], one.view(1, 1).repeat(2, 1), one, torch.zeros_like(one), 8)


# ------------------------------------------------------------------ prologue
def prologue_case(seed, ctx, M, n_axes, axes, Hq=16, Hkv=8, P=16, new_lens=None, big=False):
    gen = inputs.generator(seed, 311)
    B = len(ctx)
    c = dict(kv=inputs.paged_kv(seed, ctx, Hkv=Hkv, page_size=P), q=inputs.normal_bf16(gen, (B, M, Hq, 128)),
             k=inputs.normal_bf16(gen, (B, M, Hkv, 128)), v=inputs.normal_bf16(gen, (B, M, Hkv, 128)),
             gq=inputs.uniform_bf16(gen, (128,), 0.5, 1.5), gk=inputs.uniform_bf16(gen, (128,), 0.5, 1.5),
             pos=gen.integers(-2 ** 31, 2 ** 31, (B, M, n_axes)).astype(np.int32) if big
             else gen.integers(0, 5000, (B, M, n_axes)).astype(np.int32),
             axes=list(axes), new_lens=new_lens, n=list(new_lens) if new_lens is not None else [M] * B)
    return c


def run_prologue(c, theta=THETA, eps=1e-6, stream=None):
    dev = "cuda"
    kv = c["kv"]
    kc, vc = to_device_bf16(kv.k_cache, dev), to_device_bf16(kv.v_cache, dev)
    q_out = torch.full(c["q"].shape, SENTINEL, dtype=torch.bfloat16, device=dev)
    nl = None if c["new_lens"] is None else to_device_i32(np.array(c["new_lens"]), dev)
    pg.qk_norm_rope_append_axes(to_device_bf16(c["q"], dev), to_device_bf16(c["k"], dev), to_device_bf16(c["v"], dev),
                                to_device_bf16(c["gq"], dev), to_device_bf16(c["gk"], dev),
                                to_device_i32(c["pos"], dev), to_device_i32(kv.context_lens, dev),
                                to_device_i32(kv.block_table, dev), kc, vc, q_out, c["axes"], theta, eps, new_lens=nl,
                                stream=stream)
    torch.cuda.synchronize()
    return bf16_bits(q_out), bf16_bits(kc), bf16_bits(vc)


def check_prologue(c, theta=THETA, eps=1e-6, flags=0):
    q_out, kc, vc = run_prologue(c, theta, eps)
    kv = c["kv"]
    P, Hkv = kv.page_size, kv.k_cache.shape[1]
    want_v = kv.v_cache.copy()
    touched = np.zeros(kv.k_cache.shape[:3], dtype=bool)
    for b in range(c["q"].shape[0]):
        n = c["n"][b]
        assert (q_out[b, n:] == inputs.f32_to_bf16_bits(np.array([SENTINEL], np.float32))).all()
        if n == 0:
            continue
        pos = c["pos"][b, :n, None, :]
        for x, gamma, got in ((c["q"], c["gq"], q_out[b, :n]), (c["k"], c["gk"], None)):
            want = ref.rotate(x[b, :n], gamma, pos, c["axes"], theta, eps)
            bound = ref.rotate_bound(x[b, :n], gamma, eps)
            if got is None:
                slots = [int(kv.context_lens[b]) - n + i for i in range(n)]
                rows = [(int(kv.block_table[b, s // P]), s % P) for s in slots]
                got = np.stack([kc[p, :, o] for p, o in rows])
                for i, (p, o) in enumerate(rows):
                    want_v[p, :, o] = c["v"][b, i]
                    touched[p, :, o] = True
            err = np.abs(ref.widen(got) - want)
            assert (err <= bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)).all(), (b, float(err.max()))
    assert np.array_equal(vc, want_v)
    assert np.array_equal(kc[~touched], kv.k_cache[~touched])
    assert pg.device_error_flags() == flags


SECTIONS = [0] * 16 + [1] * 24 + [2] * 24
INTERLEAVED = [r % 3 if r < 60 else 0 for r in range(64)]


@pytest.mark.parametrize("axes,n_axes", [(SECTIONS, 3), (INTERLEAVED, 3), ([0] * 64, 1), ([3, 1] * 32, 4)])
@pytest.mark.parametrize("M", [1, 2, 7, 65, 300])
def test_prologue_axes_and_lengths(axes, n_axes, M):
    check_prologue(prologue_case(2000 + M, [M, M + 37, M + 128], M, n_axes, axes))


@pytest.mark.parametrize("Hq,Hkv,P", [(8, 8, 16), (24, 8, 64), (64, 8, 256), (4, 1, 32), (1, 1, 16), (5, 1, 128)])
def test_prologue_heads_and_pages(Hq, Hkv, P):
    check_prologue(prologue_case(2100 + Hq, [90, 33], 20, 3, SECTIONS, Hq=Hq, Hkv=Hkv, P=P))


def test_prologue_ragged():
    check_prologue(prologue_case(2200, [0, 40, 300, 9], 9, 3, SECTIONS, new_lens=[0, 9, 4, 1]))


@pytest.mark.parametrize("M,new_lens", [(460, None), (701, None), (920, [920, 919, 0]), (1401, None),
                                        (1402, [1, 1400, 1399]), (1400, [0, 2, 1400])])
def test_prologue_prompts(M, new_lens):
    """Lengths on both sides of the token counts at which a block takes one more token."""
    ctx = [n + 21 for n in (new_lens or [M] * 3)]
    check_prologue(prologue_case(2300 + M, ctx, M, 3, SECTIONS, Hq=6, Hkv=2, new_lens=new_lens))


def test_prologue_prompts_of_many_heads():
    check_prologue(prologue_case(2310, [1403, 1403, 900], 1403, 3, SECTIONS, Hq=32, Hkv=8, new_lens=[1403, 1402, 900]))


def test_prologue_positions_over_the_whole_int32_range():
    check_prologue(prologue_case(2210, [50, 20], 20, 3, SECTIONS, big=True))


@pytest.mark.parametrize("theta,eps", [(1.0, 1e-6), (1e4, 0.0), (5e6, 1e-2)])
def test_prologue_theta_and_eps(theta, eps):
    check_prologue(prologue_case(2220, [50, 20], 6, 2, [0, 1] * 32), theta, eps)


def test_prologue_zero_rows():
    """All-zero heads: the norm's eps keeps them zero."""
    c = prologue_case(2230, [30], 3, 3, SECTIONS)
    c["q"][0, 1], c["k"][0, 2] = 0, 0
    check_prologue(c)


def test_prologue_matches_the_multi_token_prologue():
    """Equal positions T - M + i on every axis: qk_norm_rope_append_multi within the two bounds."""
    M, ctx = 5, [40, 700]
    c = prologue_case(2240, ctx, M, 3, SECTIONS)
    c["pos"][:] = (np.array(ctx)[:, None] - M + np.arange(M)[None])[:, :, None]
    q_out, kc, vc = run_prologue(c)
    dev, kv = "cuda", c["kv"]
    k2, v2 = to_device_bf16(kv.k_cache, dev), to_device_bf16(kv.v_cache, dev)
    q2 = torch.empty(c["q"].shape, dtype=torch.bfloat16, device=dev)
    pg.qk_norm_rope_append_multi(to_device_bf16(c["q"], dev), to_device_bf16(c["k"], dev), to_device_bf16(c["v"], dev),
                                 to_device_bf16(c["gq"], dev), to_device_bf16(c["gk"], dev),
                                 to_device_i32(kv.context_lens, dev), to_device_i32(kv.block_table, dev), k2, v2, q2,
                                 THETA)
    torch.cuda.synchronize()
    assert np.array_equal(bf16_bits(v2), vc)
    a, b = ref.widen(q_out), ref.widen(bf16_bits(q2))
    bound = ref.rotate_bound(c["q"], c["gq"], 1e-6)
    assert (np.abs(a - b) <= 2.01 * bound + 2.0 ** -7 * np.maximum(np.abs(a), np.abs(b))).all()


def test_prologue_flags():
    c = prologue_case(2250, [60, 40, 50, 30], 8, 3, SECTIONS, new_lens=[8, 8, 8, 8])
    kv = c["kv"]
    kv.context_lens[1] = 7                              # T < n
    kv.context_lens[3] = kv.max_pages * 16 + 1
    c["new_lens"] = [8, 8, 9, 8]
    q_out, kc, vc = run_prologue(c)
    assert pg.device_error_flags() == binding.DEVERR_BAD_CONTEXT
    sentinel = inputs.f32_to_bf16_bits(np.array([SENTINEL], np.float32))
    for b in (1, 2, 3):
        assert (q_out[b] == sentinel).all()
    c = prologue_case(2251, [33, 40], 4, 3, SECTIONS)
    c["kv"].block_table[0, 2] = c["kv"].num_pages      # slot 32
    c["kv"].block_table[1, 2] = -7                     # slots 36 .. 39
    before = c["kv"].k_cache.copy()
    q_out, kc, vc = run_prologue(c)
    assert pg.device_error_flags() == binding.DEVERR_BAD_PAGE
    changed = np.any(kc != before, axis=(1, 3)).sum()
    assert changed == 3                                # slots 29, 30, 31 of the first sequence
    want = ref.rotate(c["q"], c["gq"], c["pos"][:, :, None, :], c["axes"], THETA, 1e-6)
    assert (np.abs(ref.widen(q_out) - want) <= 2.0 ** -7 * np.abs(want) + 1e-4).all()


# ------------------------------------------------------------------ commit
def commit_case(seed, L, ctx, n, M, paths, A=None, Hkv=8, P=16, shared_table=False):
    A = A or max(1, max(len(p) for p in paths))
    layers = []
    for l in range(L):
        kv = inputs.paged_kv(seed + 7 * l, ctx, Hkv=Hkv, page_size=P, fill_unused="normal")
        if shared_table and layers:
            kv.block_table = layers[0].block_table
        layers.append(kv)
    path = np.full((len(ctx), A), -99, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    return dict(layers=layers, ctx=ctx, n=n, M=M, path=path, plen=[len(p) for p in paths], paths=paths)


def run_commit(c, draft=True, keep=None, stream=None):
    dev = "cuda"
    table = None
    ks, vs, ts = [], [], []
    for kv in c["layers"]:
        ks.append(to_device_bf16(kv.k_cache, dev))
        vs.append(to_device_bf16(kv.v_cache, dev))
        if kv.block_table is c["layers"][0].block_table:
            table = table if table is not None else to_device_i32(kv.block_table, dev)
            ts.append(table)
        else:
            ts.append(to_device_i32(kv.block_table, dev))
    out = torch.full((len(c["ctx"]),), -1, dtype=torch.int32, device=dev)
    pg.kv_cache_commit_path(pg.CacheLayers(ks, vs, ts), to_device_i32(np.array(c["ctx"]), dev),
                            to_device_i32(c["path"], dev), to_device_i32(np.array(c["plen"]), dev), out, c["M"],
                            draft_lens=to_device_i32(np.array(c["n"]), dev) if draft else None, stream=stream)
    torch.cuda.synchronize()
    return [bf16_bits(t) for t in ks], [bf16_bits(t) for t in vs], out.cpu().tolist()


def commit_reference(c, keep=lambda b: True):
    ks, vs = [], []
    for kv in c["layers"]:
        k, v = kv.k_cache.copy(), kv.v_cache.copy()
        P = kv.page_size
        for b, p in enumerate(c["paths"]):
            if not keep(b):
                continue
            base = c["ctx"][b] - c["n"][b]
            for i, j in enumerate(p):
                (ps, os_), (pd, od) = divmod(base + j, P), divmod(base + i, P)
                k[kv.block_table[b, pd], :, od] = kv.k_cache[kv.block_table[b, ps], :, os_]
                v[kv.block_table[b, pd], :, od] = kv.v_cache[kv.block_table[b, ps], :, os_]
        ks.append(k)
        vs.append(v)
    return ks, vs


def check_commit(c, **kw):
    ks, vs, out = run_commit(c, **kw)
    rk, rv = commit_reference(c)
    for a, b in zip(ks + vs, rk + rv):
        assert np.array_equal(a, b)
    assert out == [t - n + len(p) for t, n, p in zip(c["ctx"], c["n"], c["paths"])]
    assert pg.device_error_flags() == 0


def test_commit_paths():
    """Nothing accepted, in place, overlapping moves (a source that is another entry's destination), the last
    token, pages that end inside the tree."""
    paths = [[], [0], [0, 1, 2], [1, 2, 3, 4], [0, 2, 3, 15], [15], [3, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15]]
    ctx = [40, 16, 16, 33, 47, 100, 29]
    check_commit(commit_case(3000, 3, ctx, [16] * 7, 16, paths), draft=False)
    check_commit(commit_case(3001, 3, ctx, [16] * 7, 16, paths, A=16))


def test_commit_long_paths_cross_chunks():
    paths = [list(range(64)), list(range(1, 64)), list(range(0, 64, 2)), [0] + list(range(20, 64))]
    check_commit(commit_case(3010, 2, [64, 90, 200, 129], [64] * 4, 64, paths, Hkv=2))


@pytest.mark.parametrize("P", [16, 64, 256])
def test_commit_ragged_drafts(P):
    paths = [[0], [], [1, 3], [0, 5]]
    check_commit(commit_case(3020 + P, 2, [300, 50, 20, 9], [1, 0, 4, 7], 7, paths, P=P))


@pytest.mark.parametrize("Hkv", [1, 5, 8])
def test_commit_of_many_sequences_and_layers(Hkv):
    """More (sequence, layer) pairs than SMs: a block moves all heads of its pair."""
    gen = inputs.generator(3025 + Hkv, 12)
    paths = [sorted(int(x) for x in gen.choice(30, int(gen.integers(0, 31)), replace=False)) for _ in range(9)]
    ctx = [30 + int(gen.integers(0, 100)) for _ in paths]
    check_commit(commit_case(3025 + Hkv, 24, ctx, [30] * 9, 30, paths, Hkv=Hkv))


def test_commit_many_layers_and_a_shared_table():
    check_commit(commit_case(3030, 128, [20], [8], 8, [[1, 4, 6]], Hkv=1, shared_table=True))


def test_commit_bad_paths_keep_nothing():
    paths = [[0, 2], [2, 2], [3, 1], [0, 8], [-1, 3], [1, 2]]
    c = commit_case(3040, 2, [40] * 6, [8, 8, 8, 8, 8, 2], 8, paths)
    ks, vs, out = run_commit(c)
    assert pg.device_error_flags() == binding.DEVERR_BAD_PATH
    rk, rv = commit_reference(dict(c, paths=[paths[0]] + [[]] * 5))
    assert all(np.array_equal(a, b) for a, b in zip(ks + vs, rk + rv))
    assert out == [34, 32, 32, 32, 32, 38]
    c = commit_case(3041, 1, [40, 40], [8, 8], 8, [[0, 2], [1, 3]])
    c["plen"] = [3, -1]  # longer than A, negative
    ks, vs, out = run_commit(c)
    assert pg.device_error_flags() == binding.DEVERR_BAD_PATH and out == [32, 32]
    assert np.array_equal(ks[0], c["layers"][0].k_cache)


def test_commit_bad_lengths_and_pages():
    c = commit_case(3050, 1, [40, 40, 40], [8, 8, 8], 8, [[1, 3]] * 3)
    c["ctx"] = [7, c["layers"][0].max_pages * 16 + 1, 40]
    c["n"] = [8, 8, 9]
    ks, vs, out = run_commit(c)
    assert pg.device_error_flags() == binding.DEVERR_BAD_CONTEXT and out == c["ctx"]
    assert np.array_equal(ks[0], c["layers"][0].k_cache) and np.array_equal(vs[0], c["layers"][0].v_cache)
    # base 30: entries 1 and 3 lie in slots 31 and 33; the second page is gone
    c = commit_case(3051, 1, [38], [8], 8, [[1, 3]])
    c["layers"][0].block_table[0, 2] = 10 ** 6
    ks, vs, out = run_commit(c)
    assert pg.device_error_flags() == binding.DEVERR_BAD_PAGE and out == [32]
    page = c["layers"][0].block_table[0, 1]
    want = c["layers"][0].k_cache.copy()
    want[page, :, 14] = want[page, :, 15]
    assert np.array_equal(ks[0], want)


def test_commit_captured():
    c = commit_case(3060, 2, [40, 60], [8, 8], 8, [[1, 4], [0, 2, 7]])
    dev = "cuda"
    ks = [to_device_bf16(kv.k_cache, dev) for kv in c["layers"]]
    vs = [to_device_bf16(kv.v_cache, dev) for kv in c["layers"]]
    layers = pg.CacheLayers(ks, vs, [to_device_i32(kv.block_table, dev) for kv in c["layers"]])
    cl, path, plen = (to_device_i32(np.array(x), dev) for x in (c["ctx"], c["path"], c["plen"]))
    out = torch.zeros(2, dtype=torch.int32, device=dev)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pg.kv_cache_commit_path(layers, cl, path, plen, out, 8)
    for k, v, kv in zip(ks, vs, c["layers"]):
        k.copy_(to_device_bf16(kv.k_cache, dev)), v.copy_(to_device_bf16(kv.v_cache, dev))
    g.replay()
    torch.cuda.synchronize()
    rk, rv = commit_reference(c)
    assert all(np.array_equal(bf16_bits(a), b) for a, b in zip(ks + vs, rk + rv))
    assert out.cpu().tolist() == [34, 55]


# ------------------------------------------------------------------ a whole step
def test_verification_steps_match_token_by_token_decoding():
    """Prologue, tree attention and commit, twice: the accepted path's outputs and the committed cache are those
    of decoding its tokens one after another (decode over a chain of the same heads and positions)."""
    dev, Hq, Hkv, P, M = "cuda", 8, 4, 16, 12
    gen = inputs.generator(4000, 320)
    prefix = [37, 5]
    B = len(prefix)
    kv = inputs.paged_kv(4000, [p + 60 for p in prefix], Hkv=Hkv, page_size=P, fill_unused="normal")
    kc, vc = to_device_bf16(kv.k_cache, dev), to_device_bf16(kv.v_cache, dev)
    bt = to_device_i32(kv.block_table, dev)
    gq, gk = (to_device_bf16(inputs.uniform_bf16(gen, (128,), 0.5, 1.5), dev) for _ in range(2))
    layers = pg.CacheLayers([kc], [vc], [bt])
    chain_k, chain_v = kc.clone(), vc.clone()
    # each side's output is within (e + e) max|V| of the formula (tree_reference's bound; e: 128 u |q||k| / sqrt(128)
    # with norms up to sqrt(128 * 1.1) + 2^-16 + 400 u + 100 u <= 1.4e-4)
    tol = 2 * 2 * 1.4e-4 * float(vc.float().abs().max())
    lens = list(prefix)
    ws = workspace(B, M, Hq, Hkv, P, kv.max_pages)
    ws1 = workspace(B, 1, Hq, Hkv, P, kv.max_pages)
    for step in range(2):
        trees = [ref.random_tree(gen, M) for _ in range(B)]
        q, k, v = (to_device_bf16(inputs.normal_bf16(gen, (B, M, h, 128)), dev) for h in (Hq, Hkv, Hkv))
        pos = np.array([[lens[b] + d for d in trees[b][1]] for b in range(B)], np.int32)
        cl = to_device_i32(np.array([l + M for l in lens]), dev)
        q_out = torch.empty_like(q)
        out = torch.empty((B, M, Hq, 128), dtype=torch.float32, device=dev)
        pg.qk_norm_rope_append_axes(q, k, v, gq, gk, to_device_i32(np.repeat(pos[:, :, None], 3, 2), dev), cl, bt, kc,
                                    vc, q_out, SECTIONS, THETA)
        pg.decode_attn_paged_tree(q_out, kc, vc, bt, cl, mask_tensor([t[0] for t in trees]), SCALE, out_f32=out,
                                  workspace=ws)
        # accept a deepest token's ancestors
        paths = []
        for masks, depth in trees:
            leaf = int(np.argmax(depth))
            paths.append([j for j in range(M) if masks[leaf] >> j & 1])
        A = max(len(p) for p in paths)
        path = np.zeros((B, A), np.int32)
        for b, p in enumerate(paths):
            path[b, :len(p)] = p
        new = torch.empty(B, dtype=torch.int32, device=dev)
        pg.kv_cache_commit_path(layers, cl, to_device_i32(path, dev), to_device_i32(np.array([len(p) for p in paths]), dev),
                                new, M)
        # the same tokens one after another
        for b in range(B):
            for i, j in enumerate(paths[b]):
                one = to_device_i32(np.array([lens[b] + i + 1]), dev)
                qo = torch.empty((1, 1, Hq, 128), dtype=torch.bfloat16, device=dev)
                of = torch.empty((1, 1, Hq, 128), dtype=torch.float32, device=dev)
                pick = lambda t: t[b:b + 1, j:j + 1].contiguous()  # noqa: E731
                pg.qk_norm_rope_append_axes(pick(q), pick(k), pick(v), gq, gk, one.view(1, 1, 1) - 1, one, bt[b:b + 1],
                                            chain_k, chain_v, qo, [0] * 64, THETA)
                pg.decode_attn_paged_tree(qo, chain_k, chain_v, bt[b:b + 1], one, mask_tensor([[1]]), SCALE, out_f32=of,
                                          workspace=ws1)
                torch.cuda.synchronize()
                assert torch.equal(qo[0, 0], q_out[b, j])
                assert (of[0, 0] - out[b, j]).abs().max().item() <= tol
        lens = [l + len(p) for l, p in zip(lens, paths)]
        torch.cuda.synchronize()
        assert new.cpu().tolist() == lens
        for b in range(B):
            rows = [(int(kv.block_table[b, s // P]), s % P) for s in range(lens[b])]
            for p, o in rows:
                assert torch.equal(kc[p, :, o], chain_k[p, :, o]) and torch.equal(vc[p, :, o], chain_v[p, :, o])
    assert pg.device_error_flags() == 0


def test_decode_may_follow_a_commit_or_a_prologue_directly():
    """decode_attn_paged reads lengths and cache rows before it waits for the kernel before it: right after the
    commit (lengths and rows written) and after a prologue of several tokens its result is that of a synchronised
    run. Repeated, with other contents before each time."""
    dev, Hq, Hkv, P, M = "cuda", 16, 8, 16, 40
    gen = inputs.generator(4100, 330)
    B, base = 6, [300, 17, 1000, 64, 5, 640]
    kv = inputs.paged_kv(4100, [x + M for x in base], Hkv=Hkv, page_size=P, fill_unused="normal")
    bt = to_device_i32(kv.block_table, dev)
    cl = to_device_i32(kv.context_lens, dev)
    paths = [sorted(int(x) for x in gen.choice(M, 9, replace=False)) for _ in range(B)]
    path, plen = to_device_i32(np.array(paths), dev), to_device_i32(np.full(B, 9), dev)
    q = to_device_bf16(inputs.normal_bf16(gen, (B, Hq, 128)), dev)
    n = pg.decode_attn_workspace_size(B, Hq, Hkv, 128, P, kv.max_pages, 0)
    ws = torch.zeros(max(16, n), dtype=torch.uint8, device=dev)
    gq, gk = (to_device_bf16(inputs.uniform_bf16(gen, (128,), 0.5, 1.5), dev) for _ in range(2))
    qs, ks, vs = (to_device_bf16(inputs.normal_bf16(gen, (B, M, h, 128)), dev) for h in (Hq, Hkv, Hkv))
    pos = to_device_i32(np.array(base)[:, None, None] + np.arange(M)[None, :, None] + np.zeros((B, M, 3), int), dev)
    q_out = torch.empty_like(qs)
    kc, vc = to_device_bf16(kv.k_cache, dev), to_device_bf16(kv.v_cache, dev)
    layers = pg.CacheLayers([kc], [vc], [bt])
    lens = torch.empty(B, dtype=torch.int32, device=dev)
    out = torch.empty((B, Hq, 128), dtype=torch.float32, device=dev)

    def run(which, sync):
        kc.copy_(to_device_bf16(kv.k_cache, dev)), vc.copy_(to_device_bf16(kv.v_cache, dev))
        lens.fill_(1), out.fill_(SENTINEL)
        torch.cuda.synchronize()
        if which == "commit":
            pg.kv_cache_commit_path(layers, cl, path, plen, lens, M)
        else:
            pg.qk_norm_rope_append_axes(qs, ks, vs, gq, gk, pos, cl, bt, kc, vc, q_out, SECTIONS, THETA)
        if sync:
            torch.cuda.synchronize()
        pg.decode_attn_paged(q, kc, vc, bt, lens if which == "commit" else cl, SCALE, out_f32=out, workspace=ws)
        torch.cuda.synchronize()
        return out.cpu()

    for which in ("commit", "prologue"):
        want = run(which, True)
        for _ in range(25):
            assert torch.equal(run(which, False), want), which
    assert pg.device_error_flags() == 0


@pytest.mark.parametrize("follower", ["step", "attention"])
def test_a_longer_decode_may_follow_a_single_token_prologue_directly(follower):
    """A prologue of one token writes slot T - 1. The fused step of T + 1 tokens, and the attention of T + 1 where T
    ends a chunk of 16 positions, request that row before they wait for the kernel before them: their results are
    those of a synchronised run. The row holds NaN before each call."""
    dev, Hq, Hkv, P = "cuda", 16, 8, 16
    gen = inputs.generator(4200, 340)
    base = [48, 16, 1024, 64, 4000, 640] if follower == "attention" else [48, 17, 1000, 64, 4001, 640]
    B = len(base)
    kv = inputs.paged_kv(4200, [x + 1 for x in base], Hkv=Hkv, page_size=P, fill_unused="normal")
    for b, t in enumerate(base):
        for cache in (kv.k_cache, kv.v_cache):
            cache[kv.block_table[b, (t - 1) // P], :, (t - 1) % P] = inputs.BF16_NAN
    new = lambda h: to_device_bf16(inputs.normal_bf16(gen, (B, 1, h, 128)), dev)  # noqa: E731
    q, k, v, q2, k2, v2 = (new(h) for h in (Hq, Hkv, Hkv) * 2)
    gq, gk = (to_device_bf16(inputs.uniform_bf16(gen, (128,), 0.5, 1.5), dev) for _ in range(2))
    bt = to_device_i32(kv.block_table, dev)
    cl, longer = to_device_i32(np.array(base), dev), to_device_i32(np.array(base) + 1, dev)
    pos = (cl - 1).view(B, 1, 1)
    n = pg.decode_attn_workspace_size(B, Hq, Hkv, 128, P, kv.max_pages, 0)
    ws = torch.zeros(max(16, n), dtype=torch.uint8, device=dev)
    kc, vc = to_device_bf16(kv.k_cache, dev), to_device_bf16(kv.v_cache, dev)
    start_k, start_v = kc.clone(), vc.clone()
    q_out = torch.empty_like(q)
    out = torch.empty((B, Hq, 128), dtype=torch.float32, device=dev)

    def run(sync):
        kc.copy_(start_k), vc.copy_(start_v), out.fill_(SENTINEL)
        torch.cuda.synchronize()
        pg.qk_norm_rope_append_axes(q, k, v, gq, gk, pos, cl, bt, kc, vc, q_out, [0] * 64, THETA)
        if sync:
            torch.cuda.synchronize()
        if follower == "step":
            pg.decode_step_paged(q2[:, 0], k2[:, 0], v2[:, 0], gq, gk, longer, bt, kc, vc, SCALE, THETA, out_f32=out,
                                 workspace=ws)
        else:
            pg.decode_attn_paged(q2[:, 0], kc, vc, bt, longer, SCALE, out_f32=out, workspace=ws)
        torch.cuda.synchronize()
        return out.cpu()

    want = run(True)
    assert torch.isfinite(want).all()
    for _ in range(25):
        assert torch.equal(run(False), want)
    assert pg.device_error_flags() == 0


@pytest.mark.parametrize("far", [-2 ** 31, -70000, 10 ** 6, 2 ** 31 - 1])
def test_a_row_own_position_cancels(far):
    """Rows that see only the prefix: slope (pos_j - pos_i) is the same for every pos_i up to a constant of the row,
    which the softmax does not see, so the result and its bound are those of pos_i = prefix, wherever pos_i lies."""
    c = Case(1870, [300, 77], 5, Hq=8, Hkv=4, masks=[[0] * 5] * 2, slopes=[0.5, 1.0, 2.0 ** -8, 0.07, 3.0, 0.3, 0.01, 0.0])
    c.positions[:] = far
    of, ob = c.run()
    c.positions[:] = np.array([295, 72], np.int32)[:, None]
    out, bound = c.reference()
    check_outputs(of, ob, out, bound, c.n)


@pytest.mark.parametrize("T", [300, 12000])
def test_slopes_that_favour_the_first_keys(T):
    """Negative slopes: the first keys weigh most, however far behind them the row is. The result and its bound are
    those of pos_i = 0 (a constant of the row again)."""
    c = Case(1880 + T, [T], 3, Hq=4, Hkv=2, masks=[[0] * 3], slopes=[-0.5, -1.0, -7.0, -0.02])
    of, ob = c.run()
    c.positions[:] = 0
    out, bound = c.reference()
    check_outputs(of, ob, out, bound, c.n)


@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_drafted_tokens_far_from_the_prefix(softcap):
    """Drafted tokens whose positions lie 10^9 past the prefix (or before it, for the heads with a negative slope): with
    slopes of at least 0.5 the prefix weighs nothing at 5000 positions already, so the result and its bound are those
    of drafted tokens that are 5000 away."""
    slopes = [0.5, 1.0, 0.7, 2.0]
    for sign in (1, -1):
        c = Case(1890, [300, 40], 24, Hq=4, Hkv=2, slopes=[sign * x for x in slopes], softcap=softcap, roots=2)
        near = c.positions.copy()
        c.positions = (near + sign * 10 ** 9).astype(np.int32)
        of, ob = c.run()
        c.positions = near + sign * 5000
        out, bound = c.reference()
        check_outputs(of, ob, out, bound, c.n)


@pytest.mark.parametrize("T", [8, 60])
def test_steep_slopes_keep_scores_of_equal_positions_apart(T):
    """Drafted tokens that all lie 40 past the prefix, seen by all rows: among them the scores decide, however steep the
    slope. A row's own position is one of them, so the bound counts the bias from there."""
    c = Case(1900 + T, [T], 8, Hq=4, Hkv=2, masks=[[255] * 8], slopes=[1e4, -1e4, 1e30, -1e30])
    c.positions[:] = T - 8 + 40
    if T > 8:
        c.slopes = np.abs(c.slopes)  # (a negative slope favours the prefix)
    c.check()


def test_prologue_of_single_tokens_that_may_be_absent():
    check_prologue(prologue_case(2260, [0, 1, 40, 33], 1, 3, INTERLEAVED, new_lens=[0, 1, 0, 1], big=True))
