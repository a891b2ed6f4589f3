"""decode_attn_paged_tree where every CTA works through many tiles: the ring of tiles wraps, both streams have steps, the
running reference moves and O is rescaled, O is moved out and added up (fp32 outputs) or stays (bf16 outputs alone),
segments follow each other in a CTA. Against the formula in 64 bits on the GPU.

A call's tiles of 128 keys are cut into equal runs, one per SM (per pair of SMs where a KV head has more than 256 query
rows), so a call needs several tiles per SM for a run to be more than one tile: `runs()` is checked in each test.

Scores: queries share a direction, and keys carry a level along it, 0, 9.5 or 19 in base 2, that changes every few tiles.
A rise by 9.5 lies above the 8 that moves a row's reference, and leaves the earlier keys a share of 2^-9.5 of the result,
far above the bounds below.

Bound on the kernel's fp32 result, in units of u = 2^-24, as in tree_reference.py (relative error e_j of weight j: score,
cap, bias, exponent, the weight's bf16 pair, fp32 sums), with the bias counted from the row's most favoured key, and the
tensor core's accumulators beside it: they round towards zero at each of the 16 products of a tile, at most 2^-23 of
sum_j p_j |V_j| a product, over the tiles of a stream between two moves of O out of it (16 for fp32 outputs, else the whole
run).
"""
import math

import numpy as np
import pytest
import torch

import paged_gqa_decode_head_gb300 as pg
import tree_reference as ref
from paged_gqa_decode_head_gb300 import binding

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SCALE = 1.0 / math.sqrt(128)
SENTINEL = 7.0
LEVEL = 9.5 * math.log(2)


@pytest.fixture(autouse=True)
def _clean_flags():
    pg.device_error_flags(clear=True)
    yield


class Long:
    """One call's tensors on the GPU."""

    def __init__(self, seed, lens, M, Hq, Hkv, P=64, draft_lens=None, softcap=0.0, slopes=None, rising=True, roots=1):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lens, self.M, self.Hq, self.Hkv, self.P = list(lens), M, Hq, Hkv, P
        self.B = B = len(lens)
        self.n = list(draft_lens) if draft_lens is not None else [M] * B
        self.draft_lens = draft_lens
        self.softcap = softcap
        need = [-(-t // P) for t in lens]
        self.max_pages = max(need) + 1
        pool = sum(need) + 1
        perm = torch.randperm(pool, generator=self.g, device="cuda").to(torch.int32)
        self.table = torch.full((B, self.max_pages), 2 ** 30, dtype=torch.int32, device="cuda")
        at = 0
        for b, c in enumerate(need):
            self.table[b, :c] = perm[at:at + c]
            at += c
        self.q, self.kc, self.vc = (self.randn(*s, 128) for s in ((B, M, Hq), (pool, Hkv, P), (pool, Hkv, P)))
        self.kc[perm[-1].long()] = self.vc[perm[-1].long()] = float("nan")  # nobody's page
        if rising:
            along = torch.where(torch.rand(128, generator=self.g, device="cuda") < 0.5, -1.0, 1.0) / math.sqrt(128)
            self.q = (self.q.float() + 8 * along).bfloat16()
            for b, t in enumerate(lens):
                level = []
                while len(level) * 128 < t:  # up by up to two levels, then back to the lowest
                    for step in range(int(rng.integers(2, 4))):
                        level += [step] * int(rng.integers(1, 5))
                keys = torch.tensor(level, device="cuda").repeat_interleave(128)[:need[b] * P].float()
                keys = torch.nn.functional.pad(keys, (0, need[b] * P - len(keys)))
                add = (keys * (LEVEL / (SCALE * 8))).view(need[b], 1, P, 1) * along
                pages = self.table[b, :need[b]].long()
                self.kc[pages] = (self.kc[pages].float() + add).bfloat16()
        for b, t in enumerate(lens):
            if t % P:  # memory behind the end holds anything
                self.kc[self.table[b, t // P].long(), :, t % P:] = float("nan")
                self.vc[self.table[b, t // P].long(), :, t % P:] = float("nan")
        trees = [ref.random_tree(rng, M, roots) for _ in range(B)]
        self.masks = np.array([[int(x) for x in t[0]] for t in trees], dtype=np.uint64)
        self.mask = torch.from_numpy(self.masks.view(np.int64)).cuda()
        self.pos = torch.tensor([[lens[b] - self.n[b] + d for d in trees[b][1]] for b in range(B)], dtype=torch.int32).cuda()
        self.slopes = None if slopes is None else torch.tensor(slopes, dtype=torch.float32).cuda()
        self.cl = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.dl = None if draft_lens is None else torch.tensor(self.n, dtype=torch.int32).cuda()
        size = pg.decode_attn_tree_workspace_size(B, M, Hq, Hkv, 128, P, self.max_pages)
        self.ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
        self.of = torch.empty(self.q.shape, dtype=torch.float32, device="cuda")
        self.ob = torch.empty(self.q.shape, dtype=torch.bfloat16, device="cuda")
        self.kept = {}  # the formula's results

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda", dtype=torch.bfloat16)

    def runs(self):
        """Tiles of a CTA's run."""
        rows = min(self.M, 128 // (self.Hq // self.Hkv))
        groups = (-(-self.M // rows) + 1) // 2
        ctas = torch.cuda.get_device_properties(0).multi_processor_count // groups
        return sum(-(-t // 128) for t, n in zip(self.lens, self.n) if n) * self.Hkv / ctas

    def launch(self, f32, bf16):
        pg.decode_attn_paged_tree(self.q, self.kc, self.vc, self.table, self.cl, self.mask, SCALE, positions=self.pos,
                                  draft_lens=self.dl, slopes=self.slopes, softcap=self.softcap,
                                  out_f32=self.of if f32 else None, out_bf16=self.ob if bf16 else None, workspace=self.ws)

    def run(self, f32, bf16):
        self.of.fill_(SENTINEL), self.ob.fill_(SENTINEL)
        self.launch(f32, bf16)
        torch.cuda.synchronize()

    def rows(self, cache, b):
        """[Hkv, T, 128] of sequence b."""
        t = self.lens[b]
        pages = self.table[b, :-(-t // self.P)].long()
        pages = torch.where((pages >= 0) & (pages < cache.shape[0]), pages, 0)
        return cache[pages].transpose(0, 1).reshape(self.Hkv, -1, 128)[:, :t]

    def formula(self, b, gone=None):
        """(out, bound without the tensor core's share, sum p |V|) [n, Hq, 128] of sequence b in 64 bits.
        gone [T]: keys that no query sees."""
        t, n, g = self.lens[b], self.n[b], self.Hq // self.Hkv
        prefix = t - n
        k, v = self.rows(self.kc, b).double(), self.rows(self.vc, b).double()
        bits = (self.mask[b, :n, None] >> torch.arange(n, device="cuda")) & 1
        seen = torch.cat([torch.ones(n, prefix, dtype=torch.bool, device="cuda"), bits.bool()], 1)
        if gone is not None:
            seen &= ~gone
        kpos = torch.cat([torch.arange(prefix, device="cuda"), self.pos[b, :n].long()]).double()
        out, bound, size = (torch.zeros(n, self.Hq, 128, dtype=torch.float64, device="cuda") for _ in range(3))
        for h in range(self.Hq):
            kh, vh, q = k[h // g], v[h // g], self.q[b, :n, h].double()
            x = q @ kh.t() * SCALE
            e = 128 * U * SCALE * (q.abs() @ kh.abs().t()) + 2 * U * x.abs()
            if self.softcap > 0:
                x = self.softcap * torch.tanh(x / self.softcap)
                e += 8 * U * x.abs()
            if self.slopes is not None:
                bias = float(self.slopes[h]) * kpos[None]
                bias = bias - bias.expand(n, t).masked_fill(~seen, -math.inf).amax(1, keepdim=True)
                e += 2 * U * (bias.abs() + x.abs())
                x = x + bias
            x = x.masked_fill(~seen, -math.inf)
            top = x.amax(1, keepdim=True)
            p = torch.exp(x - top)
            p /= p.sum(1, keepdim=True)
            e += 4 * U * (x.masked_fill(~seen, 0).abs() + top.abs()) + 8 * U + 2.0 ** -16 + 2 * (128 + t / 128 + 64) * U
            e = torch.where(seen, e, 0.0)
            out[:, h] = p @ vh
            size[:, h] = p @ vh.abs()
            bound[:, h] = (p * e) @ vh.abs() + out[:, h].abs() * (p * e).sum(1, keepdim=True)
        return out, bound, size

    def check(self, f32, bf16, rows=None, gone=None):
        """The outputs of the last run. rows[b] [n]: the tokens to look at."""
        run = math.ceil(self.runs()) + 1
        products = 16 * (16 if f32 else run)
        for b in range(self.B):
            n = self.n[b]
            assert (self.of[b, n:] == SENTINEL).all() and (self.ob[b, n:] == SENTINEL).all()
            if n == 0:
                continue
            if b not in self.kept:
                self.kept[b] = self.formula(b, None if gone is None else gone[b])
            out, bound, size = self.kept[b]
            bound = bound + products * 2.0 ** -23 * size
            at = slice(None) if rows is None else rows[b]
            for got, step in ((self.of, 2.0 ** -24) if f32 else (None, 0), (self.ob, 2.0 ** -8) if bf16 else (None, 0)):
                if got is None:
                    continue
                err = (got[b, :n].double() - out).abs() - (bound * (1 + step) + step * out.abs())
                assert torch.isfinite(got[b, :n][at]).all() and (err[at] <= 0).all(), (b, f32, bf16, float(err[at].max()))
        if not f32:
            assert (self.of == SENTINEL).all()
        if not bf16:
            assert (self.ob == SENTINEL).all()

    def check_all_outputs(self, **kw):
        for f32, bf16 in ((True, False), (False, True), (True, True)):
            self.run(f32, bf16)
            self.check(f32, bf16, **kw)


def slopes_of(Hq):
    """Gentle and steep, one negative in five, one of zero."""
    s = [2.0 ** -(2 + 9 * h / Hq) * (-1 if h % 5 == 4 else 1) for h in range(Hq)]
    s[0] = 0.0
    return s


FORMS = [(0.0, False), (25.0, False), (0.0, True), (25.0, True)]
# query rows of a KV head: one row tile (24, 128), two (256), three (320: a pair and one), four (512: two pairs)
SHAPES = [(12, 2), (64, 2), (64, 4), (40, 8), (64, 8)]


@pytest.mark.parametrize("softcap,bias", FORMS)
@pytest.mark.parametrize("M,g", SHAPES)
def test_runs_of_many_tiles(M, g, softcap, bias):
    """Some twenty tiles a CTA, the reference moving every few of them; all score forms and row layouts."""
    c = Long(7000 + M + g, [9000, 12345, 7777, 10001], M, 8 * g, 8, softcap=softcap, slopes=slopes_of(8 * g) if bias else None)
    assert c.runs() >= 15
    c.check_all_outputs()
    assert pg.device_error_flags() == 0


@pytest.mark.parametrize("M,g,softcap,bias", [(3, 1, 0.0, False), (3, 1, 25.0, True), (64, 4, 0.0, False), (64, 4, 0.0, True),
                                              (64, 8, 25.0, False)])
def test_runs_longer_than_a_span(M, g, softcap, bias):
    """More than 32 tiles a stream: O of fp32 outputs moves out several times, with rescales before, at and after."""
    c = Long(7100 + M + g, [34000, 40001, 37777], M, 8 * g, 8, softcap=softcap, slopes=slopes_of(8 * g) if bias else None)
    assert c.runs() >= (33 if M * g > 128 else 43)
    c.check_all_outputs()
    assert pg.device_error_flags() == 0


@pytest.mark.parametrize("P", [16, 128, 256])
@pytest.mark.parametrize("M,g", [(16, 2), (64, 4)])
def test_ragged_drafts_over_long_contexts(M, g, P):
    n = [M, 0, 1, M // 2, M - 1, 5, M, 3]
    c = Long(7200 + P + M, [9000, 12345, 7777, 10001, 300, 12000, 128, 8000], M, 8 * g, 8, P=P, draft_lens=n, roots=2)
    assert c.runs() >= 19
    c.check_all_outputs()
    assert pg.device_error_flags() == 0


@pytest.mark.parametrize("softcap,bias", FORMS)
def test_single_tokens_of_a_ragged_batch(softcap, bias):
    """Token decoding: three query rows a head, several segments of many tiles per CTA; scores past their cap."""
    softcap *= 0.4
    rng = np.random.default_rng(7300)
    lens = [int(x) for x in rng.integers(1, 12000, 33)]
    c = Long(7300, lens, 1, 24, 8, P=32, softcap=softcap, slopes=slopes_of(24) if bias else None)
    assert c.runs() >= 40
    c.check_all_outputs()
    assert pg.device_error_flags() == 0


@pytest.mark.parametrize("M,g,T", [(64, 4, 300), (64, 8, 200), (16, 4, 500), (64, 2, 128)])
def test_hundreds_of_short_sequences_with_nonfinite_drafted_rows(M, g, T):
    """Many short segments in a CTA, one after another. Drafted tokens' K and V rows that are not finite reach only the
    tokens that see them; a V row of +inf alone gives them +inf where it is."""
    rng = np.random.default_rng(7400 + M + g)
    B, Hkv = 320, 4
    n = [int(x) for x in rng.integers(1, M + 1, B)]
    c = Long(7400 + M + g, [x + int(rng.integers(0, T)) for x in n], M, Hkv * g, Hkv, P=16, draft_lens=n, rising=False)
    assert c.runs() >= 10
    clean_k, clean_v = c.kc.clone(), c.vc.clone()
    rows, hit = [], []
    for b in range(B):
        inf_at, nan_at = int(rng.integers(0, n[b])), int(rng.integers(0, n[b]))
        for j, x, cache in ((inf_at, math.inf, c.vc), (nan_at, math.nan, c.vc), (nan_at, math.nan, c.kc)):
            if b % 3 == 0 and j == nan_at and nan_at != inf_at:
                continue  # only an infinity
            slot = c.lens[b] - n[b] + j
            cache[int(c.table[b, slot // 16]), :, slot % 16, 5:9] = x
        sees = lambda j: ((c.masks[b, :n[b]] >> np.uint64(j)) & np.uint64(1)).astype(bool)  # noqa: E731
        only_inf = b % 3 == 0 and nan_at != inf_at
        bad = sees(inf_at) | (False if only_inf else sees(nan_at))
        rows.append(torch.from_numpy(~bad).cuda())
        hit.append(torch.from_numpy(sees(inf_at)).cuda() if only_inf else None)
    for f32, bf16 in ((True, False), (False, True)):
        c.run(f32, bf16)
        got = c.of if f32 else c.ob
        for b in range(B):
            if hit[b] is not None:
                assert (got[b, :n[b]][hit[b]][..., 5:9] == math.inf).all()
        dirty_k, dirty_v, c.kc, c.vc = c.kc, c.vc, clean_k, clean_v
        c.check(f32, bf16, rows=rows)
        c.kc, c.vc = dirty_k, dirty_v
    assert pg.device_error_flags() == 0


@pytest.mark.parametrize("M,g", [(16, 2), (64, 8)])
def test_pages_outside_the_pool_in_long_runs(M, g):
    c = Long(7500 + M, [9000, 12345, 10001], M, 8 * g, 8, P=32)
    rng = np.random.default_rng(7500)
    gone = []
    for b, t in enumerate(c.lens):
        lost = np.zeros(t, dtype=bool)
        for page in rng.choice(-(-t // 32), 60, replace=False):
            c.table[b, page] = [-1, c.kc.shape[0], 2 ** 31 - 1][page % 3]
            lost[page * 32:page * 32 + 32] = True
        gone.append(torch.from_numpy(lost).cuda())
    assert c.runs() >= 12
    c.kc[0].nan_to_num_(0.0), c.vc[0].nan_to_num_(0.0)  # the formula's stand-in for such a page
    c.check_all_outputs(gone=gone)
    assert pg.device_error_flags() == binding.DEVERR_BAD_PAGE


@pytest.mark.parametrize("M,g,softcap,bias", [(12, 2, 0.0, False), (64, 8, 25.0, True)])
def test_long_runs_give_the_same_bits_each_time(M, g, softcap, bias):
    """Alone, beside another stream's work, and replayed; with a workspace that other calls have used."""
    c = Long(7600 + M, [20000, 12345], M, 8 * g, 8, softcap=softcap, slopes=slopes_of(8 * g) if bias else None)
    for f32, bf16 in ((True, True), (False, True)):
        c.run(f32, bf16)
        want = c.of.clone(), c.ob.clone()
        side, a = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda", dtype=torch.bfloat16)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.launch(f32, bf16)
        for i in range(9):
            c.of.fill_(SENTINEL), c.ob.fill_(SENTINEL)
            c.ws.random_(0, 256, generator=c.g)
            if i % 3 == 1:
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    for _ in range(8):
                        a @ a
            graph.replay() if i % 3 == 2 else c.launch(f32, bf16)
            torch.cuda.synchronize()
            assert torch.equal(c.of, want[0]) and torch.equal(c.ob, want[1])
    assert pg.device_error_flags() == 0


def long_flat(B, M, Hq, Hkv, T):
    return Long(7700 + M, [T - 1000 * b for b in range(B)], M, Hq, Hkv, rising=False)


def test_fp32_sums_of_long_contexts():
    """fp32 outputs of 4 x 131072 keys in the 2-norm. O leaves the tensor core every 16 tiles of a stream, 256 products. A
    product's rounding towards zero loses half a unit in the last place on average, 0.36 * 2^-23 of the accumulator
    over all mantissas; the accumulator's size over a span whose terms have either sign grows as the root of the
    products so far, 2/3 of the last one on average: 256 * 2/3 * 0.36 * 2^-23 = 7.3e-6 of the span's sum, for all
    spans alike. The weights' pairs and the fp32 scores add 2^-18 / sqrt(3) = 2.2e-6 each at most, independent
    of it: 8e-6 in all. (Left in the tensor core over a run of 108 tiles a stream, O would lose some 2.3e-5.)"""
    c = long_flat(4, 2, 8, 8, 131072)
    assert c.runs() >= 200
    c.run(True, False)
    for b in range(c.B):
        out, _, _ = c.formula(b)
        rel = ((c.of[b].double() - out).norm() / out.norm()).item()
        assert rel <= 8e-6, (b, rel)
    assert pg.device_error_flags() == 0


@pytest.mark.parametrize("B,M,Hq,Hkv,T", [(4, 2, 8, 8, 131072), (3, 40, 32, 8, 40000)])
def test_bf16_outputs_alone_of_long_contexts(B, M, Hq, Hkv, T):
    """bf16 outputs alone, with no moves of O: each element within its bound, and in the 2-norm no further from the formula
    than the rounding to bf16, half a step of 2^-8 relative at most, 2^-9 in the mean of squares."""
    c = long_flat(B, M, Hq, Hkv, T)
    c.run(False, True)
    c.check(False, True)
    for b in range(B):
        out, _, _ = c.formula(b)
        rel = ((c.ob[b].double() - out).norm() / out.norm()).item()
        assert rel <= 2.0 ** -9, (b, rel)
    assert pg.device_error_flags() == 0
