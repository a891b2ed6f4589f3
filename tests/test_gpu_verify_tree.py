"""verify_drafted_tree on the GPU against the walk in 64 bits, its distribution, and its edges.

Whole outputs have to be equal wherever no comparison of the walk came nearer to a tie than MARGIN. The kernel's weights
are exp2 at 2 ulp of an argument rounded twice, (x - m) k: 2^-22 + 2 |x - m| log2 e 2^-24 relative, under 30 nats 2^-18
with the sums' own errors (partial sums of at most 2^8 terms a thread and 13 joins: 2^-16 at the most); a test joins four
of them. MARGIN = 2^-13.
"""
import numpy as np
import pytest
import torch

import paged_gqa_decode_head_gb300 as pg
import tree_int8_reference as ref
from paged_gqa_decode_head_gb300 import binding

pytestmark = pytest.mark.gpu

MARGIN = 2.0 ** -13


@pytest.fixture(autouse=True)
def _clean_flags():
    pg.device_error_flags(clear=True)
    yield


def random_parents(gen, M):
    return np.array([-1] + [int(gen.integers(max(0, (i - 4) // 3), i)) for i in range(1, M)], np.int32)


class Case:
    def __init__(self, seed, B, M, V, draft=True, dtype=torch.bfloat16, temps=None, n=None, A=None, sharp=2.0, near=0.7,
                 pad=0):
        gen = np.random.default_rng(seed)
        self.B, self.M, self.V, self.A, self.dtype, self.pad = B, M, V, A or M, dtype, pad
        as_given = lambda x: torch.from_numpy(x.astype(np.float32)).to(dtype)  # noqa: E731
        x = gen.normal(0, sharp, (B, M, V))
        self.target = as_given(x)
        y = x + gen.normal(0, near, (B, M, V))
        self.draft = as_given(y) if draft else None
        self.parents = np.stack([random_parents(gen, M) for _ in range(B)])
        self.temps = np.array([gen.choice([0.0, 0.5, 1.0, 1.7]) for _ in range(B)] if temps is None else temps, np.float32)
        self.n = np.array([M] * B if n is None else n, np.int32)
        self.draft_lens = None if n is None else self.n
        # children: the best tokens of the draft row, perturbed where they are drawn
        self.tokens = np.zeros((B, M), np.int32)
        for b in range(B):
            seen = {}
            for i in range(1, M):
                p = int(self.parents[b, i])
                row = y[b, p] / (self.temps[b] or 1.0) + (gen.gumbel(size=V) if draft and self.temps[b] else 0)
                order = [t for t in np.argsort(-row) if t not in seen.get(p, [])]
                self.tokens[b, i] = order[0] if order else seen[p][0]
                seen.setdefault(p, []).append(int(self.tokens[b, i]))
        self.u = gen.random((B, M)).astype(np.float32)
        self.noise = gen.exponential(size=(B, V)).astype(np.float32) + np.float32(1e-30)

    def rows(self, t):
        if t is None:
            return None
        if not self.pad:
            return t.cuda()
        wide = torch.full((self.B, self.M, self.V + self.pad), 1e4, dtype=self.dtype, device="cuda")
        wide[..., :self.V] = t.cuda()
        return wide[..., :self.V]

    def upload(self):
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
        B, A = self.B, self.A
        self.d = dict(target=self.rows(self.target), draft=self.rows(self.draft), tokens=i32(self.tokens),
                      parents=i32(self.parents), temps=torch.from_numpy(self.temps).cuda(),
                      u=torch.from_numpy(self.u).cuda(), noise=torch.from_numpy(self.noise).cuda(),
                      dl=None if self.draft_lens is None else i32(self.n),
                      path=torch.full((B, A), 99, dtype=torch.int32, device="cuda"),
                      plen=torch.full((B,), 99, dtype=torch.int32, device="cuda"),
                      new=torch.full((B, A), 99, dtype=torch.int32, device="cuda"),
                      logp=torch.full((B, A), 99.0, device="cuda"),
                      ws=torch.full((max(16, pg.verify_drafted_tree_workspace_size(B, self.M, self.V)),), 0xA5,
                                    dtype=torch.uint8, device="cuda"))
        return self.d

    def launch(self, stream=None, logprobs=True):
        d = self.d
        pg.verify_drafted_tree(d["target"], d["tokens"], d["parents"], d["temps"], d["u"], d["noise"], d["path"], d["plen"],
                               d["new"], logprobs=d["logp"] if logprobs else None, draft_logits=d["draft"],
                               draft_lens=d["dl"], workspace=d["ws"], stream=stream)

    def outputs(self):
        torch.cuda.synchronize()
        return [self.d[x].cpu().numpy() for x in ("path", "plen", "new", "logp")]

    def run(self):
        self.upload()
        self.launch()
        return self.outputs()

    def expected(self, b):
        f = lambda t: None if t is None else t[b].float().numpy().astype(np.float64)  # noqa: E731
        return ref.verify(f(self.target), f(self.draft), self.tokens[b].tolist(), self.parents[b].tolist(),
                          int(self.n[b]), float(self.temps[b]), self.u[b].astype(np.float64), self.noise[b], self.A)

    def check(self, flags=0, decided=0.9):
        path, plen, new, logp = self.run()
        sure = 0
        for b in range(self.B):
            p, t, lp, margin = self.expected(b)
            if margin < MARGIN:
                continue
            sure += 1
            k = len(p)
            assert plen[b] == k, (b, plen[b], p)
            assert path[b].tolist() == p + [-1] * (self.A - k), b
            assert new[b].tolist() == t + [-1] * (self.A - k), b
            # log p: the sum's relative error and the logit's scaling, (2^-16 + 2^-22 |log p|)
            lp = np.array(lp + [0.0] * (self.A - k))
            assert (np.abs(logp[b] - lp) <= 2.0 ** -16 + 2.0 ** -22 * np.abs(lp)).all(), b
        assert sure >= decided * self.B
        assert pg.device_error_flags() == flags
        return path, plen, new, logp


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 64, 65, 511, 4095, 4096, 4097, 32003])
def test_vocabularies(V, draft, dtype):
    """Rows that end inside a piece of eight, and start anywhere in 16 bytes."""
    Case(V + 1, 6, 9, V, draft=draft, dtype=dtype).check()


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("M", [1, 2, 3, 17, 63, 64])
def test_tree_sizes(M, draft):
    Case(100 + M, 9, M, 257, draft=draft, sharp=1.0).check()


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("sharp,near", [(0.1, 0.1), (0.1, 3.0), (8.0, 0.5), (8.0, 8.0), (2.0, 0.0)])
def test_flat_and_peaked_rows(sharp, near, draft):
    """Rows almost uniform or all but decided; drafts that are the target's own or far from it (many rejections)."""
    Case(200 + int(10 * sharp + near), 40, 20, 100, draft=draft, sharp=sharp, near=near).check(decided=0.8)


def test_stars_and_chains():
    """All children at one node (up to 63 rejections there), and one long chain."""
    for draft in (False, True):
        c = Case(310, 12, 64, 90, draft=draft, near=3.0, temps=[1.0] * 12)
        c.parents[:6, 1:] = 0
        c.parents[6:, 1:] = np.arange(63)
        gen = np.random.default_rng(311)
        for b in range(12):
            c.tokens[b, 1:] = gen.permutation(90)[:63]
        c.u[6:] *= 0.02
        _, plen, _, _ = c.check(decided=0.5)
        assert (plen[:6] <= 2).all() and plen[6:].max() >= 2


@pytest.mark.parametrize("V", [500, 6000, 70001])
def test_what_rejections_leave(V):
    """Given children of known probability, large ones and small ones first: each test against what is left of the row,
    while much is left and when hardly anything is. The numbers lie 5 % from the thresholds."""
    shares = [[0.4, 0.3, 0.2, 0.05, 0.02], [0.02, 0.05, 0.2, 0.3, 0.4], [0.9, 0.09, 0.005, 0.002, 0.001], [0.75, 0.2, 1e-3, 1e-4, 1e-5]]
    c = Case(317, 24, 6, V, draft=False, dtype=torch.float32, temps=[1.0] * 24, sharp=0.5)
    c.parents[:, 1:] = 0
    gen = np.random.default_rng(318)
    for b in range(24):
        tokens = gen.permutation(V)[:5]
        c.tokens[b, 1:] = tokens
        x = c.target[b, 0].numpy().astype(np.float64)
        others = np.setdiff1d(np.arange(V), tokens)
        share = np.array(shares[b % 4])
        x[others] += np.log(1 - share.sum()) - np.log(np.exp(x[others]).sum())
        x[tokens] = np.log(share)
        c.target[b, 0] = torch.from_numpy(x).float()
        left = 1 - np.concatenate([[0], np.cumsum(share)[:-1]])
        c.u[b, 1:] = np.minimum(share / left * 1.05, 0.999)
        if b // 4 < 5:
            c.u[b, 1 + b // 4] = share[b // 4] / left[b // 4] * 0.95
    path, plen, _, _ = c.check(decided=1.0)
    assert (path[:20, 1] == 1 + np.arange(20) // 4).all() and (plen[20:] == 1).all()


@pytest.mark.parametrize("draft", [False, True])
def test_a_chain_accepted_to_its_end(draft):
    """Numbers of 0 accept every token that the target allows at all: paths of 64."""
    c = Case(315, 4, 64, 90, draft=draft, temps=[1.0] * 4)
    c.parents[:, 1:] = np.arange(63)
    c.u[:] = 0
    _, plen, _, _ = c.check()
    assert (plen == 64).all()


@pytest.mark.parametrize("A", [1, 2, 5])
def test_short_paths(A):
    """A path that is full takes no further child: its last token is drawn from the node's own row."""
    c = Case(320 + A, 20, 16, 50, draft=False, A=A, near=0.1, sharp=5.0)
    _, plen, _, _ = c.check()
    assert (plen == A).any()


def test_ragged_drafts_and_empty_sequences():
    c = Case(330, 8, 12, 300, n=[0, 1, 12, 5, 0, 2, 12, 7])
    path, plen, new, logp = c.check()
    assert plen[0] == 0 and (path[0] == -1).all() and (new[0] == -1).all() and (logp[0] == 0).all()


def test_repeated_siblings_and_tokens_outside_the_vocabulary():
    """A sibling that repeats a rejected token is rejected; one outside the vocabulary is passed over."""
    for draft in (False, True):
        c = Case(340, 30, 12, 40, draft=draft, temps=[0.0, 1.0, 0.7] * 10)
        c.tokens[:, 3] = c.tokens[:, 2] = c.tokens[:, 1]
        c.tokens[:10, 5], c.tokens[10:20, 5], c.tokens[20:, 4] = -1, 40, 2 ** 31 - 1
        c.tokens[:, 0] = -7  # the root is not read as a token
        c.check(flags=binding.DEVERR_BAD_PATH, decided=0.8)


def test_parents_that_are_no_earlier_token_are_never_reached():
    c = Case(350, 20, 10, 60, draft=False)
    c.parents[:, 3], c.parents[:, 4], c.parents[:, 5] = 3, 9, -1
    c.parents[:, 6], c.parents[:, 0] = -2 ** 31, 5
    c.check()


def test_masked_nan_and_infinite_logits():
    for dtype in (torch.bfloat16, torch.float32):
        for draft in (False, True):
            c = Case(360, 16, 8, 70, draft=draft, dtype=dtype)
            lowest = torch.finfo(dtype).min
            c.target[0, :, ::2] = -np.inf
            c.target[1, :, 5:60] = np.nan
            c.target[2, :, 30] = np.inf
            c.target[3, :, 30:33] = np.inf
            c.target[4, 1:] = -np.inf            # every row but the root's
            c.target[5] = np.nan
            c.target[6, :, 1:] = lowest
            c.target[7] = lowest
            if draft:
                c.draft[0, :, ::2] = -np.inf
                c.draft[8, :, ::2] = -np.inf
                c.draft[9] = -np.inf
                c.draft[10, :, 3] = np.inf
            path, plen, new, _ = c.check(decided=0.6)
            assert plen[5] == 1 and new[5, 0] == -1
            assert new[0, :plen[0]].min() >= 0 and (new[0, :plen[0]] % 2 == 1).all()


def test_greedy_takes_the_first_maximum():
    """Ties within a piece, between threads and between blocks."""
    V = 70000
    c = Case(370, 6, 4, V, draft=False, temps=[0.0] * 6)
    for b, at in enumerate(([5, 9], [4099, 3], [69999, 40000], [0, 69999], [8191, 8192], [35000, 35001])):
        c.target[b, :, at[0]] = c.target[b, :, at[1]] = 50.0
    c.tokens[:, 1] = [5, 3, 40000, 0, 8191, 7]
    c.parents[:, 1] = 0
    _, plen, new, _ = c.check(decided=1.0)
    assert new[:, 0].tolist() == [5, 3, 40000, 0, 8191, 35000]
    assert (plen[:5] >= 2).all() and plen[5] == 1


@pytest.mark.parametrize("temperature", [1e-30, 1e-3, 50.0, 3e38])
def test_temperatures(temperature):
    c = Case(380, 10, 8, 65, draft=True, temps=[temperature] * 10)
    c.check(decided=0.5)


def test_bad_lengths_and_temperatures():
    c = Case(390, 6, 8, 65, n=[8, 9, -1, 8, 8, 8], temps=[1.0, 1.0, 1.0, -0.5, np.nan, 0.0])
    path, plen, new, _ = c.run()
    assert pg.device_error_flags() == binding.DEVERR_BAD_CONTEXT
    assert plen[1:5].tolist() == [0] * 4 and (path[1:5] == -1).all() and (new[1:5] == -1).all()
    good = Case(390, 6, 8, 65, n=[8, 9, -1, 8, 8, 8], temps=[1.0, 1.0, 1.0, -0.5, np.nan, 0.0])
    for b in (0, 5):
        p, t, _, margin = good.expected(b)
        assert margin > MARGIN and path[b, :len(p)].tolist() == p and new[b, :len(t)].tolist() == t


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [1, 3, 8, 61])
def test_padded_vocabulary_rows(pad, dtype):
    """Slices [..., :V] of wider rows, whose padding holds large numbers."""
    Case(400 + pad, 5, 8, 1001, dtype=dtype, pad=pad).check()


def test_a_vocabulary_past_32_bit_offsets():
    """Rows whose elements lie past 2^31 in the logits."""
    B, M, V = 3, 64, 150000
    wide = (1 << 31) // (B * M) + 4096
    c = Case(410, B, M, V, draft=False, temps=[0.8, 0.0, 1.0])
    c.upload()
    rows = torch.zeros((B, M, wide), dtype=torch.bfloat16, device="cuda")
    rows[..., :V] = c.d["target"]
    c.d["target"] = rows[..., :V]
    c.launch()
    path, plen, new, _ = c.outputs()
    for b in range(B):
        p, t, _, margin = c.expected(b)
        assert margin < MARGIN or (path[b, :len(p)].tolist() == p and new[b, :len(t)].tolist() == t)


@pytest.mark.parametrize("B", [1, 2, 15, 70, 300])
def test_batches(B):
    Case(420 + B, B, 6, 5000, draft=B % 2 == 0).check(decided=0.8)


def test_repeated_calls_give_the_same_bits_and_logprobs_may_be_left_out():
    c = Case(430, 20, 16, 30000)
    first = c.run()
    for _ in range(3):
        c.launch(logprobs=False)
        again = c.outputs()
        assert all(np.array_equal(x, y) for x, y in zip(first, again))


def test_two_streams_at_once():
    a, b = Case(440, 30, 16, 20000), Case(441, 3, 20, 50001, draft=False)
    ra, rb = a.run(), b.run()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        a.launch(stream=sa)
        b.launch(stream=sb)
    assert all(np.array_equal(x, y) for x, y in zip(ra, a.outputs()))
    assert all(np.array_equal(x, y) for x, y in zip(rb, b.outputs()))


def test_captured_call_follows_its_inputs():
    c, other = Case(450, 10, 12, 3000, n=[12] * 10), Case(451, 10, 12, 3000, n=[3, 12, 0, 1, 5, 12, 12, 7, 2, 12])
    want = other.run()
    c.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.launch()
    for name in ("target", "draft", "tokens", "parents", "temps", "u", "noise", "dl"):
        c.d[name].copy_(other.d[name])
    for _ in range(2):
        for name in ("path", "plen", "new", "logp"):
            c.d[name].fill_(55)
        g.replay()
        assert all(np.array_equal(x, y) for x, y in zip(want, c.outputs()))


@pytest.mark.parametrize("seed", range(16))
def test_random_calls(seed):
    gen = np.random.default_rng(500 + seed)
    M = int(gen.integers(1, 65))
    B, V = int(gen.integers(1, 40)), int(np.exp(gen.uniform(0, 10)))
    Case(500 + seed, B, M, V, draft=bool(gen.integers(0, 2)), dtype=[torch.bfloat16, torch.float32][int(gen.integers(0, 2))],
         n=[int(gen.integers(0, M + 1)) for _ in range(B)], A=int(gen.integers(1, M + 1)),
         sharp=float(gen.choice([0.3, 2.0, 5.0])), near=float(gen.choice([0.0, 0.7, 3.0])),
         pad=int(gen.integers(0, 3))).check(decided=0.7)


@pytest.mark.parametrize("draft", [False, True])
def test_new_tokens_are_distributed_as_the_target(draft):
    """The first new token of many sequences with the same rows, and the second given the first: within five standard
    deviations of softmax(target / t) in every cell, whatever the drafts were drawn from."""
    B, M, V, t = 40000, 4, 6, 0.9
    gen = np.random.default_rng(600)
    rows = gen.normal(0, 1.2, (2, V)).astype(np.float32)           # the root's row, and every child's
    drafts = (rows + gen.normal(0, 1.0, (2, V))).astype(np.float32)
    c = Case.__new__(Case)
    c.B, c.M, c.V, c.A, c.dtype, c.pad, c.draft_lens = B, M, V, M, torch.float32, 0, None
    c.n, c.temps = np.full(B, M, np.int32), np.full(B, t, np.float32)
    at = [0, 1, 1, 1]
    c.target = torch.from_numpy(np.broadcast_to(rows[at], (B, M, V)).copy())
    c.draft = torch.from_numpy(np.broadcast_to(drafts[at], (B, M, V)).copy()) if draft else None
    c.parents = np.tile(np.array([-1, 0, 0, 0], np.int32), (B, 1))
    if draft:  # three siblings drawn without replacement
        c.tokens = np.argsort(-(drafts[0] / t + gen.gumbel(size=(B, V))), 1)[:, :4].astype(np.int32)
        c.tokens = np.concatenate([np.zeros((B, 1), np.int32), c.tokens[:, :3]], 1)
    else:
        c.tokens = np.tile(np.array([0, 2, 4, 1], np.int32), (B, 1))
    c.u = gen.random((B, M)).astype(np.float32)
    c.noise = gen.exponential(size=(B, V)).astype(np.float32) + np.float32(1e-30)
    path, plen, new, _ = c.run()
    p = [ref.softmax(rows[k].astype(np.float64), t) for k in (0, 1)]
    count = np.bincount(new[:, 0], minlength=V)
    assert (np.abs(count - B * p[0]) <= 5 * np.sqrt(B * p[0] * (1 - p[0]))).all(), (count, B * p[0])
    two = plen == 2
    assert 0.05 * B < two.sum()
    count, k = np.bincount(new[two, 1], minlength=V), int(two.sum())
    assert (np.abs(count - k * p[1]) <= 5 * np.sqrt(k * p[1] * (1 - p[1]))).all()


def test_binding_refuses():
    c = Case(700, 2, 4, 33)
    d = c.upload()
    good = (d["target"], d["tokens"], d["parents"], d["temps"], d["u"], d["noise"], d["path"], d["plen"], d["new"])
    pg.verify_drafted_tree(*good, workspace=d["ws"])
    for i, bad in ((0, d["target"].half()), (0, d["target"].transpose(0, 1)), (1, d["tokens"].long()),
                   (1, d["tokens"][:1]), (2, d["parents"].cpu()), (3, d["temps"].double()), (4, d["u"][:, :3]),
                   (5, d["noise"][:, :32]), (7, d["plen"][:1]), (8, d["new"][:, :2])):
        args = list(good)
        args[i] = bad
        with pytest.raises((TypeError, ValueError)):
            pg.verify_drafted_tree(*args, workspace=d["ws"])
    for kw in (dict(draft_logits=d["draft"].float()), dict(draft_logits=d["draft"][:1]), dict(draft_lens=d["temps"]),
               dict(logprobs=d["new"]), dict(draft_logits=d["draft"][:, :, ::2])):
        with pytest.raises((TypeError, ValueError)):
            pg.verify_drafted_tree(*good, workspace=d["ws"], **kw)
