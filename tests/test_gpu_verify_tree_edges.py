"""verify_drafted_tree where its arithmetic or its loads could go wrong: what is left of q near the smallest numbers, very
high temperatures, draft rows at another alignment than the target's, rows past 32-bit offsets."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_head_gb300 as pg
from test_gpu_verify_tree import MARGIN, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_flags():
    pg.device_error_flags(clear=True)
    yield
    assert pg.device_error_flags() == 0


def siblings(B, M, V, tokens, temps, target, draft):
    """B equal sequences whose root has M - 1 children; rows of float32 logits."""
    c = Case(7000, B, M, V, draft=True, dtype=torch.float32, temps=temps)
    c.target = torch.from_numpy(np.broadcast_to(target, (B, M, V)).astype(np.float32).copy())
    c.draft = torch.from_numpy(np.broadcast_to(draft, (B, M, V)).astype(np.float32).copy())
    c.parents[:], c.parents[:, 0], c.tokens[:, 1:] = 0, -1, tokens
    return c


@pytest.mark.parametrize("low", [60.0, 80.0, 84.0, 86.0, 87.0])
def test_next_to_nothing_left_of_the_draft(low):
    """Eight children of q = 1/8 each are rejected, then one whose logit lies `low` below them: 1 / q is past the largest
    number for the last of these. The residual is p without it."""
    V = 40
    target, draft = np.full(V, -np.inf), np.full(V, -np.inf)
    target[8], target[9] = 0.0, 0.0  # p = 1/2 each: the last child's token, and one that was never drafted
    draft[:8], draft[8] = 0.0, -low
    c = siblings(1, 10, V, range(9), [1.0], target, draft)
    c.u[:] = 0.9  # p' / q' = 1/2 for the last child: rejected
    c.noise[:], c.noise[0, 8] = 1.0, 1e-3  # p itself would give token 8
    path, plen, new, logp = c.run()
    assert plen[0] == 1 and path[0, 0] == 0 and new[0, 0] == 9
    assert abs(logp[0, 0] - np.log(0.5)) < 2.0 ** -16
    c.u[0, 9] = 0.1
    path, plen, new, _ = c.run()
    assert plen[0] == 2 and path[0, 1] == 9 and new[0, 0] == 8


def test_a_long_row_of_small_remainders():
    """Rejected children of q = 1, 2^-60, 2^-110, each next to nothing beside the one before: what the residual loses to each
    adds up to a finite number, and a token that was never drafted keeps its probability."""
    V, ln2 = 24, np.log(2.0)
    target, draft = np.full(V, -np.inf), np.full(V, -np.inf)
    target[2], target[5] = 0.0, 0.0
    draft[0], draft[1], draft[2] = 0.0, -60 * ln2, -110 * ln2
    c = siblings(1, 4, V, [0, 1, 2], [1.0], target, draft)
    c.u[:], c.noise[:], c.noise[0, 2] = 0.9, 1.0, 1e-3
    path, plen, new, _ = c.run()
    assert plen[0] == 1 and new[0, 0] == 5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("draft", [False, True])
def test_an_infinite_temperature(dtype, draft):
    """All tokens of usual logits are equally likely."""
    V = 500
    c = Case(7100, 12, 6, V, draft=draft, dtype=dtype, temps=[np.inf] * 12)
    path, plen, new, logp = c.run()
    assert (plen >= 1).all() and (new[:, 0] >= 0).all()
    for b in range(12):
        assert (np.abs(logp[b, :plen[b]] + np.log(V)) < 2.0 ** -16).all()
        if plen[b] == 1 and not draft and not (c.parents[b] == 0).any():
            assert new[b, 0] == np.argmin(c.noise[b])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("temperature", [1e-30, 1.0, 1e30, 1e38, np.inf])
def test_logits_at_both_ends_of_their_type(dtype, temperature):
    """The largest number beside the lowest one: the difference is past the type, and the lowest has no weight."""
    V, most = 300, torch.finfo(dtype).max
    c = Case(7200, 4, 2, V, draft=False, dtype=dtype, temps=[temperature] * 4)
    c.target[:] = -most
    c.target[:, :, 77] = most
    c.target[1:, :, 78] = most
    c.target[2:, :, 3] = float("inf")
    c.tokens[:], c.u[:], c.noise[:] = 5, 0.5, 1.0
    path, plen, new, logp = c.run()
    assert (plen == 1).all()
    if dtype is torch.float32:  # +inf counts as the largest float32
        assert new[:, 0].tolist() == [77, 77, 3, 3]
        assert np.allclose(logp[:, 0], -np.log([1, 2, 3, 3]), atol=2.0 ** -16)
    else:
        assert new[:2, 0].tolist() == [77, 77] and (new[2:, 0] == 3).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("target_pad,draft_pad", [(0, 1), (0, 3), (0, 5), (1, 0), (3, 2), (7, 4)])
@pytest.mark.parametrize("V", [1000, 1001, 33000])
def test_draft_rows_at_another_alignment(V, target_pad, draft_pad, dtype):
    """Pieces begin on the target row's 16-byte boundaries; the draft's rows lie elsewhere."""
    c = Case(7300 + V + draft_pad, 6, 10, V, dtype=dtype)
    c.upload()
    for name, pad in (("target", target_pad), ("draft", draft_pad)):
        wide = torch.full((c.B, c.M, V + pad), 1e4, dtype=dtype, device="cuda")
        wide[..., :V] = c.d[name]
        c.d[name] = wide[..., :V]
    c.upload, kept = (lambda: kept), c.d  # check() uploads
    c.check(decided=0.5)


def test_every_decided_walk_past_32_bit_offsets():
    """Rows whose elements lie past 2^31 in the logits: paths, tails, lengths and log probabilities."""
    B, M, V = 6, 64, 60000
    wide = (1 << 31) // (B * M) * 2
    c = Case(7400, B, M, V, draft=False, temps=[0.8, 0.0, 1.0, 0.0, 0.6, 0.0])
    c.upload()
    rows = torch.zeros((B, M, wide), dtype=torch.bfloat16, device="cuda")
    rows[..., :V] = c.d["target"]
    c.d["target"] = rows[..., :V]
    c.upload, kept = (lambda: kept), c.d
    sure = sum(c.expected(b)[3] >= MARGIN for b in range(B))
    assert sure >= 4
    c.check(decided=sure / B)
