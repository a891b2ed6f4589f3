"""Drafted-tree decoding over the paged KV cache: three operators and their plain forms.

``qk_norm_rope_append_axes``  per-head RMSNorm, rotary positions with several axes (time, height,
    width; a drafted token's depth is the same on every axis) and the append of K and V;
``decode_attn_paged_tree``    attention of a tree of drafted tokens over the cached prefix and the
    tokens' own ancestors, with an optional tanh cap of the scores and an optional bias that falls
    with the distance;
``kv_cache_commit_path``      the accepted path's K and V rows moved behind the prefix, every layer
    in one call.

A case is measured as one call on tensors that a serving loop holds anyway: caches, block tables,
workspace. ``own`` selects the library's kernels; otherwise ``run`` is elementary torch in 32 bits
(64 for the rotary angles).
"""
import math
import random

import numpy as np
import torch

own = False

D = 128
THETA = 1e6
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one layer's prologue of a verification step: 16 drafted tokens behind 8192 positions
        dict(name="rope_draft_m16", op="rope", B=1, M=16, Hq=16, Hkv=8, P=16, base=8192, kind="tree", ragged=False),
        # an image's patches and the text around it, one sequence, an odd number of tokens
        dict(name="rope_image_4095", op="rope", B=1, M=4095, Hq=16, Hkv=8, P=16, base=0, kind="image", ragged=False),
        # a padded batch of prompts with images, behind prefixes of their own
        dict(name="rope_batch_32k", op="rope", B=8, M=4096, Hq=32, Hkv=8, P=64, base=513, kind="image", ragged=True),
        # the smallest verification step: a short chat, eight drafted tokens
        dict(name="tree_t512_m8", op="tree", B=1, M=8, Hq=16, Hkv=8, P=16, lens="same", T=520, cap=0.0, bias=False,
             ragged=False, out="bf16"),
        # the 28-layer decode workload's layer (T = 8192) with a tree of 16
        dict(name="tree_t8k_m16", op="tree", B=1, M=16, Hq=16, Hkv=8, P=16, lens="same", T=8192, cap=0.0, bias=False,
             ragged=False, out="bf16"),
        # the widest tree over the same layer, outputs in 32 bits
        dict(name="tree_t8k_m64_f32", op="tree", B=1, M=64, Hq=16, Hkv=8, P=16, lens="same", T=8192, cap=0.0,
             bias=False, ragged=False, out="f32"),
        # a served batch of ragged lengths up to 32768, trees of up to 16 drafted tokens
        dict(name="tree_ragged_b64", op="tree", B=64, M=16, Hq=16, Hkv=8, P=16, lens="ragged", T=32768, cap=0.0,
             bias=False, ragged=True, out="bf16"),
        # one long context with capped scores
        dict(name="tree_t128k_cap", op="tree", B=1, M=16, Hq=32, Hkv=8, P=16, lens="same", T=131072, cap=30.0,
             bias=False, ragged=False, out="bf16"),
        # many query rows per key: 64 drafted tokens times groups of 8 heads (matrix products bound it)
        dict(name="tree_wide_b8", op="tree", B=8, M=64, Hq=64, Hkv=8, P=64, lens="same", T=16384, cap=0.0, bias=False,
             ragged=False, out="bf16"),
        # plain single-token decoding of a model with distance biases and capped scores, odd sizes
        dict(name="token_bias_b33", op="tree", B=33, M=1, Hq=24, Hkv=8, P=32, lens="ragged", T=4001, cap=50.0,
             bias=True, ragged=False, out="bf16"),
        # 28 layers' caches after a step that accepted five of sixteen drafted tokens
        dict(name="commit_l28_m16", op="commit", L=28, B=1, M=16, A=5, Hkv=8, P=16, base=200, ragged=False),
        # the same for a batch with trees of 64, paths of up to 12
        dict(name="commit_l28_b24_m64", op="commit", L=28, B=24, M=64, A=12, Hkv=8, P=16, base=120, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads = [(16, 8), (32, 8), (64, 8), (24, 8), (8, 8), (4, 1), (40, 8), (56, 8)]
    kind = rng.choice(["rope", "tree", "tree", "tree", "commit"])
    Hq, Hkv = rng.choice(heads)
    P = rng.choice([16, 16, 32, 64, 128, 256])
    if kind == "rope":
        while True:
            B, M = _log_int(rng, 1, 64), _log_int(rng, 1, 8192)
            if B * M * (2 * Hq + 4 * Hkv) <= 8 * 4096 * (2 * 32 + 4 * 8):
                break
        return dict(op="rope", B=B, M=M, Hq=Hq, Hkv=Hkv, P=P, base=_log_int(rng, 1, 4096) - 1,
                    kind="tree" if M <= 64 and rng.random() < 0.5 else "image", ragged=rng.random() < 0.5)
    if kind == "tree":
        while True:
            B, M, T = _log_int(rng, 1, 128), _log_int(rng, 1, 64), _log_int(rng, 65, 131072)
            if B * T * Hkv <= 64 * 16384 * 8 and B * T * Hq * M <= 8 * 16384 * 64 * 64:
                break
        return dict(op="tree", B=B, M=M, Hq=Hq, Hkv=Hkv, P=P, lens=rng.choice(["same", "ragged"]), T=T,
                    cap=rng.choice([0.0, 0.0, 30.0, 50.0]), bias=rng.random() < 0.4, ragged=rng.random() < 0.4,
                    out=rng.choice(["bf16", "bf16", "f32"]))
    while True:
        L, B, M = rng.randint(1, 36), _log_int(rng, 1, 64), _log_int(rng, 2, 64)
        base = _log_int(rng, 16, 512)
        if L * B * Hkv * (base + M + P) <= 28 * 24 * 8 * 200:
            break
    return dict(op="commit", L=L, B=B, M=M, A=rng.randint(2, max(2, min(M, 16))), Hkv=Hkv, P=P, base=base,
                ragged=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _tables(g, lens, P, max_pages, pool=0):
    """A page table whose sequences own pages in random order, one page of the pool to spare at least."""
    need = [-(-t // P) for t in lens]
    pool = max(pool, sum(need) + 1)
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max_pages, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, pool


def _tree(rng, M):
    """Parents (-1: a root), ancestor bit masks (the token itself included) and depths of a drafted tree
    listed parents first."""
    parent = [-1] + [rng.randint(max(0, (i - 4) // 3), i - 1) for i in range(1, M)]
    mask, depth = [], []
    for i, p in enumerate(parent):
        mask.append((mask[p] if p >= 0 else 0) | (1 << i))
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return mask, depth


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def _signed64(m):
    return m - (1 << 64) if m >= 1 << 63 else m


def prepare(case, seed):
    return {"rope": _prepare_rope, "tree": _prepare_tree, "commit": _prepare_commit}[case["op"]](case, seed)


def _prepare_rope(c, seed):
    g, rng = _gen(seed), random.Random(seed)
    B, M, Hq, Hkv, P = c["B"], c["M"], c["Hq"], c["Hkv"], c["P"]
    new = [rng.randint(0, M) if c["ragged"] else M for _ in range(B)]
    lens = [c["base"] + n for n in new]
    max_pages = -(-(c["base"] + M) // P)
    table, pool = _tables(g, lens, P, max_pages, B * max_pages + 1)
    pos = np.zeros((B, M, 3), dtype=np.int32)
    for b in range(B):
        if c["kind"] == "tree":
            pos[b] = (np.asarray(_tree(rng, M)[1]) + c["base"])[:, None]
        else:
            # text, an image of h x w patches at one time step, text again from the largest position on
            lead, w = M // 8, max(1, math.isqrt(max(1, M // 2)))
            img = w * max(1, (M // 2) // w) if M >= 8 else 0
            i = np.arange(M)
            text = c["base"] + np.where(i < lead, i, i - img + max(w, img // w if w else 0))
            pos[b] = text[:, None]
            k = np.arange(min(img, M - lead))
            pos[b, lead:lead + len(k), 0] = c["base"] + lead
            pos[b, lead:lead + len(k), 1] = c["base"] + lead + k // w
            pos[b, lead:lead + len(k), 2] = c["base"] + lead + k % w
    gq = torch.rand(D, generator=g, device="cuda").add_(0.5).bfloat16()
    gk = torch.rand(D, generator=g, device="cuda").add_(0.5).bfloat16()
    return dict(op="rope", q=_randn(g, B, M, Hq, D), k=_randn(g, B, M, Hkv, D), v=_randn(g, B, M, Hkv, D), gq=gq,
                gk=gk, positions=_i32(pos), context_lens=_i32(lens), new_lens=_i32(new) if c["ragged"] else None,
                table=table, kc=_randn(g, pool, Hkv, P, D), vc=_randn(g, pool, Hkv, P, D),
                q_out=torch.zeros(B, M, Hq, D, dtype=torch.bfloat16, device="cuda"),
                # 64 frequencies: the first 16 turn with time, 24 with height, 24 with width
                axes=[0] * 16 + [1] * 24 + [2] * 24)


def _prepare_tree(c, seed):
    g, rng = _gen(seed), random.Random(seed)
    B, M, Hq, Hkv, P, T = c["B"], c["M"], c["Hq"], c["Hkv"], c["P"], c["T"]
    n_draft = [rng.randint(1, M) if c["ragged"] else M for _ in range(B)]
    lens = [max(n, rng.randint(1, T) if c["lens"] == "ragged" else T) for n in n_draft]
    max_pages = -(-max(max(lens), T) // P)
    table, pool = _tables(g, lens, P, max_pages)
    kc, vc = _randn(g, pool, Hkv, P, D), _randn(g, pool, Hkv, P, D)
    # some keys weigh more than the rest, as in real caches, so that the softmax has peaks
    strong = torch.rand(pool, 1, P, 1, generator=g, device="cuda") < 0.01
    kc.mul_(torch.where(strong, 3.0, 1.0).bfloat16())
    # memory behind a sequence's last position holds anything
    for b, t in enumerate(lens):
        if t % P:
            kc[table[b, t // P].long(), :, t % P:] = float("nan")
            vc[table[b, t // P].long(), :, t % P:] = float("nan")
    masks, pos = [], []
    for b in range(B):
        m, d = _tree(rng, M)
        masks.append([_signed64(x) for x in m])
        pos.append([lens[b] - n_draft[b] + x for x in d])
    slopes = None
    if c["bias"]:
        slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float32, device="cuda")
    out = torch.zeros(B, M, Hq, D, dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16, device="cuda")
    s = dict(op="tree", q=_randn(g, B, M, Hq, D), kc=kc, vc=vc, table=table, context_lens=_i32(lens),
             draft_lens=_i32(n_draft) if c["ragged"] else None,
             mask=torch.as_tensor(np.asarray(masks, dtype=np.int64)).cuda(), positions=_i32(pos), slopes=slopes,
             cap=c["cap"], scale=1.0 / math.sqrt(D), out=out, lens=lens, n_draft=n_draft)
    if own:
        import paged_gqa_decode_head_gb300 as pg
        n = pg.decode_attn_tree_workspace_size(B, M, Hq, Hkv, D, P, max_pages)
        s["ws"] = torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")
    return s


def _prepare_commit(c, seed):
    g, rng = _gen(seed), random.Random(seed)
    L, B, M, A, Hkv, P = c["L"], c["B"], c["M"], c["A"], c["Hkv"], c["P"]
    n_draft = [rng.randint(A, M) if c["ragged"] else M for _ in range(B)]
    lens = [c["base"] + rng.randint(0, P - 1) + n for n in n_draft]
    max_pages = -(-(c["base"] + P + M) // P)
    paths, plens = [], []
    for b in range(B):
        # the accepted path: first children first, then one sibling per level further on in the list
        a = rng.randint(1, A) if c["ragged"] else A
        later = list(range(a, n_draft[b]))
        lead = max(1, a - len(later), rng.randint(0, a))
        paths.append(list(range(lead)) + sorted(rng.sample(later, a - lead)) + [-1] * (A - a))
        plens.append(a)
    kcs, vcs, tables = [], [], []
    for _ in range(L):
        table, pool = _tables(g, lens, P, max_pages, B * max_pages + 1)
        tables.append(table)
        kcs.append(_randn(g, pool, Hkv, P, D))
        vcs.append(_randn(g, pool, Hkv, P, D))
    s = dict(op="commit", kcs=kcs, vcs=vcs, tables=tables, context_lens=_i32(lens),
             draft_lens=_i32(n_draft) if c["ragged"] else None, M=M, path=_i32(paths), path_lens=_i32(plens),
             lens_out=torch.zeros(B, dtype=torch.int32, device="cuda"))
    if own:
        import paged_gqa_decode_head_gb300 as pg
        s["layers"] = pg.CacheLayers(kcs, vcs, tables)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return {"rope": _run_rope, "tree": _run_tree, "commit": _run_commit}[state["op"]](state)


def _rotate(x, gamma, cos, sin):
    """RMSNorm over the last axis, gain, then the rotation of the pairs (i, i + 64), in 32 bits."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.float()
    a, b = x[..., :64], x[..., 64:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).bfloat16()


def _run_rope(s):
    if own:
        import paged_gqa_decode_head_gb300 as pg
        pg.qk_norm_rope_append_axes(s["q"], s["k"], s["v"], s["gq"], s["gk"], s["positions"], s["context_lens"],
                                    s["table"], s["kc"], s["vc"], s["q_out"], s["axes"], THETA, EPS,
                                    new_lens=s["new_lens"])
        return s["q_out"], s["kc"], s["vc"]
    B, M = s["q"].shape[:2]
    P = s["kc"].shape[2]
    omega = THETA ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
    axis = torch.tensor(s["axes"], device="cuda")
    phi = s["positions"][..., axis].double() * omega
    cos, sin = phi.cos().float()[:, :, None], phi.sin().float()[:, :, None]
    q = _rotate(s["q"], s["gq"], cos, sin)
    k = _rotate(s["k"], s["gk"], cos, sin)
    n = s["new_lens"] if s["new_lens"] is not None else torch.full_like(s["context_lens"], M)
    i = torch.arange(M, device="cuda")[None]
    live = i < n[:, None]
    at = (s["context_lens"] - n)[:, None] + i
    at = torch.where(live, at, 0)
    page = s["table"].long().gather(1, (at // P).long())
    s["q_out"][live] = q[live]
    s["kc"][page[live], :, (at % P)[live].long()] = k[live]
    s["vc"][page[live], :, (at % P)[live].long()] = s["v"][live]
    return s["q_out"], s["kc"], s["vc"]


def _run_tree(s):
    out = s["out"]
    if own:
        import paged_gqa_decode_head_gb300 as pg
        where = {"out_f32": out} if out.dtype == torch.float32 else {"out_bf16": out}
        pg.decode_attn_paged_tree(s["q"], s["kc"], s["vc"], s["table"], s["context_lens"], s["mask"], s["scale"],
                                  positions=s["positions"], draft_lens=s["draft_lens"], slopes=s["slopes"],
                                  softcap=s["cap"], workspace=s["ws"], **where)
        return out
    B, M, Hq, _ = s["q"].shape
    _, Hkv, P, _ = s["kc"].shape
    g = Hq // Hkv
    bit = torch.arange(64, device="cuda")
    for b, (T, n) in enumerate(zip(s["lens"], s["n_draft"])):
        pages = s["table"][b, :-(-T // P)].long()
        k = s["kc"][pages].transpose(0, 1).reshape(Hkv, -1, D)[:, :T].float()
        v = s["vc"][pages].transpose(0, 1).reshape(Hkv, -1, D)[:, :T].float()
        q = s["q"][b, :n].float().view(n, Hkv, g, D).permute(1, 2, 0, 3).reshape(Hkv, g * n, D)
        x = (q @ k.transpose(1, 2)).mul_(s["scale"]).view(Hkv, g, n, T)
        if s["cap"] > 0:
            x = torch.tanh(x / s["cap"]) * s["cap"]
        where = torch.cat([torch.arange(T - n, device="cuda"), s["positions"][b, :n].long()])
        if s["slopes"] is not None:
            far = (where[None] - s["positions"][b, :n].long()[:, None]).float()
            x = x + s["slopes"].view(Hkv, g, 1, 1) * far
        seen = torch.ones(n, T, dtype=torch.bool, device="cuda")
        seen[:, T - n:] = ((s["mask"][b, :n, None] >> bit[:n]) & 1).bool()
        x = x.masked_fill(~seen, -math.inf)
        p = torch.exp(x - x.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        o = p.view(Hkv, g * n, T) @ v
        out[b, :n] = o.view(Hkv, g, n, D).permute(2, 0, 1, 3).reshape(n, Hq, D)
    return out


def _run_commit(s):
    if own:
        import paged_gqa_decode_head_gb300 as pg
        pg.kv_cache_commit_path(s["layers"], s["context_lens"], s["path"], s["path_lens"], s["lens_out"], s["M"],
                                draft_lens=s["draft_lens"])
        return s["lens_out"], s["kcs"], s["vcs"]
    P = s["kcs"][0].shape[2]
    n = s["draft_lens"] if s["draft_lens"] is not None else torch.full_like(s["context_lens"], s["M"])
    base = (s["context_lens"] - n).long()
    i = torch.arange(s["path"].shape[1], device="cuda")[None]
    live = i < s["path_lens"][:, None]
    src = torch.where(live, base[:, None] + s["path"], 0)
    dst = torch.where(live, base[:, None] + i, 0)
    for kc, vc, table in zip(s["kcs"], s["vcs"], s["tables"]):
        ps, pd = table.long().gather(1, src // P)[live], table.long().gather(1, dst // P)[live]
        rs, rd = (src % P)[live], (dst % P)[live]
        kc[pd, :, rd] = kc[ps, :, rs]
        vc[pd, :, rd] = vc[ps, :, rs]
    s["lens_out"].copy_(base + s["path_lens"])
    return s["lens_out"], s["kcs"], s["vcs"]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "rope":
        toks = c["B"] * c["M"] * (0.5 if c["ragged"] else 1.0)
        return {"bytes": toks * ((2 * c["Hq"] + 4 * c["Hkv"]) * 2 * D + 12),
                "flops": toks * (c["Hq"] + c["Hkv"]) * D * 7}
    if c["op"] == "tree":
        keys = c["B"] * c["T"] * (0.5 if c["lens"] == "ragged" else 1.0)
        m = (c["M"] + 1) / 2 if c["ragged"] else c["M"]
        size = 4 if c["out"] == "f32" else 2
        return {"bytes": keys * c["Hkv"] * 2 * 2 * D + c["B"] * m * c["Hq"] * D * (2 + size),
                "flops": 4.0 * keys * m * c["Hq"] * D}
    a = (c["A"] + 1) / 2 if c["ragged"] else c["A"]
    moved = max(0.0, a / 2 - 0.5)  # about half of a path already lies in its place
    return {"bytes": c["L"] * c["B"] * c["Hkv"] * moved * 2 * 2 * 2 * D + c["B"] * (4 * c["A"] + 16),
            "flops": 0}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "tree": _exact_tree, "commit": _exact_commit}[case["op"]](s)


def _cells(s, b, positions, Hkv):
    """Flat row numbers [Hkv, len(positions)] in a cache seen as [rows, D]."""
    P = s["kc"].shape[2]
    pos = torch.as_tensor(positions, dtype=torch.int64, device="cuda")
    page = s["table"][b].to(torch.int64)[torch.div(pos, P, rounding_mode="floor")]
    return (page[None] * Hkv + torch.arange(Hkv, device="cuda")[:, None]) * P + torch.remainder(pos, P)[None]


def _exact_rope(s):
    B, M, Hq, _ = s["q"].shape
    Hkv = s["k"].shape[2]
    q_out, kc, vc = s["q_out"].double(), s["kc"].double(), s["vc"].double()
    turn = torch.tensor([math.exp(-math.log(THETA) * i / 64) for i in range(64)], dtype=torch.float64, device="cuda")
    lens = s["context_lens"].tolist()
    new = [M] * B if s["new_lens"] is None else s["new_lens"].tolist()

    def turned(x, gain, z):
        x = x.double()
        x = gain.double() * x / (x.square().sum(-1, keepdim=True) / D + EPS).sqrt()
        w = torch.complex(x[..., :64].contiguous(), x[..., 64:].contiguous()) * z
        return torch.cat((w.real, w.imag), dim=-1)

    for b in range(B):
        n = new[b]
        if n == 0:
            continue
        ang = torch.stack([s["positions"][b, :n, a].double() * turn[i] for i, a in enumerate(s["axes"])], dim=-1)
        z = torch.polar(torch.ones_like(ang), ang)[:, None]
        q_out[b, :n] = turned(s["q"][b, :n], s["gq"], z)
        rows = _cells(s, b, range(lens[b] - n, lens[b]), Hkv).t().reshape(-1)
        kc.view(-1, D)[rows] = turned(s["k"][b, :n], s["gk"], z).reshape(-1, D)
        vc.view(-1, D)[rows] = s["v"][b, :n].double().reshape(-1, D)
    return q_out, kc, vc


def _exact_tree(s):
    B, M, Hq, _ = s["q"].shape
    Hkv = s["kc"].shape[1]
    out = s["out"].double()
    masks, pos = s["mask"].tolist(), s["positions"].tolist()
    for b in range(B):
        T, n = s["lens"][b], s["n_draft"][b]
        rows = _cells(s, b, range(T), Hkv)
        allowed = torch.tensor([[bool(masks[b][i] >> j & 1) for j in range(n)] for i in range(n)], device="cuda")
        allowed = torch.nn.functional.pad(allowed, (T - n, 0), value=True)
        kpos = torch.cat((torch.arange(T - n, device="cuda", dtype=torch.float64),
                          torch.tensor(pos[b][:n], device="cuda", dtype=torch.float64)))
        dist = kpos[None] - kpos[T - n:, None]
        for h in range(Hkv):
            keys = s["kc"].view(-1, D)[rows[h]].double()
            vals = s["vc"].view(-1, D)[rows[h]].double()
            for j in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                e = torch.mm(s["q"][b, :n, j].double(), keys.t()) * s["scale"]
                if s["cap"] > 0:
                    e = s["cap"] * (1 - 2 / (torch.exp(2 * e / s["cap"]) + 1))
                if s["slopes"] is not None:
                    e = e + float(s["slopes"][j]) * dist
                e = torch.where(allowed, e, torch.full_like(e, -math.inf))
                out[b, :n, j] = torch.mm(torch.exp(e - torch.logsumexp(e, 1, keepdim=True)), vals)
    return out


def _exact_commit(s):
    lens = s["context_lens"].tolist()
    B = len(lens)
    nd = [s["M"]] * B if s["draft_lens"] is None else s["draft_lens"].tolist()
    paths, plens = s["path"].tolist(), s["path_lens"].tolist()
    kcs, vcs = [], []
    for kc, vc, table in zip(s["kcs"], s["vcs"], s["tables"]):
        P = kc.shape[2]
        tab = table.tolist()
        frm, to = [], []
        for b in range(B):
            for i in range(plens[b]):
                a, z = lens[b] - nd[b] + paths[b][i], lens[b] - nd[b] + i
                frm.append((tab[b][a // P], a % P))
                to.append((tab[b][z // P], z % P))
        f, t = torch.tensor(frm, device="cuda"), torch.tensor(to, device="cuda")
        for src, dst in ((kc, kcs), (vc, vcs)):
            new = src.double()
            new[t[:, 0], :, t[:, 1]] = src[f[:, 0], :, f[:, 1]].double()
            dst.append(new)
    return (torch.tensor([lens[b] - nd[b] + plens[b] for b in range(B)], device="cuda", dtype=torch.int32), kcs, vcs)
