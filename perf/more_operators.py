"""A drafted step over an INT8 cache: five operators and their plain forms.

``qk_norm_rope_append_axes_int8``  per-head RMSNorm, rotary positions on several axes, and the append
    of K and V as INT8 codes with a scale for each (position, KV head) row;
``kv_cache_read_int8``             rows of the INT8 cache read back as bf16 (measured together with the
    append: a chunk is written, then read back);
``decode_attn_paged_tree_int8``    attention of a tree of drafted tokens over the INT8 cache;
``verify_drafted_tree``            the drafted tokens accepted or rejected against the target's
    probabilities from given random numbers, and the token drawn behind the accepted path;
``kv_cache_commit_path_int8``      the accepted path's codes and scales moved behind the prefix.

A case is measured as one pass over tensors that a serving loop holds anyway. ``own`` selects the
library's kernels; otherwise ``run`` is elementary torch in 32 bits (64 for angles, and for the
probabilities of the verification, whose comparisons decide whole tokens).
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
        # one layer of a verification step: 16 drafted tokens behind 8192 positions
        dict(name="append_draft_m16", op="append", B=1, M=16, Hq=16, Hkv=8, P=16, base=8192, kind="tree", ragged=False),
        # a padded batch of prompt chunks with images, behind prefixes of their own
        dict(name="append_chunks_32k", op="append", B=8, M=4096, Hq=32, Hkv=8, P=64, base=513, kind="image",
             ragged=True),
        # the smallest verification step: a short chat, eight drafted tokens
        dict(name="tree_t520_m8", op="tree", B=1, M=8, Hq=16, Hkv=8, P=16, lens="same", T=520, cap=0.0, bias=False,
             ragged=False, out="bf16"),
        # one long context, capped scores, outputs in 32 bits
        dict(name="tree_t128k_cap_f32", op="tree", B=1, M=16, Hq=32, Hkv=8, P=16, lens="same", T=131072, cap=30.0,
             bias=False, ragged=False, out="f32"),
        # a served batch of ragged lengths up to 32768, trees of up to 16 drafted tokens
        dict(name="tree_ragged_b64", op="tree", B=64, M=16, Hq=16, Hkv=8, P=16, lens="ragged", T=32768, cap=0.0,
             bias=False, ragged=True, out="bf16"),
        # many query rows per key: 64 drafted tokens times groups of 8 heads
        dict(name="tree_wide_b8", op="tree", B=8, M=64, Hq=64, Hkv=8, P=64, lens="same", T=16384, cap=0.0, bias=False,
             ragged=False, out="bf16"),
        # plain single-token decoding of a model with distance biases and capped scores, odd sizes
        dict(name="token_bias_b33", op="tree", B=33, M=1, Hq=24, Hkv=8, P=32, lens="ragged", T=4001, cap=50.0,
             bias=True, ragged=False, out="bf16"),
        # a chat's step whose tokens were the draft model's likeliest ones (no draft probabilities)
        dict(name="verify_b1_m16", op="verify", B=1, M=16, V=151936, dtype="bf16", draft=False, ragged=False),
        # a served batch whose tokens were drawn from the draft model
        dict(name="verify_b64_m16_draft", op="verify", B=64, M=16, V=151936, dtype="bf16", draft=True, ragged=True),
        # wide trees, an odd vocabulary, logits in 32 bits
        dict(name="verify_b24_m64_f32", op="verify", B=24, M=64, V=32003, dtype="f32", draft=False, ragged=True),
        # 28 layers' caches after a step that accepted five of sixteen drafted tokens
        dict(name="commit_l28_m16", op="commit", L=28, B=1, M=16, A=5, Hkv=8, P=16, base=200, ragged=False),
        # the same for a batch with trees of 64, paths of up to 12
        dict(name="commit_l28_b24_m64", op="commit", L=28, B=24, M=64, A=12, Hkv=8, P=16, base=120, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads = [(16, 8), (32, 8), (64, 8), (24, 8), (8, 8), (4, 1), (40, 8), (56, 8)]
    kind = rng.choice(["append", "tree", "tree", "verify", "verify", "commit"])
    Hq, Hkv = rng.choice(heads)
    P = rng.choice([16, 16, 32, 64, 128, 256])
    if kind == "append":
        while True:
            B, M = _log_int(rng, 1, 64), _log_int(rng, 1, 8192)
            if B * M * (2 * Hq + 7 * Hkv) <= 8 * 4096 * (2 * 32 + 7 * 8):
                break
        return dict(op="append", B=B, M=M, Hq=Hq, Hkv=Hkv, P=P, base=_log_int(rng, 1, 4096) - 1,
                    kind="tree" if M <= 64 and rng.random() < 0.5 else "image", ragged=rng.random() < 0.5)
    if kind == "tree":
        while True:
            B, M, T = _log_int(rng, 1, 128), _log_int(rng, 1, 64), _log_int(rng, 65, 131072)
            if B * T * Hkv <= 64 * 16384 * 8 and B * T * Hq * M <= 8 * 16384 * 64 * 64:
                break
        return dict(op="tree", B=B, M=M, Hq=Hq, Hkv=Hkv, P=P, lens=rng.choice(["same", "ragged"]), T=T,
                    cap=rng.choice([0.0, 0.0, 30.0, 50.0]), bias=rng.random() < 0.4, ragged=rng.random() < 0.4,
                    out=rng.choice(["bf16", "bf16", "f32"]))
    if kind == "verify":
        while True:
            B, M, V = _log_int(rng, 1, 64), _log_int(rng, 1, 64), _log_int(rng, 500, 200000)
            dtype, draft = rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.5
            if B * M * V * (2 if dtype == "bf16" else 4) * (2 if draft else 1) <= 64 * 16 * 151936 * 4:
                break
        return dict(op="verify", B=B, M=M, V=V, dtype=dtype, draft=draft, ragged=rng.random() < 0.5)
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
    """Parents (-1: the root), ancestor bit masks (the token itself included) and depths of a drafted tree
    listed parents first. Token 0 is the token that the last step ended with."""
    parent = [-1] + [rng.randint(max(0, (i - 4) // 3), i - 1) for i in range(1, M)]
    mask, depth = [], []
    for i, p in enumerate(parent):
        mask.append((mask[p] if p >= 0 else 0) | (1 << i))
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return parent, mask, depth


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def _signed64(m):
    return m - (1 << 64) if m >= 1 << 63 else m


def _int8_cache(g, pool, Hkv, P):
    """Codes and scales of rows of N(0, 1) values."""
    x = torch.randn(pool, Hkv, P, D, generator=g, device="cuda", dtype=torch.bfloat16)
    s = x.abs().amax(-1).float() / 127
    return (x.float() / s[..., None]).round_().to(torch.int8), s


def prepare(case, seed):
    return {"append": _prepare_append, "tree": _prepare_tree, "verify": _prepare_verify,
            "commit": _prepare_commit}[case["op"]](case, seed)


def _prepare_append(c, seed):
    g, rng = _gen(seed), random.Random(seed)
    B, M, Hq, Hkv, P = c["B"], c["M"], c["Hq"], c["Hkv"], c["P"]
    new = [rng.randint(0, M) if c["ragged"] else M for _ in range(B)]
    lens = [c["base"] + n for n in new]
    max_pages = -(-(c["base"] + M) // P)
    table, pool = _tables(g, lens, P, max_pages, B * max_pages + 1)
    pos = np.zeros((B, M, 3), dtype=np.int32)
    for b in range(B):
        if c["kind"] == "tree":
            pos[b] = (np.asarray(_tree(rng, M)[2]) + c["base"])[:, None]
        else:
            # text, an image of h x w patches at one time step, text again from the largest position on
            lead, w = M // 8, max(1, math.isqrt(max(1, M // 2)))
            img = w * max(1, (M // 2) // w) if M >= 8 else 0
            i = np.arange(M)
            pos[b] = (c["base"] + np.where(i < lead, i, i - img + max(w, img // w if w else 0)))[:, None]
            k = np.arange(min(img, M - lead))
            pos[b, lead:lead + len(k), 0] = c["base"] + lead
            pos[b, lead:lead + len(k), 1] = c["base"] + lead + k // w
            pos[b, lead:lead + len(k), 2] = c["base"] + lead + k % w
    gq = torch.rand(D, generator=g, device="cuda").add_(0.5).bfloat16()
    gk = torch.rand(D, generator=g, device="cuda").add_(0.5).bfloat16()
    k8, ks = _int8_cache(g, pool, Hkv, P)
    v8, vs = _int8_cache(g, pool, Hkv, P)
    return dict(op="append", q=_randn(g, B, M, Hq, D), k=_randn(g, B, M, Hkv, D), v=_randn(g, B, M, Hkv, D), gq=gq,
                gk=gk, positions=_i32(pos), context_lens=_i32(lens), new_lens=_i32(new) if c["ragged"] else None,
                first=_i32([c["base"]] * B), table=table, k8=k8, v8=v8, ks=ks, vs=vs,
                q_out=torch.zeros(B, M, Hq, D, dtype=torch.bfloat16, device="cuda"),
                k_back=torch.zeros(B, M, Hkv, D, dtype=torch.bfloat16, device="cuda"),
                v_back=torch.zeros(B, M, Hkv, D, dtype=torch.bfloat16, device="cuda"),
                # 64 frequencies: the first 16 turn with time, 24 with height, 24 with width
                axes=[0] * 16 + [1] * 24 + [2] * 24)


def _prepare_tree(c, seed):
    g, rng = _gen(seed), random.Random(seed)
    B, M, Hq, Hkv, P, T = c["B"], c["M"], c["Hq"], c["Hkv"], c["P"], c["T"]
    n_draft = [rng.randint(1, M) if c["ragged"] else M for _ in range(B)]
    lens = [max(n, rng.randint(1, T) if c["lens"] == "ragged" else T) for n in n_draft]
    max_pages = -(-max(max(lens), T) // P)
    table, pool = _tables(g, lens, P, max_pages)
    k8, ks = _int8_cache(g, pool, Hkv, P)
    v8, vs = _int8_cache(g, pool, Hkv, P)
    # some keys weigh more than the rest, as in real caches, so that the softmax has peaks
    ks.mul_(torch.where(torch.rand(pool, 1, P, generator=g, device="cuda") < 0.01, 3.0, 1.0))
    # memory behind a sequence's last position holds anything
    for b, t in enumerate(lens):
        if t % P:
            ks[table[b, t // P].long(), :, t % P:] = float("nan")
            vs[table[b, t // P].long(), :, t % P:] = float("nan")
    masks, pos = [], []
    for b in range(B):
        _, m, d = _tree(rng, M)
        masks.append([_signed64(x) for x in m])
        pos.append([lens[b] - n_draft[b] + x for x in d])
    slopes = None
    if c["bias"]:
        slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float32, device="cuda")
    out = torch.zeros(B, M, Hq, D, dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16, device="cuda")
    s = dict(op="tree", q=_randn(g, B, M, Hq, D), k8=k8, v8=v8, ks=ks, vs=vs, table=table, context_lens=_i32(lens),
             draft_lens=_i32(n_draft) if c["ragged"] else None,
             mask=torch.as_tensor(np.asarray(masks, dtype=np.int64)).cuda(), positions=_i32(pos), slopes=slopes,
             cap=c["cap"], scale=1.0 / math.sqrt(D), out=out, lens=lens, n_draft=n_draft)
    if own:
        import paged_gqa_decode_head_gb300 as pg
        n = pg.decode_attn_tree_int8_workspace_size(B, M, Hq, Hkv, D, P, max_pages)
        s["ws"] = torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")
    return s


def _prepare_verify(c, seed):
    g, rng = _gen(seed), random.Random(seed)
    B, M, V = c["B"], c["M"], c["V"]
    dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    n_draft = [rng.randint(1, M) if c["ragged"] else M for _ in range(B)]
    temps = [rng.choice([0.0, 0.6, 0.8, 1.0]) if B > 1 else 0.8 for _ in range(B)]
    target = torch.empty(B, M, V, dtype=dtype, device="cuda")
    draft = torch.empty(B, M, V, dtype=dtype, device="cuda") if c["draft"] else None
    tokens = torch.zeros(B, M, dtype=torch.int32, device="cuda")
    parents = np.full((B, M), -1, dtype=np.int32)
    for b in range(B):
        parents[b] = _tree(rng, M)[0]
        # logits of a language model: a wide bell, and a few tokens far above it
        x = torch.randn(M, V, generator=g, device="cuda").mul_(2.0)
        at = torch.randint(0, V, (M, 8), generator=g, device="cuda")
        x.scatter_add_(1, at, 5.0 + 9.0 * torch.rand(M, 8, generator=g, device="cuda"))
        if b % 4 == 3:  # a grammar that forbids a third of the tokens
            x[:, ::3] = float("-inf")
        target[b] = x
        y = (x + 0.7 * torch.randn(M, V, generator=g, device="cuda")).to(dtype)
        if c["draft"]:
            draft[b] = y
        y = y.float()
        if c["draft"] and temps[b] > 0:  # children drawn from the draft model's distribution, without replacement
            y = y / temps[b] - torch.log(torch.empty(M, V, device="cuda").exponential_(generator=g))
        # child number k of a node is the k-th best token there
        order = torch.topk(y, min(V, max(1, M - 1)), dim=1).indices
        nth, seen = np.zeros(M, dtype=np.int64), {}
        for i in range(1, M):
            nth[i] = seen.get(parents[b, i], 0)
            seen[parents[b, i]] = nth[i] + 1
        if M > 1:
            tokens[b, 1:] = order[torch.as_tensor(parents[b, 1:].astype(np.int64)).cuda(),
                                  torch.as_tensor(nth[1:]).cuda()].int()
    s = dict(op="verify", target=target, draft=draft, tokens=tokens, parents=torch.as_tensor(parents).cuda(),
             draft_lens=_i32(n_draft) if c["ragged"] else None,
             temps=torch.tensor(temps, dtype=torch.float32, device="cuda"),
             accept=torch.rand(B, M, generator=g, device="cuda"),
             noise=torch.empty(B, V, device="cuda").exponential_(generator=g),
             path=torch.zeros(B, M, dtype=torch.int32, device="cuda"),
             path_lens=torch.zeros(B, dtype=torch.int32, device="cuda"),
             new_tokens=torch.zeros(B, M, dtype=torch.int32, device="cuda"),
             logprobs=torch.zeros(B, M, dtype=torch.float32, device="cuda"))
    if own:
        import paged_gqa_decode_head_gb300 as pg
        n = pg.verify_drafted_tree_workspace_size(B, M, V)
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
    tables = []
    for _ in range(L):
        table, pool = _tables(g, lens, P, max_pages, B * max_pages + 1)
        tables.append(table)
    k8, ks = _int8_cache(g, L * pool, Hkv, P)
    v8, vs = _int8_cache(g, L * pool, Hkv, P)
    k8, v8 = k8.view(L, pool, Hkv, P, D), v8.view(L, pool, Hkv, P, D)
    ks, vs = ks.view(L, pool, Hkv, P), vs.view(L, pool, Hkv, P)
    s = dict(op="commit", k8=k8, v8=v8, ks=ks, vs=vs, tables=torch.stack(tables), context_lens=_i32(lens),
             draft_lens=_i32(n_draft) if c["ragged"] else None, M=M, path=_i32(paths), path_lens=_i32(plens),
             lens_out=torch.zeros(B, dtype=torch.int32, device="cuda"))
    if own:
        import paged_gqa_decode_head_gb300 as pg
        s["layers"] = pg.CacheLayersInt8(list(k8), list(v8), list(ks), list(vs), list(s["tables"]))
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return {"append": _run_append, "tree": _run_tree, "verify": _run_verify, "commit": _run_commit}[state["op"]](state)


def _rotate(x, gamma, cos, sin):
    """RMSNorm over the last axis, gain, then the rotation of the pairs (i, i + 64), in 32 bits."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.float()
    a, b = x[..., :64], x[..., 64:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).bfloat16()


def _quantise(x):
    x = x.float()
    s = x.abs().amax(-1) / 127
    return torch.where(s[..., None] > 0, x / s[..., None], 0.0).round().clamp(-127, 127).to(torch.int8), s


def _run_append(s):
    if own:
        import paged_gqa_decode_head_gb300 as pg
        pg.qk_norm_rope_append_axes_int8(s["q"], s["k"], s["v"], s["gq"], s["gk"], s["positions"], s["context_lens"],
                                         s["table"], s["k8"], s["v8"], s["ks"], s["vs"], s["q_out"], s["axes"], THETA,
                                         EPS, new_lens=s["new_lens"])
        pg.kv_cache_read_int8(s["k8"], s["v8"], s["ks"], s["vs"], s["table"], s["context_lens"], s["k_back"],
                              s["v_back"], first=s["first"])
        return s["q_out"], s["k_back"], s["v_back"]
    M, P = s["q"].shape[1], s["k8"].shape[2]
    omega = THETA ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
    phi = s["positions"][..., torch.tensor(s["axes"], device="cuda")].double() * omega
    cos, sin = phi.cos().float()[:, :, None], phi.sin().float()[:, :, None]
    q = _rotate(s["q"], s["gq"], cos, sin)
    k8, ks = _quantise(_rotate(s["k"], s["gk"], cos, sin))
    v8, vs = _quantise(s["v"])
    n = s["new_lens"] if s["new_lens"] is not None else torch.full_like(s["context_lens"], M)
    i = torch.arange(M, device="cuda")[None]
    live = i < n[:, None]
    at = torch.where(live, (s["context_lens"] - n)[:, None] + i, 0)
    page, cell = s["table"].long().gather(1, (at // P).long())[live], (at % P)[live].long()
    s["q_out"][live] = q[live]
    s["k8"][page, :, cell] = k8[live]
    s["v8"][page, :, cell] = v8[live]
    s["ks"][page, :, cell] = ks[live]
    s["vs"][page, :, cell] = vs[live]
    # and read back
    at = s["first"][:, None] + i
    live = at < s["context_lens"][:, None]
    at = torch.where(live, at, 0)
    page, cell = s["table"].long().gather(1, (at // P).long())[live], (at % P)[live].long()
    s["k_back"][live] = (s["k8"][page, :, cell].float() * s["ks"][page, :, cell][..., None]).bfloat16()
    s["v_back"][live] = (s["v8"][page, :, cell].float() * s["vs"][page, :, cell][..., None]).bfloat16()
    return s["q_out"], s["k_back"], s["v_back"]


def _run_tree(s):
    out = s["out"]
    if own:
        import paged_gqa_decode_head_gb300 as pg
        where = {"out_f32": out} if out.dtype == torch.float32 else {"out_bf16": out}
        pg.decode_attn_paged_tree_int8(s["q"], s["k8"], s["v8"], s["ks"], s["vs"], s["table"], s["context_lens"],
                                       s["mask"], s["scale"], positions=s["positions"], draft_lens=s["draft_lens"],
                                       slopes=s["slopes"], softcap=s["cap"], workspace=s["ws"], **where)
        return out
    B, M, Hq, _ = s["q"].shape
    _, Hkv, P, _ = s["k8"].shape
    g, T = Hq // Hkv, s["table"].shape[1] * P
    lens = s["context_lens"].long()
    n = s["draft_lens"].long() if s["draft_lens"] is not None else torch.full_like(lens, M)
    slot, tok = torch.arange(T, device="cuda")[None], torch.arange(M, device="cuda")[None]
    table = s["table"].long()
    k = (s["k8"][table].float() * s["ks"][table][..., None]).transpose(1, 2).reshape(B, Hkv, T, D)
    v = (s["v8"][table].float() * s["vs"][table][..., None]).transpose(1, 2).reshape(B, Hkv, T, D)
    v.masked_fill_((slot >= lens[:, None])[:, None, :, None], 0.0)
    q = s["q"].float().view(B, M, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * M, D)
    x = (q @ k.transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, g, M, T)
    if s["cap"] > 0:
        x = x.div_(s["cap"]).tanh_().mul_(s["cap"])
    child = slot - (lens - n)[:, None]  # [B, T]: the drafted token in this slot
    drafted = (child >= 0) & (child < n[:, None])
    if s["slopes"] is not None:
        where = torch.where(drafted, s["positions"].long().gather(1, child.clamp(0, M - 1)), slot)
        far = (where[:, None] - s["positions"].long()[:, :, None]).float()  # [B, M, T]
        x = x.addcmul_(s["slopes"].view(1, Hkv, g, 1, 1), far[:, None, None])
    bits = (s["mask"][:, :, None] >> child.clamp(0, 63)[:, None]) & 1
    seen = (child[:, None] < 0) | (drafted[:, None] & bits.bool())
    seen &= (tok < n[:, None])[:, :, None]
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    x = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
    o = (x.view(B, Hkv, g * M, T) @ v).view(B, Hkv, g, M, D).permute(0, 3, 1, 2, 4).reshape(B, M, Hq, D)
    live = tok < n[:, None]
    out[live] = o[live].to(out.dtype)
    return out


def _run_verify(s):
    if own:
        import paged_gqa_decode_head_gb300 as pg
        pg.verify_drafted_tree(s["target"], s["tokens"], s["parents"], s["temps"], s["accept"], s["noise"], s["path"],
                               s["path_lens"], s["new_tokens"], logprobs=s["logprobs"], draft_logits=s["draft"],
                               draft_lens=s["draft_lens"], workspace=s["ws"])
        return s["path"], s["path_lens"], s["new_tokens"], s["logprobs"]
    B, M, V = s["target"].shape
    row, column = torch.arange(B, device="cuda"), torch.arange(V, device="cuda")
    n = s["draft_lens"].long() if s["draft_lens"] is not None else torch.full((B,), M, device="cuda")
    greedy = s["temps"] == 0
    heat = torch.where(greedy, 1.0, s["temps"]).double()[:, None]
    cur, count = torch.zeros_like(row), (n > 0).long()
    taken = torch.zeros(B, dtype=torch.double, device="cuda")  # how much of q the residual has lost
    tried = torch.zeros(B, V, dtype=torch.bool, device="cuda")
    path, new = torch.full((B, M + 1), -1, device="cuda"), torch.full((B, M + 1), -1, device="cuda")
    logp = torch.zeros(B, M + 1, dtype=torch.double, device="cuda")
    path[:, 0] = torch.where(n > 0, 0, -1)

    def at(cur):
        """Of the node's row: log p, the residual, its mass, q without the tried tokens, its mass, the first maximum."""
        logits = s["target"][row, cur].double()
        lp = (logits - logits.amax(1, keepdim=True)) / heat
        lp = lp - lp.exp().sum(1, keepdim=True).log()
        p = lp.exp()
        if s["draft"] is None:
            left, q, rest = p.masked_fill(tried, 0.0), None, None
        else:
            q = s["draft"][row, cur].double() / heat
            q = (q - q.amax(1, keepdim=True)).exp()
            q = (q / q.sum(1, keepdim=True)).masked_fill(tried, 0.0)
            left, rest = (p - taken[:, None] * q).clamp_(min=0.0).masked_fill_(tried, 0.0), q.sum(1)
        best = torch.where(logits == logits.amax(1, keepdim=True), column, V).amin(1)
        return lp, p, left, left.sum(1), q, rest, best

    for i in range(1, M):  # children come behind their parents, so one pass over the list walks the tree
        lp, _, left, mass, q, rest, best = at(cur)
        t = s["tokens"][:, i].long()
        wanted = s["accept"][:, i].double() * mass
        if q is not None:
            wanted = wanted * q[row, t] / rest
        here = (i < n) & (s["parents"][:, i] == cur)
        yes = here & torch.where(greedy, t == best, wanted < left[row, t])
        no = here & ~yes & ~greedy
        if q is not None:
            taken = torch.where(no, taken + mass / rest, taken)
        tried[row, t] |= no
        path[row, torch.where(yes, count, M)] = i
        new[row, torch.where(yes, count - 1, M)] = t
        logp[row, torch.where(yes, count - 1, M)] = lp[row, t]
        cur, count = torch.where(yes, i, cur), torch.where(yes, count + 1, count)
        taken, tried = torch.where(yes, 0.0, taken), tried & ~yes[:, None]
    lp, p, left, mass, _, _, best = at(cur)
    race = torch.where((mass > 0)[:, None], left, p) / s["noise"].double()
    last = torch.where(greedy, best, torch.where(race == race.amax(1, keepdim=True), column, V).amin(1))
    new[row, torch.where(n > 0, count - 1, M)] = last
    logp[row, torch.where(n > 0, count - 1, M)] = lp[row, last]
    s["path"].copy_(path[:, :M])
    s["path_lens"].copy_(count)
    s["new_tokens"].copy_(new[:, :M])
    s["logprobs"].copy_(logp[:, :M])
    return s["path"], s["path_lens"], s["new_tokens"], s["logprobs"]


def _run_commit(s):
    if own:
        import paged_gqa_decode_head_gb300 as pg
        pg.kv_cache_commit_path_int8(s["layers"], s["context_lens"], s["path"], s["path_lens"], s["lens_out"], s["M"],
                                     draft_lens=s["draft_lens"])
        return s["lens_out"], s["k8"], s["v8"], s["ks"], s["vs"]
    L, _, _, P, _ = s["k8"].shape
    n = s["draft_lens"] if s["draft_lens"] is not None else torch.full_like(s["context_lens"], s["M"])
    base = (s["context_lens"] - n).long()
    i = torch.arange(s["path"].shape[1], device="cuda")[None]
    live = i < s["path_lens"][:, None]
    src = torch.where(live, base[:, None] + s["path"], 0)
    dst = torch.where(live, base[:, None] + i, 0)
    layer = torch.arange(L, device="cuda")[:, None]
    table = s["tables"].long()
    ps = table.gather(2, (src // P).expand(L, -1, -1))[:, live]
    pd = table.gather(2, (dst // P).expand(L, -1, -1))[:, live]
    rs, rd = (src % P)[live][None], (dst % P)[live][None]
    s["k8"][layer, pd, :, rd] = s["k8"][layer, ps, :, rs]
    s["v8"][layer, pd, :, rd] = s["v8"][layer, ps, :, rs]
    s["ks"][layer, pd, :, rd] = s["ks"][layer, ps, :, rs]
    s["vs"][layer, pd, :, rd] = s["vs"][layer, ps, :, rs]
    s["lens_out"].copy_(base + s["path_lens"])
    return s["lens_out"], s["k8"], s["v8"], s["ks"], s["vs"]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "append":
        toks = c["B"] * c["M"] * (0.5 if c["ragged"] else 1.0)
        return {"bytes": toks * ((2 * c["Hq"] + 4 * c["Hkv"]) * 2 * D + 2 * c["Hkv"] * (D + 4) + 12),
                "flops": toks * (c["Hq"] + c["Hkv"]) * D * 7}
    if c["op"] == "tree":
        keys = c["B"] * c["T"] * (0.5 if c["lens"] == "ragged" else 1.0)
        m = (c["M"] + 1) / 2 if c["ragged"] else c["M"]
        size = 4 if c["out"] == "f32" else 2
        return {"bytes": keys * c["Hkv"] * 2 * (D + 4) + c["B"] * m * c["Hq"] * D * (2 + size),
                "flops": 4.0 * keys * m * c["Hq"] * D}
    if c["op"] == "verify":
        # the rows of the accepted path (some three of a tree's levels), and the noise of the last one
        rows = min(3, c["M"]) * (2 if c["draft"] else 1)
        return {"bytes": c["B"] * c["V"] * (rows * (2 if c["dtype"] == "bf16" else 4) + 4), "flops": 0}
    a = (c["A"] + 1) / 2 if c["ragged"] else c["A"]
    moved = max(0.0, a / 2 - 0.5)  # about half of a path already lies in its place
    return {"bytes": c["L"] * c["B"] * c["Hkv"] * moved * 2 * 2 * (D + 4) + c["B"] * (4 * c["A"] + 16),
            "flops": 0}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "tree": _exact_tree, "verify": _exact_verify, "commit": _exact_commit}[case["op"]](s)


def _cells(s, b, positions):
    """Flat row numbers [Hkv, len(positions)] in a cache seen as [rows, D]."""
    Hkv, P = s["k8"].shape[1:3]
    pos = torch.as_tensor(positions, dtype=torch.int64, device="cuda")
    page = s["table"][b].to(torch.int64)[torch.div(pos, P, rounding_mode="floor")]
    return (page[None] * Hkv + torch.arange(Hkv, device="cuda")[:, None]) * P + torch.remainder(pos, P)[None]


def _exact_append(s):
    B, M = s["q"].shape[:2]
    q_out, k_back, v_back = s["q_out"].double(), s["k_back"].double(), s["v_back"].double()
    turn = torch.tensor([math.exp(-math.log(THETA) * i / 64) for i in range(64)], dtype=torch.float64, device="cuda")
    new = [M] * B if s["new_lens"] is None else s["new_lens"].tolist()

    def turned(x, gain, z):
        x = x.double()
        x = gain.double() * x / (x.square().sum(-1, keepdim=True) / D + EPS).sqrt()
        w = torch.complex(x[..., :64].contiguous(), x[..., 64:].contiguous()) * z
        return torch.cat((w.real, w.imag), dim=-1)

    def stored(x):  # the values that a row's codes and scale stand for
        step = (x.abs().max(dim=-1, keepdim=True).values / 127).float().double()
        return torch.round(x / step.clamp(min=1e-300)).clamp(-127, 127) * step

    for b in range(B):
        n = new[b]
        if n == 0:
            continue
        ang = torch.stack([s["positions"][b, :n, a].double() * turn[i] for i, a in enumerate(s["axes"])], dim=-1)
        z = torch.polar(torch.ones_like(ang), ang)[:, None]
        q_out[b, :n] = turned(s["q"][b, :n], s["gq"], z)
        k_back[b, :n] = stored(turned(s["k"][b, :n], s["gk"], z).bfloat16().double())
        v_back[b, :n] = stored(s["v"][b, :n].double())
    return q_out, k_back, v_back


def _exact_tree(s):
    B, M, Hq, _ = s["q"].shape
    Hkv = s["k8"].shape[1]
    out = s["out"].double()
    masks, pos = s["mask"].tolist(), s["positions"].tolist()
    for b in range(B):
        T, n = s["lens"][b], s["n_draft"][b]
        rows = _cells(s, b, range(T))
        allowed = torch.tensor([[bool(masks[b][i] >> j & 1) for j in range(n)] for i in range(n)], device="cuda")
        allowed = torch.nn.functional.pad(allowed, (T - n, 0), value=True)
        kpos = torch.cat((torch.arange(T - n, device="cuda", dtype=torch.float64),
                          torch.tensor(pos[b][:n], device="cuda", dtype=torch.float64)))
        dist = kpos[None] - kpos[T - n:, None]
        for h in range(Hkv):
            keys = s["k8"].view(-1, D)[rows[h]].double() * s["ks"].view(-1, 1)[rows[h]].double()
            vals = s["v8"].view(-1, D)[rows[h]].double() * s["vs"].view(-1, 1)[rows[h]].double()
            for j in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                e = torch.mm(s["q"][b, :n, j].double(), keys.t()) * s["scale"]
                if s["cap"] > 0:
                    e = s["cap"] * (1 - 2 / (torch.exp(2 * e / s["cap"]) + 1))
                if s["slopes"] is not None:
                    e = e + float(s["slopes"][j]) * dist
                e = torch.where(allowed, e, torch.full_like(e, -math.inf))
                out[b, :n, j] = torch.mm(torch.exp(e - torch.logsumexp(e, 1, keepdim=True)), vals)
    return out


def _exact_verify(s):
    B, M, V = s["target"].shape
    path, new, logp = [[-1] * M for _ in range(B)], [[-1] * M for _ in range(B)], [[0.0] * M for _ in range(B)]
    lens = [M] * B if s["draft_lens"] is None else s["draft_lens"].tolist()
    tokens, parents, u = s["tokens"].tolist(), s["parents"].tolist(), s["accept"].double().tolist()
    count = [0] * B
    for b in range(B):
        if lens[b] == 0:
            continue
        t = float(s["temps"][b])
        node = 0
        while True:
            path[b][count[b]] = node
            count[b] += 1
            logits = s["target"][b, node].double()
            probs = torch.exp(logits / (t or 1.0) - torch.logsumexp(logits / (t or 1.0), 0))
            children = [i for i in range(node + 1, lens[b]) if parents[b][i] == node]
            accepted, token = None, None
            if t == 0:
                token = int(torch.nonzero(logits == logits.max())[0])
                accepted = next((i for i in children if tokens[b][i] == token), None)
            else:
                left = probs
                if s["draft"] is not None:
                    z = s["draft"][b, node].double() / t
                    q = torch.exp(z - torch.logsumexp(z, 0))
                for i in children:
                    c = tokens[b][i]
                    left = left / left.sum()
                    if s["draft"] is None:
                        ratio = float(left[c])
                    else:
                        q = q / q.sum()
                        ratio = float(left[c]) / max(float(q[c]), 1e-300)
                    if u[b][i] < ratio:
                        accepted, token = i, c
                        break
                    left = left.clone() if s["draft"] is None else torch.relu(left - q)
                    left[c] = 0
                    if s["draft"] is not None:
                        q = q.clone()
                        q[c] = 0
                if accepted is None:
                    token = int(torch.argmax((left if float(left.sum()) > 0 else probs) / s["noise"][b].double()))
            new[b][count[b] - 1] = token
            logp[b][count[b] - 1] = float(torch.log(probs[token]))
            if accepted is None:
                break
            node = accepted
    dev = dict(device="cuda")
    return (torch.tensor(path, dtype=torch.int32, **dev), torch.tensor(count, dtype=torch.int32, **dev),
            torch.tensor(new, dtype=torch.int32, **dev), torch.tensor(logp, dtype=torch.float64, **dev))


def _exact_commit(s):
    lens = s["context_lens"].tolist()
    B, P = len(lens), s["k8"].shape[3]
    nd = [s["M"]] * B if s["draft_lens"] is None else s["draft_lens"].tolist()
    paths, plens, tabs = s["path"].tolist(), s["path_lens"].tolist(), s["tables"].tolist()
    new = [s["k8"].clone(), s["v8"].clone(), s["ks"].double(), s["vs"].double()]
    frm, to = [], []
    for layer, tab in enumerate(tabs):
        for b in range(B):
            for i in range(plens[b]):
                a, z = lens[b] - nd[b] + paths[b][i], lens[b] - nd[b] + i
                frm.append((layer, tab[b][a // P], a % P))
                to.append((layer, tab[b][z // P], z % P))
    f, t = torch.tensor(frm, device="cuda").t(), torch.tensor(to, device="cuda").t()
    for k, old in enumerate((s["k8"], s["v8"], s["ks"], s["vs"])):
        new[k][t[0], t[1], :, t[2]] = old[f[0], f[1], :, f[2]].to(new[k].dtype)
    return (torch.tensor([lens[b] - nd[b] + plens[b] for b in range(B)], device="cuda", dtype=torch.int32), *new)
