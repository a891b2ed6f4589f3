"""Drafted-tree decoding in 64 bits (numpy), and how far a kernel in 32 bits may be from it.

Attention: x_j = scale <q, K_j>; capped: c tanh(x_j / c); biased: + slope (pos_j - pos_i); softmax over the
keys that the query sees; out = sum_j p_j V_j.

Bound on the kernel's fp32 output. A relative error e_j of weight j moves the output by at most
sum_j p_j |V_j| e_j + |out| sum_j p_j e_j. e_j collects, in units of u = 2^-24:
  - the score: 128 products summed in fp32 in any order, at most 128 u sum_d |q_d K_jd| scale, and its own
    scaling, 2 u |x_j|;
  - the cap: up to |x| = c a polynomial within 5e-8 (1 u) of tanh(y) / y, evaluated with at most 4 u more; past
    it 1 - 2 / (1 + e^2y), where 2 / (1 + e^2y) <= 0.24 carries exp2 and reciprocal at 2 ulp each: either way
    8 u of the capped score, the rounding of the argument counted with the score;
  - the bias: product and sum, 2 u (|bias| + |x|);
  - the exponent: argument (x_j - max) log2 e rounded twice, 4 u (|x_j| + |max|), and exp2 itself, 8 u;
  - the weight's hi + lo bf16 pair: 2^-16;
and the fp32 sums over the keys (weights, products, rescales, the merge of partial states): each adds at
most u per partial sum; with sums of T terms split over tiles of at most 128 keys 2 (128 + T / 128 + 64) u
covers them. K and V rows' own rounding is part of the input.
"""
import numpy as np

U = 2.0 ** -24


def widen(bits):
    with np.errstate(invalid="ignore"):
        return (np.ascontiguousarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def gather(cache, table_row, T, P):
    """[Hkv, T, D] bit patterns of positions 0 .. T-1."""
    n = -(-T // P)
    pages = cache[table_row[:n]]  # [n, Hkv, P, D]
    return pages.transpose(1, 0, 2, 3).reshape(cache.shape[1], n * P, cache.shape[3])[:, :T]


def attention(q, k_cache, v_cache, table, context_lens, masks, scale, draft_lens=None, positions=None, slopes=None,
              softcap=0.0, skip=None):
    """(out, bound) [B, M, Hq, D] float64; rows i >= n_b stay NaN. masks: int [B][M] (python ints or uint64).
    skip(b, j): keys left out for every query (a page outside the pool)."""
    B, M, Hq, D = q.shape
    _, Hkv, P, _ = k_cache.shape
    g = Hq // Hkv
    out = np.full((B, M, Hq, D), np.nan)
    bound = np.full((B, M, Hq, D), np.nan)
    for b in range(B):
        T = int(context_lens[b])
        n = M if draft_lens is None else int(draft_lens[b])
        prefix = T - n
        tab = np.array(table[b], copy=True)
        gone = np.zeros(T, dtype=bool)
        if skip is not None:
            gone = np.array([skip(b, j) for j in range(T)], dtype=bool)
            tab[(tab < 0) | (tab >= k_cache.shape[0])] = 0
        K = widen(gather(k_cache, tab, T, P))
        V = widen(gather(v_cache, tab, T, P))
        kpos = np.arange(T, dtype=np.float64)
        if positions is not None:
            kpos[prefix:] = positions[b][:n]
        for i in range(n):
            seen = np.ones(T, dtype=bool)
            m = int(masks[b][i])
            seen[prefix:] = [(m >> j) & 1 == 1 for j in range(n)]
            seen &= ~gone
            idx = np.nonzero(seen)[0]
            for h in range(Hq):
                if idx.size == 0:
                    out[b, i, h] = 0
                    bound[b, i, h] = 0
                    continue
                qv = widen(q[b, i, h])
                k, v = K[h // g][idx], V[h // g][idx]
                x = scale * (k @ qv)
                e = 128 * U * abs(scale) * (np.abs(k) @ np.abs(qv)) + 2 * U * np.abs(x)
                if softcap > 0:
                    x = softcap * np.tanh(x / softcap)
                    e = e + 8 * U * np.abs(x)
                if slopes is not None:
                    bias = float(slopes[h]) * (kpos[idx] - float(positions[b][i]))
                    e = e + 2 * U * (np.abs(bias) + np.abs(x))
                    x = x + bias
                e = e + 4 * U * (np.abs(x) + np.abs(x.max())) + 8 * U + 2.0 ** -16
                e = e + 2 * (128 + T / 128 + 64) * U
                p = np.exp(x - x.max())
                p /= p.sum()
                o = p @ v
                out[b, i, h] = o
                bound[b, i, h] = (p * e) @ np.abs(v) + np.abs(o) * (p @ e)
    return out, bound


def rotate(x, gamma, positions, axes, theta, eps):
    """RoPE(RMSNorm(x) gamma): x bits [..., D], positions [..., n_axes] (broadcast over the heads by the caller)."""
    x = widen(x)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * widen(gamma)
    r = np.arange(64)
    phi = positions.astype(np.float64)[..., np.asarray(axes)] * float(theta) ** (-2.0 * r / 128)
    c, s = np.cos(phi), np.sin(phi)
    a, b = y[..., :64], y[..., 64:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


def rotate_bound(x, gamma, eps):
    """|fp32 result - rotate()|: the norm (128 terms: 128 u; rsqrt 2 ulp), three products and the angle's 1e-6 rad
    each move the pair by at most that share of its length."""
    x = widen(x)
    y = np.abs(x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * widen(gamma))
    pair = np.hypot(y[..., :64], y[..., 64:])
    return np.concatenate([pair, pair], -1) * (140 * U + 1e-6)


def random_tree(gen, M, roots=1):
    """Parents first; ancestor masks (python ints, the token included) and depths."""
    parent = [-1 if i < roots else int(gen.integers(max(0, (i - 3) // 2), i)) for i in range(M)]
    masks, depth = [], []
    for i, p in enumerate(parent):
        masks.append((masks[p] if p >= 0 else 0) | (1 << i))
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return masks, depth
