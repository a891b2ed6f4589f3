"""Drafted-tree decoding over an INT8 cache, and the verification of drafted trees, in 64 bits (numpy), with how far
kernels in 32 bits may be from them.

Attention: K_j = code ks_j, V_j = code vs_j; x_j = scale <q, K_j>; capped: c tanh(x_j / c); biased: + slope (pos_j -
pos_i); softmax over the keys that the query sees; out = sum_j p_j V_j.

Bound on the kernel's fp32 output, u = 2^-24. A relative error e_j of weight j moves the output by at most sum_j p_j |V_j|
e_j + |out| sum_j p_j e_j. e_j collects:
  - the score: 128 exact products (codes and queries are exact in fp16) summed in fp32 in any order, at most 128 u sum_d
    |q_d K_jd| scale; on a tensor core that rounds towards zero twice that; the scales' products, 4 u |x_j|;
  - the cap: up to |x| = c a polynomial within 1 u of tanh(y) / y and 4 u of evaluation, past it an exponential form at 8 u
    of the capped score;
  - the bias, formed relative to a key that it favours: product and sum, 2 u (|bias| + |x|), |bias| from that key;
  - the exponent: its argument rounded twice, 4 u (|x_j| + |max|), and exp2 itself, 8 u; the reference that the
    argument is taken against lies at most 8 (in base 2) from the maximum, which the same terms cover;
  - the weight times vs_j (1 u) and its fp16 pair: 11 + 11 bits, 2^-21;
  - sums of weights and products over the keys, the two streams' and the pieces' joins: 2 (128 + T / 128 + 64) u.
The fp16 pair's rest has an absolute floor besides: weights are scaled by a power of two so that the largest V scale of a
stream's keys is at least 8; fp16's smallest step is 2^-24, half of it lost, so a key adds at most 2^-25 / 8 |code| max vs
relative to a weight of 1, and the row's sum of weights is at least 1 (the key that set the reference): T 2^-28 127 max vs.
"""
import numpy as np

from tree_reference import U, widen


def rows_of(cache, table_row, T, P):
    """[Hkv, T, ...] of positions 0 .. T - 1."""
    n = -(-T // P)
    pages = cache[table_row[:n]]
    pages = np.moveaxis(pages, 0, 1)
    return pages.reshape(cache.shape[1], n * P, *cache.shape[3:])[:, :T]


def quantize(x):
    """Codes and scales of rows [..., 128] of float32 values, in binary32 as the definition says."""
    x = np.asarray(x, np.float32)
    amax = np.abs(x).max(-1)
    s = (amax / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.rint((x / s[..., None]).astype(np.float32))
    code = np.where(s[..., None] > 0, code, 0)
    return np.clip(code, -127, 127).astype(np.int8), s


def attention(q, k8, v8, ks, vs, table, context_lens, masks, scale, n_drafted, positions=None, slopes=None, softcap=0.0,
              skip=None):
    """(out, bound) [B, M, Hq, 128] float64; rows i >= n_b stay NaN."""
    B, M, Hq, D = q.shape
    _, Hkv, P, _ = k8.shape
    g = Hq // Hkv
    out, bound = np.full((B, M, Hq, D), np.nan), np.full((B, M, Hq, D), np.nan)
    for b in range(B):
        T, n = int(context_lens[b]), int(n_drafted[b])
        prefix = T - n
        if n == 0:
            continue
        tab = np.array(table[b], copy=True)
        gone = np.zeros(T, bool)
        if skip is not None:
            gone = np.array([skip(b, j) for j in range(T)], bool)
        tab[(tab < 0) | (tab >= k8.shape[0])] = 0
        K = rows_of(k8, tab, T, P).astype(np.float64) * rows_of(ks, tab, T, P).astype(np.float64)[..., None]
        V = rows_of(v8, tab, T, P).astype(np.float64) * rows_of(vs, tab, T, P).astype(np.float64)[..., None]
        top_v = np.nan_to_num(np.abs(rows_of(vs, tab, T, P)[:, ~gone]), nan=0.0, posinf=0.0).max(1, initial=0.0)
        kpos = np.arange(T, dtype=np.float64)
        if positions is not None:
            kpos[prefix:] = positions[b][:n]
        for i in range(n):
            seen = np.ones(T, bool)
            seen[prefix:] = [(int(masks[b][i]) >> j) & 1 == 1 for j in range(n)]
            idx = np.nonzero(seen & ~gone)[0]
            if idx.size == 0:
                out[b, i], bound[b, i] = 0, 0
                continue
            for h in range(Hkv):
                qv = widen(q[b, i, h * g:(h + 1) * g])  # [g, D]
                k, v = K[h][idx], V[h][idx]
                x = scale * (qv @ k.T)
                e = 256 * U * abs(scale) * (np.abs(qv) @ np.abs(k).T) + 4 * U * np.abs(x)
                if softcap > 0:
                    x = softcap * np.tanh(x / softcap)
                    e = e + 8 * U * np.abs(x)
                if slopes is not None:
                    sl = np.asarray(slopes, np.float64)[h * g:(h + 1) * g, None]
                    favoured = np.where(sl < 0, kpos[idx].min(), kpos[idx].max())
                    bias = sl * (kpos[idx][None] - favoured)
                    e = e + 2 * U * (np.abs(bias) + np.abs(sl) * 64 + np.abs(x))
                    x = x + bias
                peak = x.max(-1, keepdims=True)
                e = e + 4 * U * (np.abs(x) + np.abs(peak)) + 9 * U + 2.0 ** -21
                e = e + 2 * (128 + T / 128 + 64) * U
                p = np.exp(x - peak)
                p /= p.sum(-1, keepdims=True)
                o = p @ v
                out[b, i, h * g:(h + 1) * g] = o
                bound[b, i, h * g:(h + 1) * g] = ((p * e) @ np.abs(v) + np.abs(o) * (p * e).sum(-1, keepdims=True) +
                                                  T * 2.0 ** -28 * 127 * top_v[h])
    return out, bound


# ------------------------------------------------------------------ verification
def usable(x):
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    return np.minimum(x, float(np.finfo(np.float32).max))


def softmax(x, t):
    if x.max() == -np.inf:
        return np.zeros_like(x)
    with np.errstate(over="ignore", invalid="ignore"):
        e = np.where(x == -np.inf, 0.0, np.exp((x - x.max()) / t))
    return e / e.sum()


def verify(target, draft, tokens, parents, n, t, u, noise, A):
    """One sequence: (path, new_tokens, logprobs, margin). target, draft [M, V] float64 or None. margin: how near any
    comparison that was made came to a tie, relative: below it a kernel in 32 bits may decide otherwise."""
    path, new, logp, margin = [], [], [], np.inf
    V = target.shape[1]
    if n == 0:
        return path, new, logp, margin
    node = 0
    while True:
        path.append(node)
        row = usable(target[node])
        p = softmax(row, t or 1.0)
        children = [i for i in range(node + 1, n) if parents[i] == node and 0 <= tokens[i] < V]
        if len(path) == A or row.max() == -np.inf:
            children = []
        accepted, token, left = None, -1, p
        if t == 0:
            if row.max() > -np.inf:
                token = int(np.nonzero(row == row.max())[0][0])
                accepted = next((i for i in children if tokens[i] == token), None)
        else:
            q = None if draft is None else softmax(usable(draft[node]), t)
            tried = set()
            for i in children:
                c = tokens[i]
                s = left.sum()
                pc = 0.0 if c in tried else left[c] / s if s > 0 else 0.0
                qs = 1.0 if q is None else q.sum()
                given = q is None or qs == 0  # nothing is left of q: the child counts as given
                qc = 1.0 if given else q[c] / qs
                if pc != u[i] * qc:
                    # p and q themselves are known to some 1e-6 of p: the residual, and so the test, to that over its share
                    margin = min(margin, abs(pc - u[i] * qc) / max(pc, u[i] * qc) * min(1.0, s))
                if u[i] * qc < pc:
                    accepted, token = i, c
                    break
                left = left.copy()
                if q is not None:
                    if not given:
                        left = np.maximum(left - s / qs * q, 0.0)
                    q = q.copy()
                    q[c] = 0.0
                left[c] = 0.0
                tried.add(c)
            if accepted is None and row.max() > -np.inf:
                if left.sum() <= 0:
                    left, margin = p, 0.0
                score = left / noise.astype(np.float64)
                token = int(np.argmax(score))
                best = np.sort(score)[-2:]
                if V > 1 and best[0] > 0:
                    margin = min(margin, (best[1] - best[0]) / best[1] * min(1.0, left[token] / p[token]))
        new.append(token)
        logp.append(float(np.log(p[token])) if token >= 0 else 0.0)
        if accepted is None:
            return path, new, logp, margin
        node = accepted
