"""Plain 64-bit implementations of the cache and beam calls (numpy), for the tests: straight
from the definitions in include/jf.h, one sequence and one kv-head at a time.  They share no
code with the kernels."""
import numpy as np

PAGE = 16


def rows_of(cache, table, t):
    """Rows t of a sequence: [len(t)][Hkv][D] of a [pages][16][Hkv][D] pool."""
    t = np.asarray(t, np.int64)
    return cache[table[t // PAGE], t % PAGE]


def attention_weight(q, k, table, prefix, nodes, lse, weight, out, scale):
    """One sequence.  q [N][Hq][D], k pool (all float64), nodes: the rows' node ids, lse
    [Hq][N], weight [Hkv][cap] or None, out [Hkv][cap] before the call.  Returns (out, tol):
    tol bounds the fp32 kernel's distance.  With u = 2^-23 (twice the rounding of one fp32
    operation, which also covers a truncating accumulation): a score's D products and sums
    are off by D u sum |q_d k_d|, the exponent by u times its size for its two products and
    one sum, the exponential by 4 u relative; adding n terms and the old weight by (n + 1) u
    of the total."""
    Hq, Hkv = q.shape[1], k.shape[2]
    G, R, D, u = Hq // Hkv, len(nodes), q.shape[2], 2.0 ** -23
    L = prefix + R
    out = out.astype(np.float64).copy()
    tol = np.zeros_like(out)
    if L == 0:
        return out, tol
    kk = rows_of(k, table, np.arange(L))
    seen = np.arange(L)[None, :] <= prefix + np.arange(R)[:, None]
    for g in range(Hkv):
        total, off = np.zeros(L), np.zeros(L)
        if weight is not None:
            total[:prefix] = weight[g, :prefix]
        for h in range(g * G, (g + 1) * G):
            s = scale * q[nodes, h] @ kk[:, g].T if R else np.zeros((0, L))
            a = scale * np.abs(q[nodes, h]) @ np.abs(kk[:, g]).T if R else s
            z = lse[h, nodes].astype(np.float64)[:, None]
            dead = np.isneginf(z)
            z = np.where(dead, 0.0, z)
            p = np.where(seen & ~dead, np.exp(s - z), 0.0)
            total += p.sum(0)
            off += (p * u * (D * a + 2 * (np.abs(s) + np.abs(z)) + 4)).sum(0)
        out[g, :L] = total
        tol[g, :L] = off + (R * G + 1) * u * np.abs(total)
    return out, tol


def select_kept(weight, seq_len, sink, recent, budget):
    B, H, cap = weight.shape
    keep = np.full((B, H, budget), -1, np.int32)
    for b in range(B):
        L = int(seq_len[b])
        for g in range(H):
            if L <= budget:
                keep[b, g, :L] = np.arange(L)
                continue
            mid = np.arange(sink, L - recent)
            w = weight[b, g, mid].astype(np.float64)
            # NaN below -inf; ties to the lowest position
            order = sorted(range(len(mid)), key=lambda i: (np.isnan(w[i]), -w[i] if not np.isnan(w[i]) else 0.0, i))
            chosen = mid[np.array(order[:budget - sink - recent], np.int64)]
            keep[b, g] = np.sort(np.concatenate([np.arange(sink), chosen, np.arange(L - recent, L)]))
    return keep, np.minimum(seq_len, budget).astype(np.int32)


def evict_kv(k, v, table, new_table, keep, kept_len, weight):
    """Copies of (k, v, weight) after the move (weight in place of the old one)."""
    k2, v2, w2 = k.copy(), v.copy(), None if weight is None else weight.copy()
    B, H, _ = keep.shape
    for b in range(B):
        n = int(kept_len[b])
        j = np.arange(n)
        for g in range(H):
            t = keep[b, g, :n].astype(np.int64)
            for new, old in ((k2, k), (v2, v)):
                new[new_table[b, j // PAGE], j % PAGE, g] = old[table[b, t // PAGE], t % PAGE, g]
            if weight is not None:
                w2[b, g, :n] = weight[b, g, t]
    return k2, v2, w2


def beam_scores(logits, score, finished, eos):
    """s(w, v) of one prompt, [W][V] float64."""
    x = logits.astype(np.float64)
    W, V = x.shape
    out = np.full((W, V), -np.inf)
    for w in range(W):
        if finished is not None and finished[w]:
            out[w, eos] = score[w]
        elif not np.isneginf(score[w]):
            m = x[w].max()
            if not np.isneginf(m):
                out[w] = np.float64(score[w]) + (x[w] - (m + np.log(np.exp(x[w] - m).sum())))
    return out


def beam_fork(table, prefix, parent, fresh):
    """(new_table, new_len, copies): copies = [(fresh page, source page, slots)]."""
    B, K = parent.shape
    W, cap = table.shape[0] // B, table.shape[1]
    new_table = np.full((B * K, cap), -1, np.int32)
    new_len = np.zeros(B * K, np.int32)
    copies = []
    for b in range(B):
        for j in range(K):
            row = b * W + int(parent[b, j])
            P = int(prefix[row])
            full = P // PAGE
            new_len[b * K + j] = P
            new_table[b * K + j, :full] = table[row, :full]
            if full < cap:
                new_table[b * K + j, full] = fresh[b, j]
                if P % PAGE:
                    copies.append((int(fresh[b, j]), int(table[row, full]), P % PAGE))
    return new_table, new_len, copies
