"""Definitions in 64 bits of the drafted-tree and token log-probability operators (numpy, CPU)."""
import numpy as np


def see_sets(parents):
    """Per sequence and node, the set A(i) (empty: no node)."""
    out = []
    for row in np.asarray(parents):
        sets = []
        for i, p in enumerate(row):
            if p == -1:
                sets.append({i})
            elif 0 <= p < i and sets[p]:
                sets.append(sets[p] | {i})
            else:
                sets.append(set())
        out.append(sets)
    return out


def tree_attention_ref(qkv, kv, lengths, parents, nh):
    """(y, bound) [B, N, C]: the attention, and sum_j p_j |v_j| (what roundings of p scale with)."""
    B, N, _, C = qkv.shape
    hs = C // nh
    y, a = np.zeros((B, N, C)), np.zeros((B, N, C))
    sees = see_sets(parents)
    for b in range(B):
        n = int(lengths[b])
        for i in range(N):
            nodes = sorted(sees[b][i])
            if not nodes:
                continue
            k = np.concatenate([kv[b, :n, 0], qkv[b, nodes, 1]]).reshape(-1, nh, hs)
            v = np.concatenate([kv[b, :n, 1], qkv[b, nodes, 2]]).reshape(-1, nh, hs)
            s = np.einsum("hd,jhd->hj", qkv[b, i, 0].reshape(nh, hs), k) / np.sqrt(hs)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            y[b, i] = np.einsum("hj,jhd->hd", p, v).reshape(-1)
            a[b, i] = np.einsum("hj,jhd->hd", p, np.abs(v)).reshape(-1)
    return y, a


def accept_ref(parents, tok, chosen, lengths, cap):
    paths, counts, nxt = [], [], []
    for b, sets in enumerate(see_sets(parents)):
        best = []
        for i, s in enumerate(sets):
            nodes = sorted(s)
            if nodes and all(tok[b][c] == chosen[b][p] for p, c in zip(nodes, nodes[1:])) and len(nodes) > len(best):
                best = nodes
        best = best[:max(0, cap - int(lengths[b]))]
        paths.append(best)
        counts.append(len(best))
        nxt.append(int(chosen[b][best[-1]]) if best else -1)
    return paths, counts, nxt


def logprob_ref(z, tokens, k, T):
    """(logp, entropy, lse, top ids, top logp) of fp64 logits [rows, V]."""
    rows, V = z.shape
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        s = z / T
        m = s.max(1, keepdims=True)
        e = s - m                      # s - lse would lose log(sum) next to a maximum beyond 2^53
        log_sum = np.log(np.exp(e).sum(1, keepdims=True))
        lse = np.where(np.isneginf(m[:, 0]), -np.inf, (m + log_sum)[:, 0])
        lp = e - log_sum
        p = np.exp(lp)
        ent = -np.where(p == 0, 0.0, p * lp).sum(1)
        ent = np.where(np.isneginf(lse), np.nan, ent)
        logp = np.where(tokens >= 0, lp[np.arange(rows), np.clip(tokens, 0, V - 1)], 0.0)
    # NaN first, then by value, equal values by index
    order = np.lexsort((np.broadcast_to(np.arange(V), z.shape), np.where(np.isnan(z), -np.inf, -z), ~np.isnan(z)))
    ids = order[:, :k]
    return logp, ent, lse, ids, np.take_along_axis(lp, ids, 1)


def logprob_grad_ref(z, tokens, g, h, T):
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        _, ent, lse, _, _ = logprob_ref(z, tokens, 0, T)
        lp = z / T - lse[:, None]      # lse is an argument of the gradient, in 32 bits
        p = np.exp(lp)
        g = np.where(tokens >= 0, g, 0.0)
        d = -p * g[:, None] - h[:, None] * np.where(p == 0, 0.0, p * (lp + ent[:, None]))
    rows = np.nonzero(tokens >= 0)[0]
    d[rows, tokens[rows]] += g[rows]
    d[np.isneginf(lse) | ((g == 0) & (h == 0))] = 0.0
    return d / T
