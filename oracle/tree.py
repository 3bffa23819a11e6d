"""Trees of drafted tokens: attention, verification, packing.

TEST INFRASTRUCTURE (oracle). The pages describe decoding one token at a time;
these are the definitions stated in include/v4kv.h, evaluated in fp64.

A tree is the list of its nodes' parents (index within the sequence, -1 for a
root), every parent before its children. Node i of a sequence with L cached
tokens sits at position L + depth(i).
"""
import numpy as np

from . import attention
from .rope import rope_rotate


def family(parents, i):
    """Node i and its ancestors, the root last. A parent that does not come
    before its child counts as none."""
    out = [i]
    while 0 <= parents[out[-1]] < out[-1]:
        out.append(int(parents[out[-1]]))
    return out


def attend_node(q, i, parents, k_tree, main, window, cached, ratio, window_len, sm_scale, topk_row=None,
                theta=1e6, rope_dim=64, rope_offset=448):
    """Output of node i, fp64 [H, D], and the sums of |weight * value| behind it.

    q [H, D]; k_tree [n, D] values of the sequence's nodes; main / window as in
    attention.decode_one. It attends to the entries that end at or before
    pos + 1 - window_len (or the non-negative top-k), the cached tokens from
    there on, and its family.
    """
    fam = family(parents, i)
    pos = cached + len(fam) - 1
    w0 = max(0, pos + 1 - window_len)
    ent = list(range(w0 // ratio)) if topk_row is None else [int(j) for j in topk_row if j >= 0]
    toks = list(range(min(w0, cached), cached))
    parts = [np.asarray(k_tree, dtype=np.float64)[fam]]
    if ent:
        parts.append(attention.gather(main["data"], main["scales"], main["dtype"], main["block_table_row"], ent))
    if toks:
        parts.append(attention.gather(window["data"], window["scales"], window["dtype"],
                                      window["block_table_row"], toks))
    v = np.concatenate(parts, axis=0)
    q = np.asarray(q, dtype=np.float64)
    s = sm_scale * (q @ v.T)
    p = np.exp(s - s.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    out = rope_rotate(p @ v, pos, theta, rope_dim, rope_offset, inverse=True)
    mass = p @ np.abs(v)
    # a rotated pair mixes its two magnitudes
    rot = slice(rope_offset, rope_offset + rope_dim)
    pair = mass[:, rot].reshape(mass.shape[0], -1, 2).sum(axis=2)
    mass[:, rot] = np.repeat(pair, 2, axis=1)
    return out, mass


def verify(target, draft, parents, tokens, accept_u, sample_u):
    """(path, next token) of one sequence: target and draft [n, V] (draft None
    for fixed guesses), fp64 arithmetic on the given values."""
    target = np.asarray(target, dtype=np.float64)
    if draft is not None:
        draft = np.asarray(draft, dtype=np.float64)
        draft = np.where(draft > 0, draft, 0.0)
    n, vocab = target.shape
    now, path = 0, [0]
    while True:
        p = np.where(target[now] > 0, target[now], 0.0)
        rest, total, accepted = p.copy(), 1.0, None
        for c in range(now + 1, n):
            if parents[c] != now or not 0 <= tokens[c] < vocab:
                continue
            x = tokens[c]
            qx = 1.0 if draft is None else float(draft[now, x])
            if float(accept_u[c]) * qx * total < rest[x]:
                accepted = c
                break
            if draft is None:
                total -= rest[x]
                rest[x] = 0.0
            else:
                rest = np.maximum(rest - total * draft[now], 0.0)
                total = rest.sum()
        if accepted is None:
            break
        now = accepted
        path.append(now)
    if not rest.sum() > 0:
        rest = p
    sums = np.cumsum(rest)
    if not (sums[-1] > 0 and np.isfinite(sums[-1])):
        return path, -1
    over = np.nonzero(sums > float(sample_u) * sums[-1])[0]
    return path, int(over[0]) if over.size else int(np.nonzero(rest > 0)[0][-1])
