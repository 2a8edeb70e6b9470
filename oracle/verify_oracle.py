"""CPU oracle of the verification of drafted tokens: fp64, one sequence and one token after the
other.

Besides the result it says how sure it is: the smallest distance, over the decisions that led to
it, between what a decision compares, in units of the probability that the weights' rounding is
relative to.  Pins live in ``tests/test_verify_host.py``.
"""

from __future__ import annotations

import numpy as np


def softmax(logits, temperature):
    """Probabilities of a row of logits (NaN: none), or None where its largest is not finite."""
    x = np.where(np.isnan(logits), -np.inf, np.asarray(logits, dtype=np.float64))
    top = x.max()
    if not np.isfinite(top):
        return None
    w = np.exp((x - top) / temperature)
    return w / w.sum()


def draw(weights, u):
    """First index whose running sum passes u times the whole sum, and the distance of that
    number to the nearest end of the index's stretch (relative to the sum)."""
    cum = np.cumsum(weights)
    goal = min(max(float(u), 0.0), 1.0) * cum[-1]
    hit = np.nonzero(cum > goal)[0]
    i = int(hit[0]) if len(hit) else int(np.nonzero(weights)[0][-1])
    low = cum[i] - weights[i]
    return i, min(abs(goal - low) if low > 0 else 1.0, abs(cum[i] - goal)) / cum[-1]


def best(logits):
    """First largest logit; None where it is not finite."""
    x = np.where(np.isnan(logits), -np.inf, np.asarray(logits, dtype=np.float64))
    return int(np.argmax(x)) if np.isfinite(x.max()) else None


def verify(logits, row_start, tokens, u_sample, max_path, parents=None, temperature=None, draft=None, u_accept=None):
    """Returns (path [S, max_path], lens [S], next [S], sure [S])."""
    vocab = logits.shape[1]
    out_path, out_len, out_next, out_sure = [], [], [], []
    for s in range(len(row_start) - 1):
        r0, n = int(row_start[s]), int(row_start[s + 1] - row_start[s])
        temp = 1.0 if temperature is None else float(temperature[s])
        if not 2.0 ** -100 <= temp <= 2.0 ** 100:
            temp = 0.0
        up = [i - 1 if parents is None else int(parents[r0 + i]) for i in range(n)]
        path, nxt, sure = [], -1, 1.0
        c = 0 if n else None
        while c is not None:
            path.append(c)
            row = logits[r0 + c]
            kids = [i for i in range(c + 1, n) if up[i] == c] if len(path) < max_path else []
            take = None
            if temp == 0.0 or draft is None:
                if temp == 0.0:
                    y = best(row)
                else:
                    p = softmax(row, temp)
                    y = None
                    if p is not None:
                        y, near = draw(p, u_sample[r0 + c])
                        sure = min(sure, near)
                nxt = -1 if y is None else y
                if y is not None:
                    take = next((i for i in kids if int(tokens[r0 + i]) == y), None)
            else:
                p = softmax(row, temp)
                if p is None:
                    nxt = -1
                    break
                q = np.where(draft[r0 + c] > 0, draft[r0 + c], 0).astype(np.float64)
                r, scale = p, 1.0
                for i in kids:
                    x = int(tokens[r0 + i])
                    if not 0 <= x < vocab:
                        continue
                    u = float(u_accept[r0 + i])
                    if p[x] > 0:  # the rounding of r(x) is relative to p(x) scale and what is taken off it
                        sure = min(sure, abs(u * q[x] - r[x]) / (scale * p[x]) if u * q[x] or r[x] else 1.0)
                    if r[x] > 0 and u * q[x] < r[x]:
                        take = i
                        break
                    rest = np.maximum(r - q, 0)
                    if rest.sum() > 0:
                        scale /= rest.sum()
                        r = rest / rest.sum()
                if take is None:
                    nxt, near = draw(r, u_sample[r0 + c])
                    sure = min(sure, near / scale)
            c = take
        out_path.append(path + [-1] * (max_path - len(path)))
        out_len.append(len(path))
        out_next.append(nxt)
        out_sure.append(sure)
    return (np.array(out_path, dtype=np.int32).reshape(-1, max_path), np.array(out_len, dtype=np.int32),
            np.array(out_next, dtype=np.int32), np.array(out_sure))
