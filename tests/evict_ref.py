"""Eviction by accumulated weight in plain form, for the tests: the choice as Python integers
and comparisons, the weights and the attention in 64 bits."""
import math

import torch

PAGE = 64


def choose(w, n, budget, sinks, recent, reach):
    """The positions that stay of a row of weights (a list of floats): sorted by score, ties by
    position."""
    if n <= budget:
        return list(range(n))
    v = [-math.inf if math.isnan(x) else x for x in w[:n]]
    score = [max(v[max(0, i - reach):i + reach + 1]) for i in range(n)]
    mid = sorted(range(sinks, n - recent), key=lambda i: (-score[i], i))
    return sorted(list(range(sinks)) + mid[:budget - sinks - recent] + list(range(n - recent, n)))


def attend(q, k, v, seen, scale):
    """q [rows, d], k, v [n, d], row i sees keys 0 .. seen[i] (a list), absent keys dropped by the
    caller -> (out [rows, d], weights [rows, n], magnitude sum p |v|), float64."""
    x = q.double() @ k.double().T * scale
    late = torch.arange(k.shape[0], device=k.device) > torch.tensor(seen, device=k.device)[:, None]
    p = torch.softmax(x.masked_fill(late, -math.inf), -1)
    return p @ v.double(), p, p @ v.double().abs()


def rows(buf, table, n, h):
    """Tokens 0 .. n - 1 of KV head h in bf16 pages [nb, hkv, 64, d]."""
    at = torch.arange(n, device=buf.device)
    return buf[table[at // PAGE].long(), h, at % PAGE]
