"""Plain implementations of beam selection and reordering, one candidate or row at a time (test infrastructure; torch on the
CPU, no code of the package)."""
import math

import torch


def log_softmax64(z):
    """fp64 log softmax of one row; NaN as -inf, infinite logits share the probability."""
    z = torch.where(torch.isnan(z), -math.inf, z.double())
    m = z.max()
    d = torch.where(z == m, 0.0, z - m)
    return d - torch.log(torch.exp(d).sum())


def select(logits, scores, num, finished=None, end=0):
    """logits [B W, V], scores [B, W]: lists of (total, beam, token) of every prompt, largest first.  A beam's own candidates
    are in the order of their logits, which rounded 64-bit totals may no longer tell apart."""
    b, w = scores.shape
    out = []
    for i in range(b):
        rows, by_logit = [], []
        for r in range(w):
            by_logit.append(r * logits.shape[1] + torch.argsort(torch.nan_to_num(logits[i * w + r].double(), nan=-math.inf,
                                                                                posinf=math.inf, neginf=-math.inf),
                                                                descending=True, stable=True))
            x, s = logits[i * w + r], float(scores[i, r])
            if not math.isfinite(s):
                t = torch.full(x.shape, -math.inf, dtype=torch.float64)
            elif finished is not None and finished[i, r]:
                t = torch.full(x.shape, -math.inf, dtype=torch.float64)
                t[end] = s
            elif torch.where(torch.isnan(x), -math.inf, x).max() == -math.inf:
                t = torch.full(x.shape, -math.inf, dtype=torch.float64)
            else:
                t = s + log_softmax64(x)
            rows.append(t)
        t, by_logit = torch.cat(rows), torch.cat(by_logit)
        order = by_logit[torch.argsort(t[by_logit], descending=True, stable=True)][:num].tolist()
        v = logits.shape[1]
        out.append([(float(t[x]), x // v, x % v) for x in order if t[x] > -math.inf])
    return out


def reorder(table, lens, parents, P):
    """table: rows of page numbers; parents: rows within the prompts (-1: itself).  Returns (new table, copies), a copy being
    (source page, destination page, tokens)."""
    new, copies = [list(r) for r in table], []
    w = len(parents[0])
    for b, par in enumerate(parents):
        par = [r if x == -1 else x for r, x in enumerate(par)]
        n = lens[b * w]
        t, part = n // P, n % P
        free = [r for r in range(w) if r not in par]
        keeper = {p: (p if par[p] == p else par.index(p)) for p in set(par)}
        for r, p in enumerate(par):
            new[b * w + r][:t] = table[b * w + p][:t]
            if not part:
                continue
            if keeper[p] == r:
                new[b * w + r][t] = table[b * w + p][t]
            else:
                dst = table[b * w + free.pop(0)][t]
                new[b * w + r][t] = dst
                copies.append((table[b * w + p][t], dst, part))
        assert not part or not free
    return new, copies
