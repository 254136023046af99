"""Plain implementations of the serving operators in 64 bits, one token or row at a time (test infrastructure; torch on
the CPU, no code of the package)."""
import math

import torch

F8 = torch.float8_e4m3fn


def e4m3_values(codes):
    """fp64 values of e4m3 codes from their bits."""
    c = codes.view(torch.uint8).to(torch.int64)
    e, f = (c >> 3) & 15, (c & 7).double()
    x = torch.where(e > 0, (1 + f / 8) * 2.0 ** (e - 7).double(), f * 2.0 ** -9)
    x = torch.where((c & 127) == 127, math.nan, x)
    return torch.where(c >= 128, -x, x)


def round_e4m3(x):
    """fp64 -> nearest e4m3 value, ties to even, +-448 beyond (infinities too); NaN stays."""
    a = x.abs().clamp(2.0 ** -70, 1e300)
    e = torch.floor(torch.log2(a))
    e = torch.where(2.0 ** e > a, e - 1, torch.where(2.0 ** (e + 1) <= a, e + 1, e)).clamp(min=-6)
    step = 2.0 ** (e - 3)
    y = (torch.round(x / step) * step).clamp(-448, 448)
    return torch.where(torch.isnan(x), x, torch.where(torch.isinf(x), torch.sign(x) * 448, y))


class RefCache:
    """Values and scales as fp64 [L, N, Hkv, P, D] and [L, N, Hkv]."""

    def __init__(self, L, N, H, P, D):
        self.P = P
        self.code = {n: torch.zeros((L, N, H, P, D), dtype=torch.float64) for n in "kv"}
        self.scale = {n: torch.zeros((L, N, H), dtype=torch.float64) for n in "kv"}

    def token(self, name, layer, table, j):
        """Token j of the sequence with page list ``table``, fp64 [Hkv, D]."""
        page = table[j // self.P]
        return self.code[name][layer, page, :, j % self.P] * self.scale[name][layer, page][:, None]

    def store(self, name, rows, table, start):
        """rows [L, n, Hkv, D] at positions start ..., page by page."""
        P, n = self.P, rows.shape[1]
        x = rows.double()
        j = start // P
        while j * P < start + n:
            lo, hi = max(start, j * P), min(start + n, j * P + P)
            new = x[:, lo - start: hi - start].transpose(1, 2)  # [L, Hkv, m, D]
            most = torch.where(torch.isfinite(new), new.abs(), 0.0).amax((2, 3))
            need = torch.zeros_like(most)
            pos = most > 0
            need[pos] = 2.0 ** torch.ceil(torch.log2(most[pos] / 448)).clamp(-120, 120)
            page = table[j]
            old = self.scale[name][:, page].clone() if j * P < start else torch.zeros_like(need)
            now = torch.maximum(need, old)
            safe = torch.where(now > 0, now, 1.0)[..., None, None]
            c = self.code[name][:, page].clone() if j * P < start else torch.zeros_like(self.code[name][:, page])
            c = torch.where((old == now)[..., None, None], c, round_e4m3(c * (old[..., None, None] / safe)))
            c[:, :, lo - j * P: hi - j * P] = round_e4m3(new / safe)
            self.code[name][:, page], self.scale[name][:, page] = c, now
            j += 1

    def attend(self, q, layer, table, n, window=0, scale=None):
        """q [T, Hq, D]: out fp64 [T, Hq, D], lse [T, Hq]."""
        t, hq, d = q.shape
        hkv = self.code["k"].shape[2]
        out, lse = torch.zeros((t, hq, d), dtype=torch.float64), torch.full((t, hq), -math.inf, dtype=torch.float64)
        if n == 0:
            return out, lse
        k, v = (torch.stack([self.token(x, layer, table, j) for j in range(n)]) for x in "kv")
        for i in range(t):
            hi = n - t + i + 1
            lo = max(0, hi - window) if window else 0
            if hi <= lo:
                continue
            for h in range(hq):
                g = h // (hq // hkv)
                z = k[lo:hi, g] @ q[i, h].double() * (scale if scale is not None else d ** -0.5)
                lse[i, h] = torch.logsumexp(z, 0)
                out[i, h] = torch.exp(z - lse[i, h]) @ v[lo:hi, g]
        return out, lse


def sample_row(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob) of one row, from the definition."""
    x = z.double().clone()
    x[torch.isnan(x)] = -math.inf
    if x.max() == -math.inf:
        return 0, -math.inf
    order = torch.argsort(x, descending=True, stable=True)
    if not temperature > 0:
        return int(order[0]), 0.0
    if top_k > 0:
        order = order[:top_k]
    top = x[order[0]]
    w = torch.where(x[order] == top, torch.ones_like(x[order]), torch.exp((x[order] - top) / temperature))
    if top_p < 1:
        before = torch.cat([torch.zeros(1, dtype=torch.float64), w.cumsum(0)[:-1]])
        n = max(1, int((before < max(top_p, 0.0) * w.sum()).sum()))
        order, w = order[:n], w[:n]
    if min_p > 0:
        # w >= min_p, asked of the logits: exp of a difference below 2^-53 rounds to 1 although it is less
        keep = x[order] >= top + temperature * math.log(min(min_p, 1.0))
        order, w = order[keep], w[keep]
    order, at = torch.sort(order)
    w = w[at]
    sums = w.cumsum(0)
    i = min(int((sums <= u * sums[-1]).sum()), len(order) - 1)
    while w[i] == 0:
        i -= 1
    return int(order[i]), float(-torch.log1p((w.sum() - w[i]) / w[i]))
