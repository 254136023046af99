"""Cases and plain forms of the serving operators: attention over an 8-bit paged cache, storing into it, loading from it,
copying its pages, and sampling a token from logits.

The cache of L layers has pages of P tokens.  K codes are e4m3 [L, N, Hkv, P, D], V codes e4m3 [L, N, Hkv, D, P]
(transposed within the page), and every (layer, page, kv head) has one fp32 scale for K and one for V, a power of two (or 0
for a page of zeros); an element is code x scale.  Sequence b's token j is slot j % P of page table[b, j // P].
"""
import math

import torch

own = False
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


# ---- cases ------------------------------------------------------------------
def listed():
    return [
        # one short sequence, the small two-layer decoder's heads: latency of a single call
        dict(name="attend_one_short", op="attend", batch=1, q_heads=4, kv_heads=2, head_dim=64, page=32, len_lo=300, len_hi=300,
             tokens=1, ragged=False, window=0),
        # the 1B shape's batch of 8 with its ragged lengths, one decode step of one layer
        dict(name="attend_1b_ragged8", op="attend", batch=8, q_heads=32, kv_heads=8, head_dim=64, page=64, len_lo=512, len_hi=4096,
             tokens=1, ragged=False, window=0),
        # the 8B shape's batch of 16 over long contexts: bound by the cache's bytes
        dict(name="attend_8b_long16", op="attend", batch=16, q_heads=32, kv_heads=8, head_dim=128, page=64, len_lo=16000, len_hi=32000,
             tokens=1, ragged=False, window=0),
        # several drafted tokens a sequence to verify, ragged, a sliding window, odd lengths, short sequences among them
        dict(name="attend_verify_window", op="attend", batch=13, q_heads=32, kv_heads=8, head_dim=128, page=32, len_lo=0, len_hi=5001,
             tokens=9, ragged=True, window=1537),
        # a decode step's new token of every sequence, all layers of the 8B shape
        dict(name="store_8b_step16", op="store", layers=36, batch=16, kv_heads=8, head_dim=128, page=64, start_lo=1500, start_hi=2500,
             tokens=1, ragged=False),
        # parking the 1B shape's ragged batch of 8: whole contexts, all layers
        dict(name="store_1b_park8", op="store", layers=16, batch=8, kv_heads=8, head_dim=64, page=64, start_lo=0, start_hi=0,
             tokens=4096, ragged=True),
        # a short prefix of the small decoder back into its cache
        dict(name="load_small", op="load", layers=2, batch=1, kv_heads=2, head_dim=64, page=32, start_lo=0, start_hi=0,
             tokens=100, ragged=False),
        # four parked sequences of the 8B shape back into bf16 caches, all layers
        dict(name="load_8b_restore4", op="load", layers=36, batch=4, kv_heads=8, head_dim=128, page=64, start_lo=0, start_hi=0,
             tokens=2048, ragged=False),
        # forking: the last page of eight children, all layers of the 1B shape
        dict(name="copy_1b_fork8", op="copy", layers=16, kv_heads=8, head_dim=64, page=64, pairs=8, pages=64, table=True),
        # compaction of a large pool of the 8B shape
        dict(name="copy_8b_compact", op="copy", layers=36, kv_heads=8, head_dim=128, page=64, pairs=300, pages=700, table=True),
        # one sequence's next token at the 1B shape's vocabulary, the usual filters
        dict(name="sample_1b_one", op="sample", batch=1, vocab=128256, dtype="float32", spread=3.0, filters="all"),
        # a batch of 16 at the 8B shape's vocabulary, every row with its own settings (greedy and unfiltered rows among them)
        dict(name="sample_8b_mixed16", op="sample", batch=16, vocab=151936, dtype="float32", spread=2.5, filters="mixed"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "store", "store", "load", "copy", "sample", "sample"))
    page, head_dim = rng.choice((32, 64)), rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    if op == "attend":
        group = rng.choice((1, 2, 3, 4, 6, 8, 16))
        tokens = rng.choice((1, 1, 1, _log_int(rng, 2, 64)))
        hi = _log_int(rng, 40, 16000)
        batch = max(1, min(_log_int(rng, 1, 64), 1 + (1 << 26) // (hi * kv_heads * head_dim * max(1, group * tokens // 16))))
        return dict(op=op, batch=batch, q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, page=page,
                    len_lo=rng.choice((0, hi // 8, hi)), len_hi=hi, tokens=tokens, ragged=tokens > 1 and rng.random() < 0.7,
                    window=rng.choice((0, 0, 0, _log_int(rng, 1, hi))))
    if op in ("store", "load"):
        layers, tokens = rng.choice((1, 2, 7, 16, 28)), rng.choice((1, 1, 5, _log_int(rng, 2, 3000)))
        start = rng.choice((0, _log_int(rng, 1, 3000)))
        row = layers * kv_heads * head_dim
        batch = max(1, min(_log_int(rng, 1, 48), (1 << 26) // (row * max(tokens, page)), (1 << 28) // (row * (start + tokens + page))))
        return dict(op=op, layers=layers, batch=batch, kv_heads=kv_heads, head_dim=head_dim, page=page, start_lo=start // 3,
                    start_hi=start, tokens=tokens, ragged=tokens > 1 and rng.random() < 0.5)
    if op == "copy":
        pairs = _log_int(rng, 1, 400)
        return dict(op=op, layers=rng.choice((1, 2, 13, 24)), kv_heads=kv_heads, head_dim=head_dim, page=page, pairs=pairs,
                    pages=2 * pairs + rng.randrange(1, 60), table=rng.random() < 0.5)
    return dict(op=op, batch=_log_int(rng, 1, 64), vocab=_log_int(rng, 1000, 262144), dtype=rng.choice(("float32", "bfloat16")),
                spread=rng.choice((1.0, 2.5, 4.0)), filters=rng.choice(("none", "top_k", "top_p", "all", "mixed")))


# ---- inputs -----------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(lo, hi, n, g):
    """n int32 in [lo, hi]."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int32)


def _pool(layers, pages, c, g, filled=True):
    """A cache whose pages hold N(0, 1) values with their scales (codes up to 448 in size), K's first channels larger, as
    keys have them; filled=False: pages that nothing has been stored in yet (zeros)."""
    hkv, p, d = c["kv_heads"], c["page"], c["head_dim"]
    out = {}
    for name, dims in (("k", (p, d)), ("v", (d, p))):
        codes = torch.zeros((layers, pages, hkv) + dims, dtype=torch.uint8, device=DEV)
        scales = torch.zeros((layers, pages, hkv), dtype=torch.float32, device=DEV)
        if filled:
            scales.copy_(torch.tensor([2.0 ** -7, 2.0 ** -6, 2.0 ** -5], device=DEV)[_ints(0, 2, scales.numel(), g).view(scales.shape)])
            for l in range(layers):
                x = torch.randn((pages, hkv) + dims, generator=g, device=DEV)
                if name == "k":
                    x[..., :4] *= 4.0
                codes[l] = (x / scales[l][..., None, None]).clamp_(-448.0, 448.0).to(F8).view(torch.uint8)
        out[name], out[name + "_scale"] = codes.view(F8), scales
    return out


def _table(batch, width, used, pages, g):
    """int32 [batch, width]: distinct pages in random order, -1 behind each sequence's `used` pages."""
    t = torch.randperm(pages, generator=g, device=DEV)[: batch * width].to(torch.int32).view(batch, width)
    return torch.where(torch.arange(width, device=DEV) < used[:, None], t, -1).to(torch.int32).contiguous()


def prepare(case, seed):
    g, c = _gen(seed), case
    s = {"case": c}
    if c["op"] == "sample":
        b, v = c["batch"], c["vocab"]
        s["logits"] = (torch.randn((b, v), generator=g, device=DEV) * c["spread"]).to(getattr(torch, c["dtype"]))
        s["u"] = torch.rand((b,), generator=g, device=DEV)
        row, f = torch.arange(b, device=DEV), c["filters"]
        on = lambda k: (row % 5 != k) if f == "mixed" else torch.ones_like(row, dtype=torch.bool)  # noqa: E731
        r = torch.rand((4, b), generator=g, device=DEV)
        if f in ("top_k", "all", "mixed"):
            s["top_k"] = torch.where(on(1), (10 + 90 * r[0]).to(torch.int32), 0).to(torch.int32)
        if f in ("top_p", "all", "mixed"):
            s["top_p"] = torch.where(on(2), 0.7 + 0.29 * r[1], 1.0)
        if f in ("all", "mixed"):
            s["min_p"] = torch.where(on(3), 0.05 * r[2], 0.0)
        if f != "none":
            s["temperature"] = torch.where(on(4), 0.5 + r[3], 0.0 if f == "mixed" else 1.0)
        return s
    p = c["page"]
    if c["op"] == "attend":
        b, t = c["batch"], c["tokens"]
        lens = _ints(c["len_lo"], c["len_hi"], b, g)
        # ragged: 0 .. t new tokens, the same numbers for every seed in another order
        count = torch.linspace(0, t, b, device=DEV)[torch.randperm(b, generator=g, device=DEV)] if c["ragged"] else torch.full((b,), t, device=DEV)
        count = count.to(torch.int32)
        lens = torch.maximum(lens, count)
        width = -(-max(c["len_hi"], t) // p)
        s["q_start"] = torch.zeros(b + 1, dtype=torch.int32, device=DEV)
        s["q_start"][1:] = count.cumsum(0)
        total = int(s["q_start"][-1]) if c["ragged"] else b * t
        shape = (total,) if c["ragged"] else (b, t)
        s["q"] = torch.randn(shape + (c["q_heads"], c["head_dim"]), generator=g, device=DEV).to(torch.bfloat16)
        s["lens"] = lens
        s["table"] = _table(b, width, (lens + p - 1) // p, b * width, g)
        s["pool"] = _pool(1, b * width, c, g)
    elif c["op"] == "copy":
        n = c["pages"]
        perm = torch.randperm(n, generator=g, device=DEV)
        s["src"], s["dst"] = perm[: c["pairs"]].tolist(), perm[c["pairs"]: 2 * c["pairs"]].tolist()
        s["table"] = _table(1, n, torch.tensor([n - 1], device=DEV), n, g) if c["table"] else None
        if c["table"]:  # only pages in use are named by a table, not those that are free to be copied to
            free = torch.zeros(n + 1, dtype=torch.bool, device=DEV)
            free[s["dst"]] = True
            s["table"].masked_fill_(free[s["table"].long()], -1)
            s["renamed"] = s["table"].clone()
        s["pool"] = _pool(c["layers"], n, c, g)
    else:
        b, t = c["batch"], c["tokens"]
        s["start"] = _ints(c["start_lo"], c["start_hi"], b, g)
        s["count"] = _ints(min(t, max(1, t // 8)), t, b, g) if c["ragged"] else torch.full((b,), t, dtype=torch.int32, device=DEV)
        width = -(-(c["start_hi"] + t) // p)
        s["table"] = _table(b, width, (s["start"] + s["count"] + p - 1) // p, b * width, g)
        s["pool"] = _pool(c["layers"], b * width, c, g, filled=c["op"] == "load" or c["start_hi"] > 0)
        # the decoder's own cache layout [L, B, Hkv, T, D], seen as [L, B, T, Hkv, D]
        for name in ("k_rows", "v_rows"):
            x = torch.empty((c["layers"], b, c["kv_heads"], t, c["head_dim"]), dtype=torch.bfloat16, device=DEV)
            if c["op"] == "store":
                for l in range(c["layers"]):
                    x[l] = torch.randn(x.shape[1:], generator=g, device=DEV)
            else:
                x.zero_()
            s[name] = x.permute(0, 1, 3, 2, 4)
    if own:
        from persistent_megakernel_decode_gb300 import kvcache
        s["cache"] = kvcache.Kv8Cache(s["pool"]["k"], s["pool"]["v"], s["pool"]["k_scale"], s["pool"]["v_scale"])
    return s


# ---- one pass ---------------------------------------------------------------
def run(s):
    return RUN[s["case"]["op"]](s)


def run_attend(s):
    c = s["case"]
    if own:
        return s["cache"].attend(s["q"], s["table"], s["lens"], q_start=s["q_start"] if c["ragged"] else None,
                                 max_tokens=c["tokens"], window=c["window"])
    return plain_attend(s["q"], s["pool"], s["table"], s["lens"], s["q_start"], c)


def run_store(s):
    if own:
        s["cache"].store(s["k_rows"], s["v_rows"], s["table"], s["start"], s["count"])
    else:
        for name in ("k", "v"):
            plain_store(s[name + "_rows"], s["pool"][name], s["pool"][name + "_scale"], s["table"], s["start"], s["count"], name == "v")
    return s["pool"]


def run_load(s):
    if own:
        s["cache"].load(s["k_rows"], s["v_rows"], s["table"], s["start"], s["count"])
    else:
        for name in ("k", "v"):
            plain_load(s[name + "_rows"], s["pool"][name], s["pool"][name + "_scale"], s["table"], s["start"], s["count"], name == "v")
    return s["k_rows"], s["v_rows"]


def run_copy(s):
    if s["table"] is not None:
        s["renamed"].copy_(s["table"])
    if own:
        s["cache"].copy_pages(s["src"], s["dst"], table=s["renamed"] if s["table"] is not None else None)
    else:
        src, dst = torch.tensor(s["src"], device=DEV), torch.tensor(s["dst"], device=DEV)
        for x in s["pool"].values():
            x = x.view(torch.uint8) if x.dtype == F8 else x
            x[:, dst] = x[:, src]
        if s["table"] is not None:
            name = torch.arange(s["case"]["pages"] + 1, device=DEV, dtype=torch.int32)
            name[-1] = -1  # an entry of -1 stays
            name[src] = dst.to(torch.int32)
            s["renamed"].copy_(name[s["renamed"].long()])
    return s["pool"] if s["table"] is None else dict(s["pool"], table=s["renamed"])


def run_sample(s):
    a = {k: s.get(k) for k in ("temperature", "top_k", "top_p", "min_p")}
    if own:
        from persistent_megakernel_decode_gb300 import runtime
        return runtime.sample(s["logits"], s["u"], **a)
    return plain_sample(s["logits"], s["u"], **a)


RUN = {"attend": run_attend, "store": run_store, "load": run_load, "copy": run_copy, "sample": run_sample}


# ---- plain forms ------------------------------------------------------------
def _rows_of(pool, scale, table, transposed):
    """Every slot of the table's pages as fp32 tokens [B, S, Hkv, D] of layer 0 (pages of -1: page 0, masked by the caller)."""
    t = table.clamp(min=0).long()
    x = pool[0].view(torch.uint8)[t].view(F8).float() * scale[0][t][..., None, None]
    x = x.transpose(-1, -2) if transposed else x
    b, w, h, p, d = x.shape
    return x.transpose(2, 3).reshape(b, w * p, h, d)


def plain_attend(q, pool, table, lens, q_start, c):
    hq, hkv, d, t = c["q_heads"], c["kv_heads"], c["head_dim"], c["tokens"]
    b = lens.numel()
    count = (q_start[1:] - q_start[:-1]).long()
    i = torch.arange(t, device=DEV)
    there = i < count[:, None]
    at = torch.where(there, q_start[:-1].long()[:, None] + i, 0)
    flat = q.reshape(-1, hq, d)
    if not flat.shape[0]:
        return q.clone(), torch.empty(q.shape[:-1], dtype=torch.float32, device=DEV)
    x = flat.float()[at].view(b, t, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    k = _rows_of(pool["k"], pool["k_scale"], table, False).permute(0, 2, 3, 1)
    v = _rows_of(pool["v"], pool["v_scale"], table, True).permute(0, 2, 1, 3)
    z = torch.matmul(x, k) * (d ** -0.5)
    z = z.view(b, hkv, hq // hkv, t, -1)
    pos = (lens.long() - count)[:, None] + i
    j = torch.arange(z.shape[-1], device=DEV)
    seen = (j <= pos[..., None]) & there[..., None]
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    z = z.masked_fill_(~seen[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(z - m)
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(b, hkv, -1, e.shape[-1]), v).view(b, hkv, hq // hkv, t, d) / l.clamp(min=1e-30)
    lse = (m + torch.log(l)).squeeze(-1)
    out = torch.empty_like(flat)
    out[at[there]] = o.permute(0, 3, 1, 2, 4).reshape(b, t, hq, d)[there].to(q.dtype)
    far = torch.empty(flat.shape[:-1], dtype=torch.float32, device=DEV)
    far[at[there]] = lse.permute(0, 3, 1, 2).reshape(b, t, hq)[there]
    return out.view(q.shape), far.view(q.shape[:-1])


def plain_store(rows, pool, scale, table, start, count, transposed):
    lay, b, t, h, d = rows.shape
    p = pool.shape[-1] if transposed else pool.shape[-2]
    n = (t + 2 * p - 2) // p  # pages that t tokens touch at most
    first = start.long() // p
    page = first[:, None] + torch.arange(n, device=DEV)
    pos = (page[..., None] * p + torch.arange(p, device=DEV)).view(b, n * p)
    src = pos - start.long()[:, None]
    new = ((src >= 0) & (src < count.long()[:, None])).view(b, n, p)
    x = torch.gather(rows.float(), 2, src.clamp(0, t - 1)[None, :, :, None, None].expand(lay, b, n * p, h, d))
    x = torch.where(new.view(1, b, n * p, 1, 1), x, 0.0).view(lay, b, n, p, h, d).transpose(3, 4)
    touched = new.any(-1)
    seq, slot = touched.nonzero(as_tuple=True)
    x, new = x[:, seq, slot], new[seq, slot][None, :, None, :, None]
    ids = table[seq, page[seq, slot]].long()
    held = (page[seq, slot] * p < start.long()[seq])[None, :, None]  # the page holds earlier tokens
    m, e = torch.frexp(x.abs().amax((-1, -2)))  # amax = m 2^e, 1/2 <= m < 1; 448 = 0.875 2^9
    power = ((e - 9) + (m > 0.875)).clamp(-120, 120).to(torch.int32)
    need = torch.where(m > 0, ((power + 127) << 23).view(torch.float32), 0.0)  # 2^power, from its bits
    before = torch.where(held, scale[:, ids], 0.0)
    now = torch.maximum(need, before)
    old = pool[:, ids].view(torch.uint8) if pool.dtype != F8 else pool.view(torch.uint8)[:, ids]
    old = old.view(F8).float()
    old = old.transpose(-1, -2) if transposed else old
    some = now.clamp(min=2.0 ** -126)[..., None, None]
    old = torch.where(held[..., None, None], old * (before[..., None, None] / some), 0.0)
    y = torch.where(new, x / some, old).clamp(-448.0, 448.0).to(F8).view(torch.uint8)
    pool.view(torch.uint8)[:, ids] = y.transpose(-1, -2) if transposed else y
    scale[:, ids] = now


def plain_load(rows, pool, scale, table, start, count, transposed):
    lay, b, t, h, d = rows.shape
    p = pool.shape[-1] if transposed else pool.shape[-2]
    i = torch.arange(t, device=DEV)
    seq, i = (i < count[:, None]).nonzero(as_tuple=True)
    pos = start.long()[seq] + i
    ids, slot = table[seq, pos // p].long(), pos % p
    codes = pool.view(torch.uint8)
    x = codes[:, ids, :, :, slot] if transposed else codes[:, ids, :, slot]  # [n, L, h, d]: the indexed axes come first
    x = x.view(F8).float() * scale[:, ids].transpose(0, 1)[..., None]
    rows[:, seq, i] = x.transpose(0, 1).to(rows.dtype)


def plain_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    b, v = logits.shape
    full = lambda x, off: torch.full((b,), off, device=DEV, dtype=torch.float64) if x is None else x.double()  # noqa: E731
    temp, tk, tp, mp = full(temperature, 1.0), full(top_k, 0.0), full(top_p, 1.0), full(min_p, 0.0)
    z, at = torch.sort(logits, dim=1, descending=True, stable=True)
    z = z.double()
    w = torch.exp((z - z[:, :1]) / torch.where(temp > 0, temp, 1.0)[:, None])
    rank = torch.arange(v, device=DEV)
    w = torch.where((rank < tk[:, None]) | (tk[:, None] <= 0), w, 0.0)
    w = torch.where((temp[:, None] > 0) | (rank == 0), w, 0.0)
    mass = w.cumsum(1)
    keep = (mass - w < tp[:, None] * mass[:, -1:]) | (rank == 0) | (tp[:, None] >= 1)
    w = torch.where(keep & (w >= mp[:, None]), w, 0.0)
    w = torch.zeros_like(w).scatter_(1, at, w)  # back in the vocabulary's order
    mass = w.cumsum(1)
    total = mass[:, -1:]
    token = torch.searchsorted(mass, u.double()[:, None] * total, right=True).clamp(max=v - 1)
    chosen = w.gather(1, token)
    logprob = -torch.log1p((w.sum(1, keepdim=True) - chosen).clamp(min=0) / chosen)
    return token.squeeze(1).to(torch.int32), logprob.squeeze(1).float()


# ---- what a pass cannot do without ------------------------------------------
def work(case):
    c = case
    if c["op"] == "sample":
        n = c["batch"] * c["vocab"]
        return {"bytes": n * (4 if c["dtype"] == "float32" else 2), "flops": 4 * n}
    if c["op"] == "copy":
        page = c["layers"] * c["kv_heads"] * (c["page"] * c["head_dim"] + 4) * 2
        return {"bytes": 2 * page * c["pairs"] + (8 * c["pages"] if c["table"] else 0), "flops": 0}
    mean = (min(c["tokens"], max(1, c["tokens"] // 8)) + c["tokens"]) / 2 if c["ragged"] else c["tokens"]
    if c["op"] == "attend":
        t = c["tokens"] / 2 if c["ragged"] else c["tokens"]
        n = max((c["len_lo"] + c["len_hi"]) / 2, t)
        n = min(n, c["window"] + t) if c["window"] else n
        rows = c["batch"] * t * c["q_heads"]
        return {"bytes": int(c["batch"] * n * c["kv_heads"] * (2 * c["head_dim"] + 8 / c["page"]) + rows * (4 * c["head_dim"] + 4)),
                "flops": int(4 * rows * max(1.0, n - t / 2) * c["head_dim"])}
    n = c["layers"] * c["batch"] * mean * c["kv_heads"] * c["head_dim"] * 2
    return {"bytes": int(3 * n), "flops": int(2 * n)}


# ---- from the definitions, in 64 bits ---------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return EXACT[case["op"]](s)


def _power(e):
    """2^e as fp64, from a table: torch's ldexp and exp2 may be off by a last place on the GPU."""
    return torch.tensor([2.0 ** i for i in range(-200, 201)], dtype=torch.float64, device=e.device)[(e + 200).long()]


def _value(code):
    """The values of e4m3 codes: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    c = code.view(torch.uint8).to(torch.int32)
    e, f = (c >> 3) & 15, (c & 7).double()
    x = torch.where(e > 0, (1 + f / 8) * _power(e - 7), f * 2.0 ** -9)
    return torch.where(c >= 128, -x, x)


def _token_rows(s, b, name, lo, hi):
    """Tokens lo .. hi - 1 of sequence b in layer 0, fp64 [n, Hkv, D]."""
    p = s["case"]["page"]
    pages = s["table"][b, lo // p: -(-hi // p)].long()
    x = _value(s["pool"][name][0].view(torch.uint8)[pages]) * s["pool"][name + "_scale"][0][pages].double()[..., None, None]
    x = x.permute(0, 3, 1, 2) if name == "v" else x.permute(0, 2, 1, 3)
    return x.reshape(-1, x.shape[2], x.shape[3])[lo % p: lo % p + hi - lo]


def exact_attend(s):
    c = s["case"]
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    flat = s["q"].reshape(-1, hq, d).double()
    out, lse = torch.zeros_like(flat), torch.full(flat.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    edge, lens = s["q_start"].tolist(), s["lens"].tolist()
    for b, n in enumerate(lens):
        t = edge[b + 1] - edge[b]
        if not t or not n:
            continue
        k, v = (_token_rows(s, b, x, 0, n).repeat_interleave(hq // hkv, 1) for x in ("k", "v"))
        for i in range(t):
            hi = n - t + i + 1
            lo = max(0, hi - c["window"]) if c["window"] else 0
            z = (k[lo:hi] * flat[edge[b] + i]).sum(-1) / math.sqrt(d)
            lse[edge[b] + i] = torch.logsumexp(z, 0)
            out[edge[b] + i] = (torch.exp(z - lse[edge[b] + i])[..., None] * v[lo:hi]).sum(0)
    return out.view(s["q"].shape), lse.view(s["q"].shape[:-1])


def _round_e4m3(x):
    """fp64 to the nearest e4m3 value, ties to even, at most 448."""
    e = torch.frexp(x.abs().clamp(min=2.0 ** -60))[1].clamp(min=-5)
    step = _power(e - 4)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact_store(s):
    c, answer = s["case"], {}
    p = c["page"]
    start, count, table = s["start"].tolist(), s["count"].tolist(), s["table"].tolist()
    if sum(count) // p * c["layers"] > 30000:
        return None
    for name in ("k", "v"):
        codes = torch.stack([_value(x) for x in s["pool"][name]])
        scales = s["pool"][name + "_scale"].double()
        for b, (first, n) in enumerate(zip(start, count)):
            for j in range(first // p, -(-(first + n) // p)):
                lo, hi = max(first, j * p), min(first + n, j * p + p)
                x = s[name + "_rows"][:, b, lo - first: hi - first].double().transpose(1, 2)  # [L, Hkv, n, D]
                most = x.abs().amax((2, 3))
                need = torch.where(most > 0, _power(torch.ceil(torch.log2(most / 448)).clamp(-120, 120)), 0.0)
                new, old = codes[:, table[b][j]], scales[:, table[b][j]]
                new = new.transpose(-1, -2) if name == "v" else new
                if first <= j * p:
                    old, new = torch.zeros_like(old), torch.zeros_like(new)
                now = torch.maximum(need, old)
                safe = torch.where(now > 0, now, 1.0)[..., None, None]
                new = _round_e4m3(new * (old[..., None, None] / safe))
                new[:, :, lo - j * p: hi - j * p] = _round_e4m3(x / safe)
                codes[:, table[b][j]] = new.transpose(-1, -2) if name == "v" else new
                scales[:, table[b][j]] = now
        answer[name], answer[name + "_scale"] = codes, scales
    return answer


def exact_load(s):
    c = s["case"]
    p = c["page"]
    answer = []
    for name in ("k", "v"):
        rows = s[name + "_rows"].double()
        for l in range(c["layers"]):
            for b, (first, n) in enumerate(zip(s["start"].tolist(), s["count"].tolist())):
                pages = s["table"][b, first // p: -(-(first + n) // p)].long()
                x = _value(s["pool"][name][l].view(torch.uint8)[pages]) * s["pool"][name + "_scale"][l][pages].double()[..., None, None]
                x = x.permute(0, 3, 1, 2) if name == "v" else x.permute(0, 2, 1, 3)
                rows[l, b, :n] = x.reshape(-1, x.shape[2], x.shape[3])[first % p: first % p + n]
        answer.append(rows)
    return tuple(answer)


def exact_copy(s):
    if s["case"]["layers"] * s["case"]["pages"] > 20000:
        return None
    answer = {}
    for name, x in s["pool"].items():
        x = torch.stack([_value(y) for y in x]) if x.dtype == F8 else x.double()
        for i, j in zip(s["src"], s["dst"]):
            x[:, j] = x[:, i]
        answer[name] = x
    if s["table"] is not None:
        to = dict(zip(s["src"], s["dst"]))
        answer["table"] = torch.tensor([[to.get(e, e) for e in r] for r in s["table"].tolist()], dtype=torch.int32)
    return answer


def exact_sample(s):
    tokens, logs = [], []
    for b in range(s["case"]["batch"]):
        x = s["logits"][b].double().cpu()
        get = lambda k, off: float(s[k][b]) if k in s else off  # noqa: E731
        temp, k, p, least, u = get("temperature", 1.0), int(get("top_k", 0)), get("top_p", 1.0), get("min_p", 0.0), float(s["u"][b])
        order = torch.argsort(x, descending=True, stable=True)
        if temp <= 0:
            order, temp = order[:1], 1.0
        order = order[:k] if k > 0 else order
        w = torch.exp((x[order] - x[order[0]]) / temp)
        if p < 1:
            before = torch.cat([torch.zeros(1, dtype=torch.float64), w.cumsum(0)[:-1]])
            n = max(1, int((before < p * w.sum()).sum()))
            order, w = order[:n], w[:n]
        order, w = order[w >= least], w[w >= least]
        order, by = torch.sort(order)
        w = w[by]
        sums = w.cumsum(0)
        i = min(int((sums <= u * sums[-1]).sum()), len(order) - 1)
        tokens.append(int(order[i]))
        logs.append(float(-torch.log1p((w.sum() - w[i]).clamp(min=0) / w[i])))
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(logs, dtype=torch.float64)


EXACT = {"attend": exact_attend, "store": exact_store, "load": exact_load, "copy": exact_copy, "sample": exact_sample}
