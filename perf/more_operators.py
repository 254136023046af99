"""Cases and plain forms of the operators for decoding several continuations of one context: attention over the 8-bit paged
cache through a sliding window whose first tokens stay visible, attention of sequences that share a prefix's pages,
beam search's selection over beams and vocabulary, and the reordering of the beams' cached states.

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
        # one stream of the small two-layer decoder's heads, the window just past: latency of a single call
        dict(name="sinks_one_short", op="sinks", batch=1, q_heads=4, kv_heads=2, head_dim=64, page=32, len_lo=700, len_hi=700,
             tokens=1, ragged=False, window=256, sinks=4),
        # eight long streams of the 1B shape, one decode step of one layer
        dict(name="sinks_1b_stream8", op="sinks", batch=8, q_heads=32, kv_heads=8, head_dim=64, page=64, len_lo=3000, len_hi=16000,
             tokens=1, ragged=False, window=2048, sinks=4),
        # drafted tokens to verify, ragged, odd lengths and window, sinks that end inside a page, sequences shorter than both
        dict(name="sinks_verify_ragged", op="sinks", batch=13, q_heads=32, kv_heads=8, head_dim=128, page=32, len_lo=0, len_hi=6001,
             tokens=9, ragged=True, window=1537, sinks=100),
        # four beams of a short prompt, the small decoder's heads: latency
        dict(name="shared_one_beams4", op="shared", groups=1, members=4, even=True, q_heads=4, kv_heads=2, head_dim=64, page=32,
             prefix_lo=300, prefix_hi=300, own_lo=1, own_hi=40, tokens=1, ragged=False),
        # four prompts of the 8B shape with eight beams each
        dict(name="shared_8b_beams32", op="shared", groups=4, members=32, even=True, q_heads=32, kv_heads=8, head_dim=128, page=64,
             prefix_lo=4000, prefix_hi=9000, own_lo=1, own_hi=300, tokens=1, ragged=False),
        # 64 conversations of the 8B shape behind one long instruction
        dict(name="shared_8b_system64", op="shared", groups=1, members=64, even=True, q_heads=32, kv_heads=8, head_dim=128, page=64,
             prefix_lo=16000, prefix_hi=16000, own_lo=100, own_hi=2000, tokens=1, ragged=False),
        # groups of uneven sizes of the 1B shape, several drafted tokens a sequence, ragged
        dict(name="shared_1b_verify", op="shared", groups=3, members=21, even=False, q_heads=32, kv_heads=8, head_dim=64, page=64,
             prefix_lo=500, prefix_hi=7000, own_lo=8, own_hi=700, tokens=5, ragged=True),
        # four beams at the 1B shape's vocabulary: latency of one step
        dict(name="beam_1b_one4", op="beam", batch=1, beams=4, num=4, vocab=128256, dtype="float32", spread=2.5, finished=0.0, first=False),
        # sixteen prompts with eight beams at the 8B shape's vocabulary, twice as many candidates as beams
        dict(name="beam_8b_16x8", op="beam", batch=16, beams=8, num=16, vocab=151936, dtype="float32", spread=2.5, finished=0.1, first=False),
        # five beams in bf16 (many equal logits) at an odd vocabulary, beams that have ended
        dict(name="beam_odd_bf16", op="beam", batch=7, beams=5, num=10, vocab=32003, dtype="bfloat16", spread=4.0, finished=0.3, first=False),
        # two prompts' four beams of the small decoder
        dict(name="reorder_small", op="reorder", layers=2, batch=2, beams=4, kv_heads=2, head_dim=64, page=32, prefix=100, own_hi=60),
        # eight prompts' eight beams, all layers of the 8B shape
        dict(name="reorder_8b_8x8", op="reorder", layers=36, batch=8, beams=8, kv_heads=8, head_dim=128, page=64, prefix=500, own_hi=120),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("sinks", "sinks", "shared", "shared", "shared", "beam", "beam", "reorder"))
    page, head_dim = rng.choice((32, 64)), rng.choice((64, 128))
    kv_heads, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 6, 8))
    tokens = rng.choice((1, 1, 1, _log_int(rng, 2, 12)))
    heads = dict(q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, page=page)
    if op == "sinks":
        hi = _log_int(rng, 40, 16000)
        batch = max(1, min(_log_int(rng, 1, 48), 1 + (1 << 25) // (hi * kv_heads * head_dim * max(1, group * tokens // 16))))
        return dict(op=op, batch=batch, **heads, len_lo=rng.choice((0, hi // 8, hi)), len_hi=hi, tokens=tokens,
                    ragged=tokens > 1 and rng.random() < 0.7, window=_log_int(rng, 1, hi), sinks=_log_int(rng, 1, 300))
    if op == "shared":
        hi = _log_int(rng, 40, 16000)
        own_hi = _log_int(rng, 16, 2000)
        groups = min(rng.choice((1, 1, _log_int(rng, 2, 8))), 1 + 20000000 // (hi * kv_heads * head_dim))
        most = min(64, 1 + (1 << 33) // (4 * (hi + own_hi) * heads["q_heads"] * head_dim * tokens), 1 + 45000000 // (own_hi * kv_heads * head_dim))
        members = max(groups, min(groups * _log_int(rng, 1, 64), most))
        return dict(op=op, groups=groups, members=members, even=rng.random() < 0.5 and members % groups == 0, **heads,
                    prefix_lo=rng.choice((0, hi // 3, hi)), prefix_hi=hi, own_lo=min(own_hi, max(tokens, rng.choice((1, own_hi // 4)))),
                    own_hi=max(own_hi, tokens), tokens=tokens, ragged=tokens > 1 and rng.random() < 0.5)
    if op == "beam":
        vocab, beams = _log_int(rng, 1000, 262144), _log_int(rng, 2, 16)
        batch = max(1, min(_log_int(rng, 1, 32), 17000000 // (vocab * beams)))
        return dict(op=op, batch=batch, beams=beams, num=beams * rng.choice((1, 2)), vocab=vocab, dtype=rng.choice(("float32", "bfloat16")),
                    spread=rng.choice((1.5, 2.5, 4.0)), finished=rng.choice((0.0, 0.2)), first=rng.random() < 0.15)
    beams, layers = _log_int(rng, 2, 16), rng.choice((1, 2, 7, 16, 28))
    batch = max(1, min(_log_int(rng, 1, 16), (1 << 26) // (layers * kv_heads * head_dim * 64 * beams)))
    return dict(op=op, layers=layers, batch=batch, beams=beams, kv_heads=kv_heads, head_dim=head_dim, page=page,
                prefix=_log_int(rng, 1, 500), own_hi=_log_int(rng, 2, 120))


# ---- inputs -----------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(lo, hi, n, g):
    """n int32 in [lo, hi]."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int32)


def _pool(layers, pages, c, g):
    """A cache whose pages hold N(0, 1) values with their scales (codes up to 448 in size), K's first channels larger, as
    keys have them."""
    hkv, p, d = c["kv_heads"], c["page"], c["head_dim"]
    out = {}
    for name, dims in (("k", (p, d)), ("v", (d, p))):
        codes = torch.zeros((layers, pages, hkv) + dims, dtype=torch.uint8, device=DEV)
        scales = torch.tensor([2.0 ** -7, 2.0 ** -6, 2.0 ** -5], device=DEV)[_ints(0, 2, layers * pages * hkv, g).long()]
        scales = scales.view(layers, pages, hkv).contiguous()
        for l in range(layers):
            x = torch.randn((pages, hkv) + dims, generator=g, device=DEV)
            if name == "k":
                x[..., :4] *= 4.0
            codes[l] = (x / scales[l][..., None, None]).clamp_(-448.0, 448.0).to(F8).view(torch.uint8)
        out[name], out[name + "_scale"] = codes.view(F8), scales
    return out


def _queries(s, b, g):
    """New tokens of b sequences: q, q_start, and how many each has (0 .. t of a ragged batch, the same numbers for every
    seed in another order)."""
    c, t = s["case"], s["case"]["tokens"]
    if c["ragged"]:
        count = torch.linspace(0, t, b, device=DEV)[torch.randperm(b, generator=g, device=DEV)].to(torch.int32)
    else:
        count = torch.full((b,), t, device=DEV, dtype=torch.int32)
    s["q_start"] = torch.zeros(b + 1, dtype=torch.int32, device=DEV)
    s["q_start"][1:] = count.cumsum(0)
    shape = (int(s["q_start"][-1]),) if c["ragged"] else (b, t)
    s["q"] = torch.randn(shape + (c["q_heads"], c["head_dim"]), generator=g, device=DEV).to(torch.bfloat16)
    return count


def _shared_table(prefix, own, first, page, g):
    """int32 table of sequences first[i] .. first[i + 1] - 1 whose full pages of prefix[i] tokens are one and the same, with
    pages of their own for the rest up to `own` tokens more; -1 behind.  All page numbers in random order."""
    full = [n // page for n in prefix]
    need = [[-(-(prefix[i] + own[b]) // page) - full[i] for b in range(first[i], first[i + 1])] for i in range(len(prefix))]
    pages = sum(full) + sum(map(sum, need))
    ids = torch.randperm(max(pages, 1), generator=g, device=DEV).tolist()
    rows, at = [], 0
    for i, n in enumerate(full):
        head, at = ids[at: at + n], at + n
        for k in need[i]:
            rows.append(head + ids[at: at + k])
            at += k
    width = max(1, max(len(r) for r in rows))
    table = torch.tensor([r + [-1] * (width - len(r)) for r in rows], dtype=torch.int32, device=DEV)
    return table, max(pages, 1)


def prepare(case, seed):
    g, c = _gen(seed), case
    s = {"case": c}
    if c["op"] == "beam":
        b, w, v = c["batch"], c["beams"], c["vocab"]
        s["logits"] = (torch.randn((b * w, v), generator=g, device=DEV) * c["spread"]).to(getattr(torch, c["dtype"]))
        s["scores"] = -20.0 * torch.rand((b, 1), generator=g, device=DEV) - torch.rand((b, w), generator=g, device=DEV).cumsum(1)
        if c["first"]:  # a first step: one beam of each prompt
            s["scores"][:, 1:] = -math.inf
        s["finished"] = torch.rand((b, w), generator=g, device=DEV) < c["finished"] if c["finished"] else None
        return s
    p = c["page"]
    if c["op"] == "sinks":
        b, t = c["batch"], c["tokens"]
        lens = torch.maximum(_ints(c["len_lo"], c["len_hi"], b, g), _queries(s, b, g))
        width = -(-max(c["len_hi"], t) // p)
        table = torch.randperm(b * width, generator=g, device=DEV).to(torch.int32).view(b, width)
        s["table"] = torch.where(torch.arange(width, device=DEV) < ((lens + p - 1) // p)[:, None], table, -1).to(torch.int32).contiguous()
        s["lens"], pages, layers = lens, b * width, 1
    elif c["op"] == "shared":
        n, b = c["groups"], c["members"]
        if c["even"]:
            first = [i * (b // n) for i in range(n + 1)]
        else:  # every group one sequence at least
            cut = (1 + torch.randperm(b - 1, generator=g, device=DEV)[: n - 1]).sort()[0].tolist() if n > 1 else []
            first = [0] + cut + [b]
        prefix = _ints(c["prefix_lo"], c["prefix_hi"], n, g).tolist()
        own_len = torch.maximum(_ints(c["own_lo"], c["own_hi"], b, g), _queries(s, b, g)).tolist()
        s["table"], pages = _shared_table(prefix, own_len, first, p, g)
        s["first"], s["prefix"], layers = first, prefix, 1
        s["groups"] = torch.tensor(first, dtype=torch.int32, device=DEV)
        s["shared"] = torch.tensor(prefix, dtype=torch.int32, device=DEV)
        of = [i for i in range(n) for _ in range(first[i], first[i + 1])]
        s["lens"] = torch.tensor([prefix[of[i]] + own_len[i] for i in range(b)], dtype=torch.int32, device=DEV)
    else:
        b, w, layers = c["batch"], c["beams"], c["layers"]
        own_len = _ints(1, c["own_hi"], b, g)
        # every beam has pages for what it may still write
        s["table"], pages = _shared_table([c["prefix"]] * b, [c["own_hi"] + p] * (b * w), [i * w for i in range(b + 1)], p, g)
        s["lens"] = (c["prefix"] + own_len).repeat_interleave(w).contiguous()
        # better beams have more children
        s["parent"] = (torch.rand((b, w), generator=g, device=DEV) ** 2 * w).to(torch.int32).clamp(max=w - 1)
        s["out"] = torch.empty_like(s["table"])
    s["pool"] = _pool(layers, pages, c, g)
    if own:
        from persistent_megakernel_decode_gb300 import kvcache
        s["cache"] = kvcache.Kv8Cache(s["pool"]["k"], s["pool"]["v"], s["pool"]["k_scale"], s["pool"]["v_scale"])
    return s


# ---- one pass ---------------------------------------------------------------
def run(s):
    return RUN[s["case"]["op"]](s)


def run_sinks(s):
    c = s["case"]
    if own:
        return s["cache"].attend(s["q"], s["table"], s["lens"], q_start=s["q_start"] if c["ragged"] else None,
                                 max_tokens=c["tokens"], window=c["window"], sinks=c["sinks"])
    return plain_sinks(s["q"], s["pool"], s["table"], s["lens"], s["q_start"], c)


def run_shared(s):
    c = s["case"]
    if own:
        return s["cache"].attend_shared(s["q"], s["table"], s["lens"], s["groups"], s["shared"],
                                        q_start=s["q_start"] if c["ragged"] else None, max_tokens=c["tokens"])
    return plain_shared(s)


def run_beam(s):
    c = s["case"]
    if own:
        from persistent_megakernel_decode_gb300 import runtime
        return runtime.beam_select(s["logits"], s["scores"], num=c["num"], finished=s["finished"], end=2)
    return plain_beam(s["logits"], s["scores"], c["num"], s["finished"], 2)


def run_reorder(s):
    if own:
        s["cache"].reorder(s["table"], s["lens"], s["parent"], out=s["out"])
    else:
        plain_reorder(s)
    return dict(s["pool"], table=s["out"])


RUN = {"sinks": run_sinks, "shared": run_shared, "beam": run_beam, "reorder": run_reorder}


# ---- plain forms ------------------------------------------------------------
def _rows_of(pool, scale, table, transposed):
    """Every slot of the table's pages as fp32 tokens [B, S, Hkv, D] of layer 0 (pages of -1: page 0, masked by the caller)."""
    t = table.clamp(min=0).long()
    x = pool[0].view(torch.uint8)[t].view(F8).float() * scale[0][t][..., None, None]
    x = x.transpose(-1, -2) if transposed else x
    b, w, h, p, d = x.shape
    return x.transpose(2, 3).reshape(b, w * p, h, d)


def _softmax_parts(z):
    """exp(z - max), its sum, and the log of the sum of exp(z), all over the last axis."""
    m = z.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(z - m)
    l = e.sum(-1, keepdim=True)
    return e, l, (m + torch.log(l)).squeeze(-1)


def plain_sinks(q, pool, table, lens, q_start, c):
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
    z = (torch.matmul(x, k) * (d ** -0.5)).view(b, hkv, hq // hkv, t, -1)
    pos = (lens.long() - count)[:, None] + i
    j = torch.arange(z.shape[-1], device=DEV)
    seen = (j <= pos[..., None]) & there[..., None] & ((j > pos[..., None] - c["window"]) | (j < c["sinks"]))
    e, l, lse = _softmax_parts(z.masked_fill(~seen[:, None, None], -math.inf))
    o = torch.matmul(e.view(b, hkv, -1, e.shape[-1]), v).view(b, hkv, hq // hkv, t, d) / l.clamp(min=1e-30)
    out = torch.empty_like(flat)
    out[at[there]] = o.permute(0, 3, 1, 2, 4).reshape(b, t, hq, d)[there].to(q.dtype)
    far = torch.empty(flat.shape[:-1], dtype=torch.float32, device=DEV)
    far[at[there]] = lse.permute(0, 3, 1, 2).reshape(b, t, hq)[there]
    return out.view(q.shape), far.view(q.shape[:-1])


def plain_shared(s):
    """Group by group: scores of all its rows with the prefix, which is taken out of its pages once, beside each sequence's
    scores with its own tokens; one softmax over both."""
    c = s["case"]
    hq, hkv, d, t, p = c["q_heads"], c["kv_heads"], c["head_dim"], c["tokens"], c["page"]
    flat = s["q"].reshape(-1, hq, d)
    out = torch.empty_like(flat)
    far = torch.empty(flat.shape[:-1], dtype=torch.float32, device=DEV)
    if not flat.shape[0]:
        return out.view(s["q"].shape), far.view(s["q"].shape[:-1])
    i = torch.arange(t, device=DEV)
    for n, lo, hi in zip(s["prefix"], s["first"], s["first"][1:]):
        m, full, rows = hi - lo, n // p, hq // hkv * t
        q0, count = s["q_start"][lo:hi].long(), (s["q_start"][lo + 1: hi + 1] - s["q_start"][lo:hi]).long()
        there = i < count[:, None]
        at = torch.where(there, q0[:, None] + i, 0)
        x = flat.float()[at].view(m, t, hkv, hq // hkv, d).permute(2, 0, 3, 1, 4)  # [hkv, m, group, t, d]
        table = s["table"][lo:hi]
        head, tail = table[:1, :full], table[:, full:]
        kh, kt = (_rows_of(s["pool"]["k"], s["pool"]["k_scale"], y, False) for y in (head, tail))
        vh, vt = (_rows_of(s["pool"]["v"], s["pool"]["v_scale"], y, True) for y in (head, tail))
        zh = torch.matmul(x.reshape(hkv, m * rows, d), kh[0].permute(1, 2, 0)).view(hkv, m, rows, full * p)
        zt = torch.matmul(x.reshape(hkv, m, rows, d), kt.permute(2, 0, 3, 1))
        pos = (s["lens"][lo:hi].long() - count)[:, None] + i - full * p
        j = torch.arange(zt.shape[-1], device=DEV)
        seen = (j <= pos[..., None]).unsqueeze(1).expand(m, hq // hkv, t, -1).reshape(m, rows, zt.shape[-1])
        z = torch.cat([zh, zt.masked_fill(~seen, -math.inf)], -1) * (d ** -0.5)
        e, l, lse = _softmax_parts(z)
        o = torch.matmul(e[..., : full * p].reshape(hkv, m * rows, full * p), vh[0].transpose(0, 1)).view(hkv, m, rows, d)
        o = (o + torch.matmul(e[..., full * p:], vt.permute(2, 0, 1, 3))) / l.clamp(min=1e-30)
        o = o.view(hkv, m, hq // hkv, t, d).permute(1, 3, 0, 2, 4).reshape(m, t, hq, d)
        out[at[there]] = o[there].to(out.dtype)
        far[at[there]] = lse.view(hkv, m, hq // hkv, t).permute(1, 3, 0, 2).reshape(m, t, hq)[there]
    return out.view(s["q"].shape), far.view(s["q"].shape[:-1])


def plain_beam(logits, scores, num, finished, end):
    """In 64 bits: the order of totals that lie close together is the result."""
    b, w = scores.shape
    v = logits.shape[1]
    z = logits.double().view(b, w, v)
    z = torch.where(torch.isnan(z), -math.inf, z)
    lse = _softmax_parts(z)[2]
    total = scores.double()[..., None] + (z - lse[..., None])
    if finished is not None:
        total.masked_fill_(finished[..., None], -math.inf)
        total[..., end] = torch.where(finished, scores.double(), total[..., end])
    total.masked_fill_(~torch.isfinite(scores)[..., None], -math.inf)
    total = total.view(b, w * v)
    best, at, index = [], [], torch.arange(w * v, device=DEV)
    for _ in range(num):
        most = total.amax(1, keepdim=True)
        i = torch.where(total == most, index, w * v).amin(1, keepdim=True)  # the lowest index of equal ones
        total.scatter_(1, i, -math.inf)
        best.append(most)
        at.append(i)
    best, at = torch.cat(best, 1), torch.cat(at, 1)
    none = best == -math.inf
    part = lambda x: torch.where(none, -1, x).to(torch.int32)  # noqa: E731
    return best.float(), part(at // v), part(at % v)


def plain_reorder(s):
    """A parent's page that is being filled stays with one child, with itself where it goes on, else with its first; the
    other children, in their order, take the pages of the beams without children, in their order, and a copy of the tokens."""
    table, par, p = s["table"], s["parent"].long(), s["case"]["page"]
    b, w = par.shape
    row = torch.arange(w, device=DEV)
    child = par[:, None, :] == row[None, :, None]  # [b, parent, child]
    first = torch.where(child, row, w).amin(2)
    keeper = torch.where(par == row, row, first)
    extra = keeper.gather(1, par) != row
    dead = ~child.any(2)
    free = torch.where(dead, row, w + row).sort(1)[0]  # rows without children first
    page_of = torch.where(extra, free.gather(1, (extra.cumsum(1) - 1).clamp(min=0)) % w, par)
    base = torch.arange(b, device=DEV)[:, None] * w
    src, tail = (base + par).view(-1), (base + page_of).view(-1)
    lens = s["lens"].long()
    full, part = lens // p, lens % p
    col = torch.arange(table.shape[1], device=DEV)
    s["out"].copy_(torch.where(col < full[:, None], table[src],
                               torch.where((col == full[:, None]) & (part[:, None] > 0), table[tail], table)))
    move = (extra.view(-1) & (part > 0)).nonzero().squeeze(1)
    at = full[move][:, None]
    a, z = table[src[move]].gather(1, at).squeeze(1).long(), table[tail[move]].gather(1, at).squeeze(1).long()
    new = torch.arange(p, device=DEV) < part[move][:, None]
    for name in ("k", "v"):
        x = s["pool"][name].view(torch.uint8)
        m = new[None, :, None, :, None] if name == "k" else new[None, :, None, None, :]
        x[:, z] = torch.where(m, x[:, a], x[:, z])
        s["pool"][name + "_scale"][:, z] = s["pool"][name + "_scale"][:, a]


# ---- what a pass cannot do without ------------------------------------------
def work(case):
    c = case
    if c["op"] == "beam":
        n = c["batch"] * (1 if c["first"] else c["beams"] * (1 - c["finished"])) * c["vocab"]  # beams that go on
        return {"bytes": int(n * (4 if c["dtype"] == "float32" else 2)) + 12 * c["batch"] * c["num"], "flops": int(4 * n)}
    if c["op"] == "reorder":
        # about 0.45 of the beams are copies, of half a page; the table is read and written
        tokens = 0.45 * c["batch"] * c["beams"] * c["page"] / 2
        rows = c["batch"] * c["beams"] * (-(-(c["prefix"] + c["own_hi"]) // c["page"]) + 1)
        return {"bytes": int(4 * c["layers"] * c["kv_heads"] * c["head_dim"] * tokens + 8 * rows), "flops": 0}
    t = c["tokens"] / 2 if c["ragged"] else c["tokens"]
    row_bytes, token_bytes = 4 * c["head_dim"] + 4, c["kv_heads"] * (2 * c["head_dim"] + 8 / c["page"])
    if c["op"] == "sinks":
        n = max((c["len_lo"] + c["len_hi"]) / 2, t)
        n = min(n, c["window"] + t + c["sinks"])
        rows = c["batch"] * t * c["q_heads"]
        return {"bytes": int(c["batch"] * n * token_bytes + rows * row_bytes), "flops": int(4 * rows * max(1.0, n - t / 2) * c["head_dim"])}
    prefix, mine = (c["prefix_lo"] + c["prefix_hi"]) / 2, max((c["own_lo"] + c["own_hi"]) / 2, t)
    rows = c["members"] * t * c["q_heads"]
    return {"bytes": int((c["groups"] * prefix + c["members"] * mine) * token_bytes + rows * row_bytes),
            "flops": int(4 * rows * (prefix + max(1.0, mine - t / 2)) * c["head_dim"])}


# ---- from the definitions, in 64 bits ---------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return EXACT[case["op"]](s)


def _value(code):
    """The values of e4m3 codes: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    c = code.view(torch.uint8).to(torch.int32)
    e, f = (c >> 3) & 15, (c & 7).double()
    power = torch.tensor([2.0 ** i for i in range(-10, 12)], dtype=torch.float64, device=c.device)
    x = torch.where(e > 0, (1 + f / 8) * power[(e + 3).long()], f * 2.0 ** -9)
    return torch.where(c >= 128, -x, x)


def _token_rows(s, b, name, n):
    """The first n tokens of sequence b in layer 0, fp64 [n, Hkv, D]."""
    pages = s["table"][b, : -(-n // s["case"]["page"])].long()
    x = _value(s["pool"][name][0].view(torch.uint8)[pages]) * s["pool"][name + "_scale"][0][pages].double()[..., None, None]
    x = x.permute(0, 3, 1, 2) if name == "v" else x.permute(0, 2, 1, 3)
    return x.reshape(-1, x.shape[2], x.shape[3])[:n]


def exact_attend(s):
    """Each sequence by itself, over every token that its queries see."""
    c = s["case"]
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    flat = s["q"].reshape(-1, hq, d).double()
    out, lse = torch.zeros_like(flat), torch.full(flat.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    edge = s["q_start"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        if edge[b + 1] == edge[b] or not n:
            continue
        k, v = (_token_rows(s, b, x, n) for x in ("k", "v"))
        for i in range(edge[b], edge[b + 1]):
            pos = n - edge[b + 1] + i
            j = torch.arange(pos + 1, device=DEV)
            if c["op"] == "sinks":
                j = j[(j > pos - c["window"]) | (j < c["sinks"])]
            z = torch.einsum("hgd,jhd->hgj", flat[i].view(hkv, hq // hkv, d), k[j]) / math.sqrt(d)
            far = torch.logsumexp(z, -1)
            lse[i] = far.reshape(-1)
            out[i] = torch.einsum("hgj,jhd->hgd", torch.exp(z - far[..., None]), v[j]).reshape(hq, d)
    return out.view(s["q"].shape), lse.view(s["q"].shape[:-1])


def exact_beam(s):
    c = s["case"]
    b, w, v, num = c["batch"], c["beams"], c["vocab"], c["num"]
    best = torch.full((b, num), -math.inf, dtype=torch.float64)
    parent, token = torch.full((b, num), -1, dtype=torch.int32), torch.full((b, num), -1, dtype=torch.int32)
    for i in range(b):
        rows = []
        for r in range(w):
            x, score = s["logits"][i * w + r].double(), float(s["scores"][i, r])
            if not math.isfinite(score):
                rows.append(torch.full_like(x, -math.inf))
            elif s["finished"] is not None and s["finished"][i, r]:
                rows.append(torch.full_like(x, -math.inf))
                rows[-1][2] = score
            else:
                rows.append(score + torch.log_softmax(x, 0))
        value, order = torch.sort(torch.cat(rows), descending=True, stable=True)
        value, order = value[:num].cpu(), order[:num].cpu()
        there = value > -math.inf
        best[i] = value
        parent[i] = torch.where(there, order // v, -1)
        token[i] = torch.where(there, order % v, -1)
    return best, parent, token


def exact_reorder(s):
    c = s["case"]
    w, p = c["beams"], c["page"]
    if c["layers"] * s["pool"]["k"].shape[1] > 30000:
        return None
    codes = {n: torch.stack([_value(x) for x in s["pool"][n]]) for n in ("k", "v")}
    scales = {n: s["pool"][n + "_scale"].double() for n in ("k", "v")}
    old, lens = s["table"].tolist(), s["lens"].tolist()
    new = [list(r) for r in old]
    for b, parents in enumerate(s["parent"].tolist()):
        n = lens[b * w]
        t, part = n // p, n % p
        dead = [r for r in range(w) if r not in parents]
        kept = set()
        for r in [r for r in range(w) if parents[r] == r] + [r for r in range(w) if parents[r] != r]:
            new[b * w + r][:t] = old[b * w + parents[r]][:t]
            if part and parents[r] not in kept:  # the parent's page goes on as this child's
                kept.add(parents[r])
                new[b * w + r][t] = old[b * w + parents[r]][t]
            elif part:
                src, dst = old[b * w + parents[r]][t], old[b * w + dead.pop(0)][t]
                new[b * w + r][t] = dst
                codes["k"][:, dst, :, :part] = codes["k"][:, src, :, :part]
                codes["v"][:, dst, :, :, :part] = codes["v"][:, src, :, :, :part]
                for x in scales.values():
                    x[:, dst] = x[:, src]
    return {"k": codes["k"], "k_scale": scales["k"], "v": codes["v"], "v_scale": scales["v"],
            "table": torch.tensor(new, dtype=torch.int32)}


EXACT = {"sinks": exact_attend, "shared": exact_attend, "beam": exact_beam, "reorder": exact_reorder}
