"""Measured cases of the 4-bit paged KV cache: the tables that place requests in it, the write into it, the read back
into 16 bits, and decode attention over it.

A row of the cache is one key or value of one KV head: D codes of 4 bits and one E4M3 scale per group of 32 elements,
value = descale * scale * (code - 8). Eight codes make a word, the lowest element in the lowest bits; a group's units
(K: 8 elements, V: 4) are dealt over the row, unit u of group i at position u * groups + i.

`own` chooses between the framework's calls and the plain form of the same operators in elementary torch operations.
"""
import math
import random

import torch

own = False

GROUP = 32
DEV = "cuda"
UNIT = {"k": 8, "v": 4}  # elements of one dealt unit


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one short sequence, few heads: the smallest decode call, its launch and merge latency
        dict(name="decode 1x300 d64", op="decode", B=1, Hq=8, Hkv=2, M=1, N=300, D=64, page=16, causal=True, window=0,
             sinks=0, ragged=False, dtype="float16"),
        # the GQA decode workload of the benchmark over its window, with the first tokens kept visible
        dict(name="decode 8x8192 window", op="decode", B=8, Hq=32, Hkv=8, M=1, N=8192, D=128, page=16, causal=True,
             window=4096, sinks=4, ragged=False, dtype="bfloat16"),
        # a serving batch in mid-flight: contexts of every length up to 16384
        dict(name="decode 64 ragged 16384", op="decode", B=64, Hq=32, Hkv=8, M=1, N=16384, D=128, page=64, causal=True,
             window=0, sinks=0, ragged=True, dtype="bfloat16"),
        # speculative decode: four rows a sequence, 16 grouped rows per KV head
        dict(name="decode 16x4 rows 8192", op="decode", B=16, Hq=32, Hkv=8, M=4, N=8192, D=128, page=128, causal=True,
             window=0, sinks=0, ragged=True, dtype="float16"),
        # one long document alone on the card
        dict(name="decode 1x131072", op="decode", B=1, Hq=32, Hkv=8, M=1, N=131072, D=128, page=256, causal=True,
             window=0, sinks=0, ragged=False, dtype="bfloat16"),
        # many short chats, a smaller head
        dict(name="decode 256 ragged 1000 d64", op="decode", B=256, Hq=16, Hkv=4, M=1, N=1000, D=64, page=32,
             causal=True, window=0, sinks=0, ragged=True, dtype="bfloat16"),
        # odd sizes: three query heads per KV head, the smallest head dimension, no causal mask
        dict(name="decode 5x777 d32", op="decode", B=5, Hq=12, Hkv=4, M=1, N=777, D=32, page=16, causal=False,
             window=500, sinks=37, ragged=True, dtype="float16"),
        # one decode step's rows written, the short contexts read back
        dict(name="append 16 rows", op="append", B=16, Hq=32, Hkv=8, N=61, new=1, pad=0, D=128, page=16, ragged=True,
             dtype="bfloat16"),
        # a prefill chunk of several requests written behind their contexts (a padded batch), then read back
        dict(name="append 16384 rows", op="append", B=8, Hq=32, Hkv=8, N=4096, new=2048, pad=256, D=128, page=64,
             ragged=False, dtype="bfloat16"),
        # a long context read back for a prefill over it
        dict(name="gather 2x32768", op="gather", B=2, Hq=32, Hkv=8, N=32768, D=128, page=128, ragged=False,
             dtype="float16"),
        # tables of one decode step
        dict(name="plan 64 requests", op="plan", B=64, N=8192, new=1, pad=0, page=16, ragged=True),
        # tables of a large mixed step, padded to a fixed number of rows
        dict(name="plan 2000 requests", op="plan", B=2000, N=16384, new=97, pad=301, page=16, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "append", "gather", "plan"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "plan":
        B = _log(rng, 1, 4000)
        new = _log(rng, 1, max(1, 200000 // B))
        return dict(op=op, B=B, N=new + _log(rng, 1, 16384), new=new, pad=rng.choice([0, _log(rng, 1, 1000)]), page=page,
                    ragged=rng.random() < 0.8)
    D = rng.choice([32, 64, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 4, 7, 8])
    dtype = rng.choice(["bfloat16", "float16"])
    ragged = rng.random() < 0.7
    room = 400_000_000 if op == "decode" else 60_000_000  # elements of K that the cache holds, at most
    B = _log(rng, 1, 128)
    N = _log(rng, 1, max(1, min(131072, room // (B * Hkv * D))))
    c = dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, N=N, D=D, page=page, ragged=ragged, dtype=dtype)
    if op == "append":
        return dict(c, new=_log(rng, 1, N), pad=rng.choice([0, _log(rng, 1, 500)]))
    if op == "gather":
        return c
    return dict(c, M=rng.choice([1, 1, 1, 2, 4, 5]), causal=rng.random() < 0.8,
                window=rng.choice([0, 0, _log(rng, 1, N)]), sinks=rng.choice([0, 0, 1, 4, _log(rng, 1, 100)]))


def _lens(c):
    """Keys of each sequence at the end of the call: all N, or spread over 1..N."""
    if not c["ragged"]:
        return [c["N"]] * c["B"]
    return [1 + int((c["N"] - 1) * ((b + 1) * 0.6180339887498949 % 1.0) + 0.5) for b in range(c["B"])]


def _news(c):
    """New rows of each request in this step: at most `new`, of its sequence's keys."""
    lens = _lens(c)
    if not c["ragged"] or c["new"] == 1:
        return [min(c["new"], L) for L in lens]
    return [min(L, int((c["new"] + 1) * ((b + 1) * 0.7548776662466927 % 1.0))) for b, L in enumerate(lens)]


def _pages(n, page):
    return -(-n // page)


def _dtype(c):
    return getattr(torch, c["dtype"])


# the power-of-two factors of the cache: scales of keys near 1 and of values near 1/8
K_DESCALE, V_DESCALE = 1.0, 0.125


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _rows(gen, n, c, which):
    """Key or value rows as a model makes them: keys with a few strong channels, values around half a unit."""
    x = torch.randn((n, c["Hkv"], c["D"]), generator=gen, device=DEV)
    d = torch.arange(c["D"], device=DEV)
    if which == "k":
        x *= 0.7 + 2.0 * (d % 19 == 3)
    else:
        x *= 0.5
    return x.to(_dtype(c))


def _cache(gen, c, num_pages):
    """A cache of quantized rows, [pages, Hkv, page, ...] codes and scales for K and V."""
    out = {}
    for which, descale in (("k", K_DESCALE), ("v", V_DESCALE)):
        codes = torch.empty((num_pages, c["Hkv"], c["page"], c["D"] // 2), dtype=torch.uint8, device=DEV)
        scales = torch.empty((num_pages, c["Hkv"], c["page"], c["D"] // GROUP), dtype=torch.float8_e4m3fn, device=DEV)
        step = max(1, 64_000_000 // (c["Hkv"] * c["page"] * c["D"]))
        for p in range(0, num_pages, step):
            n = min(step, num_pages - p)
            s, q = _quantize(_rows(gen, n * c["page"], c, which), descale)
            shape = (n, c["page"], c["Hkv"], -1)
            codes[p:p + n] = _pack(q, which).view(shape).transpose(1, 2)
            scales.view(torch.uint8)[p:p + n] = s.view(torch.uint8).view(shape).transpose(1, 2)
        out[which] = (codes, scales)
    return out


def _table(gen, c, lens):
    """Pages of every sequence, in shuffled order, and the number of pages of the pool."""
    need = torch.tensor([_pages(L, c["page"]) for L in lens], device=DEV)
    width = _pages(max(lens), c["page"])
    total = int(need.sum())
    num_pages = total + 3
    ids = torch.randperm(num_pages, generator=gen, device=DEV)[:total]
    at = torch.cumsum(need, 0) - need
    col = torch.arange(width, device=DEV)
    idx = (at[:, None] + col).clamp(max=max(total - 1, 0))
    table = torch.where(col < need[:, None], ids[idx], torch.zeros_like(idx))
    return table.to(torch.int32).contiguous(), num_pages


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    c = dict(case)
    lens = _lens(c)
    st = {"case": c}
    if c["op"] == "plan":
        news = _news(c)
        cached = [L - n for L, n in zip(lens, news)]
        held = sum(_pages(x, c["page"]) for x in cached)
        taken = sum(_pages(L, c["page"]) for L in lens) - held
        ids = torch.randperm(held + taken + 50, generator=gen, device=DEV).to(torch.int32)
        width = _pages(max(lens), c["page"])
        need = torch.tensor([_pages(x, c["page"]) for x in cached], device=DEV)
        at = torch.cumsum(need, 0) - need
        col = torch.arange(width, device=DEV)
        old = ids[(at[:, None] + col).clamp(max=held + taken)]
        st["table"] = torch.where(col < need[:, None], old, torch.full_like(old, -1)).contiguous()
        st["free"] = ids[held:].contiguous()
        st["cached"] = torch.tensor(cached, dtype=torch.int32, device=DEV)
        st["new"] = torch.tensor(news, dtype=torch.int32, device=DEV)
        st["seq_lens"] = torch.empty(c["B"], dtype=torch.int32, device=DEV)
        st["row_starts"] = torch.empty(c["B"] + 1, dtype=torch.int32, device=DEV)
        st["slots"] = torch.empty(sum(news) + c["pad"], dtype=torch.int32, device=DEV)
        st["stats"] = torch.empty(3, dtype=torch.int32, device=DEV)
        return st
    st["table"], num_pages = _table(gen, c, lens)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["cache"] = _cache(gen, c, num_pages)
    if c["op"] == "decode":
        st["q"] = torch.randn((c["B"], c["Hq"], c["M"], c["D"]), generator=gen, device=DEV).to(_dtype(c))
        st["o"] = torch.empty_like(st["q"])
        st["ws"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)  # kept by the program for all its calls
        return st
    st["k"] = torch.empty((c["B"], c["Hkv"], c["N"], c["D"]), dtype=_dtype(c), device=DEV)
    st["v"] = torch.empty_like(st["k"])
    if c["op"] == "append":
        news = _news(c)
        T = sum(news) + c["pad"]
        # K and V are parts of one projection's output: rows of Hq + 2 Hkv heads
        H, Hkv, D = c["Hq"], c["Hkv"], c["D"]
        qkv = torch.empty((T, H + 2 * Hkv, D), dtype=_dtype(c), device=DEV)
        qkv[:, :H] = 0
        qkv[:, H:H + Hkv] = _rows(gen, T, c, "k")
        qkv[:, H + Hkv:] = _rows(gen, T, c, "v")
        st["k_new"], st["v_new"] = qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        n, L = torch.tensor(news, device=DEV), torch.tensor(lens, device=DEV)
        b = torch.repeat_interleave(torch.arange(c["B"], device=DEV), n)
        pos = (L - n)[b] + torch.arange(sum(news), device=DEV) - (torch.cumsum(n, 0) - n)[b]
        slots = st["table"].long()[b, pos // c["page"]] * c["page"] + pos % c["page"]
        st["slots"] = torch.cat([slots, torch.full((c["pad"],), -1, device=DEV)]).to(torch.int32)
    return st


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _quantize(x, descale):
    """x [..., D] -> E4M3 scales [..., D/32] and codes [..., D] in 0..15. The quotient is taken in 64 bits: values next
    to a border between two codes."""
    xs = (x.float() / descale).unflatten(-1, (-1, GROUP))
    top = (xs.abs().amax(-1, keepdim=True).double() / 7.5).float()
    s = top.clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.double()
    n = torch.floor(xs.abs().double() / torch.where(sf > 0, sf, torch.ones_like(sf)) + 0.5)
    n = torch.where(sf > 0, torch.where(xs < 0, -n, n), torch.zeros_like(n)).clamp(-8, 7)
    return s.squeeze(-1), (n + 8).to(torch.uint8).flatten(-2)


def _pack(codes, which):
    """[..., D] codes -> [..., D/2] bytes in the dealt order."""
    u = codes.unflatten(-1, (-1, GROUP // UNIT[which], UNIT[which])).transpose(-3, -2)
    u = u.reshape(*codes.shape[:-1], -1, 2)
    return u[..., 0] | (u[..., 1] << 4)


def _values(codes, scales, which, descale):
    """[..., D/2] bytes and [..., D/32] scales -> [..., D] in 32 bits."""
    D = codes.shape[-1] * 2
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    n = n.unflatten(-1, (GROUP // UNIT[which], D // GROUP, UNIT[which])).transpose(-3, -2).reshape(*codes.shape[:-1], -1, GROUP)
    return ((n.float() - 8) * (scales.float() * descale).unsqueeze(-1)).flatten(-2)


def _read(st, which, descale):
    """The cache of every sequence in order, [B, Hkv, width * page, D] in 32 bits."""
    codes, scales = st["cache"][which]
    t = st["table"].long().flatten()
    x = _values(codes[t], scales.view(torch.uint8)[t].view(torch.float8_e4m3fn), which, descale)
    x = x.unflatten(0, tuple(st["table"].shape))  # [B, width, Hkv, page, D]
    return x.transpose(1, 2).flatten(2, 3)


def _gather_plain(st):
    out = []
    for which, descale in (("k", K_DESCALE), ("v", V_DESCALE)):
        x = _read(st, which, descale)[:, :, : st["case"]["N"]]
        if x.shape[2] < st["case"]["N"]:
            x = torch.nn.functional.pad(x, (0, 0, 0, st["case"]["N"] - x.shape[2]))
        held = torch.arange(x.shape[2], device=DEV) < st["lens"][:, None]
        out.append(torch.where(held[:, None, :, None], x, torch.zeros_like(x)).to(_dtype(st["case"])))
    return out


def _append_plain(st):
    c = st["case"]
    slots = st["slots"].long()
    last = slots.new_full((), st["cache"]["k"][0].shape[0] * c["page"])
    for which, descale in (("k", K_DESCALE), ("v", V_DESCALE)):
        s, q = _quantize(st[which + "_new"], descale)
        codes, scales = st["cache"][which]
        page = torch.where(slots >= 0, slots, last) // c["page"]
        for pool, rows in ((codes, _pack(q, which)), (scales.view(torch.uint8), s.view(torch.uint8))):
            # a row without a slot goes to a page behind the pool, which is dropped
            held = torch.cat([pool, pool[:1]])
            held[page, :, slots.clamp(min=0) % c["page"]] = rows
            pool.copy_(held[:-1])


def _decode_plain(st):
    c = st["case"]
    B, Hq, Hkv, M, D = c["B"], c["Hq"], c["Hkv"], c["M"], c["D"]
    k = _read(st, "k", K_DESCALE)
    q = st["q"].float().reshape(B, Hkv, Hq // Hkv * M, D)
    s = (q @ k.transpose(-1, -2)) / math.sqrt(D)
    del k
    n = s.shape[-1]
    L = st["lens"].long()
    j = torch.arange(n, device=DEV)
    p = (L[:, None] - M + torch.arange(M, device=DEV))[:, :, None]  # position of each row
    see = (j < L[:, None, None]).expand(B, M, n)
    if c["causal"]:
        see = see & (j <= p)
    if c["window"] > 0:
        see = see & ((j > p - c["window"]) | (j < c["sinks"]))
    see = see[:, None, None].expand(B, Hkv, Hq // Hkv, M, n).reshape(s.shape)
    s = torch.where(see, s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    del s, see
    total = e.sum(-1, keepdim=True)
    o = (e @ _read(st, "v", V_DESCALE)) / torch.where(total > 0, total, torch.ones_like(total))
    return o.reshape(B, Hq, M, D).to(_dtype(c))


def _plan_plain(st):
    c = st["case"]
    page = c["page"]
    cached, new, table = st["cached"].long(), st["new"].long(), st["table"]
    lens = cached + new
    ends = torch.cumsum(new, 0)
    starts = ends - new
    old = (cached + page - 1) // page
    need = (lens + page - 1) // page - old
    first = torch.cumsum(need, 0) - need
    col = torch.arange(table.shape[1], device=DEV)
    fresh = (col >= old[:, None]) & (col < (old + need)[:, None])
    pick = (first[:, None] + col - old[:, None]).clamp(0, st["free"].numel() - 1)
    table.copy_(torch.where(fresh, st["free"][pick], table))
    row = torch.arange(st["slots"].numel(), device=DEV)
    b = torch.searchsorted(ends, row, right=True).clamp(max=c["B"] - 1)
    live = row < ends[-1]
    pos = torch.where(live, cached[b] + row - starts[b], torch.zeros_like(row))
    slot = table.long()[b, pos // page] * page + pos % page
    st["slots"].copy_(torch.where(live, slot, torch.full_like(slot, -1)))
    st["seq_lens"].copy_(lens)
    st["row_starts"].copy_(torch.cat([starts, ends[-1:]]))
    st["stats"].copy_(torch.stack([ends[-1], need.sum(), torch.zeros_like(ends[-1])]))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    st, c = state, state["case"]
    if c["op"] == "plan":
        if own:
            import streaming_attention_gb300 as sa

            sa.attn_page_plan(st["cached"], st["new"], st["free"], st["table"], st["seq_lens"], st["row_starts"],
                              st["slots"], st["stats"], c["page"])
        else:
            _plan_plain(st)
        return {m: st[m] for m in ("table", "seq_lens", "row_starts", "slots", "stats")}
    if c["op"] == "decode":
        if own:
            import streaming_attention_gb300 as sa

            sa.attn_decode_paged_kv4(st["q"], *st["cache"]["k"], *st["cache"]["v"], st["table"], st["lens"], st["o"],
                                     c["N"], c["causal"], c["window"], c["sinks"], 0.0, K_DESCALE, V_DESCALE, st["ws"])
            return st["o"]
        return _decode_plain(st)
    if own:
        import streaming_attention_gb300 as sa

        if c["op"] == "append":
            sa.attn_kv4_append(st["k_new"], st["v_new"], st["slots"], *st["cache"]["k"], *st["cache"]["v"], K_DESCALE,
                               V_DESCALE)
        sa.attn_kv4_gather(*st["cache"]["k"], *st["cache"]["v"], st["table"], st["lens"], st["k"], st["v"], K_DESCALE,
                           V_DESCALE)
        return {"k": st["k"], "v": st["v"]}
    if c["op"] == "append":
        _append_plain(st)
    k, v = _gather_plain(st)
    return {"k": k, "v": v}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _spelled(codes, scales, which, descale):
    """One code at a time by its place in the row: [..., D] in 64 bits."""
    D = codes.shape[-1] * 2
    unit, groups = UNIT[which], D // GROUP
    where = [((d % GROUP) // unit * groups + d // GROUP) * unit + d % unit for d in range(D)]
    at = torch.tensor([w // 2 for w in where], device=DEV)
    shift = torch.tensor([4 * (w % 2) for w in where], dtype=torch.uint8, device=DEV)
    n = torch.bitwise_and(torch.bitwise_right_shift(codes.index_select(-1, at), shift), 15).double() - 8
    return n * torch.repeat_interleave(scales.double(), GROUP, -1) * descale


def _e4m3(a):
    """Nearest E4M3 value of a >= 0, ties to the even mantissa, at most 448: a step is 2^(e-3), e at least -6."""
    e = torch.frexp(torch.where(a > 0, a, torch.ones_like(a)))[1].double() - 1
    step = torch.exp2(e.clamp(min=-6) - 3)
    return (torch.round(a / step) * step).clamp(max=448.0)


def _sequence(st, b, L, which, descale):
    """Keys or values 0..L-1 of sequence b, [Hkv, L, D] in 64 bits."""
    codes, scales = st["cache"][which]
    page = st["case"]["page"]
    ids = st["table"][b, : _pages(L, page)].long()
    x = _spelled(codes[ids], scales.view(torch.uint8)[ids].view(torch.float8_e4m3fn), which, descale)
    return x.transpose(0, 1).flatten(1, 2)[:, :L]


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    lens = _lens(c)
    if c["op"] == "plan":
        return _plan_by_hand(st, c)
    if c["op"] == "decode":
        G, M = c["Hq"] // c["Hkv"], c["M"]
        o = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
        for b, L in enumerate(lens):
            k, v = (_sequence(st, b, L, w, f) for w, f in (("k", K_DESCALE), ("v", V_DESCALE)))
            for i in range(M):
                p = i + L - M
                j = torch.arange(L, device=DEV)
                keep = torch.ones(L, dtype=torch.bool, device=DEV)
                if c["causal"]:
                    keep &= j <= p
                if c["window"] > 0:
                    keep &= (j > p - c["window"]) | (j < c["sinks"])
                if not bool(keep.any()):
                    continue
                q = st["q"][b, :, i].double().view(c["Hkv"], G, c["D"])
                w = torch.softmax(torch.einsum("hgd,hjd->hgj", q, k[:, keep]) / math.sqrt(c["D"]), -1)
                o[b, :, i] = torch.einsum("hgj,hjd->hgd", w, v[:, keep]).reshape(c["Hq"], c["D"])
        return o
    out = {}
    for which, descale in (("k", K_DESCALE), ("v", V_DESCALE)):
        x = torch.zeros(st["k"].shape, dtype=torch.float64, device=DEV)
        rows = at = None
        if c["op"] == "append":
            y = st[which + "_new"].double() / descale
            y = y.view(*y.shape[:-1], -1, GROUP)
            s = _e4m3(y.abs().amax(-1, keepdim=True) / 7.5)
            n = torch.floor(y.abs() / s.clamp(min=2.0 ** -30) + 0.5) * torch.sign(y)
            rows = (n.clamp(-8, 7) * s * descale).flatten(-2)
            at = 0
        for b, (L, n_new) in enumerate(zip(lens, _news(c) if rows is not None else [0] * len(lens))):
            x[b, :, :L] = _sequence(st, b, L, which, descale)
            if n_new:
                x[b, :, L - n_new:L] = rows[at:at + n_new].transpose(0, 1)
                at += n_new
        out[which] = x
    return out


def _plan_by_hand(st, c):
    table, free = st["table"].tolist(), st["free"].tolist()
    starts, slots, used = [0], [], 0
    for b, (have, n) in enumerate(zip(st["cached"].tolist(), st["new"].tolist())):
        for pos in range(have, have + n):
            if pos % c["page"] == 0:
                table[b][pos // c["page"]] = free[used]
                used += 1
            slots.append(table[b][pos // c["page"]] * c["page"] + pos % c["page"])
        starts.append(len(slots))
    stats = [len(slots), used, 0]
    slots += [-1] * c["pad"]
    return {m: torch.tensor(v, dtype=torch.int32) for m, v in
            (("table", table), ("seq_lens", _lens(c)), ("row_starts", starts), ("slots", slots), ("stats", stats))}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    lens = _lens(c)
    if c["op"] == "plan":
        news = _news(c)
        taken = sum(_pages(L, c["page"]) - _pages(L - n, c["page"]) for L, n in zip(lens, news))
        words = 2 * c["B"] + 2 * taken + c["B"] + (c["B"] + 1) + sum(news) + c["pad"] + 3
        words += sum(1 for L, n in zip(lens, news) if n and (L - n) % c["page"])  # the page that is being filled
        return {"bytes": 4.0 * words, "flops": float(sum(news))}
    row = 2.0 * c["Hkv"] * (c["D"] // 2 + c["D"] // GROUP)  # one key and one value of every KV head
    wide = 2.0 * c["Hkv"] * c["D"] * 2
    table = 4.0 * sum(_pages(L, c["page"]) for L in lens) + 4.0 * c["B"]
    if c["op"] == "decode":
        keys = pairs = 0
        for L in lens:
            seen, last = 0, L
            for i in range(c["M"]):
                p = i + L - c["M"]
                hi = min(p + 1, L) if c["causal"] else L
                lo = max(0, p - c["window"] + 1) if c["window"] > 0 else 0
                hi = max(hi, 0)
                lo = min(lo, hi)
                pairs += hi - lo + min(c["sinks"], lo)
                last = min(last, lo)
                seen = max(seen, hi)
            keys += seen - last + min(c["sinks"], last)
        qo = 2.0 * 2 * c["B"] * c["Hq"] * c["M"] * c["D"]
        return {"bytes": keys * row + qo + table, "flops": 4.0 * c["D"] * c["Hq"] * pairs}
    T = sum(lens)
    padded = 1.0 * c["B"] * c["N"]
    n = {"bytes": T * row + padded * wide + table, "flops": 2.0 * T * c["Hkv"] * c["D"]}
    if c["op"] == "append":
        new = sum(_news(c))
        n["bytes"] += new * (row + wide) + 4.0 * (new + c["pad"])
        n["flops"] += 8.0 * new * c["Hkv"] * c["D"]
    return n
