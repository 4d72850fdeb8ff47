"""The 4-bit paged cache in 64 bits, from its definition: quantization, the order
of a row's codes, the tables of a step, and attention with its error bound.
Shares nothing with the library."""
import math

import numpy as np
import torch

GROUP = 32
UNIT = {"k": 8, "v": 4}


def e4m3_round(a):
    """Nearest E4M3 value of a >= 0 (ties to the even mantissa, at most 448) and its byte."""
    a = np.minimum(np.asarray(a, dtype=np.float64), 448.0)
    _, e = np.frexp(np.where(a > 0, a, 1.0))
    e = np.maximum(e - 1, -6)
    step = np.exp2(e - 3.0)
    v = np.rint(a / step) * step  # rint: halves to even; a multiple of the step is even iff its mantissa is
    _, e = np.frexp(np.where(v > 0, v, 1.0))
    e = np.maximum(e - 1, -6)
    mant = np.rint(v / np.exp2(e - 3.0)).astype(np.int64)  # 8..15 normal, 0..7 subnormal
    byte = np.where(mant >= 8, (e + 7) * 8 + (mant - 8), mant)
    return v, byte.astype(np.uint8)


def e4m3_value(byte):
    b = np.asarray(byte).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    return np.where(b & 128, -v, v)


def quantize(x, descale):
    """x [..., D] (64-bit) -> codes [..., D] in 0..15, scale bytes [..., D/32], values [..., D]."""
    g = (x / descale).reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    s, byte = e4m3_round(np.abs(g).max(-1) / 7.5)
    sd = s[..., None]
    n = np.sign(g) * np.floor(np.abs(g) / np.where(sd > 0, sd, 1.0) + 0.5)
    n = np.where(sd > 0, np.clip(n, -8, 7), 0.0)
    return (n + 8).astype(np.uint8).reshape(x.shape), byte, (n * sd * descale).reshape(x.shape)


def place(D, which):
    """Position in the row (in codes) of every element."""
    u, ng = UNIT[which], D // GROUP
    return np.array([((d % GROUP) // u * ng + d // GROUP) * u + d % u for d in range(D)])


def pack(codes, which):
    row = np.empty_like(codes)
    row[..., place(codes.shape[-1], which)] = codes
    return row[..., 0::2] | (row[..., 1::2] << 4)


def unpack(packed, which):
    D = packed.shape[-1] * 2
    row = np.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], D)
    return row[..., place(D, which)]


def values(packed, scale_bytes, which, descale):
    n = unpack(packed, which).astype(np.float64) - 8
    return n * np.repeat(e4m3_value(scale_bytes), GROUP, -1) * descale


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def bytes_of(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def visible(L, M, i, causal, window, sinks):
    """Keys that row i of M sees in a sequence of L keys."""
    p = i + L - M
    j = np.arange(L)
    see = j <= p if causal else np.ones(L, bool)
    if window > 0:
        see &= (j > p - window) | (j < sinks)
    return see


def attention(q, k, v, causal, window, sinks, scale, out_dtype, ku=None, vu=None, vd=0.125):
    """Rows q [Hq, M, D] over k, v [Hkv, L, D], 64-bit numpy: (o, bound). ku, vu: what one code stands for, per
    element (k and v themselves are codes less 8 times that). Products are taken of the codes 0..15 and of 8 times
    the unit, whose difference is the value: sums of them are up to 23 units large, whatever the values are. The
    bound per element counts
      the output's rounding                            eps/2 |o|
      two roundings to FP16, of the probability p (times 2^3 or more at the largest score) and of its product
      with the value's scale                           2 * 2^-11 A,        A = sum w |v|
      such products below FP16's normal range: each is off by at most 2^-25, times a code of at most 8 and
      the factor vd, over a sum of p that is at least 2^3; the same again for p itself
                                                       L 2 * 2^-25 8 vd / 2^3 max(1, s)
      With FP16 outputs the first rounding's remainder (itself rounded, 2^-11 of 2^-11) is multiplied by the scale and
      added before the second: 2^-11 + 2 * 2^-22 in all, and one product more that may be small (3 in place of 2).
      (Short sequences carry the second rounding's remainder too; they are held to the same bound.)
      FP32 sums over the keys, 16 a matrix instruction (L/16 + 64) 2^-23 23 sum w vu
      the logits: the query's small elements (2^-25 of the row's largest), FP32 sums over D (truncating
      adders counted: 2^-23 a term) of up to 23 ku |q| each, and the exponent's argument; a logit's error
      counts twice (weight and sum)."""
    Hq, M, D = q.shape
    Hkv, L, _ = k.shape
    G = Hq // Hkv
    scale = scale or 1.0 / math.sqrt(D)
    ku = np.abs(k) if ku is None else ku
    vu = np.abs(v) if vu is None else vu
    o, bound = np.zeros(q.shape), np.zeros(q.shape)
    half = torch.finfo(out_dtype).eps / 2
    for i in range(M):
        see = visible(L, M, i, causal, window, sinks)
        if not see.any():
            continue
        for h in range(Hq):
            kk, vv, qq = k[h // G][see], v[h // G][see], q[h, i]
            s = kk @ qq * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            o[h, i] = w @ vv
            A, U = w @ np.abs(vv), 23 * (w @ vu[h // G][see])
            size = 23 * (ku[h // G][see] @ np.abs(qq)) * abs(scale)
            logit = (D + 8) * 2.0 ** -23 * size + 2.0 ** -25 * np.abs(qq).max() * abs(scale) * np.abs(kk).sum(1)
            logit = (logit + 4 * 2.0 ** -24 * (np.abs(s) + abs(s.max()))).max()
            n = len(s)
            small = n * 2.0 ** -24 * max(vd, np.abs(vv).max())  # 8 vd s is at most the largest value and more
            p = 2.0 ** -10
            if out_dtype == torch.float16:
                small, p = 1.5 * small, 2.0 ** -11 + 2.0 ** -21
            bound[h, i] = (half * np.abs(o[h, i]) + A * (p + 2 * logit) + U * (n / 16 + 64) * 2.0 ** -23
                           + small + 1e-30)
            if out_dtype == torch.float16:
                bound[h, i] += 2.0 ** -25  # its smallest numbers
    return o, bound


def units(scale_bytes, descale):
    """What one code stands for, per element."""
    return np.repeat(e4m3_value(scale_bytes), GROUP, -1) * descale


def sequences(table, lens, packed, scales, which, descale, page_size, cap=None, unit=False):
    """Per sequence [Hkv, L, D] values (or units), through the table; a page outside the pool is zeros."""
    out = []
    pages, Hkv, _, half = packed.shape
    for b, L in enumerate(lens):
        L = max(0, min(L, table.shape[1] * page_size))
        L = L if cap is None else min(L, cap)
        x = np.zeros((Hkv, L, half * 2))
        for j0 in range(0, L, page_size):
            page, n = int(table[b, j0 // page_size]), min(page_size, L - j0)
            if 0 <= page < pages:
                if unit:
                    x[:, j0:j0 + n] = units(scales[page, :, :n], descale)
                else:
                    x[:, j0:j0 + n] = values(packed[page, :, :n], scales[page, :, :n], which, descale)
        out.append(x)
    return out


def plan(cached, new, free, table, page_size, num_rows):
    """attn_page_plan's outputs by hand: (table, seq_lens, row_starts, slots, stats)."""
    table = [list(map(int, r)) for r in table]
    width = len(table[0]) if table else 0
    starts, slots, used, lost, row = [0], [-1] * num_rows, 0, 0, 0
    for b, (c, n) in enumerate(zip(cached, new)):
        c, n = max(c, 0), max(n, 0)
        have = min(-(-c // page_size), width)
        want = min(-(-(c + n) // page_size), width)
        for k in range(have, want):
            table[b][k] = free[used] if used < len(free) else -1
            used += 1
        for pos in range(c, c + n):
            k = pos // page_size
            ok = k < width and (k < have or table[b][k] >= 0)
            slot = table[b][k] * page_size + pos % page_size if k < width and table[b][k] >= 0 else -1
            if row < num_rows:
                slots[row] = slot
            if not ok or row >= num_rows:
                lost += 1
            row += 1
        starts.append(row)
    lens = [max(c, 0) + max(n, 0) for c, n in zip(cached, new)]
    return table, lens, starts, slots, [row, min(used, len(free)), lost]
