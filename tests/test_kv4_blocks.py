"""Decode over the 4-bit cache with every 16-key block visible in the output.

A random cache hides a lost block: its weight is below what the roundings of a long
sum may add up to. Here every block stands out. Key j of KV head h and sequence b lies
in block x = j / 16 and
  its key is 7 in channel (x + h + b) mod R, R the grouped rows, and 0 elsewhere; row r
  of the group has 8 in channel r alone, so with a logit scale of 1 its logits are 56
  for the blocks with that residue and 0 for all others, whose weight e^-56 is nothing;
  its value is 7 in two channels that depend on x (modulo two primes, one in each half
  of the row), h and b, and 0 elsewhere.
So o[r, c] = 7 (keys of row r's blocks with channel c) / (keys of row r's blocks), and a
block that is lost, taken twice or read in another's place changes a channel that few
blocks share.

The bound. Logits, codes and scales are small whole numbers or powers of two, exact in
all products and sums (numerators stay below 2^24 units; what was summed before a maximum
of 56 appeared is rescaled by e^-56, which leaves less than 2^-60 of it). All logits that
count are equal, and the maximum is one of them, so every key that counts has the same
probability 2^3 (1 + d): 56 log2(e) lies between 64 and 128, where half a step is 2^-18,
so |d| <= 2^-18 ln 2 and 2^-22 more of the exponential itself. In FP16 that is 2^3; the
sum of the weights adds it as it is, in at most L / 8 additions of 2^-24 each to a lane
and ten more of lanes, warps and parts. With one division and product:
  |o| (eps / 2 + L 2^-27 + 2^-17) + 2^-24.
Segments left whole with FP16 outputs multiply what the rounding to FP16 left, 2^3 d, as
well. Their numerators are then no whole numbers: two matrix instructions per 16 keys add
to a sum of codes of at most 15 a key, and as many to 8 times the weights, each off by up
to 2^-23 of 15 + 8 units, and 64 more additions join what lanes and warps have:
  23 (L / 8 + 64) 2^-23 more. (2^-24, as for the others, was asked of them at first: the
sequence of 149 keys was 10 2^-24 off in channels whose mean is 0.)"""
import numpy as np
import pytest
import torch

import kv4_reference as ref
import streaming_attention_gb300 as sa

BF16, FP16 = torch.bfloat16, torch.float16
PRIMES = {32: (13, 11), 64: (31, 29), 128: (61, 59)}

#: lens, Hq, Hkv, M, D, page size, dtype, causal, window, sinks
LONG = [20000 + 7, 300, 16]
MANY = [1 + 389 * b % 2999 for b in range(64)]
MOST = [1 + 611 * b % 1301 for b in range(500)]
WHOLE = [1 + 37 * b % 900 for b in range(40)]
SHAPES = [
    ([131072], 32, 8, 1, 128, 256, BF16, True, 0, 0),       # four warps a team, many parts of a segment
    (LONG, 8, 1, 1, 128, 16, BF16, True, 0, 0),
    ([9000, 4097, 8192], 16, 8, 1, 128, 64, FP16, True, 0, 0),
    ([7001, 6000], 8, 2, 3, 64, 32, BF16, True, 2222, 40),
    ([12345, 1, 0, 5000], 4, 1, 1, 32, 128, FP16, False, 0, 0),
    ([16384], 8, 2, 4, 128, 128, FP16, True, 0, 0),         # 16 rows, two blocks of 8
    (MANY, 32, 8, 1, 128, 16, BF16, True, 0, 0),            # single warps as teams
    (MANY, 16, 8, 2, 64, 64, FP16, True, 1000, 33),
    (MANY, 16, 8, 1, 32, 16, BF16, True, 0, 0),
    (MOST, 8, 4, 1, 64, 32, BF16, True, 0, 0),              # more segments than teams
    (MOST, 8, 4, 3, 128, 16, FP16, True, 300, 5),
    (WHOLE, 8, 2, 2, 128, 16, BF16, True, 0, 0),            # segments left whole
    (WHOLE, 4, 2, 1, 32, 64, FP16, False, 100, 17),
]


def channels(x, h, b, D):
    m1, m2 = PRIMES[D]
    return (x + 5 * h + 3 * b) % m1, D // 2 + (x + 7 * h + b) % m2


def expected(L, h, b, R, M, D, causal, window, sinks, times=None):
    """o [R, D]; times: how often each block is taken (1)."""
    o = np.zeros((R, D))
    x = np.arange(L) // 16
    c1, c2 = channels(x, h, b, D)
    w = np.ones(L) if times is None else times[x]
    for r in range(R):
        see = ref.visible(L, M, r % M, causal, window, sinks)
        mine = see & ((x + h + b) % R == r)
        mine = mine if mine.any() else see  # none of them: all logits are 0
        total = w[mine].sum()
        if total > 0:
            o[r] = 7 * (np.bincount(c1[mine], w[mine], D) + np.bincount(c2[mine], w[mine], D)) / total
    return o


def bound(o, L, dtype, whole):
    sums = 23 * (L / 8 + 64) * 2.0 ** -23 if whole and dtype == FP16 else 0.0
    return np.abs(o) * (torch.finfo(dtype).eps / 2 + L * 2.0 ** -27 + 2.0 ** -17) + 2.0 ** -24 + sums


@pytest.mark.parametrize("n", range(len(SHAPES)))
def test_every_block_exceeds_the_bound_when_lost_doubled_or_misplaced(n):
    """What the GPU test would see of such faults, planted in the expected outputs: of every block of the longest and of
    a middling sequence, one after the other (every 7th where there are many)."""
    lens, Hq, Hkv, M, D, ps, dtype, causal, window, sinks = SHAPES[n]
    R, h = Hq // Hkv * M, Hkv - 1
    for b in {int(np.argmax(lens)), len(lens) // 2}:
        L = lens[b]
        want = expected(L, h, b, R, M, D, causal, window, sinks)
        seen = np.zeros(L, bool)
        for i in range(M):
            seen |= ref.visible(L, M, i, causal, window, sinks)
        blocks = -(-L // 16)
        step = 1 if blocks < 300 else 7 if blocks < 2000 else 97
        for x in sorted({*range(0, blocks, step), blocks - 1} if blocks else ()):
            if not seen[16 * x:16 * x + 16].any():
                continue
            for times in (0.0, 2.0):
                t = np.ones(blocks)
                t[x] = times
                got = expected(L, h, b, R, M, D, causal, window, sinks, t)
                single = ((np.arange(blocks) + h + b) % R == (x + h + b) % R).sum() == 1 or L < 16 * R
                assert single or (np.abs(got - want) > bound(want, L, dtype, max(lens) <= 1024)).any(), (b, x, times)
            if x + 1 < blocks and 16 * x + 32 <= L and seen[16 * x:16 * x + 32].all():  # the next one in its place
                t = np.ones(blocks)
                t[x], t[x + 1] = 0, 2
                got = expected(L, h, b, R, M, D, causal, window, sinks, t)
                assert L < 16 * R or (np.abs(got - want) > bound(want, L, dtype, max(lens) <= 1024)).any(), (b, x, "misplaced")


def cache_of_blocks(lens, Hkv, R, D, ps, device):
    """The cache above on shuffled pages; what no sequence holds has a scale of NaN."""
    rng = np.random.default_rng(len(lens) + D)
    need = [-(-L // ps) for L in lens]
    pages = sum(need) + 2
    ids = rng.permutation(pages)
    table = np.zeros((len(lens), max(max(need), 1)), np.int32)
    codes = [torch.full((pages, Hkv, ps, D // 2), 0x88, dtype=torch.uint8) for _ in "kv"]
    scale = torch.full((pages, Hkv, ps, D // 32), 0x7F, dtype=torch.uint8)
    h = np.arange(Hkv)[:, None]
    at = 0
    for b, L in enumerate(lens):
        mine = ids[at:at + need[b]]
        table[b, :need[b]] = mine
        at += need[b]
        n = need[b] * ps // 16  # blocks of its pages
        x = np.arange(n)[None]
        rows = {w: np.full((Hkv, n, D), 8, np.uint8) for w in "kv"}
        np.put_along_axis(rows["k"], ((x + h + b) % R)[..., None], 15, -1)
        for c in channels(x, h, b, D):
            np.put_along_axis(rows["v"], c[..., None], 15, -1)
        for pool, w in zip(codes, "kv"):
            y = torch.from_numpy(ref.pack(rows[w], w)).repeat_interleave(16, 1)  # [Hkv, keys, D / 2]
            pool[mine] = y.view(Hkv, need[b], ps, D // 2).transpose(0, 1)
        s = torch.full((Hkv, need[b] * ps, D // 32), 0x38, dtype=torch.uint8)  # 1
        s[:, L:] = 0x7F
        scale[mine] = s.view(Hkv, need[b], ps, D // 32).transpose(0, 1)
    s = scale.to(device).view(torch.float8_e4m3fn)
    return (codes[0].to(device), s, codes[1].to(device), s.clone()), table


@pytest.mark.gpu
@pytest.mark.parametrize("n", range(len(SHAPES)))
def test_every_block_is_read_once(n):
    lens, Hq, Hkv, M, D, ps, dtype, causal, window, sinks = SHAPES[n]
    dev, G = "cuda:0", Hq // Hkv
    R = G * M
    cache, table = cache_of_blocks(lens, Hkv, R, D, ps, dev)
    q = torch.zeros(len(lens), Hkv, R, D, dtype=dtype)
    q[:, :, range(R), range(R)] = 8
    q = q.view(len(lens), Hq, M, D).to(dev)
    o = torch.full_like(q, float("nan"))
    i32 = dict(dtype=torch.int32, device=dev)
    sa.attn_decode_paged_kv4(q, *cache, torch.from_numpy(table).to(dev), torch.tensor(lens, **i32), o, max(lens), causal,
                             window, sinks, 1.0)
    torch.cuda.synchronize()
    got = ref.f64(o).reshape(len(lens), Hkv, R, D)
    for b, L in enumerate(lens):
        for h in range(Hkv):
            want = expected(L, h, b, R, M, D, causal, window, sinks)
            off = np.abs(got[b, h] - want) > bound(want, L, dtype, max(lens) <= 1024)
            assert np.isfinite(got[b, h]).all() and not off.any(), (b, h, np.argwhere(off)[:5])
