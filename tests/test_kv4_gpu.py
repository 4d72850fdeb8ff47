"""The 4-bit paged cache on the GPU against its definition in 64 bits: the write
into it (exact), the read back (exact), the tables of a step (exact), decode
attention over it (within a bound derived per element in kv4_reference), and a
serving loop of them together."""
import threading

import numpy as np
import pytest
import torch

import kv4_reference as ref
import streaming_attention_gb300 as sa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP16 = torch.bfloat16, torch.float16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def model_rows(rng, shape, which):
    """Keys with a few strong channels, values around half a unit."""
    x = rng.normal(size=shape)
    return x * (0.7 + 2.0 * (np.arange(shape[-1]) % 19 == 3)) if which == "k" else x * 0.5


def make_cache(rng, pages, Hkv, ps, D, kd=1.0, vd=0.125):
    """Pools filled with quantized rows (by the reference): device tensors and numpy."""
    dev, host = [], []
    for which, d in (("k", kd), ("v", vd)):
        codes, byte, _ = ref.quantize(model_rows(rng, (pages, Hkv, ps, D), which), d)
        packed = ref.pack(codes, which)
        host += [packed, byte]
        dev += [torch.from_numpy(packed).to(DEV), torch.from_numpy(byte).to(DEV).view(torch.float8_e4m3fn)]
    return dev, host


def make_table(rng, lens, ps, pages, width=None):
    need = [-(-n // ps) for n in lens]
    width = width or max(max(need), 1)
    ids = rng.permutation(pages)
    table, at = np.zeros((len(lens), width), np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table


def run_decode(q, dev, table, lens, cap, causal=True, window=0, sinks=0, scale=0.0, kd=1.0, vd=0.125, ws=True):
    B, Hq, M, D = q.shape
    o = torch.full_like(q, float("nan"))
    work = None
    if ws:
        n = sa.attn_decode_paged_kv4_workspace_bytes(B, Hq, dev[0].shape[1], M, D, dev[0].shape[2], table.shape[1], cap,
                                                     causal, window, sinks)
        room = torch.full((n + 4096,), 255, dtype=torch.uint8, device=DEV)  # exactly n bytes, watched behind
        work = room[:n]
    sa.attn_decode_paged_kv4(q, *dev, i32(table), i32(lens), o, cap, causal, window, sinks, scale, kd, vd, work)
    torch.cuda.synchronize()
    assert not ws or bool((room[n:] == 255).all()), "written behind the workspace"
    return o


def check_decode(o, q, host, table, lens, cap, causal=True, window=0, sinks=0, scale=0.0, kd=1.0, vd=0.125):
    ps = host[0].shape[2]
    ks = ref.sequences(table, lens, host[0], host[1], "k", kd, ps, cap)
    vs = ref.sequences(table, lens, host[2], host[3], "v", vd, ps, cap)
    ku = ref.sequences(table, lens, host[0], host[1], "k", kd, ps, cap, unit=True)
    vu = ref.sequences(table, lens, host[2], host[3], "v", vd, ps, cap, unit=True)
    got, qq = ref.f64(o), ref.f64(q)
    for b in range(len(lens)):
        want, bound = ref.attention(qq[b], ks[b], vs[b], causal, window, sinks, scale, q.dtype, ku[b], vu[b], vd)
        err = np.abs(got[b] - want)
        worst = (err / np.maximum(bound, 1e-300)).max() if err.size else 0
        assert np.isfinite(got[b]).all() and (err <= bound).all(), f"sequence {b}: {worst:.3g} of the bound"


def case(seed, lens, Hq, Hkv, M, D, ps, dtype, spare=3, width=None):
    rng = np.random.default_rng(seed)
    pages = sum(-(-n // ps) for n in lens) + spare
    dev, host = make_cache(rng, pages, Hkv, ps, D)
    table = make_table(rng, lens, ps, pages, width)
    q = torch.from_numpy(rng.normal(size=(len(lens), Hq, M, D))).to(dtype).to(DEV)
    return q, dev, host, table


# ---------------------------------------------------------------------------
# append and gather
# ---------------------------------------------------------------------------
def border_rows(D, dtype, descale):
    """Rows whose elements lie on and next to the borders between codes and whose maxima lie on and
    next to the borders between scales."""
    rows = []
    for s in (1.0, 1.125, 0.8125, 2.0 ** -9, 3 * 2.0 ** -9, 448.0, 7 * 2.0 ** -7):
        x = np.zeros(D)
        ties = np.array([(n + 0.5) * s for n in range(-8, 8)])
        t = torch.from_numpy(ties * descale).to(dtype)
        up = (t.view(torch.int16) + 1).view(dtype)
        down = (t.view(torch.int16) - 1).view(dtype)
        x[:16] = t.double().numpy()
        x[16:32] = np.where(np.arange(16) % 2 == 0, up.double().numpy(), down.double().numpy())
        rows.append(x)
    for k in range(9):  # maxima 7.5 times a border between two scales, and its neighbours
        top = torch.tensor(7.5 * (1 + (2 * k + 1) / 16) * 2.0 ** -3 * descale).to(dtype)
        for step in (-1, 0, 1):
            x = np.full(D, 0.01 * descale)
            x[D - 1] = float((top.view(torch.int16) + step).view(dtype))
            rows.append(x)
    rows.append(np.zeros(D))
    rows.append(np.full(D, 2.0 ** -12 * descale))  # its scale rounds to zero
    rows.append(np.full(D, -6000.0 * descale))     # behind the largest scale: saturates
    return np.stack(rows)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("kd,vd", [(1.0, 0.125), (0.0625, 4.0)])
def test_append_and_gather_are_exact(D, dtype, kd, vd):
    rng = np.random.default_rng(D)
    Hkv, ps, pages, T = 3, 16, 9, 83
    k = model_rows(rng, (T, Hkv, D), "k")
    v = model_rows(rng, (T, Hkv, D), "v")
    bk, bv = border_rows(D, dtype, kd), border_rows(D, dtype, vd)
    k[:len(bk), 1], v[:len(bv), 2] = bk, bv
    # K and V as parts of a wider projection's output
    qkv = torch.zeros(T, 5 + 2 * Hkv, D, dtype=dtype, device=DEV)
    qkv[:, 5:5 + Hkv] = torch.from_numpy(k)
    qkv[:, 5 + Hkv:] = torch.from_numpy(v)
    kk, vv = qkv[:, 5:5 + Hkv], qkv[:, 5 + Hkv:]
    slots = rng.permutation(pages * ps)[:T].astype(np.int32)
    slots[70], slots[71], slots[72] = -1, pages * ps, 2 ** 31 - 1  # skipped rows
    dev, host = make_cache(rng, pages, Hkv, ps, D)
    sa.attn_kv4_append(kk, vv, torch.from_numpy(slots).to(DEV), *dev, kd, vd)
    torch.cuda.synchronize()
    for x, which, d, n in ((ref.f64(kk), "k", kd, 0), (ref.f64(vv), "v", vd, 2)):
        codes, byte, val = ref.quantize(x, d)
        packed, scales = host[n].copy(), host[n + 1].copy()
        for t, slot in enumerate(slots):
            if 0 <= slot < pages * ps:
                packed[slot // ps, :, slot % ps] = ref.pack(codes[t], which)
                scales[slot // ps, :, slot % ps] = byte[t]
        assert np.array_equal(bytes_np(dev[n]), packed), which
        assert np.array_equal(bytes_np(dev[n + 1]), scales), which
    # read back: sequences over shuffled pages, one with a page outside the pool, one empty
    table = np.array([[4, 1, 8], [7, -1, 0], [2, pages, 3], [5, 6, 6]], np.int32)
    lens = [41, 48, 30, 0]
    out_k = torch.full((4, Hkv, 50, D), float("nan"), dtype=dtype, device=DEV)
    out_v = out_k.clone()
    sa.attn_kv4_gather(*dev, i32(table), i32(lens), out_k, out_v, kd, vd)
    torch.cuda.synchronize()
    for out, which, d, n in ((out_k, "k", kd, 0), (out_v, "v", vd, 2)):
        seqs = ref.sequences(table, lens, bytes_np(dev[n]), bytes_np(dev[n + 1]), which, d, ps)
        for b, L in enumerate(lens):
            want = np.zeros((Hkv, 50, D))
            want[:, :L] = seqs[b]
            assert np.array_equal(ref.f64(out[b]), want), (which, b)


def bytes_np(t):
    return t.view(torch.uint8).cpu().numpy()


def test_gather_lengths_past_the_table_and_short_outputs():
    rng = np.random.default_rng(8)
    dev, host = make_cache(rng, 6, 2, 32, 64)
    table = np.array([[3, 1], [5, 0]], np.int32)
    for N, lens in ((100, [1000, -4]), (17, [64, 20]), (1, [1, 64])):
        k = torch.full((2, 2, N, 64), float("nan"), dtype=BF16, device=DEV)
        v = k.clone()
        sa.attn_kv4_gather(*dev, i32(table), i32(lens), k, v, 1.0, 0.125)
        torch.cuda.synchronize()
        ks = ref.sequences(table, lens, host[0], host[1], "k", 1.0, 32)
        for b in range(2):
            want = np.zeros((2, N, 64))
            n = min(N, ks[b].shape[1])
            want[:, :n] = ks[b][:, :n]
            assert np.array_equal(ref.f64(k[b]), want)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dtype,vd", [(BF16, 0.125), (FP16, 0.125), (FP16, 2.0 ** -20)])
def test_gather_of_nothing_is_zeros_in_every_bit(D, dtype, vd):
    """Rows behind the end and rows on pages outside the pool: no negative zeros."""
    dev, _ = make_cache(np.random.default_rng(3), 4, 2, 16, D)
    k = torch.full((3, 2, 70, D), float("nan"), dtype=dtype, device=DEV)
    v = k.clone()
    table = i32([[1, -1, 0, 2, 3], [4, 2 ** 31 - 1, -2 ** 31, 1, 1], [0, 0, 0, 0, 0]])
    sa.attn_kv4_gather(*dev, table, i32([40, 48, -1]), k, v, 1.0, vd)
    torch.cuda.synchronize()
    for x in (k.view(torch.int16), v.view(torch.int16)):
        assert not x[0, :, 16:32].any() and not x[0, :, 40:].any() and not x[1:].any()
        assert x[0, :, :16].any() and x[0, :, 32:40].any()


def test_append_one_row_of_one_head_any_stride():
    """A single row's stride is not read; a single head's neither."""
    rng = np.random.default_rng(9)
    dev, _ = make_cache(rng, 2, 1, 16, 32)
    x = torch.from_numpy(rng.normal(size=(1, 1, 32))).to(FP16).to(DEV)
    k = torch.as_strided(x, (1, 1, 32), (3, 5, 1))
    sa.attn_kv4_append(k, x, i32([17]), *dev)
    torch.cuda.synchronize()
    codes, byte, _ = ref.quantize(ref.f64(x), 1.0)
    assert np.array_equal(bytes_np(dev[0])[1, 0, 1], ref.pack(codes, "k")[0, 0])
    assert np.array_equal(bytes_np(dev[3])[1, 0, 1], byte[0, 0])


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("descale", [2.0 ** -64, 1.0, 2.0 ** 64])
def test_append_of_every_magnitude(dtype, descale):
    """Groups whose largest element is anything from the type's smallest number to its largest: exact."""
    rng = np.random.default_rng(96)
    lo, hi = (-149, 128) if dtype == BF16 else (-24, 16)
    T, D = hi - lo + 3, 64
    x = torch.from_numpy(np.ldexp(rng.uniform(-1, 1, (T, 1, D)), (lo + np.arange(T) - 1)[:, None, None]))
    x[-1] = torch.finfo(dtype).max
    x[-1, 0, ::3] *= -1
    x = x.to(dtype)
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    dev = sa.kv4_cache(-(-T // 16), 1, 16, D)
    sa.attn_kv4_append(x.to(DEV), x.to(DEV), i32(list(range(T))), *dev, descale, descale)
    torch.cuda.synchronize()
    codes, byte, _ = ref.quantize(ref.f64(x), descale)
    for n, which in ((0, "k"), (2, "v")):
        assert np.array_equal(bytes_np(dev[n]).reshape(-1, 1, D // 2)[:T], ref.pack(codes, which))
        assert np.array_equal(bytes_np(dev[n + 1]).reshape(-1, 1, D // 32)[:T], byte)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_groups_that_are_not_finite(D, dtype, bad):
    """One such element makes its group NaN, in the cache, read back, and in the rows that see it; other groups, rows and
    sequences, and rows whose window is past it, are as before. Rows without a slot may hold anything."""
    rng = np.random.default_rng(95)
    Hkv, ps, T, L = 2, 16, 200, 90  # two sequences of L keys, and rows without a slot
    x = {w: torch.from_numpy(model_rows(rng, (T, Hkv, D), w)).to(dtype) for w in "kv"}
    table = np.array([[3, 1, 4, 0, 9, 2], [6, 5, 11, 7, 10, 8]], np.int32)
    slots = [int(table[j // L, j % L // ps]) * ps + j % L % ps for j in range(2 * L)] + [-1] * (T - 2 * L)
    q = torch.from_numpy(rng.normal(size=(2, 2 * Hkv, 1, D))).to(dtype).to(DEV)

    def step(window):
        dev = sa.kv4_cache(12, Hkv, ps, D)
        sa.attn_kv4_append(x["k"].to(DEV), x["v"].to(DEV), i32(slots), *dev, 1.0, 0.125)
        out = [torch.empty(2, Hkv, L, D, dtype=dtype, device=DEV) for _ in range(2)]
        sa.attn_kv4_gather(*dev, i32(table), i32([L, L]), *out, 1.0, 0.125)
        return [t.cpu() for t in out], run_decode(q, dev, table, [L, L], L, True, window).cpu()

    clean, o_all = step(0)
    _, o_late = step(20)
    for w, at in (("k", (40, 1, D - 1)), ("v", (L + 3, 0, 0))):  # a key of the first sequence, a value of the second
        x[w][at] = bad
        x[w][2 * L:] = bad
    got, o = step(0)
    for n, (b, h, j, g) in enumerate(((0, 1, 40, D // 32 - 1), (1, 0, 3, 0))):
        hit = torch.zeros(2, Hkv, L, D, dtype=torch.bool)
        hit[b, h, j, 32 * g:32 * g + 32] = True
        assert got[n][hit].isnan().all() and torch.equal(got[n][~hit], clean[n][~hit])
    hit = torch.zeros(2, 2 * Hkv, 1, D, dtype=torch.bool)
    hit[0, 2:] = True
    hit[1, :2, :, :32] = True
    assert o[hit].isnan().all() and torch.equal(o[~hit], o_all[~hit])
    assert torch.equal(step(20)[1], o_late)


# ---------------------------------------------------------------------------
# tables of a step
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("B,ps,most,pad,short", [
    (1, 16, 40, 0, 0), (7, 16, 100, 5, 0), (64, 32, 2, 0, 0), (1000, 16, 60, 33, 0), (1024, 64, 9, 1, 0),
    (1025, 16, 3, 0, 0), (3000, 128, 300, 64, 0), (20, 16, 200, 0, 30), (20, 7, 50, -90, 4), (5, 1, 9, 2, 0)])
def test_page_plan(B, ps, most, pad, short):
    """pad < 0: slot_map too short for the step; short: pages missing from the free list."""
    rng = np.random.default_rng(B)
    cached = rng.integers(0, 5 * ps, B)
    cached[rng.random(B) < 0.3] = 0
    new = rng.integers(0, most + 1, B)
    cached[0], new[0] = ps, 1  # a full page, then one key more
    if B > 2:
        cached[1], new[1], cached[2], new[2] = -3, -1, 0, ps
    width = int(max(-(-(cached + new) // ps)))
    if short:
        width = max(width - 2, 1)  # some requests outgrow the table
    have = np.minimum(-(-np.maximum(cached, 0) // ps), width)
    need = int((np.minimum(-(-(np.maximum(cached, 0) + np.maximum(new, 0)) // ps), width) - have).sum())
    ids = rng.permutation(int(have.sum()) + need + 7)
    table, at = np.full((B, width), -7), 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    free = ids[at:at + max(need - short, 0)]
    T = max(int(np.maximum(new, 0).sum()) + pad, 0)
    want = ref.plan(cached.tolist(), new.tolist(), free.tolist(), table, ps, T)
    d_table = i32(table)
    out = [torch.full((n,), -9, dtype=torch.int32, device=DEV) for n in (B, B + 1, T, 3)]
    sa.attn_page_plan(i32(cached), i32(new), i32(free), d_table, *out, ps)
    torch.cuda.synchronize()
    assert d_table.tolist() == want[0]
    for got, w in zip(out, want[1:]):
        assert got.tolist() == w


@pytest.mark.parametrize("B,ps,most,pad,short", [
    (2, 16, 3, 0, 0), (5, 1, 4, 3, 2), (31, 7, 40, -20, 0), (256, 16, 2, 0, 0), (257, 16, 40, 9, 0), (512, 32, 70, 0, 9),
    (513, 16, 3, 1, 0), (2047, 16, 50, 0, 100), (2049, 128, 200, -3000, 5)])
def test_page_plan_counts_every_row_without_a_slot(B, ps, most, pad, short):
    """Entries that name no page, in the table of the cached keys (as a step that ran out of pages leaves them) and in the
    free list, and pages whose slots pass 32 bits, in part or wholly: their rows have no slot and are counted."""
    rng = np.random.default_rng(B + 1)
    cached, new = rng.integers(0, 4 * ps + 1, B), rng.integers(0, most + 1, B)
    cached[0], new[0] = ps - 1 if ps > 1 else 1, 3
    width = int(max(-(-(cached + new) // ps)))
    have = -(-cached // ps)
    need = int((-(-(cached + new) // ps) - have).sum())
    last = (2 ** 31 - 1) // ps  # its slots pass 32 bits behind the first few
    odd = [-1, -2 ** 31, -5, last, min(last + 1, 2 ** 31 - 1), 2 ** 31 - 1]
    table, free = rng.integers(0, 1000, (B, width)), rng.integers(0, 1000, max(need - short, 0))
    for x in (table, free):
        x[rng.random(x.shape) < 0.3] = 0  # (the same page twice is no matter here)
        at = rng.random(x.shape) < 0.3
        x[at] = rng.choice(odd, int(at.sum()))
    table[0] = -1
    T = max(int(new.sum()) + pad, 0)
    want = ref.plan(cached.tolist(), new.tolist(), free.tolist(), table, ps, T)
    want[3][:] = [x if x < 2 ** 31 else -1 for x in want[3]]
    want[4][2] = int(new.sum()) - sum(x >= 0 for x in want[3])
    assert want[4][2] > 0
    out = [torch.full((n,), -9, dtype=torch.int32, device=DEV) for n in (B, B + 1, T, 3)]
    d_table = i32(table)
    sa.attn_page_plan(i32(cached), i32(new), i32(free), d_table, *out, ps)
    torch.cuda.synchronize()
    assert d_table.tolist() == want[0]
    for got, w in zip(out, want[1:]):
        assert got.tolist() == w


def test_page_plan_after_a_step_that_ran_out():
    """15 keys, 3 more, no page left: the table's new entry is -1. The next step's rows on it have no slot either, and
    are counted; rows on a page of their own have one."""
    table, lens, starts, slots, stats = i32([[4, -7, -7]]), i32([0]), i32([0, 0]), i32([9] * 3), i32([9] * 3)
    sa.attn_page_plan(i32([15]), i32([3]), i32([]), table, lens, starts, slots, stats, 16)
    assert (table.tolist(), slots.tolist(), stats.tolist()) == ([[4, -1, -7]], [79, -1, -1], [3, 0, 2])
    sa.attn_page_plan(lens.clone(), i32([3]), i32([7, 8]), table, lens, starts, slots, stats, 16)
    assert (table.tolist(), slots.tolist(), stats.tolist()) == ([[4, -1, -7]], [-1, -1, -1], [3, 0, 3])
    slots = i32([9] * 12)
    sa.attn_page_plan(lens.clone(), i32([12]), i32([7, 8]), table, lens, starts, slots, stats, 16)
    assert (table.tolist(), slots.tolist(), stats.tolist()) == ([[4, -1, 7]], [-1] * 11 + [112], [12, 1, 11])


def test_page_plan_of_nothing_and_of_huge_lengths():
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    starts, slots, stats = i32([-9]), i32([5, 5]), i32([9, 9, 9])
    sa.attn_page_plan(e, e.clone(), e.clone(), torch.empty((0, 4), dtype=torch.int32, device=DEV), e.clone(), starts,
                      slots, stats, 16)
    torch.cuda.synchronize()
    assert starts.tolist() == [0] and slots.tolist() == [-1, -1] and stats.tolist() == [0, 0, 0]
    big = 2 ** 31 - 1  # sums of lengths pass 32 bits: saturated, nothing out of range is touched
    table, lens, starts = i32([[-7, -7]] * 3), i32([0] * 3), i32([0] * 4)
    sa.attn_page_plan(i32([big, 5, 0]), i32([big, 3, big]), i32([4, 2]), table, lens, starts, slots, stats, 16)
    torch.cuda.synchronize()
    assert lens.tolist() == [big, 8, big] and starts.tolist() == [0, big, big, big]
    assert slots.tolist() == [-1, -1] and stats.tolist() == [big, 2, big]
    assert table.tolist() == [[-7, -7], [-7, -7], [4, 2]]


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 384])
@pytest.mark.parametrize("causal,window,sinks", [(True, 0, 0), (True, 300, 0), (True, 130, 5), (False, 0, 0),
                                                 (False, 200, 70)])
def test_decode_ragged(D, ps, causal, window, sinks):
    lens = [1000, 1, 0, 1024, 517, 15, 16, 17]
    dtype = FP16 if ps in (32, 128) else BF16
    q, dev, host, table = case(D + ps, lens, 8, 2, 1, D, ps, dtype)
    o = run_decode(q, dev, table, lens, 1024, causal, window, sinks)
    check_decode(o, q, host, table, lens, 1024, causal, window, sinks)
    assert torch.all(o[2] == 0)


@pytest.mark.parametrize("D,Hq,Hkv,M", [(128, 3, 3, 1), (128, 8, 1, 1), (64, 9, 1, 1), (128, 16, 2, 2), (32, 4, 4, 8),
                                        (128, 4, 2, 9), (128, 40, 1, 1), (64, 6, 2, 7), (128, 14, 2, 5)])
@pytest.mark.parametrize("causal,window,sinks", [(True, 0, 0), (True, 40, 3), (False, 0, 0)])
def test_decode_grouped_and_speculative_rows(D, Hq, Hkv, M, causal, window, sinks):
    """Rows per KV head from 1 to 40; sequences shorter than M leave rows with no visible key."""
    lens = [301, 3, 640, 70, 0]
    q, dev, host, table = case(Hq * M, lens, Hq, Hkv, M, D, 32, FP16 if M % 2 else BF16)
    o = run_decode(q, dev, table, lens, 640, causal, window, sinks)
    check_decode(o, q, host, table, lens, 640, causal, window, sinks)
    if causal and M > 3:
        assert torch.all(o[1, :, :M - 3] == 0)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 200), (63, 64), (64, 65), (200, 16), (5000, 9), (17, 900),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (40, -3), (-1, 5)])
def test_decode_windows_and_sinks(window, sinks):
    """Windows that start inside, at and behind the sinks; sinks and windows longer than the sequence."""
    lens = [900, 64, 65, 128, 1, 333]
    q, dev, host, table = case(77, lens, 4, 2, 2, 64, 16, BF16)
    o = run_decode(q, dev, table, lens, 900, True, window, sinks)
    check_decode(o, q, host, table, lens, 900, True, window, max(sinks, 0))


def test_decode_long_context_splits_and_one_split():
    for lens, Hq, Hkv, M, window in (([20000], 4, 1, 1, 0), ([9000, 4097], 16, 8, 1, 0), ([300] * 90, 8, 8, 1, 0),
                                     ([7001], 32, 2, 1, 2222)):
        q, dev, host, table = case(len(lens), lens, Hq, Hkv, M, 128, 16, BF16)
        o = run_decode(q, dev, table, lens, max(lens), True, window, 4)
        check_decode(o, q, host, table, lens, max(lens), True, window, 4)


@pytest.mark.parametrize("scale", [0.3, -0.05, 2.0])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_decode_scales_and_workspace_of_the_library(scale, dtype):
    lens = [500, 7, 333]
    q, dev, host, table = case(5, lens, 8, 2, 2, 128, 64, dtype)
    o = run_decode(q, dev, table, lens, 500, True, 100, 3, scale, ws=False)
    check_decode(o, q, host, table, lens, 500, True, 100, 3, scale)


def test_decode_query_magnitudes():
    """Rows of very different size: the largest element of a row near 1e30, 1e-30 and 6e4, a zero row, and
    a row whose small elements fall below FP16's range relative to its largest."""
    lens = [200]
    q, dev, host, table = case(6, lens, 6, 1, 1, 64, 16, BF16)
    q[0, 0] *= 1e30
    q[0, 1] *= 1e-30
    q[0, 2] = 0
    q[0, 3, 0, 1:] *= 1e-6
    q[0, 4] *= 3e4
    qs = q.clone()
    # per-row scales that bring the logits back to order 1, one call each
    for h, scale in ((0, 1e-31), (1, 1e29), (2, 0.1), (3, 0.1), (4, 1e-5), (5, 0.1)):
        o = run_decode(qs, dev, table, lens, 200, True, 0, 0, scale)
        ks = ref.sequences(table, lens, host[0], host[1], "k", 1.0, 16)
        vs = ref.sequences(table, lens, host[2], host[3], "v", 0.125, 16)
        ku = ref.sequences(table, lens, host[0], host[1], "k", 1.0, 16, unit=True)
        vu = ref.sequences(table, lens, host[2], host[3], "v", 0.125, 16, unit=True)
        want, bound = ref.attention(ref.f64(q)[0, h:h + 1], ks[0], vs[0], True, 0, 0, scale, BF16, ku[0], vu[0])
        assert (np.abs(ref.f64(o)[0, h:h + 1] - want) <= bound).all(), h


def test_decode_rising_and_constant_logits():
    """A maximum that rises in every tile (each one rescales the state), and keys that are all equal."""
    rng = np.random.default_rng(12)
    L, D, ps = 1500, 64, 16
    pages = -(-L // ps)
    k = rng.normal(size=(pages, 1, ps, D)) * 0.1
    k[..., 0] = (np.arange(pages * ps).reshape(pages, 1, ps) / L - 0.5) * 30
    v = rng.normal(size=(pages, 1, ps, D))
    dev, host = [], []
    for x, which, d in ((k, "k", 1.0), (v, "v", 0.125)):
        codes, byte, _ = ref.quantize(x, d)
        host += [ref.pack(codes, which), byte]
        dev += [torch.from_numpy(host[-2]).to(DEV), torch.from_numpy(byte).to(DEV).view(torch.float8_e4m3fn)]
    table = np.arange(pages, dtype=np.int32)[None]
    q = torch.zeros(1, 2, 1, D, dtype=BF16, device=DEV)
    q[0, 0, 0, 0] = 16.0
    q[0, 1, 0, 0] = -16.0
    o = run_decode(q, dev, table, [L], L)
    check_decode(o, q, host, table, [L], L)
    q.zero_()  # equal logits: the mean of the values
    o = run_decode(q, dev, table, [L], L)
    check_decode(o, q, host, table, [L], L)


def faint_tail(L, mass, mag, vd, D, dtype, seed):
    """A first key that takes `mass` of the probability and has hardly a value, and a tail of L - 1 keys that share the
    rest: what an attention sink in front of a long context looks like. (q [1, 1, 1, D], pools, host, o, bound).
    The bound counts the output's rounding, both of a probability's (relative to A = sum w |v|), the logits (as
    kv4_reference does), what is lost where probabilities and their products with a scale are FP16's small numbers (at
    most 2^-25 each, times a code of at most 8, the factor and a scale, over a row sum of at least 2^3; one product
    more with FP16 outputs), and the sums of at most 256 blocks of 16 keys to a warp and 64 joins."""
    rng = np.random.default_rng(seed)
    x = np.zeros((L, 1, D))
    x[1:, 0, 0] = rng.normal(size=L - 1) * 1.5
    x[0, 0, 1] = 7
    v = rng.normal(size=(L, 1, D)) * mag + mag / 2
    v[0] *= 0.01
    host = []
    for y, which, d in ((x, "k", 1.0), (v, "v", vd)):
        codes, byte, val = ref.quantize(y, d)
        host += [ref.pack(codes, which), byte, val[:, 0]]
    k, val, unit = host[2], host[5], ref.units(host[4], vd)[:, 0]
    tail = np.log(np.exp(k[1:, 0]).sum())
    q = torch.zeros(1, 1, 1, D)
    q[..., 0], q[..., 1] = 1, (tail + np.log(mass / (1 - mass))) / k[0, 1]
    q = q.to(dtype)
    logit = k @ ref.f64(q)[0, 0, 0]
    w = np.exp(logit - logit.max())
    w /= w.sum()
    o, A, U = w @ val, w @ np.abs(val), 23 * (w @ unit)
    ku, qa = ref.units(host[1], 1.0)[:, 0], np.abs(ref.f64(q)[0, 0, 0])
    off = ((D + 8) * 2.0 ** -23 * 23 * (ku @ qa) + 2.0 ** -25 * qa.max() * np.abs(k).sum(1)
           + 4 * 2.0 ** -24 * (np.abs(logit) + logit.max())).max()
    small = L * 2.0 ** -25 * 8 * vd * (1 + unit.max() / vd) / 2.0 ** 3 * (1 if dtype == BF16 else 1.5)
    p = 2.0 ** -10 if dtype == BF16 else 2.0 ** -11 + 2.0 ** -21
    bound = (torch.finfo(dtype).eps / 2 * np.abs(o) + A * (p + 2 * off) + small
             + 320 * 2.0 ** -23 * U + (2.0 ** -25 if dtype == FP16 else 0))
    return q, host, o, bound


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("L,copies,mass,mag,vd,D", [
    (65536, 1, 0.9, 0.5, 0.125, 128), (8192, 1, 0.99, 4.0, 1.0, 64), (4096, 512, 0.99, 0.5, 0.125, 128),
    (4096, 600, 0.99, 4.0, 1.0, 32), (1000, 1, 0.995, 0.5, 0.125, 128), (1000, 300, 0.995, 0.5, 0.0625, 64)])
def test_decode_a_faint_tail_behind_a_sink(L, copies, mass, mag, vd, D, dtype):
    """Scales of the values between 1 and 448. One query row, and a batch of the same sequence (single-warp teams)."""
    q, host, want, bound = faint_tail(L, mass, mag, vd, D, dtype, 40)
    ps = 64
    n = -(-L // ps)
    dev = sa.kv4_cache(n, 1, ps, D)
    for pool, x in zip(dev, (host[0], host[1], host[3], host[4])):
        pool.view(torch.uint8).flatten(0, 2)[:L] = torch.from_numpy(x[:, 0]).to(DEV)
    table = np.tile(np.arange(n, dtype=np.int32), (copies, 1))
    o = run_decode(q.to(DEV).expand(copies, 1, 1, D).contiguous(), dev, table, [L] * copies, L, scale=1.0, vd=vd)
    err = np.abs(ref.f64(o)[:, 0, 0] - want)
    assert (err <= bound).all(), (err / bound).max()
    assert np.linalg.norm(bound) < 0.1 * np.linalg.norm(want)  # the bound says something


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("lens,Hkv", [([900], 1), ([5000, 40], 1), ([3000] * 40, 2)])
def test_decode_scales_that_rise(lens, Hkv, D, dtype):
    """Values whose scales run from the smallest to the largest along a sequence, up and down and with single peaks: what
    the probabilities were kept larger by is given back on the way."""
    rng = np.random.default_rng(41)
    ps, L = 32, max(lens)
    for way in ("up", "down", "peaks"):
        pages = -(-L // ps)
        j = np.arange(pages * ps)
        size = {"up": -9 + 17.5 * j / L, "down": 8.5 - 17.5 * j / L, "peaks": np.where(j % 501 == 77, 8.5, -9 + j % 7)}[way]
        k = model_rows(rng, (pages * ps, Hkv, D), "k") * 0.5
        v = rng.uniform(-7.5, 7.5, (pages * ps, Hkv, D)) * np.exp2(np.clip(size, -9, 8.5))[:, None, None]
        v[..., ::32] = 7.5 * np.exp2(np.clip(size, -9, 8.5))[:, None, None]
        dev, host = [], []
        for x, which in ((k, "k"), (v, "v")):
            codes, byte, _ = ref.quantize(x, 1.0)
            for y in (ref.pack(codes, which), byte):
                y = np.ascontiguousarray(y.reshape(pages, ps, Hkv, -1).transpose(0, 2, 1, 3))
                host.append(y)
                dev.append(torch.from_numpy(y).to(DEV))
        dev[1], dev[3] = (x.view(torch.float8_e4m3fn) for x in (dev[1], dev[3]))
        table = np.tile(np.arange(pages, dtype=np.int32), (len(lens), 1))
        q = torch.from_numpy(rng.normal(size=(len(lens), 2 * Hkv, 1, D))).to(dtype).to(DEV)
        o = run_decode(q, dev, table, lens, L, vd=1.0)
        some = [0, len(lens) - 1]
        check_decode(o[some], q[some], host, table[some], [lens[b] for b in some], L, vd=1.0)


def test_decode_cap_empty_problems_and_no_pages():
    lens = [640, 640]
    q, dev, host, table = case(17, lens, 4, 1, 2, 64, 32, BF16)
    o = run_decode(q, dev, table, lens, 333)
    check_decode(o, q, host, table, lens, 333)
    assert torch.all(run_decode(q, dev, table, lens, 0) == 0)
    assert torch.all(run_decode(q, dev, table, [0, -5], 640) == 0)
    empty = sa.kv4_cache(0, 1, 32, 64)
    assert torch.all(run_decode(q, empty, table, lens, 640) == 0)
    assert run_decode(q[:0].contiguous(), dev, table[:0], [], 640).shape == (0, 4, 2, 64)


@pytest.mark.parametrize("D", [32, 64, 128])
def test_decode_pages_outside_the_pool_read_zeros(D):
    lens = [500, 512, 300]
    q, dev, host, table = case(47, lens, 8, 2, 1, D, 32, BF16)
    pages = host[0].shape[0]
    table[0, 3], table[1, 0], table[2, 7], table[1, 15] = -1, pages, 2 ** 31 - 1, -2 ** 31
    o = run_decode(q, dev, table, lens, 512)
    check_decode(o, q, host, table, lens, 512)


@pytest.mark.parametrize("D", [32, 64, 128])
def test_decode_rows_behind_the_end_may_hold_anything(D):
    """NaN scales and every code in the rows behind a sequence's last key, on pages that it uses."""
    lens = [500, 1, 300, 17]
    q, dev, host, table = case(48, lens, 4, 2, 1, D, 64, FP16)
    want = run_decode(q, dev, table, lens, 512, True, 250, 3)
    used = np.zeros(host[1].shape[:3:2], bool)
    for b, L in enumerate(lens):
        for j in range(L):
            used[table[b, j // 64], j % 64] = True
    dead = torch.from_numpy(~used).to(DEV)
    for n in (1, 3):
        dev[n].view(torch.uint8).permute(0, 2, 1, 3)[dead] = 0x7F  # E4M3 NaN
    for n in (0, 2):
        dev[n].permute(0, 2, 1, 3)[dead] = 0xF0
    assert torch.equal(run_decode(q, dev, table, lens, 512, True, 250, 3), want)


def test_decode_same_result_every_time_and_for_shared_pages():
    lens = [2000, 1500, 2000]
    q, dev, host, table = case(49, lens, 8, 2, 1, 128, 16, BF16)
    table[2] = table[0]  # two requests share a prefix's pages
    first = run_decode(q, dev, table, lens, 2000)
    check_decode(first, q, host, table, lens, 2000)
    for _ in range(5):
        assert torch.equal(run_decode(q, dev, table, lens, 2000), first)


def test_pools_past_32_bits():
    """Code pools of more than 2^31 bytes: rows at their end are written and read in the right place."""
    Hkv, ps, D = 2, 16, 128
    pages = (2 ** 31 + 2 ** 28) // (Hkv * ps * D // 2)
    dev = sa.kv4_cache(pages, Hkv, ps, D)
    assert dev[0].numel() > 2 ** 31
    rng = np.random.default_rng(50)
    L = 40
    table = np.array([[pages - 1, 0, pages - 2]], np.int32)
    x = {w: torch.from_numpy(model_rows(rng, (L, Hkv, D), w)).to(BF16).to(DEV) for w in "kv"}
    slots = [int(table[0, j // ps]) * ps + j % ps for j in range(L)]
    sa.attn_kv4_append(x["k"], x["v"], i32(slots), *dev, 1.0, 0.125)
    k = torch.empty(1, Hkv, L, D, dtype=BF16, device=DEV)
    v = torch.empty_like(k)
    sa.attn_kv4_gather(*dev, i32(table), i32([L]), k, v, 1.0, 0.125)
    q = torch.from_numpy(rng.normal(size=(1, 4, 1, D))).to(BF16).to(DEV)
    o = run_decode(q, dev, table, [L], L)
    quant = [ref.quantize(ref.f64(x[w]).transpose(1, 0, 2), d) for w, d in (("k", 1.0), ("v", 0.125))]
    val, unit = [z[2] for z in quant], [ref.units(z[1], d) for z, d in zip(quant, (1.0, 0.125))]
    assert np.array_equal(ref.f64(k[0]), val[0]) and np.array_equal(ref.f64(v[0]), val[1])
    want, bound = ref.attention(ref.f64(q)[0], val[0], val[1], True, 0, 0, 0.0, BF16, *unit)
    assert (np.abs(ref.f64(o)[0] - want) <= bound).all()


# ---------------------------------------------------------------------------
# together, as a serving loop uses them
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D,ps,dtype", [(128, 16, BF16), (64, 32, FP16)])
def test_serving_loop(D, ps, dtype):
    """Prompts of different lengths are placed, written and attended to, then four decode steps (the third
    with a finished request and a padded batch): tables, cache and outputs against the definition. The
    prompt's attention reads the cache back and runs attn_fwd on it."""
    rng = np.random.default_rng(D)
    B, Hq, Hkv, pages, width = 3, 4, 2, 40, 12
    kd, vd = 1.0, 0.125
    dev = sa.kv4_cache(pages, Hkv, ps, D)
    free = rng.permutation(pages).astype(np.int32)
    d_free, taken = i32(free), 0
    table = i32(np.full((B, width), -1))
    lens = i32([0] * B)
    told = [[np.zeros((0, Hkv, D)) for _ in range(4)] for _ in range(B)]  # keys, values and their units
    for step, (news, pad) in enumerate((([70, 1, 33], 0), ([1, 1, 1], 2), ([1, 0, 1], 1), ([2, 2, 2], 0), ([1, 1, 1], 5))):
        T = sum(news) + pad
        k = torch.from_numpy(model_rows(rng, (T, Hkv, D), "k")).to(dtype).to(DEV)
        v = torch.from_numpy(model_rows(rng, (T, Hkv, D), "v")).to(dtype).to(DEV)
        seq, starts, slots, stats = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (B, B + 1, T, 3))
        sa.attn_page_plan(lens, i32(news), d_free[taken:].clone(), table, seq, starts, slots, stats, ps)
        sa.attn_kv4_append(k, v, slots, *dev, kd, vd)
        n_rows, used, lost = stats.tolist()
        assert (n_rows, lost) == (sum(news), 0) and slots.tolist()[sum(news):] == [-1] * pad
        taken += used
        lens, at = seq, 0
        for b, n in enumerate(news):
            for which, x, d in ((0, k, kd), (1, v, vd)):
                z = ref.quantize(ref.f64(x[at:at + n]), d)
                told[b][which] = np.concatenate([told[b][which], z[2]])
                told[b][2 + which] = np.concatenate([told[b][2 + which], ref.units(z[1], d)])
            at += n
        M = 2 if step == 3 else 1
        q = torch.from_numpy(rng.normal(size=(B, Hq, M, D))).to(dtype).to(DEV)
        o = torch.full_like(q, float("nan"))
        sa.attn_decode_paged_kv4(q, *dev, table, lens, o, width * ps, True, 50, 4, 0.0, kd, vd)
        torch.cuda.synchronize()
        for b in range(B):
            kk, vv, ku, vu = (x.transpose(1, 0, 2) for x in told[b])
            want, bound = ref.attention(ref.f64(q)[b], kk, vv, True, 50, 4, 0.0, dtype, ku, vu)
            assert (np.abs(ref.f64(o)[b] - want) <= bound).all(), (step, b)
        if step == 0:  # the prompt of request 0: its chunk of 33 rows over the cached context
            N, M = 70, 33
            ck, cv = (torch.empty(1, Hkv, N, D, dtype=dtype, device=DEV) for _ in range(2))
            sa.attn_kv4_gather(*dev, table[:1], lens[:1], ck, cv, kd, vd)
            qc = torch.from_numpy(rng.normal(size=(1, Hq, M, D))).to(dtype).to(DEV)
            oc = sa.attention(qc, ck, cv, causal=True)
            kk, vv = (x.transpose(1, 0, 2) for x in told[0][:2])
            want, _ = ref.attention(ref.f64(qc)[0], kk, vv, True, 0, 0, 0.0, dtype)
            assert np.abs(ref.f64(oc)[0] - want).max() <= (1e-2 if dtype == FP16 else 2e-2)


def test_whole_step_in_a_graph():
    """Plan, append and decode captured once and replayed over new lengths, rows and queries; two graphs
    with workspaces of their own replayed one after the other, and an eager call between."""
    rng = np.random.default_rng(60)
    B, Hq, Hkv, D, ps, pages, width = 4, 8, 2, 128, 16, 300, 70
    _, host = make_cache(rng, pages, Hkv, ps, D)

    def world(seed):
        r = np.random.default_rng(seed)
        t = [torch.from_numpy(x.copy()).to(DEV) for x in host]
        w = dict(dev=[t[0], t[1].view(torch.float8_e4m3fn), t[2], t[3].view(torch.float8_e4m3fn)])
        w["cached"], w["new"] = i32(r.integers(0, 1000, B)), i32([1] * B)
        w["table"] = i32(r.permutation(pages)[: B * width].reshape(B, width))
        w["free"] = i32(r.permutation(pages)[:8])
        w["lens"], w["starts"], w["slots"], w["stats"] = i32([0] * B), i32([0] * (B + 1)), i32([0] * (B + 1)), i32([0] * 3)
        w["k"] = torch.from_numpy(r.normal(size=(B + 1, Hkv, D))).to(BF16).to(DEV)
        w["v"] = torch.from_numpy(r.normal(size=(B + 1, Hkv, D))).to(BF16).to(DEV)
        w["q"] = torch.from_numpy(r.normal(size=(B, Hq, 1, D))).to(BF16).to(DEV)
        w["o"] = torch.zeros_like(w["q"])
        return w

    def step(w):
        sa.attn_page_plan(w["cached"], w["new"], w["free"], w["table"], w["lens"], w["starts"], w["slots"], w["stats"], ps)
        sa.attn_kv4_append(w["k"], w["v"], w["slots"], *w["dev"], 1.0, 0.125)
        sa.attn_decode_paged_kv4(w["q"], *w["dev"], w["table"], w["lens"], w["o"], width * ps, True, 400, 4, 0.0, 1.0,
                                 0.125)

    def load(w, seed):
        new = world(seed)
        for name, x in new.items():
            for a, b in zip(w[name], x) if name == "dev" else [(w[name], x)]:
                a.view(torch.uint8).copy_(b.view(torch.uint8))

    graphs = []
    for seed in (1, 2):
        w = world(seed)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(w)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(w)
        graphs.append((g, w))
    for seed in (3, 4, 5):
        for n, (g, w) in enumerate(graphs):
            load(w, seed + 10 * n)
        eager = world(seed)
        for g, w in graphs:
            g.replay()
        step(eager)
        torch.cuda.synchronize()
        other = world(seed + 10)
        step(other)
        torch.cuda.synchronize()
        for want, (g, w) in zip((eager, other), graphs):
            for name in ("o", "table", "lens", "slots", "stats", "starts"):
                assert torch.equal(w[name], want[name]), name
            for a, b in zip(w["dev"], want["dev"]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_calls_on_two_streams_and_two_threads():
    """Calls that overlap, each with its own workspace, from streams and from host threads."""
    jobs = []
    for seed, lens, M in ((70, [3000, 100], 1), (71, [2500], 4), (72, [40] * 60, 1)):
        q, dev, host, table = case(seed, lens, 8, 2, M, 128, 16, BF16)
        jobs.append((q, dev, i32(table), i32(lens), max(lens), run_decode(q, dev, table, lens, max(lens))))
    outs = [torch.zeros_like(j[0]) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        for j, o, s in zip(jobs, outs, streams):
            sa.attn_decode_paged_kv4(j[0], *j[1], j[2], j[3], o, j[4], k_descale=1.0, v_descale=0.125, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, j[5]) for o, j in zip(outs, jobs))
    errors = []

    def work(j, o, s):
        try:
            for _ in range(5):
                sa.attn_decode_paged_kv4(j[0], *j[1], j[2], j[3], o, j[4], k_descale=1.0, v_descale=0.125, stream=s)
        except Exception as e:  # reported below
            errors.append(e)

    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=x) for x in zip(jobs, outs, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and all(torch.equal(o, j[5]) for o, j in zip(outs, jobs))


@pytest.mark.parametrize("ps,M,sinks", [(16, 1, 0), (16, 3, 5), (64, 1, 70), (32, 9, 16)])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_decode_rows_no_query_sees_may_hold_anything(ps, M, sinks, D):
    """NaN scales in front of the window: on pages wholly behind it (given up) and in the one it begins in."""
    lens, window = [500, 90, 333, 64], 75
    q, dev, host, table = case(90 + M, lens, 4, 2, M, D, ps, BF16)
    want = run_decode(q, dev, table, lens, 512, True, window, sinks)
    seen = np.zeros(host[1].shape[:3:2], bool)
    for b, L in enumerate(lens):
        for j in range(L):
            seen[table[b, j // ps], j % ps] = j >= max(L - M - window + 1, 0) or j < sinks
    dead = torch.from_numpy(~seen).to(DEV)
    assert int(dead.sum()) > 200
    for n in (1, 3):
        dev[n].view(torch.uint8).permute(0, 2, 1, 3)[dead] = 0x7F  # E4M3 NaN
    for n in (0, 2):
        dev[n].permute(0, 2, 1, 3)[dead] = 0xF0
    assert torch.equal(run_decode(q, dev, table, lens, 512, True, window, sinks), want)


@pytest.mark.parametrize("B,Hkv,window,sinks", [(3, 2, 0, 0), (3, 2, 1100, 21), (40, 2, 0, 0), (40, 2, 1100, 21)])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_decode_dirty_rows_of_cut_segments(B, Hkv, window, sinks, D):
    """The same, and rows behind the sequences' ends, where segments are cut: teams of four warps and of one."""
    rng = np.random.default_rng(B + D)
    lens = rng.integers(1, 3001, B).tolist()
    lens[0], lens[2] = 3000, 1101
    q, dev, host, table = case(94, lens, 2 * Hkv, Hkv, 2, D, 32, BF16)
    want = run_decode(q, dev, table, lens, 3000, True, window, sinks)
    check_decode(want, q, host, table, lens, 3000, True, window, sinks)
    seen = np.zeros(host[1].shape[:3:2], bool)
    for b, L in enumerate(lens):
        for j in range(L):
            seen[table[b, j // 32], j % 32] = not window or j >= L - 2 - window + 1 or j < sinks
    dead = torch.from_numpy(~seen).to(DEV)
    for n in (1, 3):
        dev[n].view(torch.uint8).permute(0, 2, 1, 3)[dead] = 0x7F  # E4M3 NaN
    for n in (0, 2):
        dev[n].permute(0, 2, 1, 3)[dead] = 0xF0
    assert torch.equal(run_decode(q, dev, table, lens, 3000, True, window, sinks), want)


@pytest.mark.parametrize("causal,window,sinks", [(True, 0, 0), (True, 75, 0), (True, 75, 9), (False, 75, 0)])
@pytest.mark.parametrize("B,most,Hq,Hkv,M,D,dtype", [
    (4, 500, 4, 2, 4, 128, BF16), (4, 500, 2, 2, 12, 64, FP16), (4, 500, 2, 1, 5, 32, FP16),  # segments left whole
    (4, 3000, 4, 2, 4, 128, FP16), (4, 3000, 2, 1, 5, 64, BF16),                              # cut, four warps a team
    (45, 1700, 4, 2, 4, 128, BF16), (90, 1700, 1, 1, 9, 64, FP16)])                           # cut, single warps
def test_what_a_row_does_not_see_does_not_reach_it(causal, window, sinks, B, most, Hq, Hkv, M, D, dtype):
    """NaN in a key or a value that some rows of a sequence see and others do not (the last keys, which later rows see,
    and those at the rows' window edges, which earlier ones see): rows that see the key are NaN, or the elements of
    the value's group; all else is as without it."""
    rng = np.random.default_rng(97)
    lens = rng.integers(M, most + 1, B).tolist()
    lens[0], lens[1], lens[2], lens[3] = most, M, 16 * (most // 16), 16 * (most // 16) - 15
    ps, G = 16, Hq // Hkv
    q, dev, host, table = case(98, lens, Hq, Hkv, M, D, ps, dtype)
    clean = run_decode(q, dev, table, lens, most, causal, window, sinks)
    hit = torch.zeros(B, Hq, M, D, dtype=torch.bool)
    for b, L in enumerate(lens):
        # the key that the last row alone sees; the one that the first row alone sees, and its neighbour; a middle one
        spots = [L - 1, L - M - window + 1, L - M - window + 2, max(L - 1 - M // 2, 0)]
        j, key, h, g = max(spots[b % 4], 0), b // 4 % 3 == 1, b % Hkv, b % (D // 32)
        page = int(table[b, j // ps])
        dev[1 if key else 3].view(torch.uint8)[page, h, j % ps, g] = 0x7F  # E4M3 NaN
        for i in range(M):
            if ref.visible(L, M, i, causal, window, sinks)[j]:
                hit[b, h * G:(h + 1) * G, i, slice(None) if key else slice(32 * g, 32 * g + 32)] = True
    assert hit.any() and not hit.all()
    got = run_decode(q, dev, table, lens, most, causal, window, sinks).cpu()
    assert got[hit].isnan().all() and torch.equal(got[~hit], clean.cpu()[~hit])


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dtype,kd,vd", [(BF16, 2.0 ** -64, 2.0 ** 64), (BF16, 2.0 ** 64, 2.0 ** -64),
                                         (FP16, 2.0 ** -5, 2.0 ** 7), (FP16, 2.0 ** -6, 1.0), (FP16, 1.0, 2.0 ** 8),
                                         (FP16, 2.0 ** -16, 2.0 ** 10), (FP16, 2.0 ** -64, 2.0 ** -20)])
def test_factors_at_their_ends(D, dtype, kd, vd):
    """The largest and the smallest factors, and on both sides of where FP16 holds every scale times the factor as a
    normal number: write, read back (rounded once to dtype) and attention. FP16 rows are far from their factor's
    range where that is needed: all codes 8, or scales at the top."""
    rng = np.random.default_rng(91)
    Hkv, ps, pages, T = 2, 16, 8, 100
    x = {}
    for which, d in (("k", kd), ("v", vd)):
        size = d if dtype == BF16 else min(max(d, 2.0 ** -14), 2.0 ** 9)
        x[which] = torch.from_numpy(model_rows(rng, (T, Hkv, D), which) * size).to(dtype)
        x[which][5] = 0
        x[which][6] *= 2.0 ** 5
        assert torch.isfinite(x[which]).all()
    dev = sa.kv4_cache(pages, Hkv, ps, D)
    table = make_table(rng, [T], ps, pages)
    slots = [int(table[0, j // ps]) * ps + j % ps for j in range(T)]
    sa.attn_kv4_append(x["k"].to(DEV), x["v"].to(DEV), i32(slots), *dev, kd, vd)
    out = {w: torch.full((1, Hkv, T, D), float("nan"), dtype=dtype, device=DEV) for w in "kv"}
    sa.attn_kv4_gather(*dev, i32(table), i32([T]), out["k"], out["v"], kd, vd)
    val, unit = {}, {}
    for which, d, n in (("k", kd, 0), ("v", vd, 2)):
        codes, byte, val[which] = ref.quantize(ref.f64(x[which]).transpose(1, 0, 2), d)
        unit[which] = ref.units(byte, d)
        got = bytes_np(dev[n])[table[0]].transpose(1, 0, 2, 3).reshape(Hkv, -1, D // 2)[:, :T]
        assert np.array_equal(got, ref.pack(codes, which)), which
        got = bytes_np(dev[n + 1])[table[0]].transpose(1, 0, 2, 3).reshape(Hkv, -1, D // 32)[:, :T]
        assert np.array_equal(got, byte), which
        assert torch.equal(out[which][0].cpu(), torch.from_numpy(val[which]).to(dtype)), which
    # keys of order one for the query's scale; outputs of FP16 stay in its range
    q = torch.from_numpy(rng.normal(size=(1, 4, 1, D))).to(dtype)
    scale = float(1 / (np.abs(val["k"]).max() + 2.0 ** -66) / 8)
    if dtype == FP16 and np.abs(val["v"]).max() > 60000:
        return
    o = run_decode(q.to(DEV), dev, table, [T], T, True, 0, 0, scale, kd, vd)
    want, bound = ref.attention(ref.f64(q)[0], val["k"], val["v"], True, 0, 0, scale, dtype, unit["k"], unit["v"], vd)
    assert (np.abs(ref.f64(o)[0] - want) <= bound).all()


@pytest.mark.parametrize("B,Hkv,most,D", [(300, 2, 1500, 64), (130, 4, 900, 32), (229, 2, 2500, 64), (457, 1, 400, 128)])
def test_decode_many_ragged_sequences(B, Hkv, most, D):
    """More sequences than a team has threads, more segments than there are teams, some of them cut."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, most, B).tolist()
    lens[7], lens[8], lens[B - 1] = most, 0, 1
    q, dev, host, table = case(B, lens, 2 * Hkv, Hkv, 1, D, 16, BF16)
    o = run_decode(q, dev, table, lens, most)
    check_decode(o, q, host, table, lens, most)


@pytest.mark.parametrize("B,Hq,Hkv,M,D,ps,dtype,causal,window,sinks", [
    (20, 12, 2, 2, 128, 16, BF16, True, 0, 0), (20, 12, 2, 2, 128, 64, FP16, True, 100, 20),
    (400, 1, 1, 1, 64, 32, FP16, True, 0, 0), (70, 8, 1, 3, 32, 16, BF16, False, 333, 65),
    (58, 3, 1, 1, 128, 128, BF16, True, 17, 0), (30, 4, 2, 5, 64, 16, FP16, True, 1, 3),
    (800, 2, 1, 1, 32, 16, FP16, True, 600, 5)])
def test_decode_more_segments_than_a_third_of_the_sms(B, Hq, Hkv, M, D, ps, dtype, causal, window, sinks):
    """Segments to single warps: several row blocks, windows that begin anywhere, more sequences than a block's threads,
    lengths of zero and one and below the rows."""
    rng = np.random.default_rng(B + D)
    most = 1700
    lens = rng.integers(0, most, B).tolist()
    lens[0], lens[3], lens[4], lens[5], lens[B - 1] = most, 0, 1, 2, 16
    q, dev, host, table = case(B, lens, Hq, Hkv, M, D, ps, dtype)
    o = run_decode(q, dev, table, lens, most, causal, window, sinks)
    check_decode(o, q, host, table, lens, most, causal, window, sinks)
    assert torch.equal(run_decode(q, dev, table, lens, most, causal, window, sinks), o)


@pytest.mark.parametrize("cap", [1023, 1024, 1025])
@pytest.mark.parametrize("B,Hq,Hkv", [(3, 4, 2), (228, 2, 2), (229, 2, 2)])
def test_decode_on_both_sides_of_whole_segments(B, Hq, Hkv, cap):
    """16 tiles of keys and 456 segments (three teams on each of 152 SMs) are left whole, more are cut."""
    rng = np.random.default_rng(cap)
    lens = rng.integers(1, cap + 1, B).tolist()
    lens[0] = cap
    q, dev, host, table = case(cap + B, lens, Hq, Hkv, 1, 64, 64, FP16)
    o = run_decode(q, dev, table, lens, cap)
    check_decode(o, q, host, table, lens, cap)


def test_append_and_gather_on_pages_of_no_power_of_two():
    rng = np.random.default_rng(92)
    Hkv, ps, pages, D, T = 2, 384, 4, 128, 700
    x = {w: torch.from_numpy(model_rows(rng, (T, Hkv, D), w)).to(BF16).to(DEV) for w in "kv"}
    table = np.array([[2, 0], [3, 1]], np.int32)
    dev = sa.kv4_cache(pages, Hkv, ps, D)
    slots = [int(table[0, j // ps]) * ps + j % ps for j in range(T)]
    sa.attn_kv4_append(x["k"], x["v"], i32(slots), *dev, 1.0, 0.125)
    k = torch.full((2, Hkv, 800, D), float("nan"), dtype=BF16, device=DEV)
    v = k.clone()
    sa.attn_kv4_gather(*dev, i32(table), i32([T, 500]), k, v, 1.0, 0.125)
    torch.cuda.synchronize()
    for out, w, d in ((k, "k", 1.0), (v, "v", 0.125)):
        want = ref.quantize(ref.f64(x[w]).transpose(1, 0, 2), d)[2]
        assert np.array_equal(ref.f64(out[0, :, :T]), want) and not out[0, :, T:].any() and not out[1].any()


def test_one_workspace_for_calls_and_graphs_one_after_the_other():
    """Nothing in a workspace outlives a call: one of them serves calls of other shapes in turn (cut segments listed by
    segment and by team, left whole), holds any bytes before a call, and is shared by two graphs."""
    jobs, most = [], 0
    for seed, lens, Hq, Hkv, M, D in ((1, [5000], 8, 2, 1, 128), (2, list(range(1, 901, 2)), 2, 2, 1, 64),
                                      (3, [30, 900], 4, 2, 3, 32), (4, [9000, 1, 2000], 16, 8, 2, 128)):
        q, dev, host, table = case(seed, lens, Hq, Hkv, M, D, 16, BF16)
        n = sa.attn_decode_paged_kv4_workspace_bytes(len(lens), Hq, Hkv, M, D, 16, table.shape[1], max(lens))
        most = max(most, n)
        jobs.append((q, dev, i32(table), i32(lens), max(lens), run_decode(q, dev, table, lens, max(lens))))
    work = torch.empty(most, dtype=torch.uint8, device=DEV)
    outs = [torch.zeros_like(j[0]) for j in jobs]

    def call(j, o):
        sa.attn_decode_paged_kv4(j[0], *j[1], j[2], j[3], o, j[4], k_descale=1.0, v_descale=0.125, workspace=work)

    for fill in (0, 0x7F, 0xFF):
        work.fill_(fill)
        for o in outs:
            o.zero_()
        for x in (0, 1, 2, 3, 0, 2, 1, 0):
            call(jobs[x], outs[x])
        torch.cuda.synchronize()
        assert all(torch.equal(o, j[5]) for o, j in zip(outs, jobs))
    graphs = []
    for x in range(4):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(jobs[x], outs[x])
        graphs.append(g)
    for o in outs:
        o.zero_()
    for x in (3, 0, 1, 0, 2, 1, 3):
        graphs[x].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, j[5]) for o, j in zip(outs, jobs))


def test_captured_behind_copies_and_branches():
    """The calls in a graph behind copies, fills and other kernels and with two branches joined in front of them: their
    early launch must not get ahead of any of those."""
    rng = np.random.default_rng(93)
    lens = [3000, 700]
    q, dev, host, table = case(93, lens, 8, 2, 1, 128, 16, BF16)
    want = run_decode(q, dev, table, lens, 3000)
    d_table, d_lens = i32(table), i32(lens)
    x = torch.from_numpy(rng.normal(size=(64, 2, 128))).to(BF16).to(DEV)
    slots = i32(rng.permutation(3 * 16)[:40].tolist() + [-1] * 24)
    pool = sa.kv4_cache(3, 2, 16, 128)
    sa.attn_kv4_append(x, x, slots, *pool)
    k = torch.empty(1, 2, 48, 128, dtype=BF16, device=DEV)
    v = torch.empty_like(k)
    pages, n48 = i32([[0, 1, 2]]), i32([48])
    sa.attn_kv4_gather(*pool, pages, n48, k, v)
    torch.cuda.synchronize()
    w_k, w_v = k.clone(), v.clone()
    late = [torch.zeros_like(t) for t in (q, d_table, d_lens, x, slots)]
    o = torch.zeros_like(q)
    other = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for t in pool:
            t.view(torch.uint8).zero_()
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            late[0].copy_(q)
            late[3].copy_(x * 1.0)
        for n, src in ((1, d_table), (2, d_lens), (4, slots)):
            late[n].copy_(src)
        torch.cuda.current_stream().wait_stream(other)
        sa.attn_kv4_append(late[3], late[3], late[4], *pool)
        sa.attn_kv4_gather(*pool, pages, n48, k, v)
        sa.attn_decode_paged_kv4(late[0], *dev, late[1], late[2], o, 3000, k_descale=1.0, v_descale=0.125)
        sa.attn_decode_paged_kv4(late[0], *dev, late[1], late[2], o, 3000, k_descale=1.0, v_descale=0.125)
    for _ in range(5):
        for t in (*late, o, k, v):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(k, w_k) and torch.equal(v, w_v)


def test_status_word_stays_clear():
    assert sa.last_device_status() == 0
