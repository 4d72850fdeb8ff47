"""The 4-bit paged cache without a GPU: what its entry points refuse (metadata
only, nothing is launched), what the binding refuses, and the reference the GPU
tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import kv4_reference as ref
import streaming_attention_gb300 as sa
from streaming_attention_gb300 import build as B


@pytest.fixture(scope="module")
def L():
    B.build()
    return sa.lib()


def at(n):
    return ctypes.c_void_p(0x100000 * (n + 1))  # aligned, distinct, never dereferenced


OFF = ctypes.c_void_p(0x900004)  # 4-byte aligned only
ODD = ctypes.c_void_p(0x900002)


def decode(L, q=at(0), kc=at(1), ks=at(2), vc=at(3), vs=at(4), table=at(5), lens=at(6), o=at(7), B_=2, Hq=8, Hkv=2, M=1,
           D=128, pages=8, ps=16, maxp=4, max_len=64, window=0, sinks=0, kd=1.0, vd=1.0, dtype=0, ws=None, nb=0):
    return L.attn_decode_paged_kv4(q, kc, ks, vc, vs, table, lens, o, B_, Hq, Hkv, M, D, pages, ps, maxp, max_len, 1,
                                   window, sinks, 0.0, kd, vd, dtype, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), -3), (dict(dtype=7), -3),
    (dict(B_=-1), -2), (dict(M=-1), -2), (dict(Hkv=0), -2), (dict(maxp=-1), -2), (dict(max_len=-1), -2),
    (dict(pages=-1), -2), (dict(ps=0), -2), (dict(ps=24), -2), (dict(ps=192), -2),
    (dict(Hq=6, Hkv=4), -5),
    (dict(D=16), -4), (dict(D=96), -4), (dict(D=256), -4),
    (dict(pages=1 << 27, ps=16), -6),              # 2^31 slots
    (dict(B_=70000, Hq=1, Hkv=1), -6),             # grid limit B * Hkv
    (dict(B_=1 << 14, Hq=64, Hkv=2, M=64), -6),    # q
    (dict(B_=1 << 20, maxp=1 << 12), -6),          # the table
    (dict(kd=0.0), -12), (dict(kd=-1.0), -12), (dict(vd=0.3), -12), (dict(vd=float("inf")), -12),
    (dict(vd=float("nan")), -12), (dict(kd=2.0 ** -130), -12), (dict(kd=2.0 ** 127), -12),
    (dict(kd=2.0 ** -65), -12), (dict(vd=2.0 ** 65), -12),
    (dict(q=None), -1), (dict(o=None), -1), (dict(kc=None), -1), (dict(vs=None), -1), (dict(table=None), -1),
    (dict(lens=None), -1),
    (dict(q=OFF), -7), (dict(o=OFF), -7), (dict(ks=OFF), -7), (dict(table=ODD), -7), (dict(lens=ODD), -7),
])
def test_decode_refusals(L, kw, status):
    assert decode(L, **kw) == status


def test_decode_workspace(L):
    need = sa.attn_decode_paged_kv4_workspace_bytes(1, 32, 8, 1, 128, 16, 8192, 131072)
    assert need > 0
    big = dict(B_=1, Hq=32, Hkv=8, maxp=8192, max_len=131072)
    assert decode(L, ws=at(8), nb=need - 1, **big) == -8
    assert decode(L, ws=OFF, nb=need, **big) == -7
    assert sa.attn_decode_paged_kv4_workspace_bytes(1, 32, 8, 1, 48, 16, 8192, 131072) == 0
    assert sa.attn_decode_paged_kv4_workspace_bytes(0, 32, 8, 1, 128, 16, 8192, 131072) == 0
    assert sa.attn_decode_paged_kv4_workspace_bytes(1, 32, 8, 1, 128, 16, 8192, 0) == 0


def test_decode_workspace_does_not_fall_with_larger_calls():
    size = sa.attn_decode_paged_kv4_workspace_bytes
    Bs, Hs, Ms = [1, 2, 14, 15, 57, 58, 152, 444, 445, 456, 457, 2000], [1, 2, 8], [1, 2, 9]
    lens = [1, 64, 1000, 1024, 1025, 3000, 100000]
    for window in (0, 1, 500):
        n = {(B, H, M, N): size(B, 4 * H, H, M, 64, 16, 6250, N, True, window)
             for B in Bs for H in Hs for M in Ms for N in lens}
        for k, (axis, values) in enumerate((("B", Bs), ("Hkv", Hs), ("M", Ms), ("max_seq_len", lens))):
            for key, got in n.items():
                i = values.index(key[k])
                if i + 1 < len(values):
                    assert got <= n[key[:k] + (values[i + 1],) + key[k + 1:]], (axis, key, window)
        assert max(n.values()) == n[Bs[-1], Hs[-1], Ms[-1], lens[-1]] > 0


def test_decode_workspace_serves_every_smaller_call(L):
    """Query and KV heads one by one (a call needs Hq % Hkv == 0): the size does not fall along any argument, also where
    more KV heads make fewer segments (18 query heads on 2 and on 3, 36 on 4 and on 6), and a workspace of the largest
    call's size is not refused by a smaller one."""
    size = sa.attn_decode_paged_kv4_workspace_bytes
    assert size(1, 18, 2, 1, 128, 16, 125, 2000) <= size(1, 18, 3, 1, 128, 16, 125, 2000)
    assert size(1, 36, 4, 1, 128, 16, 125, 2000) <= size(1, 36, 6, 1, 128, 16, 125, 2000)
    for B, M, N, window in ((1, 1, 2000, 0), (4, 3, 1000, 0), (16, 1, 5000, 700), (60, 5, 900, 0), (200, 1, 1024, 100)):
        heads = [(q, h) for q in (1, 2, 3, 6, 8, 9, 12, 18, 24, 36, 40, 64, 72, 100) for h in range(1, q + 1) if q % h == 0]
        n = {x: size(B, *x, M, 64, 16, 400, N, True, window) for x in heads}
        for (q, h), got in n.items():
            for (q2, h2), more in n.items():
                if q <= q2 and h <= h2:
                    assert got <= more, (B, M, N, window, (q, h), (q2, h2))
            for smaller in (size(B - 1, q, h, M, 64, 16, 400, N, True, window) if B > 1 else 0,
                            size(B, q, h, M - 1, 64, 16, 400, N, True, window) if M > 1 else 0,
                            size(B, q, h, M, 64, 16, 400, N - 1, True, window)):
                assert smaller <= got
    # the smaller call itself: a workspace that is too small is told before anything else happens
    big = size(1, 18, 3, 1, 128, 16, 125, 2000)
    short = dict(B_=1, Hq=18, Hkv=2, maxp=125, max_len=2000)
    assert decode(L, ws=OFF, nb=big, **short) == -7  # large enough, not aligned
    assert decode(L, ws=at(8), nb=16, **short) == -8


def append(L, k=at(0), v=at(1), slots=at(2), kc=at(3), ks=at(4), vc=at(5), vs=at(6), T=3, Hkv=2, D=128, kst=256, vst=256,
           pages=8, ps=16, kd=1.0, vd=1.0, dtype=0):
    return L.attn_kv4_append(k, v, slots, kc, ks, vc, vs, T, Hkv, D, kst, vst, pages, ps, kd, vd, dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), -3), (dict(T=-1), -2), (dict(Hkv=-1), -2), (dict(ps=8), -2), (dict(D=80), -4),
    (dict(kst=255), -2), (dict(vst=0), -2), (dict(kst=260), -7), (dict(vst=1028), -7),
    (dict(T=1 << 24), -6), (dict(pages=1 << 28), -6), (dict(kd=3.0), -12), (dict(vd=0.0), -12),
    (dict(kd=2.0 ** 65), -12), (dict(vd=2.0 ** -65), -12),
    (dict(k=None), -1), (dict(slots=None), -1), (dict(vc=None), -1), (dict(v=OFF), -7), (dict(slots=ODD), -7),
    (dict(T=0, k=None, v=None, slots=None), 0), (dict(pages=0, kc=None, ks=None, vc=None, vs=None), 0),
])
def test_append_refusals(L, kw, status):
    assert append(L, **kw) == status


def gather(L, kc=at(0), ks=at(1), vc=at(2), vs=at(3), table=at(4), lens=at(5), k=at(6), v=at(7), B_=2, Hkv=2, N=40,
           D=64, pages=8, ps=16, maxp=4, kd=1.0, vd=1.0, dtype=1):
    return L.attn_kv4_gather(kc, ks, vc, vs, table, lens, k, v, B_, Hkv, N, D, pages, ps, maxp, kd, vd, dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), -3), (dict(N=-1), -2), (dict(B_=-1), -2), (dict(maxp=-1), -2), (dict(D=8), -4), (dict(ps=12), -2),
    (dict(N=1 << 24), -6), (dict(B_=70000, N=1), -6), (dict(kd=0.7), -12), (dict(vd=2.0 ** -65), -12), (dict(k=None), -1), (dict(lens=None), -1),
    (dict(table=None), -1), (dict(v=OFF), -7), (dict(N=0, k=None, v=None), 0),
])
def test_gather_refusals(L, kw, status):
    assert gather(L, **kw) == status


@pytest.mark.parametrize("call,kw", [
    (gather, dict(B_=1 << 15, Hkv=1 << 15, N=1 << 27, D=128)),   # 2^64 elements
    (gather, dict(B_=65535, Hkv=65535, N=(1 << 31) - 1, D=128)),
    (gather, dict(B_=1 << 15, Hkv=1 << 15, N=1 << 27, D=128, k=None, v=None)),
    (append, dict(T=1 << 30, Hkv=1 << 27, D=128)),
    (append, dict(T=(1 << 31) - 1, Hkv=(1 << 31) - 1, D=128)),
    (decode, dict(B_=1 << 15, Hq=1 << 15, Hkv=1, M=1 << 27, D=128)),
    (decode, dict(B_=1, Hq=(1 << 31) - 1, Hkv=1, M=(1 << 31) - 1, D=128)),
])
def test_sizes_whose_product_passes_64_bits(L, call, kw):
    assert call(L, **kw) == -6


def plan(L, cached=at(0), new=at(1), free=at(2), table=at(3), lens=at(4), starts=at(5), slots=at(6), stats=at(7), B_=4,
         ps=16, maxp=8, nfree=5, rows=9):
    return L.attn_page_plan(cached, new, free, table, lens, starts, slots, stats, B_, ps, maxp, nfree, rows, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B_=-1), -2), (dict(ps=0), -2), (dict(maxp=-1), -2), (dict(nfree=-1), -2), (dict(rows=-1), -2),
    (dict(B_=1 << 20, maxp=1 << 12), -6), (dict(B_=(1 << 31) - 2, maxp=0), -6),
    (dict(cached=None), -1), (dict(free=None), -1), (dict(table=None), -1), (dict(stats=None), -1),
    (dict(slots=None), -1), (dict(new=ODD), -7), (dict(slots=ODD), -7),
    (dict(lens=at(0)), -13),                             # seq_lens in place of cached_lens
    (dict(slots=ctypes.c_void_p(at(4).value + 12)), -13),  # slot_map begins inside seq_lens
    (dict(table=at(2)), -13),
])
def test_plan_refusals(L, kw, status):
    assert plan(L, **kw) == status


def test_strerror_names_the_new_codes(L):
    assert sa.strerror(-12) != "unknown status" and sa.strerror(-13) != "unknown status"
    assert sa.strerror(-14) == "unknown status"


def test_binding_refusals():
    pools = sa.kv4_cache(4, 2, 16, 64, device="cpu")
    assert pools[0].shape == (4, 2, 16, 32) and pools[1].shape == (4, 2, 16, 2)
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    table, lens = torch.zeros(1, 2, **i32), torch.zeros(1, **i32)
    with pytest.raises(ValueError, match="CUDA device"):
        sa.attn_decode_paged_kv4(q, *pools, table, lens, q.clone(), 32)
    with pytest.raises(ValueError, match="must be"):
        sa.attn_decode_paged_kv4(q[..., :32], *pools, table, lens, q[..., :32], 32)
    with pytest.raises(ValueError, match="int32"):
        sa.attn_decode_paged_kv4(q, *pools, table.long(), lens, q.clone(), 32)
    with pytest.raises(ValueError, match="scales"):
        sa.attn_decode_paged_kv4(q, pools[0], pools[1].view(torch.uint8), *pools[2:], table, lens, q.clone(), 32)
    k = torch.zeros(3, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="contiguous"):
        sa.attn_kv4_append(k.transpose(0, 1).contiguous().transpose(0, 1), k, torch.zeros(3, **i32), *pools)
    with pytest.raises(ValueError, match="slot_map"):
        sa.attn_kv4_append(k, k, torch.zeros(2, **i32), *pools)
    with pytest.raises(ValueError, match="dtype"):
        sa.attn_kv4_append(k.float(), k.float(), torch.zeros(3, **i32), *pools)
    out = torch.zeros(1, 2, 5, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="contiguous"):
        sa.attn_kv4_gather(*pools, table, lens, out.transpose(2, 3).contiguous().transpose(2, 3), out)
    with pytest.raises(ValueError, match="seq_lens"):
        sa.attn_kv4_gather(*pools, table, torch.zeros(2, **i32), out, out.clone())
    one, two, three = (torch.zeros(n, **i32) for n in (1, 2, 3))
    with pytest.raises(ValueError, match="row_starts"):
        sa.attn_page_plan(one, one, three, table, one.clone(), one.clone(), three, three, 16)
    with pytest.raises(ValueError, match="CUDA device"):
        sa.attn_page_plan(one, one.clone(), three, table, one.clone(), two, three.clone(), three.clone(), 16)


# ---- the reference ----
def test_reference_e4m3_is_the_rounding_of_the_format():
    x = np.concatenate([np.linspace(0, 2.0 ** -5, 4097), np.exp2(np.linspace(-9, 8.8, 5001)), np.arange(0, 449) * 1.0])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn)
    x32 = torch.from_numpy(x).float().double().numpy()
    v, byte = ref.e4m3_round(x32)
    assert np.array_equal(byte, want.view(torch.uint8).numpy())
    assert np.array_equal(v, want.double().numpy())
    assert np.array_equal(ref.e4m3_value(byte), v)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("which", ["k", "v"])
def test_reference_pack_is_a_reordering(D, which):
    rng = np.random.default_rng(D)
    codes = rng.integers(0, 16, (5, D)).astype(np.uint8)
    packed = ref.pack(codes, which)
    assert np.array_equal(ref.unpack(packed, which), codes)
    assert sorted(ref.place(D, which)) == list(range(D))
    # element d's unit u of group i is the row's unit u * (D / 32) + i
    u = ref.UNIT[which]
    d = D - 1
    unit = (GROUPS := 32 // u) - 1
    assert ref.place(D, which)[d] // u == unit * (D // 32) + D // 32 - 1 and GROUPS * u == 32


def test_reference_quantize_worked_example():
    x = np.zeros(32)
    x[:5] = [7.5, -7.5, 0.5, -0.5, 1.25]  # scale 1: codes 8 + (7 clamped, -8, 1, -1, 1)
    codes, byte, val = ref.quantize(x, 1.0)
    assert list(codes[:6]) == [15, 0, 9, 7, 9, 8] and byte[0] == 0x38
    assert list(val[:6]) == [7, -8, 1, -1, 1, 0]
    codes, byte, val = ref.quantize(np.zeros(32), 0.25)
    assert (codes == 8).all() and byte[0] == 0 and (val == 0).all()


def test_reference_attention_is_the_library_formula():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(4, 3, 32)), rng.normal(size=(2, 20, 32)), rng.normal(size=(2, 20, 32))
    o, bound = ref.attention(q, k, v, True, 7, 2, 0.0, torch.bfloat16)
    T = torch.from_numpy
    kk, vv = T(k).repeat_interleave(2, 0), T(v).repeat_interleave(2, 0)
    p = torch.arange(3)[:, None] + 17
    j = torch.arange(20)[None]
    mask = (j <= p) & ((j > p - 7) | (j < 2))
    want = torch.nn.functional.scaled_dot_product_attention(T(q)[None], kk[None], vv[None], attn_mask=mask)[0]
    assert np.abs(want.numpy() - o).max() < 1e-12
    assert (bound > 0).all()


def test_reference_plan_worked_example():
    # pages of 4: request 0 has 3 keys and gets 2 (one new page), request 1 starts with 5 (two pages)
    table, lens, starts, slots, stats = ref.plan([3, 0, 8], [2, 5, 0], [9, 4, 7], [[1, 0], [0, 0], [2, 3]], 4, 9)
    assert table == [[1, 9], [4, 7], [2, 3]] and lens == [5, 5, 8] and starts == [0, 2, 7, 7]
    assert slots == [7, 36, 16, 17, 18, 19, 28, -1, -1] and stats == [7, 3, 0]
