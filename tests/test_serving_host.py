"""Argument errors of the paged serving calls, on the CPU: every call below must be
refused before any CUDA work (the addresses are never dereferenced)."""
import ctypes
import math

import pytest

import long_context_attention_pair_b200 as atf

P = 1 << 20
DP = ctypes.c_double


@pytest.fixture(scope="module")
def L():
    from long_context_attention_pair_b200 import build
    build.build()
    return atf.lib()


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def table(vals):
    return (DP * len(vals))(*vals)


ORDER = {
    "rope_apply": "q qs k ks qo qos ko kos positions B T Hq Hkv D R base scale inter inv dt stream",
    "cache_append": "k ks v vs kpages vpages bt lens positions counts B T Hkv max_pages num_pages page D base rotated layout stream",
    "tree_decode_paged": "q qs kpages vpages bt lens mask positions counts out lse B T Hq Hkv max_pages num_pages page D base kwin "
                         "layout odt ws wsb stream",
    "cache_compact": "kpages vpages bt lens path acc new B M Hkv max_pages num_pages page D layout stream",
    "cache_copy_pages": "kpages vpages src dst tokens n Hkv num_pages page D layout stream",
}
GOOD = dict(q=P, qs=None, k=P, ks=None, v=P, vs=None, qo=P, qos=None, ko=P, kos=None, positions=P, B=2, T=5, Hq=8, Hkv=2, D=128, R=128,
            base=1e4, scale=1.0, inter=0, inv=0, dt=atf.BF16, stream=None, kpages=P, vpages=P, bt=P, lens=P, counts=None, max_pages=4,
            num_pages=20, page=64, rotated=1, layout=atf.KV_PACKED, mask=None, out=P, lse=None, kwin=1.0, odt=atf.BF16, ws=P, wsb=1 << 40,
            path=P, acc=P, new=None, M=4, src=P, dst=P, tokens=None, n=3)

CASES = [
    ("rope_apply", -1, [dict(q=None), dict(qo=None), dict(positions=None), dict(k=None), dict(ko=None), dict(B=0), dict(T=0), dict(Hq=0),
                        dict(Hkv=0), dict(T=1 << 31), dict(D=127), dict(D=258, R=2), dict(R=0), dict(R=130), dict(R=7), dict(base=1.0),
                        dict(base=math.nan), dict(scale=math.inf), dict(scale=math.nan), dict(inter=2), dict(inv=-1), dict(Hq=40000)]),
    ("rope_apply", -2, [dict(dt=7)]),
    ("rope_apply", -6, [dict(q=P + 2), dict(ko=P + 8)]),
    ("cache_append", -1, [dict(k=None), dict(v=None), dict(kpages=None), dict(vpages=None), dict(bt=None), dict(lens=None), dict(B=0),
                          dict(T=0), dict(Hkv=0), dict(max_pages=0), dict(num_pages=0), dict(page=32), dict(page=100), dict(base=0.5),
                          dict(rotated=2), dict(rotated=0), dict(layout=atf.KV_HND), dict(layout=9), dict(num_pages=1 << 28),
                          dict(max_pages=1 << 26), dict(B=1 << 16, T=1 << 16)]),
    ("cache_append", -2, [dict(D=96), dict(D=256)]),
    ("cache_append", -6, [dict(k=P + 8), dict(vpages=P + 2), dict(ks=strides(1280, 257, 128)), dict(vs=strides(1284, 256, 128))]),
    ("tree_decode_paged", -1, [dict(q=None), dict(kpages=None), dict(vpages=None), dict(bt=None), dict(lens=None), dict(out=None), dict(B=0),
                               dict(T=0), dict(Hq=7), dict(Hkv=0), dict(max_pages=0), dict(num_pages=-1), dict(page=0), dict(kwin=-1.0),
                               dict(kwin=math.nan), dict(base=1.0), dict(layout=atf.KV_HND), dict(B=1 << 20, T=1 << 10)]),
    ("tree_decode_paged", -2, [dict(D=96), dict(odt=3)]),
    ("tree_decode_paged", -3, [dict(ws=None), dict(wsb=0)]),
    ("tree_decode_paged", -6, [dict(q=P + 4), dict(out=P + 2), dict(ws=P + 8), dict(kpages=P + 8), dict(qs=strides(5120, 1028, 128))]),
    ("cache_compact", -1, [dict(kpages=None), dict(vpages=None), dict(bt=None), dict(lens=None), dict(path=None), dict(acc=None), dict(new=P),
                           dict(B=0), dict(M=0), dict(Hkv=0), dict(page=65), dict(layout=atf.KV_HND)]),
    ("cache_compact", -2, [dict(M=1025), dict(D=32)]),
    ("cache_compact", -6, [dict(kpages=P + 4)]),
    ("cache_copy_pages", -1, [dict(kpages=None), dict(vpages=None), dict(src=None), dict(dst=None), dict(n=0), dict(num_pages=0), dict(page=63),
                              dict(layout=atf.KV_HND)]),
    ("cache_copy_pages", -2, [dict(D=80)]),
    ("cache_copy_pages", -6, [dict(vpages=P + 2)]),
]


@pytest.mark.parametrize("name,status,changes", CASES, ids=[f"{n}{s}" for n, s, _ in CASES])
def test_bad_arguments_are_refused(L, name, status, changes):
    for ch in changes:
        a = {**GOOD, **ch}
        args = [a[x] for x in ORDER[name].split()]
        assert getattr(L, "atflash_" + name)(*args) == status, ch
        if "base" in ORDER[name].split() and "base" not in ch:
            dims = a["R"] if name == "rope_apply" else a["D"]
            if 2 <= dims <= 256 and dims % 2 == 0:
                a["base"] = table(atf.theta_table(dims, 1e4))
                args = [a[x] for x in ORDER[name].split()]
                assert getattr(L, "atflash_" + name + "_theta")(*args) == status, ch


@pytest.mark.parametrize("name", ["rope_apply", "cache_append", "tree_decode_paged"])
def test_bad_frequency_tables_are_refused(L, name):
    good = atf.theta_table(128, 1e4)
    for bad in (None, table([0.0] + good[1:]), table(good[:-1] + [1.0]), table([4.0] + good[1:]), table([math.nan] + good[1:])):
        a = {**GOOD, "base": bad}
        assert getattr(L, "atflash_" + name + "_theta")(*[a[x] for x in ORDER[name].split()]) == -1


def test_workspace_size(L):
    assert atf.tree_decode_workspace_bytes(2, 5, 8, 2, 128) > 0
    for bad in [(0, 5, 8, 2, 128), (2, 0, 8, 2, 128), (2, 5, 7, 2, 128), (2, 5, 8, 2, 96), (1 << 20, 1 << 10, 8, 2, 64)]:
        assert atf.tree_decode_workspace_bytes(*bad) == 0


def test_python_checks_come_before_the_library():
    torch = pytest.importorskip("torch")
    q, k = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
    pos = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        atf.rope_apply(q, k, pos, 1e4)
    with pytest.raises(TypeError, match="dtype"):
        atf.rope_apply(q.half(), k.half(), pos, 1e4)
    pool = torch.zeros(3, 64, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        atf.cache_copy_pages(pool, pool, pos[0], pos[0], 64)
    with pytest.raises(ValueError, match="kv_layout"):
        atf._pools(pool, pool, 64, "HND", torch.bfloat16)
    with pytest.raises(ValueError, match="page_size"):
        atf._pools(pool, pool, 128, "NHD", torch.bfloat16)
    with pytest.raises(ValueError, match="kpages"):
        atf._pools(pool, pool, 64, "PACKED", torch.bfloat16)
    with pytest.raises(TypeError, match="bfloat16"):
        atf._pools(pool.float(), pool, 64, "NHD", torch.bfloat16)
    assert atf._pools(pool, pool, 64, "NHD", torch.bfloat16)[:4] == (atf.KV_NHD, 2, 64, 3)
    with pytest.raises(TypeError, match="int32"):
        atf._flat(pos.long(), "positions", (1, 2), torch.int32)
    with pytest.raises(ValueError, match="positions"):
        atf._flat(pos, "positions", (2, 1), torch.int32)
    with pytest.raises(ValueError, match="contiguous"):
        atf._flat(torch.zeros(2, 4, dtype=torch.int32).T, "path", (4, 2), torch.int32)
    with pytest.raises(ValueError, match="last dimension"):
        atf._strided(torch.zeros(1, 2, 64, 4).transpose(2, 3), "q", (1, 2, 4, 64), torch.float32)
    with pytest.raises(ValueError, match="expanded"):
        atf._strided(torch.zeros(1, 1, 4, 64).expand(1, 2, 4, 64), "out_q", (1, 2, 4, 64), torch.float32, True)


@pytest.mark.parametrize("name", ["lens", "acc", "path", "bt"])
def test_new_lengths_must_not_overlap_an_input(L, name):
    for new in (P, P + 4, P - 4):
        a = {**GOOD, "lens": P + 4096, "acc": P + 8192, "path": P + 12288, "bt": P + 16384, "new": new, name: P}
        assert L.atflash_cache_compact(*[a[x] for x in ORDER["cache_compact"].split()]) == -1


def test_pages_beyond_32_bit_indices_are_refused(L):
    a = {**GOOD, "page": 1 << 26, "Hkv": 4, "num_pages": 2}  # 2^32 units of 16 bytes
    assert L.atflash_cache_copy_pages(*[a[x] for x in ORDER["cache_copy_pages"].split()]) == -1
    a.update(page=1 << 24, Hkv=4)  # 2^30: an index and the round of loads after it reach 2^31
    assert L.atflash_cache_copy_pages(*[a[x] for x in ORDER["cache_copy_pages"].split()]) == -1
