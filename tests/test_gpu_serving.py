"""The paged serving calls against their definitions in 64 bits (tests/serving_ref.py):
rotary positions, appending, tree attention, compaction, page copies, and a whole
drafted step of all of them."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import long_context_attention_pair_b200 as atf  # noqa: E402
import serving_ref as R  # noqa: E402

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative to the value


def randn(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.fixture(autouse=True)
def clean_status():
    yield
    torch.cuda.synchronize()
    assert atf.device_status() == 0


# ------------------------------------------------------------------ rotary positions
ROPE = [
    # B, T, Hq, Hkv, D, rotary, interleaved, scale, inverse, dtype
    (1, 1, 1, 1, 2, 2, False, 1.0, False, torch.bfloat16),
    (2, 37, 14, 2, 64, 64, False, 1.0, False, torch.bfloat16),
    (1, 300, 28, 4, 128, 128, True, 1.25, False, torch.bfloat16),
    (3, 33, 3, 3, 96, 48, False, 1.0, True, torch.bfloat16),
    (2, 19, 5, 1, 80, 6, True, 0.5, True, torch.bfloat16),
    (2, 65, 24, 8, 128, 64, True, 1.1, True, torch.float32),
    (1, 129, 7, 1, 256, 256, False, 1.0, False, torch.float32),
    (4, 5, 2, 2, 66, 34, False, 2.0, False, torch.float32),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot,inter,scale,inv,dt", ROPE)
def test_rope_equals_its_definition(B, T, Hq, Hkv, D, rot, inter, scale, inv, dt):
    q, k = randn((B, T, Hq, D), 1, dt), randn((B, T, Hkv, D), 2, dt)
    rng = np.random.default_rng(3)
    pos = rng.integers(0, 1 << 20, size=(B, T))
    pos.flat[0], pos.flat[-1] = (1 << 31) - 1, -(1 << 31) if B * T > 1 else (1 << 31) - 1
    pos = ints(pos.tolist())
    base = 1e6
    oq, ok = atf.rope_apply(q, k, pos, base, rotary_dim=rot, interleaved=inter, scale=scale, inverse=inv)
    th = R.theta_of(base, rot)
    # Positions near 2^31 times theta: the reference angle itself is good to 2^31 * 2^-53 * a few.
    for got, x in ((oq, q), (ok, k)):
        ref = R.rope(x, pos, th, rotary_dim=rot, interleaved=inter, scale=scale, inverse=inv)
        R.close(got, ref, ref.abs() * HALF[dt] + R.rope_slack(x, rot, inter, scale, HALF[dt]), "rope")
        assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt,pad", [(torch.bfloat16, 0), (torch.bfloat16, 3), (torch.float32, 2)])
def test_rope_strided_in_place_and_without_keys(inter, dt, pad):
    # q and k as views of one fused projection (rows padded so that pad = 0 is the 16-byte case), in both
    # [B, T, H, D] and head-major storage; in place; and q alone.
    B, T, Hq, Hkv, D = 2, 21, 6, 2, 64
    row = (Hq + 2 * Hkv) * D + pad
    buf = randn((B, T, row), 5, dt)
    qkv = buf[:, :, : (Hq + 2 * Hkv) * D].unflatten(-1, (Hq + 2 * Hkv, D))
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
    pos = ints([[7 * t + b for t in range(T)] for b in range(B)])
    oq, ok = atf.rope_apply(q, k, pos, 1e4, interleaved=inter)
    head_major = q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    assert torch.equal(atf.rope_apply(head_major, None, pos, 1e4, interleaved=inter), oq)
    rest = buf.clone()
    assert atf.rope_apply(q, k, pos, 1e4, interleaved=inter, out_q=q, out_k=k)[0] is q
    assert torch.equal(q, oq) and torch.equal(k, ok)
    n = (Hq + Hkv) * D
    assert torch.equal(buf[:, :, n:], rest[:, :, n:])  # values and padding untouched


def test_rope_matches_the_prefill_rotation():
    # The packed pre-pass at positions 0..N-1 and this call give the same bf16 values up to one rounding of
    # fp32 results that differ in their last bits.
    B, N, H, D, base = 1, 257, 2, 64, 1e6
    x = randn((B, N, H, D), 9)
    pack = atf.rope_pack(x, base).view(B, H, D // 16, N, 8, 2).permute(0, 3, 1, 5, 2, 4).reshape(B, N, H, D)
    got = atf.rope_apply(x, None, torch.arange(N, device="cuda", dtype=torch.int32)[None], base)
    ref = R.rope(x, torch.arange(N, device="cuda")[None], R.theta_of(base, D))
    tol = 2 * ref.abs() * HALF[torch.bfloat16] + 2 * R.rope_slack(x, D, False, 1.0, 0)
    R.close(got, pack.double(), tol, "rope against the pre-pass")


@pytest.mark.parametrize("inter,rot,scale", [(False, 64, 1.0), (True, 32, 1.3)])
def test_rope_inverse_is_the_gradient(inter, rot, scale):
    B, T, H, D = 2, 9, 3, 64
    x, dy = randn((B, T, H, D), 11, torch.float32), randn((B, T, H, D), 12, torch.float32)
    pos = ints([[1000 * b + t for t in range(T)] for b in range(B)])
    th = R.theta_of(1e4, rot)
    kw = dict(rotary_dim=rot, interleaved=inter, scale=scale)
    got = atf.rope_apply(dy, None, pos, 1e4, inverse=True, **kw)
    x64 = x.double().requires_grad_()
    a = pos.double()[..., None] * torch.as_tensor(th, device="cuda")
    c, s = scale * a.cos()[:, :, None], scale * a.sin()[:, :, None]
    r = torch.arange(rot // 2, device="cuda")
    i, j = (2 * r, 2 * r + 1) if inter else (r, r + rot // 2)
    rest = x64[..., rot:]
    loss = ((x64[..., i] * c - x64[..., j] * s) * dy[..., i].double()).sum() + \
        ((x64[..., j] * c + x64[..., i] * s) * dy[..., j].double()).sum() + (rest * dy[..., rot:].double()).sum()
    loss.backward()
    R.close(got, x64.grad, x64.grad.abs() * 2.0 ** -24 + R.rope_slack(dy, rot, inter, scale, 0), "gradient")
    # Against differences of the forward call: the map is linear, so a step of any size is exact up to fp32.
    e = randn((B, T, H, D), 13, torch.float32)
    f = lambda y: (atf.rope_apply(y, None, pos, 1e4, **kw).double() * dy.double()).sum()  # noqa: E731
    lhs, rhs = float(f(x + e) - f(x - e)) / 2, float((got.double() * e.double()).sum())
    room = float((R.rope_slack(x.abs() + e.abs(), rot, inter, scale, 0) * dy.double().abs()).sum()) * 3 + 1e-6 * abs(lhs)
    room += float(((x.abs() + e.abs()).double() * dy.double().abs()).sum()) * 2.0 ** -22
    assert abs(lhs - rhs) <= room


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D,Hkv,page,B,T,lens,counts", [
    (64, 2, 64, 1, 1, [0], None),
    (128, 4, 128, 3, 70, [60, 0, 127], [70, 1, 33]),
    (64, 1, 192, 2, 200, [191, 500], [0, 200]),
    (128, 8, 64, 2, 17, [1000, 63], [-3, 40]),
])
def test_append_equals_its_definition(packed, D, Hkv, page, B, T, lens, counts):
    base = 5e5
    kv = randn((B, T, 2 * Hkv, D), 21)
    k, v = kv[:, :, :Hkv], kv[:, :, Hkv:]
    live = [min(max(0, c), T) for c in counts] if counts else [T] * B
    c = R.Cache(B, max((n + T + page - 1) // page for n in lens), page, Hkv, D, packed, 22)
    for given in (False, True):
        pos = torch.as_tensor(np.random.default_rng(4).integers(0, 1 << 20, (B, T)), dtype=torch.int32, device="cuda") if given else None
        got = c.clone()
        atf.cache_append(k, v, got.kpages, got.vpages, c.block_table, ints(lens), page, base, positions=pos,
                         counts=ints(counts) if counts else None, kv_layout=c.layout)
        seen = got.clone()
        for b in range(B):
            slots = lens[b] + torch.arange(live[b], device="cuda")
            if not live[b]:
                continue
            gk, gv = got.read(b, slots)
            x = k[b:b + 1, :live[b]]
            ref = R.rope(x, (pos[b:b + 1, :live[b]] if given else slots[None]), R.theta_of(base, D))
            R.close(gk[None], ref, ref.abs() * 2.0 ** -8 + R.rope_slack(x, D, False, 1.0, 0), "key")
            assert torch.equal(gv, v[b, :live[b]])
            nan = torch.full_like(gk, math.nan)
            seen.write(b, slots, nan, torch.full_like(gv, math.nan))
        assert bool(torch.isnan(seen.kpages).all()) and bool(torch.isnan(seen.vpages).all())  # nothing else was written


def test_append_unrotated_feeds_the_rotating_decode():
    B, T, Hq, Hkv, D, page, base = 2, 300, 4, 2, 128, 64, 1e6
    k, v, q = randn((B, T, Hkv, D), 31), randn((B, T, Hkv, D), 32), randn((B, Hq, D), 33)
    lens, zero = ints([T, T]), ints([0, 0])
    outs = []
    for rotated in (False, True):
        c = R.Cache(B, 5, page, Hkv, D, False, 34, fill=0.0)
        atf.cache_append(k, v, c.kpages, c.vpages, c.block_table, zero, page, base, kcache_rotated=rotated)
        if not rotated:
            assert torch.equal(c.read(0, torch.arange(T, device="cuda"))[0], k[0])
        outs.append(atf.decode_paged(q, c.kpages, c.vpages, c.block_table, lens, page, base, 8.0, kcache_rotated=rotated,
                                     out_dtype=torch.float32))
    # Both calls keep |diff| <= 1e-2 against the oracle (tests/parity.py).
    assert float((outs[0] - outs[1]).abs().max()) <= 2e-2


# ------------------------------------------------------------------ tree attention
def run_tree(D, Hq, Hkv, page, packed, lens, T, counts, kind, k, base=1e4, seed=41, out_dtype=torch.bfloat16, at=0, strided=False):
    """One call against the definition; returns the cache and the outputs."""
    B = len(lens)
    live = [min(max(0, c), T) for c in counts] if counts else [T] * B
    c = R.Cache(B, max(-(-(n + t) // page) for n, t in zip(lens, live)) + 1, page, Hkv, D, packed, seed)
    for b in range(B):
        n = lens[b] + live[b]
        if n:
            c.write(b, torch.arange(n, device="cuda"), randn((n, Hkv, D), seed + 10 + b), randn((n, Hkv, D), seed + 20 + b))
    q = randn((B, T, Hq + 3, D), seed + 1)[:, :, :Hq] if strided else randn((B, T, Hq, D), seed + 1)
    pos = mask = None
    rows = torch.arange(T, device="cuda", dtype=torch.int32)
    if kind == "chain":
        m, p = torch.ones((B, T, T), dtype=torch.bool, device="cuda").tril(), ints(lens)[:, None] + rows
    elif kind == "tree":
        mask, depth = R.random_tree(B, T, seed + 2)
        pos = ints(lens)[:, None] + depth + at
        m, p = mask, pos
    else:  # any mask, any positions: entries above the diagonal, hidden selves, rows of zeros
        g = torch.Generator().manual_seed(seed + 3)
        mask = (torch.rand((B, T, T), generator=g) < 0.4).cuda()
        mask[:, 0] = False
        pos = torch.randint(0, 400, (B, T), generator=g).to(torch.int32).cuda() + at
        m, p = mask, pos
    out = torch.full((B, T, Hq, D), 7.0, dtype=out_dtype, device="cuda")
    lse = torch.full((B, Hq, T), 7.0, device="cuda")
    kw = dict(tree_mask=mask, positions=pos, counts=ints(counts) if counts else None, kv_layout=c.layout)
    call = lambda o, l: atf.tree_decode_paged(q, c.kpages, c.vpages, c.block_table, ints(lens), page, base, k, out=o, lse=l, **kw)  # noqa: E731
    call(out, lse)
    ref, rlse, err, lerr = R.tree(q, c, lens, live, p, m, R.theta_of(base, D), k)
    for b in range(B):
        t = live[b]
        assert bool((out[b, t:] == 7.0).all()) and bool((lse[b, :, t:] == 7.0).all())
        if t:
            tol = err[b, :t] + ref[b, :t].abs() * HALF[out_dtype] + 1e-30
            R.close(out[b, :t], ref[b, :t], tol.expand_as(ref[b, :t]), f"out of sequence {b}")
            R.close(lse[b, :, :t], rlse[b, :, :t], lerr[b, :, :t], f"lse of sequence {b}")
    return c, q, kw, out, lse, call


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv,page,lens,T,counts,kind,k", [
    (64, 1, 1, 64, [0], 1, None, "chain", math.inf),                     # one token, nothing cached
    (64, 14, 2, 64, [1021], 7, None, "tree", 8.0),
    (128, 24, 8, 64, [700, 5, 129, 0], 16, [16, 3, 9, 1], "tree", 2.0),
    (128, 28, 4, 128, [1000, 128], 1, None, "chain", 16.0),
    (128, 28, 4, 256, [513], 64, None, "tree", 1.0),                     # 448 rows of a KV head
    (64, 4, 4, 192, [191, 192, 193], 33, [33, 0, 20], "tree", 0.5),
    (128, 4, 1, 64, [300, 1], 50, None, "any", 1.0),                     # rows that see nothing in the tree
    (64, 3, 1, 64, [0, 64], 40, [40, 39], "any", 0.25),                  # and nothing cached: 0 and -inf
    (64, 2, 2, 64, [127], 130, None, "chain", 4.0),                      # the tree itself spans tiles
    (128, 2, 1, 64, [90], 20, None, "tree", 0.0),                        # only distance 0 (and less) keeps a pair
    (64, 40, 1, 64, [257], 5, None, "chain", math.inf),                  # 40 query heads of one KV head
    (128, 1, 1, 128, [3000], 3, None, "tree", 64.0),
])
def test_tree_equals_its_definition(packed, D, Hq, Hkv, page, lens, T, counts, kind, k):
    run_tree(D, Hq, Hkv, page, packed, lens, T, counts, kind, k)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_tree_fp32_output_strided_queries_far_positions(packed, D):
    # Positions near 2^31 with a short cache: every prefix key is far, the nodes near one another.
    run_tree(D, 6, 2, 64, packed, [150, 20], 12, None, "tree", 3.0, at=(1 << 31) - 400, out_dtype=torch.float32, strided=True)
    run_tree(D, 6, 2, 64, packed, [150, 20], 12, None, "any", math.inf, at=(1 << 31) - 500, out_dtype=torch.float32)


@pytest.mark.parametrize("packed", [False, True])
def test_tree_long_and_ragged(packed):
    run_tree(128, 7, 1, 256, packed, [9000, 1, 4097, 0, 2500], 16, [16, 16, 2, 5, 0], "tree", 16.0, base=1e7)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv,page,lens,T,k", [
    (128, 7, 1, 128, [200033], 1, math.inf),      # ten key tiles per SM, one row group, copies of the rows
    (64, 20, 2, 64, [120001, 3, 40007], 2, 8.0),
    (128, 6, 2, 64, [100100, 517], 9, 16.0),      # 27 rows
    (64, 9, 1, 256, [250001], 6, 2.0),            # 54 rows: two copies
    (128, 14, 2, 256, [90000, 60001], 21, 16.0),  # 147 rows: two row tiles
])
def test_tree_many_tiles_in_a_row(packed, D, Hq, Hkv, page, lens, T, k):
    # Long runs of key tiles on every SM, with tiles of nodes after them: every pipeline wraps many times.
    run_tree(D, Hq, Hkv, page, packed, lens, T, None, "tree", k, base=1e6, seed=311)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv,page,lens,T,counts,kind,k", [
    (128, 8, 1, 64, [300, 40], 300, [300, 150], "tree", 2.0),  # 2400 rows: three groups of seven row tiles, the last not full
    (64, 16, 2, 128, [1100, 7, 64], 129, [129, 128, 1], "any", 1.0),  # 1032 rows: two groups, of which one sequence has one row tile
    (64, 32, 1, 64, [700], 65, None, "chain", 4.0),  # 2080 rows: three groups of six
])
def test_tree_of_many_rows(packed, D, Hq, Hkv, page, lens, T, counts, kind, k):
    # More rows than the row tiles that walk the keys together: several groups of them, some without rows.
    run_tree(D, Hq, Hkv, page, packed, lens, T, counts, kind, k, seed=321)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("idle", [0, 40])
def test_tree_of_many_sequences(packed, idle):
    # More sequences than a warp has lanes, the first `idle` of them without a node.
    B, T = 75, 3
    lens = [(i * 137) % 700 for i in range(B)]
    counts = [0 if b < idle else (b * 5) % (T + 2) for b in range(B)]
    run_tree(64, 4, 2, 64, packed, lens, T, counts, "tree", 1.0, seed=331)
    if not idle:
        run_tree(128, 2, 1, 64, packed, lens, T, None, "chain", 4.0, seed=341)


@pytest.mark.parametrize("packed", [False, True])
def test_tree_every_key_counts_once(packed):
    # Uniform weights (queries of zeros) over one-hot values by key tile: output dim d is the share of the keys
    # in tiles d mod D, which one lost or doubled run of keys would change.
    B, T, Hq, Hkv, D, page, L = 3, 3, 6, 2, 64, 128, 70017
    c = R.Cache(B, (L + T + page - 1) // page, page, Hkv, D, packed, 321)
    slots = torch.arange(L + T, device="cuda")
    v = torch.nn.functional.one_hot(slots // 128 % D, D).to(torch.bfloat16)[:, None].expand(-1, Hkv, -1).contiguous()
    for b in range(B):
        c.write(b, slots, randn((L + T, Hkv, D), 322 + b), v)
    out, lse = atf.tree_decode_paged(torch.zeros((B, T, Hq, D), dtype=torch.bfloat16, device="cuda"), c.kpages, c.vpages, c.block_table,
                                     ints([L] * B), page, 1e4, 8.0, kv_layout=c.layout, return_lse=True, out_dtype=torch.float32)
    for i in range(T):
        n = L + i + 1
        want = torch.bincount(slots[:n] // 128 % D, minlength=D).double() / n
        # Powers of two times counts: every product and sum is exact in fp32, one division at the end.
        assert float(((out[:, i].double() - want).abs() / want).max()) <= 2.0 ** -22
        assert float((lse[:, :, i].double() - math.log(n)).abs().max()) <= 2.0 ** -18


@pytest.mark.parametrize("packed", [False, True])
def test_tree_scaled_frequencies(packed):
    import scaled
    D, Hq, Hkv, page, T, L = 128, 8, 2, 64, 6, 400
    th = scaled.llama3_scaled_theta(D, 5e5)
    c = R.Cache(1, 8, page, Hkv, D, packed, 51)
    c.write(0, torch.arange(L, device="cuda"), randn((L, Hkv, D), 52), randn((L, Hkv, D), 53))
    k, v, q = randn((1, T, Hkv, D), 54), randn((1, T, Hkv, D), 55), randn((1, T, Hq, D), 56)
    mask, depth = R.random_tree(1, T, 57)
    pos, lens = depth + L, ints([L])
    atf.cache_append(k, v, c.kpages, c.vpages, c.block_table, lens, page, 1e4, positions=pos, kv_layout=c.layout, theta=th)
    out, lse = atf.tree_decode_paged(q, c.kpages, c.vpages, c.block_table, lens, page, 1e4, 4.0, tree_mask=mask, positions=pos,
                                     kv_layout=c.layout, theta=th, return_lse=True, out_dtype=torch.float32)
    ref, rlse, err, lerr = R.tree(q, c, [L], [T], pos, mask, th, 4.0)
    R.close(out, ref, err.expand_as(ref) + ref.abs() * 2.0 ** -24, "out")
    R.close(lse, rlse, lerr, "lse")


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_tree_hidden_nodes_may_hold_anything(packed, bad):
    # Node 2's key and value and node 5's value are not finite; a row that sees neither is what it was, a row that
    # sees node 2 or 5 is not finite in the dims concerned.
    D, Hq, Hkv, page, T, L = 128, 4, 2, 64, 9, 200
    c, q, kw, out, lse, call = run_tree(D, Hq, Hkv, page, packed, [L], T, None, "tree", 2.0, seed=61)
    mask = kw["tree_mask"]
    kk, vv = c.read(0, torch.tensor([L + 2, L + 5], device="cuda"))
    kk, vv = kk.clone(), vv.clone()
    kk[0] = bad
    vv[0] = bad
    vv[1, :, 3] = bad
    c.write(0, torch.tensor([L + 2, L + 5], device="cuda"), kk, vv)
    out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
    call(out2, lse2)
    for i in range(T):
        two, five = bool(mask[0, i, 2]), bool(mask[0, i, 5])
        if not two:
            assert torch.equal(lse2[0, :, i], lse[0, :, i])
            keep = [d for d in range(D) if not (five and d == 3)]
            assert torch.equal(out2[0, i][:, keep], out[0, i][:, keep]), i
            if five:
                assert not bool(torch.isfinite(out2[0, i, :, 3]).any())
        else:
            assert not bool(torch.isfinite(out2[0, i]).any())


@pytest.mark.parametrize("packed", [False, True])
def test_tree_pruned_pairs_may_hold_anything(packed):
    # A key element whose pair is pruned for every query takes no part, whatever it holds.
    D, Hq, Hkv, page, T, L, base, k = 64, 4, 2, 64, 4, 300, 1e4, 0.5
    c, q, kw, out, lse, call = run_tree(D, Hq, Hkv, page, packed, [L], T, None, "chain", k, seed=71, base=base)
    slots = torch.arange(L, device="cuda")
    kk, vv = c.read(0, slots)
    kk = kk.clone()
    for r, w in enumerate(R.windows(R.theta_of(base, D), k)):
        far = slots < L - w  # pruned for every query (positions L..L+T-1)
        kk[far, :, r] = math.nan
        kk[far, :, r + D // 2] = math.inf
    c.write(0, slots, kk, vv)
    out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
    call(out2, lse2)
    assert torch.equal(out2, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("packed", [False, True])
def test_tree_of_one_token_is_the_decode(packed):
    B, Hq, Hkv, D, page, base, k = 3, 8, 2, 128, 64, 1e6, 16.0
    lens = [900, 2047, 130]
    c = R.Cache(B, 32, page, Hkv, D, packed, 81)
    for b in range(B):
        c.write(b, torch.arange(lens[b], device="cuda"), randn((lens[b], Hkv, D), 82 + b), randn((lens[b], Hkv, D), 92 + b))
    q = randn((B, Hq, D), 99)
    want = atf.decode_paged(q, c.kpages, c.vpages, c.block_table, ints(lens), page, base, k, kcache_rotated=True,
                            kv_layout=c.layout, out_dtype=torch.float32)
    got = atf.tree_decode_paged(q[:, None], c.kpages, c.vpages, c.block_table, ints([n - 1 for n in lens]), page, base, k,
                                kv_layout=c.layout, out_dtype=torch.float32)
    # Both keep |diff| <= 1e-2 against the definition.
    assert float((got[:, 0] - want).abs().max()) <= 2e-2


def test_tree_bad_pages_are_reported():
    D, Hq, Hkv, page = 128, 4, 2, 64
    c, q, kw, out, lse, call = run_tree(D, Hq, Hkv, page, True, [300, 290], 8, None, "tree", 4.0, seed=101)
    for bad in (c.n, -1, 1 << 30):
        table = c.block_table.clone()
        table[0, 2] = bad
        good = torch.zeros_like(out)
        atf.tree_decode_paged(q, c.kpages, c.vpages, table, ints([300, 290]), page, 1e4, 4.0, out=good, **kw)
        assert atf.device_status() == atf.ERR_BAD_PAGE
        assert torch.equal(good[1], out[1])  # the other sequence is not concerned
    # More tokens than the table has room for.
    atf.tree_decode_paged(q, c.kpages, c.vpages, c.block_table, ints([10 ** 6, 290]), page, 1e4, 4.0, **kw)
    assert atf.device_status() == atf.ERR_BAD_PAGE


def test_append_and_copies_report_bad_pages_and_write_elsewhere_only():
    B, T, Hkv, D, page = 2, 10, 2, 64, 64
    c = R.Cache(B, 2, page, Hkv, D, True, 111)
    k, v = randn((B, T, Hkv, D), 112), randn((B, T, Hkv, D), 113)
    table = c.block_table.clone()
    table[0, 0] = c.n
    atf.cache_append(k, v, c.kpages, c.vpages, table, ints([0, 125]), page, 1e4, kv_layout="PACKED")  # 7 slots past the row
    assert atf.device_status() == atf.ERR_BAD_PAGE
    assert int((~torch.isnan(c.vpages)).sum()) == 3 * Hkv * D
    atf.cache_append(k, v, c.kpages, c.vpages, c.block_table, ints([-20, 0]), page, 1e4, kv_layout="PACKED")
    assert atf.device_status() == atf.ERR_BAD_PAGE
    before = c.clone()
    atf.cache_copy_pages(c.kpages, c.vpages, ints([0, c.n]), ints([-1, 1]), page, kv_layout="PACKED")
    assert atf.device_status() == atf.ERR_BAD_PAGE
    atf.cache_compact(c.kpages, c.vpages, c.block_table, ints([0, 0]), ints([[-1], [999]]), ints([1, 1]), page, kv_layout="PACKED")
    assert atf.device_status() == atf.ERR_BAD_PAGE
    assert torch.equal(before.vpages.view(torch.int16), c.vpages.view(torch.int16))
    assert torch.equal(before.kpages.view(torch.int16), c.kpages.view(torch.int16))


# ------------------------------------------------------------------ compaction and page copies
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D,Hkv,page,lens,path,accepted", [
    (64, 2, 64, [60], [[0, 2, 5, 9]], [4]),
    (128, 4, 128, [0, 500, 127], [[1, 3, 4], [0, 1, 2], [5, 6, 7]], [3, 0, 2]),
    (64, 1, 64, [63, 100], [[3, 2, 1, 0], [2, 2, 0, 2]], [4, 9]),      # any order, an index twice, more than the path holds
    (128, 1, 192, [10], [list(range(1000, 0, -1))], [1000]),
])
def test_compact_equals_its_definition(packed, D, Hkv, page, lens, path, accepted):
    B, M = len(path), len(path[0])
    c = R.Cache(B, max(-(-(n + max(map(max, path)) + 1) // page) for n in lens) + 1, page, Hkv, D, packed, 121)
    c.kpages.copy_(randn(c.kpages.shape, 122))
    c.vpages.copy_(randn(c.vpages.shape, 123))
    want = c.clone()
    for b in range(B):
        n = min(accepted[b], M)
        if n:
            k, v = c.read(b, lens[b] + torch.tensor(path[b][:n], device="cuda"))
            want.write(b, lens[b] + torch.arange(n, device="cuda"), k, v)
    new = atf.cache_compact(c.kpages, c.vpages, c.block_table, ints(lens), ints(path), ints(accepted), page, kv_layout=c.layout)
    assert new.tolist() == [n + min(a, M) for n, a in zip(lens, accepted)]
    assert torch.equal(c.kpages, want.kpages) and torch.equal(c.vpages, want.vpages)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D,Hkv,page,tokens", [(64, 2, 64, None), (128, 4, 128, [0, 1, 128, 77]), (64, 1, 192, [191, 500, -4, 3])])
def test_copy_pages_equals_its_definition(packed, D, Hkv, page, tokens):
    c = R.Cache(1, 9, page, Hkv, D, packed, 131)
    c.kpages.copy_(randn(c.kpages.shape, 132))
    c.vpages.copy_(randn(c.vpages.shape, 133))
    src, dst = [3, 3, 0, 7], [1, 11, 5, 2]
    want = c.clone()
    for e in range(4):
        n = page if tokens is None else min(max(tokens[e], 0), page)
        want.vpages[dst[e], :n] = c.vpages[src[e], :n]
        if packed:
            want.kpages[dst[e], :, :, :n] = c.kpages[src[e], :, :, :n]
        else:
            want.kpages[dst[e], :n] = c.kpages[src[e], :n]
    atf.cache_copy_pages(c.kpages, c.vpages, ints(src), ints(dst), page, tokens=ints(tokens) if tokens else None, kv_layout=c.layout)
    assert torch.equal(c.kpages, want.kpages) and torch.equal(c.vpages, want.vpages)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 14, 2), (128, 8, 2)])
def test_drafted_steps_end_in_the_cache_of_plain_decoding(packed, D, Hq, Hkv):
    """Prompt appended, then three steps of append -> attend -> compact with a tree each; then the sequence is forked. The
    cache must hold the accepted tokens at their positions, and every attended row the definition's output."""
    B, page, base, kwin, T = 2, 64, 1e5, 4.0, 11
    prompts = [130, 61]
    c = R.Cache(B, 5, page, Hkv, D, packed, 141)
    P = max(prompts)
    k, v = randn((B, P, Hkv, D), 142), randn((B, P, Hkv, D), 143)
    lens = ints([0, 0])
    atf.cache_append(k, v, c.kpages, c.vpages, c.block_table, lens, page, base, counts=ints(prompts), kv_layout=c.layout)
    kept = [[(k[b, i], v[b, i]) for i in range(prompts[b])] for b in range(B)]
    lens = ints(prompts)
    rng = np.random.default_rng(144)
    for step in range(3):
        mask, depth = R.random_tree(B, T, 145 + step)
        pos = lens[:, None] + depth
        k, v, q = (randn((B, T, h, D), 150 + 10 * step + i) for i, h in enumerate((Hkv, Hkv, Hq)))
        atf.cache_append(k, v, c.kpages, c.vpages, c.block_table, lens, page, base, positions=pos, kv_layout=c.layout)
        out, lse = atf.tree_decode_paged(q, c.kpages, c.vpages, c.block_table, lens, page, base, kwin, tree_mask=mask,
                                         positions=pos, kv_layout=c.layout, return_lse=True, out_dtype=torch.float32)
        ref, rlse, err, lerr = R.tree(q, c, lens.tolist(), [T] * B, pos, mask, R.theta_of(base, D), kwin)
        R.close(out, ref, err.expand_as(ref) + ref.abs() * 2.0 ** -24, "out")
        R.close(lse, rlse, lerr, "lse")
        leaf = [int(rng.integers(0, T)) for _ in range(B)]
        paths = [[j for j in range(T) if bool(mask[b, leaf[b], j])] for b in range(B)]
        M = max(map(len, paths))
        lens = atf.cache_compact(c.kpages, c.vpages, c.block_table, lens, ints([p + [0] * (M - len(p)) for p in paths]),
                                 ints([len(p) for p in paths]), page, kv_layout=c.layout)
        for b in range(B):
            kept[b] += [(k[b, j], v[b, j]) for j in paths[b]]
    # The same tokens appended once, at their slots.
    n = lens.tolist()
    assert n == [len(x) for x in kept]
    plain = R.Cache(B, 5, page, Hkv, D, packed, 141)
    for b in range(B):
        kk, vv = (torch.stack([x[i] for x in kept[b]])[None] for i in (0, 1))
        atf.cache_append(kk, vv, plain.kpages, plain.vpages, plain.block_table[b:b + 1].contiguous(), ints([0]), page, base,
                         kv_layout=c.layout)
        for a, z in zip(c.read(b, torch.arange(n[b], device="cuda")), plain.read(b, torch.arange(n[b], device="cuda"))):
            assert torch.equal(a, z)
    # A fork of sequence 0: full pages shared, the last one copied to a page of its own.
    used = set(c.block_table.flatten().tolist())
    free = next(p for p in range(c.n) if p not in used)
    last = (n[0] - 1) // page
    table = torch.cat((c.block_table, c.block_table[:1]))
    table[2, last] = free
    atf.cache_copy_pages(c.kpages, c.vpages, table[0, last:last + 1].contiguous(), ints([free]), page, tokens=ints([n[0] - last * page]),
                         kv_layout=c.layout)
    q = randn((1, 1, Hq, D), 190)
    a, z = (atf.tree_decode_paged(q, c.kpages, c.vpages, table[i:i + 1].contiguous(), ints([n[0] - 1]), page, base, kwin,
                                  kv_layout=c.layout) for i in (0, 2))
    assert torch.equal(a, z)


def test_a_captured_step_replays_on_new_inputs_beside_eager_calls():
    """append -> attend -> compact captured once, replayed after the inputs changed in place; an eager call of another
    shape runs between replays with a workspace of its own."""
    B, T, Hq, Hkv, D, page, base, kwin = 2, 5, 8, 2, 128, 64, 1e6, 8.0
    c = R.Cache(B, 40, page, Hkv, D, True, 201, fill=0.0)
    c.kpages.copy_(randn(c.kpages.shape, 202))
    c.vpages.copy_(randn(c.vpages.shape, 203))
    k, v, q = randn((B, T, Hkv, D), 204), randn((B, T, Hkv, D), 205), randn((B, T, Hq, D), 206)
    mask, depth = R.random_tree(B, T, 207)
    lens, pos = ints([2000, 100]), torch.zeros((B, T), dtype=torch.int32, device="cuda")
    pos.copy_(ints([2000, 100])[:, None] + depth)
    path, acc = ints([[0, 1], [0, 1]]), ints([2, 1])
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros((B, T, Hq, D), device="cuda"), torch.zeros((B, Hq, T), device="cuda")
    ws = torch.empty(atf.tree_decode_workspace_bytes(B, T, Hq, Hkv, D), dtype=torch.uint8, device="cuda")

    def step():
        atf.cache_append(k, v, c.kpages, c.vpages, c.block_table, lens, page, base, positions=pos, kv_layout="PACKED")
        atf.tree_decode_paged(q, c.kpages, c.vpages, c.block_table, lens, page, base, kwin, tree_mask=mask, positions=pos,
                              kv_layout="PACKED", out=out, lse=lse, workspace=ws)
        atf.cache_compact(c.kpages, c.vpages, c.block_table, lens, path, acc, page, new_seqlens=new, kv_layout="PACKED")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in ([1500, 7], [2222, 0]):
        lens.copy_(ints(n))
        pos.copy_(ints(n)[:, None] + depth)
        q.copy_(randn(q.shape, 210 + n[0]))
        k.copy_(randn(k.shape, 211 + n[0]))
        before = c.clone()
        graph.replay()
        atf.tree_decode_paged(q[:, :1], c.kpages, c.vpages, c.block_table, lens, page, base, kwin, kv_layout="PACKED")
        torch.cuda.synchronize()
        got, got_lse = out.clone(), lse.clone()
        after = c.clone()
        c.kpages.copy_(before.kpages), c.vpages.copy_(before.vpages)
        step()
        assert torch.equal(got, out) and torch.equal(got_lse, lse)
        assert torch.equal(after.kpages, c.kpages) and torch.equal(after.vpages, c.vpages)
        assert new.tolist() == [n[0] + 2, n[1] + 1]


def test_tree_two_streams_at_once_and_again():
    """Calls on two streams at the same time, each with its own workspace, give what each gives alone, every time."""
    shapes = [(128, 28, 4, 128, True, [5000, 3], 24, None, "tree", 16.0), (64, 14, 2, 64, False, [2500], 9, None, "tree", 8.0)]
    runs = [run_tree(*s, seed=221 + i) for i, s in enumerate(shapes)]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for s, (c, q, kw, out, lse, call) in zip(streams, runs):
            with torch.cuda.stream(s):
                o, l = torch.empty_like(out), torch.empty_like(lse)
                call(o, l)
                outs.append((o, l))
        torch.cuda.synchronize()
        for (o, l), (c, q, kw, out, lse, call) in zip(outs, runs):
            assert torch.equal(o, out) and torch.equal(l, lse)


def test_append_unrotated_copies_every_bit():
    """Keys stored un-rotated keep infinities, NaN and signed zeros, and do not spread them to their partners."""
    B, T, Hkv, D, page = 1, 70, 2, 64, 64
    k, v = randn((B, T, Hkv, D), 231), randn((B, T, Hkv, D), 232)
    k[:, 3, :, 5], k[:, 4, :, 40], k[:, 5, :, 9], k[:, 6, :, 10] = math.inf, -math.inf, math.nan, -0.0
    k[:, 6, :, 42] = -1.0
    c = R.Cache(B, 2, page, Hkv, D, False, 233, fill=0.0)
    atf.cache_append(k, v, c.kpages, c.vpages, c.block_table, ints([9]), page, 1e4, kcache_rotated=False)
    slots = torch.arange(9, 9 + T, device="cuda")
    where, at = c.block_table[0].long()[slots // page], slots % page
    assert torch.equal(c.kpages[where, at].view(torch.int16), k[0].view(torch.int16))
    assert torch.equal(c.vpages[where, at].view(torch.int16), v[0].view(torch.int16))


def test_a_call_on_another_stream_does_not_wait_for_the_current_one():
    """Outputs, zeros behind the last node and workspaces of a call with stream= belong to that stream: work still queued
    on the current one neither holds them back nor overwrites them."""
    c, q, kw, want, wlse, call = run_tree(128, 8, 2, 64, True, [300, 90], 8, [8, 3], "tree", 8.0, seed=241)
    lens, other = ints([300, 90]), torch.cuda.Stream()
    path, acc, pos = ints([[0, 1], [0, 1]]), ints([2, 1]), ints([[5] * 8] * 2)
    x = torch.ones((4096, 4096), device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    for _ in range(40):
        x = x @ x * 0.0
    out, lse = atf.tree_decode_paged(q, c.kpages, c.vpages, c.block_table, lens, 64, 1e4, 8.0, return_lse=True, stream=other, **kw)
    turned = atf.rope_apply(q, None, pos, 1e4, stream=other)
    new = atf.cache_compact(c.kpages, c.vpages, c.block_table, lens, path, acc, 64, kv_layout="PACKED", stream=other)
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1, :3], want[1, :3]) and not bool(out[1, 3:].any())
    assert torch.equal(lse[0], wlse[0]) and torch.equal(lse[1, :, :3], wlse[1, :, :3])
    assert torch.equal(turned, atf.rope_apply(q, None, pos, 1e4))
    assert new.tolist() == [302, 91]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D,Hq,T", [(64, 4, 3), (128, 8, 40)])
def test_tree_waits_that_run_out_are_reported_and_leave_the_gpu_usable(packed, D, Hq, T):
    # Every sequence is about one CTA's run, its nodes in the last of 161 tiles: the warps that take the
    # nodes' tiles wait through the whole run, far beyond a limit of 1 us.
    B, page, L = 148, 256, 160 * 128 + 5
    c = R.Cache(B, L // page + 1, page, 1, D, packed, 411)
    c.kpages.copy_(randn(c.kpages.shape, 412))
    c.vpages.copy_(randn(c.vpages.shape, 413))
    q, lens = randn((B, T, Hq, D), 414), ints([L] * B)
    small = run_tree(D, Hq, 1, 64, packed, [200, 3], T, None, "tree", 4.0, seed=415)
    call = lambda: atf.tree_decode_paged(q, c.kpages, c.vpages, c.block_table, lens, page, 1e4, 8.0, kv_layout=c.layout,  # noqa: E731
                                         return_lse=True)
    want, wlse = call()
    torch.cuda.synchronize()
    assert atf.device_status() == 0
    try:
        atf.set_wait_limit_ms(0.001)
        call()
        assert atf.device_status() == atf.ERR_TIMEOUT
        out, lse = torch.empty_like(small[3]), torch.empty_like(small[4])
        small[5](out, lse)  # producers that are done early, whichever of the other waits runs out
        assert atf.device_status() in (0, atf.ERR_TIMEOUT)
    finally:
        atf.set_wait_limit_ms(2000.0)
    got, glse = call()
    assert torch.equal(got, want) and torch.equal(glse, wlse)
    small[5](out, lse)
    assert torch.equal(out, small[3]) and torch.equal(lse, small[4])


@pytest.mark.parametrize("packed", [False, True])
def test_append_of_the_most_tokens_that_a_call_takes(packed):
    # 2^31 - 1 tokens (one, repeated by strides of zero) of which five are live: the last block's threads reach index
    # 2^31 - 1, one past the last token.
    Hkv, D, page, T, live, at = 1, 128, 64, (1 << 31) - 1, 5, 61
    k, v = randn((1, 1, Hkv, D), 421), randn((1, 1, Hkv, D), 422)
    c = R.Cache(1, 2, page, Hkv, D, packed, 423)
    atf.cache_append(k.expand(1, T, Hkv, D), v.expand(1, T, Hkv, D), c.kpages, c.vpages, c.block_table, ints([at]), page, 1e4,
                     counts=ints([live]), kv_layout=c.layout)
    slots = at + torch.arange(live, device="cuda")
    gk, gv = c.read(0, slots)
    x = k.expand(1, live, Hkv, D)
    ref = R.rope(x, slots[None], R.theta_of(1e4, D))
    R.close(gk[None], ref, ref.abs() * 2.0 ** -8 + R.rope_slack(x, D, False, 1.0, 0), "key")
    assert torch.equal(gv, v[0].expand(live, Hkv, D))
    assert int((~torch.isnan(c.kpages)).sum()) == int((~torch.isnan(c.vpages)).sum()) == live * Hkv * D


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D,Hq,lens,T", [(64, 4, [300, 290], 8), (128, 6, [700, 20], 30)])
def test_tree_bad_lengths_keep_their_rows_and_bad_pages_are_zeros(packed, D, Hq, lens, T):
    Hkv, page = 2, 64
    c, q, kw, out, lse, call = run_tree(D, Hq, Hkv, page, packed, lens, T, None, "tree", 4.0, seed=431)
    args = (page, 1e4, 4.0)
    room = c.block_table.shape[1] * page
    for bad in (-1, -(1 << 31), room - T + 1, (1 << 31) - 1):
        # Rows of the caller's, and rows made by the call from memory that held something else.
        o, l = torch.full_like(out, 3.0), torch.full_like(lse, 3.0)
        atf.tree_decode_paged(q, c.kpages, c.vpages, c.block_table, ints([bad, lens[1]]), *args, out=o, lse=l, **kw)
        assert atf.device_status() == atf.ERR_BAD_PAGE
        assert bool((o[0] == 3.0).all()) and bool((l[0] == 3.0).all())
        assert torch.equal(o[1], out[1]) and torch.equal(l[1], lse[1])
        junk = [torch.full_like(x, 5.0) for x in (out, out, lse, lse)]
        del junk
        o, l = atf.tree_decode_paged(q, c.kpages, c.vpages, c.block_table, ints([bad, lens[1]]), *args, return_lse=True, **kw)
        assert atf.device_status() == atf.ERR_BAD_PAGE
        assert not bool(o[0].any()) and not bool(l[0].any())
        assert torch.equal(o[1], out[1]) and torch.equal(l[1], lse[1])
    # A page outside the pool: its keys and values count as zeros.
    zeros = c.clone()
    zeros.write(0, torch.arange(2 * page, 3 * page, device="cuda"), *(torch.zeros((page, Hkv, D), dtype=torch.bfloat16, device="cuda"),) * 2)
    ref, rlse, err, lerr = R.tree(q, zeros, lens, [T, T], kw["positions"], kw["tree_mask"], R.theta_of(1e4, D), 4.0)
    for bad in (c.n, -1, (1 << 31) - 1):
        table = c.block_table.clone()
        table[0, 2] = bad
        o, l = atf.tree_decode_paged(q, c.kpages, c.vpages, table, ints(lens), *args, return_lse=True, **kw)
        assert atf.device_status() == atf.ERR_BAD_PAGE
        R.close(o, ref, err.expand_as(ref) + ref.abs() * HALF[torch.bfloat16], "out")
        R.close(l, rlse, lerr, "lse")


@pytest.mark.parametrize("packed", [False, True])
def test_a_negative_length_moves_nothing(packed):
    # Slots that a negative length and a token's index add up to belong to the committed prefix.
    B, T, Hkv, D, page = 2, 10, 2, 64, 64
    c = R.Cache(B, 2, page, Hkv, D, packed, 441)
    c.kpages.copy_(randn(c.kpages.shape, 442))
    c.vpages.copy_(randn(c.vpages.shape, 443))
    k, v = randn((B, T, Hkv, D), 444), randn((B, T, Hkv, D), 445)
    for n in (-3, -9, -(1 << 31)):
        got, want = c.clone(), c.clone()
        atf.cache_append(k, v, got.kpages, got.vpages, c.block_table, ints([n, 7]), page, 1e4, kv_layout=c.layout)
        assert atf.device_status() == atf.ERR_BAD_PAGE
        atf.cache_append(k[1:], v[1:], want.kpages, want.vpages, c.block_table[1:], ints([7]), page, 1e4, kv_layout=c.layout)
        assert torch.equal(got.kpages, want.kpages) and torch.equal(got.vpages, want.vpages)
        got, want = c.clone(), c.clone()
        path = ints([[4, 12, 5, 11, 9, 3]] * 2)
        atf.cache_compact(got.kpages, got.vpages, c.block_table, ints([n, 7]), path, ints([6, 6]), page, kv_layout=c.layout)
        assert atf.device_status() == atf.ERR_BAD_PAGE
        atf.cache_compact(want.kpages, want.vpages, c.block_table[1:], ints([7]), path[1:], ints([6]), page, kv_layout=c.layout)
        assert torch.equal(got.kpages, want.kpages) and torch.equal(got.vpages, want.vpages)


@pytest.mark.parametrize("packed", [False, True])
def test_copying_no_pages_changes_nothing(packed):
    c = R.Cache(1, 2, 64, 2, 64, packed, 451)
    c.kpages.copy_(randn(c.kpages.shape, 452))
    c.vpages.copy_(randn(c.vpages.shape, 453))
    want, none = c.clone(), ints([])
    atf.cache_copy_pages(c.kpages, c.vpages, none, none, 64, kv_layout=c.layout)
    atf.cache_copy_pages(c.kpages, c.vpages, none, none, 64, tokens=none, kv_layout=c.layout)
    assert torch.equal(c.kpages, want.kpages) and torch.equal(c.vpages, want.vpages)
    for bad in (dict(src=ints([1])), dict(tokens=ints([3])), dict(dst=none.long())):  # still refused
        a = {**dict(src=none, dst=none, tokens=None), **bad}
        with pytest.raises((ValueError, TypeError)):
            atf.cache_copy_pages(c.kpages, c.vpages, a["src"], a["dst"], 64, tokens=a["tokens"], kv_layout=c.layout)


def fine_err(keys):
    """What probabilities in two bf16 parts (2^-16 of each) and sums that may truncate move an output by, relative to
    sum p |v|: two products and additions of at most 2^-23 for each key."""
    return 2.0 ** -16 + 2 * keys * 2.0 ** -23


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv,lens,T,kind,dt", [
    (64, 4, 2, [3, 60, 0, 120], 7, "tree", torch.bfloat16),     # rows of 1 to 127 keys, repeated in four copies
    (128, 8, 1, [128, 1, 17], 8, "chain", torch.bfloat16),      # two copies; a row of 129 keys
    (128, 12, 1, [40, 128], 30, "tree", torch.bfloat16),        # three row tiles; a second key tile
    (64, 6, 1, [0, 50], 12, "any", torch.float32),
    (128, 4, 2, [300, 10], 5, "tree", torch.float32),           # fp32 output: longer rows too
    (64, 14, 2, [257, 190], 20, "tree", torch.float32),
    (64, 2, 1, [500], 1, "chain", torch.float32),
])
def test_tree_of_few_keys_or_fp32_output_keeps_its_probabilities(packed, D, Hq, Hkv, lens, T, kind, dt):
    # Small scores (their error stays far below a bf16 rounding of P) over values of both signs.
    B, page, base, k, seed = len(lens), 64, 1e4, 8.0, 461
    c = R.Cache(B, -(-(max(lens) + T) // page), page, Hkv, D, packed, seed)
    for b in range(B):
        n = lens[b] + T
        c.write(b, torch.arange(n, device="cuda"), randn((n, Hkv, D), seed + 10 + b), randn((n, Hkv, D), seed + 20 + b))
    q = (randn((B, T, Hq, D), seed + 1, torch.float32) / 8).to(torch.bfloat16)
    rows = torch.arange(T, device="cuda", dtype=torch.int32)
    mask, pos = torch.ones((B, T, T), dtype=torch.bool, device="cuda").tril(), ints(lens)[:, None] + rows
    if kind == "tree":
        mask, depth = R.random_tree(B, T, seed + 2)
        pos = ints(lens)[:, None] + depth
    elif kind == "any":
        mask = (torch.rand((B, T, T), generator=torch.Generator().manual_seed(seed + 3)) < 0.4).cuda()
    out, lse = atf.tree_decode_paged(q, c.kpages, c.vpages, c.block_table, ints(lens), page, base, k, tree_mask=mask, positions=pos,
                                     kv_layout=c.layout, out_dtype=dt, return_lse=True)
    ref, rlse, err, lerr = R.tree(q, c, lens, [T] * B, pos, mask, R.theta_of(base, D), k, p_err=fine_err(max(lens) + T))
    R.close(out, ref, err.expand_as(ref) + ref.abs() * (HALF[dt] + 2.0 ** -21) + 1e-30, "out")
    R.close(lse, rlse, lerr, "lse")


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 2), (128, 8, 1)])
def test_tree_of_one_token_is_the_decode_for_short_sequences(packed, D, Hq, Hkv):
    # The decode computes sequences of up to 128 tokens in fp32.  (Scores here are small: queries of 1/8.)
    lens, page, base, k = [1, 2, 9, 33, 64, 65, 127, 128], 64, 1e6, 16.0
    c = R.Cache(len(lens), 2, page, Hkv, D, packed, 471)
    for b, n in enumerate(lens):
        c.write(b, torch.arange(n, device="cuda"), randn((n, Hkv, D), 472 + b), randn((n, Hkv, D), 492 + b))
    q = (randn((len(lens), Hq, D), 512, torch.float32) / 8).to(torch.bfloat16)
    want = atf.decode_paged(q, c.kpages, c.vpages, c.block_table, ints(lens), page, base, k, kcache_rotated=True, kv_layout=c.layout,
                            out_dtype=torch.float32)
    before = ints([n - 1 for n in lens])
    ones = torch.ones((len(lens), 1, 1), dtype=torch.bool, device="cuda")
    ref, _, err, _ = R.tree(q[:, None], c, before, [1] * len(lens), before[:, None], ones, R.theta_of(base, D), k, p_err=fine_err(128))
    for dt in (torch.float32, torch.bfloat16):
        got = atf.tree_decode_paged(q[:, None], c.kpages, c.vpages, c.block_table, before, page, base, k, kv_layout=c.layout, out_dtype=dt)
        # Both are within err of the definition.
        R.close(got[:, 0], want.double(), 2 * err[:, 0].expand_as(want) + want.abs() * (HALF[dt] + 2.0 ** -20), "one token")


@pytest.mark.parametrize("packed", [False, True])
def test_tree_of_a_long_chain_keeps_the_probabilities_of_its_short_rows(packed):
    # A prompt chunk of 300 tokens behind 20: rows of up to 128 keys end inside the first and the second row tile.
    D, Hq, Hkv, page, T, L, base, k = 64, 2, 2, 64, 300, 20, 1e4, 8.0
    for heads in (1, 2):  # query heads of one KV head: nodes 0..127 and 0..63 in the first tile
        kv = Hq // heads
        c = R.Cache(1, 6, page, kv, D, packed, 521)
        c.write(0, torch.arange(L + T, device="cuda"), randn((L + T, kv, D), 522), randn((L + T, kv, D), 523))
        q = (randn((1, T, Hq, D), 524, torch.float32) / 8).to(torch.bfloat16)
        out = atf.tree_decode_paged(q, c.kpages, c.vpages, c.block_table, ints([L]), page, base, k, kv_layout=c.layout)
        pos = L + torch.arange(T, device="cuda", dtype=torch.int32)[None]
        mask = torch.ones((1, T, T), dtype=torch.bool, device="cuda").tril()
        th, short = R.theta_of(base, D), 128 - L
        ref, _, err, _ = R.tree(q[:, :short], c, [L], [short], pos[:, :short], mask[:, :short, :short], th, k, p_err=fine_err(128))
        R.close(out[:, :short], ref, err.expand_as(ref) + ref.abs() * (HALF[torch.bfloat16] + 2.0 ** -21), "short rows")
        ref, _, err, _ = R.tree(q, c, [L], [T], pos, mask, th, k)
        R.close(out, ref, err.expand_as(ref) + ref.abs() * HALF[torch.bfloat16], "all rows")


def one_pair_key(q, pos, node, r, theta):
    """A rotated key [1, D] whose pair r alone is not zero: along the rotated pair of q[node, 0], scaled to a score of 8."""
    D = q.shape[-1]
    x = R.rope(q[None, node:node + 1, :1], pos[None, node:node + 1], theta)[0, 0, 0]
    a = torch.stack((x[r], x[r + D // 2]))
    key = torch.zeros((1, D), dtype=torch.float64, device="cuda")
    key[0, r], key[0, r + D // 2] = a * (8 * math.sqrt(D) / float((a * a).sum()))
    return key.to(torch.bfloat16)


# Windows of these tests run from one or a few positions to beyond the cache.
BOUNDARY = [
    # D, Hq, T, L, base, k: rows in four copies, two copies, one; prefixes that end inside a tile and with one
    (64, 1, 12, 389, 1e4, 0.5),
    (64, 4, 12, 384, 1e4, 0.5),
    (128, 2, 12, 450, 1e4, 0.25),
    (128, 8, 12, 512, 1e6, 0.25),   # more boundary pairs in a tile than are staged
    (128, 1, 1, 500, 1e4, 0.25),    # a single token
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D,Hq,T,L,base,k", BOUNDARY)
def test_tree_windows_end_where_they_should_for_every_node(packed, D, Hq, T, L, base, k):
    # A sequence for each pair r, node and side of its window: the one key that is not zero lies at distance w_r
    # (kept) or w_r + 1 (not kept) of that node. Its pair moves the log-sum-exp by units where it is kept.
    theta, page = R.theta_of(base, D), 64
    mask, depth = R.random_tree(1, T, 531)
    pos1 = L + depth[0]
    order = torch.argsort(depth[0])
    nodes = sorted({int(order[0]), int(order[T // 2]), int(order[-1])})
    cases = [(r, i, int(pos1[i]) - int(w) - over) for r, w in enumerate(R.windows(theta, k)) for i in nodes for over in (0, 1)
             if 0 <= int(pos1[i]) - int(w) - over < L]
    B = len(cases)
    q1 = randn((T, Hq, D), 532, torch.float32).mul_(4).to(torch.bfloat16)
    c = R.Cache(B, -(-(L + T) // page), page, 1, D, packed, 533, fill=0.0)
    c.vpages.copy_(randn(c.vpages.shape, 534))
    for b, (r, i, slot) in enumerate(cases):
        at = torch.tensor([slot], device="cuda")
        c.write(b, at, one_pair_key(q1, pos1, i, r, theta)[:, None], c.read(b, at)[1])
    q, pos = q1.expand(B, -1, -1, -1).contiguous(), pos1.expand(B, -1).contiguous()
    m = mask.expand(B, -1, -1).contiguous()
    out, lse = atf.tree_decode_paged(q, c.kpages, c.vpages, c.block_table, ints([L] * B), page, base, k, tree_mask=m, positions=pos,
                                     kv_layout=c.layout, return_lse=True, out_dtype=torch.float32)
    ref, rlse, err, lerr = R.tree(q, c, [L] * B, [T] * B, pos, m, theta, k)
    for b, (r, i, slot) in enumerate(cases):  # the two sides differ by far more than the tolerance
        if b % 2 and cases[b - 1][:2] == (r, i):
            assert float((rlse[b - 1, 0, i] - rlse[b, 0, i]).abs()) > 100 * float(lerr[b, 0, i])
    R.close(lse, rlse, lerr, "lse")
    R.close(out, ref, err.expand_as(ref) + ref.abs() * 2.0 ** -24, "out")


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D,Hq,base,k,L", [(64, 1, 1e4, 0.5, 60), (64, 14, 1e4, 0.5, 128), (128, 4, 1e6, 0.25, 90)])
def test_tree_windows_end_where_they_should_between_nodes(packed, D, Hq, base, k, L):
    # Node 0's key has one pair; the other nodes sit at distances around its window, on both sides.
    theta, page = R.theta_of(base, D), 64
    steps = [0, -3, -1, 0, 1, 2, 40]
    T, w = len(steps), R.windows(theta, k)
    B = len(w)
    pos = ints([[L + 7] + [max(0, L + 7 + int(x) + s) for s in steps[1:]] for x in w])
    q = randn((1, T, Hq, D), 541, torch.float32).mul_(4).to(torch.bfloat16).expand(B, -1, -1, -1).contiguous()
    c = R.Cache(B, -(-(L + T) // page), page, 1, D, packed, 542, fill=0.0)
    c.vpages.copy_(randn(c.vpages.shape, 543))
    at = torch.tensor([L], device="cuda")
    for b in range(B):
        c.write(b, at, one_pair_key(q[b], pos[b], 3, b, theta)[:, None], c.read(b, at)[1])
    m = torch.ones((B, T, T), dtype=torch.bool, device="cuda")
    out, lse = atf.tree_decode_paged(q, c.kpages, c.vpages, c.block_table, ints([L] * B), page, base, k, tree_mask=m, positions=pos,
                                     kv_layout=c.layout, return_lse=True, out_dtype=torch.float32)
    ref, rlse, err, lerr = R.tree(q, c, [L] * B, [T] * B, pos, m, theta, k)
    assert bool(((rlse[:, 0, 3] - math.log(L + T)) > 100 * lerr[:, 0, 3]).all())  # kept at distance w_r
    R.close(lse, rlse, lerr, "lse")
    R.close(out, ref, err.expand_as(ref) + ref.abs() * 2.0 ** -24, "out")


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv,B,T", [(64, 2, 1, 700, 3), (128, 8, 1, 300, 17)])
def test_tree_of_more_sequences_than_a_block_has_threads(packed, D, Hq, Hkv, B, T):
    # A few items for each CTA group, most cuts inside an item, some at its ends; sequences without nodes, and (second
    # case) two row tiles of which small trees have one.
    lens = [(i * 173) % 611 for i in range(B)]
    run_tree(D, Hq, Hkv, 64, packed, lens, T, [(i * 7) % (T + 3) - 1 for i in range(B)], "tree", 2.0, seed=551)
