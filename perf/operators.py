"""The serving operators around the paged KV cache: what each computes, on which sizes, and what it cannot do without.

Five operators of one drafted step of a served model, on the head shapes of this repository's workloads:

  rope_apply        rotary positions of queries and keys (half or interleaved pairs, part of the head, scaled), or their gradient
  cache_append      new tokens' keys (rotated) and values into the pages of a paged cache
  tree_decode       windowed attention of a tree of drafted tokens over the cached prefix and the tree itself
  cache_compact     the accepted tokens of each tree moved to the slots behind the prefix
  cache_copy_pages  the filled part of pages copied to other pages (a forked sequence's last page, a defragmented pool)

With `own` false, `run` computes them with elementary torch operations in 32 bits (angles in 64).
"""
import math

import torch

own = False

#: Head shapes (query heads, KV heads, head dim, RoPE base) of the repository's workloads.
SHAPES = {"qwen05b": (14, 2, 64, 1e6), "llama3b": (24, 8, 128, 5e5), "qwen7b": (28, 4, 128, 1e7)}


def listed():
    return [
        # One chat sequence with seven drafted tokens: a call whose latency counts (NHD cache as prefill leaves it).
        dict(name="tree_chat", op="tree", shape="qwen05b", B=1, L=1021, T=7, page=64, packed=False, k=8.0, ragged=False, chain=False),
        # A batch being served, every sequence at its own length, trees of up to 16 nodes.
        dict(name="tree_batch", op="tree", shape="llama3b", B=8, L=8192, T=16, page=64, packed=True, k=16.0, ragged=True, chain=False),
        # Single tokens (no tree) without a window over long contexts: the plain step of the same engine.
        dict(name="tree_single", op="tree", shape="qwen7b", B=4, L=65503, T=1, page=128, packed=False, k=math.inf, ragged=False, chain=True),
        # Wide trees over 128K tokens: 448 query rows for each KV head.
        dict(name="tree_wide", op="tree", shape="qwen7b", B=2, L=131072, T=64, page=256, packed=True, k=16.0, ragged=False, chain=False),
        # Queries and keys of a prompt, as views into the output of one fused projection.
        dict(name="rope_prompt", op="rope", shape="qwen7b", B=1, T=32768, f32=False, part=128, inter=False, scale=1.0, inverse=False),
        # Gradients of a training step in 32 bits: interleaved pairs in half of each head, cos and sin scaled.
        dict(name="rope_grad", op="rope", shape="llama3b", B=3, T=1367, f32=True, part=64, inter=True, scale=1.1386, inverse=True),
        # The drafted nodes of a batch written before they are attended.
        dict(name="append_nodes", op="append", shape="qwen05b", B=5, L=2000, T=7, page=64, packed=True, ragged=True),
        # Prompts of unequal lengths written whole.
        dict(name="append_prompts", op="append", shape="qwen7b", B=3, L=0, T=20011, page=256, packed=True, ragged=True),
        # A few accepted nodes of one small batch.
        dict(name="compact_step", op="compact", shape="qwen05b", B=4, L=1500, T=16, page=64, packed=False, accepted=4),
        # A large batch after wide trees.
        dict(name="compact_batch", op="compact", shape="llama3b", B=64, L=1024, T=64, page=128, packed=True, accepted=12),
        # Sequences forked into beams: the filled part of each last page.
        dict(name="copy_tails", op="copy", shape="qwen05b", n=6, page=64, packed=True, part=True),
        # A pool defragmented.
        dict(name="copy_pool", op="copy", shape="qwen7b", n=1200, page=256, packed=False, part=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["tree", "tree", "tree", "rope", "append", "compact", "copy"])
    c = dict(op=op, shape=rng.choice(sorted(SHAPES)))
    page, packed = rng.choice([64, 128, 192, 256]), rng.random() < 0.5
    if op == "tree":
        T, B = spread(1, 64), spread(1, 16)
        most = min(131072, 2 * 131072 * 64 // (T * B), 4 * 131072 // B)
        c.update(B=B, L=spread(1, most), T=T, page=page, packed=packed, k=rng.choice([1.0, 8.0, 16.0, 64.0, math.inf]),
                 ragged=rng.random() < 0.5, chain=rng.random() < 0.3)
    elif op == "rope":
        d, f32 = SHAPES[c["shape"]][2], rng.random() < 0.3
        c.update(B=spread(1, 8), T=spread(1, 2048 if f32 else 4096), f32=f32, part=rng.choice([d, d, d // 2, d // 4 * 3]),
                 inter=rng.random() < 0.5, scale=rng.choice([1.0, 1.1386]), inverse=rng.random() < 0.5)
    elif op == "append":
        c.update(B=spread(1, 8), L=spread(1, 4096) - 1, T=spread(1, 7000), page=page, packed=packed, ragged=rng.random() < 0.5)
    elif op == "compact":
        T = spread(2, 128)
        c.update(B=spread(1, 64), L=spread(1, 4096), T=T, page=page, packed=packed, accepted=rng.randint(1, T))
    else:
        c.update(n=spread(1, 600), page=page, packed=packed, part=rng.random() < 0.5)
    return c


# ------------------------------------------------------------------ the cases' sizes
def _lens(case):
    """Cached tokens of each sequence, and its new tokens."""
    B, L, T = case["B"], case["L"], case["T"]
    if not case.get("ragged"):
        return [L] * B, [T] * B
    return [max(0, L - (L * 7 * b) // (8 * B) - 5 * b) for b in range(B)], [max(1, T - (T * 3 * b) // (4 * B)) for b in range(B)]


def _windows(case):
    Hq, Hkv, D, base = SHAPES[case["shape"]]
    return [math.inf if case["k"] == math.inf else math.floor(case["k"] * 2 * math.pi * base ** (2.0 * r / D)) for r in range(D // 2)]


def work(case):
    Hq, Hkv, D, base = SHAPES[case["shape"]]
    op = case["op"]
    if op == "tree":
        lens, counts = _lens(case)
        w, total, flops = _windows(case), 0, 0
        for n, t in zip(lens, counts):
            kept = sum(min(x, n) + t for x in w)  # (key, pair) terms that some query of the tree keeps
            total += Hkv * (4 * kept + 2 * D * (n + t))  # K elements of kept pairs, V whole
            total += t * Hq * (4 * D + 4) + 4 * t + (0 if case["chain"] else t * t)
            flops += t * Hq * (4 * kept + 2 * D * (n + t))
        return {"bytes": total, "flops": flops}
    if op == "rope":
        n = case["B"] * case["T"] * (Hq + Hkv)
        return {"bytes": n * D * 2 * (4 if case["f32"] else 2) + 4 * case["B"] * case["T"], "flops": 3 * n * case["part"]}
    if op == "append":
        n = sum(_lens(case)[1])
        return {"bytes": n * Hkv * D * 8 + 4 * n, "flops": 3 * n * Hkv * D}
    if op == "compact":
        n = case["B"] * case["accepted"]
        return {"bytes": n * Hkv * D * 8 + 4 * n, "flops": 0}
    n = sum(_fill(case))
    return {"bytes": n * Hkv * D * 8 + 12 * case["n"], "flops": 0}


def _fill(case):
    """Tokens of each copied page."""
    return [case["page"] if not case["part"] else 1 + (i * 29) % case["page"] for i in range(case["n"])]


# ------------------------------------------------------------------ inputs
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pools(case, num_pages, gen):
    Hq, Hkv, D, base = SHAPES[case["shape"]]
    P = case["page"]
    kshape = (num_pages, Hkv, D // 16, P, 16) if case["packed"] else (num_pages, P, Hkv, D)
    return (torch.randn(kshape, generator=gen, device="cuda", dtype=torch.bfloat16),
            torch.randn((num_pages, P, Hkv, D), generator=gen, device="cuda", dtype=torch.bfloat16))


def _table(case, spans, gen):
    """Pages of each sequence, scattered over the pool, with a few that belong to nobody."""
    need = max(-(-s // case["page"]) for s in spans)
    n = case["B"] * need + 3
    ids = torch.randperm(n, generator=gen, device="cuda", dtype=torch.int32)[: case["B"] * need]
    return ids.reshape(case["B"], need).contiguous(), n


def _tree(case, gen):
    """Random trees: each node's parent comes before it; node i sees its ancestors and itself. Returns mask [B, T, T] and depths [B, T]."""
    B, T = case["B"], case["T"]
    u = torch.rand((B, T), generator=gen, device="cuda")
    parent = torch.clamp((u * torch.arange(T, device="cuda") * 0.7 + 0.3 * torch.arange(T, device="cuda")).long(), max=T - 1)
    parent = torch.minimum(parent, torch.clamp(torch.arange(T, device="cuda") - 1, min=0)).cpu()
    mask, depth = torch.zeros((B, T, T), dtype=torch.bool), torch.zeros((B, T), dtype=torch.int32)
    rows = torch.arange(B)
    for i in range(T):
        if i:
            mask[:, i] = mask[rows, parent[:, i]]
            depth[:, i] = depth[rows, parent[:, i]] + 1
        mask[:, i, i] = True
    return mask.cuda(), depth.cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    Hq, Hkv, D, base = SHAPES[case["shape"]]
    s = dict(case=case, base=base, D=D, Hq=Hq, Hkv=Hkv)
    op = case["op"]
    if op == "rope":
        B, T = case["B"], case["T"]
        dt = torch.float32 if case["f32"] else torch.bfloat16
        qkv = torch.randn((B, T, Hq + 2 * Hkv, D), generator=gen, device="cuda", dtype=dt)
        first = torch.randint(0, 900000, (B, 1), generator=gen, device="cuda")
        s.update(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv], positions=(first + torch.arange(T, device="cuda")).to(torch.int32))
        return s
    if op == "copy":
        s["kpages"], s["vpages"] = _pools(case, 2 * case["n"] + 1, gen)
        ids = torch.randperm(2 * case["n"] + 1, generator=gen, device="cuda", dtype=torch.int32)
        s.update(src=ids[: case["n"]].contiguous(), dst=ids[case["n"]:2 * case["n"]].contiguous(),
                 tokens=_ints(_fill(case)) if case["part"] else None)
        return s
    lens, counts = _lens(case)
    s["span"] = max(n + t for n, t in zip(lens, counts))
    s["block_table"], num_pages = _table(case, [s["span"]], gen)
    s["kpages"], s["vpages"] = _pools(case, num_pages, gen)
    s["seqlens"], s["counts"] = _ints(lens), _ints(counts)
    B, T = case["B"], case["T"]
    if op == "tree":
        s["q"] = torch.randn((B, T, Hq, D), generator=gen, device="cuda", dtype=torch.bfloat16)
        s["mask"], s["positions"] = None, None
        if not case["chain"]:
            s["mask"], depth = _tree(case, gen)
            s["positions"] = depth + s["seqlens"][:, None]
        s["out"] = torch.zeros((B, T, Hq, D), device="cuda", dtype=torch.bfloat16)
        s["lse"] = torch.zeros((B, Hq, T), device="cuda")
        s["workspace"] = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")  # scratch that a serving loop keeps between calls
    elif op == "append":
        kv = torch.randn((B, T, 2 * Hkv, D), generator=gen, device="cuda", dtype=torch.bfloat16)
        s["k"], s["v"] = kv[:, :, :Hkv], kv[:, :, Hkv:]
    else:
        # Accepted nodes: the first few of the greedy branch (numbered first), then nodes of a side branch behind it.
        a, n = case["accepted"], (B, T)
        main = torch.randint(0, a + 1, (B, 1), generator=gen, device="cuda")
        order = torch.rand(n, generator=gen, device="cuda").masked_fill(torch.arange(T, device="cuda") < a, 2.0).argsort(1)
        side = torch.cat([order[:, : max(0, T - a)], torch.full((B, a), -1, device="cuda")], 1)[:, :a]
        side = torch.where(side < 0, torch.arange(a, device="cuda"), side).sort(1).values
        at = torch.arange(a, device="cuda")
        s["path"] = torch.where((at < main) | (side < a), at, side).to(torch.int32).contiguous()
        s["accepted"] = _ints([a] * B)
        s["new_seqlens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _cos_sin(positions, theta, dtype=torch.float32):
    """cos and sin of position * theta, the angle reduced in 64 bits: [..., pairs]."""
    a = torch.remainder(positions.double()[..., None] * theta, 2 * math.pi)
    return torch.cos(a).to(dtype), torch.sin(a).to(dtype)


def _theta(base, dims):
    return base ** (-2.0 * torch.arange(dims // 2, dtype=torch.float64, device="cuda") / dims)


def _rotate(lo, hi, c, s):
    return torch.stack((lo * c - hi * s, hi * c + lo * s), -1)


def _rope_plain(s):
    case = s["case"]
    part, inter = case["part"], case["inter"]
    c, sn = _cos_sin(s["positions"], _theta(s["base"], part))
    c, sn = c[:, :, None] * case["scale"], sn[:, :, None] * (-case["scale"] if case["inverse"] else case["scale"])

    def one(x):
        y = x.float()
        rot, rest = y[..., :part], y[..., part:]
        pairs = rot.unflatten(-1, (part // 2, 2)) if inter else rot.unflatten(-1, (2, part // 2)).transpose(-1, -2)
        pairs = _rotate(pairs[..., 0], pairs[..., 1], c, sn)
        rot = (pairs if inter else pairs.transpose(-1, -2)).flatten(-2)
        return torch.cat((rot, rest), -1).to(x.dtype)

    return one(s["q"]), one(s["k"])


def _place(s, slots):
    """Page and place in the page of slots [B, n]."""
    P = s["case"]["page"]
    return s["block_table"].long().gather(1, torch.clamp(slots // P, max=s["block_table"].shape[1] - 1)), slots % P


def _append_plain(s):
    case, B, T = s["case"], s["case"]["B"], s["case"]["T"]
    i = torch.arange(T, device="cuda")
    slots = s["seqlens"].long()[:, None] + i
    live = i < s["counts"][:, None]
    c, sn = _cos_sin(slots, _theta(s["base"], s["D"]))
    H = s["D"] // 2
    k = s["k"].float()
    pairs = _rotate(k[..., :H], k[..., H:], c[:, :, None], sn[:, :, None])  # [B, T, Hkv, H, 2]
    page, at = _place(s, slots)
    page, at = page[live], at[live]
    if case["packed"]:
        s["kpages"][page, :, :, at] = pairs[live].reshape(-1, s["Hkv"], s["D"] // 16, 16).to(torch.bfloat16)
    else:
        s["kpages"][page, at] = pairs[live].transpose(-1, -2).flatten(-2).to(torch.bfloat16)
    s["vpages"][page, at] = s["v"][live]
    return s["kpages"], s["vpages"]


def _compact_plain(s):
    case = s["case"]
    n = s["seqlens"].long()[:, None]
    live = torch.arange(s["path"].shape[1], device="cuda") < s["accepted"][:, None]
    fp, fa = _place(s, n + s["path"])
    tp, ta = _place(s, n + torch.arange(s["path"].shape[1], device="cuda"))
    fp, fa, tp, ta = fp[live], fa[live], tp[live], ta[live]
    if case["packed"]:
        s["kpages"][tp, :, :, ta] = s["kpages"][fp, :, :, fa]
    else:
        s["kpages"][tp, ta] = s["kpages"][fp, fa]
    s["vpages"][tp, ta] = s["vpages"][fp, fa]
    s["new_seqlens"] = s["seqlens"] + s["accepted"]
    return s["kpages"], s["vpages"], s["new_seqlens"]


def _copy_plain(s):
    case = s["case"]
    src, dst = s["src"].long(), s["dst"].long()
    if s["tokens"] is None:
        s["kpages"][dst], s["vpages"][dst] = s["kpages"][src], s["vpages"][src]
        return s["kpages"], s["vpages"]
    i, at = (torch.arange(case["page"], device="cuda") < s["tokens"][:, None]).nonzero(as_tuple=True)
    if case["packed"]:
        s["kpages"][dst[i], :, :, at] = s["kpages"][src[i], :, :, at]
    else:
        s["kpages"][dst[i], at] = s["kpages"][src[i], at]
    s["vpages"][dst[i], at] = s["vpages"][src[i], at]
    return s["kpages"], s["vpages"]


def _tree_inputs(s):
    """The caches gathered in slot order (K as pairs [B, S, Hkv, H, 2], V [B, S, Hkv, D] with nothing behind the last node), the slots'
    and the queries' positions, and what each query sees [B, T, S]."""
    case, B, T, S = s["case"], s["case"]["B"], s["case"]["T"], s["span"]
    n, t = s["seqlens"].long()[:, None], s["counts"].long()[:, None]
    slot = torch.arange(S, device="cuda").expand(B, S)
    page, at = _place(s, slot)
    if case["packed"]:
        k = s["kpages"][page, :, :, at].reshape(B, S, s["Hkv"], s["D"] // 2, 2)
    else:
        k = s["kpages"][page, at].unflatten(-1, (2, s["D"] // 2)).transpose(-1, -2)
    v = s["vpages"][page, at].masked_fill((slot >= n + t)[..., None, None], 0)
    qpos = s["positions"].long() if s["positions"] is not None else n + torch.arange(T, device="cuda")
    node = slot - n
    inside = torch.clamp(node, 0, T - 1)
    kpos = torch.where(node < 0, slot, qpos.gather(1, inside))
    i = torch.arange(T, device="cuda")
    if s["mask"] is not None:
        sees = s["mask"].gather(2, inside[:, None].expand(B, T, S))
    else:
        sees = node[:, None] <= i[:, None]
    sees = ((node < 0)[:, None] | (sees & (node >= 0)[:, None])) & (node < t)[:, None] & (i < t)[..., None]
    return k, v, qpos, kpos, sees


def _tree_plain(s):
    B, T, S, H, Hkv, D = s["case"]["B"], s["case"]["T"], s["span"], s["D"] // 2, s["Hkv"], s["D"]
    k, v, qpos, kpos, sees = _tree_inputs(s)
    k, v = k.float(), v.float()
    w = torch.tensor([min(x, 2.0 ** 40) for x in _windows(s["case"])], device="cuda", dtype=torch.int64)
    c, sn = _cos_sin(qpos, _theta(s["base"], D))
    q = s["q"].float()
    q = _rotate(q[..., :H], q[..., H:], c[:, :, None], sn[:, :, None]).reshape(B, T, Hkv, -1, D) * D ** -0.5
    step = max(1, (1 << 28) // (B * S * Hkv * D))  # queries at a time: the kept part of K is laid out for each of them
    outs, lses = [], []
    for lo in range(0, T, step):
        dist = qpos[:, lo:lo + step, None] - kpos[:, None]
        keep = (dist[..., None] <= w)[:, :, :, None, :, None]  # pair r of the key at this distance enters the score
        kept = torch.where(keep, k[:, None], 0.0).flatten(-2)
        x = torch.einsum("bthgd,btshd->bthgs", q[:, lo:lo + step], kept)
        del kept
        x = x.masked_fill(~sees[:, lo:lo + step, None, None], -math.inf)
        m = x.amax(-1, keepdim=True).clamp(min=-3e38)
        p = torch.exp(x - m)
        total = p.sum(-1, keepdim=True)
        outs.append(torch.einsum("bthgs,bshd->bthgd", p, v) / torch.where(total == 0, 1.0, total))
        lses.append((m + torch.log(total))[..., 0])
    live = torch.arange(T, device="cuda") < s["counts"][:, None]
    out = torch.cat(outs, 1).flatten(2, 3) * live[..., None, None]
    lse = torch.where(live[..., None], torch.cat(lses, 1).flatten(2), 0.0).transpose(1, 2)
    return out.to(torch.bfloat16), lse.contiguous()


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"tree": _tree_plain, "rope": _rope_plain, "append": _append_plain, "compact": _compact_plain, "copy": _copy_plain}[op](s)
    import long_context_attention_pair_b200 as atf
    case = s["case"]
    if op == "rope":
        return atf.rope_apply(s["q"], s["k"], s["positions"], s["base"], rotary_dim=case["part"], interleaved=case["inter"], scale=case["scale"],
                              inverse=case["inverse"])
    layout = "PACKED" if case["packed"] else "NHD"
    if op == "copy":
        atf.cache_copy_pages(s["kpages"], s["vpages"], s["src"], s["dst"], case["page"], tokens=s["tokens"], kv_layout=layout)
        return s["kpages"], s["vpages"]
    if op == "append":
        atf.cache_append(s["k"], s["v"], s["kpages"], s["vpages"], s["block_table"], s["seqlens"], case["page"], s["base"],
                         counts=s["counts"], kv_layout=layout)
        return s["kpages"], s["vpages"]
    if op == "compact":
        atf.cache_compact(s["kpages"], s["vpages"], s["block_table"], s["seqlens"], s["path"], s["accepted"], case["page"],
                          new_seqlens=s["new_seqlens"], kv_layout=layout)
        return s["kpages"], s["vpages"], s["new_seqlens"]
    return atf.tree_decode_paged(s["q"], s["kpages"], s["vpages"], s["block_table"], s["seqlens"], case["page"], s["base"], case["k"],
                                 tree_mask=s["mask"], positions=s["positions"], counts=s["counts"], kv_layout=layout, out=s["out"],
                                 lse=s["lse"], workspace=s["workspace"])


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, D, H, Hkv = case["op"], s["D"], s["D"] // 2, s["Hkv"]
    if op == "rope":
        part, R = case["part"], case["part"] // 2
        r = torch.arange(R, device="cuda")
        first, second = (2 * r, 2 * r + 1) if case["inter"] else (r, r + R)
        a = s["positions"].double()[..., None, None] * torch.pow(torch.tensor(s["base"], dtype=torch.float64, device="cuda"), -2.0 * r.double() / part)
        sign = -1.0 if case["inverse"] else 1.0
        outs = []
        for x in (s["q"].double(), s["k"].double()):
            y = x.clone()
            y[..., first] = case["scale"] * (x[..., first] * torch.cos(a) - sign * x[..., second] * torch.sin(a))
            y[..., second] = case["scale"] * (x[..., second] * torch.cos(a) + sign * x[..., first] * torch.sin(a))
            outs.append(y)
        return tuple(outs)
    kp, vp = s["kpages"].double(), s["vpages"].double()
    k_at = (lambda page, at: (page, slice(None), slice(None), at)) if case["packed"] else (lambda page, at: (page, at))
    if op == "copy":
        kn, vn = kp.clone(), vp.clone()
        src, dst, fill = s["src"].tolist(), s["dst"].tolist(), _fill(case)
        for i in range(case["n"]):
            cut = (slice(None), slice(None), slice(0, fill[i])) if case["packed"] else (slice(0, fill[i]),)
            kn[dst[i]][cut] = kp[src[i]][cut]
            vn[dst[i]][: fill[i]] = vp[src[i]][: fill[i]]
        return kn, vn
    table, P = s["block_table"].long(), case["page"]
    lens, counts = _lens(case)
    if op == "compact":
        kn, vn = kp.clone(), vp.clone()
        for b in range(case["B"]):
            at = lens[b] + s["path"][b].long()
            to = lens[b] + torch.arange(case["accepted"], device="cuda")
            kn[k_at(table[b, to // P], to % P)] = kp[k_at(table[b, at // P], at % P)]
            vn[table[b, to // P], to % P] = vp[table[b, at // P], at % P]
        return kn, vn, s["seqlens"] + s["accepted"]
    theta = [s["base"] ** (-2.0 * r / D) for r in range(H)]
    if op == "append":
        for b in range(case["B"]):
            m = lens[b] + torch.arange(counts[b], device="cuda")
            x, y = s["k"][b, : counts[b]].double(), torch.empty((counts[b], Hkv, D), dtype=torch.float64, device="cuda")
            for r in range(H):
                c, sn = torch.cos(m.double() * theta[r])[:, None], torch.sin(m.double() * theta[r])[:, None]
                u, z = x[..., r] * c - x[..., r + H] * sn, x[..., r + H] * c + x[..., r] * sn
                i, j = (2 * r, 2 * r + 1) if case["packed"] else (r, r + H)
                y[..., i], y[..., j] = u, z
            kp[k_at(table[b, m // P], m % P)] = y.reshape(-1, Hkv, D // 16, 16) if case["packed"] else y
            vp[table[b, m // P], m % P] = s["v"][b, : counts[b]].double()
        return kp, vp
    # Attention, one sequence and KV head at a time, one frequency pair after the other.
    B, T, G = case["B"], case["T"], s["Hq"] // Hkv
    if sum(n + t for n, t in zip(lens, counts)) * T * s["Hq"] * H > 4e11:
        return None
    w = _windows(case)
    out = torch.zeros((B, T, s["Hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, s["Hq"], T), dtype=torch.float64, device="cuda")
    for b in range(B):
        n, t = lens[b], counts[b]
        m = torch.arange(n + t, device="cuda")
        qpos = s["positions"][b, :t].double() if s["positions"] is not None else (n + torch.arange(t, device="cuda")).double()
        dist = qpos[:, None] - torch.cat((torch.arange(n, device="cuda").double(), qpos))
        sees = torch.ones((t, n + t), dtype=torch.bool, device="cuda")
        sees[:, n:] = s["mask"][b, :t, :t] if s["mask"] is not None else torch.ones((t, t), dtype=torch.bool, device="cuda").tril()
        for h in range(Hkv):
            kr = kp[table[b, m // P], h, :, m % P].reshape(-1, D) if case["packed"] else kp[table[b, m // P], m % P, h]
            x = torch.zeros((G, t, n + t), dtype=torch.float64, device="cuda")
            for r in range(H):
                c, sn = torch.cos(qpos * theta[r])[:, None], torch.sin(qpos * theta[r])[:, None]
                a, z = s["q"][b, :t, h * G:(h + 1) * G, r].double(), s["q"][b, :t, h * G:(h + 1) * G, r + H].double()
                i, j = (2 * r, 2 * r + 1) if case["packed"] else (r, r + H)
                u, y = (a * c - z * sn).T, (z * c + a * sn).T
                x += (u[:, :, None] * kr[:, i] + y[:, :, None] * kr[:, j]) * (dist <= w[r])
            x = (x / math.sqrt(D)).masked_fill(~sees, -math.inf)
            lse[b, h * G:(h + 1) * G, :t] = torch.logsumexp(x, -1)
            out[b, :t, h * G:(h + 1) * G] = (torch.softmax(x, -1) @ vp[table[b, m // P], m % P, h]).transpose(0, 1)
    return out, lse
