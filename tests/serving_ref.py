"""64-bit references of the paged serving calls (rotary positions, append, tree
attention, compaction, page copies) and helpers that build their inputs.

The references follow the definitions element by element, in fp64, from the same
bytes the kernels get; they share no code with the package.
"""
import math

import numpy as np
import torch


def theta_of(base, dims):
    return base ** (-2.0 * np.arange(dims // 2, dtype=np.float64) / dims)


def rope(x, positions, theta, *, rotary_dim=None, interleaved=False, scale=1.0, inverse=False):
    """x [B, T, H, D] any dtype -> fp64, rotated."""
    R = rotary_dim if rotary_dim is not None else x.shape[-1]
    y = x.double().clone()
    a = positions.double()[..., None] * torch.as_tensor(theta, dtype=torch.float64, device=x.device)
    c, s = scale * torch.cos(a)[:, :, None], scale * torch.sin(a)[:, :, None] * (-1.0 if inverse else 1.0)
    r = torch.arange(R // 2, device=x.device)
    i, j = (2 * r, 2 * r + 1) if interleaved else (r, r + R // 2)
    p, q = y[..., i], y[..., j]
    out = y.clone()
    out[..., i], out[..., j] = p * c - q * s, q * c + p * s
    return out


def rope_slack(x, R, interleaved, scale, unit):
    """Largest |error| of each output element: its rounding (half a step of the type, `unit` relative to the
    value) is added by the caller; here the fp32 arithmetic, (|x| + |z|) * scale * 2^-20: the angle in half-turns
    rounded to fp32 (pi * 2^-25), cos and sin to an ulp (2^-23), two products, their sum and the scale (each 2^-24).
    For bf16 the angle in radians (three roundings of at most pi: 3 * 2^-23, which moves cos and sin by |sin| and
    |cos| times as much) and the hardware's cos and sin (2^-21.2): together with the products still below 2^-20."""
    y = x.double().abs()
    r = torch.arange(R // 2, device=x.device)
    i, j = (2 * r, 2 * r + 1) if interleaved else (r, r + R // 2)
    tot = torch.zeros_like(y)
    tot[..., i] = tot[..., j] = y[..., i] + y[..., j]
    return tot * abs(scale) * 2.0 ** -20


class Cache:
    """A paged cache with shuffled pages; every slot starts as `fill` (NaN: what nothing may read)."""

    def __init__(self, B, pages_each, page, Hkv, D, packed, seed, fill=math.nan, extra=3):
        g = torch.Generator().manual_seed(seed)
        self.n = B * pages_each + extra
        self.page, self.packed, self.Hkv, self.D, self.B = page, packed, Hkv, D, B
        self.block_table = torch.randperm(self.n, generator=g)[: B * pages_each].reshape(B, pages_each).to(torch.int32).cuda()
        kshape = (self.n, Hkv, D // 16, page, 16) if packed else (self.n, page, Hkv, D)
        self.kpages = torch.full(kshape, fill, dtype=torch.bfloat16, device="cuda")
        self.vpages = torch.full((self.n, page, Hkv, D), fill, dtype=torch.bfloat16, device="cuda")
        self.layout = "PACKED" if packed else "NHD"

    def where(self, b, slots):
        slots = slots.long()
        return self.block_table[b].long()[slots // self.page], slots % self.page

    def read(self, b, slots):
        """Rotated keys (natural dim order) and values [n, Hkv, D]."""
        p, at = self.where(b, slots)
        v = self.vpages[p, at]
        if not self.packed:
            return self.kpages[p, at], v
        k = self.kpages[p, :, :, at].reshape(len(slots), self.Hkv, self.D // 2, 2)
        return torch.cat((k[..., 0], k[..., 1]), -1), v

    def write(self, b, slots, k, v):
        """Rotated keys (natural dim order) and values [n, Hkv, D] bf16."""
        p, at = self.where(b, slots)
        self.vpages[p, at] = v
        if not self.packed:
            self.kpages[p, at] = k
        else:
            H = self.D // 2
            self.kpages[p, :, :, at] = torch.stack((k[..., :H], k[..., H:]), -1).reshape(len(slots), self.Hkv, self.D // 16, 16)

    def clone(self):
        c = object.__new__(Cache)
        c.__dict__.update(self.__dict__)
        c.kpages, c.vpages = self.kpages.clone(), self.vpages.clone()
        return c


def windows(theta, k):
    return [math.inf if math.isinf(k) else math.floor(k * 2 * math.pi / t) for t in theta]


def tree(q, cache, lens, counts, positions, mask, theta, k, p_err=2.0 ** -8):
    """fp64 (out [B, T, Hq, D], lse [B, Hq, T], err [B, T, Hq, 1], lse_err [B, Hq, T]); rows past counts are NaN.

    err: what bf16 probabilities (2^-8 of each), the rotated query kept to 2^-16 and fp32 sums can move an output
    by: (2^-8 (or p_err) + 2 e) * sum p |v| (largest over dims), with e = 2^-15 * max over keys of sum_r |terms| / sqrt(D) the
    error of a score (2^-16 for the query's two bf16 parts, 2^-16 for a 256-term fp32 sum).  lse_err: e plus fp32
    roundings of the log (2^-20 of its size and one)."""
    B, T, Hq, D = q.shape
    H, G = D // 2, Hq // cache.Hkv
    w = windows(theta, k)
    th = torch.as_tensor(theta, dtype=torch.float64, device=q.device)
    out = torch.full((B, T, Hq, D), math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq, T), math.nan, dtype=torch.float64, device=q.device)
    err = torch.zeros((B, T, Hq, 1), dtype=torch.float64, device=q.device)
    lse_err = torch.zeros((B, Hq, T), dtype=torch.float64, device=q.device)
    for b in range(B):
        n, t = int(lens[b]), int(counts[b])
        if t == 0:
            continue
        kk, vv = cache.read(b, torch.arange(n + t, device=q.device))
        kk, vv = kk.double(), vv.double()
        qpos = positions[b, :t].double()
        kpos = torch.cat((torch.arange(n, dtype=torch.float64, device=q.device), qpos))
        dist = qpos[:, None] - kpos[None]
        sees = torch.ones((t, n + t), dtype=torch.bool, device=q.device)
        sees[:, n:] = mask[b, :t, :t].bool()
        qr = rope(q[b:b + 1, :t], positions[b:b + 1, :t], theta)[0]  # [t, Hq, D]
        for h in range(cache.Hkv):
            x = torch.zeros((t, G, n + t), dtype=torch.float64, device=q.device)
            big = torch.zeros_like(x)
            for r in range(H):
                keep = (dist <= w[r])[:, None]
                qa, qb = qr[:, h * G:(h + 1) * G, r, None], qr[:, h * G:(h + 1) * G, r + H, None]
                a, z = qa * kk[:, h, r], qb * kk[:, h, r + H]
                x += torch.where(keep, a + z, 0.0)
                big += torch.where(keep, a.abs() + z.abs(), 0.0)
            hide = ~sees[:, None].expand_as(x)
            x = (x / math.sqrt(D)).masked_fill(hide, -math.inf)
            e = 2.0 ** -15 * (big / math.sqrt(D)).masked_fill(hide, 0.0).amax(-1)  # [t, G]
            m = x.amax(-1, keepdim=True)
            p = torch.where(hide, 0.0, torch.exp(x - torch.where(torch.isinf(m) & (m < 0), 0.0, m)))
            l = p.sum(-1, keepdim=True)
            p = p / torch.where(l == 0, 1.0, l)
            # What a key holds that a node does not see takes no part: drop it before the product.
            vh = torch.where(sees.any(0)[:, None], vv[:, h], 0.0)
            part = torch.stack([torch.where(sees[i][:, None], vh, 0.0).T @ p[i].T for i in range(t)]).transpose(1, 2)  # [t, G, D]
            mag = torch.stack([torch.where(sees[i][:, None], vh.abs(), 0.0).T @ p[i].T for i in range(t)]).transpose(1, 2)
            out[b, :t, h * G:(h + 1) * G] = part
            err[b, :t, h * G:(h + 1) * G, 0] = (p_err + 2 * e) * mag.amax(-1)
            ls = torch.where(l[..., 0] == 0, -math.inf, m[..., 0] + torch.log(l[..., 0]))
            lse[b, h * G:(h + 1) * G, :t] = ls.T
            lse_err[b, h * G:(h + 1) * G, :t] = (e + 2.0 ** -20 * (1 + ls.nan_to_num(0, 0, 0).abs())).T
    return out, lse, err, lse_err


def random_tree(B, T, seed):
    """Parents before children: ancestor masks [B, T, T] and depths [B, T]."""
    rng = np.random.default_rng(seed)
    mask, depth = np.zeros((B, T, T), dtype=bool), np.zeros((B, T), dtype=np.int32)
    for b in range(B):
        for i in range(T):
            if i:
                p = int(rng.integers(0, i))
                mask[b, i] = mask[b, p]
                depth[b, i] = depth[b, p] + 1
            mask[b, i, i] = True
    return torch.from_numpy(mask).cuda(), torch.from_numpy(depth).cuda()


def close(got, ref, tol, what):
    """|got - ref| <= tol elementwise, infinities and NaN in the same places."""
    got = got.double()
    same = torch.isfinite(ref) == torch.isfinite(got)
    assert bool(same.all()), f"{what}: finite in different places"
    odd = ~torch.isfinite(ref)
    assert bool((torch.isnan(got) == torch.isnan(ref))[odd].all()) and bool((got == ref)[odd & ~torch.isnan(ref)].all()), what
    d = torch.where(odd, 0.0, (got - ref).abs() - tol)
    assert float(d.max()) <= 0.0, f"{what}: {float(d.max()):.3e} over its tolerance, |diff| {float((got - ref).abs()[~odd].max()):.3e}"
