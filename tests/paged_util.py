"""Inputs and plain 64-bit forms of the paged-cache operators, for the tests.

Tolerances, from the roundings each operator makes (h = half a step of the output type
relative to the value: bf16 2^-8, fp32 2^-24):

norm + rotation: the mean of d squares and the norm's products are off by at most
  (d / 2 + 8) 2^-24 relative (a sum in lanes of 8 and a tree has fewer steps than d / 2, and
  rsqrtf is within 2 units), the cosine and sine by 2^-22 (phase to 2^-25 of a half turn times
  pi, sincospif 2 units), so with |y_i|, |y_j| the normed pair
      |err| <= h |out| + (|y_i| + |y_j|) ((d / 2 + 8) 2^-24 + 2^-21).

attention: with A = sum p |v| / sum p, each p is off by its logit's error (the product of d
  terms, d 2^-24 sum |q| |k| scale, times the exponential's slope 1, and 2^-22 of the
  exponential itself) in numerator and denominator, the sums over n keys by n 2^-24, and for
  bf16 inputs each p is rounded to bf16 for the product with V (2^-8):
      |err| <= h |out| + A (2 d 2^-24 M + 2 n 2^-24 + 2^-19 + (2^-8 if bf16)),
  M the largest scale sum |q| |k| of the row."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def rotate(y, pos, rot, theta):
    """Rotate-half on the first rot of the last axis; y fp64 [n][heads][d], pos int [n]."""
    h = rot // 2
    out = y.clone()
    if h:
        a = pos.double()[:, None] * theta ** (-2.0 * torch.arange(h, dtype=torch.float64, device=y.device) / rot)
        c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
        out[..., :h] = y[..., :h] * c - y[..., h:rot] * s
        out[..., h:rot] = y[..., h:rot] * c + y[..., :h] * s
    return out


def norm_rope(x, weight, pos, eps, w_off, rot, theta):
    """(value, tolerance) of the norm (none without a weight) and rotation of x [n][heads][d]."""
    d = x.shape[-1]
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * (weight.double() + w_off)
    out = rotate(y, pos, rot, theta)
    pair = y.abs()
    h = rot // 2
    if h:
        pair = pair.clone()
        both = y[..., :h].abs() + y[..., h:rot].abs()
        pair[..., :h], pair[..., h:rot] = both, both
    rel = (d / 2 + 8) * 2.0 ** -24 + 2.0 ** -21
    return out, HALF[x.dtype] * out.abs() * 1.01 + pair * rel


def make_batch(q_len, kv_len, page, seed, spare=2, wide=1, lead=0, tail=0, device="cuda"):
    """Packed geometry with a random page table (entries behind a sequence's pages are -7)."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in kv_len]
    n_pages = sum(need) + spare
    ids = torch.randperm(n_pages, generator=gen).to(torch.int32)
    table = torch.full((len(kv_len), max(need + [0]) + wide), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    start = (torch.tensor([0] + list(q_len)).cumsum(0) + lead).to(torch.int32)
    return dict(q_start=start.to(device), kv_len=torch.tensor(kv_len, dtype=torch.int32, device=device),
                page_table=table.to(device), n_tok=lead + sum(q_len) + tail, max_chunk=max(list(q_len) + [1]),
                page_size=page, n_pages=n_pages)


def positions(q_len, kv_len):
    """[(packed row without lead, sequence, position)]"""
    out, row = [], 0
    for b, (n, length) in enumerate(zip(q_len, kv_len)):
        for i in range(n):
            out.append((row, b, length - n + i))
            row += 1
    return out


def pools(cfg_heads, d, g, kv_len, dtype, seed, std=0.5, poison=float("nan"), device="cuda"):
    """k, v pages with `poison` in every slot that holds no token."""
    gen = torch.Generator().manual_seed(seed)
    shape = (g["n_pages"], cfg_heads, g["page_size"], d)
    out = []
    held = torch.zeros(g["n_pages"], g["page_size"], dtype=torch.bool)
    table = g["page_table"].cpu()
    for b, n in enumerate(kv_len):
        for u0 in range(0, n, g["page_size"]):
            held[table[b, u0 // g["page_size"]], : min(g["page_size"], n - u0)] = True
    for _ in range(2):
        x = torch.randn(shape, generator=gen) * std
        x[~held[:, None].expand(shape[:3])] = poison
        out.append(x.to(dtype).to(device))
    return out


def selection(q_len, kv_len, block, topk, seed):
    """Random lists as the scoring writes them: ascending complete blocks, -1 padded."""
    gen = torch.Generator().manual_seed(seed)
    sel = torch.full((sum(q_len), topk), -1, dtype=torch.int32)
    for row, _, t in positions(q_len, kv_len):
        n_c = (t + 1) // block
        pick = torch.randperm(n_c, generator=gen)[:topk].sort().values
        sel[row, : len(pick)] = pick.to(torch.int32)
    return sel


def attention(q, k_pages, v_pages, table, q_len, kv_len, scale, block=0, sel=None):
    """(value, tolerance) of every packed row in 64 bits, sequence by sequence."""
    dt = q.dtype
    n_tok, Hq, d = q.shape
    Hkv, page = k_pages.shape[1], k_pages.shape[2]
    G = Hq // Hkv
    out = torch.zeros(n_tok, Hq, d, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    row = 0
    for b, (n, length) in enumerate(zip(q_len, kv_len)):
        if n == 0:
            continue
        ids = table[b, : -(-length // page)].long()
        t = torch.arange(length - n, length, device=q.device)[:, None]
        u = torch.arange(length, device=q.device)[None]
        keep = u <= t
        if sel is not None:
            picked = torch.zeros(n, length // block + 2, dtype=torch.bool, device=q.device)
            mine = sel[row:row + n].long()
            n_c = (t + 1) // block
            good = (mine >= 0) & (mine < n_c)
            picked.scatter_(1, torch.where(good, mine, torch.full_like(mine, length // block + 1)), True)
            picked[:, length // block + 1] = False
            keep = keep & (picked[:, (u // block)[0]] | (u >= n_c * block))
        for g in range(Hkv):
            k = k_pages[ids, g].reshape(-1, d)[:length].double()
            v = v_pages[ids, g].reshape(-1, d)[:length].double()
            for h in range(g * G, (g + 1) * G):
                x = q[row:row + n, h].double()
                s = (x @ k.T * scale).masked_fill(~keep, -math.inf)
                big = (x.abs() @ k.abs().T * scale).masked_fill(~keep, 0).amax(-1, keepdim=True)
                p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e300))
                tot = p.sum(-1, keepdim=True)
                p = torch.where(tot > 0, p / tot.clamp(min=1e-300), torch.zeros_like(p))
                o, a = p @ v, p @ v.abs()
                out[row:row + n, h] = o
                rel = 2 * d * 2.0 ** -24 * big + 2 * length * 2.0 ** -24 + 2.0 ** -19
                if dt == torch.bfloat16:
                    rel = rel + 2.0 ** -8
                tol[row:row + n, h] = HALF[dt] * o.abs() * 1.01 + a * rel
        row += n
    return out, tol


def check(got, want, tol, name):
    g = got.double()
    assert torch.isfinite(g).all(), f"{name}: not finite at {(~torch.isfinite(g)).nonzero()[:4].tolist()}"
    over = (g - want).abs() - tol
    assert over.max() <= 0, (f"{name}: {int((over > 0).sum())} of {over.numel()} values off, first at "
                             f"{(over > 0).nonzero()[0].tolist()}, worst {float(over.max()):.3e} over {float(tol.max()):.3e}")
