"""Cases of the paged-cache operators: what each of them is asked to do, in sizes.

Three operators serve a paged K/V cache, in the order in which a serving step calls them:

  norm_rope     RMS norm of every query and key head and the rotary position embedding,
                in one pass over the projected rows (qsa_norm_rope)
  append        the same on the way into the cache: new keys (normed, rotated) and values
                go to their slots in the pages, indexer keys to the indexer cache, and the
                queries are normed and rotated beside them (qsa_paged_append)
  attn          attention of a chunk of new tokens per sequence over the paged cache, over
                every visible token or over the selected blocks and the trailing block
                (qsa_paged_attn)

A batch is packed: sequence b's new tokens are rows q_start[b] .. q_start[b + 1] - 1, its
cache holds kv_len[b] tokens with them, so row i of it sits at position
kv_len[b] - q_len[b] + i. A page holds page_size tokens of every KV head,
[page][KV head][slot][d], and row b of the page table lists b's pages in order.

With `own` false `run` computes the plain form in elementary torch operations; with `own`
true it makes the calls of the library's binding.
"""
import math

import torch

own = False


# --------------------------------------------------------------------------- cases
def _norm_rope(name, n_tok, Hq, Hkv, d, rot, dtype, fused):
    return dict(name=name, op="norm_rope", n_tok=n_tok, Hq=Hq, Hkv=Hkv, d=d, rot=rot, dtype=dtype, fused=fused)


def _append(name, batch, chunk, length, Hq, Hkv, d, rot, dtype, page):
    return dict(name=name, op="append", batch=batch, chunk_min=chunk[0], chunk_max=chunk[1], len_min=length[0],
                len_max=length[1], Hq=Hq, Hkv=Hkv, d=d, rot=rot, di=64, dtype=dtype, page=page)


def _attn(name, batch, chunk, length, Hq, Hkv, d, dtype, page, block, topk):
    return dict(name=name, op="attn", batch=batch, chunk_min=chunk[0], chunk_max=chunk[1], len_min=length[0],
                len_max=length[1], Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, page=page, block=block, topk=topk)


def listed():
    """topk = 0 is attention over every visible token; lengths count the chunk."""
    return [
        # one decode step of 64 sequences: launch latency decides
        _norm_rope("norm_rope_step_b64", 64, 16, 2, 128, 128, "bf16", True),
        # the padded prompt of the varlen batch, heads read out of the fused projection's rows
        _norm_rope("norm_rope_prompt_16k", 16384, 32, 4, 128, 64, "bf16", True),
        # one decode step of 64 sequences into 64-token pages
        _append("append_step_b64", 64, (1, 1), (400, 2500), 16, 2, 128, 128, "bf16", 64),
        # ragged prompt chunks of a batch of eight into small pages
        _append("append_chunks_b8", 8, (700, 2900), (2900, 4096), 32, 4, 128, 64, "bf16", 16),
        # a decode step over the whole cache, the 4K..32K lengths of the decode workload
        _attn("decode_full_b64", 64, (1, 1), (4096, 32768), 16, 2, 128, "bf16", 64, 64, 0),
        # the same step over the 32 selected blocks and the trailing one
        _attn("decode_selected_b64", 64, (1, 1), (4096, 32768), 16, 2, 128, "bf16", 64, 64, 32),
        # one user's short context: the smallest attention call
        _attn("decode_full_b1", 1, (1, 1), (1500, 1500), 16, 2, 128, "bf16", 16, 64, 0),
        # drafted tokens of a speculative step, head width 256 (the config's default)
        _attn("draft4_full_b16_hd256", 16, (3, 4), (2000, 16000), 16, 2, 256, "bf16", 32, 64, 0),
        # an 8K chunk of a long prompt over a 32K cache: the largest call
        _attn("chunk_full_8k_of_32k", 1, (8192, 8192), (32768, 32768), 16, 2, 128, "bf16", 64, 64, 0),
        # ragged chunks of a mixed batch, head width 256
        _attn("chunks_full_b6_hd256", 6, (1, 1500), (2000, 9000), 16, 2, 256, "bf16", 64, 64, 0),
        # a 4K chunk with the selection of the 64K prefill (64 blocks a token)
        _attn("chunk_selected_4k_of_24k", 1, (4096, 4096), (24000, 24000), 16, 2, 128, "bf16", 64, 64, 64),
        # the fp32 configuration of the tiny prefill, in chunks
        _attn("chunks_selected_fp32", 3, (60, 256), (256, 700), 4, 1, 64, "fp32", 16, 32, 4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attn", "attn", "attn"])
    dtype = "fp32" if rng.random() < 0.15 else "bf16"
    d = rng.choice([64, 128, 128, 128, 256]) if dtype == "bf16" else rng.choice([64, 128])
    Hq, Hkv = rng.choice([(16, 2), (16, 2), (32, 4), (4, 1), (8, 8), (24, 8), (16, 1)])
    page = rng.choice([16, 32, 64, 128, 256])
    rot = rng.choice([d, d // 2])
    if op == "norm_rope":
        return _trim(_norm_rope(None, _log_int(rng, 1, 20000), Hq, Hkv, d, rot, dtype, rng.random() < 0.5))
    if op == "append":
        hi = _log_int(rng, 1, 2900)
        lo = rng.randint(0, hi)
        batch = max(1, min(_log_int(rng, 1, 100), 16000 // hi))
        length = (hi + rng.randint(0, 300), hi + rng.randint(300, 1100))
        return _trim(_append(None, batch, (lo, hi), length, Hq, Hkv, d, rot, dtype, page))
    block = rng.choice([64, 64, 32, 128])
    topk = rng.choice([0, 0, 16, 32, 64])
    hi = rng.choice([1, 1, rng.randint(2, 9), _log_int(rng, 10, 8000)])
    hi = min(hi, int(9000 * (16 / Hq) ** 0.5 * (128 / max(d, 128)) ** 0.5))
    lo = rng.randint(0, hi) if hi > 1 else 1
    # the (row, head, key, d) quadruples and the key rows stay within the largest listed cases'
    triples = int(4e9 * 128 / max(d, 128))
    longest = max(hi, min(_log_int(rng, hi + 200, hi + 24000), triples // (hi * Hq)))
    batch = max(1, min(_log_int(rng, 1, 80), int(1.1e6 * 256 / (longest * Hkv * d)), triples // (hi * Hq * longest)))
    if dtype == "fp32":
        batch, longest, hi = min(batch, 4), min(longest, 2000), min(hi, 500)
        lo, longest = min(lo, hi), max(longest, hi + 100)
    length = (rng.randint(min(hi, longest), longest), longest)
    return _trim(_attn(None, batch, (lo, hi), length, Hq, Hkv, d, dtype, page, block, topk))


def _trim(case):
    del case["name"]
    return case


def _spread(n, lo, hi, step):
    """n whole numbers over [lo, hi]: the same for every seed, so that work() knows them; the first is hi."""
    return [hi - int((i * step) % 1.0 * (hi - lo + 1)) if hi > lo else hi for i in range(n)]


def _lengths(case):
    """(new tokens, tokens in the cache with them) of every sequence."""
    q = _spread(case["batch"], case["chunk_min"], case["chunk_max"], 0.6180339887)
    kv = _spread(case["batch"], case["len_min"], case["len_max"], 0.7548776662)
    return q, [max(a, b) for a, b in zip(q, kv)]


# --------------------------------------------------------------------------- inputs
EPS, THETA = 1e-6, 1e6


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _rows(gen, n, heads, d, dtype, pad=0):
    """[n][heads][d] rows; with pad, a view of rows that many elements longer (a fused projection's)."""
    x = torch.randn(n, heads * d + pad, generator=gen, device="cuda").to(dtype)
    return x[:, : heads * d].unflatten(1, (heads, d))


def _batch(case, gen):
    """The packed batch's geometry and page table; unused entries of the table are -1."""
    q, kv = _lengths(case)
    page = case["page"]
    need = [-(-n // page) for n in kv]
    ids = torch.randperm(sum(need) + 3, generator=gen, device="cuda").to(torch.int32)
    width = max(need) + 1
    table = torch.full((case["batch"], width), -1, dtype=torch.int32)
    table = table.cuda()
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    start = torch.tensor([0] + q).cumsum(0).to(torch.int32).cuda()
    return dict(q_start=start, kv_len=torch.tensor(kv, dtype=torch.int32).cuda(), page_table=table, n_tok=sum(q),
                max_chunk=max(q), page=page, n_pages=sum(need) + 3)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, Hq, Hkv, d = _dtype(case), case["Hq"], case["Hkv"], case["d"]
    s = dict(case=dict(case))

    def weight(n):
        return (1.0 + 0.2 * torch.randn(n, generator=gen, device="cuda")).to(dt)

    if case["op"] == "norm_rope":
        n = case["n_tok"]
        pad = (Hq + Hkv) * d if case["fused"] else 0
        s.update(q=_rows(gen, n, Hq, d, dt, pad), k=_rows(gen, n, Hkv, d, dt, pad), q_weight=weight(d), k_weight=weight(d),
                 pos=torch.randint(0, 65536, (n,), generator=gen, device="cuda").to(torch.int32),
                 q_out=torch.empty(n, Hq, d, dtype=dt, device="cuda"), k_out=torch.empty(n, Hkv, d, dtype=dt, device="cuda"))
        return s
    g = _batch(case, gen)
    s.update(g)
    n = g["n_tok"]
    pool = (g["n_pages"], Hkv, g["page"], d)
    s["k_pages"] = torch.randn(pool, generator=gen, device="cuda", dtype=torch.float32).mul_(0.5).to(dt)
    s["v_pages"] = torch.randn(pool, generator=gen, device="cuda", dtype=torch.float32).mul_(0.5).to(dt)
    if case["op"] == "append":
        cap = max(case["len_max"], case["chunk_max"])
        s.update(q=_rows(gen, n, Hq, d, dt), k=_rows(gen, n, Hkv, d, dt), v=_rows(gen, n, Hkv, d, dt),
                 ki=_rows(gen, n, 1, case["di"], dt)[:, 0], q_weight=weight(d), k_weight=weight(d),
                 q_out=torch.empty(n, Hq, d, dtype=dt, device="cuda"),
                 ki_cache=torch.zeros(case["batch"], cap, case["di"], dtype=dt, device="cuda"))
        return s
    s["q"] = _rows(gen, n, Hq, d, dt).contiguous()
    s["out"] = torch.empty(n, Hq, d, dtype=dt, device="cuda")
    s["sel"] = _selection(case, s, gen) if case["topk"] else None
    return s


def _positions(s):
    """Sequence and position of every packed row."""
    rows = torch.arange(s["n_tok"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["q_start"], rows, right=True) - 1
    return seq, s["kv_len"][seq] - s["q_start"][seq + 1] + rows


def _selection(case, s, gen):
    """topk of the complete blocks before each row by random scores, ascending, padded with -1."""
    B, k = case["block"], case["topk"]
    _, t = _positions(s)
    nb = max(1, int(s["kv_len"].max()) // B)
    block = torch.arange(nb, device="cuda")
    score = torch.rand(s["n_tok"], nb, generator=gen, device="cuda")
    score = torch.where(block < ((t + 1) // B)[:, None], score, -1.0)
    best, at = score.topk(min(k, nb), dim=1)
    at = torch.where(best >= 0, at, nb).sort(dim=1).values
    at = torch.where(at < nb, at, -1)
    pad = torch.full((s["n_tok"], k - at.shape[1]), -1, device="cuda", dtype=at.dtype)
    return torch.cat([at, pad], 1).to(torch.int32).contiguous()


# --------------------------------------------------------------------------- plain forms
def _rotate(x, pos, rot):
    """Rotate-half on the first `rot` of the last axis; x fp32 [n][heads][d]. Angles in 64 bits: fp32
    ones are off by 2^-8 at position 65536."""
    freq = THETA ** (-torch.arange(0, rot, 2, device=x.device, dtype=torch.float64) / rot)
    angle = pos.double()[:, None] * freq
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b, rest = x[..., : rot // 2], x[..., rot // 2: rot], x[..., rot:]
    return torch.cat([a * c - b * s, b * c + a * s, rest], -1)


def _normed(x, weight):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()


def _plain_norm_rope(s):
    rot = s["case"]["rot"]
    for x, w, out in (("q", "q_weight", "q_out"), ("k", "k_weight", "k_out")):
        s[out].copy_(_rotate(_normed(s[x], s[w]), s["pos"], rot))
    return s["q_out"], s["k_out"]


def _plain_append(s):
    c = s["case"]
    seq, t = _positions(s)
    page, slot = s["page_table"][seq, (t // c["page"]).long()].long(), (t % c["page"]).long()
    dt = s["k_pages"].dtype
    s["k_pages"][page, :, slot] = _rotate(_normed(s["k"], s["k_weight"]), t, c["rot"]).to(dt)
    s["v_pages"][page, :, slot] = s["v"]
    s["ki_cache"][seq, t.long()] = _rotate(s["ki"].float()[:, None], t, c["di"])[:, 0].to(dt)
    s["q_out"].copy_(_rotate(_normed(s["q"], s["q_weight"]), t, c["rot"]))
    return s["q_out"], s["k_pages"], s["v_pages"], s["ki_cache"]


def _plain_attn(s):
    c = s["case"]
    B, C, Hq, Hkv, d = c["batch"], s["max_chunk"], c["Hq"], c["Hkv"], c["d"]
    L = s["page_table"].shape[1] * c["page"]
    seq, t = _positions(s)
    row = torch.arange(s["n_tok"], device="cuda") - s["q_start"][seq]
    key = torch.arange(L, device="cuda")
    table = s["page_table"].clamp(min=0).long()
    held = (key < s["kv_len"][:, None])[:, None, :, None]

    def gathered(pages):  # [batch][Hkv][L][d], zero behind a sequence's tokens
        x = pages[table].transpose(1, 2).reshape(B, Hkv, L, d)
        return torch.where(held, x, 0).float()

    q = torch.zeros(B, C, Hkv, Hq // Hkv, d, device="cuda")
    q[seq, row] = s["q"].float().unflatten(1, (Hkv, Hq // Hkv))
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)
    score = (q @ gathered(s["k_pages"]).transpose(2, 3)).mul_(d ** -0.5).view(B, Hkv, C, Hq // Hkv, L)
    seen = key <= t[:, None]
    if s["sel"] is not None:
        nb = -(-L // c["block"])
        chosen = torch.zeros(s["n_tok"], nb + 1, dtype=torch.bool, device="cuda")
        chosen.scatter_(1, torch.where(s["sel"] < 0, nb, s["sel"]).long(), True)
        trailing = key >= ((t + 1) // c["block"] * c["block"])[:, None]
        seen &= chosen[:, key // c["block"]] | trailing
    mask = torch.zeros(B, C, L, dtype=torch.bool, device="cuda")
    mask[seq, row] = seen
    score.masked_fill_(~mask[:, None, :, None], float("-inf"))
    score.sub_(score.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = score.sum(-1)  # [batch][Hkv][C][group]
    out = (score.view(B, Hkv, -1, L) @ gathered(s["v_pages"])).view(B, Hkv, C, Hq // Hkv, d)
    out = (out / total.unsqueeze(-1)).permute(0, 2, 1, 3, 4).reshape(B, C, Hq, d)
    s["out"].copy_(out[seq, row])
    return s["out"]


# --------------------------------------------------------------------------- the library's calls
def _plan(s):
    """What a serving loop keeps between calls: config, batch description and workspace."""
    from block_sparse_long_15_b200 import qsa
    c = s["case"]
    if c["op"] == "norm_rope":
        cfg = qsa.make_config(c["Hq"], c["Hkv"], c["d"], 4, 64, 64, 32, c["dtype"])
        nr = qsa.make_norm_rope(s["q_weight"], s["k_weight"], eps=EPS, rope_theta=THETA, rotary_dim=c["rot"])
        return qsa, cfg, nr, None, None
    cfg = qsa.make_config(c["Hq"], c["Hkv"], c["d"], 4, 64, c.get("block", 64), c.get("topk") or 32, c["dtype"])
    pg = qsa.make_paged(s["q_start"], s["kv_len"], s["page_table"], n_tok=s["n_tok"], max_chunk=s["max_chunk"],
                        page_size=s["page"], n_pages=s["n_pages"])
    if c["op"] == "append":
        nr = qsa.make_norm_rope(s["q_weight"], s["k_weight"], eps=EPS, rope_theta=THETA, rotary_dim=c["rot"],
                                indexer_rotary_dim=c["di"])
        return qsa, cfg, nr, pg, torch.zeros(256, dtype=torch.uint8, device="cuda")
    return qsa, cfg, None, pg, qsa.alloc_paged_workspace(cfg, pg)


def _call(s):
    if "plan" not in s:
        s["plan"] = _plan(s)
    qsa, cfg, nr, pg, ws = s["plan"]
    op = s["case"]["op"]
    if op == "norm_rope":
        qsa.qsa_norm_rope(cfg, nr, s["pos"], s["q"], s["k"], s["q_out"], s["k_out"])
        return s["q_out"], s["k_out"]
    if op == "append":
        qsa.qsa_paged_append(cfg, nr, pg, s["k"], s["v"], s["k_pages"], s["v_pages"], ws, q=s["q"], q_out=s["q_out"],
                             ki=s["ki"], ki_cache=s["ki_cache"])
        return s["q_out"], s["k_pages"], s["v_pages"], s["ki_cache"]
    qsa.qsa_paged_attn(cfg, pg, s["q"], s["k_pages"], s["v_pages"], s["sel"], s["out"], ws)
    return s["out"]


def run(state):
    if own:
        return _call(state)
    op = state["case"]["op"]
    if op == "norm_rope":
        return _plain_norm_rope(state)
    return _plain_append(state) if op == "append" else _plain_attn(state)


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "norm_rope":
        n = case["n_tok"]
        return dict(bytes=2 * n * (Hq + Hkv) * d * e + 4 * n + 2 * d * e, flops=7 * n * (Hq + Hkv) * d)
    q, kv = _lengths(case)
    pages = sum(-(-n // case["page"]) for n in kv) * 4
    if case["op"] == "append":
        n = sum(q)
        return dict(bytes=2 * n * ((Hq + 2 * Hkv) * d + case["di"]) * e + 4 * n // case["page"], flops=7 * n * (Hq + Hkv) * d)
    pairs = rows = 0
    for n, length in zip(q, kv):
        if case["topk"]:
            kept = [min((t + 1) // case["block"], case["topk"]) * case["block"] + (t + 1) % case["block"]
                    for t in range(length - n, length)]
        else:
            kept = range(length - n + 1, length + 1)
        pairs += sum(kept)
        rows += min(length, sum(kept))
    sel = 4 * sum(q) * case["topk"]
    return dict(bytes=2 * sum(q) * Hq * d * e + 2 * rows * Hkv * d * e + pages + sel, flops=4 * pairs * Hq * d)


# --------------------------------------------------------------------------- the definition in 64 bits
def _exact_turn(x, pos, rot):
    """Each pair (x[i], x[i + rot / 2]) as a complex number, times e^(i pos theta^(-2i/rot))."""
    h = rot // 2
    w = torch.exp(-2.0 * math.log(THETA) / rot * torch.arange(h, device=x.device, dtype=torch.float64))
    z = torch.complex(x[..., :h].contiguous(), x[..., h:rot].contiguous())
    z = z * torch.polar(torch.ones_like(w), pos.double().view(-1, 1, 1) * w)
    y = x.clone()
    y[..., :h], y[..., h:rot] = z.real, z.imag
    return y


def _exact_norm(x, weight):
    x = x.double()
    return x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return [_exact_turn(_exact_norm(s[x], s[x + "_weight"]), s["pos"], case["rot"]) for x in ("q", "k")]
    q, kv = _lengths(case)
    out = torch.zeros(s["n_tok"], case["Hq"], case["d"], dtype=torch.float64, device="cuda")
    table, page, at = s["page_table"].tolist(), case["page"], 0
    if case["op"] == "append":
        k_pages, v_pages, ki = s["k_pages"].double(), s["v_pages"].double(), s["ki_cache"].double()
        for b, (n, length) in enumerate(zip(q, kv)):
            new, t = slice(at, at + n), torch.arange(length - n, length, device="cuda")
            at += n
            k = _exact_turn(_exact_norm(s["k"][new], s["k_weight"]), t, case["rot"])
            out[new] = _exact_turn(_exact_norm(s["q"][new], s["q_weight"]), t, case["rot"])
            ki[b, length - n:length] = _exact_turn(s["ki"][new].double().unsqueeze(1), t, case["di"]).squeeze(1)
            for p in range((length - n) // page, -(-length // page)):
                lo, hi = max(p * page, length - n), min((p + 1) * page, length)
                put = (slice(None), slice(lo - p * page, hi - p * page))
                k_pages[table[b][p]][put] = k[lo - length + n:hi - length + n].transpose(0, 1)
                v_pages[table[b][p]][put] = s["v"][new][lo - length + n:hi - length + n].double().transpose(0, 1)
        return [out, k_pages, v_pages, ki]
    group = case["Hq"] // case["Hkv"]
    for b, (n, length) in enumerate(zip(q, kv)):
        ids = table[b][:-(-length // page)]
        t = torch.arange(length - n, length, device="cuda")[:, None]
        u = torch.arange(length, device="cuda")
        keep = u <= t
        if s["sel"] is not None:
            mine = s["sel"][at:at + n].long()
            nb = length // case["block"] + 1
            picked = torch.zeros(n, nb + 1, device="cuda").scatter_(1, torch.where(mine < 0, nb, mine), 1.0)[:, :nb]
            keep = keep & ((picked.repeat_interleave(case["block"], 1)[:, :length] > 0) | (u // case["block"] == (t + 1) // case["block"]))
        for g in range(case["Hkv"]):
            k = s["k_pages"][ids, g].reshape(-1, case["d"])[:length].double()
            v = s["v_pages"][ids, g].reshape(-1, case["d"])[:length].double()
            for h in range(g * group, (g + 1) * group):
                a = s["q"][at:at + n, h].double() @ k.T / math.sqrt(case["d"])
                out[at:at + n, h] = torch.softmax(a.masked_fill_(~keep, float("-inf")), -1) @ v
        at += n
    return out
