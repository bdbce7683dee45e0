"""The paged-cache operators through the binding, against plain 64-bit forms (paged_util)."""
import math
import os
import subprocess
import sys

import pytest
import torch

from tests import paged_util as U

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
NAN = float("nan")


def _cfg(qsa, Hq=16, Hkv=2, d=128, di=64, block=64, topk=4, dtype="bf16", scale=0.0):
    return qsa.make_config(Hq, Hkv, d, 4, di, block, topk, dtype, scale)


# ------------------------------------------------------------------ norm + rotation
@pytest.mark.parametrize("dtype,Hq,Hkv,d,rot,w_off,pad", [
    ("bf16", 16, 2, 128, 128, 0.0, 0),
    ("bf16", 32, 4, 128, 64, 1.0, 264),    # rows of a fused projection
    ("bf16", 4, 1, 64, 32, 0.0, 8),
    ("bf16", 16, 2, 256, 256, 0.0, 0),
    ("bf16", 3, 3, 80, 80, 0.0, 0),        # a head that does not fill its lanes
    ("bf16", 33, 11, 8, 0, 0.0, 0),        # one lane a head, no rotation
    ("fp32", 4, 1, 64, 64, 0.0, 0),
    ("fp32", 5, 5, 96, 16, 1.0, 4),
    ("fp32", 2, 1, 256, 128, 0.0, 0),
])
@pytest.mark.parametrize("n", [1, 37])
def test_norm_rope(cuda_lib, dtype, Hq, Hkv, d, rot, w_off, pad, n):
    qsa, dt = cuda_lib, DT[dtype]
    g = torch.Generator().manual_seed(d + rot + n)
    q = torch.randn(n, Hq * d + pad, generator=g).to(dt).cuda()[:, : Hq * d].unflatten(1, (Hq, d))
    k = (3 * torch.randn(n, Hkv * d + pad, generator=g)).to(dt).cuda()[:, : Hkv * d].unflatten(1, (Hkv, d))
    qw, kw = ((torch.randn(d, generator=g) * 0.3 + 1 - w_off).to(dt).cuda() for _ in range(2))
    pos = torch.randint(0, 200000, (n,), generator=g).to(torch.int32)
    pos[:1] = 2 ** 31 - 1 if n == 1 else 0
    if n > 3:
        pos[1], pos[2] = -5, 2 ** 31 - 1
    pos = pos.cuda()
    nr = qsa.make_norm_rope(qw, kw, eps=1e-5, weight_offset=w_off, rope_theta=1e6, rotary_dim=rot)
    qo, ko = torch.full((n, Hq, d), NAN, dtype=dt, device="cuda"), torch.full((n, Hkv, d), NAN, dtype=dt, device="cuda")
    q0, k0 = q.clone(), k.clone()
    qsa.qsa_norm_rope(_cfg(qsa, Hq, Hkv, d, dtype=dtype), nr, pos, q, k, qo, ko)
    for name, x, x0, w, out in (("q", q, q0, qw, qo), ("k", k, k0, kw, ko)):
        want, tol = U.norm_rope(x0, w, pos, 1e-5, w_off, rot, 1e6)
        U.check(out, want, tol, name)
        assert torch.equal(x, x0)
    # in place, and one side alone: the same bits
    qsa.qsa_norm_rope(_cfg(qsa, Hq, Hkv, d, dtype=dtype), nr, pos, q, None, q, None)
    qsa.qsa_norm_rope(_cfg(qsa, Hq, Hkv, d, dtype=dtype), nr, pos, None, k, None, k)
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_norm_rope_without_weight_only_rotates(cuda_lib):
    qsa = cuda_lib
    q = torch.randn(5, 4, 64).cuda()
    pos = torch.tensor([0, 1, 2, 70000, 9], dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    nr = qsa.make_norm_rope(rope_theta=1e4, rotary_dim=32)
    qsa.qsa_norm_rope(_cfg(qsa, 4, 1, 64, dtype="fp32"), nr, pos, q, None, out, None)
    U.check(out, *U.norm_rope(q, None, pos, 0.0, 0.0, 32, 1e4), "q")
    assert torch.equal(out[..., 32:], q[..., 32:]) and torch.equal(out[0], q[0])


def test_norm_rope_extreme_rows(cuda_lib):
    """Rows of zeros stay zeros; the largest and smallest magnitudes of bf16 inputs stay finite where
    the mean of squares does in fp32."""
    qsa = cuda_lib
    q = torch.zeros(3, 2, 128)
    q[1] = 1e15
    q[2] = 1e-15
    q = q.to(torch.bfloat16).cuda()
    w = torch.ones(128, dtype=torch.bfloat16).cuda()
    out = torch.empty_like(q)
    pos = torch.tensor([3, 4, 5], dtype=torch.int32).cuda()
    nr = qsa.make_norm_rope(w, w, eps=1e-6, rope_theta=1e4, rotary_dim=128)
    qsa.qsa_norm_rope(_cfg(qsa, 2, 1, 128), nr, pos, q, None, out, None)
    assert (out[0] == 0).all()
    U.check(out, *U.norm_rope(q, w, pos, 1e-6, 0.0, 128, 1e4), "q")


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype,Hq,Hkv,d,page,q_len,kv_len,rot,rot_i", [
    ("bf16", 16, 2, 128, 64, [1] * 5, [1, 64, 65, 200, 128], 128, 64),
    ("bf16", 32, 4, 128, 16, [0, 37, 1, 16, 0], [5, 37, 16, 100, 1], 64, 32),
    ("fp32", 4, 1, 64, 32, [3, 0, 40], [33, 1, 40], 64, 0),
    ("bf16", 16, 2, 256, 256, [70], [300], 256, 64),
    ("bf16", 3, 3, 80, 16, [5, 6], [21, 6], 16, 16),
])
def test_append(cuda_lib, dtype, Hq, Hkv, d, page, q_len, kv_len, rot, rot_i):
    qsa, dt, di = cuda_lib, DT[dtype], 64
    g = U.make_batch(q_len, kv_len, page, seed=7, lead=2, tail=3)
    gen = torch.Generator().manual_seed(3)
    n = g["n_tok"]
    rows = {}
    for name, heads, width in (("q", Hq, d), ("k", Hkv, d), ("v", Hkv, d), ("ki", 1, di)):
        x = torch.randn(n, heads, width, generator=gen)
        x[:2] = NAN
        x[n - 3:] = NAN  # rows of no sequence
        rows[name] = x.to(dt).cuda()
    qw, kw = ((torch.randn(d, generator=gen) * 0.3 + 1).to(dt).cuda() for _ in range(2))
    cap = max(kv_len) + 3
    kp, vp = U.pools(Hkv, d, g, kv_len, dt, seed=1)
    ki_cache = torch.randn(len(q_len), cap, di, generator=gen).to(dt).cuda()
    q_out = torch.full((n, Hq, d), 7.0, dtype=dt, device="cuda")
    want_k, want_v, want_ki = kp.clone(), vp.clone(), ki_cache.clone()
    pg = qsa.make_paged(**g)
    nr = qsa.make_norm_rope(qw, kw, eps=1e-6, rope_theta=1e6, rotary_dim=rot, indexer_rotary_dim=rot_i)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    qsa.qsa_paged_append(_cfg(qsa, Hq, Hkv, d, di, dtype=dtype), nr, pg, rows["k"], rows["v"], kp, vp, ws, q=rows["q"],
                         q_out=q_out, ki=rows["ki"][:, 0], ki_cache=ki_cache)
    assert qsa.qsa_read_device_status(ws) == qsa.QSA_OK
    where = [(r + 2, b, t) for r, b, t in U.positions(q_len, kv_len)]
    r = torch.tensor([x[0] for x in where]).cuda()
    b = torch.tensor([x[1] for x in where]).cuda()
    t = torch.tensor([x[2] for x in where]).cuda()
    pages = g["page_table"][b, t // page].long()
    U.check(q_out[r], *U.norm_rope(rows["q"][r], qw, t, 1e-6, 0.0, rot, 1e6), "q")
    U.check(kp[pages, :, t % page], *U.norm_rope(rows["k"][r], kw, t, 1e-6, 0.0, rot, 1e6), "k")
    U.check(ki_cache[b, t][:, None], *U.norm_rope(rows["ki"][r], None, t, 0.0, 0.0, rot_i, 1e6), "ki")
    assert torch.equal(vp[pages, :, t % page], rows["v"][r])
    # nothing else moved: slots, cache rows, and the packed rows of no sequence
    for got, want, at in ((kp, want_k, (pages, slice(None), t % page)), (vp, want_v, (pages, slice(None), t % page)),
                          (ki_cache, want_ki, (b, t))):
        want[at] = got[at]
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    assert (q_out[:2] == 7).all() and (q_out[n - 3:] == 7).all()


def test_append_copies_without_norm_rope(cuda_lib):
    qsa = cuda_lib
    g = U.make_batch([4, 1], [20, 17], 16, seed=1)
    k, v = (torch.randn(5, 2, 128).to(torch.bfloat16).cuda() for _ in range(2))
    kp, vp = (torch.zeros(g["n_pages"], 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    qsa.qsa_paged_append(_cfg(qsa), None, qsa.make_paged(**g), k, v, kp, vp, ws)
    for r, b, t in U.positions([4, 1], [20, 17]):
        p = int(g["page_table"][b, t // 16])
        assert torch.equal(kp[p, :, t % 16], k[r]) and torch.equal(vp[p, :, t % 16], v[r])


# ------------------------------------------------------------------ attention
CASES = [
    # dtype Hq Hkv d page block topk q_len kv_len
    ("bf16", 16, 2, 128, 64, 64, 0, [1] * 4, [1, 63, 64, 1000]),
    ("bf16", 16, 2, 128, 16, 64, 0, [1, 0, 1], [17, 40, 16]),
    ("bf16", 16, 2, 128, 64, 64, 4, [1] * 5, [1, 63, 64, 1000, 333]),
    ("bf16", 16, 2, 128, 32, 32, 3, [2, 0, 5], [70, 9, 500]),
    ("bf16", 16, 2, 256, 64, 64, 0, [3, 4, 1], [300, 4, 129]),
    ("bf16", 16, 2, 256, 16, 64, 2, [4, 1], [300, 129]),
    ("bf16", 8, 8, 128, 128, 64, 0, [1, 7, 30], [140, 7, 300]),
    ("bf16", 24, 8, 64, 256, 64, 0, [1, 6, 40], [700, 6, 300]),
    ("bf16", 24, 8, 64, 16, 32, 5, [6, 40], [6, 300]),
    ("bf16", 16, 1, 128, 64, 128, 2, [1, 9], [700, 400]),
    ("bf16", 32, 1, 64, 32, 64, 2, [1, 3], [200, 400]),
    ("bf16", 6, 2, 80, 16, 64, 0, [2, 20], [50, 200]),
    ("bf16", 6, 2, 128, 16, 24, 3, [2, 20], [50, 200]),
    ("bf16", 16, 2, 128, 64, 64, 0, [70, 1, 129], [500, 300, 129]),
    ("bf16", 16, 2, 128, 16, 64, 4, [70, 1, 129], [500, 300, 129]),
    ("bf16", 16, 2, 256, 64, 64, 0, [70, 1, 129], [500, 300, 129]),
    ("bf16", 16, 2, 256, 16, 64, 4, [70, 1, 129], [500, 300, 129]),
    ("bf16", 24, 8, 128, 32, 64, 0, [150, 3, 0, 44], [150, 300, 10, 600]),
    ("bf16", 24, 8, 128, 32, 64, 3, [150, 3, 0, 44], [150, 300, 10, 600]),
    ("bf16", 4, 4, 128, 256, 128, 2, [200, 20], [600, 20]),
    # no more rows than one tile, split over many CTAs
    ("bf16", 16, 2, 128, 64, 64, 0, [16, 2, 9, 0], [6000, 700, 9, 50]),
    ("bf16", 16, 2, 128, 16, 64, 5, [16, 2, 9, 0], [6000, 700, 9, 50]),
    ("bf16", 24, 8, 128, 256, 64, 0, [42, 7], [3000, 2000]),
    ("bf16", 32, 1, 256, 32, 64, 0, [4, 1, 3], [5000, 1, 700]),
    ("bf16", 16, 2, 256, 16, 128, 3, [12, 8], [5000, 2300]),
    ("bf16", 24, 8, 64, 32, 64, 0, [30, 2, 500], [3000, 900, 700]),
    ("bf16", 8, 1, 64, 16, 64, 3, [3, 60], [900, 2500]),
    # many rows and many parts
    ("bf16", 16, 2, 128, 32, 64, 0, [300, 40], [4100, 40]),
    ("bf16", 16, 2, 128, 128, 192, 6, [300, 40], [4100, 2100]),
    ("bf16", 4, 4, 256, 64, 256, 2, [200, 20], [2600, 1020]),
    ("fp32", 4, 1, 64, 16, 32, 4, [30, 1, 0, 7], [200, 300, 4, 7]),
    ("fp32", 4, 1, 64, 16, 32, 0, [30, 1, 0, 7], [200, 300, 4, 7]),
    ("fp32", 8, 2, 256, 64, 48, 2, [1, 5], [300, 90]),
    ("fp32", 32, 1, 128, 32, 16, 3, [2], [80]),
    # CUDA cores: streams of many tiles a warp, heads that do not fill their lanes or entries, one to three
    # 16-byte pieces a row, tiles that cross a page
    ("fp32", 16, 2, 128, 32, 64, 0, [200, 0, 260], [1500, 10, 1400]),
    ("fp32", 16, 2, 256, 64, 64, 4, [60, 3], [1500, 1400]),
    ("fp32", 6, 2, 200, 16, 64, 0, [9, 1, 40], [300, 1, 77]),
    ("fp32", 4, 4, 136, 16, 24, 5, [9, 1, 40], [300, 1, 77]),
    ("fp32", 3, 1, 8, 16, 8, 3, [5, 33], [100, 33]),
    ("bf16", 9, 1, 16, 16, 40, 3, [5, 33], [100, 400]),
    ("bf16", 8, 2, 72, 32, 64, 0, [5, 33], [100, 400]),
    ("bf16", 12, 3, 200, 16, 24, 6, [5, 33], [100, 400]),
    ("bf16", 2, 2, 24, 16, 56, 2, [5, 33], [100, 400]),
]


def _run(qsa, case, seed=11, std=1.0, poison=NAN, lead=1, tail=2, pick=None):
    dtype, Hq, Hkv, d, page, block, topk, q_len, kv_len = case
    dt = DT[dtype]
    g = U.make_batch(q_len, kv_len, page, seed=seed, lead=lead, tail=tail)
    cfg = _cfg(qsa, Hq, Hkv, d, block=block, topk=max(topk, 1), dtype=dtype)
    kp, vp = U.pools(Hkv, d, g, kv_len, dt, seed=seed + 1, std=std, poison=poison)
    gen = torch.Generator().manual_seed(seed + 2)
    q = torch.full((g["n_tok"], Hq, d), NAN)
    q[lead:g["n_tok"] - tail] = torch.randn(sum(q_len), Hq, d, generator=gen)
    q = q.to(dt).cuda()
    sel = None
    if topk:
        sel = torch.full((g["n_tok"], topk), 12345, dtype=torch.int32)
        mine = sel[lead:g["n_tok"] - tail]
        mine[:] = -1
        mine[:, : pick or topk] = U.selection(q_len, kv_len, block, pick or topk, seed + 3)
        sel = sel.cuda()
    pg = qsa.make_paged(**g)
    out = torch.full_like(q, 7.0)
    ws = qsa.alloc_paged_workspace(cfg, pg)
    return dict(cfg=cfg, pg=pg, q=q, kp=kp, vp=vp, sel=sel, out=out, ws=ws, g=g, rows=slice(lead, g["n_tok"] - tail))


def _attn(qsa, s, stream=None):
    qsa.qsa_paged_attn(s["cfg"], s["pg"], s["q"], s["kp"], s["vp"], s["sel"], s["out"], s["ws"], stream=stream)


def _oracle(s, case):
    dtype, Hq, Hkv, d, page, block, topk, q_len, kv_len = case
    r = s["rows"]
    return U.attention(s["q"][r], s["kp"], s["vp"], s["g"]["page_table"], q_len, kv_len, 1 / math.sqrt(d), block,
                       None if s["sel"] is None else s["sel"][r])


# A large budget sends chunks with a selection to the tensor-core kernels; `pick` entries of each list
# are used, the rest is -1.
TILE_CASES = [
    # pick, case
    (5, ("bf16", 16, 2, 128, 64, 64, 256, [100, 13, 3], [4100, 700, 300])),
    (3, ("bf16", 16, 2, 128, 16, 192, 128, [16, 12, 15], [3000, 2999, 1024])),   # one tile
    (7, ("bf16", 24, 8, 128, 128, 128, 128, [90, 0, 41, 2], [2000, 5, 1300, 200])),  # G = 3: idle rows
    (1, ("bf16", 16, 2, 256, 32, 64, 256, [70, 12], [2500, 640])),
    (4, ("bf16", 8, 1, 64, 256, 64, 512, [129, 60], [3300, 900])),
    # lists longer than one segment's bits: every group of one head
    (9, ("bf16", 2, 2, 128, 64, 64, 1024, [200], [16000])),
    (9, ("bf16", 1, 1, 256, 64, 128, 1024, [40], [33000])),
]


@pytest.mark.parametrize("pick,case", TILE_CASES, ids=lambda c: str(c) if isinstance(c, int) else
                         "-".join(str(x) for x in c[:7]) + f"-q{max(c[7])}-kv{max(c[8])}")
def test_attention_selected_tiles(cuda_lib, pick, case):
    qsa = cuda_lib
    s = _run(qsa, case, pick=pick)
    n0 = qsa.qsa_kernel_launch_count()
    _attn(qsa, s)
    assert qsa.qsa_kernel_launch_count() - n0 >= 2  # a tile kernel and the merge
    assert qsa.qsa_read_device_status(s["ws"]) == qsa.QSA_OK
    U.check(s["out"][s["rows"]], *_oracle(s, case), "out")
    assert (s["out"][:1] == 7).all() and (s["out"][-2:] == 7).all()
    first = s["out"].clone()
    _attn(qsa, s)
    assert torch.equal(first, s["out"])


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:7]) + f"-q{max(c[7])}-kv{max(c[8])}")
def test_attention(cuda_lib, case):
    qsa = cuda_lib
    s = _run(qsa, case)
    _attn(qsa, s)
    assert qsa.qsa_read_device_status(s["ws"]) == qsa.QSA_OK
    U.check(s["out"][s["rows"]], *_oracle(s, case), "out")
    assert (s["out"][:1] == 7).all() and (s["out"][-2:] == 7).all()  # rows of no sequence
    first = s["out"].clone()
    s["out"].fill_(7.0)
    _attn(qsa, s)  # the workspace is as it was: the same bits again
    assert torch.equal(first, s["out"])
    assert int(s["ws"][:256].sum()) == 0


# ------------------------------------------------------------------ lists, masks and values
def test_attention_of_rows_that_see_nothing(cuda_lib):
    """A selection that lists nothing at a block boundary leaves a row empty: it is written as zeros, and
    the rows beside it are right. Both kernels."""
    qsa = cuda_lib
    for topk, q_len, kv_len in ((4, [3, 1], [64, 128]), (2048, [70, 64], [128, 64])):
        case = ("bf16", 16, 2, 128, 16, 64, topk, q_len, kv_len)
        s = _run(qsa, case, pick=1)
        rows = s["sel"][s["rows"]]
        rows[:] = -1  # row at position 63 (127): no block, no trailing token
        _attn(qsa, s)
        assert qsa.qsa_read_device_status(s["ws"]) == qsa.QSA_OK
        U.check(s["out"][s["rows"]], *_oracle(s, case), "out")
        last = s["rows"].start + q_len[0] - 1
        assert (s["out"][last] == 0).all()


def test_ids_outside_the_candidates_are_skipped(cuda_lib):
    qsa = cuda_lib
    for topk, q_len, kv_len in ((4, [2], [700]), (2048, [70], [700])):
        case = ("bf16", 16, 2, 128, 64, 64, topk, q_len, kv_len)
        s = _run(qsa, case, pick=2)
        s["sel"][s["rows"], 2] = 11      # n_c is 10: not a complete block before any of the rows
        s["sel"][s["rows"], 3] = 2 ** 30
        _attn(qsa, s)
        U.check(s["out"][s["rows"]], *_oracle(s, case), "out")


@pytest.mark.parametrize("q_len,kv_len,d", [([2], [300], 128), ([100], [400], 128), ([40], [400], 256), ([30], [90], 64)])
def test_attention_extreme_logits(cuda_lib, q_len, kv_len, d):
    """Logits of several thousand either way: one key takes (nearly) everything, the sums stay finite. The
    bf16 inputs are exact in the oracle; the logits' own rounding, 2 d 2^-24 M, is in the tolerance."""
    qsa = cuda_lib
    case = ("bf16", 16, 2, d, 64, 64, 0, q_len, kv_len)
    s = _run(qsa, case, std=4.0)
    s["q"][s["rows"]] *= 16
    _attn(qsa, s)
    U.check(s["out"][s["rows"]], *_oracle(s, case), "out")


def test_masked_infinities_in_keys(cuda_lib):
    """Keys of later tokens of the chunk may be infinite: the mask is a selection, not a product."""
    qsa = cuda_lib
    for q_len, d in (([4], 128), ([100], 128), ([60], 256)):
        case = ("bf16", 16, 2, d, 16, 64, 0, q_len, [q_len[0] + 37])
        s = _run(qsa, case)
        n = case[8][0] - 1
        s["kp"][s["g"]["page_table"][0, n // 16].long(), :, n % 16] = float("inf")
        _attn(qsa, s)
        want, tol = _oracle(s, case)
        got = s["out"][s["rows"]]
        U.check(got[:-1], want[:-1], tol[:-1], "out")  # all but the token itself


# ------------------------------------------------------------------ geometry that does not fit
BAD = [("q_start falls", lambda g: g["q_start"].__setitem__(2, 0)),
       ("q_start passes n_tok", lambda g: g["q_start"].__setitem__(3, 10 ** 6)),
       ("kv_len below the chunk", lambda g: g["kv_len"].__setitem__(1, 3)),
       ("kv_len beyond the table", lambda g: g["kv_len"].__setitem__(1, 2 ** 31 - 1)),
       ("negative kv_len", lambda g: g["kv_len"].__setitem__(1, -5)),
       ("a page outside the pool", lambda g: g["page_table"].__setitem__((1, 3), 10 ** 6)),
       ("a negative page", lambda g: g["page_table"].__setitem__((1, 2), -1)),
       ("more tokens than max_chunk", lambda g: g.__setitem__("max_chunk", 60))]


@pytest.mark.parametrize("name,spoil", BAD, ids=[b[0] for b in BAD])
@pytest.mark.parametrize("topk,d,dtype", [(0, 128, "bf16"), (0, 256, "bf16"), (2048, 128, "bf16"), (4, 128, "bf16"),
                                          (4, 64, "fp32")])
def test_bad_geometry_is_reported_and_kept_apart(cuda_lib, name, spoil, topk, d, dtype):
    """Sequence 1 is spoilt; 0 and 2 are served (unless their own rows are in dispute) and nothing faults."""
    qsa = cuda_lib
    q_len, kv_len = [50, 64, 40], [300, 200, 90]
    case = (dtype, 16, 2, d, 64, 64, topk, q_len, kv_len)
    s = _run(qsa, case, pick=2 if topk else None)
    want, tol = _oracle(s, case)
    g = {k: v.clone() if torch.is_tensor(v) else v for k, v in s["g"].items()}
    spoil(g)
    pg = qsa.make_paged(**g)
    s["ws"] = qsa.alloc_paged_workspace(s["cfg"], pg)
    qsa.qsa_paged_attn(s["cfg"], pg, s["q"], s["kp"], s["vp"], s["sel"], s["out"], s["ws"])
    assert qsa.qsa_read_device_status(s["ws"]) == qsa.QSA_ERR_DEVICE_CHECK
    r = s["rows"].start
    if name != "q_start falls":
        U.check(s["out"][r:r + 50], want[:50], tol[:50], "sequence 0")
    if not name.startswith("q_start"):
        U.check(s["out"][r + 114:r + 154], want[114:], tol[114:], "sequence 2")
    # the append: the same report, and only slots of the sequence itself may move
    dt = DT[dtype]
    k = torch.randn(g["n_tok"], 2, d, device="cuda").to(dt)
    kp, ws = s["kp"].clone(), torch.zeros(256, dtype=torch.uint8, device="cuda")
    qsa.qsa_paged_append(s["cfg"], None, pg, k, k, kp, s["vp"].clone(), ws)
    assert qsa.qsa_read_device_status(ws) == qsa.QSA_ERR_DEVICE_CHECK
    held = torch.zeros(g["n_pages"], dtype=torch.bool)
    for b, n in enumerate(kv_len):
        held[s["g"]["page_table"][b, : -(-n // 64)].cpu().long()] = True
    free = (~held).nonzero()[:, 0].cuda()
    assert torch.equal(kp[free].view(torch.uint8), s["kp"][free].view(torch.uint8))


def test_append_beyond_the_indexer_cache_is_reported(cuda_lib):
    qsa = cuda_lib
    g = U.make_batch([2, 2], [20, 9], 16, seed=5)
    k = torch.randn(4, 2, 128).to(torch.bfloat16).cuda()
    kp, vp = (torch.zeros(g["n_pages"], 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ki, ki_cache = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 19, 64, dtype=torch.bfloat16,
                                                                                     device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    qsa.qsa_paged_append(_cfg(qsa), None, qsa.make_paged(**g), k, k, kp, vp, ws, ki=ki, ki_cache=ki_cache)
    assert qsa.qsa_read_device_status(ws) == qsa.QSA_ERR_DEVICE_CHECK
    assert (ki_cache[0] == 0).all()  # the sequence that does not fit has no indexer key written
    assert (ki_cache[1, 7:9] == 1).all() and (ki_cache[1, :7] == 0).all() and (ki_cache[1, 9:] == 0).all()


# ------------------------------------------------------------------ streams, graphs, workspaces
@pytest.mark.parametrize("case", [CASES[0], CASES[3], CASES[13], CASES[15], CASES[-1]], ids=["rows", "selected", "two-tile",
                                                                                         "one-tile", "fp32"])
def test_graphs_and_streams(cuda_lib, case):
    """A captured call replays on new contents of the same tensors; two graphs and an eager call share one
    workspace one after the other; a side stream gives the same bits."""
    qsa = cuda_lib
    s = _run(qsa, case, lead=0, tail=0, poison=0.0)
    t = _run(qsa, case, seed=29, lead=0, tail=0, poison=0.0)
    _attn(qsa, s)
    want_s = s["out"].clone()
    t["ws"] = s["ws"]
    _attn(qsa, t)
    want_t = t["out"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s["out"].fill_(0)
    side.wait_stream(torch.cuda.current_stream())
    _attn(qsa, s, stream=side)
    side.synchronize()
    assert torch.equal(s["out"], want_s)
    graphs = []
    for x in (s, t):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _attn(qsa, x)
        graphs.append(g)
    for x in (s, t):
        x["out"].fill_(0)
    graphs[0].replay()
    graphs[1].replay()
    _attn(qsa, s)
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(s["out"], want_s) and torch.equal(t["out"], want_t)
    s["q"].copy_(t["q"])
    s["kp"].copy_(t["kp"]) if s["kp"].shape == t["kp"].shape else None
    graphs[0].replay()
    torch.cuda.synchronize()
    again = s["out"].clone()
    _attn(qsa, s)
    assert torch.equal(again, s["out"])
    assert qsa.qsa_read_device_status(s["ws"]) == qsa.QSA_OK


def test_append_and_norm_in_a_graph(cuda_lib):
    qsa = cuda_lib
    g = U.make_batch([1, 3], [20, 17], 16, seed=1)
    q, k, v = (torch.randn(4, h, 128).to(torch.bfloat16).cuda() for h in (16, 2, 2))
    kp, vp = (torch.zeros(g["n_pages"], 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    nr = qsa.make_norm_rope(w, w, rope_theta=1e6, rotary_dim=128)
    pg, ws = qsa.make_paged(**g), torch.zeros(256, dtype=torch.uint8, device="cuda")
    qo, pos = torch.empty_like(q), torch.arange(4, dtype=torch.int32, device="cuda")
    qsa.qsa_paged_append(_cfg(qsa), nr, pg, k, v, kp, vp, ws, q=q, q_out=qo)  # modules are loaded before the capture
    qsa.qsa_norm_rope(_cfg(qsa), nr, pos, q, None, q.clone(), None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qsa.qsa_paged_append(_cfg(qsa), nr, pg, k, v, kp, vp, ws, q=q, q_out=qo)
    k.mul_(-1)
    pg.kv_len.add_(1)
    kp.zero_()
    graph.replay()
    want = torch.zeros_like(kp)
    qsa.qsa_paged_append(_cfg(qsa), nr, pg, k, v, want, vp.clone(), ws)
    assert torch.equal(kp, want) and int((kp != 0).any(-1).sum()) == 8


def test_many_sequences(cuda_lib):
    """More sequences than one launch of the attention takes, most of them with one token."""
    qsa = cuda_lib
    gen = torch.Generator().manual_seed(4)
    q_len = torch.randint(0, 3, (1100,), generator=gen).tolist()
    q_len[600] = 30
    kv_len = [n + int(x) for n, x in zip(q_len, torch.randint(1, 60, (1100,), generator=gen))]
    for d in (128, 256):
        case = ("bf16", 8, 2, d, 16, 64, 0, q_len, kv_len)
        s = _run(qsa, case)
        _attn(qsa, s)
        assert qsa.qsa_read_device_status(s["ws"]) == qsa.QSA_OK
        U.check(s["out"][s["rows"]], *_oracle(s, case), "out")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    k = torch.randn(s["g"]["n_tok"], 2, 256, device="cuda").to(torch.bfloat16)
    qsa.qsa_paged_append(s["cfg"], None, s["pg"], k, k, s["kp"], s["vp"], ws)
    assert qsa.qsa_read_device_status(ws) == qsa.QSA_OK
    for r, b, t in U.positions(q_len, kv_len)[::97]:
        assert torch.equal(s["kp"][int(s["g"]["page_table"][b, t // 16]), :, t % 16], k[r + 1])


def test_shared_prefix_pages(cuda_lib):
    """Two sequences over the same pages of a common prefix."""
    qsa = cuda_lib
    case = ("bf16", 16, 2, 128, 64, 64, 0, [1, 40], [128 + 5, 128 + 40])
    s = _run(qsa, case)
    s["g"]["page_table"][1, :2] = s["g"]["page_table"][0, :2]
    _attn(qsa, s)
    U.check(s["out"][s["rows"]], *_oracle(s, case), "out")


def test_lengths_at_the_end_of_int32_are_refused(cuda_lib):
    """Keys are counted in int32 up to the end of a tile: a longer sequence is refused, its neighbours are
    served. (Its table names one page over and over; the table itself is long enough.)"""
    qsa = cuda_lib
    case = ("bf16", 8, 2, 128, 32768, 64, 0, [1, 1], [40, 70])
    s = _run(qsa, case, lead=0, tail=0)
    want, tol = _oracle(s, case)
    table = torch.zeros(2, 65536, dtype=torch.int32)
    table[:, :1] = s["g"]["page_table"].cpu()[:, :1]
    for length in (2**31 - 1, 2**31 - 255):
        g = dict(s["g"], page_table=table.cuda(), kv_len=torch.tensor([length, 70], dtype=torch.int32).cuda())
        pg = qsa.make_paged(**g)
        ws = qsa.alloc_paged_workspace(s["cfg"], pg)
        qsa.qsa_paged_attn(s["cfg"], pg, s["q"], s["kp"], s["vp"], None, s["out"], ws)
        assert qsa.qsa_read_device_status(ws) == qsa.QSA_ERR_DEVICE_CHECK
        U.check(s["out"][1:], want[1:], tol[1:], f"beside {length}")


def test_status_survives_a_larger_workspace(cuda_lib):
    """A recorded status is still there when a later step needs a larger workspace."""
    from block_sparse_long_15_b200.runner import QSAPaged
    qsa = cuda_lib
    run = QSAPaged(qsa.make_config(16, 2, 128, 4, 64, 64, 4, "bf16"), slots=1, max_len=640, n_pages=10, page_size=64)
    rows = lambda n: [torch.zeros(n, h, 128, dtype=torch.bfloat16, device="cuda") for h in (16, 2, 2)]
    run.step([1], *rows(1))
    small = run.ws
    small[:4].view(torch.int32)[0] = qsa.QSA_ERR_DEVICE_CHECK
    run.step([200], *rows(200))
    assert run.ws is not small, "the larger chunk needs the tensor-core kernel's partials"
    assert run.status() == qsa.QSA_ERR_DEVICE_CHECK and run.status() == qsa.QSA_OK


DEBUG_CHILD = r"""
import torch
from block_sparse_long_15_b200 import qsa
from tests import test_paged_gpu as T
assert qsa.LIB_PATH.endswith("libqsa_debug.so"), qsa.LIB_PATH
s = T._run(qsa, ("bf16", 16, 2, 128, 64, 64, 3, [4, 0, 2], [700, 9, 120]))
T._attn(qsa, s)
assert qsa.qsa_read_device_status(s["ws"]) == qsa.QSA_OK, "a valid selection was flagged"
good = s["sel"].clone()  # packed row 1 is the first of sequence 0 (n_c = 10), row 6 the last of sequence 2 (n_c = 1)
def swap(x): x[1, 0], x[1, 1] = good[1, 1], good[1, 0]
def out_of_range(x): x[1, 2] = 10
def early_end(x): x[1, 2] = -1
def one_too_many(x): x[6, 1] = 0
for spoil in (swap, out_of_range, early_end, one_too_many):
    s["sel"].copy_(good)
    spoil(s["sel"])
    T._attn(qsa, s)
    assert qsa.qsa_read_device_status(s["ws"]) == qsa.QSA_ERR_DEVICE_CHECK, spoil.__name__
print("DEBUG_CHECKS_OK")
"""


def test_debug_build_checks_packed_selections(cuda_lib):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, QSA_LIBRARY="libqsa_debug.so", PYTHONPATH=root)
    r = subprocess.run([sys.executable, "-c", DEBUG_CHILD], cwd=root, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "DEBUG_CHECKS_OK" in r.stdout, r.stdout + r.stderr


# ------------------------------------------------------------------ a run of them together
@pytest.mark.parametrize("dtype,Hq,Hkv,d,block,topk,page", [("bf16", 16, 2, 128, 64, 3, 16), ("bf16", 16, 2, 256, 64, 3, 64),
                                                          ("fp32", 4, 1, 64, 32, 4, 32)])
@pytest.mark.parametrize("selected", [False, True])
def test_serving_run(cuda_lib, dtype, Hq, Hkv, d, block, topk, page, selected):
    """Prompts in chunks, then drafted tokens and single ones, slots coming and going: every output
    against the plain form over what the cache should hold by then, every selection against
    qsa_forward's on contiguous caches."""
    from block_sparse_long_15_b200.runner import QSAPaged
    qsa, dt, di, Hi = cuda_lib, DT[dtype], 64, 4
    cfg = qsa.make_config(Hq, Hkv, d, Hi, di, block, topk, dtype)
    gen = torch.Generator().manual_seed(12)
    w = [(torch.randn(d, generator=gen) * 0.2 + 1).to(dt).cuda() for _ in range(2)]
    rot, theta = d // 2, 1e6
    nr = qsa.make_norm_rope(*w, eps=1e-6, rope_theta=theta, rotary_dim=rot, indexer_rotary_dim=64)
    run = QSAPaged(cfg, slots=3, max_len=640, n_pages=3 * 640 // page, page_size=page, norm_rope=nr)
    seen = [dict(k=[], v=[], ki=[]) for _ in range(3)]
    steps = [[200, 0, 33], [130, 64, 1], [1, 1, 1], [4, 0, 3], "release 0", [70, 1, 0], [1, 1, 1]]
    for counts in steps:
        if counts == "release 0":
            run.release(0)
            seen[0] = dict(k=[], v=[], ki=[])
            continue
        n = sum(counts)
        q, k, v = (torch.randn(n, h, d, generator=gen).to(dt).cuda() for h in (Hq, Hkv, Hkv))
        qi, ki = (torch.randn(n, Hi, di, generator=gen).to(dt).cuda(), torch.randn(n, di, generator=gen).to(dt).cuda())
        out = run.step(counts, q, k, v, qi if selected else None, ki if selected else None)
        assert run.status() == qsa.QSA_OK
        row = 0
        for s, c in enumerate(counts):
            mine = slice(row, row + c)
            row += c
            if c == 0:
                continue
            t0 = sum(len(x) for x in seen[s]["k"])
            pos = torch.arange(t0, t0 + c, device="cuda")
            # the library's own norm and rotation (tested above): the attention is in question here
            qr, kr, pos32 = torch.empty_like(q[mine]), torch.empty_like(k[mine]), pos.to(torch.int32)
            qsa.qsa_norm_rope(cfg, nr, pos32, q[mine], k[mine], qr, kr)
            kir = U.rotate(ki[mine].double()[:, None], pos, 64, theta)[:, 0].to(dt)
            for name, x in (("k", kr), ("v", v[mine]), ("ki", kir)):
                seen[s][name].append(x)
            length = t0 + c
            K, V = (torch.cat(seen[s][x]).transpose(0, 1)[None] for x in ("k", "v"))  # one page of all tokens
            sel = None
            if selected:
                assert run.length[s] == length
                # the indexer keys that were stored are the rotated ones
                U.check(run.ki_cache[s, :length], torch.cat(seen[s]["ki"]).double(),
                        torch.full((length, di), U.HALF[dt] * 8, device="cuda"), "ki")
                kbar = torch.zeros(1, 640 // block, di, device="cuda")
                lens = torch.tensor([length], dtype=torch.int32, device="cuda")
                zero = torch.zeros(1, dtype=torch.int32, device="cuda")
                qsa.qsa_compress_blocks(cfg, run.ki_cache[s:s + 1], zero, lens, kbar)
                sel = torch.empty(1, c, topk, dtype=torch.int32, device="cuda")
                ws = qsa.alloc_workspace(cfg, qsa.QSA_PREFILL, 1, c, 640)
                qsa.qsa_index_score_topk(cfg, qi[mine][None].contiguous(), kbar, lens, lens - c, 640, sel, ws)
                sel = sel[0]
            want, tol = U.attention(qr, K, V, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), [c], [length],
                                    1 / math.sqrt(d), block, sel)
            U.check(out[mine], want, tol, f"slot {s} after {t0} tokens")
    assert sorted(run.free + sum(run.pages, [])) == list(range(run.n_pages))
