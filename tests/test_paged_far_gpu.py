"""Offsets that pass 32 bits, and calls at once on two streams."""
import math

import pytest
import torch

from tests import paged_util as U
from tests import test_paged_gpu as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,Hq,Hkv,d,topk,q_len,kv_len", [
    ("bf16", 16, 2, 128, 0, [1, 2, 1], [700, 300, 64]),
    ("bf16", 16, 2, 128, 3, [1, 2, 1], [700, 300, 64]),
    ("bf16", 16, 2, 128, 0, [150, 1, 40], [700, 300, 64]),
    ("bf16", 16, 2, 256, 0, [50, 1, 40], [700, 300, 64]),
    ("fp32", 8, 2, 128, 0, [1, 20, 3], [700, 300, 64]),
])
def test_pages_behind_2_to_the_32_elements(cuda_lib, dtype, Hq, Hkv, d, topk, q_len, kv_len):
    """Append and attention in pages from both ends of a pool of more than 2^32 elements (fp32: bytes)."""
    qsa, dt, page = cuda_lib, T.DT[dtype], 64
    n_pages = 2 ** (32 if dtype == "bf16" else 31) // (Hkv * page * d) + 40
    kp, vp = (torch.empty(n_pages, Hkv, page, d, dtype=dt, device="cuda") for _ in range(2))
    need = [-(-n // page) for n in kv_len]
    ids = [i // 2 if i % 2 else n_pages - 1 - i // 2 for i in range(sum(need))]
    table = torch.full((3, max(need)), -1, dtype=torch.int32)
    gen, at = torch.Generator().manual_seed(d), 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    for x in (kp, vp):
        x[torch.tensor(ids).cuda()] = torch.randn(len(ids), Hkv, page, d, generator=gen).to(dt).cuda()
    start = torch.tensor([0] + q_len).cumsum(0).to(torch.int32)
    pg = qsa.make_paged(start.cuda(), torch.tensor(kv_len, dtype=torch.int32).cuda(), table.cuda(), n_tok=sum(q_len),
                        max_chunk=max(q_len), page_size=page, n_pages=n_pages)
    q, k, v = (torch.randn(sum(q_len), h, d, generator=gen).to(dt).cuda() for h in (Hq, Hkv, Hkv))
    cfg = T._cfg(qsa, Hq, Hkv, d, topk=max(topk, 1), dtype=dtype)
    ws = qsa.alloc_paged_workspace(cfg, pg)
    qsa.qsa_paged_append(cfg, None, pg, k, v, kp, vp, ws)
    for row, b, t in U.positions(q_len, kv_len):
        assert torch.equal(kp[table[b, t // page], :, t % page], k[row]) and torch.equal(vp[table[b, t // page], :, t % page], v[row])
    sel = U.selection(q_len, kv_len, 64, topk, 3).cuda() if topk else None
    out = torch.empty_like(q)
    qsa.qsa_paged_attn(cfg, pg, q, kp, vp, sel, out, ws)
    assert qsa.qsa_read_device_status(ws) == qsa.QSA_OK
    U.check(out, *U.attention(q, kp, vp, table.cuda(), q_len, kv_len, 1 / math.sqrt(d), 64, sel), "out")


@pytest.mark.parametrize("topk,q_len,kv_len", [(0, [1, 2], [300, 64]), (0, [150, 1], [300, 64]), (2, [20, 3], [300, 64])])
def test_rows_behind_2_to_the_32_elements(cuda_lib, topk, q_len, kv_len):
    """Packed rows that begin behind 2^32 elements of q and out, in front of them a million rows of no sequence."""
    qsa, dt, Hq, Hkv, d = cuda_lib, torch.bfloat16, 16, 2, 256
    lead, n = 2 ** 32 // (Hq * d) + 5, sum(q_len)
    g = U.make_batch(q_len, kv_len, 64, seed=4, lead=lead, tail=1)
    kp, vp = U.pools(Hkv, d, g, kv_len, dt, seed=5)
    q = torch.empty(lead + n + 1, Hq, d, dtype=dt, device="cuda")
    rows = slice(lead, lead + n)
    q[rows] = torch.randn(n, Hq, d, generator=torch.Generator().manual_seed(6)).to(dt).cuda()
    sel = None
    if topk:
        sel = torch.full((lead + n + 1, topk), -1, dtype=torch.int32, device="cuda")
        sel[rows] = U.selection(q_len, kv_len, 64, topk, 3).cuda()
    out = torch.empty_like(q)
    out[lead - 1], out[-1] = 7, 7
    cfg, pg = T._cfg(qsa, Hq, Hkv, d, topk=max(topk, 1)), qsa.make_paged(**g)
    ws = qsa.alloc_paged_workspace(cfg, pg)
    qsa.qsa_paged_attn(cfg, pg, q, kp, vp, sel, out, ws)
    assert qsa.qsa_read_device_status(ws) == qsa.QSA_OK
    U.check(out[rows], *U.attention(q[rows], kp, vp, g["page_table"], q_len, kv_len, 1 / math.sqrt(d), 64,
                                    None if sel is None else sel[rows]), "out")
    assert (out[lead - 1] == 7).all() and (out[-1] == 7).all()
    # norm and rotation of all of them, in place
    w = torch.ones(d, dtype=dt, device="cuda")
    pos = torch.arange(lead + n + 1, dtype=torch.int32, device="cuda")
    nr = qsa.make_norm_rope(w, w, rope_theta=1e6, rotary_dim=d)
    want, tol = U.norm_rope(q[rows], w, pos[rows], 1e-6, 0.0, d, 1e6)
    qsa.qsa_norm_rope(cfg, nr, pos, q, None, q, None)
    U.check(q[rows], want, tol, "q")


@pytest.mark.parametrize("a,b", [(T.CASES[0], T.CASES[13]), (T.CASES[15], T.CASES[13]), (T.CASES[20], T.CASES[31])],
                         ids=["rows and tiles", "one tile and two", "split and CUDA cores"])
def test_two_calls_at_once(cuda_lib, a, b):
    """On two streams, each with its workspace: the bits of calls one after the other."""
    qsa = cuda_lib
    calls = [T._run(qsa, a, lead=0, tail=0), T._run(qsa, b, seed=5, lead=0, tail=0)]
    want = []
    for s in calls:
        T._attn(qsa, s)
        want.append(s["out"].clone())
        s["outs"] = [torch.full_like(s["out"], 7.0) for _ in range(20)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for i in range(20):
        for s, stream in zip(calls, streams):
            s["out"] = s["outs"][i]
            T._attn(qsa, s, stream=stream)
    torch.cuda.synchronize()
    for s, w in zip(calls, want):
        assert all(torch.equal(o, w) for o in s["outs"])
        assert qsa.qsa_read_device_status(s["ws"]) == qsa.QSA_OK
