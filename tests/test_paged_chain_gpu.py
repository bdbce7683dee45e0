"""From hidden states to attention over pages: projection with every packed token as a sequence of its own, norm
and rotation on the way into the pages, selection, attention. Each link against the plain 64-bit form of what
the link before it gave.

Projection: products of bf16 are exact in fp32, and a sum of D of them is off by at most 2 D 2^-24 sum |x| |w|
(additions that round or cut), then the result is rounded to bf16 once (2^-8). At position 0 the rotation is the
identity. The other links: paged_util."""
import math

import pytest
import torch

from tests import paged_util as U

pytestmark = pytest.mark.gpu

Hq, Hkv, d, Hi, di, D, BLOCK, TOPK, PAGE, THETA = 16, 2, 128, 4, 64, 512, 64, 3, 32, 1e6


def _project(qsa, cfg, x, w, first, rot=d):
    """The projected rows of the packed tokens x [n][D], each at position first[r] of its own sequence."""
    n = x.shape[0]
    new = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda")
    q, qi, k, v, ki = new(n, 1, Hq, d), new(n, 1, Hi, di), new(n, Hkv, 1, d), new(n, Hkv, 1, d), new(n, 1, di)
    pc = qsa.qsa_proj_config_t(D, THETA, rot, di)
    ws = qsa.qsa_project(cfg, pc, x[:, None], w, first, q, qi, k, v, ki)
    assert qsa.qsa_read_device_status(ws) == qsa.QSA_OK
    return dict(q=q[:, 0], qi=qi[:, 0], k=k[:, :, 0], v=v[:, :, 0], ki=ki[:, 0])


def _weights(gen):
    n_out = Hq * d + 2 * Hkv * d + Hi * di + di
    return (torch.randn(n_out, D, generator=gen) / math.sqrt(D)).to(torch.bfloat16).cuda()


def _exact(x, w):
    """(value, tolerance) of the projection, by kind of head."""
    y, a = x.double() @ w.double().T, x.double().abs() @ w.double().abs().T
    tol = U.HALF[torch.bfloat16] * y.abs() * 1.01 + 2 * D * 2.0 ** -24 * a
    out, at = {}, 0
    for name, heads, width in (("q", Hq, d), ("k", Hkv, d), ("v", Hkv, d), ("qi", Hi, di), ("ki", 1, di)):
        cut = slice(at, at + heads * width)
        shape = (len(x), di) if name == "ki" else (len(x), heads, width)
        out[name] = y[:, cut].reshape(shape), tol[:, cut].reshape(shape)
        at += heads * width
    return out


@pytest.mark.parametrize("selected", [False, True])
def test_hidden_states_to_attention(cuda_lib, selected):
    """Three sequences in chunks and single tokens, with head norms: q_first is zero, the append rotates."""
    from block_sparse_long_15_b200.runner import QSAPaged
    qsa, dt = cuda_lib, torch.bfloat16
    cfg = qsa.make_config(Hq, Hkv, d, Hi, di, BLOCK, TOPK, "bf16")
    cfg_i = qsa.make_config(Hi, 1, di, Hi, di, BLOCK, TOPK, "bf16")  # the indexer's heads as query heads
    gen = torch.Generator().manual_seed(5)
    w = _weights(gen)
    nw = [(torch.randn(d, generator=gen) * 0.2 + 1).to(dt).cuda() for _ in range(2)]
    nr = qsa.make_norm_rope(*nw, eps=1e-6, rope_theta=THETA, rotary_dim=d, indexer_rotary_dim=di)
    nr_i = qsa.make_norm_rope(rope_theta=THETA, rotary_dim=di)
    run = QSAPaged(cfg, slots=3, max_len=512, n_pages=48, page_size=PAGE, norm_rope=nr)
    held = [0, 0, 0]
    for counts in ([200, 0, 64], [70, 3, 1], [1, 1, 1]):
        n = sum(counts)
        x = torch.randn(n, D, generator=gen).to(dt).cuda()
        rows = _project(qsa, cfg, x, w, torch.zeros(n, dtype=torch.int32, device="cuda"))
        for name, (want, tol) in _exact(x, w).items():
            U.check(rows[name], want, tol, name)
        pos = torch.cat([torch.arange(h, h + c) for h, c in zip(held, counts)]).to(torch.int32).cuda()
        qi = torch.empty_like(rows["qi"])
        qsa.qsa_norm_rope(cfg_i, nr_i, pos, rows["qi"], None, qi, None)
        U.check(qi, *U.norm_rope(rows["qi"], None, pos, 0.0, 0.0, di, THETA), "qi")
        out = run.step(counts, rows["q"], rows["k"], rows["v"], *((qi, rows["ki"]) if selected else ()))
        assert run.status() == qsa.QSA_OK
        q = torch.empty_like(rows["q"])
        qsa.qsa_norm_rope(cfg, nr, pos, rows["q"], None, q, None)
        U.check(q, *U.norm_rope(rows["q"], nw[0], pos, 1e-6, 0.0, d, THETA), "q")
        row = 0
        for s, c in enumerate(counts):
            mine, t = slice(row, row + c), torch.arange(held[s], held[s] + c).cuda()
            row += c
            held[s] += c
            if c == 0:
                continue
            pages = run.table[s].cuda()[t // PAGE].long()
            U.check(run.k_pages[pages, :, t % PAGE], *U.norm_rope(rows["k"][mine], nw[1], t, 1e-6, 0.0, d, THETA), "k")
            assert torch.equal(run.v_pages[pages, :, t % PAGE], rows["v"][mine])
            sel = None
            if selected:
                U.check(run.ki_cache[s, t][:, None], *U.norm_rope(rows["ki"][mine][:, None], None, t, 0.0, 0.0, di, THETA), "ki")
                lens = torch.tensor([held[s]], dtype=torch.int32, device="cuda")
                kbar = torch.zeros(1, 512 // BLOCK, di, device="cuda")
                qsa.qsa_compress_blocks(cfg, run.ki_cache[s:s + 1], torch.zeros_like(lens), lens, kbar)
                sel = torch.empty(1, c, TOPK, dtype=torch.int32, device="cuda")
                qsa.qsa_index_score_topk(cfg, qi[mine][None].contiguous(), kbar, lens, lens - c, 512, sel,
                                         qsa.alloc_workspace(cfg, qsa.QSA_PREFILL, 1, c, 512))
                sel = sel[0]
            want, tol = U.attention(q[mine], run.k_pages, run.v_pages, run.table[s:s + 1].cuda(), [c], [held[s]],
                                    1 / math.sqrt(d), BLOCK, sel)
            U.check(out[mine], want, tol, f"slot {s} with {held[s]} tokens")


def test_positions_given_to_the_projection(cuda_lib):
    """Without head norms the projection may rotate at each token's own position, and the append copies: the
    pages hold what the append's own rotation gives, to the roundings of both (the projection's angle is formed in
    fp32: position times 2 roundings of 2^-24, on both of a pair, and one more rounding to bf16 in the other form)."""
    qsa, dt = cuda_lib, torch.bfloat16
    cfg = qsa.make_config(Hq, Hkv, d, Hi, di, BLOCK, TOPK, "bf16")
    gen = torch.Generator().manual_seed(6)
    w = _weights(gen)
    q_len, kv_len = [40, 1], [300, 77]
    g = U.make_batch(q_len, kv_len, PAGE, seed=2)
    pos = torch.tensor([t for _, _, t in U.positions(q_len, kv_len)], dtype=torch.int32).cuda()
    x = torch.randn(41, D, generator=gen).to(dt).cuda()
    turned, plain = _project(qsa, cfg, x, w, pos), _project(qsa, cfg, x, w, torch.zeros_like(pos))
    pools = [torch.zeros(g["n_pages"], Hkv, PAGE, d, dtype=dt, device="cuda") for _ in range(4)]
    ws, pg = torch.zeros(256, dtype=torch.uint8, device="cuda"), qsa.make_paged(**g)
    nr = qsa.make_norm_rope(rope_theta=THETA, rotary_dim=d)
    qsa.qsa_paged_append(cfg, None, pg, turned["k"], turned["v"], pools[0], pools[1], ws)
    qsa.qsa_paged_append(cfg, nr, pg, plain["k"], plain["v"], pools[2], pools[3], ws)
    assert qsa.qsa_read_device_status(ws) == qsa.QSA_OK
    assert torch.equal(pools[1], pools[3])
    y, tol = _exact(x, w)["k"]
    pair = y.abs().roll(d // 2, -1) + y.abs()
    both = tol.roll(d // 2, -1) + tol
    want = U.rotate(y, pos, d, THETA)
    angle = (2 * 2.0 ** -24 * pos.double() + 2.0 ** -21)[:, None, None]
    far = U.HALF[dt] * want.abs() * 1.01 + both + pair * angle
    page, slot = g["page_table"][torch.tensor([0] * 40 + [1]).cuda(), pos // PAGE].long(), (pos % PAGE).long()
    U.check(pools[0][page, :, slot], want, far, "rotated by the projection")
    U.check(pools[2][page, :, slot], want, far + U.HALF[dt] * both, "rotated by the append")
