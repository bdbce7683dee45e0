"""Refusals of the paged-cache entry points on the host, before anything is enqueued (no GPU)."""
import ctypes

import pytest
import torch

from block_sparse_long_15_b200 import build


@pytest.fixture(scope="module")
def qsa():
    build.build()
    from block_sparse_long_15_b200 import qsa as q
    return q


GOOD, BAD = 0x10000, 0x10008  # never dereferenced


def _cfg(qsa, **kw):
    return qsa.make_config(**{**dict(Hq=16, Hkv=2, d=128, Hi=4, di=64, block=64, topk=32), **kw})


def _pg(qsa, **kw):
    f = dict(batch=2, n_tok=8, max_chunk=4, page_size=64, n_pages=10, max_pages=4, q_start=GOOD, kv_len=GOOD,
             page_table=GOOD)
    f.update(kw)
    return qsa.qsa_paged_t(**f)


def _nr(qsa, **kw):
    f = dict(eps=1e-6, weight_offset=0.0, rope_theta=1e6, rotary_dim=128, indexer_rotary_dim=64, q_weight=GOOD,
             k_weight=GOOD)
    f.update(kw)
    return qsa.qsa_norm_rope_t(**f)


def _attn(qsa, cfg=None, pg=None, q=GOOD, k=GOOD, v=GOOD, sel=None, out=GOOD, ws=GOOD, n=1 << 40):
    return qsa.library().qsa_paged_attn(ctypes.byref(cfg or _cfg(qsa)), ctypes.byref(pg or _pg(qsa)), q, k, v, sel, out,
                                        ws, n, None)


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(n_tok=-1), dict(max_chunk=-1), dict(n_pages=-1), dict(max_pages=-1),
                                dict(page_size=0), dict(page_size=-64), dict(page_size=48), dict(max_chunk=0),
                                dict(n_pages=0), dict(max_pages=0), dict(q_start=None), dict(kv_len=None),
                                dict(page_table=None)])
def test_bad_batches(qsa, kw):
    assert _attn(qsa, pg=_pg(qsa, **kw)) == qsa.QSA_ERR_INVALID_ARG
    t = qsa.qsa_append_t(k=GOOD, v=GOOD, k_row=256, v_row=256, k_pages=GOOD, v_pages=GOOD)
    assert qsa.library().qsa_paged_append(ctypes.byref(_cfg(qsa)), None, ctypes.byref(_pg(qsa, **kw)), ctypes.byref(t),
                                          GOOD, 256, None) == qsa.QSA_ERR_INVALID_ARG


@pytest.mark.parametrize("page", [1, 8, 65536])
def test_page_sizes_that_are_not_served(qsa, page):
    assert _attn(qsa, pg=_pg(qsa, page_size=page)) == qsa.QSA_ERR_UNSUPPORTED
    n = ctypes.c_size_t(0)
    assert qsa.library().qsa_paged_workspace_size(ctypes.byref(_cfg(qsa)), ctypes.byref(_pg(qsa, page_size=page)),
                                                  ctypes.byref(n)) == qsa.QSA_ERR_UNSUPPORTED


def test_bad_attention_arguments(qsa):
    L = qsa.library()
    for name in ("q", "k", "v", "out", "ws"):
        assert _attn(qsa, **{name: None}) == qsa.QSA_ERR_INVALID_ARG
        assert _attn(qsa, **{name: BAD}) == qsa.QSA_ERR_INVALID_ARG
    assert _attn(qsa, sel=BAD) == qsa.QSA_ERR_INVALID_ARG
    n = ctypes.c_size_t(0)
    cp, pp = ctypes.byref(_cfg(qsa)), ctypes.byref(_pg(qsa))
    assert L.qsa_paged_workspace_size(cp, pp, ctypes.byref(n)) == qsa.QSA_OK and n.value >= 256
    assert _attn(qsa, n=n.value - 256) == qsa.QSA_ERR_INVALID_ARG  # the workspace is too small
    assert L.qsa_paged_workspace_size(cp, pp, None) == qsa.QSA_ERR_INVALID_ARG
    assert L.qsa_paged_workspace_size(cp, None, ctypes.byref(n)) == qsa.QSA_ERR_INVALID_ARG
    assert L.qsa_paged_attn(cp, None, GOOD, GOOD, GOOD, None, GOOD, GOOD, 1 << 40, None) == qsa.QSA_ERR_INVALID_ARG
    assert _attn(qsa, cfg=_cfg(qsa, Hq=15)) == qsa.QSA_ERR_INVALID_ARG


def test_empty_batches_do_nothing(qsa):
    for kw in (dict(batch=0), dict(n_tok=0)):
        pg = _pg(qsa, **kw, q_start=None, kv_len=None, page_table=None)
        assert _attn(qsa, pg=pg, q=None, k=None, v=None, out=None, ws=None, n=0) == qsa.QSA_OK
        t = qsa.qsa_append_t()
        assert qsa.library().qsa_paged_append(ctypes.byref(_cfg(qsa)), None, ctypes.byref(pg), ctypes.byref(t), None, 0,
                                              None) == qsa.QSA_OK
    assert qsa.library().qsa_norm_rope(ctypes.byref(_cfg(qsa)), ctypes.byref(_nr(qsa)), None, 0, None, 0, None, 0, None, 0,
                                       None, 0, None) == qsa.QSA_OK


def _norm(qsa, nr=None, cfg=None, pos=GOOD, n=4, **kw):
    a = dict(q=GOOD, q_row=2048, q_out=GOOD, q_out_row=2048, k=GOOD, k_row=256, k_out=GOOD, k_out_row=256)
    a.update(kw)
    return qsa.library().qsa_norm_rope(ctypes.byref(cfg or _cfg(qsa)), ctypes.byref(nr or _nr(qsa)), pos, n, *a.values(),
                                       None)


@pytest.mark.parametrize("kw", [dict(eps=-1.0), dict(eps=float("nan")), dict(weight_offset=float("nan")),
                                dict(rotary_dim=-16), dict(rotary_dim=24), dict(rotary_dim=144), dict(rope_theta=0.0),
                                dict(rope_theta=0.5), dict(rope_theta=float("inf")), dict(rope_theta=float("nan")),
                                dict(indexer_rotary_dim=8), dict(indexer_rotary_dim=80), dict(q_weight=BAD),
                                dict(k_weight=BAD)])
def test_bad_norm_rope_parameters(qsa, kw):
    assert _norm(qsa, nr=_nr(qsa, **kw)) == qsa.QSA_ERR_INVALID_ARG
    t = qsa.qsa_append_t(k=GOOD, v=GOOD, k_row=256, v_row=256, k_pages=GOOD, v_pages=GOOD)
    assert qsa.library().qsa_paged_append(ctypes.byref(_cfg(qsa)), ctypes.byref(_nr(qsa, **kw)), ctypes.byref(_pg(qsa)),
                                          ctypes.byref(t), GOOD, 256, None) == qsa.QSA_ERR_INVALID_ARG


def test_bad_norm_rope_rows(qsa):
    assert _norm(qsa, pos=None) == qsa.QSA_ERR_INVALID_ARG
    assert _norm(qsa, n=-1) == qsa.QSA_ERR_INVALID_ARG
    for x in ("q", "k"):
        assert _norm(qsa, **{x: BAD}) == qsa.QSA_ERR_INVALID_ARG
        assert _norm(qsa, **{x + "_out": None}) == qsa.QSA_ERR_INVALID_ARG
        assert _norm(qsa, **{x + "_out": BAD}) == qsa.QSA_ERR_INVALID_ARG
        assert _norm(qsa, **{x + "_row": 248}) == qsa.QSA_ERR_INVALID_ARG      # shorter than the heads
        assert _norm(qsa, **{x + "_row": 4100}) == qsa.QSA_ERR_INVALID_ARG     # not 16-byte steps
        assert _norm(qsa, **{x + "_row": 4096}) == qsa.QSA_ERR_INVALID_ARG     # in place with another stride
    assert qsa.library().qsa_norm_rope(ctypes.byref(_cfg(qsa)), None, GOOD, 4, GOOD, 2048, GOOD, 2048, None, 0, None, 0,
                                       None) == qsa.QSA_ERR_INVALID_ARG


def test_bad_append_rows(qsa):
    L = qsa.library()
    good = dict(k=GOOD, v=GOOD, k_row=256, v_row=256, k_pages=GOOD, v_pages=GOOD, q=GOOD, q_row=2048, q_out=GOOD,
                q_out_row=2048, ki=GOOD, ki_row=64, ki_cache=GOOD, ki_cap=100)

    def call(ws=GOOD, n=256, t=True, **kw):
        a = qsa.qsa_append_t(**{**good, **kw})
        return L.qsa_paged_append(ctypes.byref(_cfg(qsa)), ctypes.byref(_nr(qsa)), ctypes.byref(_pg(qsa)),
                                  ctypes.byref(a) if t else None, ws, n, None)

    for name in ("k", "v", "k_pages", "v_pages", "q_out", "ki_cache"):
        assert call(**{name: None}) == qsa.QSA_ERR_INVALID_ARG, name
    for name in ("k", "v", "k_pages", "v_pages", "q", "q_out", "ki", "ki_cache"):
        assert call(**{name: BAD}) == qsa.QSA_ERR_INVALID_ARG, name
    for name, row in (("k_row", 248), ("v_row", 260), ("q_row", 2040), ("q_out_row", 2052), ("ki_row", 56),
                      ("ki_cap", -1)):
        assert call(**{name: row}) == qsa.QSA_ERR_INVALID_ARG, name
    assert call(q_row=4096) == qsa.QSA_ERR_INVALID_ARG
    assert call(ws=None) == qsa.QSA_ERR_INVALID_ARG
    assert call(ws=BAD) == qsa.QSA_ERR_INVALID_ARG
    assert call(n=255) == qsa.QSA_ERR_INVALID_ARG
    assert call(t=False) == qsa.QSA_ERR_INVALID_ARG


def test_binding_checks_shapes(qsa):
    import torch
    with pytest.raises(ValueError):  # a page table of another batch
        qsa.make_paged(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                       torch.zeros(3, 4, dtype=torch.int32), n_tok=1, max_chunk=1, page_size=16, n_pages=4)
    with pytest.raises(ValueError):  # q_start has one entry more than the batch
        qsa.make_paged(torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                       torch.zeros(2, 4, dtype=torch.int32), n_tok=1, max_chunk=1, page_size=16, n_pages=4)
    with pytest.raises(ValueError):  # host tensors
        qsa.make_paged(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                       torch.zeros(2, 4, dtype=torch.int32), n_tok=1, max_chunk=1, page_size=16, n_pages=4)
    with pytest.raises(ValueError):
        qsa._rows(torch.zeros(4, 2, 256)[:, :, ::2], torch.float32, (4, 2, 128), "q")


def test_page_bookkeeping(qsa):
    """Pages are handed out and taken back on the host; a step that does not fit changes nothing."""
    from block_sparse_long_15_b200.runner import QSAPaged
    r = QSAPaged(_cfg(qsa), slots=3, max_len=256, n_pages=6, page_size=64, device="cpu")
    r.reserve([65, 0, 1])
    assert [len(p) for p in r.pages] == [2, 0, 1] and r.length == [65, 0, 1] and len(r.free) == 3
    r.reserve([63, 64, 0])
    assert [len(p) for p in r.pages] == [2, 1, 1]
    for s in range(3):
        assert r.table[s, : len(r.pages[s])].tolist() == r.pages[s]
    before = ([list(p) for p in r.pages], list(r.length), list(r.free))
    for bad in ([1, 64, 64], [200, 0, 0], [0, -1, 0], [1, 1]):
        with pytest.raises(ValueError):
            r.reserve(bad)
        assert ([list(p) for p in r.pages], list(r.length), list(r.free)) == before
    r.release(0)
    assert r.length[0] == 0 and len(r.free) == 4
    assert sorted(r.free + sum(r.pages, [])) == list(range(6))
    with pytest.raises(ValueError):
        r.step([0, 0, 1], None, None, None, qi=None, ki=1)


def test_a_refused_step_changes_nothing(qsa):
    """A step whose tensors do not fit, or that selects over tokens without indexer keys, is refused
    before any length or page moves."""
    from block_sparse_long_15_b200.runner import QSAPaged
    cfg = _cfg(qsa)
    r = QSAPaged(cfg, slots=2, max_len=256, n_pages=8, page_size=64, device="cpu")
    r.reserve([64, 0])  # tokens that came without indexer keys
    before = ([list(p) for p in r.pages], list(r.length), list(r.indexed), list(r.free))

    def rows(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype)
    good = dict(q=rows(3, 16, 128), k=rows(3, 2, 128), v=rows(3, 2, 128))
    index = dict(qi=rows(3, 4, 64), ki=rows(3, 64))
    bad = [(dict(good, q=rows(2, 16, 128)), [0, 3]), (dict(good, k=rows(3, 4, 128)), [0, 3]),
           (dict(good, v=rows(3, 2, 128, dtype=torch.float32)), [0, 3]), (dict(good, **dict(index, ki=None)), [0, 3]),
           (dict(good, **dict(index, qi=rows(3, 4, 128))), [0, 3]), (dict(good, **dict(index, ki=rows(3, 32))), [0, 3]),
           (dict(good, **index), [3, 0]), (good, [300, -297])]
    for kw, counts in bad:
        with pytest.raises((ValueError, TypeError)):
            r.step(counts, **kw)
        assert ([list(p) for p in r.pages], list(r.length), list(r.indexed), list(r.free)) == before, (counts, kw.keys())
