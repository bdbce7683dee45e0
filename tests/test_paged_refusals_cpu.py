"""A refused step of the paged cache leaves the slots as they were, whichever of its calls refuses (no GPU)."""
import pytest
import torch

from block_sparse_long_15_b200 import build

CALLS = ("make_paged", "qsa_paged_workspace_size", "qsa_paged_append", "qsa_compress_blocks", "qsa_workspace_size",
         "qsa_index_score_topk", "qsa_paged_attn")


@pytest.fixture(scope="module")
def qsa():
    build.build()
    from block_sparse_long_15_b200 import qsa as q
    return q


def _state(r):
    return ([list(p) for p in r.pages], list(r.length), list(r.indexed), list(r.free), r.kbar_blocks.tolist())


def _rows(cfg, n):
    shapes = dict(q=(n, 16, 128), k=(n, 2, 128), v=(n, 2, 128), qi=(n, 4, 64), ki=(n, 64))
    return {x: torch.zeros(*s, dtype=torch.bfloat16) for x, s in shapes.items()}


@pytest.mark.parametrize("call", CALLS)
def test_a_step_refused_by_any_of_its_calls(qsa, monkeypatch, call):
    """The calls are stood in for on the host; `call` refuses once, in the second step. The slots do not move, and
    the third step sees the lengths and pages that the second one saw."""
    from block_sparse_long_15_b200.runner import QSAPaged
    cfg = qsa.make_config(Hq=16, Hkv=2, d=128, Hi=4, di=64, block=64, topk=32)
    r = QSAPaged(cfg, slots=3, max_len=512, n_pages=12, page_size=64, device="cpu")
    seen, refuse = [], [False]

    class Batch:
        def __init__(self, q_start, kv_len, page_table):
            self.kv_len = kv_len
            seen.append((q_start.tolist(), kv_len.tolist(), page_table.clone()))

    def compress(cfg, ki, kv_start, kv_len, kbar, blocks_done=None, kbar_blocks=None, stream=None):
        kbar_blocks.copy_(kv_len // 64)
    fakes = dict(make_paged=lambda q_start, kv_len, page_table, **kw: Batch(q_start, kv_len, page_table),
                 qsa_paged_workspace_size=lambda *a: 512, qsa_paged_append=lambda *a, **kw: None, qsa_compress_blocks=compress,
                 qsa_workspace_size=lambda *a: 512, qsa_index_score_topk=lambda *a: a[6].fill_(-1),
                 qsa_paged_attn=lambda *a: None)

    def stand_in(name):
        def f(*a, **kw):
            if refuse[0] and name == call:
                raise qsa.QSAError(qsa.QSA_ERR_INVALID_ARG, name)
            return fakes[name](*a, **kw)
        return f
    for name in CALLS:
        monkeypatch.setattr(qsa, name, stand_in(name))
    r.step([65, 0, 3], **_rows(cfg, 68))
    assert r.length == [65, 0, 3] and r.kbar_blocks.tolist() == [1, 0, 0]
    before = _state(r)
    refuse[0] = True
    with pytest.raises(qsa.QSAError):
        r.step([70, 64, 130], **_rows(cfg, 264))
    assert _state(r) == before
    refuse[0] = False
    r.step([70, 64, 130], **_rows(cfg, 264))
    assert r.length == [135, 64, 133] == r.indexed and r.kbar_blocks.tolist() == [2, 1, 2]
    assert [len(p) for p in r.pages] == [3, 1, 3]
    tries = seen[1:] if call != "make_paged" else [seen[1], seen[1]]
    for x, y in zip(*tries):
        assert torch.equal(x, y) if torch.is_tensor(x) else x == y
    assert sorted(r.free + sum(r.pages, [])) == list(range(12))


def test_tensors_on_another_device(qsa):
    """Right shapes and types on the host: refused by the binding, after the shapes have been looked at."""
    from block_sparse_long_15_b200.runner import QSAPaged
    cfg = qsa.make_config(Hq=16, Hkv=2, d=128, Hi=4, di=64, block=64, topk=32)
    r = QSAPaged(cfg, slots=2, max_len=256, n_pages=8, page_size=64, device="cpu")
    before = _state(r)
    rows = _rows(cfg, 3)
    for kw in (rows, {x: rows[x] for x in ("q", "k", "v")}):
        with pytest.raises(ValueError):
            r.step([3, 0], **kw)
        assert _state(r) == before


def test_counts_of_another_number_of_slots(qsa):
    from block_sparse_long_15_b200.runner import QSAPaged
    cfg = qsa.make_config(Hq=16, Hkv=2, d=128, Hi=4, di=64, block=64, topk=32)
    r = QSAPaged(cfg, slots=2, max_len=256, n_pages=8, page_size=64, device="cpu")
    before = _state(r)
    for counts in ([3], [1, 1, 1]):
        with pytest.raises(ValueError):
            r.step(counts, **_rows(cfg, 3))
        assert _state(r) == before
