"""Steps of the paged cache that the binding or the library refuses after the shapes were right: the slots are as
they were, and the same step with inputs in order gives what a cache gives that never saw the refusal."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _cache(qsa, block=64, max_len=640, weights=None, rot=128):
    from block_sparse_long_15_b200.runner import QSAPaged
    cfg = qsa.make_config(16, 2, 128, 4, 64, block, 4, "bf16")
    w = weights or [torch.linspace(0.5, 1.5, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    nr = qsa.make_norm_rope(*w, rope_theta=1e6, rotary_dim=rot, indexer_rotary_dim=64)
    return QSAPaged(cfg, slots=2, max_len=max_len, n_pages=20, page_size=64, norm_rope=nr)


def _rows(n, seed):
    gen = torch.Generator().manual_seed(seed)
    shapes = dict(q=(n, 16, 128), k=(n, 2, 128), v=(n, 2, 128), qi=(n, 4, 64), ki=(n, 64))
    return {x: torch.randn(s, generator=gen).to(torch.bfloat16).cuda() for x, s in shapes.items()}


def _state(r):
    return ([list(p) for p in r.pages], list(r.length), list(r.indexed), list(r.free), r.kbar_blocks.tolist())


def _spoilt(rows, how):
    """The same rows in a form that is not served."""
    name, how = how.split()
    x = rows[name]
    if how == "transposed":
        x = x.transpose(0, 1).contiguous().transpose(0, 1)  # [n][heads][d], head by head in memory
    elif how == "misaligned":
        x = torch.zeros(x.shape[0], x[0].numel() + 4, dtype=x.dtype, device="cuda")[:, :-4].view(x.shape)
    elif how == "shifted":
        x = torch.zeros(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape)
    elif how == "host":
        x = x.cpu()
    return dict(rows, **{name: x})


@pytest.mark.parametrize("how", ["q transposed", "k transposed", "v transposed", "q misaligned", "v misaligned",
                                 "ki misaligned", "k shifted", "q host", "ki host", "qi host"])
def test_rows_that_are_not_served(cuda_lib, how):
    qsa = cuda_lib
    r, clean = _cache(qsa), _cache(qsa)
    for c in (r, clean):
        c.step([130, 0], **_rows(130, 1))
    before = _state(r)
    with pytest.raises((ValueError, RuntimeError)):
        r.step([70, 65], **_spoilt(_rows(135, 2), how))
    assert _state(r) == before
    for counts, seed in (([3, 65], 3), ([1, 1], 4)):
        rows = _rows(sum(counts), seed)
        assert torch.equal(r.step(counts, **rows), clean.step(counts, **rows))
    assert _state(r) == _state(clean) and r.status() == qsa.QSA_OK


@pytest.mark.parametrize("what", ["weights of another width", "weights of another type", "rotation wider than a head"])
def test_parameters_that_are_not_served(cuda_lib, what):
    qsa = cuda_lib
    w = None
    if "width" in what:
        w = [torch.ones(64, dtype=torch.bfloat16, device="cuda")] * 2
    elif "type" in what:
        w = [torch.ones(128, device="cuda")] * 2
    r = _cache(qsa, weights=w, rot=144 if "rotation" in what else 128)
    before = _state(r)
    with pytest.raises((ValueError, RuntimeError)):
        r.step([70, 65], **_rows(135, 2))
    assert _state(r) == before


def test_more_blocks_than_the_scoring_serves(cuda_lib):
    """The append has been made when the selection is refused; a step over every token goes on from where the slots were."""
    qsa = cuda_lib
    r, clean = (_cache(qsa, block=8, max_len=8 * 32769) for _ in range(2))
    before = _state(r)
    with pytest.raises(RuntimeError):
        r.step([70, 65], **_rows(135, 2))
    assert _state(r) == before
    for counts, seed in (([3, 65], 3), ([1, 1], 4)):
        rows = {x: y for x, y in _rows(sum(counts), seed).items() if x in "qkv"}
        assert torch.equal(r.step(counts, **rows), clean.step(counts, **rows))
    assert _state(r) == _state(clean) and r.status() == qsa.QSA_OK
