"""Selections that neighbouring tokens share: the first blocks and the latest ones. A long unit is cut into equal
ranges of visible keys, so that many of its parts then hold no listed block, or a whole tile's none."""
import pytest
import torch

from tests import paged_util as U
from tests import test_paged_gpu as T

pytestmark = pytest.mark.gpu

# first blocks, latest blocks, case; a large budget sends chunks to the tile kernels
LISTS = [
    (2, 3, ("bf16", 16, 2, 128, 64, 64, 1024, [100], [33000])),
    (2, 0, ("bf16", 16, 2, 128, 16, 64, 1024, [100, 20], [33000, 5000])),   # the last parts hold the trailing range only
    (0, 2, ("bf16", 16, 2, 128, 64, 64, 1024, [15], [33000])),              # one tile, empty parts first
    (1, 1, ("bf16", 16, 2, 256, 32, 128, 1024, [70, 12], [30000, 640])),
    (3, 2, ("bf16", 8, 1, 64, 256, 64, 1024, [129], [33000])),
    (1, 0, ("bf16", 2, 2, 128, 64, 64, 1024, [200], [20000])),              # more segments than one a part
    (2, 3, ("bf16", 16, 2, 128, 64, 64, 32, [1, 1, 3], [33000, 700, 9000])),  # the row kernel
]


@pytest.mark.parametrize("first,last,case", LISTS, ids=[f"{f}-{z}-d{c[3]}-q{max(c[7])}" for f, z, c in LISTS])
def test_concentrated_lists(cuda_lib, first, last, case):
    qsa = cuda_lib
    block, topk, q_len, kv_len = case[5:9]
    s = T._run(qsa, case, pick=first + last)
    mine = s["sel"][s["rows"]]
    for row, _, t in U.positions(q_len, kv_len):
        n_c = (t + 1) // block
        ids = sorted(set(range(min(first, n_c))) | set(range(max(0, n_c - last), n_c)))
        mine[row] = -1
        mine[row, : len(ids)] = torch.tensor(ids, dtype=torch.int32)
    T._attn(qsa, s)
    assert qsa.qsa_read_device_status(s["ws"]) == qsa.QSA_OK
    U.check(s["out"][s["rows"]], *T._oracle(s, case), "out")
    assert (s["out"][:1] == 7).all() and (s["out"][-2:] == 7).all()
    again = s["out"].clone()
    s["out"].fill_(7.0)
    T._attn(qsa, s)
    assert torch.equal(again, s["out"])
