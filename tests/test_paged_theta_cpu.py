"""The bases of the rotary frequencies that the norm and rotation take, on the host (no GPU)."""
import ctypes
import os
import re

import pytest

from block_sparse_long_15_b200 import build

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qsa.h")


@pytest.mark.parametrize("theta,served", [(1.0, True), (1.25, True), (1e4, True), (3e38, True), (0.999, False), (0.5, False),
                                          (3.2e38, False), (float("inf"), False)])
@pytest.mark.parametrize("rot,rot_i", [(128, 0), (0, 64), (128, 64)])
def test_rotary_bases(theta, served, rot, rot_i):
    build.build()
    from block_sparse_long_15_b200 import qsa
    cfg = qsa.make_config(Hq=16, Hkv=2, d=128, Hi=4, di=64, block=64, topk=32)
    nr = qsa.qsa_norm_rope_t(1e-6, 0.0, theta, rot, rot_i, None, None)
    got = qsa.library().qsa_norm_rope(ctypes.byref(cfg), ctypes.byref(nr), None, 0, None, 0, None, 0, None, 0, None, 0, None)
    assert got == (qsa.QSA_OK if served else qsa.QSA_ERR_INVALID_ARG)


def test_the_header_names_the_bases_that_are_served():
    params = re.search(r"typedef struct \{([^}]*)\} qsa_norm_rope_t;", open(HEADER).read()).group(1)
    assert re.search(r"float rope_theta;\s*/\* 1 \.\. 3e38 ", params)
