"""Paged-cache calls at their edges: entries and counts out of range, forks of
many sequences, and how near the attention comes to float64 where the scores
are exact."""
import subprocess
import sys

import numpy as np
import pytest
import torch

import rope_aware_kv_b200 as tri
from rope_aware_kv_b200 import build as tri_build
from tests import paged_ref as R
from tests.test_gpu_paged import BF16, DEV, F32, _cache, _i32, _rows, _state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tri_build.build()
    tri.load()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("moves", [True, False])
def test_compact_flags_bad_entries(moves):
    """Entries below -1 or past the pool are left and flagged, whether or not
    a page moves; the others follow their pages."""
    page = 8
    table = np.array([[0, 4, -1], [1, -9, 6]] if moves else [[0, 1, -1], [2, -9, 6]], np.int32)
    refs = np.zeros(6, np.int32)
    refs[table[(table >= 0) & (table < 6)]] = 1
    k = torch.randn((6, page, R.D), device=DEV).to(BF16)
    want = k.clone()
    if moves:
        want[2] = k[4]
    t, c = _i32(table), _i32(refs)
    ws = tri.workspace(tri.tri_pages_workspace_bytes(2, 3, 6))
    assert tri.tri_pages_compact(k, None, t, c, ws=ws).item() == 3
    assert tri.tri_check_device_error(ws) == tri.FLAG_INDEX_RANGE
    assert t.cpu().tolist() == ([[0, 2, -1], [1, -9, 6]] if moves else [[0, 1, -1], [2, -9, 6]])
    assert c.cpu().tolist() == [1, 1, 1, 0, 0, 0]
    assert torch.equal(k, want)
    t = _i32(np.where((table < -1) | (table >= 6), -1, table))  # the same without them: no flag
    c = _i32(refs)
    tri.tri_pages_compact(want, None, t, c, ws=ws)
    assert tri.tri_check_device_error(ws) == 0
