"""The paged cache over many steps, long caches and wide tables, against the
float64 reference."""

import math

import numpy as np
import pytest

import paged_ref as ref
from test_gpu_paged import Case, check_evict, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw,keep", [
    # tables wide enough for the smaller blocks of moves, and just not
    (dict(lens=(3000, 20, 700, 1500), Hkv=8, G=1, d=64, ps=256, max_pages=64), 512),
    (dict(lens=(3000, 20, 700, 1500), Hkv=8, G=1, d=64, ps=256, max_pages=63), 512),
    (dict(lens=(2000, 3000, 0, 257, 256, 1), Hkv=2, G=1, dtype="f32", ps=256, max_pages=512), 256),
    (dict(lens=(9000, 8193), Hkv=8, G=1, d=64, ps=256, max_pages=256), 8192),
])
def test_evict_with_wide_tables(kw, keep):
    c = Case(**kw)
    check_evict(c, keep, 4, 64)
    assert status() == 0
