"""Infinite and NaN keys and values of the paged decode, against the formula in float64."""

import math

import numpy as np
import pytest

import paged_ref as ref
from hga_testlib import to_f64
from test_gpu_paged import HALF_STEP, PRODUCT, Case, status

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan


def formula(q, k, v, scale):
    """softmax(scale q.k) v of one head as it stands, the weights, and the two
    sums of the bounds over what is finite."""
    with np.errstate(invalid="ignore"):
        s = (k * q).sum(1) * scale
        p = np.exp(s - s.max())
        p = p / p.sum()
        o = (p[:, None] * v).sum(0)
        lse = s.max() + np.log(np.exp(s - s.max()).sum())
        reach = (np.abs(k) * np.abs(q)).sum(1)[np.isfinite(s)].max() * scale
        spread = (p[:, None] * np.where(np.isfinite(v), np.abs(v), 0)).sum(0)
    return o, lse, p, reach, spread


@pytest.mark.parametrize("max_pages", [None, 4096])     # one launch, two launches
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
def test_infinite_and_nan_keys_and_values(dtype, d, max_pages):
    """A score of -inf has the weight 0; one of +inf, or NaN, makes its query
    head NaN; an infinite or NaN value its element.  Nothing else is touched."""
    if max_pages is None:
        lens = (70, 1000)
    else:
        lens = (70, 3000)
    c = Case(dtype, d=d, Hkv=2, G=2, lens=lens, max_pages=max_pages, q_scale=1.0)
    table = c.table.cpu().numpy()

    def put(x, b, h, slot, e, value):
        x[int(table[b, slot // c.ps]), h, slot % c.ps, e] = value

    q = c.q
    q[0, :2] = q[0, :2].abs() + 0.125   # every product with -inf is -inf
    q[0, 2, 2], q[0, 3, 2] = 1.5, -0.75
    put(c.k, 0, 0, 5, 3, -INF)          # weight 0 for both heads
    put(c.k, 0, 0, 64, 0, -INF)
    put(c.k, 0, 1, 7, 2, INF)           # +inf for head 2, -inf for head 3
    last = lens[1] - 1
    put(c.v, 1, 0, last // 2, 9, INF)
    put(c.v, 1, 0, 17, 10, -INF)
    put(c.v, 1, 0, 4, 11, INF)          # inf - inf
    put(c.v, 1, 0, last, 11, -INF)
    put(c.v, 1, 0, 16, 12, INF)         # side by side, the same sign
    put(c.v, 1, 0, 17, 12, INF)
    put(c.v, 1, 1, 8, 1, NAN)
    before = c.host()[2]
    c.decode(True)
    assert status() == 0
    qh, (k, v, weight, _, _) = to_f64(c.q), c.host()
    o, lse = to_f64(c.o), c.lse.double().cpu().numpy()
    for b, n in enumerate(lens):
        pg, row, _ = ref.places(table[b], n, c.ps, c.k.shape[0])
        for h in range(2):
            total, e_max = np.zeros(n), 0.0
            for g in (2 * h, 2 * h + 1):
                want, want_lse, p, reach, spread = formula(qh[b, g], k[pg, h, row], v[pg, h, row],
                                                           d ** -0.5)
                total += p
                ds = (2 * d * 2.0 ** -24 + PRODUCT[dtype]) * reach
                e_max = max(e_max, 2 * ds + 2.0 ** -19 + n * 2.0 ** -23)
                tol = HALF_STEP[dtype] * np.abs(want) + (2 * ds + 2.0 ** -20 + PRODUCT[dtype]
                                                         + n * 2.0 ** -23) * spread
                fine = np.isfinite(want)
                got = o[b, g]
                assert (np.isnan(got) == np.isnan(want)).all(), (b, g, got, want)
                assert (got[np.isinf(want)] == want[np.isinf(want)]).all(), (b, g)
                assert (np.abs(got[fine] - want[fine]) <= tol[fine]).all(), (b, g)
                if math.isnan(want_lse):
                    assert math.isnan(lse[b, g])
                else:
                    assert abs(lse[b, g] - want_lse) <= ds + 2.0 ** -20 * (1 + abs(want_lse)) + n * 2.0 ** -23
            got, want = weight[pg, h, row].astype(np.float64), before[pg, h, row] + total
            assert (np.isnan(got) == np.isnan(want)).all()
            fine = np.isfinite(want)
            assert (np.abs(got[fine] - want[fine]) <= (e_max * total + 2.0 ** -23 * np.abs(want))[fine]).all()
            assert (got[total == 0] == before[pg, h, row][total == 0]).all()
    # what each of them does, said once without the formula
    assert np.isfinite(o[0, [0, 1, 3]]).all() and np.isnan(o[0, 2]).all()
    assert (o[1, :2, 9] == INF).all() and (o[1, :2, 10] == -INF).all() and np.isnan(o[1, :2, 11]).all()
    assert (o[1, :2, 12] == INF).all() and np.isnan(o[1, 2:, 1]).all()
    assert np.isfinite(np.delete(o[1, 2:], 1, axis=1)).all()


@pytest.mark.parametrize("max_pages", [None, 4096])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_values_under_weights_of_few_bits(dtype, max_pages):
    """Keys of 0: the weights, before they are divided by their sum, are 1, a
    number of one bit; an infinite value is infinite under it, and the other
    elements are the plain means of 1, 2 and 4 equal numbers."""
    c = Case(dtype, lens=(1, 2, 4), max_pages=max_pages)
    c.k.mul_(0.0).nan_to_num_(0.0)
    c.v.fill_(0.75)
    for b in range(3):
        c.v[int(c.table[b, 0]), 0, b, 5] = INF
        c.v[int(c.table[b, 0]), 1, 0, 6] = -INF
    c.decode(True)
    want = np.full(tuple(c.o.shape), 0.75)
    want[:, :4, 5], want[:, 4:, 6] = INF, -INF
    assert (to_f64(c.o) == want).all()
    assert status() == 0
