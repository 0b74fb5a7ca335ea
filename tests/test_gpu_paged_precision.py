"""What the paged decode holds in float32: softmax weights, their products and sums.

Exact answers are known here, so the bounds are of single roundings and not of
sums of n of them.
"""

import math

import numpy as np
import pytest

import paged_ref as ref
from hga_testlib import to_f64
from test_gpu_paged import HALF_STEP, Case, status

pytestmark = pytest.mark.gpu


def bf16(x):
    """Nearest bf16 numbers (ties to even) of x, in float64."""
    import torch
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("max_pages", [None, 4096])  # the one-launch kernel, and two launches
@pytest.mark.parametrize("d", [64, 128])
def test_softmax_weights_enter_their_product_in_32_bits(d, max_pages):
    """Three slots a sequence: one of weight x < 1 and value 1, two of weight 1
    whose values take away the two bf16 numbers next to x.  What is left,
    x - r1 - r2, is 17 bits and more below x.

    Bound: scores are exact up to the scale (two roundings, 2^-23 |s|), ex2
    is good to 2^-22, three products' sums are cut off at 2^-23 of values
    below 1 (2^-22 in all); then the output's rounding."""
    c = Case(lens=(3,) * 64, Hkv=1, G=1, d=d, max_pages=max_pages)
    keys = bf16(np.linspace(-16, -1, 64) * math.sqrt(d / 128))
    s = keys * float(np.float32(d ** -0.5))
    x = np.exp(s)
    r1 = bf16(x)
    r2 = bf16(x - r1)
    left = x - r1 - r2
    assert np.abs(left).max() > 2.0 ** -20
    table = c.table.cpu().numpy()
    for b in range(64):
        pg, row, _ = ref.places(table[b], 3, c.ps, c.k.shape[0])
        c.k[pg, 0, row] = 0.0
        c.k[pg[0], 0, row[0], 0] = float(keys[b])
        for i, v in enumerate((1.0, -r1[b], -r2[b])):
            c.v[pg[i], 0, row[i]] = float(v)
    c.q.zero_()
    c.q[:, :, 0] = 1.0
    c.decode()
    want = left / (x + 2)
    tol = (x * (2.0 ** -22 + 2.0 ** -23 * np.abs(s)) + 2.0 ** -22) / (x + 2) + HALF_STEP["bf16"] * np.abs(want)
    err = np.abs(to_f64(c.o)[:, 0] - want[:, None])
    assert (err <= tol[:, None]).all(), (err / tol[:, None]).max()
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_are_not_cut_off(d, dtype):
    """One slot a sequence: LSE is its score.  Queries and keys above 0, so that
    sums that are cut off instead of rounded fall short.  A sum of 32 products
    in two instructions loses 2^-24 of its size in the mean, and half of that
    when it was half as long; additions are rounded, without an error in the
    mean."""
    import torch
    c = Case(dtype, lens=(1,) * 64, Hkv=8, G=8, d=d)
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    for x in (c.q, c.k):
        x.copy_(torch.rand(x.shape, generator=g, device="cuda"))
    c.cfg.scale = 0.125
    c.decode()
    q, k = to_f64(c.q).reshape(64, 8, 8, d), to_f64(c.k)
    rows = k[c.table[:, 0].cpu().numpy(), :, 0]                     # [B, Hkv, d]
    want = np.einsum("bhgd,bhd->bhg", q, rows).reshape(64, 64) * 0.125
    rel = (c.lse.double().cpu().numpy() - want) / want
    assert abs(rel.mean()) <= 1.5 * 2.0 ** -24, rel.mean() * 2.0 ** 24
    assert np.abs(rel).max() <= d * 2.0 ** -24


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_outputs_are_not_cut_off(d, dtype):
    """Slot t and slot t + n/2 have the same key and the values 1 and -1: the
    output is 0.  A warp's sum goes up over 64 tiles to half the weights' sum L
    and down again.  Each addition's rounding is up to 2^-24 of it, 2^-24 / 3^0.5
    in the mean square, and of 64 additions 8 * 2^-24 / 3^0.5 * L / 12^0.5; over
    the four warps of a block half of that, 0.7 * 2^-24.  Bound: 2 * 2^-24,
    and 8 times that for one head of the 224 (sums that are cut off lose all
    in one direction)."""
    import torch
    n, ps, B, Hkv = 4096 * 128 // d, 256, 28, 8
    if dtype == "f32":
        n //= 2
    c = Case(dtype, lens=(n,) * B, Hkv=Hkv, G=1, d=d, ps=ps, spare=0)
    g = torch.Generator(device="cuda")
    g.manual_seed(13)
    half = n // ps // 2
    for b in range(B):
        up, down = c.table[b, :half].long(), c.table[b, half:].long()
        c.k[down] = c.k[up]
        c.v[up], c.v[down] = 1.0, -1.0
    c.decode()
    o = to_f64(c.o)
    rms = math.sqrt((o ** 2).mean())
    assert rms <= 2.0 ** -23, rms * 2.0 ** 24
    assert np.abs(o).max() <= 2.0 ** -20


@pytest.mark.parametrize("max_pages", [None, 4096])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128)])
def test_lse_is_rounded_once(dtype, d, max_pages):
    """One slot a sequence, its product with the query exact: LSE is the
    product times the scale and half a step of float32 off at most."""
    c = Case(dtype, lens=(1,) * 256, Hkv=1, G=1, d=d, max_pages=max_pages)
    keys = bf16(np.linspace(-700, 900, 256))
    c.k.zero_()
    c.k[c.table[:, 0].long(), 0, 0, 0] = c.k.new_tensor(keys)
    c.q.zero_()
    c.q[:, :, 0] = 1.0
    c.cfg.scale = float(np.float32(d ** -0.5))
    c.decode()
    want = keys * c.cfg.scale
    err = np.abs(c.lse[:, 0].double().cpu().numpy() - want)
    assert (err <= 2.0 ** -24 * np.abs(want)).all(), (err / np.abs(want)).max() * 2.0 ** 24


@pytest.mark.parametrize("lens,max_pages", [
    ((64, 30, 5), None),            # one launch
    ((64, 30, 5), 4096),            # two launches, whole heads
    ((64,) * 300 + (0, 1), 512),    # most heads whole, some split between two blocks
    ((700,), 4096),                 # one head, split
])
@pytest.mark.parametrize("offset", [300.0, -300.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_of_a_head_add_up_to_its_query_heads(dtype, offset, lens, max_pages):
    """The softmax weights of a head add up to 1 a query head, however large
    LSE is and wherever the blocks' runs are cut.  Each weight is good to
    2^-21 next to its sum (ex2 2^-22 each), the sum to 2^-20 (up to 16
    additions one after the other), the additions to the records and 1 / sum to
    2^-21: bound 2^-19."""
    import torch
    c = Case(dtype, lens=lens, Hkv=2, G=2, max_pages=max_pages)
    # every score is the offset and a little
    c.k *= 0.125
    c.k[..., 0] = 1.0
    c.q.mul_(0.5)
    c.q[..., 0] = offset * 128 ** 0.5
    c.weight.zero_()
    c.decode(True)
    lse = c.lse[torch.tensor([n > 0 for n in lens], device="cuda")]
    assert 200 < float(lse.abs().min()) and float(lse.abs().max()) < 400
    w, table = c.weight.double().cpu().numpy(), c.table.cpu().numpy()
    for b, n in enumerate(lens):
        pg, row, _ = ref.places(table[b], n, c.ps, c.k.shape[0])
        for h in range(2):
            total = w[pg, h, row].sum()
            assert abs(total - 2 * (n > 0)) <= 2 * 2.0 ** -19, (b, h, (total - 2) * 2.0 ** 20)
    assert status() == 0
