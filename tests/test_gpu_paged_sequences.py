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


@pytest.mark.parametrize("kw", [
    # one launch: two blocks an SM, and just more than that; clusters of four
    dict(lens=(33, 1, 17, 0) * 9 + (40,), Hkv=8, G=1, d=64), dict(lens=(33, 1, 17, 0) * 10, Hkv=8, G=1, d=64),
    dict(lens=(300, 2, 0, 190, 77) * 5, Hkv=4, G=2, d=64, ps=32), dict(lens=(90,) * 37, Hkv=12, G=2, ps=32),
    # as many heads as the GPU holds blocks, and one more
    dict(lens=(20, 5) * 37, Hkv=6, G=1, d=64), dict(lens=(20, 5, 9, 1, 16) * 89, Hkv=1, G=3, d=64),
])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_of_many_short_caches(kw, dtype):
    c = Case(dtype, **kw)
    before = c.host()[2]
    c.decode(True)
    c.check_decode(before)
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_through_the_steps_of_a_generation(dtype):
    """Captured steps of append + decode over a cache that is cut now and then:
    every step's share of the weights, what the append cleared and what the
    eviction moved, against the reference."""
    import torch
    from hierarchical_routed_sparse_hga_b200 import HGA_BF16, HGA_F32, Config, HgaPagedLayer
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    B, Hkv, G, d, ps = 3, 2, 2, 64, 16
    cfg = Config(B, Hkv * G, Hkv, d, 1, 1, HGA_BF16 if dtype == "bf16" else HGA_F32)
    layer = HgaPagedLayer(cfg, 24, ps, 8)
    g = torch.Generator(device="cuda")
    g.manual_seed(41)
    layer.table.copy_(torch.randperm(24, generator=g, device="cuda").view(3, 8).to(torch.int32))
    split = [Hkv * G * d, Hkv * d, Hkv * d]
    prompt = torch.tensor([60, 0, 31], dtype=torch.int32, device="cuda")
    qkv = torch.randn((B, 60, sum(split)), generator=g, device="cuda").to(tdt)
    layer.advance(prompt)
    layer.append(*qkv.split(split, -1), 1e6,
                 torch.zeros((B, Hkv * G, 60, d), dtype=tdt, device="cuda"), n_new=prompt)
    one = torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")
    qkv = torch.randn((B, 1, sum(split)), generator=g, device="cuda").to(tdt)
    q = torch.zeros((B, Hkv * G, 1, d), dtype=tdt, device="cuda")
    c = Case.__new__(Case)
    c.dtype, c.ps, c.cfg, c.cache = dtype, ps, cfg, layer.cache
    c.k, c.v, c.weight, c.slot_pos = layer.k, layer.v, layer.weight, layer.slot_pos
    c.table, c.n_slots, c.pos = layer.table, layer.n_slots, layer.pos
    c.q = q.view(B, Hkv * G, d)
    c.o = torch.zeros((B, Hkv * G, d), dtype=tdt, device="cuda")
    c.lse = torch.zeros((B, Hkv * G), device="cuda")

    def step():
        layer.advance(one)
        layer.append(*qkv.split(split, -1), 1e6, q, n_new=one)
        layer.decode(c.q, c.o, c.lse, accumulate=True)

    step()
    state = layer.n_slots.clone(), layer.pos.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    layer.n_slots.copy_(state[0]), layer.pos.copy_(state[1])
    table = layer.table.cpu().numpy()
    for i in range(40):
        qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
        before = c.host()[2]
        graph.replay()
        for b, n in enumerate(layer.n_slots.tolist()):
            if b != 1:      # the new slot's record begins at 0
                before[table[b, (n - 1) // ps], :, (n - 1) % ps] = 0.0
        c.check_decode(before)
        if max(layer.n_slots.tolist()) >= 80:
            k, v, w, p, t = c.host()
            ref.evict(k, v, w, p, t, layer.n_slots.cpu().numpy(), layer.pos.cpu().numpy(), 48, 4, 8)
            layer.evict(48, sinks=4, recent=8)
            np.testing.assert_array_equal(c.host()[2], w)
            np.testing.assert_array_equal(c.host()[3], p)
    assert layer.pos.tolist() == [60 + 41 - 1, -1, 31 + 41 - 1] and status() == 0


@pytest.mark.parametrize("kw", [
    dict(lens=(131071,), Hkv=2, d=128, ps=64, paired=True), dict(lens=(300001, 5), Hkv=1, G=8, d=64, ps=256),
    dict(lens=(4096, 4000, 4100, 3900), Hkv=4, d=128, ps=16),
])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_of_long_caches(kw, dtype):
    """Root mean square errors.  Values are independent, so an error of e in
    each product p v (root mean square) is one of e |o| in an output, and the
    sums' roundings are next to it.  Float32: the score's products (2^-23
    each, 128 of size 2, scale 0.09: 2.4e-7) and sums (1.6e-7), ex2 (1.2e-7),
    the two parts of v and p (0.8e-7, 1.2e-7), the sums of p v (1.3e-7): 3.8e-7;
    bound 2^-20, two and a half times that.  Float32 sums of all n products, or
    sums that are cut off, are above it.  Bf16: the same errors change the
    rounding of 3e-4 of the outputs (0.8 * 3.8e-7 * mean of |o|rms / |o|, about 6,
    against steps of 2^-7.5); bound 1e-3, and one output more."""
    c = Case(dtype, spare=0, **kw)
    before = c.host()[2]
    c.decode(True)
    c.check_decode(before)
    k, v, _, _, table = c.host()
    got = np.asarray(c.o.double().cpu())
    o, lse, _, _, _ = ref.decode(np.asarray(c.q.double().cpu()), k, v, table, c.lens, c.cfg.head_dim ** -0.5)
    long = [b for b, n in enumerate(c.lens) if n > 1000]
    err = got[long] - o[long]
    if dtype == "f32":
        assert math.sqrt((err ** 2).mean()) <= 2.0 ** -20 * math.sqrt((o[long] ** 2).mean())
    else:
        import torch
        rounded = torch.from_numpy(o[long]).to(torch.bfloat16).double().numpy()
        flips = (got[long] != rounded).sum()
        assert flips <= 1 + 1e-3 * rounded.size, flips / rounded.size
    assert status() == 0
