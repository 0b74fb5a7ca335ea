"""The paged cache's calls in a stream with others: what comes next reads what they wrote."""

import pytest

from test_gpu_paged import Case, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_begin,s_len", [(16384, 2048), (65536, 2048), (4096, 64)])
def test_routing_right_behind_an_append_reads_the_new_queries(q_begin, s_len, dtype):
    """The routing reads Q before it waits for the kernel in front of it: up to
    512 candidate blocks in one launch, else in the first of three.  Few new
    tokens in some sequences, so that warps of one block end far apart.  The
    selections equal those of a routing that begins when all is done."""
    import torch
    from hierarchical_routed_sparse_hga_b200 import (HGA_BF16, HGA_F32, Config, HgaPagedLayer,
                                                     hga_route, hga_route_workspace_size)
    B, Hkv, G, d = 4, 2, 4, 128
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    cfg = Config(B, Hkv * G, Hkv, d, 4, 16, HGA_BF16 if dtype == "bf16" else HGA_F32)
    ctx, n_qb = q_begin + s_len, s_len // 64
    layer = HgaPagedLayer(cfg, B * max(1, s_len // 64), 64, max(1, s_len // 64))
    g = torch.Generator(device="cuda")
    g.manual_seed(21)
    bsum = torch.randn((B, Hkv, ctx // 64, d), generator=g, device="cuda")
    gsum = torch.randn((B, Hkv, ctx // 8, d), generator=g, device="cuda")
    ws = torch.empty(max(16, hga_route_workspace_size(cfg, s_len, q_begin)), dtype=torch.uint8,
                     device="cuda")
    sel = [(torch.empty((B, Hkv, n_qb, 4), dtype=torch.int32, device="cuda"),
            torch.empty((B, Hkv, n_qb, 16), dtype=torch.int32, device="cuda")) for _ in range(2)]
    n_new = torch.tensor([s_len, 1, s_len * 3 // 5 + 1, 2], dtype=torch.int32, device="cuda")
    layer.advance(n_new)
    q_out = torch.empty((B, Hkv * G, s_len, d), dtype=tdt, device="cuda")
    other = (30 * torch.randn(q_out.shape, generator=g, device="cuda")).to(tdt)
    for _ in range(8):
        qkv = torch.randn((B, s_len, (Hkv * G + 2 * Hkv) * d), generator=g, device="cuda").to(tdt)
        parts = qkv.split([Hkv * G * d, Hkv * d, Hkv * d], -1)
        q_out.copy_(other)
        layer.append(*parts, 1e6, q_out, n_new=n_new)
        hga_route(cfg, q_out, q_begin, s_len, ctx, bsum, gsum, *sel[0], ws)
        torch.cuda.synchronize()
        hga_route(cfg, q_out, q_begin, s_len, ctx, bsum, gsum, *sel[1], ws)
        assert torch.equal(sel[0][0], sel[1][0]) and torch.equal(sel[0][1], sel[1][1])
    assert status() == 0


@pytest.mark.parametrize("as_int", [False, True])
def test_a_layer_on_its_own_stream(as_int):
    """Steps with stream=s while the current stream is busy: every call of the
    step, the counts' too, runs on s and waits for nothing else."""
    import numpy as np
    import torch
    from hierarchical_routed_sparse_hga_b200 import HGA_BF16, Config, HgaPagedLayer
    B, Hkv, G, d, ps = 2, 2, 2, 64, 16
    cfg = Config(B, Hkv * G, Hkv, d, 1, 1, HGA_BF16)
    layer = HgaPagedLayer(cfg, B * 8, ps, 8)
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    qkv = torch.randn((B, 100, (Hkv * G + 2 * Hkv) * d), generator=g, device="cuda").to(torch.bfloat16)
    step = torch.randn((B, 1, (Hkv * G + 2 * Hkv) * d), generator=g, device="cuda").to(torch.bfloat16)
    split = [Hkv * G * d, Hkv * d, Hkv * d]
    n_new = torch.tensor([100, 60], dtype=torch.int32, device="cuda")
    q_all = torch.zeros((B, Hkv * G, 100, d), dtype=torch.bfloat16, device="cuda")
    c = Case.__new__(Case)
    c.dtype, c.ps, c.cfg = "bf16", ps, cfg
    c.k, c.v, c.weight, c.slot_pos = layer.k, layer.v, layer.weight, layer.slot_pos
    c.table, c.n_slots, c.pos = layer.table, layer.n_slots, layer.pos
    q = torch.zeros((B, Hkv * G, 1, d), dtype=torch.bfloat16, device="cuda")
    c.q, c.cache = q.view(B, Hkv * G, d), layer.cache
    c.o = torch.full((B, Hkv * G, d), 7.0, dtype=torch.bfloat16, device="cuda")
    c.lse = torch.full((B, Hkv * G), 7.0, device="cuda")
    side = torch.cuda.Stream()
    s = side.cuda_stream if as_int else side

    def keep_busy(yes):
        torch.cuda.synchronize()
        if yes:
            torch.cuda._sleep(1 << 30)          # about half a second
        done = torch.cuda.Event()
        done.record()
        return done

    for yes in (False, True):                   # first use of a kernel may wait for the device
        layer.n_slots.zero_(), layer.pos.fill_(-1), layer.weight.zero_()
        done = keep_busy(yes)
        layer.advance(n_new, stream=s)
        layer.append(*qkv.split(split, -1), 1e6, q_all, n_new=n_new, stream=s)
        layer.advance(1, stream=s)
        layer.append(*step.split(split, -1), 1e6, q, stream=s)
        layer.decode(c.q, c.o, c.lse, accumulate=True, stream=s)
        with torch.cuda.stream(side):
            assert layer.n_slots.tolist() == [101, 61] and layer.pos.tolist() == [100, 60]
            assert not (yes and done.query())
            c.check_decode(np.zeros(tuple(layer.weight.shape)))
        done = keep_busy(yes)
        layer.evict(80, sinks=4, recent=16, stream=s)
        layer.advance(1, stream=s)
        layer.append(*step.split(split, -1), 1e6, q, stream=s)
        layer.decode(c.q, c.o, c.lse, stream=s)
        with torch.cuda.stream(side):
            assert layer.n_slots.tolist() == [81, 62] and layer.pos.tolist() == [101, 61]
            assert not (yes and done.query())
            c.check_decode()
    torch.cuda.synchronize()
    assert status() == 0
