"""The paged cache on the CPU: its float64 reference against closed forms, and
the host-side refusals of the C calls and of the binding (no GPU needed)."""

import math

import numpy as np
import pytest

import hierarchical_routed_sparse_hga_b200 as hga
import paged_ref as ref
from hierarchical_routed_sparse_hga_b200 import _lib

FAKE = 0x10000  # aligned, never dereferenced: every call below fails its host check


def test_reference_decode_equals_softmax_over_the_gathered_rows():
    rng = np.random.default_rng(0)
    B, Hkv, G, d, ps, n_pages = 3, 2, 2, 8, 4, 9
    k, v = rng.normal(size=(2, n_pages, Hkv, ps, d))
    table = np.array([[4, 0, 7], [8, 2, -1], [1, 3, 5]])
    n = [11, 0, 1]
    q = rng.normal(size=(B, Hkv * G, d))
    o, lse, w, _, _ = ref.decode(q, k, v, table, n, 0.5)
    for b in range(B):
        for h in range(Hkv):
            kk = k[table[b]].transpose(1, 0, 2, 3).reshape(Hkv, -1, d)[h, :n[b]]
            vv = v[table[b]].transpose(1, 0, 2, 3).reshape(Hkv, -1, d)[h, :n[b]]
            for g in (2 * h, 2 * h + 1):
                if n[b] == 0:
                    assert (o[b, g] == 0).all() and lse[b, g] == -math.inf
                    continue
                e = np.exp(0.5 * kk @ q[b, g])
                np.testing.assert_allclose(o[b, g], e @ vv / e.sum(), rtol=1e-12)
                np.testing.assert_allclose(lse[b, g], math.log(e.sum()), rtol=1e-12)
            assert abs(w[b, h][2].sum() - (G if n[b] else 0)) < 1e-12


def test_reference_rope_is_a_complex_rotation():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(5, 16))
    y = ref.rope(x, 12345, 1e6)
    z = (x[:, :8] + 1j * x[:, 8:]) * np.exp(1j * 12345 * 1e6 ** (-np.arange(8) / 8))
    np.testing.assert_allclose(y, np.concatenate([z.real, z.imag], -1), rtol=1e-10, atol=1e-10)
    assert (ref.rope(x, 77, 0.0) == x).all()


def test_reference_evict_by_hand():
    # 6 slots in pages of 2, keep 3: slot 0 is a sink, slot 5 recent, and of
    # the weights [., 5, 1, 7, 7, .] one more is kept: slot 3 (tie: lower)
    k = np.arange(3 * 1 * 2 * 1, dtype=float).reshape(3, 1, 2, 1)
    v = -k
    table = np.array([[2, 0, 1]])   # slot s -> k value [4, 5, 0, 1, 2, 3][s]
    w = np.zeros((3, 1, 2))
    p = np.zeros((3, 1, 2), dtype=int)
    for s, (ws, ps_) in enumerate(zip([0, 5, 1, 7, 7, 0], [0, 3, 4, 8, 9, 11])):
        w[table[0][s // 2], 0, s % 2], p[table[0][s // 2], 0, s % 2] = ws, ps_
    moved = ref.evict(k, v, w, p, table, [6], [11], 3, 1, 1)
    assert moved == {(0, 0): ([3, 5], [1, 2])}
    got = k[table[0]].reshape(-1)
    assert got.tolist() == [4, 1, 3, 1, 2, 3]
    assert p[table[0]].reshape(-1)[:3].tolist() == [0, 8, 11]


def cfg(**kw):
    base = dict(batch=2, n_q_heads=32, n_kv_heads=8, head_dim=128, topk_blocks=16,
                topk_groups=64)
    base.update(kw)
    return hga.Config(**base)


def pages(**kw):
    base = dict(k=FAKE, v=FAKE, table=FAKE, n_pages=100, page_stride=8 * 64 * 128, page_size=64,
                max_pages=10, weight=FAKE, slot_pos=FAKE)
    base.update(kw)
    return hga.PagedCache.raw(**base)


def status_of(fn, *args):
    with pytest.raises(hga.HgaError) as e:
        fn(*args)
    return e.value.status


def decode(c, p, q=FAKE, n=FAKE, acc=0, o=FAKE << 8, lse=FAKE, ws=FAKE, size=1 << 40):
    return status_of(hga.hga_paged_decode, c, p, q, n, acc, o, lse, ws, size, 0)


def append(c, p, q=FAKE, k=FAKE, v=FAKE, qs=32 * 128, kvs=8 * 128, s_new=1, n_new=FAKE, n=FAKE,
           pos=FAKE, base=1e6, q_out=FAKE << 8):
    return status_of(hga.hga_paged_append, c, p, q, k, v, qs, kvs, s_new, n_new, n, pos, base,
                     q_out, 0)


def evict(c, p, n=FAKE, pos=FAKE, keep=64, sinks=4, recent=16, ws=FAKE, size=1 << 40):
    return status_of(hga.hga_paged_evict, c, p, n, pos, keep, sinks, recent, ws, size, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(k=0), 1), (dict(v=0), 1), (dict(table=0), 1), (dict(k=FAKE + 8), 1),
    (dict(slot_pos=FAKE + 4), 1), (dict(page_size=8), 2), (dict(page_size=48), 2),
    (dict(page_size=512), 2), (dict(n_pages=0), 1), (dict(max_pages=0), 1),
    (dict(max_pages=1 << 25), 2), (dict(n_pages=1 << 31), 2),
    (dict(page_stride=8 * 64 * 128 - 8), 1), (dict(page_stride=8 * 64 * 128 + 4), 1),
    (dict(page_stride=1 << 41), 1),
])
def test_every_call_checks_the_cache(kw, status):
    c, p = cfg(), pages(**kw)
    assert decode(c, p) == status
    assert append(c, p) == status
    assert evict(c, p) == status
    assert hga.hga_paged_decode_workspace_size(c, p, True) == 0
    assert hga.hga_paged_evict_workspace_size(c, p) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 1), (dict(n_q_heads=33), 1), (dict(n_q_heads=72), 2), (dict(head_dim=96), 2),
    (dict(dtype=7), 2), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(batch=65536), 2),
])
def test_every_call_checks_the_config(kw, status):
    c, p = cfg(**kw), pages()
    assert decode(c, p) == status
    assert append(c, p) == status
    assert evict(c, p) == status


def test_decode_refusals():
    c, p = cfg(), pages()
    for kw in (dict(q=0), dict(n=0), dict(o=0), dict(lse=0), dict(ws=0), dict(o=FAKE + 8),
               dict(o=FAKE), dict(o=FAKE + 2 * 32 * 128 * 2 - 16), dict(acc=2)):
        assert decode(c, p, **kw) == 1, kw
    assert decode(c, pages(weight=None), acc=1) == 1
    for acc in (0, 1):
        need = hga.hga_paged_decode_workspace_size(c, p, acc)
        assert need > 0
        assert decode(c, p, acc=acc, size=need - 1) == 6


def test_decode_refuses_tables_whose_units_pass_32_bits():
    c, p = cfg(batch=1024), pages(max_pages=1 << 20)
    assert hga.hga_paged_decode_workspace_size(c, p, False) == 0
    assert decode(c, p) == 2


def test_append_refusals():
    c, p = cfg(), pages()
    for kw in (dict(k=0), dict(v=0), dict(n=0), dict(pos=0), dict(q=0), dict(q_out=0),
               dict(q=FAKE + 2), dict(q_out=FAKE), dict(s_new=-1), dict(base=-1.0), dict(base=float("nan")),
               dict(qs=32 * 128 - 8), dict(kvs=8 * 128 - 8), dict(qs=32 * 128 + 4),
               dict(kvs=8 * 128 + 4), dict(kvs=1 << 33)):
        assert append(c, p, **kw) == 1, kw


def test_evict_refusals():
    c, p = cfg(), pages()
    for kw in (dict(n=0), dict(pos=0), dict(ws=0), dict(keep=0), dict(sinks=-1), dict(recent=-1),
               dict(keep=19), dict(sinks=1 << 30, recent=(1 << 31) - 1, keep=1 << 30)):
        assert evict(c, p, **kw) == 1, kw
    assert evict(c, pages(weight=None)) == 1
    assert evict(c, pages(slot_pos=None)) == 1
    need = hga.hga_paged_evict_workspace_size(c, p)
    assert need > 0
    assert evict(c, p, size=need - 1) == 6


def test_topk_counts_are_not_used():
    # a config for routing with its counts left at 0 still describes a cache
    c = cfg(topk_blocks=0, topk_groups=0)
    assert hga.hga_paged_decode_workspace_size(c, pages(), True) > 0


def test_binding_checks_before_the_call():
    import torch
    c = cfg()
    k = torch.zeros((4, 8, 64, 128), dtype=torch.bfloat16)
    table = torch.zeros((2, 2), dtype=torch.int32)
    for kw, text in ((dict(k=k.float()), "must be"), (dict(k=k[:, :4]), "heads"),
                     (dict(k=k.transpose(2, 3).contiguous().transpose(2, 3)), "contiguous"),
                     (dict(v=k[:2]), "must be"), (dict(table=table.long()), "int32"),
                     (dict(table=table[:1]), "int32"), (dict(weight=torch.zeros(4, 8, 32)), "must"),
                     (dict(v=torch.zeros((4, 2, 8, 64, 128), dtype=torch.bfloat16)[:, 0]),
                      "stride"),
                     (dict(), "one CUDA device")):
        args = dict(k=k, v=k, table=table)
        args.update(kw)
        with pytest.raises(ValueError, match=text):
            hga.PagedCache(c, **args)
    with pytest.raises(ValueError, match="device tensors"):
        hga.hga_paged_decode(c, pages(), k, FAKE, 0, FAKE, FAKE, FAKE, 1, 0)


def test_layer_finds_the_row_stride():
    import torch
    from hierarchical_routed_sparse_hga_b200.runtime import HgaPagedLayer
    rows = HgaPagedLayer._rows
    qkv = torch.zeros((3, 5, 10 * 16))
    assert rows(qkv[..., :96], 6, 16, "q") == 160
    assert rows(qkv[..., :96].unflatten(-1, (6, 16)), 6, 16, "q") == 160
    assert rows(qkv[:, :1, :96].contiguous(), 6, 16, "q") == 96
    for bad in (qkv[:, :3, :96], qkv[..., :192:2][..., :80], qkv[..., :95],
                qkv.transpose(0, 1)[..., :96]):
        with pytest.raises(ValueError):
            rows(bad, 6 if bad.shape[-1] != 80 else 5, 16, "q")


def test_kernel_names():
    assert [hga.hga_kernel_name(i) for i in range(16, 21)] == [
        "paged_append", "paged_decode", "paged_join", "paged_evict",
        "paged_move"]
    assert _lib.HGA_K_COUNT == 21
