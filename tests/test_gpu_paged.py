"""The paged cache's kernels against the float64 reference (paged_ref).

Tolerances count what the kernels round.  Scores: a float32 sum of d products,
so |ds| <= (2 d 2^-24 + product) * sum_e |q_e k_e| * scale.  A product of bf16
numbers is exact; of float32 numbers each factor x = hi + lo + rest has
|lo| < 2^-10 |x| (11 bits, cut off) and |rest| <= 2^-11 |lo| (the next 11,
rounded), and lo * lo is left out, so it is off by at most
2 * 2^-21 + 2^-20 = 2^-19.  A softmax weight is then off by at most the factor
exp(2 ds) and a few steps of exp2 (2^-20), and the output by that, and by the
same 2^-19 of each p v, times sum_s p_s |v_s|, plus the float32 sum over n
slots (n 2^-23), plus half a step of the output's type.
"""

import math

import numpy as np
import pytest

import paged_ref as ref
from hga_testlib import to_f64

pytestmark = pytest.mark.gpu

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
PRODUCT = {"bf16": 0.0, "f32": 2.0 ** -19}


class Case:
    """A cache with random contents whose pages lie anywhere in the pool; what
    no sequence uses (rows behind the last slot, spare pages) holds NaN."""

    def __init__(self, dtype="bf16", d=128, Hkv=2, G=4, ps=16, lens=(40,), max_pages=None,
                 paired=False, spare=2, seed=0, q_scale=2.0):
        import torch
        from hierarchical_routed_sparse_hga_b200 import HGA_BF16, HGA_F32, Config, PagedCache
        self.dtype, self.ps, self.lens = dtype, ps, list(lens)
        B = len(lens)
        dev = torch.device("cuda", 0)
        tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.cfg = Config(B, Hkv * G, Hkv, d, 1, 1, HGA_BF16 if dtype == "bf16" else HGA_F32)
        rng = np.random.default_rng(seed)
        need = [-(-n // ps) for n in lens]
        max_pages = max_pages or max(1, max(need))
        n_pages = sum(need) + spare
        order = rng.permutation(n_pages)
        table = np.full((B, max_pages), -1, dtype=np.int32)
        at = 0
        for b in range(B):
            table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        shape = (n_pages, Hkv, ps, d)
        if paired:
            pool = torch.full((n_pages, 2, Hkv, ps, d), math.nan, dtype=tdt, device=dev)
            self.k, self.v = pool[:, 0], pool[:, 1]
        else:
            self.k = torch.full(shape, math.nan, dtype=tdt, device=dev)
            self.v = torch.full(shape, math.nan, dtype=tdt, device=dev)
        self.weight = torch.rand(shape[:3], generator=g, device=dev)
        self.slot_pos = torch.full(shape[:3], -7, dtype=torch.int32, device=dev)
        for b, n in enumerate(lens):
            for h in range(Hkv):
                pg, row, _ = ref.places(table[b], n, ps, n_pages)
                self.k[pg, h, row] = torch.randn((n, d), generator=g, device=dev).to(tdt)
                self.v[pg, h, row] = torch.randn((n, d), generator=g, device=dev).to(tdt)
                self.slot_pos[pg, h, row] = torch.arange(n, dtype=torch.int32, device=dev)
        self.q = (q_scale * torch.randn((B, Hkv * G, d), generator=g, device=dev)).to(tdt)
        self.table = torch.from_numpy(table).to(dev)
        self.n_slots = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.pos = torch.tensor([n - 1 for n in lens], dtype=torch.int64, device=dev)
        self.cache = PagedCache(self.cfg, self.k, self.v, self.table, self.weight, self.slot_pos)
        self.o = torch.full((B, Hkv * G, d), 7.0, dtype=tdt, device=dev)
        self.lse = torch.full((B, Hkv * G), 7.0, device=dev)

    def workspace(self, accumulate=True):
        import torch
        import hierarchical_routed_sparse_hga_b200 as hga
        size = max(hga.hga_paged_decode_workspace_size(self.cfg, self.cache, accumulate),
                   hga.hga_paged_evict_workspace_size(self.cfg, self.cache))
        # contents of a workspace do not matter
        return torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")

    def decode(self, accumulate=False, workspace=None, stream=None):
        import hierarchical_routed_sparse_hga_b200 as hga
        ws = self.workspace(accumulate) if workspace is None else workspace
        hga.hga_paged_decode(self.cfg, self.cache, self.q, self.n_slots, accumulate, self.o,
                             self.lse, ws, stream=stream)

    def host(self):
        return (to_f64(self.k), to_f64(self.v), self.weight.cpu().numpy().copy(),
                self.slot_pos.cpu().numpy().copy(), self.table.cpu().numpy())

    def check_decode(self, before=None, skip=()):
        """o and lse against the reference; with `before` (the weights before an
        accumulating call) every weight of the pool too."""
        k, v, weight, _, table = self.host()
        n = [0 if b in skip else int(x) for b, x in enumerate(self.n_slots.cpu())]
        o, lse, w, reach, spread = ref.decode(to_f64(self.q), k, v, table, n, self.cfg.head_dim ** -0.5)
        got_o, got_lse = to_f64(self.o), self.lse.double().cpu().numpy()
        G = self.cfg.n_q_heads // self.cfg.n_kv_heads
        ds = (2 * self.cfg.head_dim * 2.0 ** -24 + PRODUCT[self.dtype]) * reach      # [B, Hq]
        longest = max(n) if n else 0
        for b in range(self.cfg.batch):
            if b in skip:
                assert (got_o[b] == 7.0).all() and (got_lse[b] == 7.0).all()
                continue
            if n[b] == 0:
                assert (got_o[b] == 0.0).all() and (got_lse[b] == -math.inf).all()
                continue
            live = lse[b] > -math.inf
            assert ((got_lse[b] > -math.inf) == live).all()
            tol = HALF_STEP[self.dtype] * np.abs(o[b]) + \
                (2 * ds[b][:, None] + 2.0 ** -15 * (self.dtype == "bf16") + 2.0 ** -20
                 + PRODUCT[self.dtype] + n[b] * 2.0 ** -23) * spread[b]
            assert (np.abs(got_o[b] - o[b]) <= tol).all(), (b, np.abs(got_o[b] - o[b]).max())
            tol = ds[b] + 2.0 ** -20 * (1 + np.abs(lse[b])) + n[b] * 2.0 ** -23
            assert (np.abs(got_lse[b] - lse[b])[live] <= tol[live]).all(), b
        if before is not None:
            want, tol = before.astype(np.float64), np.zeros(before.shape)
            for (b, h), (pg, row, p) in w.items():
                np.add.at(want, (pg, h, row), p)
                e = 2 * ds[b, h * G:(h + 1) * G].max() + 2.0 ** -19 + longest * 2.0 ** -23
                np.add.at(tol, (pg, h, row), e * p)
            tol += 2.0 ** -23 * np.abs(want)
            tol[want == before] = 0.0           # slots of no sequence are untouched
            assert (np.abs(weight - want) <= tol).all(), np.abs(weight - want).max()


def status():
    from hierarchical_routed_sparse_hga_b200 import hga_get_device_status
    return hga_get_device_status()


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------

DECODE = [
    # one slot; the ends of a 16-slot step, of a page, of a 64-slot unit; idle rows
    dict(lens=(1,)), dict(lens=(2, 0, 15, 16, 17)), dict(lens=(63, 64, 65, 127, 128, 129), ps=64),
    dict(lens=(0, 0)), dict(lens=(33, 7, 250), ps=256), dict(lens=(31, 32, 33), ps=32, paired=True),
    # every number of query heads a KV head
    *[dict(lens=(77, 5), G=g, Hkv=3, seed=g) for g in range(1, 9)],
    # d = 64 (two 16-slot steps a tile), float32, K and V side by side
    dict(lens=(1, 16, 17, 47, 48, 49, 1000), d=64), dict(lens=(300, 299), d=64, ps=128, paired=True),
    dict(lens=(1, 7, 8, 9, 100), dtype="f32"), dict(lens=(515, 0, 64), dtype="f32", ps=32, G=8),
    dict(lens=(15, 16, 17, 701), dtype="f32", d=64, G=1, Hkv=5),
    dict(lens=(90, 1025), dtype="f32", d=64, G=3, paired=True, ps=128),
    # long: split over the length and joined; ragged against short ones
    dict(lens=(20001,), Hkv=1, ps=64), dict(lens=(9000, 1, 0, 4097, 333), G=2, ps=16),
    dict(lens=(6007, 6007), dtype="f32", G=5, ps=16), dict(lens=(12345, 80), d=64, G=8, ps=32),
    # more heads than the GPU holds blocks
    dict(lens=tuple(range(1, 81)), Hkv=8, G=1, d=64, ps=16),
    # a table far wider than what is in use
    dict(lens=(50, 3), max_pages=4096, ps=16),
]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kw", DECODE, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items())[:60])
def test_decode(kw, accumulate):
    c = Case(**kw)
    before = c.host()[2]
    c.decode(accumulate)
    c.check_decode(before if accumulate else None)
    if not accumulate:
        assert (c.host()[2] == before).all()
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_peaked_and_flat_scores(dtype):
    # scores over a wide range (the running maximum moves late and far), and
    # all equal ones (every weight 1/n)
    c = Case(dtype, lens=(3000, 700), ps=32, q_scale=40.0)
    n = c.lens[0]
    pg, row, _ = ref.places(c.table[0].cpu().numpy(), n, c.ps, c.k.shape[0])
    ramp = c.k.new_tensor(np.linspace(-1, 1, n))[:, None]
    c.k[pg, 0, row] = (ramp * c.q[0, 0][None]).to(c.k.dtype)
    pg, row, _ = ref.places(c.table[1].cpu().numpy(), c.lens[1], c.ps, c.k.shape[0])
    c.k[pg, 1, row] = 0.0
    before = c.host()[2]
    c.decode(True)
    c.check_decode(before)


@pytest.mark.parametrize("dtype,low", [("f32", -3.0e38), ("bf16", -3.0e38)])
def test_decode_slots_that_score_minus_infinity(dtype, low):
    # a key of the type's lowest value against a query of 8: the score
    # overflows to -inf and its weight is 0; a head whose every score is
    # -inf has nothing to attend to (o = 0, lse = -inf)
    c = Case(dtype, lens=(70, 40), G=2)
    c.q[:] = 8.0
    for b, slots in ((0, range(0, 70, 3)), (1, range(40))):
        pg, row, _ = ref.places(c.table[b].cpu().numpy(), c.lens[b], c.ps, c.k.shape[0])
        s = list(slots)
        c.k[pg[s], 0, row[s]] = low
    c.decode(True)
    assert status() == 0
    got_o, got_lse = to_f64(c.o), c.lse.cpu().numpy()
    assert (got_o[1, :2] == 0).all() and (got_lse[1, :2] == -math.inf).all()
    # the other slots' softmax: the reference without those slots
    k, v, _, _, table = c.host()
    pg, row, _ = ref.places(table[0], 70, c.ps, k.shape[0])
    left = [s for s in range(70) if s % 3]
    sc = (k[pg, 0, row][left] @ np.full(128, 8.0)) / math.sqrt(128)
    p = np.exp(sc - sc.max())
    want = (p / p.sum()) @ v[pg, 0, row][left]
    ds = (256 * 2.0 ** -24 + PRODUCT[dtype]) * (np.abs(k[pg, 0, row][left]).sum(1).max() * 8 / math.sqrt(128))
    spread = (p / p.sum()) @ np.abs(v[pg, 0, row][left])
    tol = HALF_STEP[dtype] * np.abs(want) + (2 * ds + 2.0 ** -14) * spread
    for g in range(2):
        assert (np.abs(got_o[0, g] - want) <= tol).all()


def test_decode_pages_outside_the_pool_are_left_out():
    from hierarchical_routed_sparse_hga_b200 import HGA_ERR_DEVICE_CHECK
    c = Case(lens=(200, 100, 40), ps=16)
    c.table[0, 3] = -1
    c.table[0, 12] = c.k.shape[0]
    c.table[2, :] = 1 << 30
    before = c.host()[2]
    c.decode(True)
    assert status() == HGA_ERR_DEVICE_CHECK and status() == 0
    k, v, weight, _, table = c.host()
    assert (to_f64(c.o)[2] == 0).all() and (c.lse[2].cpu().numpy() == -math.inf).all()
    # the reference leaves the same slots out
    c.n_slots[2] = 0
    c.check_decode(before)


@pytest.mark.parametrize("count", [-1, 65, 1 << 30, -(1 << 31)])
def test_decode_counts_out_of_range(count):
    from hierarchical_routed_sparse_hga_b200 import HGA_ERR_DEVICE_CHECK
    c = Case(lens=(64, 50), ps=16)
    c.n_slots[0] = count
    before = c.host()[2]
    c.decode(True)
    assert status() == HGA_ERR_DEVICE_CHECK and status() == 0
    c.check_decode(before, skip=(0,))


def test_decode_is_deterministic_and_leaves_nothing_behind():
    c = Case(lens=(5000, 17, 900), ps=64, Hkv=4)
    ws = c.workspace()
    c.decode(False, ws)
    o, lse = c.o.clone(), c.lse.clone()
    c.weight.zero_()
    c.decode(True, ws)
    w = c.weight.clone()
    assert bool((c.o == o).all()) and bool((c.lse == lse).all())
    c.weight.zero_()
    c.decode(True, ws)
    assert bool((c.weight == w).all()) and bool((c.o == o).all())


def test_decode_sequences_that_share_pages():
    # a common prefix: both sequences read its pages, and its weights receive both shares
    c = Case(lens=(100, 90), ps=16)
    c.table[1, :4] = c.table[0, :4]
    before = c.host()[2]
    c.decode(True)
    c.check_decode(before)


def test_decode_a_page_that_stands_twice_in_the_table():
    # its slots count twice, and their weights receive both shares
    c = Case(lens=(100,), ps=16)
    c.table[0, 5] = c.table[0, 1]
    before = c.host()[2]
    c.decode(True)
    c.check_decode(before)


def test_decode_captured_and_replayed_as_the_cache_grows():
    import torch
    c = Case(lens=(300, 2, 0, 64), ps=16)
    ws = c.workspace()
    for x in (c.k, c.v):
        x.nan_to_num_(0.25)
    c.decode(True, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.decode(True, ws)
    for n in ((300, 2, 0, 64), (17, 2, 1, 63), (0, 0, 0, 0), (299, 1, 0, 64)):
        c.n_slots.copy_(torch.tensor(n, dtype=torch.int32))
        if n[2]:
            c.table[2, 0] = 0
        before = c.host()[2]
        g.replay()
        torch.cuda.synchronize()
        c.check_decode(before)


def test_two_captured_graphs_share_a_workspace():
    import torch
    a, b = Case(lens=(700, 33), ps=16, seed=1), Case(lens=(40, 1200), ps=16, seed=2)
    ws = b.workspace() if b.workspace().numel() > a.workspace().numel() else a.workspace()
    graphs = []
    for c in (a, b):
        c.decode(True, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.decode(True, ws)
        graphs.append(g)
    ba, bb = a.host()[2], b.host()[2]
    for g in (graphs[0], graphs[1], graphs[0]):
        g.replay()
    torch.cuda.synchronize()
    a.weight.copy_(torch.from_numpy(ba))    # a's second replay: from the same weights
    graphs[0].replay()
    a.check_decode(ba)
    b.check_decode(bb)


def test_two_streams_with_their_own_workspaces():
    import torch
    cases = [Case(lens=(4000, 100), ps=64, seed=3), Case("f32", lens=(3000,), ps=16, seed=4)]
    streams = [torch.cuda.Stream() for _ in cases]
    before = [c.host()[2] for c in cases]
    spaces = [c.workspace() for c in cases]
    torch.cuda.synchronize()
    for c, s, ws in zip(cases, streams, spaces):
        c.decode(True, ws, s)
    torch.cuda.synchronize()
    for c, x in zip(cases, before):
        c.check_decode(x)


def test_offsets_past_32_bits():
    # pages more than 2^31 elements into the pool (bf16, 8 GB of pool of which
    # only the used pages are written)
    import torch
    import hierarchical_routed_sparse_hga_b200 as hga
    c = Case(lens=(40, 23), ps=16, spare=0)
    stride, n_pages = 1 << 26, c.k.shape[0]
    n_wide = 33
    pool = torch.empty(n_wide * stride, dtype=torch.bfloat16, device="cuda")
    shape, strides = (n_wide, 2, 16, 128), (stride, 16 * 128, 128, 1)
    k, v = pool.as_strided(shape, strides), pool.as_strided(shape, strides, 1 << 20)
    at = torch.arange(n_pages) + n_wide - n_pages      # the last pages
    k[at], v[at] = c.k, c.v
    weight = torch.zeros(shape[:3], device="cuda")
    slot_pos = torch.zeros(shape[:3], dtype=torch.int32, device="cuda")
    weight[at], slot_pos[at] = c.weight, c.slot_pos
    c.table = torch.where(c.table < 0, c.table, c.table + n_wide - n_pages)
    c.k, c.v, c.weight, c.slot_pos = k, v, weight, slot_pos
    c.cache = hga.PagedCache(c.cfg, k, v, c.table, weight, slot_pos)
    before = weight.cpu().numpy().copy()

    def small():        # the used pages on the host (nothing else was written)
        return k[at].clone(), v[at].clone()

    kk, vv = small()
    c.decode(True)
    c.k, c.v = torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(
        shape, dtype=torch.bfloat16, device="cuda")
    c.k[at], c.v[at] = kk, vv
    c.check_decode(before)
    # eviction moves rows of those pages
    kh, vh, wh, ph, table = c.host()
    moved = ref.evict(kh, vh, wh, ph, table, c.lens, [39, 22], 20, 2, 4)
    assert all(m for m, _ in moved.values())
    hga.hga_paged_evict(c.cfg, c.cache, c.n_slots, c.pos, 20, 2, 4, c.workspace())
    assert (to_f64(k[at]) == kh[at.numpy()])[~np.isnan(kh[at.numpy()])].all()
    assert (to_f64(v[at]) == vh[at.numpy()])[~np.isnan(vh[at.numpy()])].all()
    # the last token again, from new projections
    kv = torch.randn((2, 2, 1, 2, 128), device="cuda").to(torch.bfloat16)
    hga.hga_paged_append(c.cfg, c.cache, None, kv[0], kv[1], 0, 256, 1, None, c.n_slots, c.pos, 0.0,
                         None)
    for b, n in enumerate(c.lens):
        pg, row = int(c.table[b, (n - 1) // 16]), (n - 1) % 16
        assert torch.equal(k[pg, :, row], kv[0, b, 0]) and torch.equal(v[pg, :, row], kv[1, b, 0])
    assert status() == 0


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def run_append(c, s_new, n_new, base, with_q=True, fused=True, last=None, seed=5):
    """Appends to the case's cache; returns the projections and q_out."""
    import torch
    import hierarchical_routed_sparse_hga_b200 as hga
    cfg, d = c.cfg, c.cfg.head_dim
    B, Hq, Hkv = cfg.batch, cfg.n_q_heads, cfg.n_kv_heads
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    width = (Hq + 2 * Hkv) * d
    qkv = torch.randn((B, s_new, width), generator=g, device="cuda").to(c.k.dtype)
    qp, kp, vp = qkv.split([Hq * d, Hkv * d, Hkv * d], -1)
    if last is not None:
        c.pos.copy_(torch.tensor(last))
    q_out = torch.full((B, Hq, s_new, d), 7.0, dtype=c.k.dtype, device="cuda")
    nn = None if n_new is None else torch.tensor(n_new, dtype=torch.int32, device="cuda")
    elt = qkv.element_size()
    if fused:
        at = qkv.data_ptr()
        args = (at if with_q else None, at + Hq * d * elt, at + (Hq + Hkv) * d * elt, width, width)
    else:
        parts = [x.contiguous() for x in (qp, kp, vp)]
        args = (parts[0] if with_q else None, parts[1], parts[2], Hq * d, Hkv * d)
    hga.hga_paged_append(cfg, c.cache, *args, s_new, nn, c.n_slots, c.pos, base,
                         q_out if with_q else None)
    torch.cuda.synchronize()
    return to_f64(qp.unflatten(-1, (Hq, d))), to_f64(kp.unflatten(-1, (Hkv, d))), \
        to_f64(vp.unflatten(-1, (Hkv, d))), q_out


def check_append(c, before, got, s_new, n_new, base, with_q=True, untouched=(), no_page=()):
    """Everything the call wrote, and that nothing else changed.  Bound: half a
    step of the type, and for the rotation 16 * 2^-24 of the pair's size (the
    angle's float32 rounding after its reduction, the sine, the products)."""
    qp, kp, vp, q_out = got
    k0, v0, w0, p0, table = before
    k1, v1, w1, p1, _ = c.host()
    half = c.cfg.head_dim // 2
    want_k, want_v, want_w, want_p = k0.copy(), v0.copy(), w0.copy(), p0.copy()
    tol_k = np.zeros_like(k0)
    want_q = np.full(q_out.shape, 7.0)
    tol_q = np.zeros(q_out.shape)

    def bound(x, y):
        size = np.abs(x[..., :half]) + np.abs(x[..., half:])
        return HALF_STEP[c.dtype] * np.abs(y) + 16 * 2.0 ** -24 * np.concatenate([size, size], -1)

    for b in range(c.cfg.batch):
        if b in untouched:
            continue
        m = s_new if n_new is None else n_new[b]
        for i in range(m):
            p = int(c.pos[b]) - m + 1 + i
            y = ref.rope(qp[b, i], p, base)
            want_q[b, :, i] = y
            tol_q[b, :, i] = bound(qp[b, i], y) if base > 1 else 0
            s = int(c.n_slots[b]) - m + i
            if (b, s // c.ps) in no_page:
                continue
            pg, row = table[b, s // c.ps], s % c.ps
            y = ref.rope(kp[b, i], p, base)
            want_k[pg, :, row] = y
            tol_k[pg, :, row] = bound(kp[b, i], y) if base > 1 else 0
            want_v[pg, :, row] = vp[b, i]
            want_w[pg, :, row], want_p[pg, :, row] = 0.0, p

    def close(x, y, tol):
        return (np.isnan(x) & np.isnan(y)) | (np.abs(x - y) <= tol)

    assert close(k1, want_k, tol_k).all()
    assert close(v1, want_v, 0).all()
    assert (w1 == want_w).all() and (p1 == want_p).all()
    if with_q:
        assert close(to_f64(q_out), want_q, tol_q).all()
    else:
        assert (to_f64(q_out) == 7.0).all()


APPEND = [
    (dict(lens=(1,)), 1, None, 1e6, {}),
    (dict(lens=(17, 300, 16, 64)), 1, (1, 1, 0, 1), 1e6, {}),
    (dict(lens=(40, 33), ps=32, paired=True, G=3), 33, (33, 0), 1e6, {}),
    (dict(lens=(100, 129, 64), ps=64, d=64, G=8, Hkv=1), 100, (100, 1, 64), 1e4, {}),
    (dict(lens=(70, 20), dtype="f32", G=2), 20, (3, 20), 1e6, {}),
    (dict(lens=(70, 20), dtype="f32", d=64, G=1, Hkv=5, ps=256), 9, None, 0.0, {}),
    (dict(lens=(50, 20), G=2), 8, None, 1.0, dict(with_q=False)),
    (dict(lens=(50, 20), G=5), 8, (8, 3), 1e6, dict(fused=False)),
    # positions far behind the slots (a cache that was cut), and the last there are
    (dict(lens=(50, 20)), 4, None, 1e6, dict(last=(131071, 2 ** 31 - 1))),
    (dict(lens=(700,), ps=16, Hkv=8), 700, None, 1e6, {}),
]


@pytest.mark.parametrize("kw,s_new,n_new,base,more", APPEND)
def test_append(kw, s_new, n_new, base, more):
    c = Case(**kw)
    before = c.host()
    got = run_append(c, s_new, n_new, base, **more)
    assert status() == 0
    check_append(c, before, got, s_new, n_new, base, more.get("with_q", True))


def test_append_without_records():
    import torch
    import hierarchical_routed_sparse_hga_b200 as hga
    c = Case(lens=(20, 9))
    before = c.host()
    c.cache = hga.PagedCache(c.cfg, c.k, c.v, c.table)
    w0, p0 = c.weight.clone(), c.slot_pos.clone()
    run_append(c, 5, None, 1e6)
    assert bool((c.weight == w0).all()) and bool((c.slot_pos == p0).all())
    assert not (to_f64(c.k) == before[0]).all()
    # nothing to append
    k1 = c.k.clone()
    run_append(c, 0, None, 1e6)
    assert torch.equal(c.k.nan_to_num(5.0), k1.nan_to_num(5.0))


def test_append_refuses_counts_and_positions_out_of_range():
    from hierarchical_routed_sparse_hga_b200 import HGA_ERR_DEVICE_CHECK
    # more new tokens than rows; than slots; a negative count; a position
    # before 0; one past 2^31; more slots than the table has; the last is right
    c = Case(lens=(40,) * 7, ps=16)
    c.n_slots[1] = 3
    c.n_slots[5] = 49
    before = c.host()
    n_new = (5, 4, -1, 4, 4, 4, 4)
    got = run_append(c, 4, n_new, 1e6, last=(39, 39, 39, 2, 2 ** 31, 39, 39))
    assert status() == HGA_ERR_DEVICE_CHECK and status() == 0
    check_append(c, before, got, 4, n_new, 1e6, untouched=range(6))


def test_append_to_a_page_outside_the_pool():
    from hierarchical_routed_sparse_hga_b200 import HGA_ERR_DEVICE_CHECK
    c = Case(lens=(40, 40), ps=16)
    c.table[0, 1] = c.k.shape[0]
    c.table[1, 2] = -1
    before = c.host()
    got = run_append(c, 30, None, 1e6)
    assert status() == HGA_ERR_DEVICE_CHECK and status() == 0
    check_append(c, before, got, 30, None, 1e6, no_page={(0, 1), (1, 2)})


# ---------------------------------------------------------------------------
# evict
# ---------------------------------------------------------------------------

def check_evict(c, keep, sinks, recent):
    import hierarchical_routed_sparse_hga_b200 as hga
    k, v, w, p, table = c.host()
    ref.evict(k, v, w, p, table, c.n_slots.cpu().numpy(), c.pos.cpu().numpy(), keep, sinks, recent)
    hga.hga_paged_evict(c.cfg, c.cache, c.n_slots, c.pos, keep, sinks, recent, c.workspace())
    k1, v1, w1, p1, _ = c.host()
    np.testing.assert_array_equal(p1, p)
    np.testing.assert_array_equal(w1, w)
    np.testing.assert_array_equal(k1, k)
    np.testing.assert_array_equal(v1, v)


EVICT = [
    # nothing to do; one to drop; everything but one; exactly the page
    (dict(lens=(40, 0, 1)), 40, 0, 0), (dict(lens=(41, 3)), 40, 4, 8), (dict(lens=(300, 2)), 1, 0, 0),
    (dict(lens=(300, 2)), 1, 1, 0), (dict(lens=(300, 2)), 1, 0, 1),
    (dict(lens=(64, 65, 63, 0, 128), ps=64), 64, 4, 16),
    (dict(lens=(1000, 513, 512), ps=16, paired=True), 512, 4, 100),
    (dict(lens=(1000, 77), dtype="f32", d=64, Hkv=5, G=1, ps=128), 70, 0, 70),
    (dict(lens=(257, 600), dtype="f32", ps=32), 256, 128, 128),
    (dict(lens=(500, 90), d=64, G=2, paired=True), 80, 4, 16),
    (dict(lens=(20000, 9000), Hkv=1, d=64, ps=64), 8192, 4, 64),
    (dict(lens=(5000,) * 3, d=64, ps=16, paired=True), 4990, 4, 64),
    (dict(lens=(70000,), Hkv=1, d=64, ps=256), 33333, 10, 1000),
]


@pytest.mark.parametrize("kw,keep,sinks,recent", EVICT)
def test_evict(kw, keep, sinks, recent):
    c = Case(**kw)
    check_evict(c, keep, sinks, recent)
    assert status() == 0


@pytest.mark.parametrize("n,keep", [(200, 64), (3000, 1000), (9001, 9000)])
def test_evict_ties_zeros_and_values_that_are_no_numbers(n, keep):
    # few different weights (ties go to the lower slot), both zeros (equal),
    # infinities, NaN (below everything), denormals
    import torch
    c = Case(lens=(n, n), ps=16, seed=8)
    pool = torch.tensor([0.0, -0.0, 1.0, 1.0, -1.0, math.inf, -math.inf, math.nan, 1e-40, 2e-40],
                        device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    c.weight.copy_(pool[torch.randint(0, 10, c.weight.shape, generator=g, device="cuda")])
    c.weight[:, 1] = 0.5                 # one head: all equal
    check_evict(c, keep, 4, 32)


@pytest.mark.parametrize("levels", [0, 50])
def test_evict_a_head_longer_than_the_blocks_hold(levels):
    # more slots a block than its shared memory holds keys, and than one round
    # of ranks covers; with 50 different weights the edge is a long tie
    c = Case(lens=(540001,), Hkv=1, G=1, d=64, ps=256, spare=0)
    if levels:
        c.weight.copy_((c.weight * levels).floor())
    check_evict(c, 270007, 4, 1000)
    assert status() == 0


def test_evict_positions_that_hold_more_than_is_kept():
    # repeated positions hold more slots than `keep`: the lower ones are kept
    c = Case(lens=(500,), ps=16)
    c.slot_pos.fill_(1)
    check_evict(c, 100, 2, 0)
    c = Case(lens=(500,), ps=16)
    c.pos[0] = -50                       # every position is recent
    check_evict(c, 100, 0, 1)


def test_evict_positions_in_any_order_then_again():
    # two cuts in a row, the second of a cache whose slots are no longer in order
    import torch
    c = Case(lens=(700, 650), ps=16, Hkv=3)
    check_evict(c, 400, 4, 64)
    c.n_slots.clamp_(max=400)
    c.weight.copy_(torch.rand(c.weight.shape, device="cuda"))
    check_evict(c, 200, 4, 64)
    c.n_slots.clamp_(max=200)
    check_evict(c, 200, 4, 64)           # at its length: nothing moves


def test_evict_leaves_bad_sequences_alone():
    from hierarchical_routed_sparse_hga_b200 import HGA_ERR_DEVICE_CHECK
    c = Case(lens=(100, 100, 100, 20), ps=16)
    c.table[0, 6] = c.k.shape[0]
    c.n_slots[1] = 113
    c.table[3, 1] = -5                   # 20 slots, not cut: not looked at
    check_evict_ref = [0, 0, 100, 20]
    import hierarchical_routed_sparse_hga_b200 as hga
    k, v, w, p, table = c.host()
    ref.evict(k, v, w, p, table, check_evict_ref, c.pos.cpu().numpy(), 64, 4, 16)
    hga.hga_paged_evict(c.cfg, c.cache, c.n_slots, c.pos, 64, 4, 16, c.workspace())
    assert status() == HGA_ERR_DEVICE_CHECK and status() == 0
    k1, v1, w1, p1, _ = c.host()
    np.testing.assert_array_equal(p1, p)
    np.testing.assert_array_equal(w1, w)
    np.testing.assert_array_equal(k1, k)
    np.testing.assert_array_equal(v1, v)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_generation_with_a_bounded_cache(dtype):
    """Prompts, then steps of append + decode captured in one graph, the cache
    cut whenever it is over its budget: every step's output against the
    reference on the cache as it stands, an idle row in between."""
    import torch
    from hierarchical_routed_sparse_hga_b200 import HGA_BF16, HGA_F32, Config, HgaPagedLayer
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    B, Hkv, G, d, ps = 3, 2, 4, 128, 16
    cfg = Config(B, Hkv * G, Hkv, d, 1, 1, HGA_BF16 if dtype == "bf16" else HGA_F32)
    layer = HgaPagedLayer(cfg, 3 * 8, ps, 8)
    layer.table.copy_(torch.randperm(24, device="cuda").view(3, 8).to(torch.int32))
    g = torch.Generator(device="cuda")
    g.manual_seed(9)

    def draw(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(tdt)

    prompt = torch.tensor([70, 0, 33], dtype=torch.int32, device="cuda")
    qkv = draw(B, 70, (Hkv * G + 2 * Hkv) * d)
    split = [Hkv * G * d, Hkv * d, Hkv * d]
    q_out = torch.zeros((B, Hkv * G, 70, d), dtype=tdt, device="cuda")
    layer.advance(prompt)
    layer.append(*qkv.split(split, -1), 1e6, q_out, n_new=prompt)

    qkv = draw(B, 1, (Hkv * G + 2 * Hkv) * d)
    q = torch.zeros((B, Hkv * G, 1, d), dtype=tdt, device="cuda")
    o = torch.zeros((B, Hkv * G, d), dtype=tdt, device="cuda")
    lse = torch.zeros((B, Hkv * G), device="cuda")
    one = torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")

    def step():
        layer.advance(one)
        layer.append(*qkv.split(split, -1), 1e6, q, n_new=one)
        layer.decode(q.view(B, Hkv * G, d), o, lse, accumulate=True)

    c = Case.__new__(Case)
    c.dtype, c.ps, c.cfg = dtype, ps, cfg
    c.k, c.v, c.weight, c.slot_pos = layer.k, layer.v, layer.weight, layer.slot_pos
    c.table, c.n_slots, c.pos = layer.table, layer.n_slots, layer.pos
    c.q, c.o, c.lse, c.cache = q.view(B, Hkv * G, d), o, lse, layer.cache

    step()
    graph = torch.cuda.CUDAGraph()
    state = layer.n_slots.clone(), layer.pos.clone()
    with torch.cuda.graph(graph):
        step()
    layer.n_slots.copy_(state[0]), layer.pos.copy_(state[1])
    for i in range(60):
        qkv.copy_(draw(*qkv.shape))
        graph.replay()
        if i % 7 == 3:
            w0 = c.host()[2]
            # undo this step's share of the weights to check it
            torch.cuda.synchronize()
            c.check_decode()
            assert int(layer.n_slots[1]) == 0
            sums = [sum(w0[pg, h, row].sum() for pg, row in [ref.places(
                layer.table[2].cpu().numpy(), int(layer.n_slots[2]), ps, 24)[:2]])
                for h in range(Hkv)]
            assert all(x > 0 for x in sums)
        if int(layer.n_slots.max()) >= 96:
            k, v, w, p, table = c.host()
            ref.evict(k, v, w, p, table, layer.n_slots.cpu().numpy(), layer.pos.cpu().numpy(),
                      64, 4, 16)
            layer.evict(64, sinks=4, recent=16)
            np.testing.assert_array_equal(c.host()[3], p)
            np.testing.assert_array_equal(c.host()[0], k)
            assert int(layer.n_slots.max()) <= 64
    assert status() == 0
    # positions went on while the cache was cut
    assert layer.pos.tolist() == [70 + 61 - 1, -1, 33 + 61 - 1]
    held = p_held = c.host()[3]
    pg, row, _ = ref.places(layer.table[0].cpu().numpy(), int(layer.n_slots[0]), ps, 24)
    for h in range(Hkv):
        pos = sorted(held[pg, h, row])
        assert len(set(pos)) == len(pos) and pos[:4] == [0, 1, 2, 3]
        assert pos[-1] == 130
    assert p_held is held


def test_queries_of_the_append_feed_the_next_call():
    """Back to back on one stream: the mean queries are read from what the
    append wrote, not from what the buffer held."""
    import torch
    from hierarchical_routed_sparse_hga_b200 import (HGA_BF16, Config, HgaPagedLayer,
                                                     hga_build_query_summaries)
    B, Hkv, G, d, S = 2, 8, 4, 128, 2048
    cfg = Config(B, Hkv * G, Hkv, d, 4, 16, HGA_BF16)
    layer = HgaPagedLayer(cfg, B * S // 64, 64, S // 64)
    layer.advance(S)
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    qsum = torch.zeros((B, Hkv, S // 64, d), device="cuda")
    for _ in range(5):
        qkv = torch.randn((B, S, (Hkv * G + 2 * Hkv) * d), generator=g, device="cuda").to(torch.bfloat16)
        q_out = torch.full((B, Hkv * G, S, d), math.nan, dtype=torch.bfloat16, device="cuda")
        layer.append(*qkv.split([Hkv * G * d, Hkv * d, Hkv * d], -1), 1e6, q_out)
        hga_build_query_summaries(cfg, q_out, 0, S, S, qsum)
        want = q_out.view(B, Hkv, G, S // 64, 64, d).double().mean((2, 4))
        # float32 sums of 256 values of size up to 6
        assert float((qsum.double() - want).abs().max()) <= 256 * 6 * 2.0 ** -23
    # nothing to append is no call
    layer.append(qkv[:, :0, :4096], qkv[:, :0, :1024], qkv[:, :0, :1024], 1e6, q_out)


def test_paged_and_routed_decode_agree_when_everything_is_selected():
    """The routed decode over a contiguous cache whose top-k covers it, and the
    paged decode over the same tokens."""
    import torch
    from hierarchical_routed_sparse_hga_b200 import (HGA_F32, Config, HgaPagedLayer,
                                                     hga_build_summaries, hga_decode)
    B, Hkv, G, d, T = 2, 2, 2, 64, 512
    cfg = Config(B, Hkv * G, Hkv, d, 64, 256, HGA_F32)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    k, v = (torch.randn((B, Hkv, T, d), generator=g, device="cuda") for _ in range(2))
    q = torch.randn((B, Hkv * G, d), generator=g, device="cuda")
    pos = torch.tensor([400, 63], dtype=torch.int64, device="cuda")
    gsum = torch.zeros((B, Hkv, T // 8, d), device="cuda")
    bsum = torch.zeros((B, Hkv, T // 64, d), device="cuda")
    hga_build_summaries(cfg, k, T, 0, T, gsum, bsum)
    o = torch.zeros((2, B, Hkv * G, d), device="cuda")
    lse = torch.zeros((2, B, Hkv * G), device="cuda")
    hga_decode(cfg, q, k, v, T, pos, bsum, gsum, None, None, o[0], lse[0])
    layer = HgaPagedLayer(cfg, B * T // 64, 64, T // 64)
    layer.advance((pos + 1).to(torch.int32))
    rows = [x.transpose(1, 2).contiguous()[:, :401] for x in (k, v)]
    n_new = (pos + 1).to(torch.int32)
    layer.append(None, rows[0].contiguous(), rows[1].contiguous(), 0.0, None, n_new=n_new)
    layer.decode(q, o[1], lse[1])
    # both are float32 sums of the same terms, each within 1e-4 of the formula
    assert float((o[0] - o[1]).abs().max()) <= 2e-4
    assert float((lse[0] - lse[1]).abs().max()) <= 2e-4
    assert status() == 0


def test_binding_refuses_other_devices_types_and_sizes():
    import torch
    import hierarchical_routed_sparse_hga_b200 as hga
    c = Case(lens=(20, 9))
    ws = c.workspace()
    ok = [c.cfg, c.cache, c.q, c.n_slots, False, c.o, c.lse, ws]
    for i, bad in ((2, c.q.float()), (2, c.q[:1]), (2, c.q.transpose(1, 2)), (3, c.n_slots.long()),
                   (3, c.n_slots[:1]), (3, c.n_slots.cpu()), (5, c.o.float()), (6, c.lse.double()),
                   (6, c.lse[:1])):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            hga.hga_paged_decode(*args)
    with pytest.raises(ValueError):
        hga.hga_paged_evict(c.cfg, c.cache, c.n_slots, c.pos.int(), 8, 0, 0, ws)
    for other in (hga.Config(2, 8, 2, 64, 1, 1), hga.Config(2, 8, 4, 128, 1, 1),
                  hga.Config(2, 8, 2, 128, 1, 1, hga.HGA_F32)):
        with pytest.raises(ValueError):
            hga.hga_paged_decode(other, *ok[1:])
    with pytest.raises(ValueError):
        cfg3 = hga.Config(3, 8, 2, 128, 1, 1)
        hga.hga_paged_evict(cfg3, c.cache, torch.zeros(3, dtype=torch.int32, device="cuda"),
                            torch.zeros(3, dtype=torch.int64, device="cuda"), 8, 0, 0, ws)
    assert (to_f64(c.o) == 7.0).all()
