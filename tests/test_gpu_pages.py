"""GPU tests of a paged cache's pages (kdt_page_assign), rows written to slots (kdt_latent_write_paged) and
compaction (kdt_kv_compact_paged), against the plain oracle (oracle/paged.py, oracle/q8.py).

Pages are whole numbers: equal. Written rows: y in float32 is off by below 2^-20 of itself (21 roundings of the sum of
squares, halved by the root, then a root, a division and two products), k by 8e-7 (|k0| + |k1|) (angle, sine and cosine,
three roundings), then half a bf16 step, 2^-8 of the value. Moved rows: the same bytes.
"""
import numpy as np
import pytest

from oracle import paged as op
from oracle import q8 as oq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kdt():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_tree_absorb_gb300 import build_lib
    build_lib.build()
    import speculative_decoding_tree_absorb_gb300 as k
    return k


def _cu(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _state(rng, B, W, page, n_pages, top):
    """Lengths up to `top` rows, their pages anywhere, stale entries behind them."""
    lens = rng.randint(0, top + 1, B)
    held = (-(-lens // page)).astype(np.int32)
    while held.sum() > n_pages:
        held[np.argmax(held)] = 0
    lens = np.minimum(lens, held * page)
    ids = rng.permutation(n_pages).astype(np.int32)
    table = rng.randint(-5, n_pages + 5, (B, W)).astype(np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    return table, held, np.concatenate([ids[at:], ids[:at]]).astype(np.int32), n_pages - at, lens.astype(np.int32)


def _assign(kdt, state, new_len, page, start=None, T=0, wide=False):
    import torch
    table, held, free, n_free, _ = state
    t = _cu(table)
    if wide:                                # a table that is a part of a larger one
        big = torch.full((table.shape[0], table.shape[1] + 9), 77, dtype=torch.int32, device="cuda")
        big[:, :table.shape[1]] = t
        t = big[:, :table.shape[1]]
    h, f, n, e = _cu(held), _cu(free), _cu(np.array([n_free], dtype=np.int32)), _cu(np.array([9], dtype=np.int32))
    slots = kdt.page_assign(t, h, f, n, _cu(new_len.astype(np.int32)), page, start=None if start is None else _cu(start), T=T,
                            err=e)
    torch.cuda.synchronize()
    if wide:
        assert (big[:, table.shape[1]:] == 77).all()
    return (t.cpu().numpy(), h.cpu().numpy(), f.cpu().numpy(), int(n.item()), None if slots is None else slots.cpu().numpy(),
            int(e.item()))


def _same(got, want):
    for g, w, name in zip(got, want, ("table", "held", "free", "n_free", "slots", "err")):
        assert np.array_equal(g, w) if w is not None else g is None, name


@pytest.mark.parametrize("B,page,T", [(1, 8, 1), (7, 16, 5), (40, 64, 33), (300, 8, 70), (1025, 16, 1), (2100, 256, 40),
                                      (16384, 8, 1), (3, 1024, 4096), (64, 32, 2048)])
def test_pages_and_slots(kdt, B, page, T):
    rng = np.random.RandomState(B + T)
    W = -(-(900 + T) // page) + 1
    n_pages = max(1, B * W * 2 // 3)
    state = _state(rng, B, W, page, n_pages, 900)
    for kind in ("grow", "shrink", "mixed", "nothing", "all back", "too much"):
        lens = state[4]
        new = {"grow": lens + rng.randint(0, T + 1, B), "shrink": rng.randint(0, lens + 1), "mixed": rng.randint(0, 900, B),
               "nothing": lens, "all back": 0 * lens, "too much": np.full(B, W * page)}[kind]
        start = np.maximum(lens - rng.randint(0, 3, B), 0).astype(np.int32)
        want = op.page_assign(state[0], state[1], state[2], state[3], new, page, start, T)
        _same(_assign(kdt, state, new, page, start, T, wide=kind == "mixed"), want)
        if kind in ("grow", "mixed"):       # and on from there, without slots
            state = want[:4] + (np.where(want[1] == -(-new // page), new, 0 * new),)
            back = rng.randint(0, 900, B)
            want = op.page_assign(*state[:4], back, page)
            _same(_assign(kdt, state, back, page), want)


def test_starts_anywhere(kdt):
    """Rows before the first and behind the last have no slot, however far off."""
    start = np.array([-5, 2 ** 31 - 1, -(2 ** 31), 3, 39, -40], dtype=np.int64)
    state = _state(np.random.RandomState(8), 6, 6, 8, 40, 40)
    new = np.array([40, 40, 40, 40, 40, 0])
    for T in (1, 7, 33, 700):
        want = op.page_assign(*state[:4], new, 8, start, T)
        _same(_assign(kdt, state, new, 8, start.astype(np.int32), T), want)


def test_refused_requests(kdt):
    rng = np.random.RandomState(5)
    state = _state(rng, 50, 6, 8, 120, 40)
    new = rng.randint(0, 48, 50)
    new[[3, 17]] = -1, 49                    # a negative length, more than W pages
    state[1][30] = 7                         # more held than a table row has
    state[1][31] = -2
    want = op.page_assign(*state[:4], new, 8, np.zeros(50, dtype=np.int32), 9)
    assert want[5] == 4
    _same(_assign(kdt, state, new, 8, np.zeros(50, dtype=np.int32), 9), want)
    new[[3, 17]] = 2 ** 31 - 1, 0
    want = op.page_assign(*state[:4], new, 8)
    _same(_assign(kdt, state, new, 8), want)


def test_a_shortage_in_the_middle(kdt):
    B = 3000
    table, held = np.full((B, 2), -1, dtype=np.int32), np.zeros(B, dtype=np.int32)
    free = np.random.RandomState(1).permutation(2000).astype(np.int32)
    state = (table, held, free, 2000, held)
    new = np.where(np.arange(B) % 3 == 0, 16, 8)
    want = op.page_assign(table, held, free, 2000, new, 8, held, 16)
    assert want[5] > 1000 and want[3] <= 1
    _same(_assign(kdt, state, new, 8, held, 16), want)


def test_round_trips_inside_a_graph(kdt):
    """A step's pages taken and given back, captured and replayed: the state comes back every time, and the slots
    are those of a plain call."""
    import torch
    rng = np.random.RandomState(9)
    state = _state(rng, 33, 40, 16, 900, 300)
    t, h, f, n = (_cu(x) for x in (state[0], state[1], state[2], np.array([state[3]], dtype=np.int32)))
    lens = _cu(state[4])
    new = lens + 100
    before = [x.clone() for x in (h, f, n)]
    plain = kdt.page_assign(t, h, f, n, new, 16, start=lens, T=100)
    kdt.page_assign(t, h, f, n, lens, 16)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        slots = kdt.page_assign(t, h, f, n, new, 16, start=lens, T=100)
        kdt.page_assign(t, h, f, n, lens, 16)
    for _ in range(3):
        slots.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(slots, plain)
        for a, b in zip((h, f, n), before):
            assert torch.equal(a, b)


# ---------------------------------------------------------------------------------- writing --
def _bits(t):
    import torch
    return t.view(torch.int16).cpu().numpy()


@pytest.mark.parametrize("B,T", [(1, 1), (64, 1), (3, 37), (2, 1000), (13, 700)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm,rope", [(True, True), (False, True), (True, False), (False, False)])
def test_rows_written(kdt, B, T, dtype, norm, rope):
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(B * T)
    page = 16
    n_pages = -(-B * T * 2 // page)
    c = torch.full((n_pages, page, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    k = torch.full((n_pages, page, 64), -7.0, dtype=torch.bfloat16, device="cuda")
    wide = torch.randn(B, T, 640, device="cuda", generator=g).to(dt)        # slices of a wider buffer
    x, kk = wide[..., :512], wide[..., 560:624]
    gamma = (0.5 + torch.rand(512, device="cuda", generator=g)).to(dt) if norm else None
    pos = torch.randint(0, 1 << 20, (B, T), device="cuda", generator=g).to(torch.int32) if rope else None
    slots = torch.randperm(n_pages * page, device="cuda", generator=g)[:B * T].view(B, T).to(torch.int32)
    drop = torch.rand(B, T, device="cuda", generator=g) < 0.2
    slots[drop] = torch.where(torch.rand(B, T, device="cuda", generator=g) < 0.5, -1, n_pages * page)[drop].to(torch.int32)
    kdt.latent_write_paged(x, kk, c, k, slots, gamma=gamma, eps=1e-5, pos=pos, base=5000.0)
    torch.cuda.synchronize()
    keep = (~drop).cpu().numpy()
    at = slots.cpu().numpy()[keep]
    y = oq.norm(x.double().cpu().numpy(), None if gamma is None else gamma.double().cpu().numpy(), 1e-5)[keep]
    kin = kk.double().cpu().numpy()[keep]
    rot = oq.rope(kin, pos.cpu().numpy()[keep], 5000.0) if rope else kin
    got_c, got_k = c.view(-1, 512).double().cpu().numpy(), k.view(-1, 64).double().cpu().numpy()
    assert (np.abs(got_c[at] - y) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(y)).all()
    mag = np.tile(np.abs(kin[:, :32]) + np.abs(kin[:, 32:]), 2)
    assert (np.abs(got_k[at] - rot) <= 2.0 ** -8 * np.abs(rot) + (8.1e-7 * mag if rope else 0)).all()
    rest = np.setdiff1d(np.arange(n_pages * page), at)
    assert (got_c[rest] == 7.0).all() and (got_k[rest] == -7.0).all()


def test_written_infinities_and_nan(kdt):
    """Without a norm every value goes its own way; with one a NaN or infinity takes its row."""
    import torch
    x = torch.randn(1, 4, 512, device="cuda")
    x[0, 1, 3], x[0, 2, 5] = float("inf"), float("nan")
    k = torch.zeros(1, 4, 64, device="cuda")
    slots = torch.tensor([[2, 9, 4, 0]], dtype=torch.int32, device="cuda")
    for gamma in (None, torch.ones(512, device="cuda")):
        c = torch.zeros(2, 8, 512, dtype=torch.bfloat16, device="cuda")
        kp = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda")
        kdt.latent_write_paged(x, k, c, kp, slots, gamma=gamma)
        got = c.view(16, 512)
        assert torch.isfinite(got[[2, 0]]).all()
        if gamma is None:
            assert torch.isinf(got[9, 3]) and torch.isfinite(got[9, :3]).all() and torch.isnan(got[4, 5])
        else:
            assert torch.isnan(got[9, 3]) and torch.isnan(got[4]).all()


# ------------------------------------------------------------------------------- compaction --
@pytest.mark.parametrize("B,T,page", [(1, 2, 8), (5, 64, 64), (40, 256, 16), (400, 17, 128), (2, 4096, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_compaction(kdt, B, T, page, dtype):
    """As the dense cache's compaction on the same rows; the pages' other rows stay."""
    import torch
    rng = np.random.RandomState(B + T)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    pre = rng.randint(0, 100, B).astype(np.int32)
    W = -(-(100 + T) // page) + 1
    n_pages = B * W + 3
    table = rng.permutation(n_pages)[:B * W].reshape(B, W).astype(np.int32)
    c, k = torch.randn(n_pages, page, 512, device="cuda").to(dt), torch.randn(n_pages, page, 64, device="cuda").to(dt)
    n = rng.randint(0, T + 1, B).astype(np.int32)
    acc = np.full((B, T), -1, dtype=np.int32)
    for b in range(B):
        acc[b, :n[b]] = np.sort(rng.choice(T, n[b], replace=False))
    L = W * page
    t = _cu(table).long()
    rows = (t[:, :, None] * page + torch.arange(page, device="cuda")).view(B, L)
    dense_c, dense_k = c.view(-1, 512)[rows], k.view(-1, 64)[rows]
    p1, p2 = _cu(pre), _cu(pre)
    kdt.kv_compact(dense_c, dense_k, p1, _cu(acc), _cu(n))
    want_c, want_k = c.clone(), k.clone()
    want_c.view(-1, 512)[rows.view(-1)] = dense_c.view(-1, 512)
    want_k.view(-1, 64)[rows.view(-1)] = dense_k.view(-1, 64)
    big = torch.full((B, W + 2), 1 << 30, dtype=torch.int32, device="cuda")
    big[:, :W] = _cu(table)
    kdt.kv_compact_paged(c, k, big[:, :W], p2, _cu(acc), _cu(n))
    assert torch.equal(p1, p2) and torch.equal(c, want_c) and torch.equal(k, want_k)


def test_compaction_skips_pages_that_are_none(kdt):
    import torch
    table = torch.tensor([[3, -1, 9, 2]], dtype=torch.int32, device="cuda")
    c, k = torch.randn(6, 8, 512, device="cuda"), torch.randn(6, 8, 64, device="cuda")
    acc = torch.tensor([[0, 5, 11, 20, 26]], dtype=torch.int32, device="cuda")     # rows 9 (page -1), 15, 24 (2), 30 (2)
    c0 = c.clone()
    pre = torch.tensor([4], dtype=torch.int32, device="cuda")
    acc = torch.nn.functional.pad(acc, (0, 22), value=-1)
    kdt.kv_compact_paged(c, k, table, pre, acc, torch.tensor([5], dtype=torch.int32, device="cuda"))
    want = c0.clone()
    # k = 1, 2: sources on pages -1; k = 3, 4: rows 24 and 30 (page 2) to row 7 (page 3) and row 8 (page -1: not copied)
    want[3, 7] = c0[2, 0]
    assert torch.equal(c, want) and int(pre.item()) == 9


def test_another_device_memory_is_refused(kdt):
    import torch
    with pytest.raises(kdt.KdtError) as e:
        kdt.page_assign(*(torch.zeros(s, dtype=torch.int32).pin_memory() for s in ((2, 3), 2, 6, 1, 2)), 8)
    assert e.value.status == 6


def test_batches_around_the_shared_memory_given_unasked(kdt):
    """Sizes on both sides of the leave that larger scans need, in a process that no larger batch has run in before."""
    import os
    import subprocess
    import sys
    code = """
import numpy as np
import speculative_decoding_tree_absorb_gb300 as kdt
from oracle import paged as op
from tests.test_gpu_pages import _assign, _same, _state
for B in (6015, 6016, 6017, 6110, 6111, 6144, 6145):
    rng = np.random.RandomState(B)
    state = _state(rng, B, 4, 8, 2 * B, 20)
    new, start = rng.randint(0, 33, B), np.zeros(B, dtype=np.int32)
    _same(_assign(kdt, state, new, 8, start, 3), op.page_assign(*state[:4], new, 8, start, 3))
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
