"""GPU tests of the 8-bit latent cache: rows written (norm, rotation, quantisation), read
back and compacted, against the float64 oracle (oracle/q8.py).

Tolerances, from the roundings each result goes through:
 * a code is y * 2^-e rounded to e4m3: off by at most half a step, 2^-4 |y| or, in the
   subnormals, 2^-10 * 2^e;
 * y itself is computed in float32: the sum of squares takes 16 fused adds and 5 shuffle
   adds (21 roundings, halved by the square root) and then a square root, a division and
   two products: below 16 * 2^-24 = 2^-20 relative;
 * k_pe: float32 angles within 2e-7 of the exact ones (rounding of the turn fraction to 24
   bits, times pi), sine and cosine within 2 units (2.4e-7), three roundings of 2^-24, then
   half a bf16 step, 2^-8 relative: 2^-8 |r| + 8e-7 (|k0| + |k1|).
"""
import numpy as np
import pytest

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


def _gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def _cache(B, L, fill=0xA5):
    """Cache arrays that hold one byte everywhere, so that an untouched row shows."""
    import torch
    return (torch.full((B, L, 512), fill, dtype=torch.uint8, device="cuda"),
            torch.full((B, L, 16), fill, dtype=torch.uint8, device="cuda"),
            torch.full((B, L, 128), fill, dtype=torch.uint8, device="cuda").view(torch.bfloat16))


def _np(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


def _check_rows(y, k, codes, scale, k_pe):
    """Stored rows [N, ...] against float64 y [N,512] (before quantisation) and k [N,64] (rotated),
    kin = |k0| + |k1| bound folded into k's second entry."""
    krot, kmag = k
    g = np.abs(y).reshape(-1, 16, 32).max(-1)
    e = scale.astype(np.int64) - 127
    slack = 2.0 ** -20
    assert ((e >= -100) & (e <= 100)).all()
    fits = (g <= 448.0 * np.exp2(e) * (1 + slack)) | (e == 100)
    least = (g > 448.0 * np.exp2(e - 1.0) * (1 - slack)) | (e == -100)
    assert fits.all() and least.all()
    v = oq.dequantise(codes, scale)
    unit = np.repeat(np.exp2(e.astype(np.float64)), 32, axis=-1)
    tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * unit) + slack * np.abs(y)
    big = np.abs(y) > 448.0 * unit
    assert (np.abs(v - np.where(big, np.sign(y) * 448.0 * unit, y)) <= tol).all()
    assert (np.abs(k_pe - krot) <= 2.0 ** -8 * np.abs(krot) + 8e-7 * kmag).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,norm,rot", [(1, 1, True, True), (3, 7, True, True), (2, 300, False, True),
                                          (5, 64, True, False), (1, 5000, True, True)])
def test_write_matches_oracle_and_leaves_other_rows(kdt, dtype, B, T, norm, rot):
    import torch
    g = _gen(B * 1000 + T)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    kv = (torch.randn(B, T, 576, device="cuda", generator=g) * 3).to(dt)
    gamma = (0.1 + torch.rand(512, device="cuda", generator=g)).to(dt) if norm else None
    pre = torch.tensor([(37 * b) % 50 for b in range(B)], dtype=torch.int32, device="cuda")
    L = 50 + T + 4
    pos = (torch.randint(0, 1 << 20, (B, T), device="cuda", generator=g)).to(torch.int32) if rot else None
    c8, sc, kp = _cache(B, L)
    old = [t.clone() for t in (c8, sc, kp)]
    kdt.latent_write_q8(kv[..., :512], kv[..., 512:], c8, sc, kp, pre, gamma=gamma, eps=1e-5, pos=pos, base=10000.0)
    x = _np(kv)
    y = oq.norm(x[..., :512], None if gamma is None else _np(gamma), 1e-5)
    k = oq.rope(x[..., 512:], pos.cpu().numpy(), 10000.0) if rot else x[..., 512:]
    mag = np.abs(x[..., 512:544]) + np.abs(x[..., 544:])
    mag = np.concatenate([mag, mag], -1)
    for b, p in enumerate(pre.tolist()):
        r = slice(p, p + T)
        _check_rows(y[b], (k[b], mag[b]), c8[b, r].cpu().numpy(), sc[b, r].cpu().numpy(), _np(kp[b, r]))
        for t, o in zip((c8, sc, kp), old):
            t, o = (t.view(torch.int16), o.view(torch.int16)) if t.dtype == torch.bfloat16 else (t, o)
            assert torch.equal(t[b, :p], o[b, :p]) and torch.equal(t[b, p + T:], o[b, p + T:])


def test_write_padded_batch_and_rows_outside_the_cache(kdt):
    import torch
    g = _gen(5)
    B, T, L = 4, 9, 12
    kv = torch.randn(B, T, 576, device="cuda", generator=g)
    pre = torch.tensor([0, 8, -3, 2 ** 31 - 4], dtype=torch.int32, device="cuda")     # all, 4, 6 and no rows inside
    n = torch.tensor([5, 9, 9, 9], dtype=torch.int32, device="cuda")
    c8, sc, kp = _cache(B, L)
    kdt.latent_write_q8(kv[..., :512], kv[..., 512:], c8, sc, kp, pre, n_rows=n)
    full = [_cache(1, T)[i] for i in range(3)]
    written = np.zeros((B, L), dtype=bool)
    for b, (p, m) in enumerate(zip(pre.tolist(), n.tolist())):
        full = _cache(1, T)
        kdt.latent_write_q8(kv[b:b + 1, :, :512], kv[b:b + 1, :, 512:], *full, torch.zeros(1, dtype=torch.int32, device="cuda"))
        for i in range(m):
            if 0 <= p + i < L:
                written[b, p + i] = True
                assert torch.equal(c8[b, p + i], full[0][0, i]) and torch.equal(sc[b, p + i], full[1][0, i])
                assert torch.equal(kp[b, p + i], full[2][0, i])
    left = torch.from_numpy(~written).cuda()
    assert (c8[left] == 0xA5).all() and (sc[left] == 0xA5).all()
    assert (kp.view(torch.uint8)[left] == 0xA5).all()
    assert written.sum() == 5 + 4 + 6


def test_write_special_values(kdt):
    """Zeros, one huge or tiny element, infinities and NaN: the group with them reads as NaN, the
    others of the row are not touched by it (no norm)."""
    import torch
    x = torch.zeros(8, 1, 576, device="cuda")
    x[1, 0, 5] = float("nan")
    x[2, 0, 40] = float("-inf")
    x[3, 0, :512] = 1e-38
    x[4, 0, :512] = 3e38
    x[5, 0, 0], x[5, 0, 1] = 448.0, 0.001
    x[6, 0, 0] = 448.00003
    x[7, 0, 1], x[7, 0, 33] = -0.0, 2.0 ** -120
    x[1, 0, 100] = 3.0
    c8, sc, kp = _cache(8, 1)
    zero = torch.zeros(8, dtype=torch.int32, device="cuda")
    kdt.latent_write_q8(x[..., :512], x[..., 512:], c8, sc, kp, zero)
    s = sc[:, 0].cpu().numpy()
    assert (s[0] == 27).all() and (c8[0] == 0).all()
    assert s[1, 0] == 255 and (c8[1, 0, :32] == 0).all() and s[1, 3] == 127 + (-7)     # 3 <= 448 * 2^-7 = 3.5
    assert s[2, 1] == 255 and (np.delete(s[2], 1) == 27).all()
    assert (s[3] == 27).all() and (c8[3] == 0).all()
    assert (s[4] == 227).all() and (c8[4] == 0x7E).all()                                # saturates at 448 * 2^100
    assert s[5, 0] == 127 and c8[5, 0, 0] == 0x7E and c8[5, 0, 1] == 1                  # 0.001 -> 2^-9 * 1 (step 2^-9)
    assert s[6, 0] == 128
    assert s[7, 1] == 27 and (c8[7, 0, 32:64] == 0).all()
    c, _ = kdt.latent_read_q8(c8, sc, kp, None, 1)
    nan = torch.isnan(c[:, 0]).cpu().numpy()
    want = np.zeros((8, 512), dtype=bool)
    want[1, :32] = want[2, 32:64] = True
    assert np.array_equal(nan, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,R,L", [(1, 1, 1), (3, 17, 40), (4, 700, 701)])
def test_read_is_exact(kdt, dtype, B, R, L):
    """Every code (but the two NaN ones) under every valid scale byte reads as its value."""
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = _gen(B + R)
    c8 = torch.randint(0, 256, (B, L, 512), device="cuda", generator=g).to(torch.uint8)
    c8 = torch.where((c8 & 127) == 127, torch.zeros_like(c8), c8)
    sc = torch.randint(27, 228, (B, L, 16), device="cuda", generator=g).to(torch.uint8)
    sc[:, L // 2, 3] = 255
    kp = torch.randn(B, L, 64, device="cuda", generator=g).to(torch.bfloat16)
    start = torch.tensor([(3 * b) % max(1, L - R + 1) - (1 if b == 2 else 0) for b in range(B)], dtype=torch.int32,
                         device="cuda")                                    # sequence 2 may start at row -1
    c, k = kdt.latent_read_q8(c8, sc, kp, start, R, dtype=dt)
    assert c.dtype == dt and k.dtype == dt
    v, kk = oq.dequantise(c8.cpu().numpy(), sc.cpu().numpy()), _np(kp)
    got_c, got_k = _np(c), _np(k)
    for b, s in enumerate(start.tolist()):
        for i in range(R):
            if 0 <= s + i < L:
                assert np.array_equal(got_c[b, i], v[b, s + i], equal_nan=True) and np.array_equal(got_k[b, i], kk[b, s + i])
            else:
                assert (got_c[b, i] == 0).all() and (got_k[b, i] == 0).all()


def test_read_ragged_leaves_rows_behind(kdt):
    import torch
    c8, sc, kp = _cache(3, 20)
    sc.fill_(127)
    n = torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda")
    out_c = torch.full((3, 9, 512), 7.0, device="cuda")
    out_k = torch.full((3, 9, 64), 7.0, device="cuda")
    kdt.latent_read_q8(c8, sc, kp, None, 9, n_rows=n, out_c=out_c, out_k=out_k)
    for b, m in enumerate(n.tolist()):
        assert (out_c[b, m:] == 7.0).all() and (out_k[b, m:] == 7.0).all()
        assert (out_c[b, :m] == float(oq.CODES[0xA5])).all()


def test_far_rows_pass_32_bits(kdt):
    """Row offsets of the last sequence pass 2^31 elements and bytes of c_q8."""
    import torch
    B, L, T = 3, 2_200_000, 5
    c8 = torch.zeros(B, L, 512, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(B, L, 16, dtype=torch.uint8, device="cuda")
    kp = torch.zeros(B, L, 64, dtype=torch.bfloat16, device="cuda")
    kv = torch.randn(B, T, 576, device="cuda", generator=_gen(1)).to(torch.bfloat16)
    pre = torch.full((B,), L - T, dtype=torch.int32, device="cuda")
    kdt.latent_write_q8(kv[..., :512], kv[..., 512:], c8, sc, kp, pre)
    small = [t[:, L - T:].contiguous() for t in (c8, sc, kp)]
    ref = _cache(B, T)
    kdt.latent_write_q8(kv[..., :512], kv[..., 512:], *ref, torch.zeros_like(pre))
    for t, r in zip(small, ref):
        assert torch.equal(t, r)
    c, k = kdt.latent_read_q8(c8, sc, kp, pre, T)
    c2, k2 = kdt.latent_read_q8(*ref, None, T)
    assert torch.equal(c, c2) and torch.equal(k, k2)
    acc = torch.tensor([[0, 2, 4, -1, -1]] * B, dtype=torch.int32, device="cuda")
    n_acc = torch.full((B,), 3, dtype=torch.int32, device="cuda")
    kdt.kv_compact_q8(c8, sc, kp, pre, acc, n_acc)
    for t, r in zip((c8, sc, kp), ref):
        assert torch.equal(t[:, L - T:L - T + 3], r[:, [0, 2, 4]])
    assert (pre == L - T + 3).all()


@pytest.mark.parametrize("B,T", [(1, 1), (4, 64), (7, 300), (2, 4096)])
def test_compact_moves_the_path(kdt, B, T):
    import torch
    g = _gen(T)
    L = 40 + T
    c8 = torch.randint(0, 256, (B, L, 512), device="cuda", generator=g).to(torch.uint8)
    sc = torch.randint(0, 256, (B, L, 16), device="cuda", generator=g).to(torch.uint8)
    kp = torch.randn(B, L, 64, device="cuda", generator=g).to(torch.bfloat16)
    ref = [t.clone() for t in (c8, sc, kp)]
    pre = [(11 * b) % 38 for b in range(B)]
    rng = np.random.RandomState(T)
    acc = np.full((B, T), -1, dtype=np.int32)
    n = []
    for b in range(B):
        path = [0] + sorted(rng.permutation(np.arange(1, T))[:rng.randint(0, T)].tolist())
        acc[b, :len(path)] = path
        n.append(len(path))
    d_pre = torch.tensor(pre, dtype=torch.int32, device="cuda")
    kdt.kv_compact_q8(c8, sc, kp, d_pre, torch.from_numpy(acc).cuda(), torch.tensor(n, dtype=torch.int32, device="cuda"))
    for b in range(B):
        for r, t in zip(ref, (c8, sc, kp)):
            old = r[b].clone()
            for k in range(n[b]):
                r[b, pre[b] + k] = old[pre[b] + acc[b, k]]
            assert torch.equal(r[b], t[b])
    assert d_pre.tolist() == [p + m for p, m in zip(pre, n)]


def test_write_and_read_in_a_captured_graph_on_another_stream(kdt):
    import torch
    g = _gen(9)
    kv = torch.randn(2, 6, 576, device="cuda", generator=g)
    pre = torch.zeros(2, dtype=torch.int32, device="cuda")
    c8, sc, kp = _cache(2, 6)
    out_c, out_k = torch.empty(2, 6, 512, device="cuda"), torch.empty(2, 6, 64, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            kdt.latent_write_q8(kv[..., :512], kv[..., 512:], c8, sc, kp, pre)
            kdt.latent_read_q8(c8, sc, kp, None, 6, out_c=out_c, out_k=out_k)
    for seed in (1, 2):
        kv.copy_(torch.randn(2, 6, 576, device="cuda", generator=_gen(seed)))
        graph.replay()
        torch.cuda.synchronize()
        ref = _cache(2, 6)
        kdt.latent_write_q8(kv[..., :512], kv[..., 512:], *ref, pre)
        c, k = kdt.latent_read_q8(*ref, None, 6, dtype=torch.float32)
        assert torch.equal(c, out_c) and torch.equal(k, out_k)


@pytest.mark.parametrize("B,T", [(1, 1024), (30, 256), (100, 256), (250, 300), (700, 40), (1300, 5)])
def test_compaction_of_every_split(kdt, B, T):
    """Batches that get eight CTAs a sequence, fewer and one: both caches' rows as copied one by one, rows
    beside the path as they were, prefixes advanced; paths of any length, none and one among them."""
    import torch
    rng = np.random.RandomState(B)
    L = T + 40
    pre = rng.randint(0, 40, B).astype(np.int32)
    n = np.minimum(rng.choice([0, 1, 2, 6, T // 2, T], B), T).astype(np.int32)
    acc = np.full((B, T), -1, dtype=np.int32)
    for b in range(B):
        if n[b]:
            acc[b, :n[b]] = np.concatenate([[0], 1 + np.sort(rng.choice(T - 1, n[b] - 1, replace=False))])
    g = torch.Generator(device="cuda").manual_seed(B)
    big = lambda d, t: torch.randint(-2 ** 15, 2 ** 15 - 1, (B, L, d), device="cuda", generator=g).to(torch.int16).view(t)
    q8 = [big(256, torch.uint8), big(8, torch.uint8), big(64, torch.bfloat16)]
    kv = [big(512, torch.bfloat16), big(64, torch.bfloat16)]
    was = [x.clone().view(torch.uint8) for x in q8 + kv]
    move = [(b, int(pre[b]) + k, int(pre[b]) + int(acc[b, k])) for b in range(B) for k in range(1, n[b])]
    if move:
        bb, to, at = (torch.tensor(x, device="cuda") for x in zip(*move))
        for x in was:
            x[bb, to] = x[bb, at]
    dev = [torch.from_numpy(x).cuda() for x in (acc, n)]
    p8, p16 = (torch.from_numpy(pre).cuda() for _ in range(2))
    kdt.kv_compact_q8(*q8, p8, *dev)
    kdt.kv_compact(*kv, p16, *dev)
    torch.cuda.synchronize()
    for x, w in zip(q8 + kv, was):
        assert torch.equal(x.view(torch.uint8), w)
    assert p8.tolist() == p16.tolist() == (pre + n).tolist()
