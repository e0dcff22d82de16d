"""GPU tests of kdt_sample against the float64 oracle (oracle/paged.py).

Tokens are equal unless the draw, or top-p's border, lies within 2^-38 of the kept mass of one: the weights are held to
2^-44 of the largest and off by at most 2^-40 of themselves, and float64's own exponentials are no better than 2^-52.
logp: 1e-6 + 2^-23 of its size.
"""
import numpy as np
import pytest

from oracle import paged as op

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


def _check(kdt, logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, skip=0, **kw):
    """Settings as arrays or numbers; `skip` rows may be too near a border to be compared."""
    import torch
    R, V = logits.shape
    err = torch.full((1,), 5, dtype=torch.int32, device="cuda")

    def dev(v, dt):
        return torch.from_numpy(np.asarray(v, dtype=dt)).cuda() if np.ndim(v) else v
    tok, logp = kdt.sample(logits, torch.from_numpy(u).cuda(), temperature=dev(temperature, np.float32), top_k=dev(top_k, np.int32),
                           top_p=dev(top_p, np.float32), min_p=dev(min_p, np.float32), err=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    tok, logp, l = tok.cpu().numpy(), logp.cpu().numpy(), logits.double().cpu().numpy()

    def one(v, r, dt):
        return float(np.asarray(v, dtype=dt)[r]) if np.ndim(v) else v
    near = 0
    for r in range(R):
        t, lp, gap = op.sample(l[r], u[r], one(temperature, r, np.float32), int(one(top_k, r, np.int32)), one(top_p, r, np.float32),
                               one(min_p, r, np.float32))
        if gap < 2.0 ** -38 and tok[r] != t:
            near += 1
            continue
        assert tok[r] == t, (r, tok[r], t, gap)
        assert abs(logp[r] - lp) <= 1e-6 + 2.0 ** -23 * abs(lp), (r, logp[r], lp)
    assert near <= skip
    return tok, logp


def _logits(rng, R, V, kind, dtype):
    import torch
    if kind == "peaked":
        l = 14.0 - rng.uniform(0.8, 2.0, (R, 1)) * np.log1p(rng.rand(R, V).argsort(-1)) + 0.4 * rng.randn(R, V)
    elif kind == "normal":
        l = 2.0 * rng.randn(R, V)
    elif kind == "ties":
        l = rng.randint(-3, 4, (R, V)) * 0.5
    else:                                   # "flat"
        l = np.full((R, V), 3.25)
    t = torch.from_numpy(l).cuda()
    return t.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 32000, 50257])
@pytest.mark.parametrize("kind", ["peaked", "normal", "ties", "flat"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_settings_of_every_row(kdt, V, kind, dtype):
    rng = np.random.RandomState(V)
    R = 24 if V < 10000 else 8
    logits = _logits(rng, R, V, kind, dtype)
    u = rng.rand(R).astype(np.float32)
    u[0] = 0.0
    u[-1] = np.float32(1.0 - 2.0 ** -24)
    _check(kdt, logits, u, temperature=rng.choice([0.5, 1.0, 1.3], R), top_k=rng.choice([0, -1, 1, 2, 17, 50, V, V + 5, max(1, V // 3)], R),
           top_p=rng.choice([1.0, 0.95, 0.5, 0.1, 0.0, -1.0, 2.0], R), min_p=rng.choice([0.0, 0.01, 0.1, 0.5, 1.0, 3.0, -1.0], R))
    _check(kdt, logits, u)
    _check(kdt, logits, u, top_p=0.9, temperature=0.8)
    _check(kdt, logits, u, top_k=5)
    _check(kdt, logits, u, min_p=0.05)


@pytest.mark.parametrize("R,V", [(1, 160000), (200, 9001), (3, 524288), (600, 130), (17, 151936)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sizes(kdt, R, V, dtype):
    rng = np.random.RandomState(R)
    logits = _logits(rng, R, V, "peaked", dtype)
    u = rng.rand(R).astype(np.float32)
    _check(kdt, logits, u, top_k=40, top_p=0.95, min_p=0.01, temperature=0.7)
    _check(kdt, logits, u, top_p=rng.uniform(0.2, 1.0, R))
    _check(kdt, logits, u)


def test_rows_apart_and_odd_starts(kdt):
    import torch
    rng = np.random.RandomState(3)
    for dtype in (torch.bfloat16, torch.float32):
        big = torch.full((9, 5003), float("nan"), dtype=dtype, device="cuda")
        big[:, 3:4804] = _logits(rng, 9, 4801, "peaked", "f32").to(dtype)
        _check(kdt, big[:, 3:4804], rng.rand(9).astype(np.float32), top_p=0.8, top_k=900)


def test_masked_tokens(kdt):
    """-inf logits, and logits far below (weight 0), are never drawn; a row with one token left gives it."""
    import torch
    rng = np.random.RandomState(4)
    logits = _logits(rng, 6, 3000, "normal", "f32")
    logits[0, 1:] = -float("inf")
    logits[1, :2990] = -float("inf")
    logits[2, 7:] = torch.finfo(torch.float32).min
    logits[3] = -1e30
    logits[3, 2999] = 4.0
    logits[4, ::2] = -float("inf")
    u = np.array([0.99, 0.999, 0.9999, 0.5, 0.7, 0.2], dtype=np.float32)
    for kw in (dict(), dict(top_k=2000), dict(top_p=0.99), dict(top_k=2995, top_p=0.999, min_p=1e-9)):
        tok, _ = _check(kdt, logits, u, **kw)
        assert tok[0] == 0 and tok[1] >= 2990 and tok[2] < 7 and tok[3] == 2999 and tok[4] % 2 == 1


@pytest.mark.parametrize("V", [700, 9000])
@pytest.mark.parametrize("spread,temp", [(1000.0, 900.0), (2.0 ** -11, 1e-3), (2.0 ** -9, 2e-3), (60000.0, 1000.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_spreads_that_one_bin_holds(kdt, V, spread, temp, dtype):
    """Logits far below the largest, or all within a hair of zero, that have weights all the same."""
    import torch
    rng = np.random.RandomState(V)
    l = torch.from_numpy(rng.uniform(-spread, spread, (9, V))).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    l[4, ::3] = float("-inf")
    u = rng.rand(9).astype(np.float32)
    _check(kdt, l, u, temperature=temp)
    _check(kdt, l, u, temperature=temp, top_p=rng.uniform(0.05, 0.99, 9))
    _check(kdt, l, u, temperature=temp, top_k=rng.randint(1, V, 9), min_p=0.02)
    _check(kdt, l, u, temperature=temp, top_k=V - 5, top_p=0.9, min_p=rng.uniform(0, 0.3, 9))


def test_greedy_rows(kdt):
    rng = np.random.RandomState(5)
    logits = _logits(rng, 8, 7000, "ties", "bf16")
    temp = np.array([0, 1, 0, 0.5, 0, 1, 0, 0], dtype=np.float32)
    tok, logp = _check(kdt, logits, rng.rand(8).astype(np.float32), temperature=temp, top_p=0.9)
    first = logits.float().cpu().numpy().argmax(-1)
    assert (tok[temp == 0] == first[temp == 0]).all() and (logp[temp == 0] == 0).all()
    _check(kdt, logits, rng.rand(8).astype(np.float32), temperature=0.0)


def test_signed_zeros_are_equal(kdt):
    import torch
    logits = torch.tensor([[-0.0, 0.0, -0.0, 0.0, -1.0]], device="cuda")
    for k in (1, 2, 3):
        tok, _ = _check(kdt, logits, np.array([0.999], dtype=np.float32), top_k=k)
        assert tok[0] == k - 1


def test_rows_without_a_token(kdt):
    """A NaN, a +inf, nothing but -inf, settings that are no numbers in range: token -1, named, the others as ever."""
    import torch
    rng = np.random.RandomState(6)
    logits = _logits(rng, 9, 2000, "peaked", "f32")
    good = logits.clone()
    logits[2, 5], logits[4, 1999], logits[5] = float("nan"), float("inf"), -float("inf")
    temp = torch.ones(9, device="cuda")
    temp[6], temp[7] = -1.0, 2e3
    top_p = torch.full((9,), 0.9, device="cuda")
    top_p[8] = float("nan")
    u = torch.from_numpy(rng.rand(9).astype(np.float32)).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    tok, logp = kdt.sample(logits, u, temperature=temp, top_p=top_p, err=err)
    assert int(err.item()) == 3
    bad = [2, 4, 5, 6, 7, 8]
    assert (tok[bad] == -1).all() and (logp[bad] == 0).all()
    want, _ = kdt.sample(good, u, top_p=0.9, err=err)
    # (0.9 as a double and as a float32 differ: the array's rows are compared with an array's)
    want, _ = kdt.sample(good, u, top_p=torch.full((9,), 0.9, device="cuda"), err=err)
    assert int(err.item()) == 0 and torch.equal(tok[[0, 1, 3]], want[[0, 1, 3]])


def test_numbers_and_arrays_agree(kdt):
    import torch
    rng = np.random.RandomState(7)
    logits = _logits(rng, 33, 12345, "peaked", "bf16")
    u = torch.from_numpy(rng.rand(33).astype(np.float32)).cuda()
    full = lambda v, dt=torch.float32: torch.full((33,), v, dtype=dt, device="cuda")
    a = kdt.sample(logits, u, temperature=0.75, top_k=100, top_p=0.875, min_p=0.03125)
    b = kdt.sample(logits, u, temperature=full(0.75), top_k=full(100, torch.int32), top_p=full(0.875), min_p=full(0.03125))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert kdt.sample(logits, u, want_logp=False)[1] is None


def test_captured_and_replayed_on_new_logits(kdt):
    import torch
    rng = np.random.RandomState(8)
    logits = _logits(rng, 12, 32000, "peaked", "f32")
    u = torch.from_numpy(rng.rand(12).astype(np.float32)).cuda()
    kdt.sample(logits, u, top_k=30, top_p=0.9)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        tok, logp = kdt.sample(logits, u, top_k=30, top_p=0.9)
    for k in range(3):
        logits.copy_(_logits(rng, 12, 32000, "peaked", "f32"))
        graph.replay()
        torch.cuda.synchronize()
        want = kdt.sample(logits, u, top_k=30, top_p=0.9)
        assert torch.equal(tok, want[0]) and torch.equal(logp, want[1])


def test_not_device_memory_is_refused(kdt):
    import torch
    with pytest.raises(kdt.KdtError) as e:
        kdt.sample(torch.zeros(2, 8, device="cuda"), torch.zeros(2).pin_memory())
    assert e.value.status == 6


@pytest.mark.parametrize("V,most", [(1000, 200), (32000, 200), (160003, 80)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logp_has_no_order(kdt, V, most, dtype):
    """A row's log-probability, before the filters by its definition, has the same bits alone and in batches of any size
    (other clusters, other slices), under every filter, and from rows that start on no 16-byte boundary."""
    import torch
    rng = np.random.RandomState(V)
    logits = _logits(rng, most, V, "normal", dtype)
    logits[:, 0] = logits.amax(1) + 0.5          # u = 0 draws this token under every filter
    off = torch.zeros((most, V + 3), dtype=logits.dtype, device="cuda")[:, 1:V + 1]
    off.copy_(logits)
    u = torch.zeros(most, device="cuda")
    temp = torch.from_numpy(rng.uniform(0.5, 1.5, most).astype(np.float32)).cuda()
    tok, want = kdt.sample(logits, u, temperature=temp)
    assert (tok == 0).all()
    for kw in (dict(), dict(top_p=0.9), dict(top_k=50), dict(top_k=V // 2, top_p=0.99), dict(min_p=1e-3)):
        for n in (1, 2, 12, 30, 70, most):
            for lg in (logits, off):
                tok, logp = kdt.sample(lg[most - n:], u[:n], temperature=temp[most - n:], **kw)
                assert (tok == 0).all() and torch.equal(logp, want[most - n:]), (kw, n)
