"""GPU tests of the sampled tree verification (kdt_tree_sample) against the float64 oracle
(oracle/q8.py): paths, counts and bonus tokens are whole numbers and have to be equal.

The oracle's weights are float64 exponentials rounded to 2^-44 of the largest, the
library's the same numbers to within 2^-40 of each, so a running sum is off by at most
V 2^-40 / Z of the rest: a threshold would have to fall that near to a border (chance below
1e-6 a case at the sizes here, and the seeds are fixed). logp is float32 of a float64 value
whose sum is within 4e-5 of exact on the fast path: 4e-5 + 2^-23 |logp|.
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


def _tree(rng, T, back=6):
    return np.array([-1] + [rng.randint(max(0, i - back), i) for i in range(1, T)], dtype=np.int32)


def _inputs(seed, B, T, V, dtype, pad=0, agree=0.8):
    import torch
    rng = np.random.RandomState(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    parent = np.stack([_tree(rng, T) for _ in range(B)])
    tok = rng.randint(0, V, (B, T)).astype(np.int32)
    buf = torch.randn(B, T, V + pad, device="cuda", generator=g) * 2
    lift = np.where(rng.rand(B, T) < agree, 15.0, 4.0)
    for b in range(B):
        for i in range(1, T):
            buf[b, parent[b, i], tok[b, i]] = lift[b, i]
    buf = buf.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return dict(parent=parent, tok=tok, logits=buf[..., :V], u=rng.rand(B, T).astype(np.float32),
                ub=rng.rand(B).astype(np.float32), temp=1.0)


def _run(kdt, d, **kw):
    import torch
    err = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    acc, n, bonus, logp = kdt.tree_sample(torch.from_numpy(d["parent"]).cuda(), torch.from_numpy(d["tok"]).cuda(),
                                          d["logits"], torch.from_numpy(d["u"]).cuda(), torch.from_numpy(d["ub"]).cuda(),
                                          temperature=d["temp"], err=err, **kw)
    torch.cuda.synchronize()
    return acc.cpu().numpy(), n.cpu().numpy(), bonus.cpu().numpy(), logp.cpu().numpy(), int(err.item())


def _check(d, got, err=0):
    acc, n, bonus, logp, e = got
    assert e == err
    for b in range(len(n)):
        path, want, lp = oq.tree_sample(d["parent"][b], d["tok"][b], lambda i: d["logits"][b, i].double().cpu().numpy(),
                                        d["u"][b].astype(np.float64), float(d["ub"][b]), d["temp"])
        assert acc[b, :n[b]].tolist() == path and (acc[b, n[b]:] == -1).all(), (b, acc[b], path)
        assert bonus[b] == want, (b, bonus[b], want)
        assert (np.abs(logp[b, :n[b]] - lp) <= 4e-5 + 2.0 ** -23 * np.abs(lp)).all()
        assert (logp[b, n[b]:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,V,pad", [(1, 1, 1, 0), (2, 5, 7, 0), (3, 9, 997, 0), (4, 17, 32000, 0), (1, 6, 160000, 0),
                                       (40, 12, 5000, 3), (200, 4, 1030, 0), (3, 8, 4099, 5)])
def test_matches_oracle(kdt, dtype, B, T, V, pad):
    d = _inputs(B * 1000 + V, B, T, V, dtype, pad)
    d["temp"] = [1.0, 0.7, 1.9][V % 3]
    _check(d, _run(kdt, d))


def test_vocabulary_larger_than_shared_memory(kdt):
    for dtype in ("f32", "bf16"):
        _check((d := _inputs(3, 1, 4, 524288, dtype)), _run(kdt, d))
        _check((d := _inputs(4, 160, 2, 120001, dtype)), _run(kdt, d))        # one CTA a sequence, rows unaligned


def test_chain_accepted_to_the_end_and_rejected_at_once(kdt):
    d = _inputs(7, 2, 64, 3000, "f32")
    d["parent"][:] = np.arange(64) - 1
    for i in range(1, 64):
        d["logits"][:, i - 1, :] = 0
        for b in range(2):
            d["logits"][b, i - 1, d["tok"][b, i]] = 30.0
    d["u"][1, 1] = np.float32(1 - 2.0 ** -24)
    d["logits"][1, 0, d["tok"][1, 1]] = -40.0
    got = _run(kdt, d)
    assert got[1].tolist() == [64, 1]
    _check(d, got)


def test_equal_numbers_at_the_border(kdt):
    """Two tokens of equal weight: u 0.5 is not below one half, the float before it is; and
    thresholds that fall on a running sum exactly go to the next token."""
    d = _inputs(8, 4, 2, 2, "f32")
    d["parent"][:, 1], d["tok"][:, 1] = 0, 0
    d["logits"][:] = 1.5
    d["u"][:, 1] = [0.5, np.nextafter(np.float32(0.5), np.float32(0)), 0.0, np.float32(1 - 2.0 ** -24)]
    d["ub"][:] = [0.0, 0.5, np.nextafter(np.float32(0.5), np.float32(0)), np.float32(1 - 2.0 ** -24)]
    got = _run(kdt, d)
    assert got[1].tolist() == [1, 2, 2, 1]
    assert got[2].tolist() == [1, 1, 0, 1]
    _check(d, got)


def test_tests_near_the_border_use_exact_sums(kdt):
    """u_node next to p(child), on both sides, closer than the fast sums resolve."""
    d = _inputs(9, 64, 2, 4000, "bf16", agree=1.0)
    for b in range(64):
        d["parent"][b, 1] = 0
        row = d["logits"][b, 0].double().cpu().numpy()
        w = oq.sample_weights(row, 1.0)
        u = np.float32(w[d["tok"][b, 1]] / w.sum())
        for _ in range(b % 5):
            u = np.nextafter(u, np.float32(b % 2))
        d["u"][b, 1] = u
    got = _run(kdt, d)
    assert 8 < (got[1] == 2).sum() < 56
    _check(d, got)


def test_repeated_and_invalid_tokens(kdt):
    d = _inputs(10, 3, 8, 500, "f32")
    d["parent"][:] = [-1, 0, 0, 0, 0, 1, 2, 3]
    d["tok"][0, 1:5] = 17                                # one token drafted four times: counted once
    d["logits"][0, 0, 17] = 7.0
    d["u"][0, 1:5] = [0.99999, 0.0, 0.0, 0.0]
    _check({k: (v[:1] if not isinstance(v, float) else v) for k, v in d.items()},
           _run(kdt, {k: (v[:1] if not isinstance(v, float) else v) for k, v in d.items()}))
    d["tok"][1, 2], d["tok"][2, 3] = -1, 500             # outside the vocabulary: never accepted, reported
    d["u"][1:] = 0.0
    d["tok"][1, 1] = d["tok"][1, 3]
    d["logits"][1:, 0, :] = -np.inf
    d["logits"][1:, 0, 3] = 1.0                          # nothing but token 3 can be drawn
    got = _run(kdt, d)
    assert got[4] == 1 + 8 + 2
    _check(d, got, err=1 + 8 + 2)


def test_rows_without_a_distribution(kdt):
    """NaN, +inf or nothing but -inf on the way: the walk ends there with bonus -1; elsewhere they
    do not matter."""
    d = _inputs(11, 4, 4, 900, "f32")
    d["parent"][:] = [-1, 0, 1, 2]
    for b in range(4):
        for i in range(1, 4):
            d["logits"][b, i - 1, d["tok"][b, i]] = 60.0
    d["logits"][0, 2, 899] = float("nan")
    d["logits"][1, 2, 0] = float("inf")
    d["logits"][2, 1] = -float("inf")
    d["logits"][3, 0, 5] = 90.0                          # the walk of sequence 3 stops at the root
    d["logits"][3, 3, 7] = float("nan")
    got = _run(kdt, d)
    assert got[1].tolist() == [3, 3, 2, 1] and got[2].tolist() == [-1, -1, -1, 5]
    assert got[4] == 1 + 2                               # the first one: node 2 of sequence 0
    _check(d, got, err=3)


def test_masked_tokens_are_never_drawn(kdt):
    d = _inputs(12, 64, 1, 2000, "bf16")
    keep = np.random.RandomState(1).rand(2000) < 0.01
    d["logits"][:, :, np.flatnonzero(~keep)] = -float("inf")
    d["ub"][:4] = [0.0, np.float32(1 - 2.0 ** -24), 0.5, 2.0 ** -24]
    got = _run(kdt, d)
    assert keep[got[2]].all()
    _check(d, got)


def test_star_of_4095_children_and_malformed_parents(kdt):
    d = _inputs(13, 1, 4096, 300, "f32")
    d["parent"][0, 1:] = 0
    d["logits"][0, 0] = 0.0
    d["tok"][0, 1:4000] = np.arange(3999) % 250
    d["u"][0] = 0.999
    _check(d, _run(kdt, d))
    d["parent"][0, 9] = 9
    d["parent"][0, 77] = -2
    got = _run(kdt, d)
    assert got[4] == 10


def test_distribution_of_the_first_token(kdt):
    """20000 sequences with the same logits and random numbers of their own: the first emitted
    token is distributed as softmax(logits), children drafted or not (chi square, 23 degrees of
    freedom: above 60 has probability 4e-5)."""
    import torch
    B, V, T = 20000, 24, 4
    rng = np.random.RandomState(2)
    row = rng.randn(V).astype(np.float32)
    d = dict(parent=np.tile(np.array([-1, 0, 0, 0], dtype=np.int32), (B, 1)),
             tok=np.tile(np.array([0, 3, 11, 3], dtype=np.int32), (B, 1)),
             logits=torch.from_numpy(row).cuda().expand(B, T, V).contiguous(), u=rng.rand(B, T).astype(np.float32),
             ub=rng.rand(B).astype(np.float32), temp=1.3)
    acc, n, bonus, _, err = _run(kdt, d)
    assert err == 0
    first = np.where(n > 1, d["tok"][np.arange(B), np.maximum(acc[:, 1], 0)], bonus)
    p = np.exp(row / 1.3) / np.exp(row / 1.3).sum()
    chi = ((np.bincount(first, minlength=V) - B * p) ** 2 / (B * p)).sum()
    assert chi < 60


def test_captured_and_replayed_beside_another_stream(kdt):
    import torch
    d = _inputs(14, 4, 20, 20000, "bf16")
    t = [torch.from_numpy(d[k]).cuda() for k in ("parent", "tok", "u", "ub")]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = kdt.tree_sample(t[0], t[1], d["logits"], t[2], t[3])
    for k in range(3):
        rng = np.random.RandomState(k)
        d["u"], d["ub"] = rng.rand(4, 20).astype(np.float32), rng.rand(4).astype(np.float32)
        t[2].copy_(torch.from_numpy(d["u"])), t[3].copy_(torch.from_numpy(d["ub"]))
        torch.cuda.synchronize()
        other = kdt.tree_sample(t[0], t[1], d["logits"], t[2], t[3])
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        _check(d, [x.cpu().numpy() for x in out] + [0])
        assert all(torch.equal(a, b) for a, b in zip(out, other))


@pytest.mark.parametrize("dtype,B,temp", [("f32", 80, 1.0), ("bf16", 80, 0.3), ("f32", 2, 1.7)])
def test_the_largest_vocabulary_in_a_large_batch(kdt, dtype, B, temp):
    """524288 tokens with one CTA a sequence (and eight): the longest float32 sums there are. Many weights
    of one size, so that their roundings count; a child's test just on either side of its border, from
    within the fast sums' error to beyond the margin; and log-probabilities within the stated bounds."""
    import torch
    V, T = 524288, 2
    d = _inputs(21, B, T, V, dtype, agree=1.0)
    d["logits"] = d["logits"] * 0.2 + 1.0                    # of T rows each the first matters for the test
    d["logits"][:, :, 5] = 9.0
    d["parent"][:, 1], d["temp"] = 0, temp
    for b in range(B):
        d["logits"][b, 0, d["tok"][b, 1]] = 11.0 + 0.01 * (b % 7)
        w = oq.sample_weights(d["logits"][b, 0].double().cpu().numpy(), temp)
        off = [1e-7, 3e-6, 1e-5, 2e-5, 5e-5, 1e-3][b % 6] * (1 if b % 2 else -1)
        d["u"][b, 1] = np.float32(w[d["tok"][b, 1]] / w.sum() * (1 + off))
    got = _run(kdt, d)
    assert got[4] == 0 and 0.2 * B < (got[1] == 2).sum() < 0.8 * B
    for b in range(B):
        path, want, lp = oq.tree_sample(d["parent"][b], d["tok"][b], lambda i: d["logits"][b, i].double().cpu().numpy(),
                                        d["u"][b].astype(np.float64), float(d["ub"][b]), temp)
        n = got[1][b]
        assert got[0][b, :n].tolist() == path and got[2][b] == want
        off = np.abs(got[3][b, :n] - lp)
        assert (off[:-1] <= 2e-5 + 2.0 ** -23 * np.abs(lp[:-1])).all() and off[-1] <= 3e-7 + 2.0 ** -23 * abs(lp[-1]), (b, off)
