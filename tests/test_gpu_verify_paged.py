"""GPU parity of kdt_verify_attn_paged against the float64 oracle (oracle/q8.py's attention) on the rows the
table names, at the sizes and masks where it can go wrong.

Tolerances. Scores: n = 576 products summed in float32, off by at most ds = n 2^-24 scale sum|q||c| (with the largest
such sum of the case), times ln 2 log2 e = 1 through the exponent. Weights: 2^(+-ds) from the scores, 2^-21 from the
exponential and the two float32 products around it, 2^-8 from the rounding to bf16, so an output is off by at most
(2^-8 + 2 ds + 2^-20) sum_j p_j |c_j|, then rounded to its type (2^-8 or 2^-24 of its value); splits add one rounding of
2^-22. lse: ds, the sum's roundings (at most N / 32 + 24 adds in a row) and 2^-20 for the logarithm's and the reference's
products, relative to 1 + |lse|.
"""
import numpy as np
import pytest

from oracle import paged as op
from oracle import q8 as oq

pytestmark = pytest.mark.gpu
SCALE = 1.0 / np.sqrt(192.0)


@pytest.fixture(scope="module")
def kdt():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_tree_absorb_gb300 import build_lib
    build_lib.build()
    import speculative_decoding_tree_absorb_gb300 as k
    return k


def _inputs(seed, T, H, prefix, page=64, spare=3, amp=1.0, n=None):
    """Queries, random trees, and a cache whose rows are NaN wherever no sequence has a row; table entries behind a
    sequence's pages are no pages at all."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.RandomState(seed)
    B = len(prefix)
    n = [T] * B if n is None else n
    held = [-(-(p + k) // page) if k else 0 for p, k in zip(prefix, n)]
    n_pages, W = sum(held) + spare, max(-(-(max(prefix) + T) // page), 1)
    ids = rng.permutation(n_pages).astype(np.int32)
    table = rng.choice([-1, -(2 ** 31), 2 ** 31 - 1, n_pages], (B, W)).astype(np.int32)
    c = torch.full((n_pages, page, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    k = torch.full((n_pages, page, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    at, rows = 0, []
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
        N = prefix[b] + n[b] if n[b] else 0
        r = op.rows_of(table[b], N, page)
        rows.append(r)
        i = torch.from_numpy(r).cuda()
        c.view(-1, 512)[i] = torch.randn(N, 512, device="cuda", generator=g).to(torch.bfloat16)
        k.view(-1, 64)[i] = torch.randn(N, 64, device="cuda", generator=g).to(torch.bfloat16)
    q = (torch.randn(B, T, H, 576, device="cuda", generator=g) * amp).to(torch.bfloat16)
    parent = np.full((B, T), -1, dtype=np.int32)
    for b in range(B):
        for i in range(1, T):
            parent[b, i] = rng.randint(max(0, i - 8), i)
    return dict(q=q, c=c, k=k, table=table, parent=parent, prefix=list(prefix), T=T, H=H, B=B, page=page, rows=rows, n=n)


def _bits(see, T):
    import torch
    bits = np.zeros(see.shape[:2] + ((T + 31) // 32,), dtype=np.uint32)
    for t in range(T):
        bits[..., t // 32] |= see[..., t].astype(np.uint32) << np.uint32(t % 32)
    return torch.from_numpy(bits.view(np.int32)).cuda()


def _args(d):
    import torch
    return (d["q"][..., :512], d["q"][..., 512:], d["c"], d["k"], torch.from_numpy(d["table"]).cuda(),
            torch.tensor(d["prefix"], dtype=torch.int32, device="cuda"))


def _call(kdt, d, see=None, want_err=0, **kw):
    import torch
    err = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    if see is not None:
        kw["vis"] = _bits(see, d["T"])
    elif d["T"] > 1 or kw.pop("with_parent", False):
        kw["parent"] = torch.from_numpy(d["parent"]).cuda()
    kw.setdefault("max_kv_len", max(d["prefix"]) + d["T"])
    out, lse = kdt.verify_attn_paged(*_args(d), scale=SCALE, err=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == want_err
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def _check(d, got, out_eps, see=None, nodes=None):
    """Against the oracle, for all nodes or some (the others' rows are then only required to be finite)."""
    out, lse = got
    for b, P in enumerate(d["prefix"]):
        n = d["n"][b]
        if n == 0:
            continue
        c = d["c"].view(-1, 512)[d["rows"][b]].double().cpu().numpy()
        k = d["k"].view(-1, 64)[d["rows"][b]].double().cpu().numpy()
        some = list(range(n)) if nodes is None else [i for i in nodes if i < n]
        if nodes is not None:
            assert np.isfinite(out[b, :n]).all()
        q = d["q"][b, some].double().cpu().numpy()
        sb = (oq.ancestors(d["parent"][b]) if see is None else see[b])[some][:, :n]
        ref_o, ref_l = oq.attention(q, c, k, P, sb, SCALE)
        for m, i in enumerate(some):
            keys = np.concatenate([np.arange(P), P + np.flatnonzero(sb[m])])
            if not len(keys):
                assert (out[b, i] == 0).all() and (lse[b, i] == -np.inf).all()
                continue
            kc = np.concatenate([c[keys], k[keys]], -1)
            p = np.exp(SCALE * (q[m] @ kc.T) - ref_l[m][:, None])
            ds = 576 * 2.0 ** -24 * abs(SCALE) * (np.abs(q[m]) @ np.abs(kc).T).max()
            tol = (2.0 ** -8 + 2 * ds + 2.0 ** -20) * (p @ np.abs(c[keys])) + (out_eps + 2.0 ** -22) * np.abs(ref_o[m])
            assert (np.abs(out[b, i] - ref_o[m]) <= tol).all(), (b, i, np.abs(out[b, i] - ref_o[m]).max())
            tol = ds + (2.0 ** -20 + (len(keys) / 32 + 24) * 2.0 ** -24) * (1 + np.abs(ref_l[m]))
            assert (np.abs(lse[b, i] - ref_l[m]) <= tol).all(), (b, i, np.abs(lse[b, i] - ref_l[m]).max())


CASES = [(1, 1, [0]), (1, 64, [0, 1, 62, 63, 64, 65, 1000]), (1, 16, [700]), (9, 8, [37, 37]), (5, 20, [300, 11, 2000]),
         (33, 3, [65, 600]), (64, 64, [200]), (70, 1, [130, 0]), (1, 128, [9000]), (2, 1024, [70]), (13, 32, [1500, 77]),
         (1, 200, [500, 3]), (3, 40, [127, 128])]


@pytest.mark.parametrize("splits", [0, 1, 3, 50])
@pytest.mark.parametrize("T,H,prefix", CASES)
def test_parity(kdt, T, H, prefix, splits):
    import torch
    d = _inputs(T * 100 + H, T, H, prefix, page=[8, 16, 32, 64, 128, 1024][(T + H + splits) % 6])
    bf16 = (T + H + splits) % 2 == 0
    got = _call(kdt, d, num_splits=splits, out_dtype=torch.bfloat16 if bf16 else torch.float32)
    _check(d, got, 2.0 ** -8 if bf16 else 2.0 ** -24)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 512, 1024])
@pytest.mark.parametrize("T,H", [(1, 64), (20, 4)])
def test_page_sizes(kdt, page, T, H):
    """Lengths that end at every kind of place in a page, and in a block of keys."""
    d = _inputs(page + T, T, H, [0, 7, 8, page - T if page > T else 9, page, page + 1, 3 * page + 5, 1023, 1024, 1025], page=page)
    _check(d, _call(kdt, d), 2.0 ** -24)
    _check(d, _call(kdt, d, num_splits=7), 2.0 ** -24)


@pytest.mark.parametrize("splits", [0, 1, 2, 5])
@pytest.mark.parametrize("T,H,n", [(1, 64, [1, 0, 1, 0, 0]), (7, 20, [7, 3, 0, 1, 5]), (40, 8, [0, 40, 33, 1, 0]), (40, 8, [0] * 5)])
def test_padded_batches(kdt, T, H, n, splits):
    """Rows behind a sequence's nodes, and sequences that are not there, are left as they were."""
    import torch
    d = _inputs(T, T, H, [200, 1000, 64, 0, 300], n=n)
    out = torch.full((5, T, H, 512), 3.0, device="cuda")
    lse = torch.full((5, T, H), -4.0, device="cuda")
    got = _call(kdt, d, n_rows=torch.tensor(n, dtype=torch.int32, device="cuda"), out=out, lse=lse, num_splits=splits)
    _check(d, got, 2.0 ** -24)
    for b in range(5):
        assert (got[0][b, n[b]:] == 3.0).all() and (got[1][b, n[b]:] == -4.0).all()


def test_caller_bits_and_rows_that_see_nothing(kdt):
    d = _inputs(11, 40, 6, [0, 0, 130])
    rng = np.random.RandomState(3)
    see = rng.rand(3, 40, 40) < 0.3
    see[0, 5] = see[1] = see[0, 39] = False
    for splits in (0, 1, 3):
        _check(d, _call(kdt, d, see=see, num_splits=splits), 2.0 ** -24, see=see)
    d = _inputs(12, 1, 16, [0, 5, 64])
    no = np.zeros((3, 1, 1), dtype=bool)
    _check(d, _call(kdt, d, see=no), 2.0 ** -24, see=no)


def test_one_row_with_and_without_its_parent(kdt):
    d = _inputs(13, 1, 32, [0, 64, 200])
    a, b = _call(kdt, d), _call(kdt, d, with_parent=True)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("T,H", [(12, 4), (64, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_reaches_only_the_rows_that_see_it(kdt, T, H, bad):
    """NaN or infinity in a tree node's latent, and in another's rope key: rows that see neither are bit for bit as
    without them; no row that sees the latent stays finite throughout."""
    d = _inputs(21, T, H, [300, 64])
    clean = _call(kdt, d)
    d["c"].view(-1, 512)[d["rows"][0][300 + 5], 130] = bad
    d["k"].view(-1, 64)[d["rows"][1][64 + 3], 7] = bad
    out, lse = _call(kdt, d)
    for b, t in ((0, 5), (1, 3)):
        sees = oq.ancestors(d["parent"][b])[:, t]
        assert sees.any() and not sees.all()
        assert np.array_equal(out[b, ~sees], clean[0][b, ~sees]) and np.array_equal(lse[b, ~sees], clean[1][b, ~sees])
        if b == 0:
            assert not np.isfinite(out[b, sees]).all(-1).any()
        else:                                       # scores of +-inf (or NaN): -inf has weight 0
            s = d["q"][b, :, :, 512 + 7].double().cpu().numpy()[sees] * bad
            up = ~(s < 0)
            assert np.isnan(out[b, sees][up]).all() and np.isfinite(out[b, sees][~up]).all()
    d["c"].view(-1, 512)[d["rows"][0][7], 0] = float("nan")      # in the prefix: every row sees it
    out, lse = _call(kdt, d)
    assert np.isnan(out[0]).any(-1).all() and np.isnan(lse[0]).all()


def test_outlier_keys_raise_the_reference(kdt):
    """Keys far larger than the rest, late in the sequence, in several blocks: the running reference rises block after
    block and old sums are rescaled."""
    d = _inputs(31, 3, 64, [1500, 700], amp=3.0)
    for b, P in enumerate(d["prefix"]):
        for k, j in enumerate(range(100, P, 190)):
            d["c"].view(-1, 512)[d["rows"][b][j]] *= 2.0 ** (k % 4)
    _check(d, _call(kdt, d, num_splits=1), 2.0 ** -24)
    _check(d, _call(kdt, d), 2.0 ** -24)


def _scored_minus_inf(d, keys):
    """Infinite rope values at these rows of every sequence, against queries that are all negative there."""
    d["q"][..., 512 + 3] = -(d["q"][..., 512 + 3].abs() + 0.5)
    for r in d["rows"]:
        d["k"].view(-1, 64)[r[list(keys)], 3] = float("inf")


def _without(d, keys):
    """What the oracle sees of the same problem without these prefix rows."""
    gone = set(keys)
    return dict(d, rows=[np.array([x for j, x in enumerate(r) if j not in gone], dtype=np.int64) for r in d["rows"]],
                prefix=[p - len(gone) for p in d["prefix"]])


# prefix, rows that score -inf: all of the first block, of the first two, of the last whole ones, all but one row
MINUS_INF = [(191, range(0, 64)), (383, range(0, 128)), (384, range(0, 129)), (700, range(130, 700)), (640, range(1, 640))]


@pytest.mark.parametrize("splits", [0, 1, 2, 5])
@pytest.mark.parametrize("T,H", [(1, 4), (9, 8), (40, 8)])
@pytest.mark.parametrize("prefix,keys", MINUS_INF)
def test_blocks_that_score_minus_inf_have_weight_0(kdt, prefix, keys, T, H, splits):
    d = _inputs(91, T, H, [prefix])
    _scored_minus_inf(d, keys)
    _check(_without(d, keys), _call(kdt, d, num_splits=splits), 2.0 ** -24)


@pytest.mark.parametrize("splits", [0, 1, 2])
def test_nothing_but_minus_inf(kdt, splits):
    no = np.zeros((1, 1, 1), dtype=bool)
    for prefix in (0, 128, 383):
        d = _inputs(93, 1, 4, [prefix])
        _scored_minus_inf(d, range(prefix + 1))
        got = _call(kdt, d, num_splits=splits)
        assert (got[0] == 0).all() and (got[1] == -np.inf).all()
    d["k"].view(-1, 64)[d["rows"][0][200], 5] = float("nan")       # a NaN among them is not lost
    out, lse = _call(kdt, d, num_splits=splits)
    assert np.isnan(out).all() and np.isnan(lse).all()


@pytest.mark.parametrize("T,H", [(1, 64), (9, 16)])
def test_sequences_that_share_pages(kdt, T, H):
    """A common prefix in the same pages, and a page that one sequence names twice."""
    d = _inputs(61, T, H, [200, 150, 200, 129], page=16)
    for b in range(1, 4):
        d["table"][b, :8] = d["table"][0, :8]
        d["rows"][b][:128] = d["rows"][0][:128]
    d["table"][2, 5] = d["table"][2, 2]
    d["rows"][2][80:96] = d["rows"][2][32:48]
    _check(d, _call(kdt, d), 2.0 ** -24)


def test_pages_that_are_none(kdt):
    """An entry outside the cache among those a sequence needs: named, its rows read as zeros, the others untouched."""
    import torch
    d = _inputs(41, 1, 16, [500, 100, 640], page=32)
    clean = _call(kdt, d)
    for bad in (-1, -(2 ** 31), d["c"].shape[0], 2 ** 31 - 1):
        e = dict(d, table=d["table"].copy())
        e["table"][2, 3] = bad
        out, lse = _call(kdt, e, want_err=1 + 3 + 2)
        assert np.array_equal(out[:2], clean[0][:2]) and np.array_equal(lse[:2], clean[1][:2])
        z = dict(d, c=d["c"].clone(), k=d["k"].clone())
        z["c"][int(d["table"][2, 3])] = 0
        z["k"][int(d["table"][2, 3])] = 0
        want = _call(kdt, z)
        assert np.array_equal(out, want[0]) and np.array_equal(lse, want[1])
    e["table"][1, 0] = -1
    _call(kdt, e, want_err=1 + 3 + 1)


@pytest.mark.parametrize("T", [9, 32, 33])
def test_malformed_parents_are_recorded(kdt, T):
    d = _inputs(72, T, 4, [10, 0, 130])
    good = dict(d, parent=d["parent"].copy())
    d["parent"][1, 4], d["parent"][2, 6] = 4, -2            # its own parent; below -1
    good["parent"][1, 4] = good["parent"][2, 6] = -1        # a walk ends there
    a, b = _call(kdt, d, want_err=T + 4 + 1), _call(kdt, good)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_lengths_outside_the_bound_are_brought_into_it(kdt):
    import torch
    d = _inputs(73, 2, 8, [100, 100])
    par = torch.from_numpy(d["parent"]).cuda()
    a = list(_args(d))
    want = kdt.verify_attn_paged(*a, parent=par, max_kv_len=102)
    low = kdt.verify_attn_paged(*a[:5], torch.tensor([0, 0], dtype=torch.int32, device="cuda"), parent=par, max_kv_len=102)
    for pre, w in ((torch.tensor([2 ** 31 - 1, 101]), want), (torch.tensor([-5, -(2 ** 31)]), low)):
        got = kdt.verify_attn_paged(*a[:5], pre.to(torch.int32).cuda(), parent=par, max_kv_len=102)
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])


@pytest.mark.parametrize("T,H,prefix", [(1, 64, [3000, 5]), (20, 64, [700, 1300]), (1, 16, [200, 9])])
def test_captured_graph_two_streams_and_fresh_inputs(kdt, T, H, prefix):
    """Two calls captured on two streams with workspaces of their own, replayed on rewritten inputs and lengths; results
    as from plain calls, bit for bit."""
    import torch
    d = [_inputs(61 + k, T, H, prefix) for k in (0, 1)]
    N = max(prefix) + T
    need = kdt.verify_attn_paged_workspace_size(2, T, H, N, 64)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in d]
    outs = [torch.empty(2, T, H, 512, device="cuda") for _ in d]
    lses = [torch.empty(2, T, H, device="cuda") for _ in d]
    args = [_args(x) for x in d]
    par = [torch.from_numpy(x["parent"]).cuda() for x in d]

    def call(k, out, lse, w):
        kdt.verify_attn_paged(*args[k], parent=par[k] if T > 1 else None, max_kv_len=N, scale=SCALE, out=out, lse=lse, workspace=w)

    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=a):
        b.wait_stream(a)
        call(0, outs[0], lses[0], ws[0])
        with torch.cuda.stream(b):
            call(1, outs[1], lses[1], ws[1])
        a.wait_stream(b)
    for seed in (1, 2, 3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for k, x in enumerate(d):
            x["q"].copy_(torch.randn(x["q"].shape, device="cuda", generator=g).to(torch.bfloat16))
            args[k][5].copy_(torch.tensor([p // seed for p in prefix]))
        for w in ws:
            w.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for k in (0, 1):
            o, l = torch.empty_like(outs[k]), torch.empty_like(lses[k])
            call(k, o, l, torch.empty_like(ws[k]))
            torch.cuda.synchronize()
            assert torch.equal(o, outs[k]) and torch.equal(l, lses[k])


@pytest.mark.parametrize("T,H", [(1, 4), (1, 128), (6, 50)])
def test_more_sequences_than_sms(kdt, T, H):
    rng = np.random.RandomState(3)
    d = _inputs(82, T, H, [int(x) for x in rng.randint(0, 300, 170)], page=16)
    _check(d, _call(kdt, d), 2.0 ** -24)


def test_pages_beyond_32_bits_of_offset(kdt):
    """Cache rows whose byte offsets pass 2^32, and a table row far from its neighbour."""
    import torch
    d = _inputs(81, 1, 16, [0, 3, 260], page=64)
    n_big = 70000                                            # 4.6 GB of latents
    c = torch.zeros(n_big, 64, 512, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(n_big, 64, 64, dtype=torch.bfloat16, device="cuda")
    shift = n_big - d["c"].shape[0]
    c[shift:], k[shift:] = d["c"], d["k"]
    d["table"] = np.where((d["table"] >= 0) & (d["table"] < d["c"].shape[0]), d["table"] + shift, -1).astype(np.int32)
    d.update(c=c, k=k, rows=[r + shift * 64 for r in d["rows"]])
    wide = torch.full((3, 1 << 16), -1, dtype=torch.int32, device="cuda")
    W = d["table"].shape[1]
    wide[:, 5:5 + W] = torch.from_numpy(d["table"]).cuda()
    a = list(_args(d))
    out, lse = kdt.verify_attn_paged(*a[:4], wide[:, 5:5 + W], a[5], max_kv_len=261, scale=SCALE)
    _check(d, (out.double().cpu().numpy(), lse.double().cpu().numpy()), 2.0 ** -24)


@pytest.mark.parametrize("T,H,prefix", [(1, 64, [0, 1, 5]), (9, 8, [130, 3, 0, 300]), (40, 20, [70])])
@pytest.mark.parametrize("splits", [0, 700])
def test_a_bound_far_above_the_lengths(kdt, T, H, prefix, splits):
    """max_kv_len left at the table's width: the split is planned for many more blocks than there are."""
    d = _inputs(98, T, H, prefix)
    W = d["table"].shape[1]
    d["table"] = np.concatenate([d["table"], np.full((len(prefix), 500), -1, dtype=np.int32)], 1)
    _check(d, _call(kdt, d, max_kv_len=None, num_splits=splits), 2.0 ** -24)
    assert d["table"].shape[1] == W + 500


@pytest.mark.parametrize("scale", [0.0, -0.05, 2.0])
def test_other_scales(kdt, scale, monkeypatch):
    import sys
    d = _inputs(99, 20, 8, [300, 2], amp=0.25)
    for splits in (0, 1):
        monkeypatch.setattr(sys.modules[__name__], "SCALE", scale)
        got = _call(kdt, d, num_splits=splits)
        _check(d, got, 2.0 ** -24)


def test_queries_far_apart(kdt):
    """Query rows 2048 elements apart, NaN between them."""
    import torch
    d = _inputs(100, 7, 12, [400, 130], spare=0)
    wide = torch.full((2, 7, 12, 2048), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[..., 64:640] = d["q"]
    d["q"] = wide[..., 64:640]
    _check(d, _call(kdt, d), 2.0 ** -24)


def test_queries_that_are_not_finite_stay_in_their_rows(kdt):
    d = _inputs(102, 3, 20, [300, 64])
    clean = _call(kdt, d)
    d["q"][0, 1, 7, 5], d["q"][1, 2, 19, 570] = float("nan"), float("inf")
    out, lse = _call(kdt, d)
    hit = np.zeros((2, 3, 20), dtype=bool)
    hit[0, 1, 7] = hit[1, 2, 19] = True
    assert np.array_equal(out[~hit], clean[0][~hit]) and np.array_equal(lse[~hit], clean[1][~hit])
    assert np.isnan(out[hit]).all()


WIDE = [(127, 3, [1, 300]), (128, 2, [0, 128]), (129, 5, [64, 70]), (513, 1, [127, 0]), (1000, 3, [90]), (2500, 1, [5, 200]),
        (4096, 2, [130])]


def _some_nodes(T, n=24):
    edge = [i + e for i in range(0, T, 64) for e in (-1, 0, 1, 31, 32)]
    pick = np.random.RandomState(T).choice(T, min(T, n), replace=False).tolist()
    return sorted({i for i in [T - 2] + edge[:15] + edge[-10:] + pick + [T - 1] if 0 <= i < T})


@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("kind", ["random", "chain"])
@pytest.mark.parametrize("T,H,prefix", WIDE)
def test_wide_trees_and_prompt_chunks(kdt, T, H, prefix, kind, splits):
    d = _inputs(T, T, H, prefix, page=32)
    if kind == "chain":
        d["parent"] = np.tile(np.arange(T, dtype=np.int32) - 1, (len(prefix), 1))
    _check(d, _call(kdt, d, num_splits=splits), 2.0 ** -24, nodes=_some_nodes(T))


@pytest.mark.parametrize("T,H", [(161, 3), (1030, 2)])
def test_wide_caller_bits(kdt, T, H):
    d = _inputs(T + 1, T, H, [0, 70])
    rng = np.random.RandomState(T)
    see = rng.rand(2, T, T) < 0.02
    see[0, ::7] = False
    see[0, 3, T - 1] = see[1, 5, T - 33] = True
    _check(d, _call(kdt, d, see=see), 2.0 ** -24, see=see, nodes=_some_nodes(T))


def test_each_call_sees_its_own_tree(kdt):
    """Calls in a row on one workspace with two trees in turn."""
    import torch
    T, H = 64, 8
    d = _inputs(96, T, H, [40, 3, 300])
    chain = np.tile(np.arange(T, dtype=np.int32) - 1, (3, 1))
    par = [torch.from_numpy(x).cuda() for x in (d["parent"], chain)]
    ws = torch.empty(kdt.verify_attn_paged_workspace_size(3, T, H, 300 + T, 64), dtype=torch.uint8, device="cuda")
    args = _args(d)
    outs = [kdt.verify_attn_paged(*args, parent=par[k % 2], max_kv_len=300 + T, workspace=ws, scale=SCALE) for k in range(30)]
    torch.cuda.synchronize()
    for k, tree in enumerate((d["parent"], chain)):
        _check(dict(d, parent=tree), [x.double().cpu().numpy() for x in outs[k]], 2.0 ** -24)
    for k in range(2, 30):
        assert torch.equal(outs[k][0], outs[k % 2][0]) and torch.equal(outs[k][1], outs[k % 2][1])


@pytest.mark.parametrize("T,H,prefix", [(1, 64, [900, 2100, 1500, 77]), (9, 128, [4000, 12])])
def test_runs_repeat_their_bits(kdt, T, H, prefix):
    """In every one of many runs, alone and with other work on the device, the result is the same bit for bit."""
    import torch
    d = _inputs(95, T, H, prefix)
    par = torch.from_numpy(d["parent"]).cuda() if T > 1 else None
    args = _args(d)
    out, lse = kdt.verify_attn_paged(*args, parent=par, max_kv_len=max(prefix) + T)
    side, junk = torch.cuda.Stream(), torch.empty(1 << 26, device="cuda")
    for k in range(60):
        if k % 2:
            with torch.cuda.stream(side):
                junk.add_(1.0)
        o, l = kdt.verify_attn_paged(*args, parent=par, max_kv_len=max(prefix) + T)
        assert torch.equal(o, out) and torch.equal(l, lse), k
    torch.cuda.synchronize()


def test_a_busy_side_stream_keeps_its_workspace_and_outputs(kdt):
    """A call queued on a stream that is still busy: what the call allocated is not handed out before it has run."""
    import torch
    T, H, prefix = 40, 16, [3000, 700]
    d = _inputs(97, T, H, prefix)
    want = _call(kdt, d)
    par = torch.from_numpy(d["parent"]).cuda()
    args = _args(d)
    need = kdt.verify_attn_paged_workspace_size(2, T, H, max(prefix) + T, 64)
    side, a = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):
            a = (a @ a).clamp_(-1, 1)
    out, lse = kdt.verify_attn_paged(*args, parent=par, scale=SCALE, max_kv_len=max(prefix) + T, stream=side)
    junk = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), want[0]) and np.array_equal(lse.double().cpu().numpy(), want[1])
    del junk


def test_same_as_the_dense_cache(kdt):
    """On the same rows in a dense cache kdt_verify_attn gives the same within both bounds."""
    import torch
    d = _inputs(51, 16, 64, [500, 900])
    out, lse = _call(kdt, d)
    L = 916
    c, k = torch.zeros(2, L, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, L, 64, dtype=torch.bfloat16, device="cuda")
    for b, r in enumerate(d["rows"]):
        c[b, :len(r)], k[b, :len(r)] = d["c"].view(-1, 512)[r], d["k"].view(-1, 64)[r]
    q = d["q"]
    o2, l2 = kdt.verify_attn(q[..., :512], q[..., 512:], c, k, torch.tensor(d["prefix"], dtype=torch.int32, device="cuda"),
                             parent=torch.from_numpy(d["parent"]).cuda(), max_kv_len=L, scale=SCALE)
    assert np.abs(out - o2.double().cpu().numpy()).max() <= 2 * 2e-2
    assert np.abs(lse - l2.double().cpu().numpy()).max() <= 1e-3


def test_not_device_memory_is_refused(kdt):
    import torch
    d = _inputs(71, 33, 8, [10])            # a tree whose visibility takes a workspace
    par = torch.from_numpy(d["parent"]).cuda()
    a = list(_args(d))
    with pytest.raises(kdt.KdtError) as e:
        kdt.verify_attn_paged(*a[:4], torch.from_numpy(d["table"]).pin_memory(), a[5], parent=par)
    assert e.value.status == 6
    with pytest.raises(kdt.KdtError) as e:
        kdt.verify_attn_paged(*a, parent=par, max_kv_len=43, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")[128:])
    assert e.value.status == 4


@pytest.mark.parametrize("captured", [False, True])
def test_a_batch_without_nodes_ends_behind_its_visibility(kdt, captured):
    """Where n_rows leaves every sequence without a node the attention reads no visibility word; the call still ends only
    once the words' kernel has: what it reports of the parents (in a chain of 4096, from its last walks) is there for what
    follows on the stream. Rows of out and lse are left as they were."""
    import torch
    B, T, H = 3, 4096, 1
    d = _inputs(91, 1, H, [5] * B)
    i32 = dict(dtype=torch.int32, device="cuda")
    parent = torch.arange(-1, T - 1, **i32).repeat(B, 1)
    parent[1, T - 1] = T - 1
    q = torch.zeros(B, T, H, 576, dtype=torch.bfloat16, device="cuda")
    table, prefix, none = torch.zeros(B, 65, **i32), torch.zeros(B, **i32), torch.zeros(B, **i32)
    out, lse = torch.full((B, T, H, 512), 3.0, device="cuda"), torch.full((B, T, H), 4.0, device="cuda")
    err = torch.zeros(1, **i32)
    ws = torch.empty(kdt.verify_attn_paged_workspace_size(B, T, H, 65 * 64, 64), dtype=torch.uint8, device="cuda")

    def call():
        kdt.verify_attn_paged(q[..., :512], q[..., 512:], d["c"], d["k"], table, prefix, n_rows=none, parent=parent, out=out,
                              lse=lse, err=err, workspace=ws)
        return err.clone()
    call()
    torch.cuda.synchronize()
    if captured:
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=s):
            seen = [call() for _ in range(3)]
        graph.replay()
    else:
        seen = [call() for _ in range(3)]
    torch.cuda.synchronize()
    assert [int(e.item()) for e in seen] == [2 * T] * 3
    assert (out == 3.0).all() and (lse == 4.0).all()


@pytest.mark.parametrize("splits", [29, 30, 31, 32, 33, 48, 64])
@pytest.mark.parametrize("T,H", [(1, 64), (3, 30)])
def test_both_joins_where_they_meet(kdt, T, H, splits):
    """Two groups in shares on both sides of the number that decides how their pieces are joined."""
    d = _inputs(T + splits, T, H, [4000, 3100])
    _check(d, _call(kdt, d, num_splits=splits), 2.0 ** -24)
