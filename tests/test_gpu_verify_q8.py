"""GPU parity of kdt_verify_attn_q8 against the float64 oracle (oracle/q8.py) on the cache's own
values, at the sizes and masks where it can go wrong.

Tolerances. Scores: n = 576 products summed in float32, off by at most ds = n 2^-24 scale
sum|q||c| (with the largest such sum of the case) -- times ln 2 log2 e = 1 through the
exponent. Weights: 2^(+-ds) from the scores, 2^-21 from the exponential and the two float32
products around it, 2^-8 from the rounding to bf16, so an output is off by at most
(2^-8 + 2 ds + 2^-20) sum_j p_j |c_j|, then rounded to its type (2^-8 or 2^-24 of its value);
splits add one rounding of 2^-22. lse: ds, the sum's roundings (at most N / 128 + 12 adds
in a row) and 2^-20 for the logarithm's and the reference's products, relative to 1 + |lse|.
"""
import numpy as np
import pytest

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


def _inputs(seed, T, H, prefix, pad=5, amp=1.0):
    """Queries, a cache written by quantising random rows, and random trees; rows behind the
    last tree row hold NaN scales and NaN rope keys."""
    import torch
    import speculative_decoding_tree_absorb_gb300 as kdt
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, L = len(prefix), max(prefix) + T + pad
    c8 = torch.full((B, L, 512), 0x33, dtype=torch.uint8, device="cuda")
    sc = torch.full((B, L, 16), 255, dtype=torch.uint8, device="cuda")
    kp = torch.full((B, L, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    n = torch.tensor([p + T for p in prefix], dtype=torch.int32, device="cuda")
    kv = torch.randn(B, max(prefix) + T, 576, device="cuda", generator=g)
    kdt.latent_write_q8(kv[..., :512], kv[..., 512:], c8, sc, kp, torch.zeros(B, dtype=torch.int32, device="cuda"), n_rows=n)
    q = (torch.randn(B, T, H, 576, device="cuda", generator=g) * amp).to(torch.bfloat16)
    rng = np.random.RandomState(seed)
    parent = np.full((B, T), -1, dtype=np.int32)
    for b in range(B):
        for i in range(1, T):
            parent[b, i] = rng.randint(max(0, i - 8), i)
    return dict(q=q, c8=c8, sc=sc, kp=kp, parent=parent, prefix=list(prefix), T=T, H=H, B=B, L=L)


def _call(kdt, d, see=None, **kw):
    import torch
    pre = torch.tensor(d["prefix"], dtype=torch.int32, device="cuda")
    err = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    if see is None:
        kw["parent"] = torch.from_numpy(d["parent"]).cuda()
    else:
        W = (d["T"] + 31) // 32
        bits = np.zeros(see.shape[:2] + (W,), dtype=np.uint32)
        for t in range(d["T"]):
            bits[..., t // 32] |= see[..., t].astype(np.uint32) << np.uint32(t % 32)
        kw["vis"] = torch.from_numpy(bits.view(np.int32)).cuda()
    out, lse = kdt.verify_attn_q8(d["q"][..., :512], d["q"][..., 512:], d["c8"], d["sc"], d["kp"], pre, scale=SCALE,
                                  err=err, max_kv_len=max(d["prefix"]) + d["T"], **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def _check(d, got, out_eps, see=None):
    out, lse = got
    for b, P in enumerate(d["prefix"]):
        N = P + d["T"]
        c = oq.dequantise(d["c8"][b, :N].cpu().numpy(), d["sc"][b, :N].cpu().numpy())
        k = d["kp"][b, :N].double().cpu().numpy()
        q = d["q"][b].double().cpu().numpy()
        sb = oq.ancestors(d["parent"][b]) if see is None else see[b]
        ref_o, ref_l = oq.attention(q, c, k, P, sb, SCALE)
        # sum_j p_j |c_j|, with the same weights
        for i in range(d["T"]):
            keys = np.concatenate([np.arange(P), P + np.flatnonzero(sb[i])])
            if not len(keys):
                assert (out[b, i] == 0).all() and (lse[b, i] == -np.inf).all()
                continue
            kc = np.concatenate([c[keys], k[keys]], -1)
            s = SCALE * (q[i] @ kc.T)
            p = np.exp(s - ref_l[i][:, None])
            mag = p @ np.abs(c[keys])
            ds = 576 * 2.0 ** -24 * SCALE * (np.abs(q[i]) @ np.abs(kc).T).max()
            tol = (2.0 ** -8 + 2 * ds + 2.0 ** -20) * mag + (out_eps + 2.0 ** -22) * np.abs(ref_o[i])
            assert (np.abs(out[b, i] - ref_o[i]) <= tol).all(), (b, i, np.abs(out[b, i] - ref_o[i]).max())
            tol = ds + (2.0 ** -20 + (len(keys) / 128 + 12) * 2.0 ** -24) * (1 + np.abs(ref_l[i]))
            assert (np.abs(lse[b, i] - ref_l[i]) <= tol).all(), (b, i, np.abs(lse[b, i] - ref_l[i]).max())


CASES = [(1, 1, [0]), (1, 64, [0, 1, 126, 127, 128, 129, 1000]), (9, 8, [37, 37]), (5, 20, [300, 11, 2000]),
         (33, 3, [65, 600]), (64, 64, [200]), (70, 1, [130, 0]), (1, 128, [9000]), (2, 1024, [70])]


@pytest.mark.parametrize("impl,splits", [("auto", 0), ("q8_rows", 0), ("q8_rows", 1), ("q8_rows", 5), ("tcgen05", 0),
                                         ("tcgen05", 1), ("tcgen05", 3)])
@pytest.mark.parametrize("T,H,prefix", CASES)
def test_parity(kdt, T, H, prefix, impl, splits):
    import torch
    d = _inputs(T * 100 + H, T, H, prefix)
    bf16 = (T + H + splits) % 2 == 0
    got = _call(kdt, d, impl=impl, num_splits=splits, out_dtype=torch.bfloat16 if bf16 else torch.float32)
    _check(d, got, 2.0 ** -8 if bf16 else 2.0 ** -24)


@pytest.mark.parametrize("impl", ["tcgen05", "q8_rows"])
def test_caller_bits_and_rows_that_see_nothing(kdt, impl):
    d = _inputs(11, 40, 6, [0, 0, 130])
    rng = np.random.RandomState(3)
    see = rng.rand(3, 40, 40) < 0.3
    see[0, 5] = see[1] = see[0, 39] = False
    _check(d, _call(kdt, d, see=see, impl=impl), 2.0 ** -24, see=see)
    _check(d, _call(kdt, d, see=see, impl=impl, num_splits=3), 2.0 ** -24, see=see)


@pytest.mark.parametrize("impl", ["tcgen05", "q8_rows"])
@pytest.mark.parametrize("T,H", [(12, 4), (64, 64)])
def test_nan_reaches_exactly_the_rows_that_see_it(kdt, impl, T, H):
    """NaN in a tree node's codes (its group flagged) and an infinity in another's rope key:
    rows that see neither are bit for bit as without them; rows that see them are NaN."""
    import torch
    d = _inputs(21, T, H, [300, 64])
    clean = _call(kdt, d, impl=impl)
    d["sc"][0, 300 + 5, 2] = 255
    d["kp"][1, 64 + 3, 7] = float("inf")
    out, lse = _call(kdt, d, impl=impl)
    for b, t in ((0, 5), (1, 3)):
        sees = oq.ancestors(d["parent"][b])[:, t]
        assert sees.any() and not sees.all()
        assert np.array_equal(out[b, ~sees], clean[0][b, ~sees]) and np.array_equal(lse[b, ~sees], clean[1][b, ~sees])
        if b == 0:
            assert np.isnan(out[b, sees]).all() and np.isnan(lse[b, sees]).all()
        else:                                       # scores of +-inf (or NaN): no finite answer but -inf scores
            s = d["q"][b, :, :, 512 + 7].double().cpu().numpy()[sees]
            up = s > 0
            assert np.isnan(out[b, sees][up]).all()
    d["sc"][0, 7, 0] = 255                            # in the prefix: every row sees it
    out, lse = _call(kdt, d, impl=impl)
    assert np.isnan(out[0]).all() and np.isnan(lse[0]).all()


@pytest.mark.parametrize("impl", ["tcgen05", "q8_rows"])
def test_outlier_keys_raise_the_reference(kdt, impl):
    """Keys far larger than the rest, late in the sequence, in several blocks: the running
    reference rises block after block and old sums are rescaled."""
    d = _inputs(31, 3, 64, [1500, 700], amp=3.0)
    for b, P in enumerate(d["prefix"]):
        for k, row in enumerate(range(100, P, 190)):
            d["sc"][b, row] += k % 4
    _check(d, _call(kdt, d, impl=impl, num_splits=1), 2.0 ** -24)
    _check(d, _call(kdt, d, impl=impl), 2.0 ** -24)


@pytest.mark.parametrize("impl", ["tcgen05", "q8_rows"])
def test_scales_over_the_whole_range(kdt, impl):
    """Scale bytes from the smallest to above 2^7 (where widening takes a second product)."""
    import torch
    d = _inputs(41, 2, 16, [260], amp=2.0 ** -12)
    g = torch.Generator(device="cuda").manual_seed(2)
    d["sc"][:, :262] = torch.randint(27, 139, (1, 262, 16), device="cuda", generator=g).to(torch.uint8)
    _check(d, _call(kdt, d, impl=impl), 2.0 ** -24)


def test_same_as_the_bf16_cache(kdt):
    """On the rows read back to a bf16 cache kdt_verify_attn gives the same within both bounds."""
    import torch
    d = _inputs(51, 16, 64, [500, 900])
    out, lse = _call(kdt, d)
    pre = torch.tensor(d["prefix"], dtype=torch.int32, device="cuda")
    c, k = kdt.latent_read_q8(d["c8"], d["sc"], d["kp"], None, d["L"])
    q = d["q"]
    o2, l2 = kdt.verify_attn(q[..., :512], q[..., 512:], c, k, pre, parent=torch.from_numpy(d["parent"]).cuda(),
                             max_kv_len=916, scale=SCALE)
    assert np.abs(out - o2.double().cpu().numpy()).max() <= 2 * 2e-2
    assert np.abs(lse - l2.double().cpu().numpy()).max() <= 1e-3


@pytest.mark.parametrize("T,H,prefix", [(1, 64, [3000, 5]), (64, 64, [700, 1300])])
def test_captured_graph_two_streams_and_fresh_inputs(kdt, T, H, prefix):
    """Two calls captured on two streams with workspaces of their own, replayed on rewritten
    inputs; results as from plain calls, bit for bit."""
    import torch
    d = [_inputs(61 + k, T, H, prefix) for k in (0, 1)]
    pre = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    par = [torch.from_numpy(x["parent"]).cuda() for x in d]
    N = max(prefix) + T
    ws = [torch.empty(kdt.verify_attn_q8_workspace_size(2, T, H, N), dtype=torch.uint8, device="cuda") for _ in d]
    outs = [torch.empty(2, T, H, 512, device="cuda") for _ in d]
    lses = [torch.empty(2, T, H, device="cuda") for _ in d]

    def call(k, out, lse, w):
        x = d[k]
        kdt.verify_attn_q8(x["q"][..., :512], x["q"][..., 512:], x["c8"], x["sc"], x["kp"], pre, parent=par[k],
                           max_kv_len=N, scale=SCALE, out=out, lse=lse, workspace=w)

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
        for x in d:
            x["q"].copy_(torch.randn(x["q"].shape, device="cuda", generator=g).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        for k in (0, 1):
            o, l = torch.empty_like(outs[k]), torch.empty_like(lses[k])
            call(k, o, l, torch.empty_like(ws[k]))
            torch.cuda.synchronize()
            assert torch.equal(o, outs[k]) and torch.equal(l, lses[k])


@pytest.mark.parametrize("impl", ["q8_rows", "tcgen05"])
def test_infinite_rope_keys(kdt, impl):
    """A key with an infinite rope value scores +inf or -inf by the sign of the row's query there: NaN, or
    a key of weight 0."""
    d = _inputs(84, 5, 4, [200])
    d["kp"][0, 17, 3] = float("inf")
    out, lse = _call(kdt, d, impl=impl)
    up = (d["q"][0, ..., 512 + 3] > 0).cpu().numpy()
    assert up.any() and (d["q"][0, ..., 512 + 3] < 0).any()
    assert np.isnan(out[0][up]).all() and np.isnan(lse[0][up]).all()
    # the others: as without the key
    import torch
    keep = torch.tensor([j for j in range(205) if j != 17], device="cuda")
    e = dict(d, c8=d["c8"][:, keep].contiguous(), sc=d["sc"][:, keep].contiguous(), kp=d["kp"][:, keep].contiguous(),
             prefix=[199])
    without = _call(kdt, e, impl=impl)
    _check(e, (np.where(up[..., None], without[0][0], out[0])[None], np.where(up, without[1][0], lse[0])[None]), 0.0)


@pytest.mark.parametrize("impl", ["q8_rows", "tcgen05"])
def test_far_sequences_pass_32_bits(kdt, impl):
    """Code offsets of the last sequence are beyond 2^31 (and its queries few)."""
    d = _inputs(81, 9, 4, [0, 3, 260], pad=2200000)
    assert 2 * d["L"] * 512 > 2 ** 31
    _check(d, _call(kdt, d, impl=impl), 0.0)


@pytest.mark.parametrize("impl", ["q8_rows", "tcgen05"])
@pytest.mark.parametrize("T,H", [(1, 4), (6, 50)])
def test_more_sequences_than_sms(kdt, impl, T, H):
    rng = np.random.RandomState(3)
    d = _inputs(82, T, H, [int(x) for x in rng.randint(0, 300, 170)])
    _check(d, _call(kdt, d, impl=impl), 0.0)


def test_not_device_memory_is_refused(kdt):
    import torch
    d = _inputs(71, 33, 8, [10])            # a tree whose visibility takes a workspace
    pre = torch.tensor([10], dtype=torch.int32)
    with pytest.raises(kdt.KdtError) as e:
        kdt.verify_attn_q8(d["q"][..., :512], d["q"][..., 512:], d["c8"], d["sc"], d["kp"], pre.pin_memory(),
                           parent=torch.from_numpy(d["parent"]).cuda())
    assert e.value.status == 6
    with pytest.raises(kdt.KdtError) as e:
        kdt.verify_attn_q8(d["q"][..., :512], d["q"][..., 512:], d["c8"], d["sc"], d["kp"], pre.cuda(),
                           parent=torch.from_numpy(d["parent"]).cuda(),
                           workspace=torch.empty(256, dtype=torch.uint8, device="cuda")[128:])
    assert e.value.status == 4


@pytest.mark.parametrize("impl", ["q8_rows", "tcgen05"])
@pytest.mark.parametrize("T", [9, 32, 33])
def test_malformed_parents_are_recorded(kdt, T, impl):
    import torch
    d = _inputs(72, T, 4, [10, 0, 130])
    good = d["parent"].copy()
    d["parent"][1, 4], d["parent"][2, 6] = 4, -2            # its own parent; below -1
    good[1, 4] = good[2, 6] = -1                            # a walk ends there
    err = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    pre = torch.tensor(d["prefix"], dtype=torch.int32, device="cuda")
    got = []
    for par in (d["parent"], good):
        got.append(kdt.verify_attn_q8(d["q"][..., :512], d["q"][..., 512:], d["c8"], d["sc"], d["kp"], pre,
                                      parent=torch.from_numpy(par).cuda(), max_kv_len=130 + T, impl=impl, err=err))
        assert int(err.item()) == (T + 4 + 1 if par is not good else 0)
    for a, b in zip(*got):
        assert torch.equal(a, b)


def _scored_minus_inf(d, keys):
    """Infinite rope values at these cache rows of every sequence, against queries that are all negative
    there: each of those keys scores -inf for each row."""
    d["q"][..., 512 + 3] = -(d["q"][..., 512 + 3].abs() + 0.5)
    d["kp"][:, list(keys), 3] = float("inf")


def _without(d, keys):
    """The same problem without these prefix rows."""
    import torch
    keep = torch.tensor([j for j in range(d["L"]) if j not in set(keys)], device="cuda")
    return dict(d, c8=d["c8"][:, keep].contiguous(), sc=d["sc"][:, keep].contiguous(), kp=d["kp"][:, keep].contiguous(),
                prefix=[p - len(keys) for p in d["prefix"]])


# prefix, rows that score -inf: all of the first block, of the first two, of the last whole block, all but one row
MINUS_INF = [(383, range(0, 128)), (383, range(0, 256)), (384, range(0, 129)), (700, range(130, 700)), (640, range(1, 640))]


@pytest.mark.parametrize("splits", [0, 1, 2, 5])
@pytest.mark.parametrize("T,H", [(1, 4), (9, 8), (40, 8)])
@pytest.mark.parametrize("prefix,keys", MINUS_INF)
def test_blocks_that_score_minus_inf_have_weight_0_in_the_rows_kernel(kdt, prefix, keys, T, H, splits):
    """Whole 128-key blocks whose every score is -inf, an item's first block among them: as without these keys,
    however the work is cut."""
    d = _inputs(91, T, H, [prefix])
    _scored_minus_inf(d, keys)
    _check(_without(d, keys), _call(kdt, d, impl="q8_rows", num_splits=splits), 2.0 ** -24)


@pytest.mark.parametrize("splits", [0, 1, 2])
def test_nothing_but_minus_inf_in_the_rows_kernel(kdt, splits):
    """A token whose own key scores -inf behind a block of finite ones, and one whose every key does: what is
    left of the keys, and a row of zeros with lse -inf."""
    no = np.zeros((1, 1, 1), dtype=bool)
    d = _inputs(92, 1, 4, [128])
    _scored_minus_inf(d, [128])
    _check(d, _call(kdt, d, impl="q8_rows", num_splits=splits), 2.0 ** -24, see=no)
    for prefix in (0, 128, 383):
        d = _inputs(93, 1, 4, [prefix])
        _scored_minus_inf(d, range(prefix + 1))
        _check(dict(d, prefix=[0]), _call(kdt, d, impl="q8_rows", num_splits=splits), 0.0, see=no)
    # a NaN among them is not lost
    d["kp"][0, 200, 5] = float("nan")
    out, lse = _call(kdt, d, impl="q8_rows", num_splits=splits)
    assert np.isnan(out).all() and np.isnan(lse).all()


@pytest.mark.parametrize("splits", [0, 1, 2, 5])
@pytest.mark.parametrize("T,H", [(1, 4), (9, 8), (40, 8)])
@pytest.mark.parametrize("prefix,keys", MINUS_INF)
def test_blocks_that_score_minus_inf_have_weight_0_in_the_cluster_kernel(kdt, prefix, keys, T, H, splits):
    """The same there, whose blocks end at the last tree row: halves of 64 keys without a mask, all -inf."""
    d = _inputs(91, T, H, [prefix])
    _scored_minus_inf(d, keys)
    _check(_without(d, keys), _call(kdt, d, impl="tcgen05", num_splits=splits), 2.0 ** -24)


@pytest.mark.parametrize("splits", [0, 1, 2])
def test_nothing_but_minus_inf_in_the_cluster_kernel(kdt, splits):
    no = np.zeros((1, 1, 1), dtype=bool)
    d = _inputs(92, 1, 4, [128])
    _scored_minus_inf(d, [128])
    _check(d, _call(kdt, d, impl="tcgen05", num_splits=splits), 2.0 ** -24, see=no)
    for prefix in (0, 128, 383):
        d = _inputs(93, 1, 4, [prefix])
        _scored_minus_inf(d, range(prefix + 1))
        _check(dict(d, prefix=[0]), _call(kdt, d, impl="tcgen05", num_splits=splits), 0.0, see=no)
    d["kp"][0, 200, 5] = float("nan")
    out, lse = _call(kdt, d, impl="tcgen05", num_splits=splits)
    assert np.isnan(out).all() and np.isnan(lse).all()


@pytest.mark.parametrize("T,H,prefix", [(64, 64, [900, 2100, 1500, 77]), (9, 128, [4000, 12])])
def test_cluster_kernel_repeats_its_bits(kdt, T, H, prefix):
    """Both CTAs of a pair widen the tiles that one CTA's MMAs read: in every one of many runs, alone and with
    other work on the device, the result is the same bit for bit."""
    import torch
    d = _inputs(95, T, H, prefix)
    _check(d, _call(kdt, d, impl="tcgen05"), 2.0 ** -24)
    pre = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    par = torch.from_numpy(d["parent"]).cuda()
    args = (d["q"][..., :512], d["q"][..., 512:], d["c8"], d["sc"], d["kp"], pre)
    out, lse = kdt.verify_attn_q8(*args, parent=par, max_kv_len=max(prefix) + T, impl="tcgen05")
    side, junk = torch.cuda.Stream(), torch.empty(1 << 26, device="cuda")
    for k in range(60):
        if k % 2:
            with torch.cuda.stream(side):
                junk.add_(1.0)
        o, l = kdt.verify_attn_q8(*args, parent=par, max_kv_len=max(prefix) + T, impl="tcgen05")
        assert torch.equal(o, out) and torch.equal(l, lse), k
    torch.cuda.synchronize()


@pytest.mark.parametrize("impl", ["q8_rows", "tcgen05"])
@pytest.mark.parametrize("T,H", [(64, 8), (150, 2)])
def test_each_call_sees_its_own_tree(kdt, impl, T, H):
    """Calls in a row on one workspace with two trees in turn: the attention starts while the visibility
    kernel of its call still writes the words over those of the call before."""
    import torch
    d = _inputs(96, T, H, [40, 3, 300])
    pre = torch.tensor(d["prefix"], dtype=torch.int32, device="cuda")
    chain = np.tile(np.arange(T, dtype=np.int32) - 1, (3, 1))
    par = [torch.from_numpy(x).cuda() for x in (d["parent"], chain)]
    ws = torch.empty(kdt.verify_attn_q8_workspace_size(3, T, H, 300 + T, impl=impl), dtype=torch.uint8, device="cuda")
    args = (d["q"][..., :512], d["q"][..., 512:], d["c8"], d["sc"], d["kp"], pre)
    outs = [kdt.verify_attn_q8(*args, parent=par[k % 2], max_kv_len=300 + T, impl=impl, workspace=ws, scale=SCALE)
            for k in range(30)]
    torch.cuda.synchronize()
    for k, tree in enumerate((d["parent"], chain)):
        _check(dict(d, parent=tree), [x.double().cpu().numpy() for x in outs[k]], 2.0 ** -24)
    for k in range(2, 30):
        assert torch.equal(outs[k][0], outs[k % 2][0]) and torch.equal(outs[k][1], outs[k % 2][1])


@pytest.mark.parametrize("T,H,prefix", [(40, 16, [3000, 700])])
def test_a_busy_side_stream_keeps_its_workspace_and_outputs(kdt, T, H, prefix):
    """A call queued on a stream that is still busy: what the call allocated is not handed out to the current
    stream before it has run."""
    import torch
    d = _inputs(97, T, H, prefix)
    want = _call(kdt, d)
    pre = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    par = torch.from_numpy(d["parent"]).cuda()
    need = kdt.verify_attn_q8_workspace_size(2, T, H, max(prefix) + T)
    side, a = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):
            a = (a @ a).clamp_(-1, 1)
    out, lse = kdt.verify_attn_q8(d["q"][..., :512], d["q"][..., 512:], d["c8"], d["sc"], d["kp"], pre, parent=par, scale=SCALE,
                                  max_kv_len=max(prefix) + T, stream=side)
    junk = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), want[0]) and np.array_equal(lse.double().cpu().numpy(), want[1])
    del junk


def _check_nodes(d, got, out_eps, see, nodes):
    """_check for some nodes of each sequence: the others' rows are only required to be finite."""
    out, lse = got
    assert np.isfinite(out).all()
    for b, P in enumerate(d["prefix"]):
        N = P + d["T"]
        c = oq.dequantise(d["c8"][b, :N].cpu().numpy(), d["sc"][b, :N].cpu().numpy())
        k = d["kp"][b, :N].double().cpu().numpy()
        q = d["q"][b, nodes].double().cpu().numpy()
        ref_o, ref_l = oq.attention(q, c, k, P, see[b][nodes], SCALE)
        for n, i in enumerate(nodes):
            keys = np.concatenate([np.arange(P), P + np.flatnonzero(see[b][i])])
            if not len(keys):
                assert (out[b, i] == 0).all() and (lse[b, i] == -np.inf).all()
                continue
            kc = np.concatenate([c[keys], k[keys]], -1)
            p = np.exp(SCALE * (q[n] @ kc.T) - ref_l[n][:, None])
            ds = 576 * 2.0 ** -24 * SCALE * (np.abs(q[n]) @ np.abs(kc).T).max()
            tol = (2.0 ** -8 + 2 * ds + 2.0 ** -20) * (p @ np.abs(c[keys])) + (out_eps + 2.0 ** -22) * np.abs(ref_o[n])
            assert (np.abs(out[b, i] - ref_o[n]) <= tol).all(), (b, i, np.abs(out[b, i] - ref_o[n]).max())
            tol = ds + (2.0 ** -20 + (len(keys) / 128 + 12) * 2.0 ** -24) * (1 + np.abs(ref_l[n]))
            assert (np.abs(lse[b, i] - ref_l[n]) <= tol).all(), (b, i, np.abs(lse[b, i] - ref_l[n]).max())


def _some_nodes(T, n=24):
    """First and last nodes, those around words' and blocks' ends, and a few between."""
    edge = [i + e for i in range(0, T, 128) for e in (-1, 0, 1, 31, 32)]
    pick = np.random.RandomState(T).choice(T, min(T, n), replace=False).tolist()
    return sorted({i for i in [T - 2] + edge[:15] + edge[-10:] + pick + [T - 1] if 0 <= i < T})


WIDE = [(127, 3, [1, 300]), (128, 2, [0, 128]), (129, 5, [64, 70]), (200, 7, [0, 33, 500]), (513, 1, [127, 0]),
        (1000, 3, [90]), (2500, 1, [5, 200]), (4096, 2, [130]), (4095, 1, [0])]


@pytest.mark.parametrize("impl,splits", [("q8_rows", 0), ("q8_rows", 3), ("tcgen05", 0), ("tcgen05", 2), ("auto", 0)])
@pytest.mark.parametrize("kind", ["random", "chain"])
@pytest.mark.parametrize("T,H,prefix", WIDE)
def test_wide_trees_and_prompt_chunks(kdt, T, H, prefix, kind, impl, splits):
    """Trees over many visibility words and key blocks, up to the largest, and chains: a prompt's chunk."""
    d = _inputs(T, T, H, prefix)
    if kind == "chain":
        d["parent"] = np.tile(np.arange(T, dtype=np.int32) - 1, (len(prefix), 1))
    see = [oq.ancestors(p) for p in d["parent"]]
    _check_nodes(d, _call(kdt, d, impl=impl, num_splits=splits), 2.0 ** -24, see, _some_nodes(T))


@pytest.mark.parametrize("impl", ["q8_rows", "tcgen05"])
@pytest.mark.parametrize("T,H", [(161, 3), (1030, 2), (4096, 1)])
def test_wide_caller_bits(kdt, impl, T, H):
    """Any bits over many words, rows that see nothing among them."""
    d = _inputs(T + 1, T, H, [0, 70])
    rng = np.random.RandomState(T)
    see = rng.rand(2, T, T) < 0.02
    see[0, ::7] = False
    see[0, 3, T - 1] = see[1, 5, T - 33] = True
    _check_nodes(d, _call(kdt, d, see=see, impl=impl), 2.0 ** -24, see, _some_nodes(T))


@pytest.mark.parametrize("impl", ["q8_rows", "tcgen05"])
def test_same_as_the_bf16_cache_by_element(kdt, impl):
    """As test_same_as_the_bf16_cache, with each element's own bound: twice _check's, once for either kernel."""
    import torch
    d = _inputs(51, 16, 64, [500, 900])
    out, lse = _call(kdt, d, impl=impl)
    pre = torch.tensor(d["prefix"], dtype=torch.int32, device="cuda")
    c, k = kdt.latent_read_q8(d["c8"], d["sc"], d["kp"], None, d["L"])
    q = d["q"]
    o2, l2 = (x.double().cpu().numpy() for x in kdt.verify_attn(
        q[..., :512], q[..., 512:], c, k, pre, parent=torch.from_numpy(d["parent"]).cuda(), max_kv_len=916, scale=SCALE,
        impl="tcgen05"))
    for b, P in enumerate(d["prefix"]):
        kc = torch.cat([c[b, :P + 16], k[b, :P + 16]], -1).double().cpu().numpy()
        qb, see = q[b].double().cpu().numpy(), oq.ancestors(d["parent"][b])
        for i in range(16):
            keys = np.concatenate([np.arange(P), P + np.flatnonzero(see[i])])
            s = SCALE * (qb[i] @ kc[keys].T)
            p = np.exp(s - s.max(-1, keepdims=True))
            mag = (p / p.sum(-1, keepdims=True)) @ np.abs(kc[keys, :512])
            ds = 576 * 2.0 ** -24 * SCALE * (np.abs(qb[i]) @ np.abs(kc[keys]).T).max()
            tol = 2 * ((2.0 ** -8 + 2 * ds + 2.0 ** -20) * mag + (2.0 ** -24 + 2.0 ** -22) * np.abs(o2[b, i]))
            assert (np.abs(out[b, i] - o2[b, i]) <= tol).all(), (b, i)
            tol = 2 * (ds + (2.0 ** -20 + (len(keys) / 128 + 12) * 2.0 ** -24) * (1 + np.abs(l2[b, i])))
            assert (np.abs(lse[b, i] - l2[b, i]) <= tol).all(), (b, i)


@pytest.mark.parametrize("impl,splits", [("auto", 0), ("q8_rows", 0), ("q8_rows", 700), ("tcgen05", 0)])
@pytest.mark.parametrize("T,H,prefix", [(1, 64, [0, 1, 5]), (9, 8, [130, 3, 0, 300]), (40, 20, [70])])
def test_a_bound_far_above_the_lengths(kdt, T, H, prefix, impl, splits):
    """max_kv_len left at the cache's size: the split is planned for many more blocks than there are."""
    import torch
    d = _inputs(98, T, H, prefix, pad=30000)
    pre = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    out, lse = kdt.verify_attn_q8(d["q"][..., :512], d["q"][..., 512:], d["c8"], d["sc"], d["kp"], pre,
                                  parent=torch.from_numpy(d["parent"]).cuda(), scale=SCALE, impl=impl, num_splits=splits)
    _check(d, (out.double().cpu().numpy(), lse.double().cpu().numpy()), 2.0 ** -24)


@pytest.mark.parametrize("impl", ["q8_rows", "tcgen05"])
@pytest.mark.parametrize("scale", [0.0, -0.05, 2.0])
def test_other_scales(kdt, impl, scale, monkeypatch):
    """A scale of 0 (the plain mean), a negative and a large one. The bounds hold n 2^-24 |scale| sum |q||c|, so
    a negative scale is checked as the positive one over the negated queries: the same scores."""
    import sys
    d = _inputs(99, 20, 8, [300, 2], amp=0.25)
    for splits in (0, 1):
        monkeypatch.setattr(sys.modules[__name__], "SCALE", scale)
        got = _call(kdt, d, impl=impl, num_splits=splits)
        monkeypatch.setattr(sys.modules[__name__], "SCALE", abs(scale))
        _check(dict(d, q=-d["q"]) if scale < 0 else d, got, 2.0 ** -24)


@pytest.mark.parametrize("impl", ["q8_rows", "tcgen05"])
def test_queries_far_apart_and_a_cache_without_room_to_spare(kdt, impl):
    """Query rows 2048 elements apart; the last sequence's last row is the cache's last."""
    import torch
    d = _inputs(100, 7, 12, [400, 130], pad=0)
    wide = torch.full((2, 7, 12, 2048), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[..., 64:640] = d["q"]
    d["q"] = wide[..., 64:640]
    _check(d, _call(kdt, d, impl=impl), 2.0 ** -24)


def test_a_given_stream_inside_a_capture(kdt):
    """Capturing with ``stream=`` a side stream that joined the capture, workspace and outputs made by the call:
    replays give what plain calls give."""
    import torch
    d = _inputs(101, 40, 16, [900, 30])
    pre = torch.tensor(d["prefix"], dtype=torch.int32, device="cuda")
    par = torch.from_numpy(d["parent"]).cuda()
    args = (d["q"][..., :512], d["q"][..., 512:], d["c8"], d["sc"], d["kp"], pre)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=a):
        b.wait_stream(a)
        one = kdt.verify_attn_q8(*args, parent=par, max_kv_len=940, stream=b)
        two = kdt.verify_attn_q8(*args, parent=par, max_kv_len=940, stream=a)
        a.wait_stream(b)
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        d["q"].copy_(torch.randn(d["q"].shape, device="cuda", generator=g).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        want = kdt.verify_attn_q8(*args, parent=par, max_kv_len=940)
        torch.cuda.synchronize()
        for got in (one, two):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
