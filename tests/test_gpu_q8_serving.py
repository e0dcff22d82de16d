"""GPU test of the 8-bit cache's operators as a serving loop uses them: prompts are written, then each
step writes a drafted tree's rows behind the prefix, attends, samples the path that stands and moves its
rows to the prefix. Every call is checked against the float64 oracle on what it read, and after the
steps the cache holds, byte for byte, the rows of the emitted tokens written in one line."""
import numpy as np
import pytest

from tests import test_gpu_tree_sample as ts
from tests import test_gpu_verify_q8 as tv

pytestmark = pytest.mark.gpu
kdt = tv.kdt

B, T, H, V, L, STEPS, TEMP = 3, 12, 8, 600, 160, 4, 0.9
PROMPT = [40, 5, 77]


class Model:
    """Rows of the cache and queries by token; logits from the attention's outputs."""

    def __init__(self):
        import torch
        g = torch.Generator(device="cuda").manual_seed(5)

        def rnd(*shape, dtype=torch.bfloat16):
            return torch.randn(*shape, device="cuda", generator=g).to(dtype)
        self.kv, self.q, self.gamma = rnd(V, 576), rnd(V, H, 576), rnd(512) * 0.1 + 1
        self.w = rnd(H * 512, V, dtype=torch.float32) * 0.05
        self.prompt = torch.randint(0, V, (B, max(PROMPT)), device="cuda", generator=g)


def _cache():
    import torch
    return (torch.zeros(B, L, 512, dtype=torch.uint8, device="cuda"), torch.full((B, L, 16), 255, dtype=torch.uint8, device="cuda"),
            torch.full((B, L, 64), float("nan"), dtype=torch.bfloat16, device="cuda"))


def _write(kdt, m, cache, tok, pos, prefix, n_rows=None):
    kv = m.kv[tok]
    kdt.latent_write_q8(kv[..., :512], kv[..., 512:], *cache, prefix, gamma=m.gamma, pos=pos, n_rows=n_rows)


def _drafts(seed):
    """Trees of STEPS steps: parents, depths, drafted tokens (node 0's is the token to continue), random numbers
    and how strongly the logits favour each drafted token."""
    rng = np.random.RandomState(seed)
    out = []
    for _ in range(STEPS):
        parent = np.stack([ts._tree(rng, T, 3) for _ in range(B)])
        depth = np.zeros_like(parent)
        for i in range(1, T):
            depth[:, i] = depth[np.arange(B), parent[:, i]] + 1
        out.append((parent, depth, rng.randint(0, V, (B, T)).astype(np.int32), rng.rand(B, T).astype(np.float32),
                    rng.rand(B).astype(np.float32), np.where(rng.rand(B, T) < 0.7, 12.0, 0.0).astype(np.float32)))
    return out


def _step(kdt, m, cache, prefix, ws, t):
    """One step on device tensors t = (parent, depth, tok, u_node, u_bonus, lift); tok's node 0 is the root."""
    import torch
    parent, depth, tok, un, ub, lift = t
    _write(kdt, m, cache, tok.long(), prefix[:, None] + depth, prefix)
    q = m.q[tok.long()]
    out, lse = kdt.verify_attn_q8(q[..., :512], q[..., 512:], *cache, prefix, parent=parent, max_kv_len=L, scale=tv.SCALE,
                                  out_dtype=torch.float32, workspace=ws)
    logits = out.reshape(B, T, H * 512) @ m.w
    b = torch.arange(B, device="cuda")[:, None].expand(B, T - 1)
    logits.index_put_((b, parent[:, 1:].long(), tok[:, 1:].long()), lift[:, 1:], accumulate=True)
    acc, n, bonus, logp = kdt.tree_sample(parent, tok, logits, un, ub, temperature=TEMP)
    before = prefix.clone()
    kdt.kv_compact_q8(*cache, prefix, acc, n)
    return dict(q=q, out=out, lse=lse, logits=logits, acc=acc, n=n, bonus=bonus, logp=logp, before=before)


def _run(kdt, m, drafts, graph):
    """All steps, eagerly or as replays of one captured step; what each step returned, the cache, the tokens."""
    import torch
    cache = _cache()
    prefix = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens = torch.tensor(PROMPT, dtype=torch.int32, device="cuda")
    pos = torch.arange(max(PROMPT), dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    _write(kdt, m, cache, m.prompt, pos, prefix, n_rows=lens)
    prefix.copy_(lens)
    need = kdt.verify_attn_q8_workspace_size(B, T, H, L)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    root = np.arange(B, dtype=np.int32)
    emitted = [m.prompt[b, :PROMPT[b]].tolist() for b in range(B)]
    steps, g, t = [], None, None
    for parent, depth, tok, un, ub, lift in drafts:
        tok = tok.copy()
        tok[:, 0] = root
        new = [torch.from_numpy(x).cuda() for x in (parent, depth, tok, un, ub, lift)]
        if not graph:
            r = _step(kdt, m, cache, prefix, ws, new)
        else:
            if g is None:
                t = new
                saved = [x.clone() for x in (*cache, prefix)]
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    _step(kdt, m, cache, prefix, ws, t)      # warm-up
                torch.cuda.current_stream().wait_stream(side)
                for x, y in zip((*cache, prefix), saved):
                    x.copy_(y)
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    held = _step(kdt, m, cache, prefix, ws, t)
            for x, y in zip(t, new):
                x.copy_(y)
            g.replay()
            r = {k: v.clone() for k, v in held.items()}
        torch.cuda.synchronize()
        r["tok"], r["parent"], r["u"], r["ub"] = tok, parent, un, ub
        r["cache"] = [x.clone() for x in cache]
        steps.append(r)
        for b in range(B):
            emitted[b] += tok[b, r["acc"][b, :r["n"][b]].tolist()].tolist()
        root = r["bonus"].cpu().numpy()
    return steps, cache, prefix, emitted


def test_steps_of_a_serving_loop(kdt):
    import torch
    m, drafts = Model(), _drafts(9)
    steps, cache, prefix, emitted = _run(kdt, m, drafts, False)
    longest = 0
    for r in steps:
        P = r["before"].tolist()
        # attention and sampling against the oracle, on the cache as it was (moved rows lie at or before
        # their sources, so the tree's rows are written again where the path was moved over them)
        c = [x.clone() for x in r["cache"]]
        depth = np.zeros((B, T), dtype=np.int32)
        for i in range(1, T):
            depth[:, i] = depth[np.arange(B), r["parent"][:, i]] + 1
        _write(kdt, m, c, torch.from_numpy(r["tok"]).cuda().long(), r["before"][:, None] + torch.from_numpy(depth).cuda(), r["before"])
        d = dict(q=r["q"], c8=c[0], sc=c[1], kp=c[2], parent=r["parent"], prefix=P, T=T, H=H, B=B, L=L)
        tv._check(d, (r["out"].double().cpu().numpy(), r["lse"].double().cpu().numpy()), 0.0)
        s = dict(parent=r["parent"], tok=r["tok"], logits=r["logits"], u=r["u"], ub=r["ub"], temp=TEMP)
        ts._check(s, tuple(r[k].cpu().numpy() for k in ("acc", "n", "bonus", "logp")) + (0,))
        longest = max(longest, int(r["n"].max()))
    assert longest >= 3
    # the cache holds the emitted tokens' rows as if written in one line
    n = [len(e) for e in emitted]
    assert prefix.tolist() == n and max(n) <= L - T
    line = torch.zeros(B, max(n), dtype=torch.long, device="cuda")
    for b in range(B):
        line[b, :n[b]] = torch.tensor(emitted[b])
    want = _cache()
    pos = torch.arange(max(n), dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    _write(kdt, m, want, line, pos, torch.zeros(B, dtype=torch.int32, device="cuda"),
           n_rows=torch.tensor(n, dtype=torch.int32, device="cuda"))
    for b in range(B):
        for x, y in zip(cache, want):
            assert torch.equal(x[b, :n[b]], y[b, :n[b]])


def test_captured_step_replayed(kdt):
    import torch
    m, drafts = Model(), _drafts(10)
    a, ca, pa, ea = _run(kdt, m, drafts, False)
    b, cb, pb, eb = _run(kdt, m, drafts, True)
    assert ea == eb and torch.equal(pa, pb)
    for x, y in zip(a, b):
        for k in ("acc", "n", "bonus", "logp", "out", "lse"):
            assert torch.equal(x[k], y[k]), k
    for x, y in zip(ca, cb):
        for k in range(B):
            assert torch.equal(x[k, :pa[k]], y[k, :pa[k]])
