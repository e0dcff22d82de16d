"""GPU test of the paged cache's operators as a server uses them: prompts get pages and are written, then a step gives
every request room for a drafted tree, writes its rows at their slots, attends, samples the path that stands, moves its
rows to the prefix and gives the pages behind it back; then one token more is decoded, drawn under top-k and top-p.
Every call is checked against the float64 oracle on what it read, and after the steps the cache holds, byte for byte,
the rows of the emitted tokens, in pages that no two requests share."""
import numpy as np
import pytest

from oracle import paged as op
from tests import test_gpu_sample as tp
from tests import test_gpu_tree_sample as ts
from tests import test_gpu_verify_paged as tv
from tests.test_gpu_q8_serving import Model, _drafts, B, T, H, V, STEPS, TEMP, PROMPT

pytestmark = pytest.mark.gpu
kdt = tv.kdt

PAGE, W, PAGES = 8, 20, 48
DRAW = dict(temperature=0.8, top_k=40, top_p=0.9)


class Server:
    def __init__(self, kdt, m, seed):
        import torch
        self.kdt, self.m = kdt, m
        self.c = torch.full((PAGES, PAGE, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.k = torch.full((PAGES, PAGE, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
        self.held = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.free = torch.from_numpy(np.random.RandomState(seed).permutation(PAGES).astype(np.int32)).cuda()
        self.n_free = torch.tensor([PAGES], dtype=torch.int32, device="cuda")
        self.prefix = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.root = torch.arange(B, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(4, dtype=torch.int32, device="cuda")
        need = max(kdt.verify_attn_paged_workspace_size(B, t, H, W * PAGE, PAGE) for t in (1, T))
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def state(self):
        return (self.c, self.k, self.table, self.held, self.free, self.n_free, self.prefix, self.root)

    def room(self, new_len, n=0, err=None):
        return self.kdt.page_assign(self.table, self.held, self.free, self.n_free, new_len, PAGE, start=self.prefix if n else None,
                                    T=n, err=err)

    def write(self, tok, pos, slots):
        kv = self.m.kv[tok.long()]
        self.kdt.latent_write_paged(kv[..., :512], kv[..., 512:], self.c, self.k, slots, gamma=self.m.gamma, pos=pos)

    def attend(self, tok, **kw):
        import torch
        q = self.m.q[tok.long()]
        seen = dict(q=q, c=self.c.clone(), k=self.k.clone(), table=self.table.clone(), prefix=self.prefix.clone())
        out, lse = self.kdt.verify_attn_paged(q[..., :512], q[..., 512:], self.c, self.k, self.table, self.prefix, scale=tv.SCALE,
                                              out_dtype=torch.float32, workspace=self.ws, **kw)
        return dict(seen, out=out, lse=lse, logits=out.reshape(B, -1, H * 512) @ self.m.w)

    def prompts(self):
        import torch
        lens = torch.tensor(PROMPT, dtype=torch.int32, device="cuda")
        slots = self.room(lens, max(PROMPT))
        pos = torch.arange(max(PROMPT), dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
        self.write(self.m.prompt, pos, slots)
        self.prefix.copy_(lens)

    def step(self, t):
        """One step on device tensors (parent, depth, tok, u_node, u_bonus, lift, u): a tree, then a single token."""
        import torch
        parent, depth, tok, un, ub, lift, u = t
        tok[:, 0] = self.root
        slots = self.room(self.prefix + T, T, self.err[0:1])
        self.write(tok, self.prefix[:, None] + depth, slots)
        r = self.attend(tok, parent=parent, err=self.err[1:2])
        b = torch.arange(B, device="cuda")[:, None].expand(B, T - 1)
        r["logits"].index_put_((b, parent[:, 1:].long(), tok[:, 1:].long()), lift[:, 1:], accumulate=True)
        acc, n, bonus, logp = self.kdt.tree_sample(parent, tok, r["logits"], un, ub, temperature=TEMP)
        self.kdt.kv_compact_paged(self.c, self.k, self.table, self.prefix, acc, n)
        self.room(self.prefix)                               # what the path did not fill
        # decoded: the bonus token's row, then the next token
        one = bonus[:, None]
        slots = self.room(self.prefix + 1, 1, self.err[2:3])
        self.write(one, self.prefix[:, None].contiguous(), slots)
        s = self.attend(one, err=self.err[3:4])
        nxt, nlogp = self.kdt.sample(s["logits"].reshape(B, V), u, **DRAW)
        self.prefix += 1
        self.root.copy_(nxt)
        r.update(tok=tok.clone(), acc=acc, n=n, bonus=bonus, logp=logp, nxt=nxt, nlogp=nlogp, err=self.err.clone(),
                 held=self.held.clone(), n_free=self.n_free.clone())
        r.update({"one_" + key: v for key, v in s.items()})
        return r


def _run(kdt, m, seed, graph):
    import torch
    sv = Server(kdt, m, seed)
    sv.prompts()
    rng = np.random.RandomState(seed + 1)
    emitted = [m.prompt[b, :PROMPT[b]].tolist() for b in range(B)]
    steps, g, t = [], None, None
    for d in _drafts(seed):
        new = [torch.from_numpy(x).cuda() for x in (*d, rng.rand(B).astype(np.float32))]
        if not graph:
            r = sv.step(new)
        else:
            if g is None:
                t = new
                saved = [x.clone() for x in sv.state()]
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    sv.step(t)                               # warm-up
                torch.cuda.current_stream().wait_stream(side)
                for x, y in zip(sv.state(), saved):
                    x.copy_(y)
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    kept = sv.step(t)
            for x, y in zip(t, new):
                x.copy_(y)
            g.replay()
            r = {key: v.clone() for key, v in kept.items()}
        torch.cuda.synchronize()
        r.update(parent_np=d[0], u_np=(d[3], d[4], new[6].cpu().numpy()))
        steps.append(r)
        tok = r["tok"].cpu().numpy()
        for b in range(B):
            emitted[b] += tok[b, r["acc"][b, :r["n"][b]].tolist()].tolist() + [int(r["bonus"][b])]
    return steps, sv, emitted


def _attention(r, n, parent, pre=""):
    d = dict(q=r[pre + "q"], c=r[pre + "c"], k=r[pre + "k"], table=r[pre + "table"].cpu().numpy(), prefix=r[pre + "prefix"].tolist(),
             T=n, H=H, B=B, page=PAGE, parent=parent, n=[n] * B)
    d["rows"] = [op.rows_of(d["table"][b], d["prefix"][b] + n, PAGE) for b in range(B)]
    tv._check(d, (r[pre + "out"].double().cpu().numpy(), r[pre + "lse"].double().cpu().numpy()), 2.0 ** -24)


def test_steps_of_a_server(kdt):
    import torch
    m = Model()
    steps, sv, emitted = _run(kdt, m, 11, False)
    longest = 0
    for r in steps:
        assert r["err"].tolist() == [0] * 4
        _attention(r, T, r["parent_np"])
        _attention(r, 1, np.full((B, 1), -1, dtype=np.int32), "one_")
        un, ub, u = r["u_np"]
        ts._check(dict(parent=r["parent_np"], tok=r["tok"].cpu().numpy(), logits=r["logits"], u=un, ub=ub, temp=TEMP),
                  tuple(r[key].cpu().numpy() for key in ("acc", "n", "bonus", "logp")) + (0,))
        tok, logp = tp._check(kdt, r["one_logits"].reshape(B, V), u, **DRAW)
        assert (tok == r["nxt"].cpu().numpy()).all() and (logp == r["nlogp"].cpu().numpy()).all()
        longest = max(longest, int(r["n"].max()))
    assert longest >= 3
    # pages: as many as the rows need, every one in one place
    n = [len(e) for e in emitted]
    assert sv.prefix.tolist() == n and sv.held.tolist() == [-(-x // PAGE) for x in n]
    table, free = sv.table.cpu().numpy(), sv.free[:int(sv.n_free)].tolist()
    used = [int(p) for b in range(B) for p in table[b, :-(-n[b] // PAGE)]]
    assert sorted(used + free) == list(range(PAGES))
    # the cache holds the emitted tokens' rows as if written in one line
    for b in range(B):
        rows = torch.from_numpy(op.rows_of(table[b], n[b], PAGE)).cuda()
        c = torch.zeros(-(-n[b] // PAGE), PAGE, 512, dtype=torch.bfloat16, device="cuda")
        k = torch.zeros(c.shape[0], PAGE, 64, dtype=torch.bfloat16, device="cuda")
        kv = m.kv[torch.tensor([emitted[b]], device="cuda")]
        line = torch.arange(n[b], dtype=torch.int32, device="cuda")[None]
        kdt.latent_write_paged(kv[..., :512], kv[..., 512:], c, k, line, gamma=m.gamma, pos=line)
        for x, y, D in ((sv.c, c, 512), (sv.k, k, 64)):
            assert torch.equal(x.view(-1, D)[rows].view(torch.int16), y.view(-1, D)[:n[b]].view(torch.int16))


def test_captured_steps_replayed(kdt):
    import torch
    m = Model()
    a, sa, ea = _run(kdt, m, 12, False)
    b, sb, eb = _run(kdt, m, 12, True)
    assert ea == eb
    for x, y in zip(a, b):
        for key in ("acc", "n", "bonus", "logp", "out", "lse", "one_out", "one_lse", "nxt", "nlogp", "held", "n_free", "err"):
            assert torch.equal(x[key], y[key]), key
    for x, y in zip(sa.state()[2:], sb.state()[2:]):
        assert torch.equal(x, y)
    n = sa.prefix.tolist()
    table = sa.table.cpu().numpy()
    for i in range(B):
        rows = torch.from_numpy(op.rows_of(table[i], n[i], PAGE)).cuda()
        for x, y, D in ((sa.c, sb.c, 512), (sa.k, sb.k, 64)):
            assert torch.equal(x.view(-1, D)[rows].view(torch.int16), y.view(-1, D)[rows].view(torch.int16))
