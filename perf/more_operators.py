"""Measured cases of serving from a paged latent cache.

A server of many requests keeps the latent cache in pages. One step of it is: give every
request the pages its new rows need and say where each row goes (``assign``), norm, rotate
and store the new rows there (``write``), attend over the pages, one token or a small draft
tree a request (``attn``), draw the next token under each request's temperature, top-k, top-p
and min-p (``sample``), or, after a draft tree, close the gaps of the branches that lost
(``compact``). A cache row is 512 latent and 64 rope values in bf16.
"""
import math

import torch

own = False

D_C, D_R = 512, 64
SCALE = 1.0 / math.sqrt(192.0)
BASE, EPS = 10000.0, 1e-6
WEIGHT_UNIT = 2.0 ** 44                     # sampling weights are held to 2^-44 of the row's largest


def listed():
    return [
        # a batched tree step: room for 64 drafted rows each, and back after the step; latency counts
        {"name": "assign tree step", "op": "assign", "B": 8, "T": 64, "lo": 100, "hi": 2000, "page": 64},
        # many prompts admitted at once, small pages, and their requests finished
        {"name": "assign prompts", "op": "assign", "B": 256, "T": 2001, "lo": 0, "hi": 0, "page": 16},
        # plain decoding: one new row of each of 64 requests, bf16 activations
        {"name": "write single rows", "op": "write", "B": 64, "T": 1, "lo": 100, "hi": 2000, "page": 64, "dtype": "bf16",
         "norm": True, "ragged": False},
        # a padded batch of long prompt chunks, fp32 activations
        {"name": "write prompts", "op": "write", "B": 12, "T": 4095, "lo": 0, "hi": 700, "page": 32, "dtype": "f32",
         "norm": True, "ragged": True},
        # one short conversation, a tensor-parallel share of the heads; latency counts
        {"name": "attn one request", "op": "attn", "B": 1, "T": 1, "H": 16, "lo": 700, "hi": 700, "page": 64},
        # plain decoding of a batch, ragged contexts: cache bandwidth counts
        {"name": "attn single tokens", "op": "attn", "B": 64, "T": 1, "H": 64, "lo": 1024, "hi": 8192, "page": 64},
        # two long contexts, all heads on one device, large pages: split over the length
        {"name": "attn long contexts", "op": "attn", "B": 2, "T": 1, "H": 128, "lo": 60001, "hi": 99990, "page": 128},
        # small draft trees, few heads, small pages
        {"name": "attn small trees", "op": "attn", "B": 8, "T": 13, "H": 32, "lo": 2500, "hi": 12000, "page": 16},
        # one request, a small vocabulary, fp32 logits; latency counts
        {"name": "sample one", "op": "sample", "R": 1, "V": 32000, "dtype": "f32", "peak": 1.4, "temp": 0.8, "top_k": 50,
         "top_p": 0.9, "min_p": 0.0, "mixed": False},
        # a batch with settings of its own for every request, a large vocabulary, bf16 logits
        {"name": "sample batch", "op": "sample", "R": 64, "V": 160000, "dtype": "bf16", "peak": 1.2, "temp": 1.0,
         "top_k": 0, "top_p": 0.95, "min_p": 0.02, "mixed": True},
        # accepted paths after a usual tree step
        {"name": "compact step", "op": "compact", "B": 8, "T": 64, "path": 6, "lo": 500, "hi": 2500, "page": 64},
        # many sequences with deep accepted paths, small pages
        {"name": "compact deep", "op": "compact", "B": 96, "T": 256, "path": 120, "lo": 100, "hi": 1000, "page": 16},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["assign", "write", "attn", "attn", "attn", "sample", "sample", "compact"])
    page = rng.choice([8, 16, 32, 64, 64, 128, 256])
    if op == "assign":
        B = _log_int(rng, 1, 256)
        lo = rng.choice([0, rng.randint(0, 600)])
        return {"op": op, "B": B, "T": _log_int(rng, 1, min(4096, 500000 // B)), "lo": lo,
                "hi": lo + (rng.randint(0, 1500) if lo else 0), "page": page}
    if op == "write":
        B = _log_int(rng, 1, 64)
        T = _log_int(rng, 1, min(4096, 48000 // B))
        lo = rng.randint(0, 600)
        return {"op": op, "B": B, "T": T, "lo": lo, "hi": lo + rng.randint(0, 1500), "page": page,
                "dtype": rng.choice(["bf16", "f32"]), "norm": rng.random() < 0.75, "ragged": rng.random() < 0.5}
    if op == "attn":
        T = rng.choice([1, 1, 1, _log_int(rng, 2, 64)])
        H = rng.choice([1, 8, 16, 20, 32, 64, 128, rng.randint(2, 128)])
        # no dearer than the batch of single tokens: rows x keys, and the cache, at most as large
        hi = _log_int(rng, 1, min(60000, 64 * 64 * 4608 // (T * H)))
        lo = rng.randint(0, hi) if rng.random() < 0.6 else hi
        most = min(64, 64 * 64 * 4608 // (T * H * (hi + T)), 290000 // (hi + T))
        return {"op": op, "B": _log_int(rng, 1, max(1, most)), "T": T, "H": H, "lo": lo, "hi": hi, "page": page}
    if op == "sample":
        R = _log_int(rng, 1, 256)
        return {"op": op, "R": R, "V": _log_int(rng, 900, min(160000, 10_000_000 // R)), "dtype": rng.choice(["bf16", "f32"]),
                "peak": round(rng.uniform(0.9, 1.8), 2), "temp": rng.choice([1.0, 0.7, 1.2]),
                "top_k": rng.choice([0, 0, 20, 50, 400]), "top_p": rng.choice([1.0, 0.95, 0.9, 0.5]),
                "min_p": rng.choice([0.0, 0.0, 0.02, 0.1]), "mixed": rng.random() < 0.5}
    T = _log_int(rng, 2, 256)
    lo = rng.randint(0, 800)
    return {"op": op, "B": _log_int(rng, 1, 96), "T": T, "path": rng.randint(1, max(1, T // 2)), "lo": lo,
            "hi": lo + rng.randint(0, 1500), "page": page}


# ------------------------------------------------------------------------------ inputs --
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lens(case):
    """Sequence b's prefix length: spread evenly over [lo, hi], in a fixed mixed order."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    order = [(b * 7 + 3) % B if B % 7 else b for b in range(B)]
    return [hi if B == 1 else lo + (hi - lo) * k // (B - 1) for k in order]


def _new_rows(case):
    """Rows of sequence b that are written (a padded batch holds fewer than T)."""
    B, T = case["B"], case["T"]
    return [T if not case["ragged"] else max(0, T - (T * b) // B) for b in range(B)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _pages(rows, page):
    return (rows + page - 1) // page


def _table(g, lens, page, spare):
    """A page table as a running server leaves it: a request's pages anywhere, behind them what was there before.
    Returns it, the pages of each request (int32, on the GPU) and the number of all pages."""
    held = [_pages(n, page) for n in lens]
    n_pages, W = sum(held) + spare, max(max(held), 1)
    order = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
    table = torch.randint(0, n_pages, (len(lens), W), device="cuda", generator=g).to(torch.int32)
    h = torch.tensor(held, device="cuda")
    table[torch.arange(W, device="cuda") < h.unsqueeze(1)] = order[:sum(held)]
    return table, h.to(torch.int32), n_pages, order


def _cache(g, n_pages, page):
    """A filled cache: normed latents with a learned weight, as a model leaves them."""
    gamma = 0.5 + torch.rand(D_C, device="cuda", generator=g)
    c_kv = torch.empty(n_pages, page, D_C, dtype=torch.bfloat16, device="cuda")
    for a in range(0, n_pages, max(1, 65536 // page)):
        part = c_kv[a:a + max(1, 65536 // page)]
        part.copy_(torch.randn(part.shape, device="cuda", generator=g) * gamma)
    k_pe = torch.randn(n_pages, page, D_R, device="cuda", generator=g).to(torch.bfloat16)
    return c_kv, k_pe


def _tree(g, B, T):
    """Parents with a bias to recent nodes, node 0 the root."""
    back = torch.empty(B, T, device="cuda").exponential_(0.3, generator=g).floor().to(torch.int64) + 1
    i = torch.arange(T, device="cuda").expand(B, T)
    parent = torch.where(i == 0, torch.full_like(i, -1), (i - back).clamp(min=0))
    return parent.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "sample":
        R, V = case["R"], case["V"]
        # a few likely tokens and a long tail: the logit falls with the log of the rank
        rank = torch.rand(R, V, device="cuda", generator=g).argsort(-1).to(torch.float32)
        logits = 14.0 - case["peak"] * torch.log(1.0 + rank) + 0.4 * torch.randn(R, V, device="cuda", generator=g)
        s["logits"] = logits.to(_DT[case["dtype"]])
        s["u"] = torch.rand(R, device="cuda", generator=g)
        for k in ("temp", "top_k", "top_p", "min_p"):
            s[k] = case[k]
        if case["mixed"]:                   # every request brings its own settings
            r = torch.rand(4, R, device="cuda", generator=g)
            s["temp"] = case["temp"] * (0.7 + 0.5 * r[0])
            s["top_k"] = torch.where(r[1] < 0.5, torch.full_like(r[1], case["top_k"]), 5 + 100 * r[1]).to(torch.int32)
            s["top_p"] = torch.where(r[2] < 0.2, torch.ones_like(r[2]), case["top_p"] - 0.1 * r[2])
            s["min_p"] = torch.where(r[3] < 0.5, torch.zeros_like(r[3]), torch.full_like(r[3], case["min_p"]))
        return s
    B, T, page = case["B"], case["T"], case["page"]
    lens = _lens(case)
    s["prefix_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if op == "assign":
        add = [max(1, T - (T * b) // (2 * B)) for b in range(B)]
        room = sum(_pages(n + a, page) for n, a in zip(lens, add))
        table, held, n_pages, order = _table(g, lens, page, room - sum(_pages(n, page) for n in lens) + 5)
        W = max(_pages(n + a, page) for n, a in zip(lens, add))
        s["table"] = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
        s["table"][:, :table.shape[1]] = table[:, :W]
        s["held"] = held
        used = sum(_pages(n, page) for n in lens)
        s["free"] = torch.cat([order[used:], order[:used]])     # a stack: the first n_free of it are free
        s["n_free"] = torch.tensor([n_pages - used], dtype=torch.int32, device="cuda")
        s["new_len"] = s["prefix_len"] + torch.tensor(add, dtype=torch.int32, device="cuda")
        return s
    s["table"], _, n_pages, _ = _table(g, [n + T for n in lens], page, 7)
    s["c_kv"], s["k_pe"] = _cache(g, n_pages, page)
    if op == "write":
        kv = torch.randn(B, T, D_C + D_R, device="cuda", generator=g) * 1.7
        s["kv"] = kv.to(_DT[case["dtype"]])
        if case["norm"]:
            s["gamma"] = (0.5 + torch.rand(D_C, device="cuda", generator=g)).to(_DT[case["dtype"]])
        i = torch.arange(T, device="cuda")
        rows = s["prefix_len"].long().unsqueeze(1) + i
        s["pos"] = rows.to(torch.int32)
        at = s["table"].long().gather(1, rows // page) * page + rows % page
        n = torch.tensor(_new_rows(case), device="cuda").unsqueeze(1)
        s["slots"] = torch.where(i < n, at, torch.full_like(at, -1)).to(torch.int32)
    elif op == "attn":
        s["max_kv"] = max(lens) + T
        s["q"] = torch.randn(B, T, case["H"], D_C + D_R, device="cuda", generator=g).to(torch.bfloat16)
        if T > 1:
            s["parent"] = _tree(g, B, T)
    else:                                   # compact: increasing paths of about the asked length
        steps = torch.rand(B, T - 1, device="cuda", generator=g).argsort(-1)
        n = (1 + torch.randint(0, 2 * case["path"], (B,), device="cuda", generator=g)).clamp(max=T)
        chosen = steps < (n - 1).unsqueeze(1)                       # n - 1 nodes below the root
        i = torch.arange(1, T, device="cuda").expand(B, T - 1)
        path = torch.where(chosen, i, torch.full_like(i, T + 1)).sort(-1).values
        path = torch.where(path > T, torch.full_like(path, -1), path)
        s["acc"] = torch.cat([torch.zeros(B, 1, device="cuda", dtype=torch.int64), path], 1).to(torch.int32)
        s["n_acc"] = n.to(torch.int32)
    return s


# ------------------------------------------------------------------- one pass, each operator --
def run(s):
    return {"assign": _run_assign, "write": _run_write, "attn": _run_attn, "sample": _run_sample,
            "compact": _run_compact}[s["case"]["op"]](s)


def _resize(s, new_len, page):
    """Every request to the pages of new_len rows: what it gives up goes on top of the stack, the first given
    uppermost, then what others need comes off the top."""
    B, W = s["table"].shape
    cap = s["free"].numel()
    col = torch.arange(W, device="cuda")
    need, have = ((new_len + page - 1) // page).unsqueeze(1), s["held"].unsqueeze(1)
    gives, takes = (col >= need) & (col < have), (col >= have) & (col < need)
    k_give = torch.cumsum(gives.flatten(), 0).view(B, W)
    k_take = torch.cumsum(takes.flatten(), 0).view(B, W)
    top = s["n_free"].long() + k_give[-1, -1]
    stack = torch.cat([s["free"], s["free"][:1]])               # one place more for what is not written
    stack[torch.where(gives, top - k_give, torch.full_like(k_give, cap))] = s["table"]
    s["table"].copy_(torch.where(takes, stack[(top - k_take).clamp(0, cap - 1)], s["table"]))
    top = top - k_take[-1, -1]
    s["free"].copy_(torch.where(torch.arange(cap, device="cuda") < top, stack[:cap], s["free"]))
    s["n_free"].copy_(top)
    s["held"].copy_(need.squeeze(1))


def _run_assign(s):
    """The step's rows get their pages and slots, and the pages go back behind the step."""
    case = s["case"]
    T, page = case["T"], case["page"]
    if own:
        import speculative_decoding_tree_absorb_gb300 as kdt
        slots = kdt.page_assign(s["table"], s["held"], s["free"], s["n_free"], s["new_len"], page,
                                start=s["prefix_len"], T=T)
        kdt.page_assign(s["table"], s["held"], s["free"], s["n_free"], s["prefix_len"], page)
    else:
        _resize(s, s["new_len"], page)
        rows = s["prefix_len"].long().unsqueeze(1) + torch.arange(T, device="cuda")
        at = s["table"].long().gather(1, (rows // page).clamp(max=s["table"].shape[1] - 1)) * page + rows % page
        slots = torch.where(rows < s["new_len"].unsqueeze(1), at, torch.full_like(at, -1)).to(torch.int32)
        _resize(s, s["prefix_len"], page)
    return slots, s["table"], s["held"], s["free"], s["n_free"]


def _run_write(s):
    kv = s["kv"]
    if own:
        import speculative_decoding_tree_absorb_gb300 as kdt
        kdt.latent_write_paged(kv[..., :D_C], kv[..., D_C:], s["c_kv"], s["k_pe"], s["slots"], gamma=s.get("gamma"),
                               eps=EPS, pos=s["pos"], base=BASE)
        return s["c_kv"], s["k_pe"]
    x = kv[..., :D_C].to(torch.float32)
    if "gamma" in s:
        x = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * s["gamma"].to(torch.float32)
    freq = BASE ** (-2.0 * torch.arange(D_R // 2, device="cuda", dtype=torch.float64) / D_R)
    a = s["pos"].to(torch.float64).unsqueeze(-1) * freq
    c, n = torch.cos(a).to(torch.float32), torch.sin(a).to(torch.float32)
    k1, k2 = kv[..., D_C:].to(torch.float32).chunk(2, -1)
    k = torch.cat([k1 * c - k2 * n, k2 * c + k1 * n], -1)
    keep = s["slots"] >= 0
    at = s["slots"][keep].long()
    s["c_kv"].view(-1, D_C)[at] = x[keep].to(torch.bfloat16)
    s["k_pe"].view(-1, D_R)[at] = k[keep].to(torch.bfloat16)
    return s["c_kv"], s["k_pe"]


def _closure(parent):
    """[B, T, T]: whether node t is node i itself or an ancestor of it."""
    B, T = parent.shape
    up = torch.eye(T, device="cuda").expand(B, T, T).clone()
    i = torch.arange(T, device="cuda").expand(B, T)
    b = torch.arange(B, device="cuda").unsqueeze(1).expand(B, T)
    has = parent >= 0
    up[b[has], i[has], parent.long()[has]] = 1.0
    for _ in range(max(1, (T - 1).bit_length())):
        up = (up @ up).clamp(max=1.0)
    return up > 0.5


def _run_attn(s):
    case, q, page = s["case"], s["q"], s["case"]["page"]
    B, T, H, N = case["B"], case["T"], case["H"], s["max_kv"]
    if own:
        import speculative_decoding_tree_absorb_gb300 as kdt
        if "ws" not in s:                   # a server keeps its workspace
            s["ws"] = torch.empty(kdt.verify_attn_paged_workspace_size(B, T, H, N, page, out_dtype=torch.bfloat16),
                                  dtype=torch.uint8, device="cuda")
        return kdt.verify_attn_paged(q[..., :D_C], q[..., D_C:], s["c_kv"], s["k_pe"], s["table"], s["prefix_len"],
                                     parent=s.get("parent"), max_kv_len=N, scale=SCALE, out_dtype=torch.bfloat16,
                                     workspace=s["ws"])
    j = torch.arange(N, device="cuda")
    t = j - s["prefix_len"].unsqueeze(1)                                    # tree index of each key
    at = torch.where(t < T, s["table"].long()[:, j // page] * page + j % page, 0)
    c = s["c_kv"].view(-1, D_C)[at].to(torch.float32)
    k = torch.cat([c, s["k_pe"].view(-1, D_R)[at].to(torch.float32)], -1)
    if T > 1:
        see = torch.gather(_closure(s["parent"]), 2, t.clamp(0, T - 1).unsqueeze(1).expand(B, T, N))
        see = (see & (t < T).unsqueeze(1)) | (t < 0).unsqueeze(1)           # [B, T, N]
    else:
        see = (t < 1).unsqueeze(1)
    x = torch.matmul(q.to(torch.float32).reshape(B, T * H, D_C + D_R), k.transpose(1, 2)) * SCALE
    x = x.view(B, T, H, N).masked_fill_(~see.unsqueeze(2), -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp_(x.sub_(m))
    z = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, T * H, N), c).view(B, T, H, D_C) / z
    return out.to(torch.bfloat16), (m + torch.log(z)).squeeze(-1)


def _column(v, R, dtype):
    """A setting of all rows, or one a row, as [R, 1]."""
    return (v.to(dtype) if torch.is_tensor(v) else torch.full((R,), v, dtype=dtype, device="cuda")).unsqueeze(1)


def _run_sample(s):
    case = s["case"]
    R, V = case["R"], case["V"]
    if own:
        import speculative_decoding_tree_absorb_gb300 as kdt
        return kdt.sample(s["logits"], s["u"], temperature=s["temp"], top_k=s["top_k"], top_p=s["top_p"],
                          min_p=s["min_p"])
    # 64 bits: a threshold falls between two of many thousand tokens' running sums
    temp, top_p, min_p = (_column(s[k], R, torch.float64) for k in ("temp", "top_p", "min_p"))
    top_k = _column(s["top_k"], R, torch.int64)
    top_k = torch.where(top_k > 0, top_k, V)
    y = s["logits"].to(torch.float64)
    y = (y - y.amax(-1, keepdim=True)) / temp
    w = torch.round(torch.exp(y) * WEIGHT_UNIT)
    order = torch.sort(y, dim=-1, descending=True, stable=True).indices     # equal logits: the lower token first
    ws = w.gather(1, order)
    ws = torch.where(torch.arange(V, device="cuda") < top_k, ws, 0.0)
    before = torch.cumsum(ws, -1) - ws                                      # mass in front of each
    keep = ((before < top_p * ws.sum(-1, keepdim=True)) | (top_p >= 1.0)) & (ws >= min_p * WEIGHT_UNIT)
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, 0.0))
    total = torch.cumsum(kept, -1)
    at = s["u"].to(torch.float64).unsqueeze(1) * total[:, -1:]
    token = torch.searchsorted(total, at, right=True).clamp(max=V - 1)
    logp = y.gather(1, token) - torch.log(w.sum(-1, keepdim=True) / WEIGHT_UNIT)
    return token.squeeze(1).to(torch.int32), logp.squeeze(1).to(torch.float32)


def _run_compact(s):
    case, page = s["case"], s["case"]["page"]
    if own:
        import speculative_decoding_tree_absorb_gb300 as kdt
        kdt.kv_compact_paged(s["c_kv"], s["k_pe"], s["table"], s["prefix_len"], s["acc"], s["n_acc"], update_prefix=False)
        return s["c_kv"], s["k_pe"]
    i = torch.arange(case["T"], device="cuda")
    keep = i < s["n_acc"].unsqueeze(1)
    b = torch.arange(case["B"], device="cuda").unsqueeze(1).expand_as(keep)[keep]
    src = (s["prefix_len"].unsqueeze(1) + s["acc"])[keep].long()
    dst = (s["prefix_len"].unsqueeze(1) + i)[keep].long()
    table = s["table"].long()
    src, dst = table[b, src // page] * page + src % page, table[b, dst // page] * page + dst % page
    for a in (s["c_kv"].view(-1, D_C), s["k_pe"].view(-1, D_R)):
        a[dst] = a[src]
    return s["c_kv"], s["k_pe"]


# -------------------------------------------------------------------------------- work --
def work(case):
    """Inputs read once, outputs written once, and the products of the two contractions."""
    op = case["op"]
    if op == "sample":
        esz = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["R"] * (case["V"] * esz + 12), "flops": 4 * case["R"] * case["V"]}
    B, T = case["B"], case["T"]
    row = 2 * (D_C + D_R)
    if op == "assign":
        pages = sum(_pages(n + T, case["page"]) - _pages(n, case["page"]) for n in _lens(case))
        return {"bytes": 4 * B * T + 2 * 8 * pages + 24 * B, "flops": 0}
    if op == "write":
        esz = 2 if case["dtype"] == "bf16" else 4
        n = sum(_new_rows(case))
        return {"bytes": n * ((D_C + D_R) * esz + row + 8), "flops": n * (4 * D_C + 3 * D_R)}
    if op == "attn":
        H, rows = case["H"], B * T * case["H"]
        kv = sum(_lens(case)) + B * T
        seen = T * H * sum(_lens(case)) + rows * (T + 1) / 2
        return {"bytes": kv * row + rows * (row + 2 * D_C + 4), "flops": 2 * seen * (2 * D_C + D_R)}
    return {"bytes": 2 * B * min(case["path"], T) * row, "flops": 0}


# ------------------------------------------------------------------- the definition, 64 bits --
def exact(case, seed):
    if case["op"] == "assign":
        return None                         # whole numbers only
    s = prepare(case, seed)
    return {"write": _exact_write, "attn": _exact_attn, "sample": _exact_sample, "compact": _exact_compact}[case["op"]](case, s)


def _row_of(s, b, j, page):
    """Cache rows of positions j (a list or range) of sequence b."""
    t = s["table"][b].tolist()
    return torch.tensor([t[n // page] * page + n % page for n in j], device="cuda", dtype=torch.int64)


def _exact_write(case, s):
    c_kv, k_pe = s["c_kv"].to(torch.float64), s["k_pe"].to(torch.float64)
    j = torch.arange(D_R // 2, device="cuda", dtype=torch.float64)
    for b, (n, p) in enumerate(zip(_new_rows(case), _lens(case))):
        if n == 0:
            continue
        x = s["kv"][b, :n].to(torch.float64)
        c, k = x[:, :D_C], x[:, D_C:]
        if "gamma" in s:
            c = c / torch.sqrt(torch.sum(c * c, -1, keepdim=True) / D_C + EPS) * s["gamma"].to(torch.float64)
        at = _row_of(s, b, range(p, p + n), case["page"])
        c_kv.view(-1, D_C)[at] = c
        a = torch.outer(torch.arange(p, p + n, device="cuda", dtype=torch.float64), torch.pow(BASE, -j / (D_R // 2)))
        z = torch.polar(torch.ones_like(a), a) * torch.complex(k[:, :D_R // 2].contiguous(), k[:, D_R // 2:].contiguous())
        k_pe.view(-1, D_R)[at] = torch.cat([z.real, z.imag], -1)
    return c_kv, k_pe


def _ancestors(parent):
    """parent: a list; [T, T] truth values, node by node."""
    T = len(parent)
    see = torch.zeros(T, T, dtype=torch.bool)
    for i, p in enumerate(parent):
        if p >= 0:
            see[i] = see[p]
        see[i, i] = True
    return see


def _exact_attn(case, s):
    B, T, H = case["B"], case["T"], case["H"]
    out = torch.empty(B, T, H, D_C, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, T, H, dtype=torch.float64, device="cuda")
    for b, p in enumerate(_lens(case)):
        at = _row_of(s, b, range(p + T), case["page"])
        c, k = s["c_kv"].view(-1, D_C)[at].to(torch.float64), s["k_pe"].view(-1, D_R)[at].to(torch.float64)
        q = s["q"][b].to(torch.float64)
        hide = torch.zeros(T, 1, p + T, dtype=torch.bool, device="cuda")
        hide[:, 0, p:] = ~_ancestors(s["parent"][b].tolist() if T > 1 else [-1]).to("cuda")
        x = SCALE * (q[..., :D_C] @ c.T + q[..., D_C:] @ k.T)
        x = torch.where(hide, -math.inf, x)
        lse[b] = torch.logsumexp(x, -1)
        out[b] = torch.softmax(x, -1) @ c
    return out, lse


def _exact_sample(case, s):
    R, V = case["R"], case["V"]
    token, logp = torch.zeros(R, dtype=torch.int32), torch.zeros(R, dtype=torch.float64)

    def setting(k, r):
        return s[k][r].item() if torch.is_tensor(s[k]) else s[k]
    for r in range(R):
        y = (s["logits"][r].double() - s["logits"][r].max().double()) / setting("temp", r)
        w = torch.floor(torch.exp(y) * WEIGHT_UNIT + 0.5).to(torch.int64)
        # tokens from the most likely down, equal ones in the vocabulary's order
        order = torch.argsort(-y, stable=True)
        k, p, low = setting("top_k", r), setting("top_p", r), setting("min_p", r)
        order = order[:k] if k > 0 else order
        if p < 1.0:
            mass = torch.cumsum(w[order], 0)
            order = order[:int((mass.double() < p * float(mass[-1])).sum()) + 1]
        order = order[w[order].double() >= low * WEIGHT_UNIT]
        left = torch.sort(order).values
        up = torch.cumsum(w[left], 0)
        token[r] = left[min(int((up.double() <= float(s["u"][r].double()) * float(up[-1])).sum()), len(left) - 1)]
        logp[r] = y[int(token[r])] - math.log(float(w.double().sum()) / WEIGHT_UNIT)
    return token, logp


def _exact_compact(case, s):
    c_kv, k_pe = s["c_kv"].to(torch.float64), s["k_pe"].to(torch.float64)
    for b, p in enumerate(_lens(case)):
        path = s["acc"][b, :int(s["n_acc"][b])].tolist()
        src, dst = _row_of(s, b, [p + a for a in path], case["page"]), _row_of(s, b, range(p, p + len(path)), case["page"])
        for t in (c_kv.view(-1, D_C), k_pe.view(-1, D_R)):
            t[dst] = t[src].clone()
    return c_kv, k_pe
