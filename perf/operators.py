"""Measured cases of the 8-bit latent cache and the sampled tree verification.

One step of a tree-speculation server on an 8-bit cache is: quantise the new rows as they
are written (``write``), attend over the cache (``attn``), accept drafted tokens by the
target's probabilities (``sample``), drop the rows of the branches that lost
(``compact``); ``read`` hands rows back in 16 or 32 bits, e.g. to move a sequence to a
16-bit cache. A cache row is 512 e4m3 codes, one power-of-two scale byte (E8M0) for each
32 of them, and 64 bf16 rope values.
"""
import math

import torch

own = False

D_C, D_R, GROUP = 512, 64, 32
SCALE = 1.0 / math.sqrt(192.0)
BASE, EPS = 10000.0, 1e-6
WEIGHT_UNIT = 2.0 ** 44                     # sampling weights are held to 2^-44 of the row's largest


def listed():
    return [
        # the rows of one tree step (64 nodes for each of 8 sequences), bf16 activations
        {"name": "write tree step", "op": "write", "B": 8, "T": 64, "lo": 100, "hi": 2000, "dtype": "bf16",
         "norm": True, "ragged": False},
        # a padded batch of long prompt chunks, fp32 activations
        {"name": "write prompts", "op": "write", "B": 12, "T": 4095, "lo": 0, "hi": 700, "dtype": "f32",
         "norm": True, "ragged": True},
        # a short stretch of every sequence read back, e.g. for a prompt chunk's expanded keys
        {"name": "read stretch", "op": "read", "B": 8, "R": 129, "L": 1500, "dtype": "bf16"},
        # whole sequences moved to a 16-bit cache
        {"name": "read sequences", "op": "read", "B": 8, "R": 8256, "L": 8256, "dtype": "bf16"},
        # the smallest step: a short conversation, few heads; latency counts
        {"name": "attn tiny tree", "op": "attn", "B": 2, "T": 9, "H": 8, "lo": 37, "hi": 37, "out": "bf16"},
        # plain decoding, one token a sequence, ragged contexts: cache bandwidth counts
        {"name": "attn single tokens", "op": "attn", "B": 64, "T": 1, "H": 64, "lo": 1024, "hi": 8192, "out": "bf16"},
        # the batched tree step that the framework's headline workload has
        {"name": "attn tree step", "op": "attn", "B": 8, "T": 64, "H": 64, "lo": 8192, "hi": 8192, "out": "bf16"},
        # few heads (a tensor-parallel share), an odd tree, long ragged contexts
        {"name": "attn long ragged", "op": "attn", "B": 3, "T": 13, "H": 16, "lo": 5000, "hi": 32768, "out": "bf16"},
        # one sequence with a small tree and vocabulary, fp32 logits; latency counts
        {"name": "sample one", "op": "sample", "B": 1, "T": 9, "V": 32000, "dtype": "f32", "agree": 0.7, "temp": 1.0},
        # a batched tree step with a large vocabulary, bf16 logits
        {"name": "sample tree step", "op": "sample", "B": 8, "T": 64, "V": 160000, "dtype": "bf16", "agree": 0.8,
         "temp": 0.8},
        # accepted paths after a usual step
        {"name": "compact step", "op": "compact", "B": 8, "T": 64, "path": 6, "lo": 500, "hi": 3000},
        # many sequences with deep accepted paths
        {"name": "compact deep", "op": "compact", "B": 96, "T": 256, "path": 120, "lo": 100, "hi": 1000},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "attn", "sample", "compact"])
    if op == "write":
        B = rng.randint(1, 16)
        T = _log_int(rng, 1, min(4096, 48000 // B))
        lo = rng.randint(0, 600)
        return {"op": op, "B": B, "T": T, "lo": lo, "hi": lo + rng.randint(0, 1500), "dtype": rng.choice(["bf16", "f32"]),
                "norm": rng.random() < 0.75, "ragged": rng.random() < 0.5}
    if op == "read":
        B = rng.randint(1, 16)
        R = _log_int(rng, 1, 60000 // B)
        return {"op": op, "B": B, "R": R, "L": R + rng.randint(0, 2000), "dtype": rng.choice(["bf16", "f32"])}
    if op == "attn":
        T = rng.choice([1, 1, _log_int(rng, 2, 80)])
        H = rng.choice([1, 8, 16, 20, 32, 64, 128, rng.randint(2, 128)])
        hi = _log_int(rng, 1, 24000)
        lo = rng.randint(0, hi) if rng.random() < 0.6 else hi
        # no dearer than the tree step: rows x keys, and the cache, at most as large
        most = min(64, int(8 * 64 * 64 * 8256 // (T * H * (hi + T))), 500000 // (hi + T))
        return {"op": op, "B": _log_int(rng, 1, max(1, most)), "T": T, "H": H, "lo": lo, "hi": hi,
                "out": "bf16"}
    if op == "sample":
        B, T = _log_int(rng, 1, 32), _log_int(rng, 2, 128)
        V = _log_int(rng, 900, min(160000, 80_000_000 // (B * T)))
        return {"op": op, "B": B, "T": T, "V": V, "dtype": rng.choice(["bf16", "f32"]), "agree": round(rng.uniform(0.2, 0.9), 2),
                "temp": rng.choice([1.0, 0.6, 1.3])}
    T = _log_int(rng, 2, 256)
    lo = rng.randint(0, 800)
    return {"op": op, "B": _log_int(rng, 1, 96), "T": T, "path": rng.randint(1, max(1, T // 2)), "lo": lo,
            "hi": lo + rng.randint(0, 1500)}


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


def _quantise_groups(y):
    """Codes (float8_e4m3fn) and scale bytes of y [..., 512] fp32: one power of two a group of
    32, the least 2^e with max|y| <= 448 * 2^e, e clamped to [-100, 100]."""
    g = y.unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1)
    m, k = torch.frexp(top)
    e = torch.where(m <= 0.875, k - 9, k - 8).clamp(-100, 100)
    e = torch.where(top == 0, torch.full_like(e, -100), e)
    codes = torch.ldexp(g, -e.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.flatten(-2), (e + 127).to(torch.uint8)


def _values(codes, scale):
    return (codes.to(torch.float32).unflatten(-1, (-1, GROUP))
            * torch.ldexp(torch.ones((), device=scale.device), scale.to(torch.int32) - 127).unsqueeze(-1)).flatten(-2)


def _cache(g, B, L):
    """A filled cache: normed latents with a learned weight, as a model leaves them."""
    gamma = 0.5 + torch.rand(D_C, device="cuda", generator=g)
    codes = torch.empty(B, L, D_C, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(B, L, D_C // GROUP, dtype=torch.uint8, device="cuda")
    for b in range(B):
        codes[b], scale[b] = _quantise_groups(torch.randn(L, D_C, device="cuda", generator=g) * gamma)
    k_pe = torch.randn(B, L, D_R, device="cuda", generator=g).to(torch.bfloat16)
    return codes, scale, k_pe


def _tree(g, B, T):
    """Parents with a bias to recent nodes, node 0 the root."""
    back = torch.empty(B, T, device="cuda").exponential_(0.3, generator=g).floor().to(torch.int64) + 1
    i = torch.arange(T, device="cuda").expand(B, T)
    parent = torch.where(i == 0, torch.full_like(i, -1), (i - back).clamp(min=0))
    return parent.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op, B = case["op"], case["B"]
    s = {"case": case}
    if op == "read":
        s["codes"], s["scale"], s["k_pe"] = _cache(g, B, case["L"])
        s["start"] = torch.tensor([(case["L"] - case["R"]) * b // B for b in range(B)], dtype=torch.int32, device="cuda")
        return s
    T = case["T"]
    if op == "sample":
        V = case["V"]
        s["parent"] = _tree(g, B, T)
        tok = torch.randint(0, V, (B, T), device="cuda", generator=g)
        logits = torch.randn(B, T, V, device="cuda", generator=g) * 2.0
        # the target often agrees with a draft: lift a node's children in its row
        p = s["parent"].long().clamp(min=0)
        lift = torch.where(torch.rand(B, T, device="cuda", generator=g) < case["agree"], 16.0, 7.0)
        lift[:, 0] = 0.0
        b = torch.arange(B, device="cuda").unsqueeze(1).expand(B, T)
        logits[b, p, tok] = logits[b, p, tok] * (lift == 0) + lift
        s["logits"] = logits.to(_DT[case["dtype"]])
        s["tok"] = tok.to(torch.int32)
        s["u_node"] = torch.rand(B, T, device="cuda", generator=g)
        s["u_bonus"] = torch.rand(B, device="cuda", generator=g)
        return s
    lens = _lens(case)
    s["prefix_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    L = max(lens) + T + 3
    s["codes"], s["scale"], s["k_pe"] = _cache(g, B, L)
    if op == "write":
        kv = torch.randn(B, T, D_C + D_R, device="cuda", generator=g) * 1.7
        s["kv"] = kv.to(_DT[case["dtype"]])
        if case["norm"]:
            s["gamma"] = (0.5 + torch.rand(D_C, device="cuda", generator=g)).to(_DT[case["dtype"]])
        s["pos"] = (s["prefix_len"].unsqueeze(1) + torch.arange(T, device="cuda")).to(torch.int32)
        if case["ragged"]:
            s["n_rows"] = torch.tensor(_new_rows(case), dtype=torch.int32, device="cuda")
    elif op == "attn":
        s["max_kv"] = max(lens) + T
        s["q"] = torch.randn(B, T, case["H"], D_C + D_R, device="cuda", generator=g).to(torch.bfloat16)
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
def _scale_values(scale):
    return scale.view(torch.float8_e8m0fnu)


def run(s):
    return {"write": _run_write, "read": _run_read, "attn": _run_attn, "sample": _run_sample,
            "compact": _run_compact}[s["case"]["op"]](s)


def _run_write(s):
    case, kv = s["case"], s["kv"]
    T = case["T"]
    if own:
        import speculative_decoding_tree_absorb_gb300 as kdt
        kdt.latent_write_q8(kv[..., :D_C], kv[..., D_C:], s["codes"], s["scale"], s["k_pe"], s["prefix_len"],
                            gamma=s.get("gamma"), eps=EPS, pos=s["pos"], base=BASE, n_rows=s.get("n_rows"))
        return s["codes"], _scale_values(s["scale"]), s["k_pe"]
    x = kv[..., :D_C].to(torch.float32)
    if "gamma" in s:
        x = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * s["gamma"].to(torch.float32)
    codes, scale = _quantise_groups(x)
    freq = BASE ** (-2.0 * torch.arange(D_R // 2, device="cuda", dtype=torch.float64) / D_R)
    a = s["pos"].to(torch.float64).unsqueeze(-1) * freq
    c, n = torch.cos(a).to(torch.float32), torch.sin(a).to(torch.float32)
    k1, k2 = kv[..., D_C:].to(torch.float32).chunk(2, -1)
    k = torch.cat([k1 * c - k2 * n, k2 * c + k1 * n], -1).to(torch.bfloat16)
    i = torch.arange(T, device="cuda")
    rows = s["prefix_len"].long().unsqueeze(1) + i
    b = torch.arange(case["B"], device="cuda").unsqueeze(1).expand_as(rows)
    if "n_rows" in s:
        keep = i < s["n_rows"].unsqueeze(1)
        b, rows, codes, scale, k = b[keep], rows[keep], codes[keep], scale[keep], k[keep]
    s["codes"].view(torch.uint8)[b, rows] = codes.view(torch.uint8)
    s["scale"][b, rows] = scale
    s["k_pe"][b, rows] = k
    return s["codes"], _scale_values(s["scale"]), s["k_pe"]


def _run_read(s):
    case = s["case"]
    if own:
        import speculative_decoding_tree_absorb_gb300 as kdt
        return kdt.latent_read_q8(s["codes"], s["scale"], s["k_pe"], s["start"], case["R"], dtype=_DT[case["dtype"]])
    rows = s["start"].long().unsqueeze(1) + torch.arange(case["R"], device="cuda")
    b = torch.arange(case["B"], device="cuda").unsqueeze(1).expand_as(rows)
    c = _values(s["codes"].view(torch.uint8)[b, rows].view(torch.float8_e4m3fn), s["scale"][b, rows])
    return c.to(_DT[case["dtype"]]), s["k_pe"][b, rows].to(_DT[case["dtype"]])


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
    case, q = s["case"], s["q"]
    B, T, H, N = case["B"], case["T"], case["H"], s["max_kv"]
    dt = _DT[case["out"]]
    if own:
        import speculative_decoding_tree_absorb_gb300 as kdt
        if "ws" not in s:                   # a server keeps its workspace
            s["ws"] = torch.empty(kdt.verify_attn_q8_workspace_size(B, T, H, N, out_dtype=dt), dtype=torch.uint8,
                                  device="cuda")
        return kdt.verify_attn_q8(q[..., :D_C], q[..., D_C:], s["codes"], s["scale"], s["k_pe"], s["prefix_len"],
                                  parent=s["parent"], max_kv_len=N, scale=SCALE, out_dtype=dt, workspace=s["ws"])
    c = _values(s["codes"][:, :N], s["scale"][:, :N])
    k = torch.cat([c, s["k_pe"][:, :N].to(torch.float32)], -1)
    j = torch.arange(N, device="cuda")
    t = j - s["prefix_len"].unsqueeze(1)                                    # tree index of each key
    see = torch.gather(_closure(s["parent"]), 2, t.clamp(0, T - 1).unsqueeze(1).expand(B, T, N))
    see = (see & (t < T).unsqueeze(1)) | (t < 0).unsqueeze(1)               # [B, T, N]
    x = torch.matmul(q.to(torch.float32).reshape(B, T * H, D_C + D_R), k.transpose(1, 2)) * SCALE
    x = x.view(B, T, H, N).masked_fill_(~see.unsqueeze(2), -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp_(x.sub_(m))
    z = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, T * H, N), c).view(B, T, H, D_C) / z
    return out.to(dt), (m + torch.log(z)).squeeze(-1)


def _children(parent, tok):
    """For every node c: mask over earlier siblings, and whether one of those drafts the same token."""
    T = parent.shape[1]
    i = torch.arange(T, device="cuda")
    sib = (parent.unsqueeze(2) == parent.unsqueeze(1)) & (i.unsqueeze(0) < i.unsqueeze(1)) & (parent >= 0).unsqueeze(1)
    return sib, (sib & (tok.unsqueeze(2) == tok.unsqueeze(1))).any(-1)


def _run_sample(s):
    case, parent, tok = s["case"], s["parent"], s["tok"]
    B, T, V = case["B"], case["T"], case["V"]
    if own:
        import speculative_decoding_tree_absorb_gb300 as kdt
        return kdt.tree_sample(parent, tok, s["logits"], s["u_node"], s["u_bonus"], temperature=case["temp"])
    # 64 bits: a threshold falls between two of many thousand tokens' running sums
    y = s["logits"].to(torch.float64)
    y = (y - y.amax(-1, keepdim=True)) / case["temp"]
    w = torch.round(torch.exp(y) * WEIGHT_UNIT)
    z = w.sum(-1)
    b = torch.arange(B, device="cuda").unsqueeze(1).expand(B, T)
    p = parent.long().clamp(min=0)
    wc = w[b, p, tok.long()]
    sib, again = _children(parent, tok)
    rem = z[b, p] - torch.matmul((sib & ~again.unsqueeze(1)).to(torch.float64), wc.unsqueeze(-1)).squeeze(-1)
    take = (s["u_node"].to(torch.float64) * rem < wc) & ~again & (parent >= 0)
    first = take & ~(sib & take.unsqueeze(1)).any(-1)
    first[:, 0] = True
    on = (first.unsqueeze(1) | ~_closure(parent)).all(-1)                   # the whole way from the root was taken
    i = torch.arange(T, device="cuda").expand(B, T)
    n = on.sum(-1)
    path = torch.where(on, i, torch.full_like(i, T)).sort(-1).values
    last = path.gather(1, (n - 1).unsqueeze(1)).squeeze(1)
    row = w[torch.arange(B, device="cuda"), last].clone()
    kid = parent == last.unsqueeze(1)
    row[b[kid], tok.long()[kid]] = 0.0
    total = torch.cumsum(row, -1)
    at = s["u_bonus"].to(torch.float64).unsqueeze(1) * total[:, -1:]
    bonus = torch.searchsorted(total, at, right=True).clamp(max=V - 1).squeeze(1)
    step = path.clamp(max=T - 1)
    after = torch.cat([tok.long().gather(1, step)[:, 1:], torch.zeros(B, 1, dtype=torch.int64, device="cuda")], 1)
    after = torch.where(i == (n - 1).unsqueeze(1), bonus.unsqueeze(1), after)   # the token after each path node
    logp = torch.where(i < n.unsqueeze(1), y[b, step, after] - torch.log(z / WEIGHT_UNIT)[b, step], 0.0)
    return (torch.where(path < T, path, -1).to(torch.int32), n.to(torch.int32), bonus.to(torch.int32),
            logp.to(torch.float32))


def _run_compact(s):
    case = s["case"]
    if own:
        import speculative_decoding_tree_absorb_gb300 as kdt
        kdt.kv_compact_q8(s["codes"], s["scale"], s["k_pe"], s["prefix_len"], s["acc"], s["n_acc"], update_prefix=False)
        return s["codes"], _scale_values(s["scale"]), s["k_pe"]
    i = torch.arange(case["T"], device="cuda")
    keep = i < s["n_acc"].unsqueeze(1)
    b = torch.arange(case["B"], device="cuda").unsqueeze(1).expand_as(keep)[keep]
    src = (s["prefix_len"].unsqueeze(1) + s["acc"])[keep].long()
    dst = (s["prefix_len"].unsqueeze(1) + i)[keep].long()
    codes = s["codes"].view(torch.uint8)
    codes[b, dst] = codes[b, src]
    s["scale"][b, dst] = s["scale"][b, src]
    s["k_pe"][b, dst] = s["k_pe"][b, src]
    return s["codes"], _scale_values(s["scale"]), s["k_pe"]


# -------------------------------------------------------------------------------- work --
def work(case):
    """Inputs read once, outputs written once, and the products of the two contractions."""
    op, B = case["op"], case["B"]
    row8 = D_C + D_C // GROUP + 2 * D_R
    if op == "read":
        esz = 2 if case["dtype"] == "bf16" else 4
        n = B * case["R"]
        return {"bytes": n * (row8 + (D_C + D_R) * esz), "flops": n * D_C}
    T = case["T"]
    if op == "write":
        esz = 2 if case["dtype"] == "bf16" else 4
        n = sum(_new_rows(case))
        return {"bytes": n * ((D_C + D_R) * esz + row8 + 4), "flops": n * (6 * D_C + 3 * D_R)}
    if op == "attn":
        H, rows = case["H"], B * T * case["H"]
        kv = sum(_lens(case)) + B * T
        seen = T * H * sum(_lens(case)) + rows * (T + 1) / 2
        out = 2 if case["out"] == "bf16" else 4
        return {"bytes": kv * row8 + rows * ((D_C + D_R) * 2 + D_C * out + 4), "flops": 2 * seen * (2 * D_C + D_R)}
    if op == "sample":
        # the rows on the way: the root's, and one more for every accepted token (a path cannot be read short)
        esz = 2 if case["dtype"] == "bf16" else 4
        deep = max(1, int(math.log2(T)))
        rows = B * sum(case["agree"] ** k for k in range(deep + 1))
        return {"bytes": rows * case["V"] * esz, "flops": 3 * rows * case["V"]}
    return {"bytes": 2 * B * min(case["path"], T) * row8, "flops": 0}


# ------------------------------------------------------------------- the definition, 64 bits --
def _exact_groups(y):
    """Codes' values and scales of y [N, 512] float64, group by group from the definition."""
    g = y.reshape(-1, D_C // GROUP, GROUP)
    top = g.abs().max(-1).values
    e = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 448.0))
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp(-100, 100)
    x = g / torch.exp2(e).unsqueeze(-1)
    # e4m3: a multiple of 2^(k - 3) for |x| in [2^k, 2^(k + 1)), k at least -6
    k = torch.floor(torch.log2(torch.clamp(x.abs(), min=2.0 ** -6))).clamp(-6, 8)
    unit = torch.exp2(k - 3)
    v = (torch.round(x / unit) * unit).clamp(-448, 448)
    return v.reshape(-1, D_C), torch.exp2(e)


def exact(case, seed):
    s = prepare(case, seed)
    return {"write": _exact_write, "read": _exact_read, "attn": _exact_attn, "sample": _exact_sample,
            "compact": _exact_compact}[case["op"]](case, s)


def _as64(s):
    return (s["codes"].to(torch.float64), torch.exp2(s["scale"].to(torch.float64) - 127.0), s["k_pe"].to(torch.float64))


def _exact_write(case, s):
    codes, scale, k_pe = _as64(s)
    j = torch.arange(D_R // 2, device="cuda", dtype=torch.float64)
    for b in range(case["B"]):
        n, p = _new_rows(case)[b], _lens(case)[b]
        x = s["kv"][b, :n].to(torch.float64)
        c, k = x[:, :D_C], x[:, D_C:]
        if "gamma" in s:
            c = c / torch.sqrt(torch.sum(c * c, -1, keepdim=True) / D_C + EPS) * s["gamma"].to(torch.float64)
        codes[b, p:p + n], scale[b, p:p + n] = _exact_groups(c)
        a = torch.outer(torch.arange(p, p + n, device="cuda", dtype=torch.float64), torch.pow(BASE, -j / (D_R // 2)))
        z = torch.polar(torch.ones_like(a), a) * torch.complex(k[:, :D_R // 2], k[:, D_R // 2:])
        k_pe[b, p:p + n] = torch.cat([z.real, z.imag], -1)
    return codes, scale, k_pe


def _exact_read(case, s):
    codes, scale, k_pe = _as64(s)
    c = codes * scale.repeat_interleave(GROUP, -1)
    at = s["start"].tolist()
    return (torch.stack([c[b, r:r + case["R"]] for b, r in enumerate(at)]),
            torch.stack([k_pe[b, r:r + case["R"]] for b, r in enumerate(at)]))


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
        c = s["codes"][b, :p + T].to(torch.float64)
        c = c * torch.exp2(s["scale"][b, :p + T].to(torch.float64) - 127.0).repeat_interleave(GROUP, -1)
        k = s["k_pe"][b, :p + T].to(torch.float64)
        q = s["q"][b].to(torch.float64)
        hide = torch.zeros(T, 1, p + T, dtype=torch.bool, device="cuda")
        hide[:, 0, p:] = ~_ancestors(s["parent"][b].tolist()).to("cuda")
        x = SCALE * (q[..., :D_C] @ c.T + q[..., D_C:] @ k.T)
        x = torch.where(hide, -math.inf, x)
        lse[b] = torch.logsumexp(x, -1)
        out[b] = torch.softmax(x, -1) @ c
    return out, lse


def _exact_sample(case, s):
    B, T = case["B"], case["T"]
    acc = torch.full((B, T), -1, dtype=torch.int32)
    count, bonus = torch.zeros(B, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    logp = torch.zeros(B, T, dtype=torch.float64)
    for b in range(B):
        parent, tok, u = s["parent"][b].tolist(), s["tok"][b].tolist(), s["u_node"][b].double().tolist()
        node, n = 0, 0
        while True:
            acc[b, n] = node
            y = s["logits"][b, node].to(torch.float64) / case["temp"]
            y = y - y.max()
            w = torch.floor(torch.exp(y) * WEIGHT_UNIT + 0.5)
            ln = y - math.log(float(w.sum()) / WEIGHT_UNIT)
            left, step = w.clone(), None
            for c in range(node + 1, T):
                if parent[c] == node:
                    if u[c] * float(left.sum()) < float(left[tok[c]]):
                        step = c
                        break
                    left[tok[c]] = 0.0
            if step is None:
                break
            logp[b, n] = ln[tok[step]]
            node, n = step, n + 1
        up = torch.cumsum(left, 0)
        bonus[b] = int((up <= float(s["u_bonus"][b].double()) * float(up[-1])).sum())
        logp[b, n] = ln[int(bonus[b])]
        count[b] = n + 1
    return acc, count, bonus, logp


def _exact_compact(case, s):
    codes, scale, k_pe = _as64(s)
    for b, p in enumerate(_lens(case)):
        for t in (codes, scale, k_pe):
            old = t[b].clone()
            for k, node in enumerate(s["acc"][b, :int(s["n_acc"][b])].tolist()):
                t[b, p + k] = old[p + node]
    return codes, scale, k_pe
