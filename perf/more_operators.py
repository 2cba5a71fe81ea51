"""The attention of a verify step over a paged cache, and what stands around it: cases, inputs, plain
forms, exact results.

Four operators, in the order in which a step of tree drafting calls them:
  append   the nodes' keys and values into a cache's pages, with the position rotation of keys and
           queries on the way; a prompt's in the same manner
  attend   attention of the nodes over the cached tokens before them and over their ancestors
  tree     greedy verify of a drafted tree: the path on which the drafts are the target's argmaxes
  keep     the accepted path's tokens moved to the places right after the cached ones

An entry of a step is one sequence and its nodes: row starts[i] + t of the inputs is node t, whose
place in the sequence is lengths[seq] + t.  Node 0 is the token fed before the drafts; parents[row]
is a node's parent, below its own number; a chain's parent is the node before.  A node's position is
lengths[seq] + its depth.  A node sees the cached tokens, its ancestors and itself, with a window W
only those whose position is above its own minus W.  Pages are page_tokens tokens of kv_heads x
head_dim elements; the query heads h * G .. h * G + G - 1 read the key head h, G = q_heads / kv_heads.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # one request, one token, a short context: latency decides
        {"name": "attend_one", "op": "attend", "n": 1, "T": 1, "q_heads": 32, "kv_heads": 8, "D": 128,
         "pt": 16, "lo": 1000, "hi": 1000, "dtype": "bf16", "window": 0, "tree": 0},
        # a served batch with small trees, contexts of all lengths
        {"name": "attend_batch", "op": "attend", "n": 64, "T": 8, "q_heads": 32, "kv_heads": 8,
         "D": 128, "pt": 16, "lo": 300, "hi": 8200, "dtype": "bf16", "window": 0, "tree": 1},
        # one long document: the work has to be split over the tokens
        {"name": "attend_long", "op": "attend", "n": 1, "T": 5, "q_heads": 32, "kv_heads": 8,
         "D": 128, "pt": 64, "lo": 250001, "hi": 250001, "dtype": "bf16", "window": 0, "tree": 0},
        # the widest trees: 512 rows read each key, so that the matrix units decide
        {"name": "attend_wide", "op": "attend", "n": 16, "T": 64, "q_heads": 64, "kv_heads": 8,
         "D": 128, "pt": 32, "lo": 8000, "hi": 16000, "dtype": "bf16", "window": 0, "tree": 1},
        # float32, a head per query head, an odd page, a sliding window, empty contexts among them
        {"name": "attend_f32", "op": "attend", "n": 24, "T": 5, "q_heads": 12, "kv_heads": 12, "D": 64,
         "pt": 7, "lo": 0, "hi": 5000, "dtype": "f32", "window": 2000, "tree": 1},
        # one token of one request
        {"name": "append_one", "op": "append", "n": 1, "T": 1, "q_heads": 32, "kv_heads": 8, "D": 128,
         "rot": 128, "inter": 0, "pt": 16, "lo": 1000, "hi": 1000, "dtype": "bf16", "tree": 0},
        # the nodes of a served batch, far positions among them
        {"name": "append_batch", "op": "append", "n": 256, "T": 9, "q_heads": 32, "kv_heads": 8,
         "D": 128, "rot": 128, "inter": 0, "pt": 16, "lo": 0, "hi": 16000, "dtype": "bf16", "tree": 1},
        # prompts of unequal lengths, part of each head rotated, in pairs of neighbours
        {"name": "append_prompts", "op": "append", "n": 6, "T": 4100, "q_heads": 32, "kv_heads": 8,
         "D": 128, "rot": 64, "inter": 1, "pt": 16, "lo": 0, "hi": 0, "dtype": "bf16", "tree": 0},
        # the smallest tree
        {"name": "tree_small", "op": "tree", "B": 1, "T": 8, "V": 1000, "depth": 4, "dtype": "f32",
         "accept": 0.7},
        # the widest trees of a served batch
        {"name": "tree_large", "op": "tree", "B": 64, "T": 64, "V": 128256, "depth": 8, "dtype": "bf16",
         "accept": 0.7},
        # two layers, one request
        {"name": "keep_small", "op": "keep", "n": 1, "T": 8, "depth": 4, "pools": 4, "elems": 1024,
         "pt": 16, "lo": 1000, "hi": 1000},
        # the keys and values of 32 layers, a served batch
        {"name": "keep_large", "op": "keep", "n": 128, "T": 64, "depth": 8, "pools": 64, "elems": 1024,
         "pt": 16, "lo": 0, "hi": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "tree", "keep"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    pt = rng.choice([1, 5, 8, 16, 32, 64, 100])
    if op == "tree":
        T, V = rng.randint(1, 64), _log(rng, 500, 152064)
        B = _log(rng, 1, max(1, min(64, int(5e8 / (V * T)))))
        return {"op": op, "B": B, "T": T, "V": V, "depth": rng.randint(0, min(10, T - 1)), "dtype": dt,
                "accept": rng.choice([0.3, 0.6, 0.8])}
    if op == "keep":
        T, pools = rng.randint(2, 64), rng.choice([1, 2, 8, 32, 64])
        n = _log(rng, 1, 128)
        return {"op": op, "n": n, "T": T, "depth": rng.randint(1, min(10, T - 1)), "pools": pools,
                "elems": 8 * _log(rng, 4, 256), "pt": pt, "lo": 0, "hi": rng.choice([0, 30])}
    kv, G, D = rng.choice([1, 2, 4, 8, 12]), rng.choice([1, 2, 3, 4, 6, 8]), rng.choice([64, 80, 128, 128, 256])
    case = {"op": op, "q_heads": kv * G, "kv_heads": kv, "D": D, "pt": pt, "dtype": dt}
    if op == "attend":
        T = rng.choice([1, 1, rng.randint(2, 9), rng.randint(2, 64)])
        n = _log(rng, 1, 64)
        # keys and values of a gigabyte; float32 products take longer
        most = min((1 if dt == "f32" else 2) * 1.2e8 / (n * kv * D), (5e7 if dt == "f32" else 3e8) / (n * kv * G * T))
        hi = _log(rng, 16, max(17, min(200000, int(most))))
        return {**case, "n": n, "T": T, "lo": rng.choice([0, hi // 2, hi]), "hi": hi,
                "window": rng.choice([0, 0, 0, max(1, hi // 3)]), "tree": rng.randint(0, 1)}
    tree = rng.randint(0, 1)
    T = rng.choice([1, rng.randint(2, 9), rng.randint(10, 64)]) if tree else _log(rng, 1, 5000)
    n = _log(rng, 1, max(1, min(256, int(3e7 / (T * kv * (G + 2) * D)))))
    hi = rng.choice([0, 100, max(1, min(100000, int(1e8 / (n * kv * D))))])
    return {**case, "n": n, "T": T, "rot": rng.choice([D, D, D // 2, 0]), "inter": rng.randint(0, 1),
            "lo": 0, "hi": hi, "tree": tree}


def _spread(lo, hi, n):
    """n lengths over lo .. hi, the same for each seed up to their order."""
    return [lo + (hi - lo) * (2 * i + 1) // (2 * n) for i in range(n)]


def _counts(case):
    """Nodes of each entry: a prompt's lengths are spread, every fourth tree is smaller."""
    n, T = case["n"], case["T"]
    if T > 64:
        return _spread(T // 8, T, n)
    return [T - (T // 3 if i % 4 == 3 else 0) for i in range(n)]


# ---------------------------------------------------------------------------------- inputs

class _Handle:
    """A handle that lives as long as the state that holds it."""

    def __init__(self, value, destroy):
        self.value, self._destroy = value, destroy

    def __del__(self):
        self._destroy(self.value)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] == "tree":
        _prepare_tree(state, case, g)
    else:
        _prepare_pages(state, case, g)
        {"attend": _prepare_attend, "append": _prepare_append, "keep": _prepare_keep}[case["op"]](state, case, g)
    if own:
        _handles(state, case)
    return state


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def _randint(g, hi, shape):
    """Whole numbers below hi, a tensor of bounds or a number."""
    return (torch.rand(shape, generator=g, device="cuda") * hi).floor().long()


def _parents(n, T, tree, g):
    """[n, T] parents: a chain's, or a tree's in which every other node continues the one before."""
    t = torch.arange(T, device="cuda").expand(n, T)
    if not tree:
        return (t - 1).int().contiguous()
    far = torch.minimum(_randint(g, t, (n, T)), (t - 1).clamp_min(0))
    par = torch.where(torch.rand(n, T, generator=g, device="cuda") < 0.5, t - 1, far)
    par[:, 0] = -1
    return par.int().contiguous()


def _prepare_pages(state, case, g):
    """A cache of 1 to 3 sequences more than the step has entries, its pages in any order."""
    n, pt = case["n"], case["pt"]
    S = n + 1 + n % 3
    perm = lambda k: torch.randperm(k, generator=g, device="cuda")          # noqa: E731
    order = perm(n)
    counts = torch.tensor(_counts(case), device="cuda")
    lens = torch.tensor(_spread(case["lo"], case["hi"], n), device="cuda")[order]
    seqs = perm(S)[:n]
    held = (lens + counts + pt - 1) // pt
    # the sizes go by the case alone
    mb = (case["hi"] + case["T"] + pt - 1) // pt
    P = sum((x + case["T"] + pt - 1) // pt for x in _spread(case["lo"], case["hi"], n)) + 3
    blocks = torch.zeros(S, dtype=torch.long, device="cuda")
    lengths = torch.zeros(S, dtype=torch.long, device="cuda")
    blocks[seqs], lengths[seqs] = held, lens
    before = torch.cumsum(blocks, 0) - blocks
    j = torch.arange(mb, device="cuda")
    pages = perm(P)
    at = (before[:, None] + j).clamp_max(P - 1)
    tables = torch.where(j < blocks[:, None], pages[at], -1)
    refs = torch.zeros(P, dtype=torch.long, device="cuda")
    refs[pages[:int(held.sum().item())]] = 1
    state.update(P=P, S=S, mb=mb, refs=refs.int(), tables=tables.int().contiguous(), blocks=blocks.int(),
                 lengths=lengths.int(), seqs=seqs.int(), counts=counts.int(),
                 starts=(torch.cumsum(counts, 0) - counts).int(), rows=int(counts.sum().item()),
                 longest=int((lens + counts).max().item()))


def _step_rows(state, case, g):
    """Parents by row, and the rows as the model's projection leaves them: q, k and v side by side."""
    n, T = case["n"], case["T"]
    by_entry = _parents(n, T, case["tree"], g)
    alive = torch.arange(T, device="cuda") < state["counts"][:, None]
    state["parents"] = by_entry[alive].contiguous() if case["tree"] else None
    wide = (case["q_heads"] + 2 * case["kv_heads"]) * case["D"]
    x = torch.randn(state["rows"], wide, generator=g, device="cuda").to(DTYPES[case["dtype"]])
    a, b = case["q_heads"] * case["D"], (case["q_heads"] + case["kv_heads"]) * case["D"]
    state.update(wide=wide, q=x[:, :a], k=x[:, a:b], v=x[:, b:])


def _pools(state, case, g, num, elems):
    dt = DTYPES[case.get("dtype", "bf16")]
    return torch.randn(num, state["P"], case["pt"] * elems, generator=g, device="cuda", dtype=dt)


def _prepare_attend(state, case, g):
    _step_rows(state, case, g)
    state["pools"] = _pools(state, case, g, 2, case["kv_heads"] * case["D"])
    state["scale"] = 1.0 / math.sqrt(case["D"])


def _prepare_append(state, case, g):
    _step_rows(state, case, g)
    state["pools"] = _pools(state, case, g, 2, case["kv_heads"] * case["D"])
    half = case["rot"] // 2
    state["inv_freq"] = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float32) / max(half, 1))


def _moves(case):
    """Accepted drafts of each entry, and how many of the first of them stay where they are.  A path's
    other nodes come from behind all destinations, so that the same moves give the same again."""
    got = []
    for i, m in enumerate(_counts(case)):
        acc = min(case["depth"] - i % (case["depth"] + 1), m - 1)
        same = i * 5 // (case["depth"] + 1) % (acc + 1)
        got.append((same + min(acc - same, max(0, m - case["depth"] - 1)), same))
    return got


def _prepare_keep(state, case, g):
    n, T, depth = case["n"], case["T"], case["depth"]
    state["pools"] = _pools(state, case, g, case["pools"], case["elems"])
    behind = torch.rand(n, T, generator=g, device="cuda").tolist()
    paths = []
    for (acc, same), m, w in zip(_moves(case), _counts(case), behind):
        more = sorted(sorted(range(depth + 1, m), key=w.__getitem__)[:acc - same])
        paths.append([*range(same + 1), *more, *[-1] * (depth - acc)])
    state["path"] = _i32(paths)
    state["accepted"] = _i32([a for a, _ in _moves(case)])


def _prepare_tree(state, case, g):
    B, T, V, dt = case["B"], case["T"], case["V"], DTYPES[case["dtype"]]
    par = _parents(B, T, 1, g)
    tok = _randint(g, V, (B, T))
    # a node's best id is one of its children's with probability `accept`
    t = torch.arange(T, device="cuda")
    child = (par.long()[:, None, :] == t[None, :, None]) & (t > 0)
    pick = (child * torch.rand(B, T, T, generator=g, device="cuda")).argmax(2)
    hit = child.any(2) & (torch.rand(B, T, generator=g, device="cuda") < case["accept"])
    best = torch.where(hit, tok.gather(1, pick), _randint(g, V, (B, T)))
    x = torch.empty(B, T, V, dtype=dt, device="cuda")
    for b in range(0, B, 8):
        x[b:b + 8] = torch.randn(min(B, b + 8) - b, T, V, generator=g, device="cuda")
    x.scatter_(2, best[:, :, None], 8.0)
    state.update(logits=x, tokens=tok.int(), parents=par,
                 counts=_i32([T - (T // 3 if b % 4 == 3 else 0) for b in range(B)]))


def _handles(state, case):
    from rejection_sampling_verification_row_amd import binding as sv
    state["sv"] = sv
    dt = sv.SPECVERIFY_F32 if case.get("dtype") == "f32" else sv.SPECVERIFY_BF16
    if case["op"] == "tree":
        B, T, D1 = case["B"], case["T"], case["depth"] + 1
        state.update(h=_Handle(sv.specverify_create(0, B, T - 1, case["V"]), sv.specverify_destroy),
                     dt=dt, out=tuple(torch.empty(s, dtype=torch.int32, device="cuda")
                                      for s in ((B,), (B, D1), (B, D1))))
        return
    pools = state["pools"]
    size = pools[0, 0].numel() * pools.element_size()
    state["c"] = _Handle(sv.specverify_cache_create(
        0, state["P"], case["pt"], state["S"], state["mb"], size, [pools[i] for i in range(len(pools))],
        state["refs"], state["tables"], state["blocks"], state["lengths"]), sv.specverify_cache_destroy)
    if case["op"] == "keep":
        return
    n, T = case["n"], case["T"]
    state["h"] = _Handle(sv.specverify_attn_create(state["c"].value, dt, case["q_heads"],
                                                   case["kv_heads"], case["D"], n, min(T, 64)),
                         sv.specverify_attn_destroy)
    state["nodes"] = sv.SpecVerifyNodes(seqs=state["seqs"], starts=state["starts"],
                                        counts=state["counts"], parents=state["parents"])
    state["out"] = torch.empty(state["rows"], case["q_heads"], case["D"], dtype=DTYPES[case["dtype"]],
                               device="cuda")
    if case["op"] == "attend":
        state["lse"] = torch.empty(state["rows"], case["q_heads"], device="cuda")
    else:
        state["rotation"] = sv.SpecVerifyRotation(state["inv_freq"], case["rot"], case["inter"])


# ---------------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if op == "attend":
        return _own_attend(state) if own else _plain_attend(state)
    if op == "append":
        return _own_append(state) if own else _plain_append(state)
    if op == "tree":
        return _own_tree(state) if own else _plain_tree(state)
    return _own_keep(state) if own else _plain_keep(state)


def _own_attend(s):
    c = s["case"]
    s["sv"].specverify_attn_attend(s["h"].value, None, 0, 1, c["n"], c["T"], s["rows"], s["nodes"],
                                   s["scale"], c["window"], s["q"], s["wide"], s["out"],
                                   c["q_heads"] * c["D"], s["lse"])
    return s["out"], s["lse"]


def _own_append(s):
    c = s["case"]
    s["sv"].specverify_attn_append(s["h"].value, None, 0, 1, c["n"], c["T"], s["rows"], s["nodes"],
                                   s["rotation"], s["k"], s["wide"], s["v"], s["wide"], s["q"],
                                   s["wide"], s["out"], c["q_heads"] * c["D"])
    return s["out"], s["pools"]


def _own_tree(s):
    c, (acc, path, tok) = s["case"], s["out"]
    s["sv"].specverify_run_greedy_tree(s["h"].value, None, s["dt"], c["B"], c["T"], c["V"], c["depth"],
                                       s["logits"], s["tokens"], s["parents"], s["counts"], acc, path,
                                       tok)
    return acc, path, tok


def _own_keep(s):
    c = s["case"]
    s["sv"].specverify_cache_keep_path(s["c"].value, None, c["n"], c["depth"] + 1, s["seqs"],
                                       s["accepted"], s["path"])
    return s["pools"].view(torch.int16)


# ---------------------------------------------------------------------------------- plain forms

def _ancestors(s):
    """[n, T, T] whether node j is node t or an ancestor of it, and [n, T] depths."""
    n, T = s["case"]["n"], s["case"]["T"]
    t = torch.arange(T, device="cuda")
    par = (t - 1).expand(n, T)
    if s["parents"] is not None:
        row = s["starts"].long()[:, None] + t
        par = s["parents"].long()[row.clamp_max(s["rows"] - 1)]
    step = ((par[:, :, None] == t) & (t[:, None] > 0)).double()
    anc = torch.linalg.matrix_power(torch.eye(T, dtype=torch.float64, device="cuda") + step, T) > 0
    return anc, anc.sum(2) - 1


def _slots(s, places):
    """Places [n, m] of the entries' sequences as numbers of tokens in a pool; -1: no page."""
    pt, tab = s["case"]["pt"], s["tables"].long()[s["seqs"].long()]
    pg = tab.gather(1, (places // pt).clamp(0, s["mb"] - 1))
    return torch.where(pg >= 0, pg * pt + places % pt, -1)


def _plain_attend(s):
    c = s["case"]
    n, T, H, Hk, D, W = c["n"], c["T"], c["q_heads"], c["kv_heads"], c["D"], c["window"]
    G, L = H // Hk, s["longest"]
    lens, counts = s["lengths"].long()[s["seqs"].long()], s["counts"].long()
    j, t = torch.arange(L, device="cuda"), torch.arange(T, device="cuda")
    slot = _slots(s, j.expand(n, L)).clamp_min(0)
    k, v = (p.view(-1, Hk, D)[slot].float().permute(0, 2, 1, 3) for p in s["pools"])
    row = (s["starts"].long()[:, None] + t).clamp_max(s["rows"] - 1)
    q = s["q"].reshape(-1, Hk, G, D)[row].float().permute(0, 2, 1, 3, 4).reshape(n, Hk, T * G, D)
    anc, depth = _ancestors(s)
    # [n, T, L]: cached tokens within the window, then ancestors within it
    node = (j - lens[:, None]).clamp(0, T - 1)
    seen = anc.gather(2, node[:, None, :].expand(n, T, L))
    at = torch.where(j < lens[:, None], j, lens[:, None] + depth.gather(1, node))
    seen = torch.where(j < lens[:, None, None], True, seen) & (j < (lens + counts)[:, None, None])
    if W:
        seen &= at[:, None, :] > (lens[:, None] + depth)[:, :, None] - W
    x = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["scale"])
    x = x.view(n, Hk, T, G, L).masked_fill_(~seen[:, None, :, None, :], -math.inf).view(n, Hk, T * G, L)
    top = x.amax(3, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    x = x.sub_(top).exp_()
    z = x.sum(3, keepdim=True)
    o = torch.matmul(x, v.contiguous()) / z
    lse = (z.log() + top)[..., 0].view(n, Hk, T, G).permute(0, 2, 1, 3).reshape(n, T, H)
    o = o.view(n, Hk, T, G, D).permute(0, 2, 1, 3, 4).reshape(n, T, H, D)
    alive = t < counts[:, None]
    return o[alive].to(s["q"].dtype), lse[alive]


def _rotated(x, cos, sin, inter):
    """x [..., D] with its first 2 * cos.shape[-1] elements rotated, in 32 bits."""
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if inter else (x[..., :half], x[..., half:2 * half])
    u, w = a * cos - b * sin, b * cos + a * sin
    head = torch.stack((u, w), -1).flatten(-2) if inter else torch.cat((u, w), -1)
    return torch.cat((head, x[..., 2 * half:]), -1)


def _entry_rows(s):
    """Entry and node of each row."""
    counts = s["counts"].long()
    entry = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), counts,
                                    output_size=s["rows"])
    return entry, torch.arange(s["rows"], device="cuda") - s["starts"].long()[entry]


def _plain_append(s):
    c = s["case"]
    H, Hk, D, dt = c["q_heads"], c["kv_heads"], c["D"], s["q"].dtype
    entry, node = _entry_rows(s)
    lens = s["lengths"].long()[s["seqs"].long()]
    depth = node if s["parents"] is None else _ancestors(s)[1][entry, node]
    ang = (lens[entry] + depth).double()[:, None] * s["inv_freq"].double()
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    q = _rotated(s["q"].float().view(-1, H, D), cos, sin, c["inter"]).to(dt)
    k = _rotated(s["k"].float().view(-1, Hk, D), cos, sin, c["inter"]).to(dt)
    pt = c["pt"]
    place = lens[entry] + node
    slot = s["tables"].long()[s["seqs"].long()[entry], place // pt] * pt + place % pt
    s["pools"][0].view(-1, Hk, D)[slot] = k
    s["pools"][1].view(-1, Hk, D)[slot] = s["v"].reshape(-1, Hk, D)
    return q, s["pools"]


def _plain_tree(s):
    c = s["case"]
    B, T, D1 = c["B"], c["T"], c["depth"] + 1
    best = s["logits"].float().argmax(2)
    t = torch.arange(T, device="cuda")
    # follows[b, i]: the first child of node i that holds its best id, T: none
    fits = (s["parents"].long()[:, None, :] == t[:, None]) & (t > 0) & (t < s["counts"][:, None, None])
    fits &= s["tokens"].long()[:, None, :] == best[:, :, None]
    follows = torch.where(fits, t, T).amin(2)
    follows = torch.cat((follows, torch.full((B, 1), T, device="cuda")), 1)
    path = torch.zeros(B, D1, dtype=torch.long, device="cuda")
    for j in range(1, D1):
        path[:, j] = follows.gather(1, path[:, j - 1:j])[:, 0]
    on = path < T
    tok = torch.where(on, best.gather(1, path.clamp_max(T - 1)), -1)
    return (on.sum(1) - 1).int(), torch.where(on, path, -1).int(), tok.int()


def _plain_keep(s):
    c = s["case"]
    j = torch.arange(c["depth"] + 1, device="cuda")
    lens = s["lengths"].long()[s["seqs"].long()][:, None]
    moved = (j > 0) & (j <= s["accepted"].long()[:, None])
    src = _slots(s, lens + s["path"].long().clamp_min(0))[moved]
    dst = _slots(s, (lens + j).expand_as(s["path"]))[moved]
    p = s["pools"].view(c["pools"], -1, c["elems"])
    p[:, dst] = p[:, src]
    return s["pools"].view(torch.int16)


# ---------------------------------------------------------------------------------- exact results

def _see(parents, count, window):
    """For each node its depth and the nodes that it sees, from its parents one by one."""
    depth, seen = [0] * count, []
    for t in range(count):
        chain, at = [t], t
        while at > 0:
            at = int(parents[at]) if parents is not None else at - 1
            chain.append(at)
        depth[t] = len(chain) - 1
        seen.append([a for i, a in enumerate(chain) if not window or i < window])
    return depth, seen


def _places(s, i):
    """Pool places of entry i's tokens, cached ones and nodes, in order."""
    c, q = s["case"], int(s["seqs"][i])
    total = int(s["lengths"][q]) + int(s["counts"][i])
    pages = s["tables"][q, :(total + c["pt"] - 1) // c["pt"]].long()
    inside = torch.arange(c["pt"], device=pages.device)
    return (pages[:, None] * c["pt"] + inside).reshape(-1)[:total]


def exact(case, seed):
    if case["op"] == "keep":
        return None                      # copies: nothing is computed
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(s)
    c = case
    H, Hk, D = c["q_heads"], c["kv_heads"], c["D"]
    G = H // Hk
    par = None if s["parents"] is None else s["parents"].cpu()
    starts, counts = s["starts"].tolist(), s["counts"].tolist()
    lens = s["lengths"][s["seqs"].long()].tolist()
    q64 = s["q"].double().reshape(-1, H, D)
    if c["op"] == "attend":
        out = torch.zeros_like(q64)
        lse = torch.zeros(len(q64), H, dtype=torch.float64, device="cuda")
        for i in range(c["n"]):
            a, m, ln = starts[i], counts[i], lens[i]
            depth, seen = _see(None if par is None else par[a:a + m], m, c["window"])
            at = _places(s, i)
            k, v = (p.view(-1, Hk, D)[at].double() for p in s["pools"])
            ok = torch.zeros(m, len(at), dtype=torch.bool)
            for t in range(m):
                low = max(0, ln + depth[t] - c["window"] + 1) if c["window"] else 0
                ok[t, low:ln] = True
                ok[t, [ln + b for b in seen[t]]] = True
            ok = ok.cuda()
            for h in range(Hk):
                x = q64[a:a + m, h * G:(h + 1) * G].reshape(m * G, D) @ k[:, h].T.contiguous()
                x = (x * s["scale"]).view(m, G, -1).masked_fill(~ok[:, None], -math.inf)
                z = torch.logsumexp(x, 2)
                lse[a:a + m, h * G:(h + 1) * G] = z
                w = torch.exp(x - z[..., None])
                out[a:a + m, h * G:(h + 1) * G] = (w.view(m * G, -1) @ v[:, h].contiguous()).view(m, G, D)
        return out, lse
    pools = s["pools"].double()
    half = c["rot"] // 2
    freq = s["inv_freq"].double()
    for i in range(c["n"]):
        a, m, ln = starts[i], counts[i], lens[i]
        depth = list(range(m)) if par is None else _see(par[a:a + m], m, 0)[0]
        pos = torch.tensor(depth, dtype=torch.float64, device="cuda") + ln
        turn = torch.polar(torch.ones(m, half, dtype=torch.float64, device="cuda"), pos[:, None] * freq)
        k64 = s["k"][a:a + m].double().reshape(m, Hk, D)
        for x in (q64[a:a + m], k64):
            if not half:
                continue
            pair = x[..., :c["rot"]].reshape(m, -1, half, 2) if c["inter"] else \
                x[..., :c["rot"]].reshape(m, -1, 2, half).transpose(2, 3)
            r = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[:, None])
            x[..., :c["rot"]] = (r if c["inter"] else r.transpose(2, 3)).reshape(m, -1, c["rot"])
        at = _places(s, i)[ln:]
        pools[0].view(-1, Hk, D)[at] = k64
        pools[1].view(-1, Hk, D)[at] = s["v"][a:a + m].double().reshape(m, Hk, D)
    return q64, pools


def _exact_tree(s):
    c = s["case"]
    best = s["logits"].double().cpu() if s["logits"].numel() < 1 << 26 else None
    par, tok, counts = s["parents"].tolist(), s["tokens"].tolist(), s["counts"].tolist()
    acc, paths, toks = [], [], []
    for b in range(c["B"]):
        at, path, out = 0, [0], []
        while True:
            row = best[b, at] if best is not None else s["logits"][b, at].double().cpu()
            g = int((row == row.max()).nonzero()[0, 0])
            out.append(g)
            nxt = [i for i in range(1, counts[b]) if par[b][i] == at and tok[b][i] == g]
            if not nxt or len(path) > c["depth"]:
                break
            at = nxt[0]
            path.append(at)
        fill = [-1] * (c["depth"] + 1 - len(path))
        acc.append(len(path) - 1)
        paths.append(path + fill)
        toks.append(out + fill)
    return tuple(torch.tensor(x, dtype=torch.int32) for x in (acc, paths, toks))


# ---------------------------------------------------------------------------------- the least work

def work(case):
    es = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if case["op"] == "tree":
        # the rows on the path: the root's, and one more for each accepted draft
        rows = case["B"] * sum(case["accept"] ** j for j in range(case["depth"] + 1))
        return {"bytes": rows * case["V"] * es + case["B"] * 4 * (2 * case["T"] + 2 * case["depth"] + 4),
                "flops": rows * case["V"]}
    n, counts = case["n"], _counts(case)
    rows = sum(counts)
    if case["op"] == "keep":
        moved = sum(a - same for a, same in _moves(case))
        return {"bytes": 2 * moved * case["pools"] * case["elems"] * 2 + n * 4 * (case["depth"] + 4),
                "flops": n}
    Hq, Hk, D = case["q_heads"], case["kv_heads"], case["D"]
    if case["op"] == "append":
        move = 2 * rows * (Hq + 2 * Hk) * D * es
        return {"bytes": move + 12 * n + 4 * rows, "flops": 3 * rows * (Hq + Hk) * case["rot"]}
    lens = _spread(case["lo"], case["hi"], n)
    if case["window"]:
        lens = [min(x, case["window"] - 1) for x in lens]
    mean = sum(lens) / n
    read = (sum(lens) + rows) * 2 * Hk * D * es
    return {"bytes": read + 2 * rows * Hq * D * es + 4 * rows * Hq + 4 * (sum(lens) + rows) // case["pt"],
            "flops": 4 * Hq * D * rows * (mean + 4)}
