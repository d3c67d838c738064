"""Operators that read the paged cache under a mask of their own, as cases to be measured: attention
of a tree of drafted tokens, the commit of its accepted path, and decoding over a few blocks of a long
context: the bounds of the blocks' keys, the selection by a score against them, the attention over
the selected blocks.  Each case computes its operator in a plain torch form, or, where `own` is set,
through the package's calls."""
import math
import random

import torch

own = False

# Trees of n_lo..n_hi drafted tokens (the root, which is a token that stands, counted) of `seqs`
# sequences, behind p_lo..p_hi tokens of context.
TREE = [
    # one user's speculation over a short chat, where latency counts
    dict(name="tree_small", op="tree", seqs=1, n_lo=8, n_hi=8, p_lo=300, p_hi=300,
         hq=32, hkv=8, d=128, bs=16, type="bf16", cache="same", pick=1),
    # a serving batch that verifies a tree for each of its sequences
    dict(name="tree_batch", op="tree", seqs=24, n_lo=20, n_hi=64, p_lo=500, p_hi=6000,
         hq=32, hkv=8, d=128, bs=16, type="bf16", cache="same", pick=2),
    # trees behind very long contexts
    dict(name="tree_far", op="tree", seqs=4, n_lo=48, n_hi=63, p_lo=50000, p_hi=62000,
         hq=64, hkv=8, d=128, bs=32, type="f16", cache="same", pick=3),
]

# The accepted path of each tree, and its rows of every layer's pools moved together.
COMMIT = [
    # one sequence, a draft model of two layers
    dict(name="commit_small", op="commit", seqs=1, n_lo=8, n_hi=8, p_lo=300, p_hi=300, layers=2,
         hkv=8, d=128, bs=16, type="bf16", pick=4),
    # a batch of 64 sequences and 32 layers
    dict(name="commit_layers", op="commit", seqs=64, n_lo=16, n_hi=64, p_lo=50, p_hi=300, layers=32,
         hkv=8, d=128, bs=16, type="bf16", pick=5),
]

# Bounds of the blocks that hold n_lo..n_hi new tokens behind p_lo..p_hi.
BOUNDS = [
    # after a decode step: one new token per sequence
    dict(name="bounds_step", op="bounds", seqs=32, n_lo=1, n_hi=1, p_lo=500, p_hi=4000,
         hkv=8, d=128, bs=16, type="bf16", pick=6),
    # after prompts
    dict(name="bounds_prompt", op="bounds", seqs=5, n_lo=6000, n_hi=15000, p_lo=0, p_hi=100,
         hkv=8, d=128, bs=16, type="f16", pick=7),
]

# Selection of `keep` blocks (the first `first` and the last `last` among them) for each query token
# and kv head.
SELECT = [
    # a few sequences of ordinary length
    dict(name="select_step", op="select", seqs=4, q_len=1, p_lo=3000, p_hi=8000, keep=64, first=1, last=4,
         hq=32, hkv=8, d=128, bs=16, type="bf16", pick=8),
    # a batch of long contexts
    dict(name="select_far", op="select", seqs=20, q_len=1, p_lo=60000, p_hi=131072, keep=128, first=1, last=8,
         hq=32, hkv=8, d=128, bs=16, type="bf16", pick=9),
]

# Attention over selected blocks.
SPARSE = [
    # one user behind a long document
    dict(name="sparse_small", op="sparse", seqs=1, q_len=1, p_lo=9000, p_hi=9000, keep=64, first=1, last=4,
         hq=32, hkv=8, d=128, bs=16, type="bf16", cache="same", pick=10),
    # a batch behind long contexts
    dict(name="sparse_batch", op="sparse", seqs=48, q_len=1, p_lo=12000, p_hi=32000, keep=128, first=1, last=8,
         hq=32, hkv=8, d=128, bs=16, type="bf16", cache="same", pick=11),
    # two query tokens each over an 8-bit cache
    dict(name="sparse_fp8", op="sparse", seqs=40, q_len=2, p_lo=8000, p_hi=20000, keep=96, first=2, last=4,
         hq=64, hkv=8, d=128, bs=32, type="bf16", cache="fp8", pick=12),
]

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
K_SCALE, V_SCALE = 0.03125, 0.015625   # of the 8-bit pools: |values| up to 14 and 7 are held


def listed():
    return [dict(c) for c in TREE + COMMIT + BOUNDS + SELECT + SPARSE]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "commit", "bounds", "select", "sparse", "sparse"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        hkv = rng.choice([1, 2, 3, 4, 8, 16])
        base = dict(op=op, hkv=hkv, d=rng.choice([64, 128]), bs=rng.choice([16, 32]), type=rng.choice(["bf16", "f16"]),
                    pick=rng.randint(100, 10 ** 6))
        heads = hkv * rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if g * hkv <= 64])
        fp8 = rng.random() < 0.3
        if op == "tree":
            n, p = _log(rng, 1, 160), _log(rng, 1, 60000)
            c = dict(base, hq=heads, seqs=_log(rng, 1, 40), n_lo=max(1, n // 2), n_hi=n, p_lo=p // 4, p_hi=p,
                     cache="fp8" if fp8 and base["d"] == 128 else "same")
        elif op == "commit":
            n = _log(rng, 1, 160)
            c = dict(base, seqs=_log(rng, 1, 100), n_lo=max(1, n // 2), n_hi=n, p_lo=0, p_hi=_log(rng, 1, 400),
                     layers=_log(rng, 1, 48), type="fp8" if fp8 else base["type"])
        elif op == "bounds":
            n = rng.choice([1, _log(rng, 1, 10000)])
            c = dict(base, seqs=_log(rng, 1, 64), n_lo=max(1, n // 3), n_hi=n, p_lo=0, p_hi=_log(rng, 1, 4000),
                     type="fp8" if fp8 else base["type"])
        else:
            p = _log(rng, 100, 131072)
            keep = _log(rng, 4, 256)
            first = rng.randint(0, 2)
            c = dict(base, hq=heads, seqs=_log(rng, 1, 48), q_len=rng.choice([1, 1, 1, 2, 3, 5]), p_lo=p // 3 + 5, p_hi=p,
                     keep=keep, first=first, last=rng.randint(0, min(keep - first, 8)))
            if op == "sparse":
                c["cache"] = "fp8" if fp8 and base["d"] == 128 else "same"
        # no more work than the largest listed case of the operator, and pools and scores of ordinary size
        lens = _lengths(c)
        rows = max(n * l for n, l in lens) * c.get("hq", 0)
        if (_cost(c) <= most and rows <= 2 ** 29
                and sum(l for _, l in lens) * hkv * c["d"] * c.get("layers", 1) <= (2 ** 31 if op != "select" else 2 ** 33)):
            return c


def _lengths(c):
    """New tokens (or query tokens) and context length, the new ones counted, of each sequence."""
    r = random.Random(c["pick"])
    got = []
    for _ in range(c["seqs"]):
        n = c["q_len"] if "q_len" in c else r.randint(c["n_lo"], c["n_hi"])
        got.append((n, n + r.randint(c["p_lo"], c["p_hi"])))
    return got


def _trees(c):
    """Parents of each tree's nodes (-1 for the root) and the nodes of its accepted path.  The path's
    nodes past the root stand behind the places that they move to."""
    r = random.Random(c["pick"] + 1)
    got = []
    for n, _ in _lengths(c):
        longest = min((n + 1) // 2, 9)
        take = r.randint(1, longest)
        path = [0] + sorted(r.sample(range(take, n), take - 1))
        parents = [-1] + [r.randrange(max(0, i - 12), i) for i in range(1, n)]
        for a, b in zip(path, path[1:]):
            parents[b] = a
        got.append((parents, path))
    return got


def work(c):
    lens = _lengths(c)
    item = 1 if c.get("cache") == "fp8" or c["type"] == "fp8" else 2
    if c["op"] == "tree":
        q = sum(n for n, _ in lens)
        seen = 0
        for (n, l), (parents, _) in zip(lens, _trees(c)):
            depth = []
            for p in parents:
                depth.append(1 if p < 0 else depth[p] + 1)
            seen += n * (l - n) + sum(depth)
        moved = sum(l for _, l in lens) * c["hkv"] * c["d"] * 2 * item + 2 * q * c["hq"] * c["d"] * 2
        masks = sum(-(-n // 32) * 4 * n for n, _ in lens)
        tables = 4 * sum(-(-l // c["bs"]) for _, l in lens)
        return {"bytes": moved + masks + tables, "flops": 4 * c["d"] * c["hq"] * seen}
    if c["op"] == "commit":
        rows = sum(sum(j != i for j, i in enumerate(path)) for _, path in _trees(c))
        tokens = sum(n for n, _ in lens)
        masks = sum(-(-n // 32) * 4 * n for n, _ in lens)
        return {"bytes": 4 * rows * c["layers"] * c["hkv"] * c["d"] * item + 16 * tokens + masks, "flops": tokens}
    if c["op"] == "bounds":
        # the rows of every block that holds a new token, and what is written for it
        rows = blocks = 0
        for n, l in lens:
            first = (l - n) // c["bs"]
            rows += l - first * c["bs"]
            blocks += -(-l // c["bs"]) - first
        return {"bytes": c["hkv"] * (rows * c["d"] * item + blocks * (2 * c["d"] + 4)), "flops": 2 * rows * c["hkv"] * c["d"]}
    if c["op"] == "select":
        read = written = scored = 0
        for n, l in lens:
            seen = [-(-(l - n + j + 1) // c["bs"]) for j in range(n)]
            mid = [max(s - c["first"] - c["last"], 0) if s > c["keep"] else 0 for s in seen]
            read += max(mid)
            scored += sum(mid)
            written += n * c["keep"]
        b = read * c["hkv"] * (2 * c["d"] + 4) + 4 * written * c["hkv"] + 2 * len(lens) * c["q_len"] * c["hq"] * c["d"]
        return {"bytes": b, "flops": 4 * scored * c["hkv"] * c["d"]}
    tokens, q = _selected_tokens(c), len(lens) * c["q_len"]
    moved = tokens * c["hkv"] * c["d"] * 2 * item
    return {"bytes": moved + 4 * q * c["hq"] * c["d"] + 4 * q * c["hkv"] * c["keep"],
            "flops": 4 * tokens * c["hq"] * c["d"]}


def _selected_tokens(c):
    """Tokens of the selected blocks, per kv head (the last block, which may end early, among them)."""
    total = 0
    for n, l in _lengths(c):
        for j in range(n):
            seen = l - n + j + 1
            blocks = -(-seen // c["bs"])
            if c["last"] or blocks <= c["keep"]:
                total += (min(blocks, c["keep"]) - 1) * c["bs"] + (seen - (blocks - 1) * c["bs"])
            else:
                total += c["keep"] * c["bs"]
    return total


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, g, kind):
    """N(0, 1) values, made in pieces of bounded size."""
    out = torch.empty(shape, dtype=kind, device="cuda")
    flat = out.view(-1)
    for at in range(0, flat.numel(), 2 ** 28):
        part = flat[at:at + 2 ** 28]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    return out


def _pool(shape, g, kind, scale):
    """A pool of N(0, 1) rows in the cache's type."""
    if kind == "fp8":
        x = _normal(shape, g, torch.float16)
        return (x / scale).to(torch.float8_e4m3fn).view(torch.uint8)
    return _normal(shape, g, TYPES[kind])


def _cells(c, g, lens):
    """A block table over blocks in random order, lengths, and the blocks of the pool."""
    need = [-(-l // c["bs"]) for _, l in lens]
    ids = torch.randperm(sum(need) + sum(need) // 10 + 1, generator=g, device="cuda").to(torch.int32)
    at = torch.zeros(len(lens), max(need), dtype=torch.int64)
    keep = torch.zeros(len(lens), max(need), dtype=torch.bool)
    first = 0
    for s, n in enumerate(need):
        at[s, :n] = torch.arange(first, first + n)
        keep[s, :n] = True
        first += n
    tables = torch.where(keep.cuda(), ids[at.cuda()], -1).to(torch.int32).contiguous()
    lens_d = torch.tensor([l for _, l in lens], dtype=torch.int32, device="cuda")
    return tables, lens_d, len(ids)


def _starts(lens):
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    return starts


def _masks(c, trees):
    """Bit i of word w of a node's row: the node sees node 32 w + i of its tree."""
    words = max(-(-len(p) // 32) for p, _ in trees)
    rows = []
    for parents, _ in trees:
        seen = []
        for i, p in enumerate(parents):
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        rows += [[(m >> 32 * w) & 0xFFFFFFFF for w in range(words)] for m in seen]
    return torch.tensor(rows, dtype=torch.int64).to(torch.int32).cuda()


def prepare(c, seed):
    g = _generator(seed)
    lens = _lengths(c)
    s = dict(case=c, lens=lens, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    s["tables"], s["lens_d"], blocks = _cells(c, g, lens)
    s["longest"] = max(l for _, l in lens)
    s["starts"] = _starts(lens)
    s["starts_d"] = torch.tensor(s["starts"], dtype=torch.int32, device="cuda")
    hkv, d, bs = c["hkv"], c["d"], c["bs"]
    shape = (blocks, hkv, bs, d)
    cache = "fp8" if c.get("cache") == "fp8" else c["type"]
    if c["op"] == "tree":
        s.update(q=_normal((s["starts"][-1], c["hq"], d), g, TYPES[c["type"]]), masks=_masks(c, _trees(c)),
                 k=_pool(shape, g, cache, K_SCALE), v=_pool(shape, g, cache, V_SCALE), scale=d ** -0.5)
        s["out"] = torch.zeros_like(s["q"])
    elif c["op"] == "commit":
        trees = _trees(c)
        total = s["starts"][-1]
        # the model's choices; drafted tokens that differ from them off the accepted paths
        target = torch.randint(0, 32000, (total,), generator=g, device="cuda")
        parent = torch.tensor([max(p, 0) + a for (parents, _), a in zip(trees, s["starts"]) for p in parents])
        taken = torch.zeros(total, dtype=torch.bool)
        for (_, path), a in zip(trees, s["starts"]):
            taken[[a + i for i in path]] = True
        wrong = torch.randint(1, 32000, (total,), generator=g, device="cuda")
        draft = (target[parent.cuda()] + torch.where(taken.cuda(), 0, wrong)) % 32000
        s["pools"] = _pool((c["layers"], 2) + shape, g, c["type"], K_SCALE)
        s["keys"] = [s["pools"][i, 0] for i in range(c["layers"])]
        s["values"] = [s["pools"][i, 1] for i in range(c["layers"])]
        s.update(target=target, draft=draft, masks=_masks(c, trees), most=16)
        s["accepted"] = torch.zeros(c["seqs"], s["most"], dtype=torch.int32, device="cuda")
        s["count"] = torch.zeros(c["seqs"], dtype=torch.int32, device="cuda")
        s["next"] = torch.zeros(c["seqs"], dtype=torch.int64, device="cuda")
        s["new_lens"] = torch.zeros(c["seqs"], dtype=torch.int32, device="cuda")
    elif c["op"] == "bounds":
        s["k"] = _pool(shape, g, c["type"], K_SCALE)
        s["new"] = max(n for n, _ in lens)
        s["bounds"] = torch.zeros((blocks, hkv, 2, d), dtype=torch.int8, device="cuda")
        s["steps"] = torch.zeros((blocks, hkv), device="cuda")
        # the blocks that hold new tokens, for the plain form: sequence, block
        touched = [(i, b) for i, (n, l) in enumerate(lens) for b in range((l - n) // bs, -(-l // bs))]
        s["touched"] = torch.tensor(touched, device="cuda").t().contiguous()
    elif c["op"] == "select":
        s["q"] = _normal((c["seqs"], c["q_len"], c["hq"], d), g, TYPES[c["type"]])
        # each head's dimensions have a place of their own, around which the blocks' keys spread
        place = 30 * torch.randn((hkv, d), generator=g, device="cuda")
        s["bounds"] = torch.empty((blocks, hkv, 2, d), dtype=torch.int8, device="cuda")
        for a in range(0, blocks, 8192):
            part = s["bounds"][a:a + 8192]
            for i, sign in ((0, 1), (1, -1)):
                wide = torch.randn(part[:, :, 0].shape, generator=g, device="cuda").mul_(8).add_(25)
                part[:, :, i] = wide.mul_(sign).add_(place).round_().clamp_(-127, 127).to(torch.int8)
        s["steps"] = 2.0 ** torch.randint(-6, -4, (blocks, hkv), generator=g, device="cuda").float()
        s["chosen"] = torch.zeros((c["seqs"], c["q_len"], hkv, c["keep"]), dtype=torch.int32, device="cuda")
    else:
        s.update(q=_normal((c["seqs"], c["q_len"], c["hq"], d), g, TYPES[c["type"]]),
                 k=_pool(shape, g, cache, K_SCALE), v=_pool(shape, g, cache, V_SCALE), scale=d ** -0.5)
        s["out"] = torch.zeros_like(s["q"])
        score = torch.rand((c["seqs"], c["q_len"], hkv, s["tables"].shape[1]), generator=g, device="cuda")
        s["chosen"] = _best(score, _seen(s), c)
    return s


def _seen(s):
    """Tokens that each query token sees: [sequences, query tokens]."""
    n = s["case"]["q_len"]
    return s["lens_d"].long()[:, None] - n + 1 + torch.arange(n, device="cuda")


def _best(score, seen, c):
    """The blocks of each row [.., blocks]: the first and last ones of its context and the best of the
    others, ties to the lowest index, in ascending order, then -1."""
    blocks = (seen + c["bs"] - 1) // c["bs"]
    at = torch.arange(score.shape[-1], device=score.device)
    blocks = blocks[..., None, None]
    score = score.masked_fill((at < c["first"]) | (at >= blocks - c["last"]), math.inf)
    score = score.masked_fill(at >= blocks, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :c["keep"]]
    if order.shape[-1] < c["keep"]:
        order = torch.nn.functional.pad(order, (0, c["keep"] - order.shape[-1]), value=score.shape[-1])
    order = torch.where(order < blocks, order, 2 ** 30).sort(-1).values
    return torch.where(order < 2 ** 30, order, -1).to(torch.int32)


def run(s):
    return {"tree": _tree, "commit": _commit, "bounds": _bounds, "select": _select, "sparse": _sparse}[s["case"]["op"]](s)


def _workspace(s, need):
    """The program's workspace, made on its first call."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(need(), 256), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _values(x, cache, scale):
    return x.view(torch.float8_e4m3fn).float() * scale if cache == "fp8" else x.float()


def _tree(s):
    c = s["case"]
    if own:
        import paged_kv_cache_187_gb300 as pa
        ws = _workspace(s, lambda: pa.pa_decode_tree_workspace_size(
            s["q"].shape[0], len(s["lens"]), c["hq"], c["hkv"], c["d"], s["longest"]))
        args = (s["out"], s["q"], s["k"], s["v"], s["tables"], s["lens_d"], s["starts_d"], s["masks"], s["longest"],
                s["scale"])
        if c["cache"] == "fp8":
            pa.pa_decode_tree_fp8(*args, K_SCALE, V_SCALE, workspace=ws, status=s["status"])
        else:
            pa.pa_decode_tree(*args, workspace=ws, status=s["status"])
        return s["out"]
    hkv, d, g = c["hkv"], c["d"], c["hq"] // c["hkv"]
    bit = torch.arange(32, device="cuda", dtype=torch.int32)
    for i, (n, length) in enumerate(s["lens"]):
        rows = slice(s["starts"][i], s["starts"][i + 1])
        ids = s["tables"][i, :-(-length // c["bs"])].long()
        k, v = (_values(p[ids], c["cache"], scale).transpose(0, 1).reshape(hkv, 1, -1, d)[:, :, :length]
                for p, scale in ((s["k"], K_SCALE), (s["v"], V_SCALE)))
        q = s["q"][rows].float().view(n, hkv, g, d).permute(1, 2, 0, 3)
        scores = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])          # [hkv, g, n, length]
        sees = ((s["masks"][rows, :, None] >> bit) & 1).flatten(1)[:, :n].bool()
        scores[..., length - n:].masked_fill_(~sees, -math.inf)
        scores.sub_(scores.amax(-1, keepdim=True)).exp_()
        o = torch.matmul(scores, v).div_(scores.sum(-1, keepdim=True))
        s["out"][rows] = o.permute(2, 0, 1, 3).reshape(n, c["hq"], d).to(s["out"].dtype)
    return s["out"]


def _commit(s):
    c = s["case"]
    if own:
        import paged_kv_cache_187_gb300 as pa
        pa.pa_tree_accept(s["accepted"], s["count"], s["next"], s["new_lens"], s["draft"], s["target"], s["masks"],
                          s["starts_d"], s["lens_d"], status=s["status"])
        pa.pa_move_tokens(s["keys"], s["values"], s["tables"], s["new_lens"], s["accepted"], s["count"],
                          status=s["status"])
        return s["accepted"], s["count"], s["next"], s["new_lens"], _held(s["pools"])
    # the trees side by side: [sequences, nodes]
    S, n = c["seqs"], max(m for m, _ in s["lens"])
    starts = s["starts_d"].long()
    size = starts[1:] - starts[:-1]
    at = (starts[:-1, None] + torch.arange(n, device="cuda")).clamp_max(s["starts"][-1] - 1)
    here = torch.arange(n, device="cuda") < size[:, None]
    bit = torch.arange(32, device="cuda", dtype=torch.int32)
    sees = ((s["masks"][:, :, None] >> bit) & 1).flatten(1)[:, :n].bool()[at]    # [S, n, n]
    if sees.shape[-1] < n:
        sees = torch.nn.functional.pad(sees, (0, n - sees.shape[-1]))
    i = torch.arange(n, device="cuda")
    above = sees & (i[None, :] < i[:, None]) & here[..., None]
    parent = torch.where(above, i, -1).amax(-1)                                   # -1: none
    draft, target = s["draft"][at], s["target"][at]
    agrees = (parent >= 0) & (draft == target.gather(1, parent.clamp_min(0))) & here
    agrees[:, 0] = here[:, 0]
    # the path of each node: its ancestors, all of which have to agree
    depth = above.sum(-1)
    good = here & agrees & ~(above & ~agrees[:, None, :]).any(-1)
    best = torch.where(good, depth * n + (n - 1 - i), -1).amax(-1)
    last = n - 1 - best % n
    on = (above | (i[None, :] == i[:, None]))[torch.arange(S, device="cuda"), last] & (best >= 0)[:, None]
    order = torch.where(on, i, n).sort(-1).values
    order = torch.nn.functional.pad(order, (0, max(0, s["most"] - n)), value=n)[:, :s["most"]]
    s["accepted"].copy_(torch.where(order < n, order, -1))
    s["count"].copy_(on.sum(-1).clamp_max(s["most"]))
    count = s["count"].long()
    end = s["accepted"].long().gather(1, (count - 1).clamp_min(0)[:, None])
    s["next"].copy_(torch.where(count > 0, target.gather(1, end.clamp_min(0))[:, 0], -1))
    s["new_lens"].copy_(s["lens_d"] - size + count)
    base = (s["lens_d"].long() - size)[:, None]
    j = torch.arange(s["most"], device="cuda")
    used = j < count[:, None]
    # (places without a node: the root's row over itself)
    src = (base + torch.where(used, s["accepted"], 0)).clamp_min(0)
    dst = (base + torch.where(used, j, 0)).clamp_min(0)
    bs = c["bs"]
    sb, db = s["tables"].gather(1, src // bs).long(), s["tables"].gather(1, dst // bs).long()
    s["pools"][:, :, db, :, dst % bs] = s["pools"][:, :, sb, :, src % bs]
    return s["accepted"], s["count"], s["next"], s["new_lens"], _held(s["pools"])


def _held(pool):
    """A pool's values: 8-bit ones in units of their scale."""
    return pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool


def _exponent(x):
    """floor(log2 x), -100 at least, of x >= 0."""
    return torch.frexp(x.clamp_min(2.0 ** -100)).exponent - 1


def _power(e):
    """2^e, exactly."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _bounds(s):
    c = s["case"]
    if own:
        import paged_kv_cache_187_gb300 as pa
        pa.pa_key_bounds(s["bounds"], s["steps"], s["k"], s["tables"], s["lens_d"], s["new"],
                         query_starts=s["starts_d"], status=s["status"])
        return s["bounds"], s["steps"]
    bs = c["bs"]
    row, col = s["touched"]
    filled = (s["lens_d"].long()[row] - col * bs).clamp_max(bs)
    block = s["tables"][row, col].long()
    for a in range(0, len(block), 4096):
        b = block[a:a + 4096]
        k = _held(s["k"])[b].float()                                               # [n, hkv, bs, d]
        past = (torch.arange(bs, device="cuda") >= filled[a:a + 4096, None])[:, None, :, None]
        step = _power(_exponent(k.masked_fill(past, 0).abs().amax((2, 3))).clamp_max(96) - 6)
        x = (k / step[..., None, None]).round().clamp(-127, 127)
        s["bounds"][b, :, 0] = x.masked_fill(past, -math.inf).amax(2).to(torch.int8)
        s["bounds"][b, :, 1] = x.masked_fill(past, math.inf).amin(2).to(torch.int8)
        s["steps"][b] = step
    return s["bounds"], s["steps"]


def _select(s):
    c = s["case"]
    if own:
        import paged_kv_cache_187_gb300 as pa
        ws = _workspace(s, lambda: pa.pa_select_blocks_workspace_size(c["seqs"], c["q_len"], c["hkv"], c["bs"], s["longest"]))
        pa.pa_select_blocks(s["chosen"], s["q"], s["bounds"], s["steps"], s["tables"], s["lens_d"], c["bs"], s["longest"],
                            c["first"], c["last"], workspace=ws, status=s["status"])
        return s["chosen"]
    S, n, hkv, d = c["seqs"], c["q_len"], c["hkv"], c["d"]
    q = s["q"].float().view(S, n, hkv, -1, d)
    q = (q / _power(_exponent(q.abs().amax((3, 4), keepdim=True)) - 5)).round()
    up, down = q.clamp_min(0).sum(3), q.clamp_max(0).sum(3)                        # [S, n, hkv, d], whole numbers
    score = torch.empty((S, n, hkv, s["tables"].shape[1]), device="cuda")
    for i in range(S):
        ids = s["tables"][i].long().clamp_min(0)
        b = s["bounds"][ids].float().permute(1, 2, 3, 0)                           # [hkv, 2, d, blocks]
        sums = torch.matmul(up[i].transpose(0, 1), b[:, 0]) + torch.matmul(down[i].transpose(0, 1), b[:, 1])
        score[i] = (sums * s["steps"][ids].t()[:, None]).transpose(0, 1)
    s["chosen"].copy_(_best(score, _seen(s), c))
    return s["chosen"]


def _sparse(s):
    c = s["case"]
    if own:
        import paged_kv_cache_187_gb300 as pa
        ws = _workspace(s, lambda: pa.pa_decode_sparse_workspace_size(
            c["seqs"], c["q_len"], c["hq"], c["hkv"], c["d"], c["bs"], c["keep"]))
        args = (s["out"], s["q"], s["k"], s["v"], s["tables"], s["lens_d"], s["chosen"], s["scale"])
        if c["cache"] == "fp8":
            pa.pa_decode_sparse_fp8(*args, K_SCALE, V_SCALE, workspace=ws, status=s["status"])
        else:
            pa.pa_decode_sparse(*args, workspace=ws, status=s["status"])
        return s["out"]
    S, n, hkv, d, bs = c["seqs"], c["q_len"], c["hkv"], c["d"], c["bs"]
    seen = _seen(s)
    for i in range(S):
        pick = s["chosen"][i].long()                                               # [n, hkv, keep]
        ids = s["tables"][i][pick.clamp_min(0)].long()
        head = torch.arange(hkv, device="cuda")[None, :, None]
        k, v = (_values(p[ids, head], c["cache"], scale).reshape(n, hkv, -1, d)
                for p, scale in ((s["k"], K_SCALE), (s["v"], V_SCALE)))
        pos = pick[..., None] * bs + torch.arange(bs, device="cuda")
        hide = ((pick < 0)[..., None] | (pos >= seen[i][:, None, None, None])).flatten(2)
        q = s["q"][i].float().view(n, hkv, -1, d)
        scores = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(hide[:, :, None], -math.inf)
        scores.sub_(scores.amax(-1, keepdim=True)).exp_()
        o = torch.matmul(scores, v).div_(scores.sum(-1, keepdim=True))
        s["out"][i] = o.view(n, c["hq"], d).to(s["out"].dtype)
    return s["out"]


def exact(c, seed):
    """From the definitions, in 64 bits."""
    if c["op"] in ("tree", "sparse") and work(c)["flops"] > 2e12:
        return None
    if c["op"] == "select" and work(c)["flops"] / c["d"] > 1.2e8:      # (query token, head, block) scores, four each
        return None
    s = prepare(c, seed)
    hkv, bs, d = c["hkv"], c["bs"], c["d"]
    if c["op"] == "tree":
        g = c["hq"] // hkv
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for i, ((n, length), (parents, _)) in enumerate(zip(s["lens"], _trees(c))):
            sees = torch.ones(n, length, dtype=torch.bool)
            for a in range(n):
                sees[a, length - n:] = False
                b = a
                while b >= 0:
                    sees[a, length - n + b] = True
                    b = parents[b]
            sees = sees.cuda()
            ids = s["tables"][i, :-(-length // bs)].long()
            for h in range(hkv):
                k, v = (_values(p[ids, h], c["cache"], 1.0).double().reshape(-1, d)[:length] for p in (s["k"], s["v"]))
                if c["cache"] == "fp8":
                    k, v = k * K_SCALE, v * V_SCALE
                for j in range(h * g, (h + 1) * g):
                    x = s["q"][s["starts"][i]:s["starts"][i + 1], j].double() @ k.t() * s["scale"]
                    out[s["starts"][i]:s["starts"][i + 1], j] = torch.softmax(x.masked_fill(~sees, -math.inf), -1) @ v
        return out
    if c["op"] == "commit":
        draft, target = s["draft"].tolist(), s["target"].tolist()
        accepted = torch.full((c["seqs"], s["most"]), -1, dtype=torch.int32)
        count, following, new_lens = [], [], []
        pools = s["pools"].clone()
        for i, ((n, length), (parents, _)) in enumerate(zip(s["lens"], _trees(c))):
            a = s["starts"][i]
            paths = {0: [0]}
            for b in range(1, n):
                if parents[b] in paths and draft[a + b] == target[a + parents[b]]:
                    paths[b] = paths[parents[b]] + [b]
            path = max(paths.values(), key=lambda p: (len(p), -p[-1]))[:s["most"]]
            accepted[i, :len(path)] = torch.tensor(path)
            count.append(len(path))
            following.append(target[a + path[-1]])
            new_lens.append(length - n + len(path))
            table = s["tables"][i].tolist()
            for j, b in enumerate(path):
                to, at = length - n + j, length - n + b
                pools[:, :, table[to // bs], :, to % bs] = s["pools"][:, :, table[at // bs], :, at % bs]
        return (accepted, torch.tensor(count, dtype=torch.int32), torch.tensor(following),
                torch.tensor(new_lens, dtype=torch.int32), _held(pools))
    if c["op"] == "bounds":
        bounds, steps = s["bounds"].clone(), s["steps"].clone()
        for i, (n, length) in enumerate(s["lens"]):
            lo = (length - n) // bs
            ids = s["tables"][i, lo:-(-length // bs)].long()
            k = _held(s["k"])[ids].double()
            valid = torch.arange(lo * bs, lo * bs + len(ids) * bs, device="cuda").view(-1, 1, bs, 1) < length
            k0 = torch.where(valid, k, 0.0)
            step = torch.exp2(torch.floor(torch.log2(k0.abs().amax((2, 3)).clamp_min(2.0 ** -100))).clamp(-100, 96) - 6)
            x = torch.clamp(torch.round(k / step[..., None, None]), -127, 127)
            bounds[ids, :, 0] = torch.where(valid, x, -1000.0).amax(2).to(torch.int8)
            bounds[ids, :, 1] = torch.where(valid, x, 1000.0).amin(2).to(torch.int8)
            steps[ids] = step.float()
        return bounds, steps
    if c["op"] == "select":
        chosen = torch.empty(s["chosen"].shape, dtype=torch.int32)
        g = c["hq"] // hkv
        for i, (n, length) in enumerate(s["lens"]):
            ids = s["tables"][i, :-(-length // bs)].long()
            hi, lo = (s["bounds"][ids, :, a].double() * s["steps"][ids].double()[..., None] for a in (0, 1))
            for j in range(n):
                blocks = -(-(length - n + j + 1) // bs)
                q = s["q"][i, j].double().view(hkv, g, d)
                top = q.abs().amax((1, 2)).clamp_min(2.0 ** -100)
                q = torch.round(q * torch.exp2(5 - torch.floor(torch.log2(top)))[:, None, None])
                score = torch.zeros(blocks, hkv, dtype=torch.float64, device="cuda")
                for r in range(g):
                    score += torch.maximum(q[:, r] * hi[:blocks], q[:, r] * lo[:blocks]).sum(-1)
                for h, row in enumerate(score.t().tolist()):
                    if blocks <= c["keep"]:
                        got = list(range(blocks))
                    else:
                        got = list(range(c["first"])) + list(range(blocks - c["last"], blocks))
                        middle = sorted(range(c["first"], blocks - c["last"]), key=lambda b: (-row[b], b))
                        got = sorted(got + middle[:c["keep"] - len(got)])
                    chosen[i, j, h] = torch.tensor(got + [-1] * (c["keep"] - len(got)))
        return chosen
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    g = c["hq"] // hkv
    for i, (n, length) in enumerate(s["lens"]):
        for j in range(n):
            limit = length - n + j + 1
            for h in range(hkv):
                got = s["chosen"][i, j, h]
                got = got[got >= 0].long()
                seen = (got[:, None] * bs + torch.arange(bs, device="cuda")).view(-1) < limit
                k, v = (_values(p[s["tables"][i, got].long(), h], c["cache"], 1.0).double().reshape(-1, d)[seen]
                        for p in (s["k"], s["v"]))
                if c["cache"] == "fp8":
                    k, v = k * K_SCALE, v * V_SCALE
                x = s["q"][i, j, h * g:(h + 1) * g].double() @ k.t() * s["scale"]
                out[i, j, h * g:(h + 1) * g] = torch.softmax(x, -1) @ v
    return out
