"""The chunk operators of the paged cache, as cases to be measured: attention of a ragged batch of
new tokens over the cache, rotary positions fused with the write into the cache, and the moving of
blocks when a pool shrinks.  Each case computes its operator in a plain torch form, or, where `own`
is set, through the package's calls."""
import math
import random

import torch

own = False

# Attention of new tokens over the cache: `chunks` sequences with q_lo..q_hi new tokens and `singles`
# sequences with one, each behind p_lo..p_hi tokens that are in the cache already.
ATTENTION = [
    # the smallest call: one short continuation of a chat, where latency counts
    dict(name="chunk_short", op="attention", chunks=1, singles=0, q_lo=17, q_hi=17, p_lo=300, p_hi=300,
         hq=32, hkv=8, d=128, bs=16, type="bf16", cache="same", pick=1),
    # a serving step: two prompts' chunks beside 61 sequences that decode one token each
    dict(name="chunk_mixed", op="attention", chunks=2, singles=61, q_lo=400, q_hi=900, p_lo=200, p_hi=4000,
         hq=32, hkv=8, d=128, bs=16, type="bf16", cache="same", pick=2),
    # a whole long prompt in one call
    dict(name="prompt_long", op="attention", chunks=1, singles=0, q_lo=8192, q_hi=8192, p_lo=0, p_hi=0,
         hq=32, hkv=8, d=128, bs=16, type="bf16", cache="same", pick=3),
    # a few tokens each behind very long contexts: few rows, the work has to be split along the context
    dict(name="chunk_far", op="attention", chunks=4, singles=0, q_lo=20, q_hi=28, p_lo=50000, p_hi=62000,
         hq=64, hkv=8, d=128, bs=32, type="f16", cache="same", pick=4),
    # short prompts of odd lengths, one query head per kv head, head size 64
    dict(name="prompts_mha64", op="attention", chunks=9, singles=0, q_lo=37, q_hi=1500, p_lo=0, p_hi=0,
         hq=16, hkv=16, d=64, bs=16, type="f16", cache="same", pick=5),
    # chunks of long prompts over an 8-bit cache
    dict(name="chunk_fp8", op="attention", chunks=2, singles=3, q_lo=1000, q_hi=1100, p_lo=9000, p_hi=14000,
         hq=32, hkv=8, d=128, bs=16, type="bf16", cache="fp8", pick=6),
]

# Rotary positions and the write into the cache: `tokens` new tokens with `axes` position axes.
ROPE = [
    # a decode step of three sequences
    dict(name="rope_step", op="rope", tokens=3, axes=1, hq=32, hkv=8, d=128, rot=128, bs=16,
         interleaved=False, type="bf16", cache="same"),
    # text around images: time, height and width positions, q / k / v slices of one fused projection
    dict(name="rope_image", op="rope", tokens=8200, axes=3, hq=32, hkv=8, d=128, rot=128, bs=16,
         interleaved=False, type="bf16", cache="same"),
    # half of the dimensions rotated in adjacent pairs, into an 8-bit cache
    dict(name="rope_fp8", op="rope", tokens=4099, axes=1, hq=32, hkv=8, d=128, rot=64, bs=16,
         interleaved=True, type="f16", cache="fp8"),
]

# Moving blocks to lower places in every layer's pools, and the tables with them.
MOVE = [
    # a handful of blocks of a small pool
    dict(name="move_few", op="move", layers=4, pairs=7, blocks=64, seqs=5, hkv=8, d=128, bs=16, type="bf16"),
    # a pool of 32 layers that gives back two fifths of its blocks
    dict(name="move_layers", op="move", layers=32, pairs=201, blocks=512, seqs=64, hkv=8, d=128, bs=16,
         type="bf16"),
]

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
K_SCALE, V_SCALE = 0.03125, 0.015625   # of the 8-bit pools: |values| up to 14 and 7 are held


def listed():
    return [dict(c) for c in ATTENTION + ROPE + MOVE]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    most = max(_cost(c) for c in ATTENTION)
    op = rng.choice(["attention", "attention", "attention", "rope", "move"])
    hkv = rng.choice([1, 2, 3, 4, 8, 16])
    hq = hkv * rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if g * hkv <= 64])
    d = rng.choice([64, 128])
    bs = rng.choice([16, 32])
    kind = rng.choice(["bf16", "f16"])
    if op == "rope":
        axes = rng.choice([1, 2, 3, 4])
        return dict(op="rope", tokens=_log(rng, 1, 16384), axes=axes, hq=hq, hkv=hkv, d=d,
                    rot=16 * rng.randint(2, d // 16), bs=bs, interleaved=rng.random() < 0.4, type=kind,
                    cache=rng.choice(["same", "fp8"]))
    if op == "move":
        layers = _log(rng, 1, 48)
        pairs = _log(rng, 1, 6400 // max(layers, 16))
        return dict(op="move", layers=layers, pairs=pairs, blocks=2 * pairs + rng.randint(3, 99),
                    seqs=_log(rng, 1, 200), hkv=min(hkv, 8), d=d, bs=bs, type=rng.choice(["bf16", "f16", "fp8"]))
    cache = "fp8" if d == 128 and rng.random() < 0.3 else "same"
    while True:
        q, p = _log(rng, 1, 4096), _log(rng, 1, 60000) - 1
        c = dict(op="attention", chunks=_log(rng, 1, 24), singles=rng.choice([0, 0, rng.randint(1, 40)]),
                 q_lo=max(1, q // 3), q_hi=q, p_lo=p // 4, p_hi=p, hq=hq, hkv=hkv, d=d, bs=bs, type=kind,
                 cache=cache, pick=rng.randint(100, 10 ** 6))
        # no more work than the largest listed case, and scores that the plain form can hold
        if (_cost(c) <= most and max(n * n_q * l for n_q, n, l in _groups(c)) * hq <= 2 ** 31
                and max(n * l for _, n, l in _groups(c)) * hkv * d <= 2 ** 31):
            return c


def _lengths(c):
    """New tokens and context length (the new ones counted) of each sequence, in a mixed order."""
    r = random.Random(c["pick"])
    seqs = [r.randint(c["q_lo"], c["q_hi"]) for _ in range(c["chunks"])] + [1] * c["singles"]
    r.shuffle(seqs)
    return [(n, n + r.randint(c["p_lo"], c["p_hi"])) for n in seqs]


def _groups(c):
    """(new tokens, sequences with so many, their longest context)."""
    lens = _lengths(c)
    return [(n, sum(m == n for m, _ in lens), max(l for m, l in lens if m == n))
            for n in sorted({m for m, _ in lens})]


def work(c):
    if c["op"] == "attention":
        lens = _lengths(c)
        q = sum(n for n, _ in lens)
        item = 1 if c["cache"] == "fp8" else 2
        seen = sum(n * l - n * (n - 1) // 2 for n, l in lens)     # (token, context token) pairs
        moved = sum(l for _, l in lens) * c["hkv"] * c["d"] * 2 * item + 2 * q * c["hq"] * c["d"] * 2
        tables = 4 * sum(-(-l // c["bs"]) for _, l in lens)
        return {"bytes": moved + tables, "flops": 4 * c["d"] * c["hq"] * seen}
    if c["op"] == "rope":
        item = 1 if c["cache"] == "fp8" else 2
        per = 4 * c["hq"] * c["d"] + 2 * c["hkv"] * c["d"] * (2 + item) + 8 * c["axes"] + 4
        return {"bytes": c["tokens"] * per, "flops": 3 * c["tokens"] * (c["hq"] + c["hkv"]) * c["rot"]}
    item = 1 if c["type"] == "fp8" else 2
    block = c["hkv"] * c["bs"] * c["d"] * item
    return {"bytes": 4 * c["layers"] * c["pairs"] * block + 8 * c["blocks"], "flops": 0}


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, g, kind):
    return torch.randn(shape, generator=g, device="cuda").to(kind)


def _pool(shape, g, kind, scale):
    """A pool of N(0, 1) rows in the cache's type."""
    if kind == "fp8":
        return (torch.randn(shape, generator=g, device="cuda") / scale).to(torch.float8_e4m3fn).view(torch.uint8)
    return _normal(shape, g, TYPES[kind])


def prepare(c, seed):
    g = _generator(seed)
    if c["op"] == "attention":
        lens = _lengths(c)
        bs, total = c["bs"], sum(n for n, _ in lens)
        need = [-(-l // bs) for _, l in lens]
        places = torch.randperm(sum(need) + sum(need) // 10 + 1, generator=g, device="cuda").to(torch.int32)
        tables = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
        at, ids = 0, places.cpu()
        for s, n in enumerate(need):
            tables[s, :n] = ids[at:at + n]
            at += n
        starts = [0]
        for n, _ in lens:
            starts.append(starts[-1] + n)
        cache = c["type"] if c["cache"] == "same" else "fp8"
        shape = (len(places), c["hkv"], bs, c["d"])
        groups = []      # the sequences with as many new tokens each, for the plain form
        for n, _, longest in _groups(c):
            at = torch.tensor([i for i, (m, _) in enumerate(lens) if m == n], device="cuda")
            groups.append((n, at, -(-longest // bs)))
        return dict(case=c, lens=lens, starts=starts, groups=groups, longest=max(l for _, l in lens), scale=c["d"] ** -0.5,
                    q=_normal((total, c["hq"], c["d"]), g, TYPES[c["type"]]),
                    k=_pool(shape, g, cache, K_SCALE), v=_pool(shape, g, cache, V_SCALE),
                    out=torch.zeros((total, c["hq"], c["d"]), dtype=TYPES[c["type"]], device="cuda"),
                    tables=tables.cuda(), lens_d=torch.tensor([l for _, l in lens], dtype=torch.int32, device="cuda"),
                    starts_d=torch.tensor(starts, dtype=torch.int32, device="cuda"),
                    status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if c["op"] == "rope":
        t, hq, hkv, d, bs = c["tokens"], c["hq"], c["hkv"], c["d"], c["bs"]
        blocks = -(-t // bs) + 3
        qkv = _normal((t, hq + 2 * hkv, d), g, TYPES[c["type"]])
        cache = c["type"] if c["cache"] == "same" else "fp8"
        if c["axes"] == 1:      # a text far into its context
            first = int(torch.randint(0, 100000, (1,), generator=g, device="cuda"))
            positions = (torch.arange(t, device="cuda") + first)[None]
        else:                   # frames of 24 x 36 patches: the axes count frames, rows, columns, and so on
            i = torch.arange(t, device="cuda") + int(torch.randint(0, 9000, (1,), generator=g, device="cuda"))
            positions = torch.stack([i // 864, i // 36 % 24, i % 36, i % 5][:c["axes"]])
        half = c["rot"] // 2
        # pairs in runs, one per axis, the last axis with what is left
        axes = [min(i * c["axes"] // half, c["axes"] - 1) for i in range(half)]
        freq = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        return dict(case=c, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:],
                    q_out=torch.zeros((t, hq, d), dtype=TYPES[c["type"]], device="cuda"),
                    k_pool=_pool((blocks, hkv, bs, d), g, cache, K_SCALE),
                    v_pool=_pool((blocks, hkv, bs, d), g, cache, V_SCALE),
                    slots=torch.randperm(blocks * bs, generator=g, device="cuda")[:t].to(torch.int32),
                    positions=positions.to(torch.int64).contiguous(), freq=freq, axes=axes,
                    axes_d=torch.tensor(axes, device="cuda"),
                    status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    n, keep = c["blocks"], c["blocks"] - c["pairs"]
    shape = (c["layers"], 2, n, c["hkv"], c["bs"], c["d"])
    pools = _pool(shape, g, c["type"], K_SCALE)
    order = torch.randperm(keep, generator=g, device="cuda")
    pairs = torch.stack([torch.arange(keep, n, device="cuda"), order[:c["pairs"]]], 1).to(torch.int32)
    used = torch.cat([order[c["pairs"]:], pairs[:, 0].long()])
    used = used[torch.randperm(len(used), generator=g, device="cuda")]
    width = max(1, -(-len(used) // c["seqs"]))
    tables = torch.full((c["seqs"] * width,), -1, dtype=torch.int32, device="cuda")
    tables[:len(used)] = used.to(torch.int32)
    return dict(case=c, pools=pools, keys=[pools[l, 0] for l in range(c["layers"])],
                values=[pools[l, 1] for l in range(c["layers"])], pairs=pairs.contiguous(),
                tables=tables.view(c["seqs"], width), status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def run(s):
    return {"attention": _attention, "rope": _rope, "move": _move}[s["case"]["op"]](s)


def _workspace(s, need):
    """The program's workspace, made on its first call."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(need(), 256), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _attention(s):
    c = s["case"]
    if own:
        import paged_kv_cache_187_gb300 as pa
        ws = _workspace(s, lambda: pa.pa_prefill_workspace_size(
            s["q"].shape[0], len(s["lens"]), c["hq"], c["hkv"], c["d"], s["longest"]))
        args = (s["out"], s["q"], s["k"], s["v"], s["tables"], s["lens_d"], s["starts_d"], s["longest"], s["scale"])
        if c["cache"] == "fp8":
            pa.pa_prefill_fp8(*args, K_SCALE, V_SCALE, workspace=ws, status=s["status"])
        else:
            pa.pa_prefill(*args, workspace=ws, status=s["status"])
        return s["out"]
    out = s["out"]
    hkv, d, g = c["hkv"], c["d"], c["hq"] // c["hkv"]
    for n, at, blocks in s["groups"]:
        rows = s["starts_d"][at].long()[:, None] + torch.arange(n, device="cuda")
        tables = s["tables"][at, :blocks].long().clamp_min(0)
        k, v = (_values(p[tables], c["cache"], scale).transpose(1, 2).reshape(len(at), hkv, 1, -1, d)
                for p, scale in ((s["k"], K_SCALE), (s["v"], V_SCALE)))
        q = s["q"][rows].float().view(len(at), n, hkv, g, d).permute(0, 2, 3, 1, 4)
        scores = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
        limit = (s["lens_d"][at].long()[:, None] - n + torch.arange(n, device="cuda") + 1)[:, None, None, :, None]
        scores.masked_fill_(torch.arange(scores.shape[-1], device="cuda") >= limit, -math.inf)
        scores.sub_(scores.amax(-1, keepdim=True)).exp_()
        o = torch.matmul(scores, v).div_(scores.sum(-1, keepdim=True))
        out[rows] = o.permute(0, 3, 1, 2, 4).reshape(len(at), n, c["hq"], d).to(out.dtype)
    return out


def _values(x, cache, scale):
    return x.view(torch.float8_e4m3fn).float() * scale if cache == "fp8" else x.float()


def _rope(s):
    c = s["case"]
    if own:
        import paged_kv_cache_187_gb300 as pa
        args = (s["q_out"], s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["slots"], s["positions"], s["freq"])
        more = dict(pair_axes=s["axes"], interleaved=c["interleaved"], status=s["status"])
        if c["cache"] == "fp8":
            pa.pa_rope_and_cache_fp8(*args, K_SCALE, V_SCALE, **more)
        else:
            pa.pa_rope_and_cache(*args, **more)
        return s["q_out"], _held(s["k_pool"]), _held(s["v_pool"])
    angle = s["positions"][s["axes_d"]].t().double() * s["freq"].double()        # [tokens, pairs]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    half, rot = c["rot"] // 2, c["rot"]
    block, offset = s["slots"].long() // c["bs"], s["slots"].long() % c["bs"]

    def turn(x):
        y = x.float()
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["interleaved"] else (y[..., :half], y[..., half:rot])
        a, b = a * cos - b * sin, a * sin + b * cos
        both = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
        return torch.cat([both, y[..., rot:]], -1)

    s["q_out"].copy_(turn(s["q"]))
    for pool, x, scale in ((s["k_pool"], turn(s["k"]), K_SCALE), (s["v_pool"], s["v"].float(), V_SCALE)):
        if c["cache"] == "fp8":
            x = (x * (1.0 / scale)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        pool[block, :, offset] = x.to(pool.dtype)
    return s["q_out"], _held(s["k_pool"]), _held(s["v_pool"])


def _held(pool):
    """A pool's values: 8-bit ones in units of their scale."""
    return pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool


def _move(s):
    if own:
        import paged_kv_cache_187_gb300 as pa
        pa.pa_move_blocks(s["keys"], s["values"], s["pairs"], block_tables=s["tables"], status=s["status"])
        return _held(s["pools"]), s["tables"]
    at, to = s["pairs"].long().t()
    s["pools"][:, :, to] = s["pools"][:, :, at]
    place = torch.arange(s["case"]["blocks"] + 1, dtype=torch.int32, device="cuda")
    place[-1] = -1                                                               # the padding stays
    place[at] = s["pairs"][:, 1]
    s["tables"].copy_(place[s["tables"].long()])
    return _held(s["pools"]), s["tables"]


def exact(c, seed):
    """From the definitions, in 64 bits."""
    s = prepare(c, seed)
    if c["op"] == "move":
        pools, tables = s["pools"].clone(), s["tables"].cpu()
        for a, b in s["pairs"].tolist():
            pools[:, :, b] = s["pools"][:, :, a]
        new = dict(s["pairs"].tolist())
        tables = torch.tensor([[new.get(x, x) for x in row] for row in tables.tolist()], dtype=torch.int32)
        return _held(pools), tables
    if c["op"] == "rope":
        pos = torch.stack([s["positions"][a] for a in s["axes"]]).double().t()
        w = torch.polar(torch.ones_like(pos), pos * s["freq"].double())[:, None]

        def rotated(x):
            y = x.double().clone()
            first = slice(0, c["rot"], 2) if c["interleaved"] else slice(0, c["rot"] // 2)
            second = slice(1, c["rot"], 2) if c["interleaved"] else slice(c["rot"] // 2, c["rot"])
            z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * w
            y[..., first], y[..., second] = z.real, z.imag
            return y

        held = []
        for pool, x, scale in ((s["k_pool"], rotated(s["k"]), K_SCALE), (s["v_pool"], s["v"].double(), V_SCALE)):
            p = _held(pool).double().transpose(1, 2).reshape(-1, c["hkv"], c["d"])
            p[s["slots"].long()] = x / scale if c["cache"] == "fp8" else x
            held.append(p.view(-1, c["bs"], c["hkv"], c["d"]).transpose(1, 2).contiguous())
        return rotated(s["q"]), held[0], held[1]
    if work(c)["flops"] > 3e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    g = c["hq"] // c["hkv"]
    for i, (n, length) in enumerate(s["lens"]):
        ids = s["tables"][i, :-(-length // c["bs"])].long()
        for h in range(c["hkv"]):
            k, v = (_values(p[ids, h], c["cache"], 1.0).double().reshape(-1, c["d"])[:length]
                    for p in (s["k"], s["v"]))
            if c["cache"] == "fp8":
                k, v = k * K_SCALE, v * V_SCALE
            rows = slice(s["starts"][i], s["starts"][i + 1])
            for j in range(h * g, (h + 1) * g):
                x = s["q"][rows, j].double() @ k.t() * s["scale"]
                keep = torch.ones(n, length, dtype=torch.bool, device="cuda").tril(length - n)
                out[rows, j] = torch.softmax(x.masked_fill(~keep, -math.inf), -1) @ v
    return out
