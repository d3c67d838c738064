"""GPU: attention of trees of new tokens over the paged cache (pa_decode_tree, _fp8) against the
plain 64-bit form, the accepted paths (pa_tree_accept) and the moves of their rows
(pa_move_tokens)."""
import math
import random

import pytest
import torch

import masked_reference as M
from test_gpu_prefill import make

pytestmark = pytest.mark.gpu


def random_tree(n, seed, reach=9):
    r = random.Random(seed)
    return [-1] + [r.randrange(max(0, i - reach), i) for i in range(1, n)] if n else []


def trees(b, kind, seed):
    """The trees' bool matrices: paths of random trees, any bits below the diagonal (rows that see
    nothing of the tree among them), or every token before."""
    g = torch.Generator().manual_seed(seed)
    sees = []
    for s in range(len(b["lens"])):
        n = int(b["starts"][s + 1] - b["starts"][s])
        if kind == "paths":
            sees.append(M.paths(random_tree(n, seed + s)))
        elif kind == "any":
            m = torch.rand((n, n), generator=g) < torch.rand((n, 1), generator=g)
            m[::5] = False
            sees.append(m)
        else:
            sees.append(torch.ones((n, n), dtype=torch.bool).tril())
    return sees


def workspace(b, mcl):
    import paged_kv_cache_187_gb300 as pa
    T, Hq, D = b["q"].shape
    n = pa.pa_decode_tree_workspace_size(T, len(b["lens"]), Hq, b["kc"].shape[1], D, mcl)
    return torch.full((max(n, 256),), 0xA5, dtype=torch.uint8, device="cuda")


def call(b, mask, out, ws=None, mcl=None, status=None, stream=None):
    import paged_kv_cache_187_gb300 as pa
    mcl = max(b["lens"] + [0]) if mcl is None else mcl
    ws = workspace(b, mcl) if ws is None else ws
    args = (out, b["q"], b["kc"], b["vc"], b["tables"], b["lens_d"], b["starts_d"], mask, mcl, b["scale"])
    if b["fp8"]:
        pa.pa_decode_tree_fp8(*args, b["ks"], b["vs"], workspace=ws, status=status, stream=stream)
    else:
        pa.pa_decode_tree(*args, workspace=ws, status=status, stream=stream)
    return out


def check(b, sees, out):
    want, tol = M.tree(b["q"], b["kc"], b["vc"], b["tables"], b["lens"], b["starts"], sees, b["scale"],
                       b["ks"], b["vs"])
    n = int(b["starts"][-1])
    err = (out[:n].double() - want[:n]).abs()
    assert torch.isfinite(out[:n]).all()
    bad = err > tol[:n]
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} beyond tolerance, worst ratio "
                           f"{float((err / tol[:n].clamp_min(1e-30))[bad].max()):.3g}, first at "
                           f"{bad.nonzero()[0].tolist()}")


def run(b, sees, words=None):
    words = words or max(1, -(-max([m.shape[0] for m in sees] + [1]) // 32))
    mask = M.masks(sees, words, "cuda")
    if b["q"].shape[0] > mask.shape[0]:
        mask = torch.cat([mask, mask.new_full((b["q"].shape[0] - mask.shape[0], words), -1)])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(b, mask, torch.full_like(b["q"], 7.0), status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    check(b, sees, out)
    return out


# one token to several row tiles; trees that begin at, before and behind the edges of tiles,
# halves of tiles, blocks and mask words; trees that are the whole context, and longer than it
SEQS = [(1, 1), (5, 5), (8, 308), (33, 161), (64, 192), (64, 191), (31, 160), (0, 40), (65, 66), (32, 32),
        (40, 300), (7, 135), (130, 140), (9, 6)]


@pytest.mark.parametrize("kind", ["paths", "any"])
@pytest.mark.parametrize("Hq,Hkv,D,bs,dtype,fp8", [
    (4, 4, 128, 16, torch.bfloat16, False),
    (8, 2, 128, 16, torch.bfloat16, False),
    (8, 2, 64, 32, torch.float16, False),
    (16, 1, 128, 32, torch.float16, False),
    (7, 1, 64, 16, torch.bfloat16, False),
    (8, 2, 128, 16, torch.bfloat16, True),
    (13, 1, 128, 32, torch.float16, True),
])
def test_trees(cuda_device, Hq, Hkv, D, bs, dtype, fp8, kind):
    b = make(SEQS, Hq, Hkv, D, bs, dtype, 31 + Hq + D, fp8, extra=3)
    out = run(b, trees(b, kind, 5))
    assert bool((out[int(b["starts"][-1]):] == 7.0).all())      # rows behind the last sequence


@pytest.mark.parametrize("seqs,Hq,Hkv,D,bs,dtype,fp8", [
    # few units, cut into shares; rows for one stream (whose tiles the streams share) and both
    ([(8, 5000)], 8, 1, 128, 16, torch.bfloat16, False),
    ([(60, 9001), (1, 77), (33, 2600)], 16, 2, 128, 32, torch.float16, False),
    ([(64, 20000)], 8, 2, 64, 16, torch.bfloat16, False),
    ([(20, 6000), (1, 8191), (70, 4000)], 16, 2, 128, 16, torch.float16, True),
    # many units
    ([(1 + i * 7 % 64, 1 + i * 7 % 64 + i * 131 % 1500) for i in range(120)], 8, 2, 128, 16, torch.bfloat16, False),
    ([(1 + i * 7 % 64, 1 + i * 7 % 64 + i * 131 % 1500) for i in range(120)], 4, 4, 64, 32, torch.float16, False),
    # a wide tree: more mask words than rows of a tile
    ([(700, 3000), (300, 300)], 4, 2, 128, 16, torch.bfloat16, False),
])
def test_trees_over_long_contexts(cuda_device, seqs, Hq, Hkv, D, bs, dtype, fp8):
    b = make(seqs, Hq, Hkv, D, bs, dtype, 3 + Hq, fp8)
    run(b, trees(b, "paths", 9))


@pytest.mark.parametrize("D,dtype,fp8", [(64, torch.float16, False), (128, torch.bfloat16, False),
                                         (128, torch.bfloat16, True)])
def test_a_chain_is_a_chunk(cuda_device, D, dtype, fp8):
    """With every token before it set, and garbage past it, a tree is a chunk: the same bits."""
    import paged_kv_cache_187_gb300 as pa
    b = make([(40, 300), (1, 2500), (5, 64), (200, 200), (64, 7000)], 6, 2, D, 16, dtype, 73, fp8)
    sees = [torch.ones((int(n), int(n)), dtype=torch.bool) for n in (40, 1, 5, 200, 64)]
    mask = M.masks(sees, 7, "cuda")
    out = call(b, mask, torch.zeros_like(b["q"]))
    mcl = max(b["lens"])
    want = torch.zeros_like(out)
    args = (want, b["q"], b["kc"], b["vc"], b["tables"], b["lens_d"], b["starts_d"], mcl, b["scale"])
    if fp8:
        pa.pa_prefill_fp8(*args, b["ks"], b["vs"], workspace=workspace(b, mcl))
    else:
        pa.pa_prefill(*args, workspace=workspace(b, mcl))
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_rows_that_see_nothing(cuda_device):
    b = make([(6, 6), (40, 40), (3, 2)], 4, 2, 128, 16, torch.bfloat16, 8)
    sees = [torch.zeros((n, n), dtype=torch.bool) for n in (6, 40, 3)]
    sees[1][7, 3] = True
    out = run(b, sees)
    rows = [i for i in range(49) if i != 6 + 7]
    assert bool((out[rows] == 0).all()) and bool((out[13] != 0).any())


@pytest.mark.parametrize("seqs,Hq,fp8", [([(12, 12), (40, 150), (20, 700)], 8, False),
                                         ([(64, 6000)], 8, False),
                                         ([(12, 12), (40, 150), (20, 700)], 8, True)])
def test_infinite_and_nan_values_stay_with_the_rows_that_see_them(cuda_device, seqs, Hq, fp8):
    """V rows of single nodes hold +inf, -inf, both and NaN, K rows NaN: a row that does not see
    them has the bits that it has without them, one that does is infinite or NaN where they are."""
    b = make(seqs, Hq, 2, 128, 16, torch.bfloat16, 17, fp8)
    sees = trees(b, "paths", 3)
    words = max(-(-m.shape[0] // 32) for m in sees)
    mask = M.masks(sees, words, "cuda")
    clean = call(b, mask, torch.zeros_like(b["q"]))
    torch.cuda.synchronize()
    check(b, sees, clean)
    g, D, bs = Hq // 2, 128, 16
    nan = 0x7F if fp8 else math.nan
    for s, (n, L) in enumerate(seqs):
        plans = [(2, [(5, math.nan)]), (n - 1, [(9, math.nan)])]
        if not fp8:
            plans += [(3, [(0, math.inf), (70, -math.inf)]), (4, [(0, -math.inf)]), (6, [(1, -math.inf)])]
        for node, put in plans:
            kc, vc = b["kc"].clone(), b["vc"].clone()
            pos = L - n + node
            block = int(b["tables"][s, pos // bs])
            for d, x in put:
                vc[block, 1, pos % bs, d] = nan if math.isnan(x) else x
            out = call(dict(b, kc=kc, vc=vc), mask, torch.zeros_like(b["q"]))
            torch.cuda.synchronize()
            want = clean.clone()
            a = int(b["starts"][s])
            for j in range(n):
                if sees[s][j, node]:
                    for d, x in put:
                        want[a + j, g:2 * g, d] = x
            same = (out == want) | (torch.isnan(out) & torch.isnan(want))
            assert bool(same.all()), (s, node, (~same).nonzero()[:4].tolist())
            # a NaN key: the rows that see it are NaN throughout
            kc[block, 0, pos % bs, 3] = nan
            out = call(dict(b, kc=kc), mask, torch.zeros_like(b["q"]))
            torch.cuda.synchronize()
            want = clean.clone()
            for j in range(n):
                if sees[s][j, node]:
                    want[a + j, :g] = math.nan
            same = (out == want) | (torch.isnan(out) & torch.isnan(want))
            assert bool(same.all()), (s, node, "key", (~same).nonzero()[:4].tolist())


def test_two_infinities_of_one_element(cuda_device):
    """+inf at one node and -inf at another: infinite for rows that see one, NaN for both."""
    b = make([(10, 200)], 4, 1, 64, 16, torch.float16, 4)
    sees = [M.paths([-1, 0, 0, 1, 1, 2, 3, 5, 4, 6])]
    for node, x in ((1, math.inf), (6, -math.inf), (2, math.inf)):
        pos = 190 + node
        b["vc"][int(b["tables"][0, pos // 16]), 0, pos % 16, 40] = x
    out = call(b, M.masks(sees, 1, "cuda"), torch.zeros_like(b["q"]))
    torch.cuda.synchronize()
    got = out[:, 0, 40].tolist()
    for j in range(10):
        plus, minus = bool(sees[0][j, 1] or sees[0][j, 2]), bool(sees[0][j, 6])
        if plus and minus:
            assert math.isnan(got[j])
        elif plus or minus:
            assert got[j] == (math.inf if plus else -math.inf)
        else:
            assert math.isfinite(got[j])


def test_bad_metadata_is_flagged(cuda_device):
    import paged_kv_cache_187_gb300 as pa
    seqs = [(40, 300), (8, 64)]
    b = make(seqs, 4, 2, 128, 16, torch.bfloat16, 5)
    sees = trees(b, "paths", 2)
    good = run(b, sees)

    def flagged(bit, mask=None, **kw):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = call(dict(b, **kw), M.masks(sees, 2, "cuda") if mask is None else mask,
                   torch.full_like(b["q"], 7.0), mcl=300, status=status)
        torch.cuda.synchronize()
        assert int(status) == bit
        return out

    # a tree of 40 tokens and one word of masks: the rows below 32 do not change, and no row sees
    # the tokens past them
    out = flagged(pa.PA_DEVERR_BAD_LEN, mask=M.masks(sees, 1, "cuda"))
    assert torch.equal(out[:32], good[:32]) and torch.equal(out[40:], good[40:])
    cut = [sees[0].clone(), sees[1]]
    cut[0][:, 32:] = False
    check(b, cut, out)
    flagged(pa.PA_DEVERR_BAD_LEN, starts_d=torch.tensor([0, 40, 99], dtype=torch.int32, device="cuda"))
    flagged(pa.PA_DEVERR_BAD_LEN, starts_d=torch.tensor([0, 40, 30], dtype=torch.int32, device="cuda"))
    flagged(pa.PA_DEVERR_BAD_LEN, lens_d=torch.tensor([100000, 64], dtype=torch.int32, device="cuda"))
    flagged(pa.PA_DEVERR_BAD_LEN, lens_d=torch.tensor([300, -5], dtype=torch.int32, device="cuda"))
    tables = b["tables"].clone()
    tables[1, 2] = b["kc"].shape[0] + 7
    out = flagged(pa.PA_DEVERR_BAD_BLOCK, tables=tables)
    assert torch.equal(out[:40], good[:40])


def test_graphs_streams_and_guards(cuda_device):
    """Captured and replayed with new masks, on another stream, with guards behind the workspace."""
    import paged_kv_cache_187_gb300 as pa
    b = make([(40, 1300), (64, 64), (9, 5000)], 8, 2, 128, 16, torch.bfloat16, 6)
    T, mcl = b["q"].shape[0], 5000
    need = pa.pa_decode_tree_workspace_size(T, 3, 8, 2, 128, mcl)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    mask = torch.zeros((T, 2), dtype=torch.int32, device="cuda")
    out = torch.zeros_like(b["q"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(b, mask, out, ws=ws[:need], mcl=mcl)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(b, mask, out, ws=ws[:need], mcl=mcl)
    for seed in (1, 2):
        sees = trees(b, "paths" if seed == 1 else "any", seed)
        mask.copy_(M.masks(sees, 2, "cuda"))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        check(b, sees, out)
        with torch.cuda.stream(side):
            again = call(b, mask, torch.zeros_like(out), ws=ws[:need], mcl=mcl, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, again)
    assert bool((ws[need:] == 0x5A).all())


# ------------------------------------------------------------------ the accepted path
def accept_call(parents, draft, target, most, lens=None, words=None, extra=0):
    import paged_kv_cache_187_gb300 as pa
    S = len(parents)
    n = [len(p) for p in parents]
    words = words or max(1, -(-max(n + [1]) // 32))
    mask = M.masks([M.paths(p) for p in parents], words, "cuda")
    starts = torch.tensor([sum(n[:i]) for i in range(S + 1)], dtype=torch.int32, device="cuda")
    lens = torch.tensor(lens or [10 * i + k for i, k in enumerate(n)], dtype=torch.int32, device="cuda")
    accepted = torch.full((S, most), 77, dtype=torch.int32, device="cuda")
    count = torch.full((S,), 77, dtype=torch.int32, device="cuda")
    follow = torch.full((S,), 77, dtype=torch.int64, device="cuda")
    new = torch.full((S,), 77, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = torch.tensor([x for t in draft for x in t], dtype=torch.int64, device="cuda")
    t = torch.tensor([x for t in target for x in t], dtype=torch.int64, device="cuda")
    pa.pa_tree_accept(accepted, count, follow, new, d, t, mask, starts, lens, status=status)
    torch.cuda.synchronize()
    return accepted, count, follow, new, lens, int(status)


@pytest.mark.parametrize("sizes,most,vocab", [
    ([1, 2, 8, 0, 33, 64, 65], 16, 3),
    ([5, 300, 31, 32], 4, 2),
    ([1], 1, 5),
    ([2048, 7], 40, 2),
    ([3, 0], 600, 1),            # every token matches: the deepest path
    ([500], 600, 1),
])
def test_accepted_paths(cuda_device, sizes, most, vocab):
    r = random.Random(sum(sizes) + vocab)
    # (large tokens: no 32-bit comparison)
    word = lambda: r.randrange(vocab) * (1 << 33) + 5  # noqa: E731
    parents = [random_tree(n, 3 + i, reach=4 if i % 2 else n) for i, n in enumerate(sizes)]
    draft = [[word() for _ in range(n)] for n in sizes]
    target = [[word() for _ in range(n)] for n in sizes]
    accepted, count, follow, new, lens, status = accept_call(parents, draft, target, most)
    assert status == 0
    for s, n in enumerate(sizes):
        path, token = M.accept(parents[s], draft[s], target[s], most)
        assert accepted[s].tolist() == path + [-1] * (most - len(path))
        assert int(count[s]) == len(path) and int(follow[s]) == token
        assert int(new[s]) == int(lens[s]) - n + len(path)


def test_a_node_without_a_parent_is_not_accepted(cuda_device):
    import paged_kv_cache_187_gb300 as pa
    mask = torch.tensor([[1], [2], [6], [9]], dtype=torch.int32, device="cuda")   # 1 and 2 hang on no root
    starts = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20], dtype=torch.int32, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    accepted = torch.zeros((1, 5), dtype=torch.int32, device="cuda")
    count, follow = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    pa.pa_tree_accept(accepted, count, follow, lens, ids, ids, mask, starts, lens)     # (lengths in place)
    assert accepted[0].tolist() == [0, 3, -1, -1, -1] and int(count) == 2 and int(lens) == 18


def test_accept_flags_bad_lengths(cuda_device):
    parents = [random_tree(6, 1), random_tree(4, 2)]
    ids = [[1] * 6, [1] * 4]
    *_, status = accept_call(parents, ids, ids, 8, lens=[5, 4])
    assert status == 4


def moves_reference(pools, tables, new, accepted, count, bs):
    want = [p.clone() for p in pools]
    for s in range(tables.shape[0]):
        n = int(count[s])
        base = int(new[s]) - n
        for j in range(n):
            at, to = base + int(accepted[s, j]), base + j
            for w, p in zip(want, pools):
                w[int(tables[s, to // bs]), :, to % bs] = p[int(tables[s, at // bs]), :, at % bs]
    return want


@pytest.mark.parametrize("Hkv,D,bs,dtype,layers,most", [
    (8, 128, 16, torch.bfloat16, 3, 12),
    (1, 64, 32, torch.float16, 70, 5),          # two launches
    (5, 64, 16, torch.uint8, 2, 130),           # more rows than a pass of the table of places
    (33, 128, 32, torch.uint8, 1, 9),
    (3, 80, 8, torch.bfloat16, 2, 20),          # rows of 160 bytes, blocks of 8
])
def test_moved_rows(cuda_device, Hkv, D, bs, dtype, layers, most):
    import paged_kv_cache_187_gb300 as pa
    r = random.Random(Hkv * D)
    sizes = [1, 7, 64, 200, 40, 3]
    S, g = len(sizes), torch.Generator(device="cuda").manual_seed(4)
    lens = [n + r.randrange(0, 90) for n in sizes]
    width = -(-max(lens) // bs) + 1
    NB = S * width + 3
    tables = torch.randperm(NB, generator=g, device="cuda")[:S * width].to(torch.int32).view(S, width)
    pools = [torch.randint(0, 255, (NB, Hkv, bs, D * (1 if dtype == torch.uint8 else 2)), generator=g,
                           device="cuda", dtype=torch.uint8) for _ in range(2 * layers)]
    pools = [p if dtype == torch.uint8 else p.view(dtype) for p in pools]
    accepted = torch.full((S, most), -1, dtype=torch.int32, device="cuda")
    count = torch.zeros(S, dtype=torch.int32, device="cuda")
    for s, n in enumerate(sizes):
        k = min(most, n) if s % 2 else r.randint(1, min(most, n))
        path = sorted(r.sample(range(n), k))
        accepted[s, :k] = torch.tensor(path, dtype=torch.int32)
        count[s] = k
    count[2] = 0
    new = (torch.tensor(lens, device="cuda") - torch.tensor(sizes, device="cuda")).to(torch.int32) + count
    raw = [p.view(torch.uint8) for p in pools]
    want = moves_reference(raw, tables.cpu(), new, accepted.cpu(), count, bs)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_move_tokens(pools[:layers], pools[layers:], tables, new, accepted, count, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    for i, (a, b) in enumerate(zip(raw, want)):
        assert torch.equal(a, b), i


def test_moves_flag_bad_entries(cuda_device):
    """An entry that does not ascend, a position past the table, a block outside the pool, counts
    out of range: flagged, the rest moved."""
    import paged_kv_cache_187_gb300 as pa
    NB, bs = 12, 16
    key = torch.arange(NB * bs, device="cuda").view(NB, 1, bs, 1).expand(NB, 1, bs, 64).to(torch.float16).contiguous()
    cases = [([0, 3, 2, 5], 4, 20, [0, 1], 1, {1: 3, 3: 5}),          # (2 behind 3)
             ([0, 40, 41], 3, 19, [0, 1], 4, {}),                     # past 32 tokens
             ([0, 2, 20], 3, 5, [0, 99], 2, {1: 2}),                  # a block that is not there
             ([0, 2], 9, 20, [0, 1], 4, {}),                          # more than the row holds
             ([0, 2], 2, 1, [0, 1], 4, {}),                           # before the context's start
             ([-3, 4], 2, 8, [0, 1], 1, {1: 4})]
    for path, n, new, table, bit, moved in cases:
        k, v = key.clone(), key.clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pa.pa_move_tokens([k], [v], torch.tensor([table], dtype=torch.int32, device="cuda"),
                          torch.tensor([new], dtype=torch.int32, device="cuda"),
                          torch.tensor([path], dtype=torch.int32, device="cuda"),
                          torch.tensor([n], dtype=torch.int32, device="cuda"), status=status)
        torch.cuda.synchronize()
        want = key.clone()
        for j, node in moved.items():
            to, at = new - n + j, new - n + node
            want[table[to // bs], 0, to % bs] = key[table[at // bs], 0, at % bs]
        assert int(status) == bit, path
        assert torch.equal(k, want) and torch.equal(v, want), path


def test_accept_and_move_in_a_graph(cuda_device):
    """Captured once, replayed with other choices of the model."""
    import paged_kv_cache_187_gb300 as pa
    sizes, bs, layers, most = [9, 30, 12], 16, 2, 8
    S, T, g = 3, 51, torch.Generator(device="cuda").manual_seed(4)
    parents = [random_tree(n, i) for i, n in enumerate(sizes)]
    mask = M.masks([M.paths(p) for p in parents], 1, "cuda")
    starts = torch.tensor([0, 9, 39, 51], dtype=torch.int32, device="cuda")
    lens = torch.tensor([50, 30, 100], dtype=torch.int32, device="cuda")
    tables = torch.randperm(24, generator=g, device="cuda").to(torch.int32).view(3, 8)
    fresh = [torch.randn((24, 2, bs, 64), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2 * layers)]
    pools = [p.clone() for p in fresh]
    accepted = torch.zeros((S, most), dtype=torch.int32, device="cuda")
    count, new = (torch.zeros(S, dtype=torch.int32, device="cuda") for _ in range(2))
    follow = torch.zeros(S, dtype=torch.int64, device="cuda")
    draft, target = (torch.zeros(T, dtype=torch.int64, device="cuda") for _ in range(2))

    def step():
        pa.pa_tree_accept(accepted, count, follow, new, draft, target, mask, starts, lens)
        pa.pa_move_tokens(pools[:layers], pools[layers:], tables, new, accepted, count)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    r = random.Random(8)
    for _ in range(4):
        d, t = ([r.randrange(2) for _ in range(T)] for _ in range(2))
        draft.copy_(torch.tensor(d))
        target.copy_(torch.tensor(t))
        for p, f in zip(pools, fresh):
            p.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        for s, n in enumerate(sizes):
            a = int(starts[s])
            path, token = M.accept(parents[s], d[a:a + n], t[a:a + n], most)
            assert accepted[s, :len(path)].tolist() == path and int(follow[s]) == token
        want = moves_reference(fresh, tables.cpu(), new, accepted.cpu(), count, bs)
        assert all(torch.equal(p, w) for p, w in zip(pools, want))


@pytest.mark.parametrize("seqs,Hq,Hkv,D,bs,dtype,fp8", [
    # two row tiles (and four, and three with one left over) of a sequence, taken in pairs
    ([(60, 9001), (50, 7000), (64, 12000)], 16, 2, 128, 16, torch.bfloat16, False),
    ([(55, 20000)], 8, 1, 128, 32, torch.float16, False),
    ([(120, 9001), (97, 8000)], 16, 2, 128, 16, torch.bfloat16, False),
    ([(33, 9001), (64, 300), (34, 15000), (0, 40), (64, 64)], 16, 2, 64, 16, torch.float16, False),
    ([(60, 9001), (50, 7000)], 16, 2, 128, 16, torch.float16, True),
    ([(400, 8000), (300, 9000)], 4, 1, 128, 16, torch.bfloat16, False),
    # too many left over for pairs
    ([(60, 9001), (5, 7000), (9, 12000), (31, 8000)], 16, 2, 128, 16, torch.bfloat16, False),
])
def test_row_tiles_in_pairs(cuda_device, seqs, Hq, Hkv, D, bs, dtype, fp8):
    b = make(seqs, Hq, Hkv, D, bs, dtype, 41 + Hq, fp8)
    run(b, trees(b, "paths", 19))


@pytest.mark.parametrize("seqs,kind", [([(2000, 2000), (3, 900)], "chain"), ([(1700, 2600)], "any"),
                                       ([(2048, 2050), (2047, 4000)], "paths")])
def test_large_trees(cuda_device, seqs, kind):
    b = make(seqs, 4, 2, 64, 16, torch.float16, 12)
    run(b, trees(b, kind, 3))


def test_two_graphs_share_a_workspace(cuda_device):
    """One whose contexts are cut, one without a plan, replayed in turn."""
    import paged_kv_cache_187_gb300 as pa
    cases = [make([(40, 9000), (64, 7000)], 8, 2, 128, 16, torch.bfloat16, 6), make([(9, 300)], 8, 2, 128, 16, torch.bfloat16, 7)]
    need = max(pa.pa_decode_tree_workspace_size(b["q"].shape[0], len(b["lens"]), 8, 2, 128, max(b["lens"])) for b in cases)
    ws = torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda")
    side, graphs, sees, outs = torch.cuda.Stream(), [], [], []
    for b in cases:
        sees.append(trees(b, "paths", 5))
        mask, out = M.masks(sees[-1], 2, "cuda"), torch.zeros_like(b["q"])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(b, mask, out, ws=ws)
        graphs.append((graph, mask))
        outs.append(out)
    for turn in range(3):
        for i, b in enumerate(cases):
            outs[i].fill_(7.0)
            graphs[i][0].replay()
        torch.cuda.synchronize()
        for i, b in enumerate(cases):
            check(b, sees[i], outs[i])


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_scales(cuda_device, scale):
    b = make([(20, 300), (5, 5), (33, 2000)], 8, 2, 128, 16, torch.bfloat16, 21)
    b["scale"] = scale
    run(b, trees(b, "any", 4))
