"""GPU: the tree and sparse operators in a row, as a server uses them: drafts decoded over selected
blocks, the drafted tree's tokens written with their rotary positions, verified over the whole cache,
the accepted path committed in every layer, the touched blocks bounded anew -- several rounds, after
which the cache has to hold what appending the accepted tokens alone would have put there."""
import random

import numpy as np
import pytest
import torch

import chunk_reference as R
import masked_reference as M

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prompts,rounds", [([500, 33, 1300], 4), ([1], 3)])
def test_rounds_of_speculation(cuda_device, prompts, rounds, fp8):
    import paged_kv_cache_187_gb300 as pa
    Hq, Hkv, D, bs, layers, dtype, dev = 16, 4, 128, 16, 2, torch.bfloat16, "cuda"
    S, width, mcl, keep, vocab = len(prompts), 100, 1600, 12, 3
    NB = S * width + 10
    ks, vs = (0.03, 0.02) if fp8 else (1.0, 1.0)
    g, r = torch.Generator(device=dev).manual_seed(5), random.Random(3)
    scale = D ** -0.5
    alloc = pa.PagedAllocator(NB, bs, 9)
    cdt = torch.uint8 if fp8 else dtype
    keys, values = ([torch.full((NB, Hkv, bs, D), 0, dtype=cdt, device=dev) for _ in range(layers)] for _ in range(2))
    bounds = [torch.zeros((NB, Hkv, 2, D), dtype=torch.int8, device=dev) for _ in range(layers)]
    steps = [torch.zeros((NB, Hkv), device=dev) for _ in range(layers)]
    freq = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().to(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    held = [[] for _ in range(S)]         # per sequence and layer: the rows that have to be in the cache

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def write(l, q, k, v, slots, pos):
        out = torch.empty_like(q)
        if fp8:
            pa.pa_rope_and_cache_fp8(out, q, k, v, keys[l], values[l], slots, pos[None], freq, ks, vs, status=status)
        else:
            pa.pa_rope_and_cache(out, q, k, v, keys[l], values[l], slots, pos[None], freq, status=status)
        return out

    def rows(l, slots):
        b, o = slots.long() // bs, slots.long() % bs
        return [(keys[l][x, :, y].clone(), values[l][x, :, y].clone()) for x, y in zip(b, o)]

    # the prompts
    starts = np.concatenate([[0], np.cumsum(prompts)])
    slots = []
    for s, n in enumerate(prompts):
        alloc.pa_alloc_add_seq(s, n)
        slots += alloc.pa_alloc_slots(s, 0, n).tolist()
    ids = list(range(S))
    slots_d = i32(slots)
    pos = torch.cat([torch.arange(n, device=dev) for n in prompts])
    for l in range(layers):
        q, k, v = (torch.randn((int(starts[-1]), h, D), generator=g, device=dev).to(dtype) for h in (Hq, Hkv, Hkv))
        write(l, q, k, v, slots_d, pos)
        got = rows(l, slots_d)
        for s in range(S):
            held[s].append(got[starts[s]:starts[s + 1]])
    tables = torch.from_numpy(alloc.pa_alloc_block_tables(ids, width)).to(dev)
    lens = torch.from_numpy(alloc.pa_alloc_context_lens(ids)).to(dev)
    for l in range(layers):
        pa.pa_key_bounds(bounds[l], steps[l], keys[l], tables, lens, max(prompts), query_starts=i32(starts.tolist()),
                         status=status)
    ws = torch.empty(max(pa.pa_select_blocks_workspace_size(S, 1, Hkv, bs, mcl), 256), dtype=torch.uint8, device=dev)
    moved = 0
    for _ in range(rounds):
        length = alloc.pa_alloc_context_lens(ids)
        # a draft step over selected blocks, every layer
        for l in range(layers):
            q = torch.randn((S, Hq, D), generator=g, device=dev).to(dtype)
            sel = torch.empty((S, Hkv, keep), dtype=torch.int32, device=dev)
            pa.pa_select_blocks(sel, q, bounds[l], steps[l], tables, lens, bs, mcl, 1, 3, workspace=ws, status=status)
            out = torch.zeros_like(q)
            if fp8:
                pa.pa_decode_sparse_fp8(out, q, keys[l], values[l], tables, lens, sel, scale, ks, vs, status=status)
            else:
                pa.pa_decode_sparse(out, q, keys[l], values[l], tables, lens, sel, scale, status=status)
            for s in range(S):
                L, n_blocks = int(length[s]), -(-int(length[s]) // bs)
                k, v = M.gather(keys[l], tables[s], L, ks), M.gather(values[l], tables[s], L, vs)
                seen = torch.zeros((1, Hkv, n_blocks * bs), dtype=torch.bool, device=dev)
                for h in range(Hkv):
                    picked = [x for x in sel[s, h].tolist() if x >= 0]
                    assert len(picked) == min(keep, n_blocks) and picked == sorted(set(picked))
                    assert 0 in picked and n_blocks - 1 in picked
                    for x in picked:
                        seen[0, h, x * bs:(x + 1) * bs] = True
                want, tol = M.attend(q[s:s + 1], k, v, seen[..., :L], scale, dtype, 2.0 ** -11 if fp8 else 2.0 ** -16,
                                     2.0 ** -24)
                assert ((out[s:s + 1].double() - want).abs() <= tol).all()
        # the trees: written behind the contexts, verified, committed
        sizes = [r.randint(1, 40) for _ in range(S)]
        T = sum(sizes)
        parents = [[-1] + [r.randrange(max(0, i - 5), i) for i in range(1, n)] for n in sizes]
        sees = [M.paths(p) for p in parents]
        mask = M.masks(sees, 2, dev)
        starts = np.concatenate([[0], np.cumsum(sizes)])
        starts_d = i32(starts.tolist())
        slots, depth = [], []
        for s, n in enumerate(sizes):
            alloc.pa_alloc_reserve_batch([s], n)
            table = alloc.pa_alloc_block_tables([s], width)[0]
            slots += [int(table[t // bs]) * bs + t % bs for t in range(int(length[s]), int(length[s]) + n)]
            depth += [int(length[s]) + int(m.sum()) - 1 for m in sees[s]]
        tables = torch.from_numpy(alloc.pa_alloc_block_tables(ids, width)).to(dev)
        with_tree = i32([int(length[s]) + sizes[s] for s in range(S)])
        slots_d, pos = i32(slots), torch.tensor(depth, dtype=torch.int64, device=dev)
        tws = torch.empty(pa.pa_decode_tree_workspace_size(T, S, Hq, Hkv, D, mcl), dtype=torch.uint8, device=dev)
        tree_rows = []
        for l in range(layers):
            q, k, v = (torch.randn((T, h, D), generator=g, device=dev).to(dtype) for h in (Hq, Hkv, Hkv))
            q = write(l, q, k, v, slots_d, pos)
            tree_rows.append(rows(l, slots_d))
            out = torch.zeros_like(q)
            args = (out, q, keys[l], values[l], tables, with_tree, starts_d, mask, mcl, scale)
            if fp8:
                pa.pa_decode_tree_fp8(*args, ks, vs, workspace=tws, status=status)
            else:
                pa.pa_decode_tree(*args, workspace=tws, status=status)
            want, tol = M.tree(q, keys[l], values[l], tables, with_tree.tolist(), starts, sees, scale, ks, vs)
            assert ((out.double() - want).abs() <= tol).all()
        draft, target = ([r.randrange(vocab) for _ in range(T)] for _ in range(2))
        accepted = torch.zeros((S, 8), dtype=torch.int32, device=dev)
        count = torch.zeros(S, dtype=torch.int32, device=dev)
        follow = torch.zeros(S, dtype=torch.int64, device=dev)
        lens = with_tree.clone()
        pa.pa_tree_accept(accepted, count, follow, lens, torch.tensor(draft, device=dev), torch.tensor(target, device=dev),
                          mask, starts_d, lens, status=status)
        pa.pa_move_tokens(keys, values, tables, lens, accepted, count, status=status)
        # (the host appends the accepted tokens, into the blocks that it reserved)
        for s in range(S):
            a = int(starts[s])
            path, token = M.accept(parents[s], draft[a:a + sizes[s]], target[a:a + sizes[s]], 8)
            assert accepted[s, :len(path)].tolist() == path and int(follow[s]) == token
            moved += sum(i != j for j, i in enumerate(path))
            for _ in path:
                alloc.pa_alloc_append(s)
            for l in range(layers):
                held[s][l] = held[s][l] + [tree_rows[l][a + i] for i in path]
        assert lens.tolist() == alloc.pa_alloc_context_lens(ids).tolist()
        for l in range(layers):
            pa.pa_key_bounds(bounds[l], steps[l], keys[l], tables, lens, 8, status=status)
    assert moved > 0 or S == 1
    assert int(status) == 0
    largest = 448.0 if fp8 else 3.3895313892515355e38
    for s in range(S):
        L = int(lens[s])
        for l in range(layers):
            assert len(held[s][l]) == L
            block, offset = tables[s, torch.arange(L, device=dev) // bs].long(), torch.arange(L, device=dev) % bs
            assert torch.equal(keys[l][block, :, offset], torch.stack([k for k, _ in held[s][l]]))
            assert torch.equal(values[l][block, :, offset], torch.stack([v for _, v in held[s][l]]))
            for b in range(-(-L // bs)):
                at = int(tables[s, b])
                hi, lo, step = M.bounds(R.cache_values(keys[l][at, 1, :min(bs, L - b * bs)]), largest)
                assert torch.equal(bounds[l][at, 1, 0].double(), hi) and torch.equal(bounds[l][at, 1, 1].double(), lo)
                assert float(steps[l][at, 1]) == step


@pytest.mark.parametrize("fp8", [False, True])
def test_pools_past_four_gigabytes(cuda_device, fp8):
    """The same blocks at the end of large pools and in small ones: the same bits."""
    import paged_kv_cache_187_gb300 as pa
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(3)
    Hkv, D, bs, used, NB = 8, 128, 16, 60, (400_000 if fp8 else 200_000)
    dtype = torch.uint8 if fp8 else torch.bfloat16
    lens, n = torch.tensor([470, 350], dtype=torch.int32, device="cuda"), 20
    small = [torch.randn((used, Hkv, bs, D), generator=g, device="cuda") for _ in range(2)]
    small = [x.to(torch.float8_e4m3fn).view(dtype) if fp8 else x.to(dtype) for x in small]
    large = [torch.empty((NB, Hkv, bs, D), dtype=dtype, device="cuda") for _ in range(2)]
    where = torch.arange(used, device="cuda") * 7 + NB - 7 * used
    for x, y in zip(large, small):
        x[where] = y
    tables = torch.randperm(used, generator=g, device="cuda").to(torch.int32)[:2 * 30].view(2, 30)
    far = where[tables.long()].to(torch.int32)
    q = torch.randn((2 * n, 16, D), generator=g, device="cuda").to(torch.bfloat16)
    starts = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    mask = torch.randint(-2 ** 31, 2 ** 31, (2 * n, 1), generator=g, device="cuda").to(torch.int32)
    path = torch.tensor([[0, 2, 5, 6], [0, 1, 4, -1]], dtype=torch.int32, device="cuda")
    count = torch.tensor([4, 3], dtype=torch.int32, device="cuda")
    new = lens - n + count
    got = []
    for (kc, vc), table in ((small, tables), (large, far)):
        bounds = torch.zeros((kc.shape[0], Hkv, 2, D), dtype=torch.int8, device="cuda")
        steps = torch.zeros((kc.shape[0], Hkv), device="cuda")
        pa.pa_key_bounds(bounds, steps, kc, table, lens, int(lens.max()))
        chosen = torch.zeros((2, Hkv, 9), dtype=torch.int32, device="cuda")
        ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
        pa.pa_select_blocks(chosen, q[::n].contiguous(), bounds, steps, table, lens, bs, 470, 1, 2, workspace=ws)
        near, tree = torch.zeros_like(q[::n].contiguous()), torch.zeros_like(q)
        args = (near, q[::n].contiguous(), kc, vc, table, lens, chosen, 0.1)
        if fp8:
            pa.pa_decode_sparse_fp8(*args, 0.5, 0.5)
            pa.pa_decode_tree_fp8(tree, q, kc, vc, table, lens, starts, mask, 470, 0.1, 0.5, 0.5, workspace=ws)
        else:
            pa.pa_decode_sparse(*args)
            pa.pa_decode_tree(tree, q, kc, vc, table, lens, starts, mask, 470, 0.1, workspace=ws)
        pa.pa_move_tokens([kc], [vc], table, new, path, count)
        torch.cuda.synchronize()
        at = table[:, :30].long()
        got.append((bounds[at], steps[at], chosen, near, tree, kc[at], vc[at]))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert bool(got[0][3].any()) and bool(got[0][4].any())


FIRST_CALLS = """
import torch
import test_gpu_sparse as S
import test_gpu_tree as T
import paged_kv_cache_187_gb300 as pa
lens = [900, 40]
att = S.sparse_case(lens, 1, 8, 2, 128, 16, torch.bfloat16, 40, 1)
sel = S.select_case(lens, 1, 8, 2, 128, 16, torch.bfloat16, 1)
far = S.select_case([40000], 1, 8, 2, 128, 16, torch.bfloat16, 1)
tree = T.make([(12, 90), (5, 700)], 8, 2, 128, 16, torch.bfloat16, 2)
sees = T.trees(tree, "paths", 1)
mask = T.M.masks(sees, 1, "cuda")
out, o = torch.zeros_like(tree["q"]), torch.zeros_like(att["q"])
ws, ws2 = T.workspace(tree, 700), torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
a, f = (torch.zeros((len(x["lens"]), 1, 2, 40), dtype=torch.int32, device="cuda") for x in (sel, far))
ids = torch.zeros(17, dtype=torch.int64, device="cuda")
moved = tree["kc"].clone(), tree["vc"].clone()
i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")
path, count, follow, new = i32(2, 4), i32(2), torch.zeros(2, dtype=torch.int64, device="cuda"), i32(2)
bounds, steps = torch.zeros((tree["kc"].shape[0], 2, 2, 128), dtype=torch.int8, device="cuda"), torch.zeros(
    (tree["kc"].shape[0], 2), device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    S.sparse_call(att, out=o, ws=ws2)
    S.select_call(sel, 40, 1, 2, out=a, ws=ws2)
    S.select_call(far, 40, 1, 2, out=f, ws=ws2)
    T.call(tree, mask, out, ws=ws, mcl=700)
    pa.pa_tree_accept(path, count, follow, new, ids, ids, mask, tree["starts_d"], tree["lens_d"])
    pa.pa_move_tokens([moved[0]], [moved[1]], tree["tables"], new, path, count)
    pa.pa_key_bounds(bounds, steps, tree["kc"], tree["tables"], tree["lens_d"], 700)
graph.replay()
torch.cuda.synchronize()
S.sparse_check(att, o)
S.select_check(sel, a, 40, 1, 2)
S.select_check(far, f, 40, 1, 2)
T.check(tree, sees, out)
assert int(count.min()) >= 1 and int(new[0]) == 90 - 12 + int(count[0])
assert bool(steps.any())
print("captured")
"""


def test_first_calls_of_a_process_in_a_capture(cuda_device):
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], env=env, cwd=here, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-3000:]
