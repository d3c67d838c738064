"""GPU: edges of the tree and sparse operators -- scores of -inf before and within a tree, more new
tokens than a context holds, negative entries of a list."""
import math

import pytest
import torch

import chunk_reference as R
import masked_reference as M
from test_gpu_prefill import make
from test_gpu_sparse import LARGEST, layout, pool_of, sparse_call, sparse_case, sparse_check
from test_gpu_tree import call, trees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,Hq,Hkv,D,dtype", [
    ([(20, 300), (1, 200), (40, 150)], 8, 2, 128, torch.bfloat16),
    ([(8, 5000)], 8, 1, 64, torch.float16),                   # cut into shares, rows for one stream
    ([(64, 9000), (33, 2600)], 16, 2, 128, torch.bfloat16),
    ([(1 + i * 7 % 64, 200 + i * 131 % 1500) for i in range(60)], 4, 4, 64, torch.float16),
])
@pytest.mark.parametrize("where", ["first tile", "a late token", "all before the tree", "everything"])
def test_scores_of_minus_infinity_in_and_before_a_tree(cuda_device, seqs, Hq, Hkv, D, dtype, where):
    """Infinite keys where every query is positive: those tokens have no weight, and a row that sees
    no other is a zero row."""
    b = make(seqs, Hq, Hkv, D, 16, dtype, 19)
    sees = trees(b, "paths", 4)
    b["q"][..., 3] = b["q"][..., 3].abs() + 0.5
    want = torch.zeros(b["q"].shape, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(want)
    for s, (n, L) in enumerate(seqs):
        hide = torch.zeros(L, dtype=torch.bool, device="cuda")
        if where == "first tile":
            hide[:64] = True
        elif where == "a late token":
            hide[L - n - 1:L - n + 1] = True
        elif where == "all before the tree":
            hide[:L - n] = True
        else:
            hide[:] = True
        t = hide.nonzero()[:, 0]
        b["kc"][b["tables"][s, t // 16].long(), :, t % 16, 3] = -math.inf
        k = M.gather(b["kc"], b["tables"][s], L)
        k[t] = 0
        v = M.gather(b["vc"], b["tables"][s], L)
        seen = torch.ones((n, L), dtype=torch.bool, device="cuda")
        seen[:, L - n:] = sees[s].cuda().tril()
        seen &= ~hide
        a = int(b["starts"][s])
        want[a:a + n], tol[a:a + n] = M.attend(b["q"][a:a + n], k, v, seen[:, None].expand(n, Hkv, L), b["scale"], dtype,
                                               R.half_step(dtype), 2.0 ** -32 if dtype == torch.float16 else 0.0)
    mask = M.masks(sees, 2, "cuda")
    out = call(b, mask, torch.full_like(b["q"], 7.0))
    assert bool(torch.isfinite(out).all())
    assert bool(((out.double() - want).abs() <= tol).all())
    if where == "everything":
        assert not bool(out.any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.uint8])
def test_more_new_tokens_than_the_context_bound_every_block(cuda_device, dtype):
    """Without a flag, as a bound on new tokens may be larger than a context."""
    import paged_kv_cache_187_gb300 as pa
    g = torch.Generator(device="cuda").manual_seed(8)
    lens, bs, D = [1, 40, 0, 200], 16, 64
    tables, lens_d, NB = layout(lens, bs, g)
    k = pool_of((NB, 2, bs, D), dtype, g)
    starts = torch.tensor([0, 300, 341, 350, 551], dtype=torch.int32, device="cuda")
    got = []
    for query_starts in (starts, None):
        bounds = torch.full((NB, 2, 2, D), 99, dtype=torch.int8, device="cuda")
        steps = torch.full((NB, 2), 99.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pa.pa_key_bounds(bounds, steps, k, tables, lens_d, 300, query_starts=query_starts, status=status)
        assert int(status) == 0
        got.append((bounds, steps))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    value = (lambda x: x.view(torch.float8_e4m3fn).double()) if dtype == torch.uint8 else (lambda x: x.double())
    for s, L in enumerate(lens):
        for x in range(-(-L // bs)):
            ph = int(tables[s, x])
            for h in range(2):
                hi, lo, step = M.bounds(value(k[ph, h, :min(bs, L - x * bs)]), LARGEST[dtype])
                assert torch.equal(got[0][0][ph, h, 0].double(), hi) and torch.equal(got[0][0][ph, h, 1].double(), lo)
                assert float(got[0][1][ph, h]) == step


@pytest.mark.parametrize("entry", [-2, -77, -2 ** 31])
def test_negative_entries_of_a_list_are_skipped(cuda_device, entry):
    b = sparse_case([500, 320], 1, 4, 2, 128, 16, torch.bfloat16, 40, 8, pick=20)
    b["selected"][:, :, :, 7:9] = -1
    clean = sparse_call(b)
    sparse_check(b, clean)
    b["selected"][:, :, :, 7:9] = entry
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = sparse_call(b, status=status)
    assert torch.equal(out, clean) and int(status) == 0
