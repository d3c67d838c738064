"""GPU: edges of the tree and sparse operators -- more new tokens than a context holds, negative
entries of a list."""
import pytest
import torch

import masked_reference as M
from test_gpu_sparse import LARGEST, layout, pool_of, sparse_call, sparse_case, sparse_check

pytestmark = pytest.mark.gpu


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
