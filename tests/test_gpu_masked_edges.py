"""GPU: edges of the tree and sparse operators -- negative entries of a list."""
import pytest
import torch

from test_gpu_sparse import sparse_call, sparse_case, sparse_check

pytestmark = pytest.mark.gpu


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
