"""GPU: attention over selected blocks (pa_decode_sparse, _fp8) where scores are -inf (such a token
has no weight, wherever it stands in the tiles of a row), and over the longest lists."""
import math

import pytest
import torch

import masked_reference as M
from test_gpu_sparse import sparse_call, sparse_case, sparse_check, sparse_reference, sparse_run

pytestmark = pytest.mark.gpu

# (sequences, query heads, kv heads, head size, type): rows with a cluster each, and whole rows; query
# heads one to a kv head and in groups of up to 8 and up to 16
ROWS = [
    (1, 8, 2, 128, torch.bfloat16),
    (1, 16, 1, 64, torch.float16),
    (1, 2, 2, 128, torch.float16),
    (1, 3, 3, 64, torch.bfloat16),
    (120, 8, 4, 128, torch.float16),
    (80, 36, 4, 64, torch.bfloat16),
    (320, 2, 2, 64, torch.bfloat16),
    (320, 2, 2, 128, torch.float16),
]


def low_case(seqs, tokens, Hq, Hkv, D, bs, dtype, hidden, seed=41):
    """Lists of all blocks of `tokens` tokens each, and the same without the blocks that `hidden` (block
    -> bool) names, whose keys have -inf where every query is positive: scores of -inf, weights of 0,
    so both are the same attention."""
    blocks = -(-tokens // bs)
    b = sparse_case([tokens] * seqs, 1, Hq, Hkv, D, bs, dtype, blocks, seed, pick=blocks)
    b["q"][..., 5] = b["q"][..., 5].abs() + 0.5
    gone = [x for x in range(blocks) if hidden(x)]
    b["kc"][b["tables"][:, gone].reshape(-1).long(), :, :, 5] = -math.inf
    left = [x for x in range(blocks) if not hidden(x)]
    row = torch.tensor(left + [-1] * len(gone), dtype=torch.int32, device="cuda")
    return b, dict(b, selected=row.expand(b["selected"].shape).contiguous())


def low_check(b, reduced):
    """Every row against the 64-bit form over the reduced lists (a few sequences of many)."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = sparse_call(b, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert bool(torch.isfinite(out).all())
    for s in sorted({0, len(b["lens"]) // 2, len(b["lens"]) - 1}):
        one = dict(reduced, q=b["q"][s:s + 1], tables=b["tables"][s:s + 1], lens=b["lens"][s:s + 1],
                   selected=reduced["selected"][s:s + 1])
        sparse_check(one, out[s:s + 1])


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("seqs,Hq,Hkv,D,dtype", ROWS)
@pytest.mark.parametrize("where", ["last token", "first block", "first half", "last half"])
def test_scores_of_minus_infinity_have_no_weight(cuda_device, where, seqs, Hq, Hkv, D, dtype, bs):
    blocks = 33
    tokens = (blocks - 1) * bs + 1                 # the last block holds one token
    hidden = {"last token": lambda x: x == blocks - 1, "first block": lambda x: x == 0,
              "first half": lambda x: x < 17, "last half": lambda x: x > 16}[where]
    low_check(*low_case(seqs, tokens, Hq, Hkv, D, bs, dtype, hidden))


@pytest.mark.parametrize("seqs,Hq,Hkv,D", [(1, 8, 2, 128), (1, 16, 1, 64), (120, 8, 4, 128), (80, 36, 4, 64)])
def test_minus_infinity_for_one_head_of_a_group(cuda_device, seqs, Hq, Hkv, D):
    """Products past fp32's range in the first block, of the first query head of each group alone."""
    b, reduced = low_case(seqs, 500, Hq, Hkv, D, 16, torch.bfloat16, lambda x: x == 0)
    g = Hq // Hkv
    b["kc"][b["tables"][:, 1:].reshape(-1).long(), :, :, 5] = 0
    b["kc"][b["tables"][:, 0].long(), :, :, 5] = -1e20
    b["q"][..., 5] = 0
    b["q"][:, :, ::g, 5] = 1e20
    out = sparse_call(b)
    for s in sorted({0, seqs // 2, seqs - 1}):
        for lists in (b, reduced):
            one = dict(b, q=b["q"][s:s + 1], tables=b["tables"][s:s + 1], lens=b["lens"][s:s + 1],
                       selected=lists["selected"][s:s + 1])
            want, tol = sparse_reference(one)
            heads = torch.zeros(Hq, dtype=torch.bool, device="cuda")
            heads[::g] = True
            heads = heads if lists is reduced else ~heads
            got = out[s:s + 1, :, heads].double()
            assert bool(((got - want[:, :, heads]).abs() <= tol[:, :, heads]).all())


@pytest.mark.parametrize("seqs", [1, 100])
@pytest.mark.parametrize("Hq,Hkv,bs,dtype", [(8, 2, 16, torch.bfloat16), (16, 1, 32, torch.float16), (4, 4, 16, torch.float16)])
def test_rows_of_nothing_but_minus_infinity_are_zero_over_8_bits(cuda_device, seqs, Hq, Hkv, bs, dtype):
    """(An 8-bit cache has no infinities: the query brings them.)"""
    b = sparse_case([300] * seqs, 1, Hq, Hkv, 128, bs, dtype, 20, 43, fp8=True, pick=20)
    one = torch.ones((), device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    b["kc"][..., 5] = torch.where(b["kc"][..., 5] == 0x7F, b["kc"][..., 5], one)
    clean = sparse_run(b) if seqs == 1 else sparse_call(b)
    b["q"][:, :, 0, 5] = -math.inf
    out = sparse_call(b)
    assert not bool(out[:, :, 0].any())
    assert torch.equal(out[:, :, 1:], clean[:, :, 1:])


@pytest.mark.parametrize("seqs,Hq,Hkv,D,dtype", ROWS)
def test_rows_of_nothing_but_minus_infinity_are_zero(cuda_device, seqs, Hq, Hkv, D, dtype):
    b, _ = low_case(seqs, 500, Hq, Hkv, D, 16, dtype, lambda x: True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = sparse_call(b, status=status)
    assert not bool(out.any()) and int(status) == 0


@pytest.mark.parametrize("seqs,Hq,Hkv,D,dtype", ROWS)
def test_a_nan_beside_minus_infinity_is_nan(cuda_device, seqs, Hq, Hkv, D, dtype):
    """One NaN score in a tile of -inf, which is otherwise without weight."""
    b, _ = low_case(seqs, 500, Hq, Hkv, D, 16, dtype, lambda x: x < 4)
    b["kc"][int(b["tables"][0, 2]), 0, 9, 7] = math.nan
    out = sparse_call(b)
    g = Hq // Hkv
    want = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    want[0, 0, :g] = True
    assert torch.equal(torch.isnan(out), want)


@pytest.mark.parametrize("seqs,Hq,dtype", [(300, 1, torch.bfloat16), (300, 4, torch.float16), (1, 4, torch.bfloat16)])
def test_the_longest_lists(cuda_device, seqs, Hq, dtype):
    """65,536 entries, in whole rows and in a cluster: every wait within its limit."""
    g = torch.Generator(device="cuda").manual_seed(6)
    blocks, bs, D = 65536, 16, 64
    L = blocks * bs - 5
    kc, vc = (torch.randn((blocks, 1, bs, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    kc[-1, :, bs - 5:] = vc[-1, :, bs - 5:] = math.nan
    row = torch.arange(blocks, dtype=torch.int32, device="cuda")
    b = dict(q=torch.randn((seqs, 1, Hq, D), generator=g, device="cuda").to(dtype), kc=kc, vc=vc,
             tables=row.expand(seqs, blocks).contiguous(), lens=[L] * seqs,
             lens_d=torch.full((seqs,), L, dtype=torch.int32, device="cuda"),
             selected=row.expand(seqs, 1, 1, blocks).contiguous(), scale=D ** -0.5, fp8=False)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = sparse_call(b, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    k, v = kc.transpose(1, 2).reshape(-1, 1, D)[:L].double(), vc.transpose(1, 2).reshape(-1, 1, D)[:L].double()
    seen = torch.ones((1, 1, L), dtype=torch.bool, device="cuda")
    for s in sorted({0, seqs // 2, seqs - 1}):
        want, tol = M.attend(b["q"][s], k, v, seen, b["scale"], dtype, 2.0 ** -16,
                             2.0 ** -24 if dtype == torch.float16 else 0.0)
        assert bool(((out[s].double() - want).abs() <= tol).all())
