"""GPU: attention of ragged chunks (pa_prefill, pa_prefill_fp8) where its parts meet: values that
are infinite or NaN behind vanishing weights, on every way the work can be shared out."""
import pytest
import torch

from test_gpu_prefill import call, make, reference

pytestmark = pytest.mark.gpu


def check_classes(b, out):
    """Infinities and NaN where the 64-bit form has them, the rest within its tolerance."""
    want, tol = reference(b)
    n = int(b["starts"][-1])
    got, want, tol = out[:n].double(), want[:n], tol[:n]
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    odd = ~torch.isfinite(want)
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
    assert bool((((got - want).abs() <= tol) | odd).all())
    return want


# (new tokens, context, the token with nearly all the weight, tokens with infinite and NaN values):
# values before and after the large weight, in tiles that every row sees whole and in the last
# ones; calls without a plan, units taken whole, units cut into shares, rows that both streams share
@pytest.mark.parametrize("seqs,Hq,Hkv,mcl", [
    ([(40, 300, 3, 200, 290)], 8, 2, 300),                        # not planned
    ([(40, 300, 299, 5, 270)], 8, 2, 300),
    ([(200, 700, 400, 90, 650)], 8, 2, 700),                      # rows for both streams
    ([(1, 5000, 17, 4998, 2600)], 8, 1, 5000),                    # cut; shared rows
    ([(1, 5000, 4990, 20, 2600)], 8, 1, 5000),
    ([(90, 9000, 30, 8950, 4321)], 16, 1, 9000),                  # cut; rows for both streams
    ([(33, 2600, 2580, 1, 2599), (2, 9001, 100, 9000, 7000)], 4, 2, 9001),
    ([(3, 60 + i, 1, 50, 20) for i in range(400)], 4, 2, 2000),   # units taken whole
])
@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (64, torch.float16), (128, torch.float16)])
@pytest.mark.parametrize("gap", [40.0, 200.0])
def test_infinite_values_behind_vanishing_weights(cuda_device, seqs, Hq, Hkv, mcl, D, dtype, gap):
    """A softmax weight is never 0, however small: an infinite value that a row sees comes out as
    infinity, two of both signs and NaN as NaN.  Against the token with nearly all the weight the
    others' weights are about 2^-gap: below fp16's range, and below fp32's."""
    inf, nan = float("inf"), float("nan")
    b = make([s[:2] for s in seqs], Hq, Hkv, D, 16, dtype, 97)
    b["q"] *= 0.1
    b["q"][..., 0] = 16.0
    key = gap / (16.0 * b["scale"] * 1.4426950408889634)
    for s, (_, L, top, t0, t1) in enumerate(seqs):
        at = lambda t: (int(b["tables"][s, t // 16]), slice(None), t % 16)
        live = b["tables"][s, :-(-L // 16)].long()
        b["kc"][live, :, :, 0] = 0
        b["kc"][at(top)][..., 0] = key
        for t, dims in ((t0, {5: inf, 7: -inf, 11: inf, 13: nan, D - 1: inf}),
                        (t1, {11: -inf, 17: inf, 33: -inf, D - 2: nan})):
            for d, x in dims.items():
                b["vc"][at(t)][:, d] = x
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(b, torch.full_like(b["q"], 7.0), mcl=mcl, status=status)
    assert int(status) == 0
    want = check_classes(b, out)
    assert bool(torch.isinf(want).any()) and bool(torch.isnan(want).any())
