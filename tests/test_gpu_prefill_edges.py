"""GPU: attention of ragged chunks (pa_prefill, pa_prefill_fp8) where its parts meet: values that
are infinite or NaN behind vanishing weights, bad metadata and rows with nothing to attend to, on
every way the work can be shared out."""
import pytest
import torch

import chunk_reference as R
from test_gpu_prefill import call, check, make, reference, run

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


GUARD = 1 << 16


def guarded(b, mcl):
    """A workspace of exactly the size asked for, with a guard behind it."""
    import paged_kv_cache_187_gb300 as pa
    T, Hq, D = b["q"].shape
    n = pa.pa_prefill_workspace_size(T, len(b["lens"]), Hq, b["kc"].shape[1], D, mcl)
    whole = torch.full((n + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
    assert whole.data_ptr() % 256 == 0
    return whole[:n], whole[n:]


def shared_out(ws):
    """How the last call on a workspace was shared out: its plan's third word, unless it had none."""
    cut = int(ws[8:12].view(torch.int32))
    return {0: "whole", 1: "cut"}.get(cut, "no plan")


def flags_of(b, mcl, how, **change):
    """The status of a call with some of its metadata replaced; it writes nothing past its
    workspace and its output."""
    b = dict(b, **change)
    ws, guard = guarded(b, mcl)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    room = torch.full((b["q"].numel() + 4096,), 7.0, dtype=b["q"].dtype, device="cuda")
    call(b, room[:b["q"].numel()].view(b["q"].shape), ws=ws, mcl=mcl, status=status)
    torch.cuda.synchronize()
    assert bool((guard == 0x5A).all()) and bool((room[b["q"].numel():] == 7.0).all())
    assert shared_out(ws) == how
    return int(status)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# contexts up to 1024 tokens and a unit per CTA: no plan; a longer limit: the plan kernel
@pytest.mark.parametrize("mcl,how", [(200, "no plan"), (4096, "whole")])
@pytest.mark.parametrize("D,dtype,fp8", [(128, torch.bfloat16, False), (64, torch.float16, False),
                                         (128, torch.bfloat16, True)])
def test_bad_metadata_with_and_without_a_plan(cuda_device, mcl, how, D, dtype, fp8):
    import paged_kv_cache_187_gb300 as pa
    b = make([(30, 200), (20, 100)], 4, 2, D, 16, dtype, 37, fp8)
    assert flags_of(b, mcl, how) == 0
    for starts in ([0, 40, 30], [-5, 30, 50], [0, 30, 2 ** 31 - 1], [50, 0, 50], [-2 ** 31, -7, -1]):
        assert flags_of(b, mcl, how, starts_d=i32(starts)) == pa.PA_DEVERR_BAD_LEN, starts
    for lens in ([300, 100], [-1, 100], [-2 ** 31, 100]):
        assert flags_of(b, mcl, how, lens_d=i32(lens)) == pa.PA_DEVERR_BAD_LEN, lens
    # the second row of the tables is padding past its 100 tokens, and the clamped length reaches it
    assert flags_of(b, mcl, how, lens_d=i32([200, 2 ** 31 - 1])) == pa.PA_DEVERR_BAD_LEN | pa.PA_DEVERR_BAD_BLOCK
    bad = b["tables"].clone()
    bad[0, 3], bad[1, 0] = b["kc"].shape[0], -7
    assert flags_of(b, mcl, how, tables=bad) == pa.PA_DEVERR_BAD_BLOCK
    check(b, call(b, torch.zeros_like(b["q"]), mcl=mcl))              # and all is well


@pytest.mark.parametrize("L,mcl,how", [(20, 20, "no plan"), (20, 4096, "whole"), (5000, 5000, "cut")])
@pytest.mark.parametrize("starts", [[0, 240] * 6 + [0], [0] + [240, 0] * 6, [0, 240] + [0] * 11])
def test_overlapping_chunks_stay_within_the_workspace(cuda_device, L, mcl, how, starts):
    """Chunks that overlap ask for more row tiles than the workspace has room for: flagged, and
    neither the workspace nor the output is written past its end."""
    import paged_kv_cache_187_gb300 as pa
    b = make([(20, L)] * 12, 16, 1, 128, 16, torch.bfloat16, 38)
    assert flags_of(b, mcl, how, starts_d=i32(starts)) == pa.PA_DEVERR_BAD_LEN
    check(b, call(b, torch.zeros_like(b["q"]), mcl=mcl))


# chunks whose first tokens lie before the context's start, and empty contexts: row tiles without
# a single tile of tokens, next to others
@pytest.mark.parametrize("seqs,mcl,how", [
    ([(10, 4), (3, 0), (140, 130), (1, 0), (300, 1)], 300, "no plan"),
    ([(10, 4), (3, 0), (140, 130), (1, 0), (300, 1)], 4096, "whole"),
    ([(300, 1), (1, 30000), (500, 100), (2, 0), (40, 40)], 30000, "cut"),   # such units first,
    ([(1, 30000), (600, 30), (5, 0)], 30000, "cut"),                        # .. and last
    ([(400, 0), (200, 190), (7, 9000), (0, 50), (90, 3)], 9000, "cut"),
    ([(400, 0), (3, 0)], 4096, "whole"),                                    # nothing else
])
@pytest.mark.parametrize("Hq,Hkv,D,dtype,fp8", [(8, 1, 128, torch.bfloat16, False), (8, 2, 64, torch.float16, False),
                                                (8, 2, 128, torch.float16, True)])
def test_row_tiles_without_tokens(cuda_device, seqs, mcl, how, Hq, Hkv, D, dtype, fp8):
    b = make(seqs, Hq, Hkv, D, 16, dtype, 3, fp8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws, guard = guarded(b, mcl)
    out = call(b, torch.full_like(b["q"], 7.0), ws=ws, mcl=mcl, status=status)
    assert int(status) == 0 and bool((guard == 0x5A).all()) and shared_out(ws) == how
    check(b, out)
    for s, (n, L) in enumerate(seqs):
        a = int(b["starts"][s])
        assert not out[a:a + max(n - L, 0)].any()


@pytest.mark.parametrize("mcl", [10, 4096])
def test_calls_without_a_row_of_query(cuda_device, mcl):
    b = make([(0, 10), (0, 0)], 4, 2, 128, 16, torch.float16, 61, extra=4)
    ws, guard = guarded(b, mcl)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(b, torch.full_like(b["q"], 3.0), ws=ws, mcl=mcl, status=status)
    assert int(status) == 0 and bool((out == 3).all()) and bool((guard == 0x5A).all())


@pytest.mark.parametrize("seqs,Hq,Hkv", [([(33, 1400), (1, 3000), (200, 900), (5, 256)], 8, 1),
                                         ([(2, 9001), (40, 2600)], 4, 2)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_references_move_over_8_bit_caches(cuda_device, seqs, Hq, Hkv, dtype):
    """Keys that grow along the context under large queries: most rows find their largest score
    late, and the accumulators are rescaled there, several times in a row."""
    b = make(seqs, Hq, Hkv, 128, 32, dtype, 17, True, spread=3.0)
    b["q"] *= 8.0
    moved = rows = 0
    for s, (n, L) in enumerate(seqs):
        for t, i in enumerate(b["tables"][s, :-(-L // 32)].tolist()):
            k = b["kc"][i].view(torch.float8_e4m3fn).float() * (0.1 + 2.0 * t * 32 / L)
            b["kc"][i] = k.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        # rows whose largest score in bits lies more than 16 (2^8 and 2^7 of fp16's weights, and
        # one) above that of their first 128 tokens: their reference moves
        ids = b["tables"][s, :-(-L // 32)].long()
        k = R.cache_values(b["kc"][ids], b["ks"]).transpose(1, 2).reshape(-1, Hkv, 128)[:L - n]
        x = b["q"][int(b["starts"][s]):int(b["starts"][s]) + n].double()
        y = torch.einsum("nhd,thd->nht", x, k.repeat_interleave(Hq // Hkv, 1)) * b["scale"] / 0.6931471805599453
        if L - n > 128:
            moved += int((y.amax(-1) > y[..., :128].amax(-1) + 16).sum())
            rows += y.shape[0] * y.shape[1]
    assert moved > rows // 2
    run(b)
