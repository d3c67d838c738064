"""GPU: attention of ragged chunks of new tokens over the paged cache (pa_prefill,
pa_prefill_fp8) against the plain 64-bit form, within the tolerance derived there."""
import numpy as np
import pytest
import torch

import chunk_reference as R

pytestmark = pytest.mark.gpu


def make(seqs, Hq, Hkv, D, bs, dtype, seed, fp8=False, spread=1.0, extra=0, dev="cuda"):
    """seqs: (new tokens, context length) each.  Unused blocks and the rows of used blocks
    past their context hold NaN."""
    g = torch.Generator(device=dev).manual_seed(seed)
    need = [-(-L // bs) for _, L in seqs]
    NB = sum(need) + sum(need) // 5 + 2
    order = torch.randperm(NB, generator=g, device=dev).to(torch.int32)
    tables = torch.full((len(seqs), max(max(need), 1)), -1, dtype=torch.int32, device=dev)
    shape = (NB, Hkv, bs, D)
    kf = torch.randn(shape, generator=g, device=dev) * spread
    vf = torch.randn(shape, generator=g, device=dev)
    ks, vs = (0.03, 0.02) if fp8 else (1.0, 1.0)
    if fp8:
        kc = (kf / ks).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        vc = (vf / vs).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        nan = 0x7F
    else:
        kc, vc, nan = kf.to(dtype), vf.to(dtype), float("nan")
    at = 0
    for s, n in enumerate(need):
        ids = order[at:at + n]
        at += n
        tables[s, :n] = ids
        if seqs[s][1] % bs:
            kc[ids[-1].long(), :, seqs[s][1] % bs:] = nan
            vc[ids[-1].long(), :, seqs[s][1] % bs:] = nan
    kc[order[at:].long()] = nan
    vc[order[at:].long()] = nan
    starts = np.concatenate([[0], np.cumsum([n for n, _ in seqs])]).astype(np.int32)
    T = int(starts[-1]) + extra
    q = torch.randn((T, Hq, D), generator=g, device=dev).to(dtype)
    return dict(q=q, kc=kc, vc=vc, tables=tables, lens=[L for _, L in seqs], starts=starts,
                lens_d=torch.tensor([L for _, L in seqs], dtype=torch.int32, device=dev),
                starts_d=torch.from_numpy(starts).to(dev), scale=D ** -0.5, fp8=fp8, ks=ks, vs=vs)


def workspace(b, mcl):
    import paged_kv_cache_187_gb300 as pa
    T, Hq, D = b["q"].shape
    n = pa.pa_prefill_workspace_size(T, len(b["lens"]), Hq, b["kc"].shape[1], D, mcl)
    # (stale contents must not matter)
    return torch.full((max(n, 256),), 0xA5, dtype=torch.uint8, device="cuda")


def call(b, out, ws=None, mcl=None, status=None, stream=None):
    import paged_kv_cache_187_gb300 as pa
    mcl = max(b["lens"] + [0]) if mcl is None else mcl
    ws = workspace(b, mcl) if ws is None else ws
    args = (out, b["q"], b["kc"], b["vc"], b["tables"], b["lens_d"], b["starts_d"], mcl, b["scale"])
    if b["fp8"]:
        pa.pa_prefill_fp8(*args, b["ks"], b["vs"], workspace=ws, status=status, stream=stream)
    else:
        pa.pa_prefill(*args, workspace=ws, status=status, stream=stream)
    return out


def reference(b):
    return R.prefill(b["q"], b["kc"], b["vc"], b["tables"], b["lens"], b["starts"], b["scale"],
                     b["ks"], b["vs"])


def check(b, out, ref=None):
    want, tol = ref or reference(b)
    n = int(b["starts"][-1])
    err = (out[:n].double() - want[:n]).abs()
    assert torch.isfinite(out[:n]).all()
    bad = err > tol[:n]
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} beyond tolerance, worst ratio "
                           f"{float((err / tol[:n].clamp_min(1e-30))[bad].max()):.3g}, first at "
                           f"{bad.nonzero()[0].tolist()}")


def run(b):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(b, torch.full_like(b["q"], 7.0), status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    check(b, out)
    return out


# from one token to several tiles; chunk and context around the tile's and blocks' edges
SEQS = [(1, 1), (5, 5), (1, 130), (17, 317), (128, 128), (129, 129), (31, 31), (0, 40), (40, 300)]


@pytest.mark.parametrize("Hq,Hkv,D,bs,dtype,fp8", [
    (4, 4, 128, 16, torch.bfloat16, False),
    (8, 2, 128, 16, torch.bfloat16, False),
    (8, 2, 64, 32, torch.float16, False),
    (4, 4, 64, 16, torch.bfloat16, False),
    (16, 1, 128, 32, torch.float16, False),
    (7, 1, 128, 16, torch.float16, False),      # 18 tokens of 7 heads per stream
    (10, 2, 64, 32, torch.bfloat16, False),     # groups of 5
    (6, 2, 128, 32, torch.bfloat16, False),     # groups of 3
    (8, 2, 128, 16, torch.bfloat16, True),
    (8, 8, 128, 32, torch.float16, True),
    (13, 1, 128, 32, torch.bfloat16, True),
])
def test_ragged_chunks(cuda_device, Hq, Hkv, D, bs, dtype, fp8):
    run(make(SEQS, Hq, Hkv, D, bs, dtype, 11 + Hq + D, fp8))


@pytest.mark.parametrize("Hq,Hkv,D,bs,dtype,fp8", [
    (8, 2, 128, 16, torch.bfloat16, False),
    (4, 4, 64, 32, torch.float16, False),
    (8, 2, 128, 32, torch.float16, True),
])
def test_many_items_and_tiles_per_cta(cuda_device, Hq, Hkv, D, bs, dtype, fp8):
    """Several items in a row on each CTA, each of many tiles of which only the last few are
    partly masked, next to items where all are: the tile ring wraps at different places."""
    rng = np.random.default_rng(7)
    seqs = [(int(n), int(n + p)) for n, p in zip(rng.integers(1, 60, 150), rng.integers(0, 2500, 150))]
    seqs += [(0, 0), (700, 700), (3, 4001), (257, 1500)]
    run(make(seqs, Hq, Hkv, D, bs, dtype, 5, fp8))


# Few units, so that the work is cut into shares at places that move with every length: units
# begun in one share and ended several later, shares that hold the ends of two, rows for one
# stream only (whose tiles the streams share) and for both, odd and even numbers of tiles.
@pytest.mark.parametrize("seqs,Hq,Hkv,D,bs,dtype,fp8", [
    ([(1, 5000)], 8, 1, 128, 16, torch.bfloat16, False),
    ([(1, 129)], 2, 2, 128, 16, torch.float16, False),
    ([(2, 9001), (1, 77), (33, 2600)], 4, 2, 128, 32, torch.float16, False),
    ([(20, 6000), (1, 8191), (70, 4000)], 16, 2, 128, 16, torch.bfloat16, False),
    ([(100, 3000)], 3, 1, 64, 16, torch.bfloat16, False),
    ([(1, 20000), (64, 700)], 5, 1, 64, 32, torch.float16, False),
    ([(1, 5000)], 8, 1, 128, 32, torch.bfloat16, True),
    ([(20, 6000), (1, 8191), (70, 4000)], 16, 2, 128, 16, torch.float16, True),
    ([(300, 300)], 16, 1, 128, 16, torch.bfloat16, False),
    ([(5, 640), (5, 641), (5, 639), (0, 100), (5, 5)], 6, 6, 128, 16, torch.bfloat16, False),
])
def test_work_cut_into_shares(cuda_device, seqs, Hq, Hkv, D, bs, dtype, fp8):
    run(make(seqs, Hq, Hkv, D, bs, dtype, 23 + Hq, fp8))
