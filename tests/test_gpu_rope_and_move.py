"""GPU: rotary positions with the cache write (pa_rope_and_cache, _fp8) and block moves
(pa_move_blocks) against plain forms."""
import math

import numpy as np
import pytest
import torch

import chunk_reference as R

pytestmark = pytest.mark.gpu


def freqs(half, dev="cuda"):
    return (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(dev)


def rope_case(T, Hq, Hkv, D, rot, bs, axes, dtype, fp8, seed, top=60000, fused=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    NB = -(-T // bs) + 3
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda").to(dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    slots = torch.randperm(NB * bs, generator=g, device="cuda")[:T].to(torch.int32)
    pos = torch.randint(0, top, (axes, T), generator=g, device="cuda")
    cdt = torch.uint8 if fp8 else dtype
    pools = [torch.randint(0, 100, (NB, Hkv, bs, D), generator=g, device="cuda").to(cdt) for _ in range(2)]
    half = rot // 2
    pair_axes = None if axes == 1 else [i * axes // half for i in range(half)]
    return dict(q=q, k=k, v=v, slots=slots, pos=pos, kp=pools[0], vp=pools[1], freq=freqs(half),
                pair_axes=pair_axes, fp8=fp8)


def rope_call(b, out, interleaved=False, status=None, **kw):
    import paged_kv_cache_187_gb300 as pa
    args = (out, b["q"], b["k"], b["v"], b["kp"], b["vp"], b["slots"], b["pos"], b["freq"])
    kw = dict(pair_axes=b["pair_axes"], interleaved=interleaved, status=status, **kw)
    if b["fp8"]:
        pa.pa_rope_and_cache_fp8(*args, 0.03, 0.02, **kw)
    else:
        pa.pa_rope_and_cache(*args, **kw)
    return out


def angle_error(b):
    """Bound on |rotated - exact| over |u| + |v| of the pair, [T, 1, rot dims' pairs]: the
    fraction of a turn rounded to fp32 (pi 2^-24), cos and sin good to 2^-23, three fp32
    roundings (2^-24 each), and the frequency as a 64-bit fraction (2^-51 of the angle)."""
    far = float((b["pos"].abs().amax().double() * b["freq"].double().amax()).cpu())
    return (math.pi + 2 + 3) * 2.0 ** -24 + far * 2.0 ** -51


def check_rope(b, out, before, interleaved):
    dtype = b["q"].dtype
    u = R.half_step(dtype)
    eps = angle_error(b)
    want, size = R.rope(b["q"], b["pos"], b["freq"], b["pair_axes"], interleaved)
    assert ((out.double() - want).abs() <= u * want.abs() + eps * size).all()
    rot = 2 * b["freq"].numel()
    assert torch.equal(out[..., rot:], b["q"][..., rot:])
    want, size = R.rope(b["k"], b["pos"], b["freq"], b["pair_axes"], interleaved)
    bs = b["kp"].shape[2]
    live = b["slots"] >= 0
    s = b["slots"][live].long()
    got_k, got_v = b["kp"][s // bs, :, s % bs], b["vp"][s // bs, :, s % bs]
    if b["fp8"]:
        got = got_k.view(torch.float8_e4m3fn).double() * 0.03
        y = want[live]
        # half a step of e4m3: 2^-4 of the value, or 2^-10 scale below its normal range; the
        # reciprocal scale and the product one fp32 rounding each
        assert ((got - y).abs() <= (2.0 ** -4 + 2.0 ** -22) * y.abs() + 2.0 ** -10 * 0.03 + 2 * eps * size[live]).all()
        r = torch.tensor(1.0, dtype=torch.float32) / torch.tensor(0.02, dtype=torch.float32)
        v8 = (b["v"][live].float() * r.cuda()).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(got_v, v8)
    else:
        y = want[live]
        assert ((got_k.double() - y).abs() <= u * y.abs() + eps * size[live]).all()
        assert torch.equal(got_v, b["v"][live])
        assert torch.equal(got_k[..., rot:], b["k"][live][..., rot:])
    # every other slot is as it was
    for pool, old in zip((b["kp"], b["vp"]), before):
        a, o = pool.transpose(1, 2).reshape(-1, *pool.shape[1:2], pool.shape[3]), old.transpose(1, 2).reshape(-1, *old.shape[1:2], old.shape[3])
        rest = torch.ones(a.shape[0], dtype=torch.bool, device="cuda")
        rest[s] = False
        assert torch.equal(a[rest], o[rest])


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,bs,axes,dtype,fp8,interleaved", [
    (1, 4, 4, 64, 64, 16, 1, torch.bfloat16, False, False),
    (3, 32, 8, 128, 128, 16, 1, torch.bfloat16, False, False),
    (37, 8, 2, 128, 128, 32, 3, torch.float16, False, False),
    (130, 5, 1, 128, 48, 16, 2, torch.bfloat16, False, True),
    (65, 6, 3, 64, 32, 16, 4, torch.float16, False, True),
    (33, 8, 8, 256, 256, 16, 3, torch.bfloat16, False, False),
    (41, 8, 2, 128, 128, 16, 3, torch.bfloat16, True, False),
    (9, 7, 1, 64, 64, 32, 1, torch.float16, True, True),
    (18, 2, 2, 96, 16, 16, 1, torch.float16, True, False),
    (5, 2, 1, 80, 80, 16, 2, torch.bfloat16, False, False),
])
def test_rope_matches_the_formula(cuda_device, T, Hq, Hkv, D, rot, bs, axes, dtype, fp8, interleaved):
    b = rope_case(T, Hq, Hkv, D, rot, bs, axes, dtype, fp8, 5 + T)
    before = (b["kp"].clone(), b["vp"].clone())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = rope_call(b, torch.empty((T, Hq, D), dtype=dtype, device="cuda"), interleaved, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    check_rope(b, out, before, interleaved)


def test_rope_far_and_negative_positions(cuda_device):
    for top, shift in ((2 ** 31, 0), (2 ** 31, -2 ** 31), (4000, -2000)):
        b = rope_case(50, 4, 2, 128, 128, 16, 1, torch.float16, False, 3, top=top)
        b["pos"] += shift
        before = (b["kp"].clone(), b["vp"].clone())
        out = rope_call(b, torch.empty((50, 4, 128), dtype=torch.float16, device="cuda"))
        check_rope(b, out, before, False)


def test_rope_padding_bad_slots_and_in_place(cuda_device):
    b = rope_case(23, 8, 2, 128, 128, 16, 1, torch.bfloat16, False, 4, fused=False)
    b["slots"][::3] = -1
    before = (b["kp"].clone(), b["vp"].clone())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = b["q"].clone()
    rope_call(b, b["q"], status=status)                 # in place
    assert int(status) == 0
    out, b["q"] = b["q"], q
    check_rope(b, out, before, False)
    import paged_kv_cache_187_gb300 as pa
    b["slots"][1] = b["kp"].shape[0] * 16               # just past the pool
    kp, vp = b["kp"].clone(), b["vp"].clone()
    rope_call(b, torch.empty_like(q), status=status)
    assert int(status) == pa.PA_DEVERR_BAD_SLOT
    assert torch.equal(kp, b["kp"]) and torch.equal(vp, b["vp"])   # nothing new was written


def test_rope_without_turning_is_reshape_and_cache(cuda_device):
    """At position 0 nothing turns: the pools are what pa_reshape_and_cache leaves."""
    import paged_kv_cache_187_gb300 as pa
    for fp8 in (False, True):
        b = rope_case(29, 4, 2, 128, 128, 16, 1, torch.bfloat16, fp8, 6, fused=False)
        b["pos"].zero_()
        kp, vp = b["kp"].clone(), b["vp"].clone()
        out = rope_call(b, torch.empty_like(b["q"]))
        if fp8:
            pa.pa_reshape_and_cache_fp8(b["k"], b["v"], kp, vp, b["slots"], 0.03, 0.02)
        else:
            pa.pa_reshape_and_cache(b["k"], b["v"], kp, vp, b["slots"])
        assert torch.equal(out, b["q"])
        assert torch.equal(kp.view(torch.uint8), b["kp"].view(torch.uint8))
        assert torch.equal(vp.view(torch.uint8), b["vp"].view(torch.uint8))


@pytest.mark.parametrize("layers,NB,Hkv,bs,D,dtype", [
    (1, 9, 1, 16, 64, torch.float16),
    (3, 64, 8, 16, 128, torch.bfloat16),
    (65, 20, 2, 32, 64, torch.bfloat16),        # two launches
    (2, 40, 3, 16, 128, torch.uint8),
    (2, 24, 1, 16, 8, torch.float16),
])
def test_move_blocks(cuda_device, layers, NB, Hkv, bs, D, dtype):
    import paged_kv_cache_187_gb300 as pa
    rng = np.random.default_rng(layers + NB)
    keep = NB - NB // 3
    src = np.sort(rng.choice(np.arange(keep, NB), NB - keep - 1, replace=False))
    dst = rng.permutation(keep)[:src.size]
    pairs = torch.from_numpy(np.stack([src, dst], 1).astype(np.int32)).cuda()
    pools = [torch.randint(0, 120, (NB, Hkv, bs, D), device="cuda").to(dtype) for _ in range(2 * layers)]
    want = [p.clone() for p in pools]
    for p in want:
        p[torch.from_numpy(dst).cuda()] = p[torch.from_numpy(src).cuda()]
    tables = rng.integers(-1, NB, size=(17, 23)).astype(np.int32)
    t = torch.from_numpy(tables).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_move_blocks(pools[:layers], pools[layers:], pairs, block_tables=t, status=status)
    place = dict(zip(src.tolist(), dst.tolist()))
    assert np.array_equal(t.cpu().numpy(), np.vectorize(lambda b: place.get(b, b))(tables))
    for a, b in zip(pools, want):
        assert torch.equal(a, b)
    assert int(status) == 0
    # pairs outside the pool are skipped and reported, the others moved
    pairs[0, 1] = NB
    status.zero_()
    pa.pa_move_blocks(pools[:layers], pools[layers:], pairs, status=status)
    assert int(status) == pa.PA_DEVERR_BAD_BLOCK
    for a, b in zip(pools, want):
        assert torch.equal(a, b)


def test_move_flags_pairs_out_of_order_and_moves_tables_alone(cuda_device):
    import paged_kv_cache_187_gb300 as pa
    pools = [torch.randint(0, 100, (12, 2, 16, 64), device="cuda").to(torch.float16) for _ in range(2)]
    want = pools[0].clone()
    pairs = torch.tensor([[9, 1], [8, 0]], dtype=torch.int32, device="cuda")
    want[1], want[0] = want[9], want[8]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_move_blocks(pools[:1], pools[1:], pairs, status=status)
    assert int(status) == pa.PA_DEVERR_BAD_BLOCK             # reported, and copied all the same
    assert torch.equal(pools[0], want)


def test_rope_and_move_in_a_graph(cuda_device):
    import paged_kv_cache_187_gb300 as pa
    b = rope_case(33, 8, 2, 128, 128, 16, 3, torch.bfloat16, False, 8)
    out = torch.zeros((33, 8, 128), dtype=torch.bfloat16, device="cuda")
    before = (b["kp"].clone(), b["vp"].clone())
    NB = b["kp"].shape[0]
    free = torch.zeros((2 * NB, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    pairs = torch.tensor([[NB, 0], [NB + 1, 1]], dtype=torch.int32, device="cuda")
    table = torch.arange(2 * NB, dtype=torch.int32, device="cuda")[None].contiguous()
    rope_call(b, out)
    torch.cuda.synchronize()
    eager = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rope_call(b, out)
        pa.pa_move_blocks([free], [free.clone()], pairs, block_tables=table)
    out.zero_()
    b["kp"].copy_(before[0])
    b["vp"].copy_(before[1])
    free[NB:NB + 2] = 3.0
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    check_rope(b, out, before, False)
    assert (free[:2] == 3).all() and table[0, NB:NB + 2].tolist() == [0, 1]
