"""GPU: rotary positions with frequencies of every size and sign and with wide heads, and block
tables rewritten without pools or with millions of entries."""
import math

import numpy as np
import pytest
import torch

import chunk_reference as R
from test_gpu_rope_and_move import check_rope, rope_call, rope_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,dtype,fp8,interleaved", [
    (19, 3, 2, 512, 256, torch.bfloat16, False, False),
    (5, 2, 1, 1024, 256, torch.float16, False, True),
    (7, 2, 1, 1024, 16, torch.bfloat16, True, False),
    (11, 5, 1, 336, 144, torch.float16, True, True),      # 21 units a head: one thread stays idle
    (3, 1, 1, 544, 240, torch.bfloat16, False, False),    # 34 units: one head at a time
])
def test_rope_of_wide_heads(cuda_device, T, Hq, Hkv, D, rot, dtype, fp8, interleaved):
    b = rope_case(T, Hq, Hkv, D, rot, 16, 1, dtype, fp8, 5 + D)
    before = (b["kp"].clone(), b["vp"].clone())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = rope_call(b, torch.empty((T, Hq, D), dtype=dtype, device="cuda"), interleaved, status)
    assert int(status) == 0
    check_rope(b, out, before, interleaved)


@pytest.mark.parametrize("top", [1, 1000, 2 ** 28])
def test_rope_frequencies_of_every_size_and_sign(cuda_device, top):
    """64 frequencies from fp32's smallest subnormal to just below 2^24, of both signs, and 0.
    Position times frequency is exact in fp64 (28 and 24 bits), and so is its reduction there."""
    bits = [0x00000001, 0x00000400, 0x007FFFFF, 0x00800000, 0x0B7FFFFF]
    exps = np.linspace(2, 150, 53).astype(int)
    rng = np.random.default_rng(top)
    freq = np.array([np.uint32(x).view(np.float32) for x in bits]
                    + [np.uint32((int(e) << 23) | int(rng.integers(0, 1 << 23))).view(np.float32) for e in exps]
                    + [0.0, 2.0 ** -9, 2.0 ** -10, 1.0, 2.0 ** 23, np.float32(2.0 ** 24 - 1)], dtype=np.float32)
    freq[1::2] *= -1
    assert freq.size == 64 and np.abs(freq).max() < 2 ** 24
    b = rope_case(40, 4, 2, 128, 128, 16, 1, torch.float16, False, 3, top=top)
    b["pos"][0, ::2] *= -1
    b["freq"] = torch.from_numpy(freq).cuda()
    out = rope_call(b, torch.empty((40, 4, 128), dtype=torch.float16, device="cuda"))
    # a turn's fraction rounded to fp32 (pi 2^-24), cos and sin good to 2^-23, three fp32 roundings
    # (2^-24 each), and the step of a turn, off by at most 2^-64 turns a position
    eps = (math.pi + 2 + 3) * 2.0 ** -24 + 2 * math.pi * top * 2.0 ** -64
    bs = b["kp"].shape[2]
    s = b["slots"].long()
    for x, got in ((b["q"], out), (b["k"], b["kp"][s // bs, :, s % bs])):
        want, size = R.rope(x.cpu(), b["pos"].cpu(), b["freq"].cpu(), None, False)
        err = (got.cpu().double() - want).abs()
        assert bool((err <= R.half_step(torch.float16) * want.abs() + eps * size + 2.0 ** -25).all())


def move(keys, values, pairs, tables, shape, dtype, status):
    """The call of the C library: pools as lists of tensors, which may be empty."""
    import paged_kv_cache_187_gb300 as pa
    NB, Hkv, bs, D = shape
    host = np.array([t.data_ptr() for t in keys + values] + [0], dtype=np.uint64)
    base = host.ctypes.data
    return pa.raw().pa_move_blocks(
        base if keys else None, base + 8 * len(keys) if keys else None, len(keys), pairs.data_ptr(),
        pairs.shape[0], tables.data_ptr(), tables.shape[0], tables.shape[1], Hkv, D, bs, NB, dtype,
        status.data_ptr(), torch.cuda.current_stream().cuda_stream)


def test_tables_are_rewritten_without_a_pool(cuda_device):
    import paged_kv_cache_187_gb300 as pa
    NB = 50
    rng = np.random.default_rng(3)
    tables = rng.integers(-1, NB + 2, size=(13, 29)).astype(np.int32)      # some outside the pool
    pairs = np.array([[30, 2], [31, 0], [40, 7], [49, 1]], np.int32)
    place = dict(pairs.tolist())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = torch.from_numpy(tables).cuda()
    assert move([], [], torch.from_numpy(pairs).cuda(), t, (NB, 2, 16, 64), pa.PA_F16, status) == 0
    assert np.array_equal(t.cpu().numpy(), np.vectorize(lambda b: place.get(b, b))(tables))
    assert int(status) == 0
    # a pair outside the pool is skipped and reported, the others' entries rewritten
    pairs[2, 1] = NB
    del place[40]
    t = torch.from_numpy(tables).cuda()
    assert move([], [], torch.from_numpy(pairs).cuda(), t, (NB, 2, 16, 64), pa.PA_F16, status) == 0
    assert np.array_equal(t.cpu().numpy(), np.vectorize(lambda b: place.get(b, b))(tables))
    assert int(status) == pa.PA_DEVERR_BAD_BLOCK


@pytest.mark.parametrize("rows,width", [(256, 8192), (1, 3_000_001), (1000, 777)])
def test_move_with_wide_tables(cuda_device, rows, width):
    """Tables as wide as the longest context allows, mostly padding; nothing past their end is
    written."""
    import paged_kv_cache_187_gb300 as pa
    NB = 400
    g = torch.Generator(device="cuda").manual_seed(rows)
    whole = torch.full((rows * width + 64,), -1, dtype=torch.int32, device="cuda")
    used = torch.randperm(rows * width, generator=g, device="cuda")[:200_000]
    whole[used] = torch.randint(0, NB, used.shape, generator=g, device="cuda", dtype=torch.int32)
    whole[rows * width:] = 399
    src = torch.arange(200, 400, device="cuda")
    dst = torch.randperm(200, generator=g, device="cuda")
    pairs = torch.stack([src, dst], 1).to(torch.int32).contiguous()
    place = torch.arange(NB, device="cuda")
    place[src] = dst
    want = torch.where(whole >= 0, place[whole.clamp_min(0).long()].to(torch.int32), whole)
    want[rows * width:] = 399
    pools = [torch.randint(0, 100, (NB, 1, 16, 64), device="cuda").to(torch.float16) for _ in range(2)]
    moved = [p.clone() for p in pools]
    for p in moved:
        p[dst] = p[src]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_move_blocks(pools[:1], pools[1:], pairs, block_tables=whole[:rows * width].view(rows, width), status=status)
    assert int(status) == 0
    assert torch.equal(whole, want)
    for p, m in zip(pools, moved):
        assert torch.equal(p, m)
