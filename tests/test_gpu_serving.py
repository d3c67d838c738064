"""GPU: the chunk operators in a row, as a server uses them -- prompts taken in pieces of
different lengths beside decoding sequences (rotary positions and cache write, attention of
the chunk), a sequence freed, the pools compacted, and the decode going on over the moved
blocks."""
import numpy as np
import pytest
import torch

import chunk_reference as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
def test_prompts_in_pieces_then_compaction(cuda_device, fp8):
    import paged_kv_cache_187_gb300 as pa
    Hq, Hkv, D, bs, layers, dtype = 16, 4, 128, 16, 2, torch.bfloat16
    NB, width, mcl = 200, 40, 600
    ks, vs = (0.03, 0.02) if fp8 else (1.0, 1.0)
    dev, g = "cuda", torch.Generator(device="cuda").manual_seed(5)
    alloc = pa.PagedAllocator(NB, bs, 9)
    cdt = torch.uint8 if fp8 else dtype
    keys = [torch.full((NB, Hkv, bs, D), 127, dtype=cdt, device=dev) for _ in range(layers)]
    values = [torch.full((NB, Hkv, bs, D), 127, dtype=cdt, device=dev) for _ in range(layers)]
    freq = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().to(dev)
    axes = [0] * 24 + [1] * 20 + [2] * 20
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    lens = {s: 0 for s in range(5)}
    for s in lens:
        alloc.pa_alloc_add_seq(s, 0)
    # pieces of each step: (sequence, new tokens)
    steps = [[(0, 100), (1, 37)], [(0, 1), (1, 200), (2, 64)], [(0, 1), (1, 1), (2, 130), (3, 17), (4, 300)],
             [(0, 1), (1, 1), (2, 1), (3, 5), (4, 9)]]
    scale = D ** -0.5
    for step in steps:
        slots, starts, pos = [], [0], []
        for s, n in step:
            alloc.pa_alloc_reserve_batch([s], n)
            slots += [int(alloc.pa_alloc_append(s)) for _ in range(n)]
            t = np.arange(lens[s], lens[s] + n)
            pos.append(np.stack([t, t // 7, t % 7]))
            lens[s] += n
            starts.append(starts[-1] + n)
        ids = [s for s, _ in step]
        T = starts[-1]
        tables = torch.from_numpy(alloc.pa_alloc_block_tables(ids, width)).to(dev)
        lens_d = torch.from_numpy(alloc.pa_alloc_context_lens(ids)).to(dev)
        starts_d = torch.tensor(starts, dtype=torch.int32, device=dev)
        slots_d = torch.tensor(slots, dtype=torch.int32, device=dev)
        pos_d = torch.from_numpy(np.concatenate(pos, 1).astype(np.int64)).to(dev)
        ws = torch.empty(pa.pa_prefill_workspace_size(T, len(ids), Hq, Hkv, D, mcl), dtype=torch.uint8, device=dev)
        for l in range(layers):
            qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=dev).to(dtype)
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
            rotated, out = torch.empty((T, Hq, D), dtype=dtype, device=dev), torch.zeros((T, Hq, D), dtype=dtype, device=dev)
            if fp8:
                pa.pa_rope_and_cache_fp8(rotated, q, k, v, keys[l], values[l], slots_d, pos_d, freq, ks, vs,
                                         pair_axes=axes, status=status)
                pa.pa_prefill_fp8(out, rotated, keys[l], values[l], tables, lens_d, starts_d, mcl, scale, ks, vs,
                                  workspace=ws, status=status)
            else:
                pa.pa_rope_and_cache(rotated, q, k, v, keys[l], values[l], slots_d, pos_d, freq,
                                     pair_axes=axes, status=status)
                pa.pa_prefill(out, rotated, keys[l], values[l], tables, lens_d, starts_d, mcl, scale,
                              workspace=ws, status=status)
            want, tol = R.prefill(rotated, keys[l], values[l], tables, lens_d.tolist(), starts, scale, ks, vs)
            assert ((out.double() - want).abs() <= tol).all()
            spun, size = R.rope(q, pos_d, freq, axes, False)
            assert ((rotated.double() - spun).abs() <= 2.0 ** -8 * spun.abs() + 2.0 ** -20 * size).all()
    torch.cuda.synchronize()
    assert int(status) == 0
    # sequence 1 ends; the pool shrinks to what the others need, and a decode step goes on
    ids = [0, 2, 3, 4]
    alloc.pa_alloc_free_seq(1)
    old = alloc.pa_alloc_block_tables(ids, width)
    tables, lens_d = torch.from_numpy(old).to(dev), torch.from_numpy(alloc.pa_alloc_context_lens(ids)).to(dev)
    q = torch.randn((4, Hq, D), generator=g, device=dev).to(dtype)

    def decode(l, n):
        out = torch.zeros_like(q)
        need = pa.pa_decode_auto_workspace_size(4, Hq, Hkv, D, bs, mcl)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        pools = (keys[l][:n], values[l][:n])
        if fp8:
            pa.pa_decode_fp8(out, q, *pools, tables, lens_d, mcl, scale, ks, vs, workspace=ws, status=status)
        else:
            pa.pa_decode_auto(out, q, *pools, tables, lens_d, mcl, scale, workspace=ws, status=status)
        return out

    before = [decode(l, NB) for l in range(layers)]
    keep = NB - alloc.num_free
    pairs = alloc.pa_alloc_shrink(keep)
    assert len(pairs) > 0
    pa.pa_move_blocks(keys, values, torch.from_numpy(pairs).to(dev), block_tables=tables, status=status)
    assert np.array_equal(tables.cpu().numpy(), alloc.pa_alloc_block_tables(ids, width))
    for l in range(layers):
        assert torch.equal(before[l], decode(l, keep))       # the tail of the pools is unused now
    assert int(status) == 0
