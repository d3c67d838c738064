"""CPU-only: argument checks of the chunk operators (every call below is rejected, or
accepted as empty, before any device work; the addresses are never touched), the
allocator's shrink against a plain model, and the 64-bit forms that the GPU tests use
against the oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

import chunk_reference as R
import oracle

OK, INVALID, UNSUPPORTED, NO_BLOCKS, CUDA, WORKSPACE = 0, 1, 2, 3, 4, 5
F16, BF16, FP8 = 0, 1, 2
A = 0x10000          # 16-byte (and 256-byte) aligned
MIS = 0x10008        # 8-byte aligned only


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_187_gb300 import build
    build.build()
    import paged_kv_cache_187_gb300 as pkg
    return pkg


@pytest.fixture(scope="module")
def lib(pa):
    return pa.raw()


def _err(lib):
    return (lib.pa_last_error() or b"").decode()


def _prefill(lib, fp8=False, **kw):
    p = dict(out=A, q=A, kc=A, vc=A, bt=A, maxb=64, lens=A, starts=A, T=100, S=3, Hq=8, Hkv=2, D=128,
             bs=16, NB=64, mcl=900, scale=0.1, ks=0.5, vs=0.5, dt=BF16, ws=A, wb=1 << 40)
    p.update(kw)
    head = [p[k] for k in ("out", "q", "kc", "vc", "bt", "maxb", "lens", "starts", "T", "S", "Hq", "Hkv",
                           "D", "bs", "NB", "mcl", "scale")]
    tail = [p["dt"], p["ws"], p["wb"], None, None]
    if fp8:
        return lib.pa_prefill_fp8(*head, p["ks"], p["vs"], *tail)
    return lib.pa_prefill(*head, *tail)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,code,word", [
    (dict(T=-1), INVALID, "positive"),
    (dict(S=-1), INVALID, "positive"),
    (dict(Hkv=0), INVALID, "positive"),
    (dict(NB=0), INVALID, "positive"),
    (dict(maxb=0), INVALID, "positive"),
    (dict(mcl=-1), INVALID, "positive"),
    (dict(T=(1 << 24) + 1), UNSUPPORTED, "num_tokens"),
    (dict(dt=FP8), UNSUPPORTED, "dtype"),
    (dict(D=96), UNSUPPORTED, "head_size"),
    (dict(bs=64), UNSUPPORTED, "block_size"),
    (dict(Hq=9), INVALID, "num_kv_heads"),
    (dict(Hq=34), UNSUPPORTED, "group"),
    (dict(NB=1 << 27), UNSUPPORTED, "rows"),
    (dict(scale=float("nan")), INVALID, "scale"),
    (dict(scale=float("inf")), INVALID, "scale"),
    (dict(out=0), INVALID, "null"),
    (dict(starts=0), INVALID, "null"),
    (dict(q=MIS), INVALID, "aligned"),
    (dict(vc=MIS), INVALID, "aligned"),
    (dict(ws=0), WORKSPACE, "workspace"),
    (dict(wb=1000), WORKSPACE, "workspace"),
    (dict(ws=A + 16), INVALID, "256-byte"),
])
def test_prefill_refusals(lib, fp8, kw, code, word):
    assert _prefill(lib, fp8, **kw) == code
    assert word in _err(lib)


def test_prefill_fp8_refusals_and_empty_calls(lib):
    for kw, word in ((dict(ks=0.0), "k_scale"), (dict(vs=-1.0), "k_scale"), (dict(ks=float("nan")), "k_scale")):
        assert _prefill(lib, True, **kw) == INVALID and word in _err(lib)
    assert _prefill(lib, True, D=64) == UNSUPPORTED and "head_size 128" in _err(lib)
    none = dict(out=0, q=0, kc=0, vc=0, bt=0, lens=0, starts=0, ws=0, wb=0)
    assert _prefill(lib, T=0, **none) == OK
    assert _prefill(lib, S=0, **none) == OK


def test_prefill_workspace_size(pa):
    size = pa.pa_prefill_workspace_size
    assert size(100, 3, 8, 2, 128, 900) > 0
    assert size(0, 0, 8, 2, 128, 0) > 0
    # rows of the chunk, not the context, set what grows
    assert size(100, 3, 8, 2, 128, 900) == size(100, 3, 8, 2, 128, 900_000)
    assert size(100_000, 3, 8, 2, 128, 900) > size(100, 3, 8, 2, 128, 900)
    # contexts of one tile are never cut: no room for partial results
    assert size(100, 3, 8, 2, 128, 128) < 1 << 16
    for bad in ((-1, 3, 8, 2, 128, 9), (1, -3, 8, 2, 128, 9), (1, 3, 0, 2, 128, 9), (1, 3, 8, 0, 128, 9),
                (1, 3, 8, 2, 0, 9), (1, 3, 8, 2, 128, -9), ((1 << 24) + 1, 3, 8, 2, 128, 9)):
        assert size(*bad) == 0


def _rope(lib, fp8=False, **kw):
    axes = np.asarray(kw.pop("axes", [0] * 64), np.int32)
    p = dict(out=A, q=A + 16, k=A, v=A, qs=1024, ks=256, vs=256, kc=A, vc=A, slots=A, pos=A, na=1,
             ax=axes.ctypes.data, freq=A, rot=128, il=0, T=5, Hq=8, Hkv=2, D=128, bs=16, NB=64, dt=BF16,
             k_scale=0.5, v_scale=0.5)
    p.update(kw)
    head = [p[k] for k in ("out", "q", "k", "v", "qs", "ks", "vs", "kc", "vc", "slots", "pos", "na", "ax",
                           "freq", "rot", "il", "T", "Hq", "Hkv", "D", "bs", "NB", "dt")]
    if fp8:
        return lib.pa_rope_and_cache_fp8(*head, p["k_scale"], p["v_scale"], None, None)
    return lib.pa_rope_and_cache(*head, None, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(T=-1), INVALID, "positive"),
    (dict(Hkv=0), INVALID, "positive"),
    (dict(dt=FP8), UNSUPPORTED, "dtype"),
    (dict(D=72, rot=64, qs=1024), UNSUPPORTED, "head_size"),
    (dict(D=2048, rot=64, qs=1 << 20, ks=1 << 20, vs=1 << 20), UNSUPPORTED, "head_size"),
    (dict(rot=8), UNSUPPORTED, "rot_dim"),
    (dict(rot=24), UNSUPPORTED, "rot_dim"),
    (dict(rot=144), UNSUPPORTED, "rot_dim"),
    (dict(D=512, rot=272, qs=4096, ks=1024, vs=1024), UNSUPPORTED, "rot_dim"),
    (dict(na=0), UNSUPPORTED, "num_axes"),
    (dict(na=5), UNSUPPORTED, "num_axes"),
    (dict(na=2, ax=None), INVALID, "pair_axes"),
    (dict(na=2, axes=[0] * 63 + [2]), INVALID, "pair_axes[63]"),
    (dict(na=2, axes=[-1] + [0] * 63), INVALID, "pair_axes[0]"),
    (dict(qs=1016), INVALID, "stride"),
    (dict(ks=260), INVALID, "multiples of 8"),
    (dict(Hq=1 << 20, qs=1 << 27), UNSUPPORTED, "heads"),
    (dict(slots=0), INVALID, "null"),
    (dict(freq=0), INVALID, "null"),
    (dict(v=MIS), INVALID, "aligned"),
    (dict(out=A + 16, qs=2048), INVALID, "in place"),
])
def test_rope_refusals(lib, kw, code, word):
    assert _rope(lib, **dict(kw)) == code
    assert word in _err(lib)
    assert _rope(lib, True, **dict(kw)) == code


def test_rope_fp8_refusals_and_empty_calls(lib):
    assert _rope(lib, True, k_scale=0.0) == INVALID and "scales" in _err(lib)
    none = dict(T=0, out=0, q=0, k=0, v=0, kc=0, vc=0, slots=0, pos=0, freq=0)
    assert _rope(lib, **none) == OK
    assert _rope(lib, True, **none) == OK


def _move(lib, **kw):
    pools = np.asarray(kw.pop("pools", [A, A, A, A]), np.uint64)
    p = dict(keys=pools.ctypes.data, values=pools.ctypes.data + 16, L=2, pairs=A, n=3, bt=None, rows=0,
             maxb=0, Hkv=2, D=128, bs=16, NB=64, dt=BF16)
    p.update(kw)
    return lib.pa_move_blocks(*[p[k] for k in ("keys", "values", "L", "pairs", "n", "bt", "rows", "maxb",
                                               "Hkv", "D", "bs", "NB", "dt")], None, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(L=-1), INVALID, "positive"),
    (dict(n=-1), INVALID, "positive"),
    (dict(NB=0), INVALID, "positive"),
    (dict(n=65), INVALID, "65 pairs"),
    (dict(dt=7), UNSUPPORTED, "dtype"),
    (dict(bt=A, rows=-1, maxb=4), INVALID, "num_rows"),
    (dict(bt=A, rows=2, maxb=0), INVALID, "num_rows"),
    (dict(pairs=0), INVALID, "null"),
    (dict(keys=None), INVALID, "null"),
    (dict(pools=[A, 0, A, A]), INVALID, "null pool"),
    (dict(pools=[A, A, A, MIS]), INVALID, "aligned"),
    (dict(D=1, bs=1, Hkv=1), INVALID, "16-byte multiples"),
])
def test_move_refusals(lib, kw, code, word):
    assert _move(lib, **kw) == code
    assert word in _err(lib)


def test_move_without_pairs_is_a_no_op(lib):
    assert _move(lib, n=0, pairs=0) == OK


def test_binding_refuses_before_the_library(pa):
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    pool = torch.zeros(3, 2, 16, 128, dtype=torch.bfloat16)
    t, l, s = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    import paged_kv_cache_187_gb300._binding as B

    class Here(B._Call):       # a machine without a GPU has no current device
        def __init__(self):
            self.dev = 0

    old, B._Call = B._Call, Here
    try:
        with pytest.raises(ValueError, match="CUDA tensor"):
            pa.pa_prefill(q, q, pool, pool, t, l, s, 10, 0.1)
        with pytest.raises(ValueError, match="query_starts"):
            pa.pa_prefill(q, q, pool, pool, t, l, s[:1], 10, 0.1)
        with pytest.raises(ValueError, match="inconsistent"):
            pa.pa_prefill(q[:2], q, pool, pool, t, l, s, 10, 0.1)
        with pytest.raises(TypeError, match="uint8"):
            pa.pa_prefill_fp8(q, q, pool, pool, t, l, s, 10, 0.1, 1.0, 1.0)
        k = q[:, :2]
        pos, freq, slots = torch.zeros(1, 4, dtype=torch.int64), torch.zeros(64), torch.zeros(4, dtype=torch.int32)
        with pytest.raises(ValueError, match="CUDA tensor"):
            pa.pa_rope_and_cache(q, q, k, k, pool, pool, slots, pos, freq)
        with pytest.raises(ValueError, match="one axis per pair"):
            pa.pa_rope_and_cache(q, q, k, k, pool, pool, slots, pos, freq, pair_axes=[0] * 63)
        with pytest.raises(ValueError, match="positions"):
            pa.pa_rope_and_cache(q, q, k, k, pool, pool, slots, pos[0], freq)
        with pytest.raises(ValueError, match="at least one layer"):
            pa.pa_move_blocks([], [], t)
        with pytest.raises(ValueError, match="pairs"):
            pa.pa_move_blocks([pool], [pool], t)
    finally:
        B._Call = old


# ------------------------------------------------------------------ shrink
def _model(alloc, ids, width, num_blocks):
    tables = alloc.pa_alloc_block_tables(ids, width)
    counts = [alloc.pa_alloc_refcount(b) for b in range(num_blocks)]
    return tables, counts


@pytest.mark.parametrize("seed", range(6))
def test_shrink_moves_the_high_blocks_to_the_low_free_ones(pa, seed):
    rng = np.random.default_rng(seed)
    NB, bs = 60, 4
    a = pa.PagedAllocator(NB, bs, seed)
    for s in range(6):
        a.pa_alloc_add_seq(s, int(rng.integers(0, 25)))
    a.pa_alloc_fork(0, 10, int(a.pa_alloc_context_lens([0])[0]))
    a.pa_alloc_free_seq(2)
    ids = [0, 1, 3, 4, 5, 10]
    tables, counts = _model(a, ids, 8, NB)
    used = NB - a.num_free
    assert used == sum(c > 0 for c in counts)
    with pytest.raises(pa.PANoBlocks):
        a.pa_alloc_shrink(used - 1)
    assert np.array_equal(_model(a, ids, 8, NB)[0], tables)
    keep = used + int(rng.integers(0, 5))
    high = [b for b in range(keep, NB) if counts[b]]
    low = [b for b in range(keep) if not counts[b]][:len(high)]
    pairs = a.pa_alloc_shrink(keep)
    assert pairs.tolist() == [list(x) for x in zip(high, low)]
    place = dict(zip(high, low))
    new, c2 = _model(a, ids, 8, keep)
    assert np.array_equal(new, np.vectorize(lambda b: place.get(b, b))(tables))
    for b in range(keep):
        assert c2[b] == (counts[b] or (counts[high[low.index(b)]] if b in low else 0))
    assert a.pa_alloc_refcount(keep) == -1 and a.num_blocks == keep
    # every block that is left can be handed out once
    left = a.num_free
    assert left == keep - used
    if left:
        a.pa_alloc_add_seq(99, left * bs)
        got = a.pa_alloc_block_tables([99], left)[0]
        assert len(set(got.tolist())) == left and got.max() < keep and got.min() >= 0
        assert not set(got.tolist()) & set(new[new >= 0].ravel().tolist())
    assert a.pa_alloc_shrink(keep).shape == (0, 2)
    a.pa_alloc_free_seq(0)          # the fork still holds its blocks
    assert all(a.pa_alloc_refcount(int(b)) >= 1 for b in new[5] if b >= 0)


def test_shrink_refusals(pa):
    a = pa.PagedAllocator(10, 16, 1)
    for n in (0, -3, 11):
        with pytest.raises(pa.PAError):
            a.pa_alloc_shrink(n)
    a.pa_alloc_add_seq(0, 20)
    a.pa_alloc_fork(0, 1, 20)
    a.pa_alloc_append(0)             # a private copy is pending
    with pytest.raises(pa.PAError, match="pending"):
        a.pa_alloc_shrink(8)
    a.pa_alloc_take_copies()
    n = ctypes.c_int32(-1)
    before = a.pa_alloc_block_tables([0, 1], 4)
    room = np.zeros((1, 2), np.int32)
    lib = pa.raw()
    high = int((np.unique(before[before >= 0]) >= 4).sum())
    if high > 1:
        assert lib.pa_alloc_shrink(a._h, 4, room.ctypes.data, 1, ctypes.byref(n)) == INVALID
        assert n.value == high and np.array_equal(a.pa_alloc_block_tables([0, 1], 4), before)
    assert lib.pa_alloc_shrink(None, 4, room.ctypes.data, 1, ctypes.byref(n)) == INVALID
    assert lib.pa_alloc_shrink(a._h, 4, room.ctypes.data, 1, None) == INVALID


# ------------------------------------------------------------------ the 64-bit forms
@pytest.mark.parametrize("dtype,QL,Hq,Hkv,D", [("bf16", 3, 8, 2, 64), ("f16", 5, 4, 4, 128)])
def test_attention_form_agrees_with_the_oracle(dtype, QL, Hq, Hkv, D):
    from oracle_side import bits, err_stats
    g = torch.Generator().manual_seed(QL)
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float16
    NB, bs, lens = 40, 16, np.array([1, 2, 40, 17, 90], np.int32)
    kc, vc = (torch.randn(NB, Hkv, bs, D, generator=g).to(tdt) for _ in range(2))
    q = torch.randn(5, QL, Hq, D, generator=g).to(tdt)
    tables = torch.randperm(NB, generator=g)[:30].view(5, 6).to(torch.int32)
    starts = np.arange(6) * QL
    out, tol = R.prefill(q.view(-1, Hq, D), kc, vc, tables, lens, starts, D ** -0.5)
    ref = oracle.decode_mq(bits(q), bits(kc), bits(vc), tables.numpy(), lens, np.float32(D ** -0.5), dtype)
    assert err_stats(bits(out.to(tdt).view(5, QL, Hq, D)), ref, dtype).ok(dtype)
    assert (tol[out != 0] > 0).all()


def test_rotary_form_turns_pairs():
    x = torch.zeros(2, 1, 8, dtype=torch.float16)
    x[:, 0, 0], x[:, 0, 1] = 1.0, 2.0
    pos = torch.tensor([[0, 3], [0, 7]])
    freq = torch.tensor([0.5, 0.25])
    y, _ = R.rope(x, pos, freq, [0, 1], False)             # pairs (0, 2) and (1, 3)
    assert y[0, 0].tolist() == [1, 2, 0, 0, 0, 0, 0, 0]
    assert y[1, 0, :4].tolist() == pytest.approx([math.cos(1.5), 2 * math.cos(1.75), math.sin(1.5),
                                                  2 * math.sin(1.75)])
    y, _ = R.rope(x, pos, freq, [1, 1], True)              # pairs (0, 1) and (2, 3)
    assert y[1, 0, :4].tolist() == pytest.approx([math.cos(3.5) - 2 * math.sin(3.5),
                                                  math.sin(3.5) + 2 * math.cos(3.5), 0, 0])
