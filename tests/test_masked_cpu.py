"""CPU-only: argument checks of the tree and sparse operators (every call below is rejected, or
accepted as empty, before any device work; the addresses are never touched), the sizes of their
workspaces, and the 64-bit forms that the GPU tests use against the oracle and by hand."""
import math

import numpy as np
import pytest
import torch

import masked_reference as M
import oracle

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = 0, 1, 2, 4, 5
F16, BF16, FP8 = 0, 1, 2
A = 0x10000
MIS = 0x10008


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


def _tree(lib, fp8=False, **kw):
    p = dict(out=A, q=A, kc=A, vc=A, bt=A, maxb=64, lens=A, starts=A, mask=A, W=2, T=100, S=3, Hq=8, Hkv=2,
             D=128, bs=16, NB=64, mcl=900, scale=0.1, ks=0.5, vs=0.5, dt=BF16, ws=A, wb=1 << 40)
    p.update(kw)
    head = [p[k] for k in ("out", "q", "kc", "vc", "bt", "maxb", "lens", "starts", "mask", "W", "T", "S", "Hq",
                           "Hkv", "D", "bs", "NB", "mcl", "scale")]
    tail = [p["dt"], p["ws"], p["wb"], None, None]
    if fp8:
        return lib.pa_decode_tree_fp8(*head, p["ks"], p["vs"], *tail)
    return lib.pa_decode_tree(*head, *tail)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,code,word", [
    (dict(T=-1), INVALID, "positive"),
    (dict(S=-1), INVALID, "positive"),
    (dict(W=0), INVALID, "mask_words"),
    (dict(W=-3), INVALID, "mask_words"),
    (dict(mask=0), INVALID, "tree_mask"),
    (dict(T=(1 << 24) + 1), UNSUPPORTED, "num_tokens"),
    (dict(dt=FP8), UNSUPPORTED, "dtype"),
    (dict(D=96), UNSUPPORTED, "head_size"),
    (dict(bs=8), UNSUPPORTED, "block_size"),
    (dict(Hq=34), UNSUPPORTED, "group"),
    (dict(scale=float("nan")), INVALID, "scale"),
    (dict(lens=0), INVALID, "null"),
    (dict(q=MIS), INVALID, "aligned"),
    (dict(ws=0), WORKSPACE, "workspace"),
    (dict(ws=A + 16), INVALID, "256-byte"),
])
def test_tree_refusals(lib, fp8, kw, code, word):
    assert _tree(lib, fp8, **kw) == code
    assert word in _err(lib) and "decode_tree" in _err(lib)


def test_tree_empty_calls_and_sizes(lib, pa):
    none = dict(out=0, q=0, kc=0, vc=0, bt=0, lens=0, starts=0, mask=0, ws=0, wb=0)
    assert _tree(lib, T=0, **none) == OK and _tree(lib, S=0, **none) == OK
    assert _tree(lib, True, D=64) == UNSUPPORTED
    size = pa.pa_decode_tree_workspace_size
    assert size(100, 3, 8, 2, 128, 900) == pa.pa_prefill_workspace_size(100, 3, 8, 2, 128, 900) > 0
    assert size(-1, 3, 8, 2, 128, 900) == 0


def _accept(lib, **kw):
    p = dict(acc=A, most=8, cnt=A, nxt=A, new=A, d=A, t=A, mask=A, W=2, starts=A, lens=A, T=40, S=3)
    p.update(kw)
    return lib.pa_tree_accept(*[p[k] for k in ("acc", "most", "cnt", "nxt", "new", "d", "t", "mask", "W", "starts",
                                               "lens", "T", "S")], None, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(T=-1), INVALID, "positive"),
    (dict(S=-1), INVALID, "positive"),
    (dict(most=0), INVALID, "positive"),
    (dict(W=0), INVALID, "positive"),
    (dict(W=65), UNSUPPORTED, "mask_words"),
    (dict(acc=0), INVALID, "null"),
    (dict(new=0), INVALID, "null"),
    (dict(d=0), INVALID, "null"),
    (dict(mask=0), INVALID, "null"),
])
def test_accept_refusals(lib, kw, code, word):
    assert _accept(lib, **kw) == code
    assert word in _err(lib)


def test_accept_of_no_sequence(lib):
    assert _accept(lib, S=0, acc=0, cnt=0, nxt=0, new=0, d=0, t=0, mask=0, starts=0, lens=0) == OK


def _move(lib, pools=(A, A), **kw):
    arr = np.array(list(pools), dtype=np.uint64)
    p = dict(k=arr.ctypes.data, v=arr.ctypes.data, L=len(pools), bt=A, maxb=9, new=A, acc=A, most=8, cnt=A, S=3,
             Hkv=2, D=64, bs=16, NB=30, dt=BF16)
    p.update(kw)
    return lib.pa_move_tokens(*[p[k] for k in ("k", "v", "L", "bt", "maxb", "new", "acc", "most", "cnt", "S", "Hkv",
                                               "D", "bs", "NB", "dt")], None, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(L=-1), INVALID, "positive"),
    (dict(S=-1), INVALID, "positive"),
    (dict(maxb=0), INVALID, "positive"),
    (dict(most=0), INVALID, "positive"),
    (dict(Hkv=0), INVALID, "positive"),
    (dict(dt=7), UNSUPPORTED, "dtype"),
    (dict(D=4), INVALID, "16-byte"),
    (dict(D=8, dt=FP8), INVALID, "16-byte"),
    (dict(Hkv=1 << 30, D=1024), UNSUPPORTED, "heads"),
    (dict(k=0), INVALID, "null"),
    (dict(acc=0), INVALID, "null"),
    (dict(pools=(A, 0)), INVALID, "null pool"),
    (dict(pools=(A, MIS)), INVALID, "aligned"),
])
def test_move_refusals(lib, kw, code, word):
    assert _move(lib, **kw) == code
    assert word in _err(lib)


def test_move_of_nothing(lib):
    assert _move(lib, S=0, k=0, v=0, bt=0, new=0, acc=0, cnt=0) == OK
    assert _move(lib, L=0, k=0, v=0, bt=0, new=0, acc=0, cnt=0) == OK


def _bounds(lib, **kw):
    p = dict(b=A, st=A, k=A, bt=A, maxb=64, lens=A, starts=0, new=1, S=3, Hkv=2, D=128, bs=16, NB=64, dt=BF16)
    p.update(kw)
    return lib.pa_key_bounds(*[p[k] for k in ("b", "st", "k", "bt", "maxb", "lens", "starts", "new", "S", "Hkv", "D",
                                              "bs", "NB", "dt")], None, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(S=-1), INVALID, "positive"),
    (dict(new=-1), INVALID, "positive"),
    (dict(Hkv=0), INVALID, "positive"),
    (dict(maxb=0), INVALID, "positive"),
    (dict(dt=9), UNSUPPORTED, "dtype"),
    (dict(D=256), UNSUPPORTED, "head_size"),
    (dict(bs=64), UNSUPPORTED, "block_size"),
    (dict(b=0), INVALID, "null"),
    (dict(lens=0), INVALID, "null"),
    (dict(k=MIS), INVALID, "aligned"),
    (dict(b=MIS), INVALID, "aligned"),
    (dict(S=1 << 20, new=1 << 30, maxb=1 << 26), UNSUPPORTED, "blocks"),
])
def test_bounds_refusals(lib, kw, code, word):
    assert _bounds(lib, **kw) == code
    assert word in _err(lib)


def test_bounds_of_nothing(lib):
    assert _bounds(lib, S=0, b=0, st=0, k=0, bt=0, lens=0) == OK
    assert _bounds(lib, new=0, b=0, st=0, k=0, bt=0, lens=0) == OK


def _select(lib, **kw):
    p = dict(sel=A, q=A, b=A, st=A, bt=A, maxb=64, lens=A, S=3, QL=1, Hq=8, Hkv=2, D=128, bs=16, NB=64, mcl=900, n=8,
             first=1, last=2, dt=BF16, ws=A, wb=1 << 40)
    p.update(kw)
    return lib.pa_select_blocks(*[p[k] for k in ("sel", "q", "b", "st", "bt", "maxb", "lens", "S", "QL", "Hq", "Hkv",
                                                 "D", "bs", "NB", "mcl", "n", "first", "last", "dt", "ws", "wb")],
                                None, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(S=-1), INVALID, "positive"),
    (dict(QL=0), INVALID, "positive"),
    (dict(n=0), INVALID, "positive"),
    (dict(mcl=-1), INVALID, "positive"),
    (dict(first=-1), INVALID, "num_first"),
    (dict(last=-1), INVALID, "num_last"),
    (dict(first=5, last=4), INVALID, "num_first"),
    (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), INVALID, "num_first"),
    (dict(dt=FP8), UNSUPPORTED, "dtype"),
    (dict(D=96), UNSUPPORTED, "head_size"),
    (dict(bs=8), UNSUPPORTED, "block_size"),
    (dict(Hq=9), INVALID, "num_kv_heads"),
    (dict(Hq=34), UNSUPPORTED, "group"),
    (dict(Hq=70000, Hkv=70000), UNSUPPORTED, "heads"),
    (dict(S=1 << 20, QL=1 << 12), UNSUPPORTED, "rows"),
    (dict(mcl=1 << 30, maxb=1 << 27), UNSUPPORTED, "contexts"),
    (dict(NB=1 << 30), UNSUPPORTED, "pool"),
    (dict(sel=0), INVALID, "null"),
    (dict(st=0), INVALID, "null"),
    (dict(q=MIS), INVALID, "aligned"),
    (dict(b=MIS), INVALID, "aligned"),
    (dict(ws=0), WORKSPACE, "workspace"),
    (dict(wb=100), WORKSPACE, "workspace"),
    (dict(ws=A + 16), INVALID, "256-byte"),
])
def test_select_refusals(lib, kw, code, word):
    assert _select(lib, **kw) == code
    assert word in _err(lib)


def test_select_of_nothing_and_sizes(lib, pa):
    assert _select(lib, S=0, sel=0, q=0, b=0, st=0, bt=0, lens=0, ws=0, wb=0) == OK
    size = pa.pa_select_blocks_workspace_size
    assert size(3, 1, 2, 16, 900) >= 4 * 3 * 2 * 57
    assert size(3, 4, 2, 16, 900) >= 4 * size(3, 1, 2, 16, 900) - 1024
    for bad in ((-1, 1, 2, 16, 9), (1, 0, 2, 16, 9), (1, 1, 0, 16, 9), (1, 1, 2, 0, 9), (1, 1, 2, 16, -1)):
        assert size(*bad) == 0


def _sparse(lib, fp8=False, **kw):
    p = dict(out=A, q=A, kc=A, vc=A, bt=A, maxb=64, lens=A, sel=A, n=8, S=3, QL=1, Hq=8, Hkv=2, D=128, bs=16, NB=64,
             scale=0.1, ks=0.5, vs=0.5, dt=BF16, ws=A, wb=1 << 40)
    p.update(kw)
    head = [p[k] for k in ("out", "q", "kc", "vc", "bt", "maxb", "lens", "sel", "n", "S", "QL", "Hq", "Hkv", "D", "bs",
                           "NB", "scale")]
    tail = [p["dt"], p["ws"], p["wb"], None, None]
    if fp8:
        return lib.pa_decode_sparse_fp8(*head, p["ks"], p["vs"], *tail)
    return lib.pa_decode_sparse(*head, *tail)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,code,word", [
    (dict(S=-1), INVALID, "positive"),
    (dict(QL=0), INVALID, "positive"),
    (dict(n=0), INVALID, "positive"),
    (dict(NB=0), INVALID, "positive"),
    (dict(dt=FP8), UNSUPPORTED, "dtype"),
    (dict(D=96), UNSUPPORTED, "head_size"),
    (dict(bs=64), UNSUPPORTED, "block_size"),
    (dict(Hq=9), INVALID, "num_kv_heads"),
    (dict(Hq=34), UNSUPPORTED, "group"),
    (dict(NB=1 << 27), UNSUPPORTED, "rows"),
    (dict(S=1 << 20, QL=64), UNSUPPORTED, "rows"),
    (dict(n=(1 << 16) + 1), UNSUPPORTED, "num_selected"),
    (dict(scale=float("inf")), INVALID, "scale"),
    (dict(sel=0), INVALID, "null"),
    (dict(out=0), INVALID, "null"),
    (dict(q=MIS), INVALID, "aligned"),
    (dict(vc=MIS), INVALID, "aligned"),
])
def test_sparse_refusals(lib, fp8, kw, code, word):
    assert _sparse(lib, fp8, **kw) == code
    assert word in _err(lib) and "decode_sparse" in _err(lib)


def test_sparse_fp8_refusals_empty_calls_and_sizes(lib, pa):
    for kw in (dict(ks=0.0), dict(vs=-1.0), dict(ks=float("nan"))):
        assert _sparse(lib, True, **kw) == INVALID and "k_scale" in _err(lib)
    assert _sparse(lib, True, D=64) == UNSUPPORTED
    assert _sparse(lib, S=0, out=0, q=0, kc=0, vc=0, bt=0, lens=0, sel=0, ws=0, wb=0) == OK
    # (the parts of a row meet in shared memory)
    assert pa.pa_decode_sparse_workspace_size(3, 1, 8, 2, 128, 16, 8) == 0


def test_binding_refuses_before_the_library(pa, monkeypatch):
    import paged_kv_cache_187_gb300._binding as B

    class Here(B._Call):       # a machine without a GPU has no current device
        def __init__(self):
            self.dev = 0

    monkeypatch.setattr(B, "_Call", Here)
    t = torch.zeros
    with pytest.raises(ValueError):
        pa.pa_tree_accept(t((2, 4), dtype=torch.int32), t(3, dtype=torch.int32), t(2), t(2), t(5), t(5), t((5, 1)), t(3), t(2))
    with pytest.raises(ValueError):
        pa.pa_move_tokens([], [], t((2, 4)), t(2), t((2, 3)), t(2))
    with pytest.raises(ValueError):
        pa.pa_key_bounds(t((9, 2, 2, 64)), t((9, 3)), t((9, 2, 16, 64)), t((1, 2)), t(1), 1)
    with pytest.raises(ValueError):
        pa.pa_select_blocks(t((2, 2, 8)), t((3, 4, 64)), t((9, 2, 2, 64)), t((9, 2)), t((3, 4)), t(3), 16, 64, 0, 0)
    with pytest.raises(ValueError):
        pa.pa_select_blocks(t((2, 8)), t((3, 4, 64)), t((9, 2, 2, 64)), t((9, 2)), t((3, 4)), t(3), 16, 64, 0, 0)
    with pytest.raises(ValueError):
        pa.pa_decode_sparse(t((3, 4, 64)), t((3, 4, 64)), t((9, 2, 16, 64)), t((9, 2, 16, 64)), t((3, 4)), t(3),
                            t((3, 3, 8)), 0.1)
    with pytest.raises(ValueError):
        pa.pa_decode_tree(t((5, 4, 64)), t((5, 4, 64)), t((9, 2, 16, 64)), t((9, 2, 16, 64)), t((1, 4)), t(1), t(2),
                          t((4, 1)), 64, 0.1)
    with pytest.raises(TypeError):
        pa.pa_decode_tree(t((5, 4, 64)), t((5, 4, 64)), t((9, 2, 16, 64)), t((9, 2, 16, 64)), t((1, 4)), t(1), t(2),
                          None, 64, 0.1)
    with pytest.raises(ValueError):          # a tensor of the host
        pa.pa_key_bounds(t((9, 2, 2, 64), dtype=torch.int8), t((9, 2)), t((9, 2, 16, 64), dtype=torch.float16),
                         t((1, 2), dtype=torch.int32), t(1, dtype=torch.int32), 1)


# ------------------------------------------------------------------ the 64-bit forms
def _bits(x):
    return x.view(torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_the_tree_form_of_a_chain_agrees_with_the_oracle(dtype):
    t = torch.float16 if dtype == "f16" else torch.bfloat16
    g = torch.Generator().manual_seed(3)
    S, QL, Hq, Hkv, D, bs = 3, 4, 4, 2, 64, 16
    lens = [40, 4, 100]
    tables = torch.randperm(24, generator=g).to(torch.int32).view(3, 8)
    kc, vc = (torch.randn((24, Hkv, bs, D), generator=g).to(t) for _ in range(2))
    q = torch.randn((S * QL, Hq, D), generator=g).to(t)
    sees = [torch.ones((QL, QL), dtype=torch.bool)] * S
    out, _ = M.tree(q, kc, vc, tables, lens, [0, 4, 8, 12], sees, D ** -0.5)
    want = oracle.decode_mq(_bits(q.view(S, QL, Hq, D)), _bits(kc), _bits(vc), tables.numpy(),
                            np.array(lens, np.int32), np.float32(D ** -0.5), dtype)
    # (the oracle takes the scale as an fp32, scores up to 2^4: relative errors of 2^-24 * 2^4 twice)
    err = (out.view(S, QL, Hq, D) - torch.from_numpy(want)).abs().max()
    assert err <= 2.0 ** -19 * float(vc.double().abs().max())


def test_masks_and_paths_by_hand():
    m = M.paths([-1, 0, 0, 1, 2])
    assert m.int().tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 1, 0, 1, 0], [1, 0, 1, 0, 1]]
    assert M.masks([m], 1, "cpu")[:, 0].tolist() == [1, 3, 5, 11, 21]
    wide = M.masks([torch.ones((33, 33), dtype=torch.bool).tril()], 2, "cpu")
    assert wide[31].tolist() == [-1, 0] and wide[32].tolist() == [-1, 1]
    assert M.accept([-1, 0, 0, 1, 2], [9, 5, 6, 7, 8], [6, 0, 8, 0, 4], 9) == ([0, 2, 4], 4)
    assert M.accept([-1, 0, 0, 1, 2], [9, 5, 6, 7, 8], [6, 0, 8, 0, 4], 2) == ([0, 2], 8)


def test_bounds_scores_and_selection_by_hand():
    k = torch.tensor([[1.0, -3.0, 0.0], [2.5, 0.1, 0.0]], dtype=torch.float64)
    hi, lo, step = M.bounds(k, 65504.0)                       # the largest is 3: step 2 / 64
    assert step == 2.0 ** -5
    assert hi.tolist() == [80, 3, 0] and lo.tolist() == [32, -96, 0]
    assert M.bounds(torch.zeros((2, 3), dtype=torch.float64), 65504.0)[2] == 2.0 ** -106
    assert math.isnan(M.bounds(torch.tensor([[1.0, math.nan]], dtype=torch.float64), 65504.0)[2])
    # 127.5 of a step is clamped to 127
    assert M.bounds(torch.tensor([[255 / 128]], dtype=torch.float64), 65504.0)[0].tolist() == [127]
    q = torch.tensor([[1.0, -2.0, 0.0], [0.5, 0.0, 0.0]], dtype=torch.float64)    # |p| of 2 is 32
    got = M.scores(q, hi[None], lo[None], torch.tensor([step], dtype=torch.float64), 65504.0)
    assert got.tolist() == [(16 * 80 + 32 * 96 + 8 * 80) * step]
    assert M.select([5, 9, 9, 1, 9], 5, 2, 0, 0) == [1, 2]
    assert M.select([5, 9, 9, 1, 9], 5, 3, 1, 1) == [0, 1, 4]
    assert M.select([5, 9], 2, 3, 1, 1) == [0, 1, -1]


def test_a_score_bounds_the_groups_scores():
    """Up to the rounding: |p| <= 64 and bounds to half a step each."""
    g = torch.Generator().manual_seed(1)
    for _ in range(20):
        k = torch.randn((16, 64), generator=g, dtype=torch.float64) * 2
        q = torch.randn((4, 64), generator=g, dtype=torch.float64)
        hi, lo, step = M.bounds(k, 65504.0)
        unit = 2.0 ** (M.exponent(float(q.abs().max())) - 5)
        score = float(M.scores(q, hi[None], lo[None], torch.tensor([step], dtype=torch.float64), 65504.0)) * unit
        slack = float(q.abs().sum()) * step / 2 + 4 * 64 * unit / 2 * (float(k.abs().max()) + step)
        assert score + slack >= float((q @ k.t()).sum(0).max())
