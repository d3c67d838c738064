"""GPU: decoding over selected blocks -- bounds of the blocks' keys (pa_key_bounds) and the
selection (pa_select_blocks), both exact, and the attention over the selected blocks
(pa_decode_sparse, _fp8) against the plain 64-bit forms."""
import math
import random

import pytest
import torch

import masked_reference as M

pytestmark = pytest.mark.gpu

LARGEST = {torch.bfloat16: 3.3895313892515355e38, torch.float16: 65504.0, torch.uint8: 448.0}


def pool_of(shape, dtype, g, spread=1.0):
    x = torch.randn(shape, generator=g, device="cuda") * spread
    return x.to(torch.float8_e4m3fn).view(torch.uint8) if dtype == torch.uint8 else x.to(dtype)


def layout(lens, bs, g, spare=3):
    need = [-(-L // bs) for L in lens]
    NB = sum(need) + spare
    order = torch.randperm(NB, generator=g, device="cuda").to(torch.int32)
    tables = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = order[at:at + n]
        at += n
    return tables, torch.tensor(lens, dtype=torch.int32, device="cuda"), NB


# ------------------------------------------------------------------ bounds
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.uint8])
@pytest.mark.parametrize("D,bs,Hkv", [(128, 16, 3), (64, 32, 1), (64, 16, 8), (128, 32, 2)])
@pytest.mark.parametrize("new", [[1, 1, 1, 1, 1, 1], [5, 0, 40, 33, 16, 2]])
def test_bounds(cuda_device, dtype, D, bs, Hkv, new):
    """Also zeros, tiny and huge values, infinities and NaN, rows past the context, and blocks that
    no new token is in, which keep what they have."""
    import paged_kv_cache_187_gb300 as pa
    g = torch.Generator(device="cuda").manual_seed(D + bs)
    lens = [1, 33, 40, 65, 16, 200]
    tables, lens_d, NB = layout(lens, bs, g)
    k = pool_of((NB, Hkv, bs, D), dtype, g)
    value = (lambda x: x.view(torch.float8_e4m3fn).double()) if dtype == torch.uint8 else (lambda x: x.double())
    last = [int(tables[s, (L - 1) // bs]) for s, L in enumerate(lens)]
    k[last[0]] = 0                                                      # nothing but zeros
    if dtype == torch.uint8:
        k[last[2], 0, (lens[2] - 1) % bs, 7] = 0xFF                     # NaN
        k[last[3], 0] = 1                                               # the smallest number
        k[last[4], 0, 0, 5] = 0x7E                                      # the largest
    else:
        k[last[2], 0, (lens[2] - 1) % bs, 7] = math.nan
        k[last[2], 0, :, 9] = math.nan                                  # a dim of NaN alone
        k[last[3], 0] *= 2.0 ** -14 if dtype == torch.float16 else 1e-38
        k[last[4], 0, 0, 5] = -math.inf
        k[last[4], -1, 3, 6] = math.inf
        k[last[5], 0] = (k[last[5], 0].double() * (6e4 if dtype == torch.float16 else 1e37) / 5).to(dtype)
    for s, L in enumerate(lens):
        if L % bs:
            k[last[s], :, L % bs:] = 0x7F if dtype == torch.uint8 else math.nan
    starts = torch.tensor([sum(new[:i]) for i in range(7)], dtype=torch.int32, device="cuda")
    bounds = torch.full((NB, Hkv, 2, D), 99, dtype=torch.int8, device="cuda")
    steps = torch.full((NB, Hkv), 99.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ones = new == [1] * 6
    pa.pa_key_bounds(bounds, steps, k, tables, lens_d, max(new), query_starts=None if ones else starts, status=status)
    torch.cuda.synchronize()
    n_over = any(n > L for n, L in zip(new, lens))
    assert int(status) == 0, n_over
    want, want_steps = torch.full_like(bounds, 99), torch.full_like(steps, 99.0)
    for s, L in enumerate(lens):
        for b in range(max(L - new[s], 0) // bs, -(-L // bs) if new[s] else 0):
            ph = int(tables[s, b])
            for h in range(Hkv):
                hi, lo, step = M.bounds(value(k[ph, h, :min(bs, L - b * bs)]), LARGEST[dtype])
                want[ph, h, 0], want[ph, h, 1], want_steps[ph, h] = hi.to(torch.int8), lo.to(torch.int8), step
    assert torch.equal(bounds, want)
    assert torch.equal(steps.nan_to_num(-1.0), want_steps.nan_to_num(-1.0))
    assert int(torch.isnan(steps).sum()) == int(torch.isnan(want_steps).sum())


def test_bounds_of_long_prompts_and_bad_metadata(cuda_device):
    import paged_kv_cache_187_gb300 as pa
    g = torch.Generator(device="cuda").manual_seed(2)
    lens, new, bs = [3000, 17, 1200], [2990, 17, 640], 16
    tables, lens_d, NB = layout(lens, bs, g)
    k = pool_of((NB, 2, bs, 64), torch.bfloat16, g)
    starts = torch.tensor([0, 2990, 3007, 3647], dtype=torch.int32, device="cuda")
    bounds = torch.zeros((NB, 2, 2, 64), dtype=torch.int8, device="cuda")
    steps = torch.zeros((NB, 2), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_key_bounds(bounds, steps, k, tables, lens_d, 2990, query_starts=starts, status=status)
    assert int(status) == 0
    for s, L in enumerate(lens):
        for b in range(0, -(-L // bs)):
            ph = int(tables[s, b])
            if b < (L - new[s]) // bs:
                assert not bool(bounds[ph].any()) and not bool(steps[ph].any())
                continue
            if b % 7 and b < L // bs - 1:
                continue
            hi, lo, step = M.bounds(k[ph, 1, :min(bs, L - b * bs)].double(), LARGEST[torch.bfloat16])
            assert torch.equal(bounds[ph, 1, 0].double(), hi) and torch.equal(bounds[ph, 1, 1].double(), lo)
            assert float(steps[ph, 1]) == step
    # more new tokens than the call allows for, lengths past the table, a block outside the pool
    for kw, bit in ((dict(new=100), 4), (dict(lens=[3000, 17, 99999]), 4), (dict(lens=[-1, 17, 1200]), 4),
                    (dict(bad=NB), 2), (dict(bad=-1), 2)):
        status.zero_()
        t = tables.clone()
        if "bad" in kw:
            t[1, 0] = kw["bad"]
        if "lens" in kw:
            t[t < 0] = 0
        pa.pa_key_bounds(bounds, steps, k, t, torch.tensor(kw.get("lens", lens), dtype=torch.int32, device="cuda"),
                         kw.get("new", 2990), query_starts=starts, status=status)
        assert int(status) == bit, kw


# ------------------------------------------------------------------ selection
def select_case(lens, q_len, Hq, Hkv, D, bs, dtype, seed, values=None, spare=3):
    """Bounds as keys give them; `values`: few different ones, so that many scores are equal."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    tables, lens_d, NB = layout(lens, bs, g, spare)
    q = torch.randn((len(lens), q_len, Hq, D), generator=g, device="cuda").to(dtype)
    if values:
        pick = torch.randint(0, values, (NB, Hkv, 1, 1), generator=g, device="cuda")
        bounds = (pick * 3 - 4).expand(NB, Hkv, 2, D).to(torch.int8).contiguous()
        steps = torch.full((NB, Hkv), 0.5, device="cuda")
    else:
        hi = torch.randint(-127, 128, (NB, Hkv, D), generator=g, device="cuda")
        lo = (hi - torch.randint(0, 80, (NB, Hkv, D), generator=g, device="cuda")).clamp_min(-127)
        bounds = torch.stack([hi, lo], 2).to(torch.int8)
        steps = 2.0 ** torch.randint(-7, -3, (NB, Hkv), generator=g, device="cuda").float()
    return dict(q=q, bounds=bounds, steps=steps, tables=tables, lens=lens, lens_d=lens_d, bs=bs)


def select_call(b, keep, first, last, mcl=None, status=None, ws=None, out=None, stream=None):
    import paged_kv_cache_187_gb300 as pa
    S, QL = b["q"].shape[:2]
    Hkv, mcl = b["bounds"].shape[1], mcl or max(max(b["lens"]), 1)
    if out is None:
        out = torch.full((S, QL, Hkv, keep), 77, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = torch.full((max(pa.pa_select_blocks_workspace_size(S, QL, Hkv, b["bs"], mcl), 256),), 0xA5,
                        dtype=torch.uint8, device="cuda")
    pa.pa_select_blocks(out, b["q"], b["bounds"], b["steps"], b["tables"], b["lens_d"], b["bs"], mcl, first, last,
                        workspace=ws, status=status, stream=stream)
    return out


def select_check(b, out, keep, first, last):
    S, QL, Hq, D = b["q"].shape
    Hkv, bs = b["bounds"].shape[1], b["bs"]
    g = Hq // Hkv
    for s, L in enumerate(b["lens"]):
        ids = b["tables"][s, :-(-L // bs)].long()
        for j in range(QL):
            seen = max(L - QL + j + 1, 0)
            for h in range(Hkv):
                score = M.scores(b["q"][s, j, h * g:(h + 1) * g].double(), b["bounds"][ids, h, 0].double(),
                                 b["bounds"][ids, h, 1].double(), b["steps"][ids, h].double(),
                                 LARGEST[b["q"].dtype]).tolist()
                want = M.select(score, -(-seen // bs), keep, first, last)
                assert out[s, j, h].tolist() == want, (s, j, h)


LENS = [1, 16, 17, 63 * 16, 64 * 16, 65 * 16, 64 * 16 + 1, 2000, 5000, 0]


@pytest.mark.parametrize("q_len,Hq,Hkv,D,bs,dtype,keep,first,last", [
    (1, 8, 2, 128, 16, torch.bfloat16, 64, 1, 4),
    (1, 16, 1, 64, 16, torch.float16, 64, 0, 0),
    (2, 4, 4, 128, 32, torch.float16, 7, 2, 5),          # nothing left to rank
    (5, 6, 2, 64, 16, torch.bfloat16, 33, 0, 1),
    (3, 20, 20, 128, 16, torch.bfloat16, 5, 1, 0),       # more kv heads than groups of lanes
    (1, 39, 13, 64, 32, torch.float16, 1, 0, 0),
    (4, 35, 5, 128, 16, torch.bfloat16, 100, 3, 2),
    (6, 33, 33, 64, 16, torch.float16, 16, 1, 1),
])
def test_selection(cuda_device, q_len, Hq, Hkv, D, bs, dtype, keep, first, last):
    b = select_case(LENS, q_len, Hq, Hkv, D, bs, dtype, 7 + Hq)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = select_call(b, keep, first, last, status=status)
    assert int(status) == 0
    select_check(b, out, keep, first, last)


@pytest.mark.parametrize("seqs", [2, 40])
@pytest.mark.parametrize("q_len,Hq,Hkv,D,dtype", [(1, 16, 4, 128, torch.bfloat16), (2, 14, 2, 64, torch.float16)])
def test_one_launch_and_three_select_alike(cuda_device, seqs, q_len, Hq, Hkv, D, dtype):
    """Few rows of short contexts take one launch, more rows or longer contexts three."""
    for blocks in (1024, 1025, 300):
        b = select_case([blocks * 16 - 5 - 7 * (i % 3) for i in range(seqs)], q_len, Hq, Hkv, D, 16, dtype, blocks)
        select_check(dict(b, lens=b["lens"][:3]), select_call(b, 37, 2, 3), 37, 2, 3)


@pytest.mark.parametrize("values", [1, 2, 5])
def test_equal_scores_go_to_the_lowest_block(cuda_device, values):
    b = select_case([400, 5000, 9000, 20000, 1024], 1, 8, 2, 64, 16, torch.bfloat16, 3, values=values)
    for keep, first, last in ((20, 1, 2), (500, 0, 0), (64, 0, 64), (3, 0, 1)):
        select_check(b, select_call(b, keep, first, last), keep, first, last)


def test_long_rows(cuda_device):
    """More blocks than the threads keep in registers, and a row of a million tokens."""
    b = select_case([16 * 8192 + 5, 16 * 9000, 16 * 65000 + 3], 1, 4, 2, 64, 16, torch.float16, 5)
    for keep, first, last in ((300, 1, 8), (9100, 0, 1)):
        select_check(b, select_call(b, keep, first, last), keep, first, last)
    b = select_case([16 * 20000, 16 * 70000], 1, 2, 1, 64, 16, torch.float16, 5, values=3)
    select_check(b, select_call(b, 10000, 2, 3), 10000, 2, 3)


def test_odd_values_of_queries_and_steps(cuda_device):
    """Queries of zeros, tiny and huge numbers, infinities and NaN; NaN steps."""
    for dtype in (torch.bfloat16, torch.float16):
        b = select_case([3000, 3000, 3000, 3000, 3000], 1, 4, 2, 128, 16, dtype, 9)
        b["q"][0, 0, :2] = 0
        b["q"][1] *= 2.0 ** -15 if dtype == torch.float16 else 1e-37
        b["q"][2, 0, 1, 5], b["q"][2, 0, 1, 6] = math.nan, -0.0
        b["q"][3, 0, 0, 9], b["q"][3, 0, 3, 2] = math.inf, -math.inf
        b["q"][4] *= 1e4 if dtype == torch.float16 else 1e38
        b["steps"][b["tables"][2, 5:70:9].long(), 0] = math.nan
        b["steps"][b["tables"][2, 50:52].long(), 1] = 2.0 ** -106
        for keep in (40, 5):
            select_check(b, select_call(b, keep, 1, 2), keep, 1, 2)


def test_selection_flags_bad_metadata(cuda_device):
    b = select_case([1500, 900], 2, 4, 2, 64, 16, torch.float16, 4)
    good = select_call(b, 20, 1, 2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = b["tables"].clone()
    t[0, 30] = b["bounds"].shape[0]
    out = select_call(dict(b, tables=t), 20, 1, 2, status=status)
    assert int(status) == 2 and torch.equal(out[1], good[1])
    status.zero_()
    lens = torch.tensor([1500, 90000], dtype=torch.int32, device="cuda")
    full = b["tables"].clone()
    full[full < 0] = 0
    out = select_call(dict(b, tables=full, lens_d=lens), 20, 1, 2, status=status)
    assert int(status) == 4 and torch.equal(out[0], good[0])
    status.zero_()
    out = select_call(dict(b, lens_d=torch.tensor([1500, -7], dtype=torch.int32, device="cuda")), 20, 1, 2, status=status)
    assert int(status) == 4 and torch.equal(out[0], good[0]) and bool((out[1] == -1).all())


# ------------------------------------------------------------------ attention
def sparse_case(lens, q_len, Hq, Hkv, D, bs, dtype, keep, seed, fp8=False, pick=None):
    """Rows of used blocks past their context, and blocks that no list names, hold NaN."""
    r = random.Random(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    tables, lens_d, NB = layout(lens, bs, g)
    cdt = torch.uint8 if fp8 else dtype
    kc, vc = pool_of((NB, Hkv, bs, D), cdt, g, 30.0 if fp8 else 1.0), pool_of((NB, Hkv, bs, D), cdt, g, 30.0 if fp8 else 1.0)
    nan = 0x7F if fp8 else math.nan
    lists, used = [], set()
    for s, L in enumerate(lens):
        for j in range(q_len):
            blocks = -(-max(L - q_len + j + 1, 0) // bs)
            for h in range(Hkv):
                n = r.randint(0, min(keep, blocks)) if pick is None else min(pick, keep, blocks)
                got = sorted(r.sample(range(blocks), n))
                if r.random() < 0.5 and blocks and n:
                    got = sorted(set(got[:-1] + [blocks - 1]))
                lists.append(got + [-1] * (keep - len(got)))
                used.update((int(tables[s, b]), h) for b in got)
        if L % bs:
            at = int(tables[s, L // bs])
            kc[at, :, L % bs:] = nan
            vc[at, :, L % bs:] = nan
    dead = torch.ones((NB, Hkv), dtype=torch.bool)
    for at, h in used:
        dead[at, h] = False
    kc[dead.cuda()] = nan
    vc[dead.cuda()] = nan
    selected = torch.tensor(lists, dtype=torch.int32, device="cuda").view(len(lens), q_len, Hkv, keep)
    q = torch.randn((len(lens), q_len, Hq, D), generator=g, device="cuda").to(dtype)
    return dict(q=q, kc=kc, vc=vc, tables=tables, lens=lens, lens_d=lens_d, selected=selected, scale=D ** -0.5,
                fp8=fp8, ks=0.03, vs=0.02)


def sparse_call(b, out=None, status=None, ws=None, stream=None):
    import paged_kv_cache_187_gb300 as pa
    S, QL, Hq, D = b["q"].shape
    Hkv, bs = b["kc"].shape[1:3]
    if ws is None:
        n = pa.pa_decode_sparse_workspace_size(S, QL, Hq, Hkv, D, bs, b["selected"].shape[3])
        ws = torch.full((max(n, 256),), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full_like(b["q"], 7.0) if out is None else out
    args = (out, b["q"], b["kc"], b["vc"], b["tables"], b["lens_d"], b["selected"], b["scale"])
    if b["fp8"]:
        pa.pa_decode_sparse_fp8(*args, b["ks"], b["vs"], workspace=ws, status=status, stream=stream)
    else:
        pa.pa_decode_sparse(*args, workspace=ws, status=status, stream=stream)
    return out


def sparse_reference(b):
    """The weights enter PV as two 16-bit terms (2^-16 of bf16's, and of fp16's, which lose 2^-25
    each below its range) or, over 8 bits, as fp16 (2^-11)."""
    S, QL, Hq, D = b["q"].shape
    bs, Hkv = b["kc"].shape[2], b["kc"].shape[1]
    ks, vs = (b["ks"], b["vs"]) if b["fp8"] else (1.0, 1.0)
    out = torch.zeros(b["q"].shape, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    half = b["fp8"] or b["q"].dtype == torch.float16
    for s, L in enumerate(b["lens"]):
        k, v = M.gather(b["kc"], b["tables"][s], L, ks), M.gather(b["vc"], b["tables"][s], L, vs)
        if L == 0:
            continue
        seen = torch.zeros((QL, Hkv, -(-L // bs) * bs), dtype=torch.bool)
        for j in range(QL):
            for h in range(Hkv):
                for x in b["selected"][s, j, h].tolist():
                    if x >= 0:
                        seen[j, h, x * bs:(x + 1) * bs] = True
                seen[j, h, max(L - QL + j + 1, 0):] = False
        out[s], tol[s] = M.attend(b["q"][s], k, v, seen[..., :L].cuda(), b["scale"], b["q"].dtype,
                                  2.0 ** -11 if b["fp8"] else 2.0 ** -16, 2.0 ** -24 if half else 0.0)
    return out, tol


def sparse_check(b, out):
    want, tol = sparse_reference(b)
    assert torch.isfinite(out).all()
    err = (out.double() - want).abs()
    bad = err > tol
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} beyond tolerance, worst ratio "
                           f"{float((err / tol.clamp_min(1e-30))[bad].max()):.3g}, first at {bad.nonzero()[0].tolist()}")


def sparse_run(b):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = sparse_call(b, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    sparse_check(b, out)
    return out


@pytest.mark.parametrize("q_len,Hq,Hkv,D,bs,dtype,keep,fp8", [
    (1, 8, 2, 128, 16, torch.bfloat16, 20, False),
    (1, 8, 2, 128, 32, torch.float16, 33, False),
    (3, 4, 4, 128, 16, torch.bfloat16, 40, False),        # a query head to a kv head
    (1, 16, 1, 64, 32, torch.bfloat16, 9, False),
    (2, 10, 2, 64, 16, torch.float16, 1, False),
    (5, 6, 2, 64, 16, torch.bfloat16, 64, False),
    (1, 3, 3, 64, 32, torch.float16, 31, False),
    (2, 8, 2, 128, 16, torch.bfloat16, 33, True),
    (1, 16, 1, 128, 32, torch.float16, 12, True),
    (1, 4, 4, 128, 16, torch.bfloat16, 40, True),
])
def test_selected_blocks(cuda_device, q_len, Hq, Hkv, D, bs, dtype, keep, fp8):
    sparse_run(sparse_case([1, 2, 16, 17, 300, 0, 1000, 33, 640], q_len, Hq, Hkv, D, bs, dtype, keep, 3 + Hq, fp8))


@pytest.mark.parametrize("lens,Hq,Hkv,D,bs,dtype,keep,fp8", [
    ([9000], 8, 2, 128, 16, torch.bfloat16, 300, False),                       # few rows: long lists cut
    ([40000], 4, 1, 128, 32, torch.float16, 1000, False),
    ([9000, 50, 7000], 16, 1, 64, 16, torch.bfloat16, 400, False),
    ([3000 + 10 * i for i in range(60)], 16, 4, 128, 16, torch.bfloat16, 64, False),   # many rows
    ([900 + 10 * i for i in range(130)], 8, 8, 64, 16, torch.float16, 12, False),
    ([9000, 50, 7000], 8, 2, 128, 16, torch.bfloat16, 300, True),
    ([2000 + 10 * i for i in range(60)], 8, 4, 128, 32, torch.bfloat16, 40, True),
])
def test_long_lists_and_many_rows(cuda_device, lens, Hq, Hkv, D, bs, dtype, keep, fp8):
    sparse_run(sparse_case(lens, 1, Hq, Hkv, D, bs, dtype, keep, 5 + Hq, fp8, pick=keep))


def test_all_blocks_are_a_decode(cuda_device):
    import paged_kv_cache_187_gb300 as pa
    lens = [700, 33, 512]
    b = sparse_case(lens, 1, 8, 2, 128, 16, torch.bfloat16, 44, 6, pick=44)
    out = sparse_run(b)
    ws = torch.empty(max(pa.pa_decode_auto_workspace_size(3, 8, 2, 128, 16, 700), 256), dtype=torch.uint8, device="cuda")
    want = torch.zeros_like(b["q"][:, 0])
    pa.pa_decode_auto(want, b["q"][:, 0].contiguous(), b["kc"], b["vc"], b["tables"], b["lens_d"], 700, b["scale"],
                      workspace=ws)
    assert (out[:, 0].double() - want.double()).abs().max() <= 2.0 ** -7 * want.double().abs().max()


def test_bad_lists_are_flagged_and_left_out(cuda_device):
    b = sparse_case([500, 320], 1, 4, 2, 128, 16, torch.bfloat16, 40, 8, pick=40)
    clean = sparse_run(b)
    # (entries: the first list as it is, so that every block it names holds numbers)
    full = [x for x in b["selected"][0, 0, 0].tolist() if x >= 0]
    for edit, keep in (([5, 3, 9], [5, 9]), ([2, 2, 4], [2, 4]), ([4, -1, 7], [4, 7]), ([1, 3, 99999], [1, 3]),
                       ([1, 3, 32], [1, 3]), ([-5, 3], [3]), ([2 ** 31 - 1, 0, 4], [0, 4]), ([31, 30, 29], [31])):
        sel = torch.full_like(b["selected"], -1)
        sel[1] = b["selected"][1]
        sel[0, 0, 1] = b["selected"][0, 0, 1]
        sel[0, 0, 0, 3:3 + len(edit)] = torch.tensor(edit, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = sparse_call(dict(b, selected=sel), status=status)
        torch.cuda.synchronize()
        assert int(status) == (0 if edit == [4, -1, 7] or edit == [-5, 3] else 2), edit
        assert torch.equal(out[1], clean[1]) and torch.equal(out[0, 0, 2:], clean[0, 0, 2:])
        assert all(x in full for x in keep)
        good = torch.full_like(sel, -1)
        good[:] = sel
        good[0, 0, 0] = -1
        good[0, 0, 0, :len(keep)] = torch.tensor(keep, dtype=torch.int32, device="cuda")
        sparse_check(dict(b, selected=good), out)


def test_bad_lengths_and_blocks_are_flagged(cuda_device):
    b = sparse_case([500, 320], 1, 4, 2, 128, 16, torch.bfloat16, 40, 8, pick=40)
    clean = sparse_run(b)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = b["tables"].clone()
    t[1, 3] = b["kc"].shape[0]
    out = sparse_call(dict(b, tables=t), status=status)
    assert int(status) == 2 and torch.equal(out[0], clean[0])
    status.zero_()
    out = sparse_call(dict(b, lens_d=torch.tensor([500, -3], dtype=torch.int32, device="cuda")), status=status)
    assert int(status) & 4 and torch.equal(out[0], clean[0]) and bool((out[1] == 0).all())


def test_sparse_step_in_a_graph_and_on_streams(cuda_device):
    """Bounds, selection and attention captured as one step, replayed over new keys; guards behind
    the workspaces; the same on another stream."""
    import paged_kv_cache_187_gb300 as pa
    lens, Hq, Hkv, D, bs, keep, first, last = [3000, 700, 5000], 8, 2, 128, 16, 24, 1, 3
    g = torch.Generator(device="cuda").manual_seed(2)
    tables, lens_d, NB = layout(lens, bs, g)
    kc, vc = (torch.zeros((NB, Hkv, bs, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((3, Hq, D), dtype=torch.bfloat16, device="cuda")
    bounds = torch.zeros((NB, Hkv, 2, D), dtype=torch.int8, device="cuda")
    steps = torch.zeros((NB, Hkv), device="cuda")
    selected = torch.zeros((3, Hkv, keep), dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    n1 = pa.pa_select_blocks_workspace_size(3, 1, Hkv, bs, 5000)
    n2 = pa.pa_decode_sparse_workspace_size(3, 1, Hq, Hkv, D, bs, keep)
    w1 = torch.full((n1 + 1024,), 0x5A, dtype=torch.uint8, device="cuda")
    w2 = torch.full((n2 + 1024,), 0x5A, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        pa.pa_key_bounds(bounds, steps, kc, tables, lens_d, 5000, status=status)
        pa.pa_select_blocks(selected, q, bounds, steps, tables, lens_d, bs, 5000, first, last, workspace=w1[:n1],
                            status=status)
        pa.pa_decode_sparse(out, q, kc, vc, tables, lens_d, selected, D ** -0.5, workspace=w2[:n2], status=status)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    for _ in range(3):
        for t in (kc, vc, q):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        b = dict(q=q[:, None], bounds=bounds, steps=steps, tables=tables, lens=lens, lens_d=lens_d, bs=bs, kc=kc,
                 vc=vc, selected=selected[:, None], scale=D ** -0.5, fp8=False)
        for s, L in enumerate(lens):
            hi, lo, st = M.bounds(kc[int(tables[s, 3]), 1].double(), LARGEST[torch.bfloat16])
            ph = int(tables[s, 3])
            assert torch.equal(bounds[ph, 1, 0].double(), hi) and float(steps[ph, 1]) == st
        select_check(b, selected[:, None], keep, first, last)
        sparse_check(b, out[:, None])
        before = out.clone()
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        assert torch.equal(before, out)
    assert int(status) == 0
    assert bool((w1[n1:] == 0x5A).all()) and bool((w2[n2:] == 0x5A).all())


@pytest.mark.parametrize("Hq,Hkv,D,bs,dtype,keep,fp8", [
    (4, 1, 64, 16, torch.float16, 9001, False),          # a cluster's CTAs take their pieces in several goes
    (8, 1, 128, 16, torch.bfloat16, 8999, True),         # .. whose blocks pair across the goes
    (2, 2, 128, 32, torch.bfloat16, 1200, False),
])
def test_very_long_lists(cuda_device, Hq, Hkv, D, bs, dtype, keep, fp8):
    sparse_run(sparse_case([200000, 150007, 900], 1, Hq, Hkv, D, bs, dtype, keep, 12, fp8, pick=keep))


def test_lists_longer_than_a_go_on_every_kind_of_row(cuda_device):
    """Whole rows of 700 entries (more rows than SMs have places), the first entries -1."""
    b = sparse_case([12000] * 250, 1, 8, 8, 64, 16, torch.bfloat16, 700, 13, pick=650)
    b["selected"] = torch.cat([torch.full_like(b["selected"][..., :30], -1), b["selected"]], -1).contiguous()
    out = sparse_call(b)
    torch.cuda.synchronize()
    for s in (0, 17, 249):
        one = dict(b, q=b["q"][s:s + 1], tables=b["tables"][s:s + 1], lens=[12000], selected=b["selected"][s:s + 1])
        sparse_check(one, out[s:s + 1])


@pytest.mark.parametrize("lens,Hq,Hkv,D,dtype", [
    ([700], 8, 2, 128, torch.bfloat16),                 # a cluster per row
    ([700, 90] * 60, 8, 4, 128, torch.float16),         # a CTA
    ([700], 2, 2, 64, torch.float16),                   # single heads, a cluster
    ([700, 90] * 160, 2, 2, 64, torch.bfloat16),
])
def test_nan_keys_and_values_that_a_row_sees(cuda_device, lens, Hq, Hkv, D, dtype):
    b = sparse_case(lens, 1, Hq, Hkv, D, 16, dtype, 40, 31, pick=40)
    good = sparse_call(b)
    assert bool(torch.isfinite(good).all())
    first = [int(b["tables"][0, int(b["selected"][0, 0, h, 3])]) for h in range(2)]
    b["kc"][first[0], 0, 5] = math.nan                  # kv head 0: all of it
    b["vc"][first[1], 1, 7, 11] = math.nan              # kv head 1: dim 11
    out = sparse_call(b)
    g = Hq // Hkv
    want = torch.zeros(good.shape, dtype=torch.bool, device="cuda")
    want[0, 0, :g] = True
    want[0, 0, g:2 * g, 11] = True
    assert torch.equal(torch.isnan(out), want)
    assert torch.equal(out[~want], good[~want])


def test_lists_with_room_for_every_block_of_a_long_context(cuda_device):
    b = select_case([16 * 20000 + 3, 16 * 131072, 5], 1, 2, 1, 64, 16, torch.float16, 5)
    keep = 131072
    out = select_call(b, keep, 3, 4)
    for s, L in enumerate(b["lens"]):
        n = -(-L // 16)
        assert torch.equal(out[s, 0, 0, :n], torch.arange(n, dtype=torch.int32, device="cuda"))
        assert bool((out[s, 0, 0, n:] == -1).all())
    for keep in (131071, 50):
        select_check(b, select_call(b, keep, 3, 4), keep, 3, 4)


@pytest.mark.parametrize("seqs", [1, 40])
def test_a_block_outside_the_pool_scores_zero(cuda_device, seqs):
    """Not -0, whatever stands in the pool's first block."""
    b = select_case([16 * 50] * seqs, 1, 8, 4, 64, 16, torch.bfloat16, 5)
    b["q"].abs_()
    b["bounds"].zero_()
    b["bounds"][0] = -5
    for at, block in ((3, -1), (17, b["bounds"].shape[0]), (30, 1 << 30)):
        b["tables"][:, at] = block
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = select_call(b, 25, 1, 2, status=status)
    assert int(status) == 2
    for s in range(seqs):
        worst = [i for i, x in enumerate(b["tables"][s].tolist()) if x == 0]
        want = [i for i in range(48) if i not in worst][:23] + [48, 49]
        if worst and worst[0] in (0, 48, 49):
            want = list(range(23)) + [48, 49]
        for h in range(4):
            assert out[s, 0, h].tolist() == want, (s, h)


def test_two_host_threads_and_streams_at_once(cuda_device):
    import threading
    jobs = []
    for i, (lens, keep) in enumerate((([900, 4000], 40), ([300] * 50, 9))):
        sel = select_case(lens, 1, 8, 2, 128, 16, torch.bfloat16, i)
        att = sparse_case(lens, 1, 8, 2, 128, 16, torch.bfloat16, keep, i)
        jobs.append((sel, att, keep, select_call(sel, keep, 1, 2), sparse_call(att)))
    torch.cuda.synchronize()
    wrong = []

    def work(sel, att, keep, chosen, alone):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(60):
                a = select_call(sel, keep, 1, 2, stream=stream)
                b = sparse_call(att, stream=stream)
                stream.synchronize()
                if not torch.equal(a, chosen) or not torch.equal(b, alone):
                    wrong.append(keep)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
@pytest.mark.parametrize("lens,Hq,dtype,fp8", [([700, 33], 8, torch.bfloat16, False), ([300] * 100, 2, torch.float16, False),
                                               ([700, 33], 8, torch.float16, True)])
def test_scales(cuda_device, lens, Hq, dtype, fp8, scale):
    b = sparse_case(lens, 1, Hq, 2, 128, 16, dtype, 20, 33, fp8=fp8)
    b["scale"] = scale
    sparse_check(b, sparse_call(b))
