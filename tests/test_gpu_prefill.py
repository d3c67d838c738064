"""GPU: attention of ragged chunks of new tokens over the paged cache (pa_prefill,
pa_prefill_fp8) against the plain 64-bit form, within the tolerance derived there."""
import math

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


@pytest.mark.parametrize("seqs,fp8", [
    # more sequences, and more row tiles, than the plan holds in shared memory: whole units ..
    ([(1 + (i * 37) % 90, 1 + (i * 37) % 90 + (i * 13) % 50) for i in range(900)], False),
    ([(1 + i % 3, 40 + i % 90) for i in range(600)], True),
    # .. and shares, cut through one long context among 2100 short ones
    ([(1, 1 + i % 9) for i in range(1500)] + [(2, 60000)] + [(1, 3)] * 600, False),
])
def test_batches_past_the_plans_tables(cuda_device, seqs, fp8):
    D = 128 if fp8 else 64
    run(make(seqs, 16, 1, D, 16, torch.float16, 61, fp8))


@pytest.mark.parametrize("D,dtype,fp8", [(64, torch.float16, False), (128, torch.bfloat16, False),
                                         (128, torch.bfloat16, True)])
def test_output_at_any_16_bytes(cuda_device, D, dtype, fp8):
    """Rows are stored 32 bytes at a time where the output's address allows it, else 16."""
    b = make([(40, 300), (1, 2500), (5, 64)], 6, 2, D, 16, dtype, 73, fp8)
    want = run(b)
    flat = torch.full((b["q"].numel() + 32,), 7.0, dtype=dtype, device="cuda")
    for skip in (8, 16, 24):
        flat.fill_(7.0)
        out = flat[skip:skip + b["q"].numel()].view(b["q"].shape)
        call(b, out)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert bool((flat[:skip] == 7.0).all()) and bool((flat[skip + out.numel():] == 7.0).all())


def test_two_threads_at_once(cuda_device):
    """Calls from two host threads, each on its own stream with its own workspace, give the
    bits that they give alone."""
    import threading
    jobs = [make([(90, 1000), (1, 1700)], 8, 2, 128, 16, torch.bfloat16, 67),
            make([(3, 4000), (200, 300)], 8, 2, 128, 16, torch.bfloat16, 71)]
    alone = [run(b) for b in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(b, want):
        st = torch.cuda.Stream()
        mcl = max(b["lens"])
        with torch.cuda.stream(st):
            ws, status = workspace(b, mcl), torch.zeros(1, dtype=torch.int32, device="cuda")
            for _ in range(20):
                out = call(b, torch.zeros_like(b["q"]), ws=ws, mcl=mcl, status=status)
                if not torch.equal(out, want) or int(status):
                    wrong.append(1)

    threads = [threading.Thread(target=work, args=j) for j in zip(jobs, alone)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_chunks_longer_than_the_context_and_empty_contexts(cuda_device):
    """Rows with nothing to attend to are zero rows: chunks whose first tokens lie before the
    context's start (clamped metadata), and empty contexts."""
    for fp8 in (False, True):
        b = make([(10, 4), (3, 0), (140, 130), (1, 0), (300, 1)], 8, 2, 128, 16, torch.float16, 3, fp8)
        out = run(b)
        for s, (n, L) in enumerate([(10, 4), (3, 0), (140, 130), (1, 0), (300, 1)]):
            a = int(b["starts"][s])
            assert not out[a:a + max(n - L, 0)].any()


@pytest.mark.parametrize("Hq,Hkv,D,bs,dtype,fp8", [
    (8, 2, 128, 16, torch.bfloat16, False), (4, 4, 64, 32, torch.float16, False),
    (8, 1, 128, 32, torch.float16, True)])
@pytest.mark.parametrize("spread", [12.0, 40.0])
def test_references_move(cuda_device, Hq, Hkv, D, bs, dtype, fp8, spread):
    """Scores that spread over hundreds: the largest of a row turns up in late tiles, and the
    accumulators are rescaled there."""
    b = make([(33, 1400), (1, 3000), (200, 900), (5, 128)], Hq, Hkv, D, bs, dtype, 17, fp8,
             spread=spread if not fp8 else min(spread, 3.0))
    # growing along the context
    for s, L in enumerate(b["lens"]):
        for t, i in enumerate(b["tables"][s, :-(-L // bs)].tolist()):
            f = 0.1 + 2.0 * t * bs / L
            if not fp8:
                b["kc"][i] = (b["kc"][i].float() * f).to(dtype)
    run(b)


@pytest.mark.parametrize("D,dtype,fp8", [(128, torch.float16, False), (64, torch.float16, False),
                                         (128, torch.bfloat16, False), (128, torch.bfloat16, True)])
@pytest.mark.parametrize("C,L", [(1, 8192), (130, 3000)])
def test_a_long_tail_behind_one_large_weight(cuda_device, D, dtype, fp8, C, L):
    """Token 0 has nearly all the weight and a value of 0; the others, 2^-23.5 each, a value
    near 1.  Relative to the largest weight they lie below fp16's smallest step, 2^-24, by a
    rounding of a third."""
    b = make([(C, L)], 4, 1, D, 16, dtype, 29, fp8)
    ids = b["tables"][0, :-(-L // 16)].long()
    b["q"].zero_()
    b["q"][..., 0] = 16.0
    key = 23.5 * math.log(2.0) / b["scale"] / 16.0
    if fp8:
        b["kc"][ids] = 0
        b["vc"][ids] = torch.tensor(1.0 / b["vs"], device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
        b["kc"][ids[0], 0, 0, 0] = torch.tensor(key / b["ks"], device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        b["kc"][ids] = 0
        b["vc"][ids] = 1.0
        b["kc"][ids[0], 0, 0, 0] = key
    b["vc"][ids[0], 0, 0] = 0
    run(b)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-4, 2.0])
def test_scales(cuda_device, scale):
    for fp8 in (False, True):
        b = make([(40, 500), (1, 900)], 4, 2, 128, 16, torch.float16, 19, fp8)
        b["scale"] = scale
        run(b)


def test_rows_outside_the_chunks_are_left_alone(cuda_device):
    b = make([(9, 100), (0, 50), (130, 400)], 4, 2, 128, 16, torch.bfloat16, 29, extra=37)
    shift = 11                                     # rows before the first chunk as well
    b["starts"] = b["starts"] + shift
    b["starts_d"] += shift
    out = call(b, torch.full_like(b["q"], 7.0))
    want, tol = reference(b)
    n = int(b["starts"][-1])
    assert (out[:shift] == 7).all() and (out[n:] == 7).all()
    assert ((out[shift:n].double() - want[shift:n]).abs() <= tol[shift:n]).all()


@pytest.mark.parametrize("D,dtype,fp8", [(128, torch.bfloat16, False), (64, torch.float16, False),
                                         (128, torch.float16, True)])
@pytest.mark.parametrize("seqs,at", [([(40, 300)], 270), ([(3, 200)], 198), ([(90, 1000), (5, 1700)], 950),
                                     ([(1, 400), (20, 40)], 399), ([(257, 257)], 100)])
def test_infinities_and_nan_in_masked_places(cuda_device, D, dtype, fp8, seqs, at):
    """Token `at` of each sequence (or its last) holds infinite and NaN elements of V, and the
    one after it NaN in K: rows before them come out as if they were not there, rows that see
    the V elements get them, rows that see the K get NaN."""
    Hq, Hkv, bs = 8, 2, 16
    b = make(seqs, Hq, Hkv, D, bs, dtype, 31, fp8)
    clean = {k: b[k].clone() for k in ("kc", "vc")}
    nan, inf = (0x7F, None) if fp8 else (float("nan"), float("inf"))
    hurt = []
    for s, (n, L) in enumerate(seqs):
        t = min(at, L - 1)
        block = int(b["tables"][s, t // bs])
        b["vc"][block, 0, t % bs, 5] = nan
        if not fp8:
            b["vc"][block, 0, t % bs, 7] = inf
            b["vc"][block, 1, t % bs, 9] = -inf
        t2 = min(t + 1, L - 1)
        b["kc"][int(b["tables"][s, t2 // bs]), 1, t2 % bs] = nan
        hurt.append((t, t2))
    out = call(b, torch.zeros_like(b["q"]))
    b["kc"], b["vc"] = clean["kc"], clean["vc"]
    want, tol = reference(b)
    g = Hq // Hkv
    for s, (n, L) in enumerate(seqs):
        a, (t, t2) = int(b["starts"][s]), hurt[s]
        for j in range(n):
            pos, row, w, e = L - n + j, out[a + j].double(), want[a + j], tol[a + j]
            good = torch.ones(Hq, D, dtype=torch.bool, device="cuda")
            if pos >= t:
                assert torch.isnan(row[:g, 5]).all()
                good[:g, 5] = False
                if not fp8:
                    assert (row[:g, 7] == inf).all() and (pos >= t2 or (row[g:, 9] == -inf).all())
                    good[:g, 7] = False
                    good[g:, 9] = False
            if pos >= t2:
                assert torch.isnan(row[g:]).all()
                good[g:] = False
            assert ((row - w).abs() <= e)[good].all(), (s, j)


def test_bad_metadata_is_flagged_and_never_faults(cuda_device):
    import paged_kv_cache_187_gb300 as pa
    b = make([(30, 200), (20, 100)], 4, 2, 128, 16, torch.bfloat16, 37)
    ws = workspace(b, 4096)
    out = torch.zeros_like(b["q"])

    def flags(**change):
        c = dict(b, **change)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(c, out, ws=ws, mcl=change.get("mcl", 200), status=status)
        torch.cuda.synchronize()
        return int(status)

    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    assert flags() == 0
    assert flags(starts_d=i32([0, 40, 30])) == pa.PA_DEVERR_BAD_LEN          # descending
    assert flags(starts_d=i32([-5, 30, 50])) == pa.PA_DEVERR_BAD_LEN
    assert flags(starts_d=i32([0, 30, 2 ** 31 - 1])) == pa.PA_DEVERR_BAD_LEN
    assert flags(starts_d=i32([50, 0, 50])) == pa.PA_DEVERR_BAD_LEN
    assert flags(lens_d=i32([300, 100])) == pa.PA_DEVERR_BAD_LEN             # > max_context_len
    assert flags(lens_d=i32([-1, 100])) == pa.PA_DEVERR_BAD_LEN
    assert flags(lens_d=i32([2 ** 31 - 1, 100]), mcl=4096) == pa.PA_DEVERR_BAD_LEN   # > the row
    bad = b["tables"].clone()
    bad[0, 3], bad[1, 0] = b["kc"].shape[0], -7
    assert flags(tables=bad) == pa.PA_DEVERR_BAD_BLOCK
    # overlapping chunks want more row tiles than there is room for
    many = make([(20, 20)] * 12, 16, 1, 128, 16, torch.bfloat16, 38)
    many["starts_d"] = i32([0, 240] * 6 + [0])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(many, torch.zeros_like(many["q"]), status=status)
    torch.cuda.synchronize()
    assert int(status) == pa.PA_DEVERR_BAD_LEN
    check(b, call(b, out, ws=ws))                                            # and all is well


def test_streams_graphs_and_shared_workspaces(cuda_device):
    """Captured calls give the eager results bit for bit, replayed with other inputs in place
    too; two graphs on one workspace take turns; a call on a side stream with its own."""
    shapes = [[(40, 900), (1, 3000)], [(1, 700), (300, 300), (5, 64)]]
    bs = [make(s, 8, 2, 128, 16, torch.bfloat16, 41 + i) for i, s in enumerate(shapes)]
    ws = max((workspace(b, 3000) for b in bs), key=lambda w: w.numel())
    eager = [call(b, torch.zeros_like(b["q"]), ws=ws, mcl=3000) for b in bs]
    torch.cuda.synchronize()
    outs, graphs = [torch.zeros_like(b["q"]) for b in bs], []
    for b, o in zip(bs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(b, o, ws=ws, mcl=3000)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for e, o in zip(eager, outs):
            assert torch.equal(e, o)
    # new contents in the captured buffers
    new = make(shapes[0], 8, 2, 128, 16, torch.bfloat16, 77)
    for k in ("q", "kc", "vc", "tables"):
        bs[0][k].copy_(new[k])
    graphs[0].replay()
    torch.cuda.synchronize()
    check(bs[0], outs[0])
    # two streams at once, each with its own workspace
    side = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.zeros_like(ws) for _ in range(2)]
    got = [torch.zeros_like(b["q"]) for b in bs]
    want = [call(b, torch.zeros_like(b["q"]), ws=ws, mcl=3000) for b in bs]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, o, w, st in zip(bs, got, spaces, side):
            call(b, o, ws=w, mcl=3000, stream=st)
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert torch.equal(o, w)


def test_the_same_call_gives_the_same_bits(cuda_device):
    for fp8 in (False, True):
        b = make([(70, 5000), (1, 900), (20, 8000)], 16, 2, 128, 16, torch.bfloat16, 43, fp8)
        first = call(b, torch.zeros_like(b["q"]))
        for _ in range(5):
            assert torch.equal(first, call(b, torch.zeros_like(b["q"])))


@pytest.mark.parametrize("Hq,Hkv,D,dtype,fp8", [(6, 2, 64, torch.bfloat16, False), (6, 2, 128, torch.bfloat16, True),
                                               (7, 1, 128, torch.float16, False)])
def test_bits_do_not_depend_on_rows_without_a_query(cuda_device, Hq, Hkv, D, dtype, fp8):
    """Groups of 3 and 7 leave rows of a stream's 128 unused, and short chunks leave more: what
    an earlier call left there changes nothing."""
    b = make([(40, 300), (1, 2500), (5, 64), (18, 900)], Hq, Hkv, D, 16, dtype, 79, fp8)
    loud = make([(200, 400), (60, 2000)], Hq, Hkv, D, 16, dtype, 83, fp8)
    loud["q"] *= 50.0
    quiet = dict(loud, q=loud["q"] * 1e-4)
    want = run(b)
    for other in (loud, quiet, b, loud):
        call(other, torch.empty_like(other["q"]))
        assert torch.equal(call(b, torch.zeros_like(b["q"])), want)


def test_single_tokens_agree_with_the_decode(cuda_device):
    """One new token per sequence is an ordinary decode: both within tolerance of the formula."""
    import paged_kv_cache_187_gb300 as pa
    lens = [1, 5, 128, 129, 700, 2500]
    b = make([(1, L) for L in lens], 32, 8, 128, 16, torch.bfloat16, 47)
    ref = reference(b)
    check(b, call(b, torch.zeros_like(b["q"])), ref)
    out = torch.zeros_like(b["q"])
    pa.pa_decode_v1(out, b["q"], b["kc"], b["vc"], b["tables"], b["lens_d"], 2500, b["scale"])
    check(b, out, ref)


def test_offsets_past_32_bits(cuda_device):
    """A pool of more than 2^32 bytes and 2^31 elements, the sequences in its last blocks."""
    NB, Hkv, bs, D = 150_000, 8, 16, 128
    small = make([(50, 700), (1, 300)], 16, Hkv, D, bs, torch.bfloat16, 53)
    n = small["kc"].shape[0]
    big = {}
    for k in ("kc", "vc"):
        big[k] = torch.empty((NB, Hkv, bs, D), dtype=torch.bfloat16, device="cuda")
        big[k][NB - n:] = small[k]
    t = small["tables"]
    b = dict(small, **big, tables=torch.where(t >= 0, t + (NB - n), t))
    assert b["kc"].numel() > 2 ** 31
    assert torch.equal(call(b, torch.zeros_like(b["q"])), call(small, torch.zeros_like(b["q"])))
    check(small, call(b, torch.zeros_like(b["q"])))


def test_long_context(cuda_device):
    run(make([(3, 70_001)], 8, 1, 128, 32, torch.float16, 59))


def test_empty_calls(cuda_device):
    b = make([(0, 10), (0, 0)], 4, 2, 128, 16, torch.float16, 61, extra=4)
    out = call(b, torch.full_like(b["q"], 3.0))
    torch.cuda.synchronize()
    assert (out == 3).all()


@pytest.mark.parametrize("Hq,Hkv,D,bs,dtype,fp8", [
    (8, 2, 128, 16, torch.bfloat16, False), (4, 1, 64, 32, torch.float16, False),
    (16, 1, 128, 16, torch.float16, True)])
@pytest.mark.parametrize("seqs", [
    [(17, 317)], [(1, 1)], [(1, 1024)], [(0, 3), (0, 0), (5, 70), (0, 9), (40, 40), (0, 1)],
    [(1, 7 * i + 1) for i in range(32)], [(1, 40)] * 33, [(100, 1000), (3, 1), (9, 4)], [(1, 1025)],
    [(600, 1000)]])
def test_small_calls_without_a_plan_and_their_neighbours(cuda_device, Hq, Hkv, D, bs, dtype, fp8, seqs):
    """Up to 32 sequences, a unit per CTA and contexts up to 1024 tokens are not planned; one
    sequence, token or unit more are."""
    run(make(seqs, Hq, Hkv, D, bs, dtype, 67, fp8))
