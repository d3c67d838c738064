"""Plain 64-bit forms of the operators whose reads of the cache follow a mask: trees of new
tokens, key bounds, the selection of blocks, attention over selected blocks; with the error
that each attention result may have (the bounds and selections are exact)."""
import math

import torch

import chunk_reference as R

FP32 = R.FP32


def gather(pool, table, length, scale=1.0):
    """Rows of a sequence's first `length` tokens, fp64 [length, Hkv, D]."""
    bs = pool.shape[2]
    ids = table[:(length + bs - 1) // bs].long()
    return R.cache_values(pool[ids], scale).transpose(1, 2).reshape(-1, pool.shape[1], pool.shape[3])[:length]


def attend(q, k, v, seen, scale, out_dtype, weight_step, lost=0.0):
    """(out, tolerance) fp64 [n, Hq, D] of query rows q [n, Hq, D] over tokens k, v [L, Hkv, D]
    (fp64) that `seen` [n, Hkv, L] names; rows without any are 0.

    Tolerance of a row, with W = sum_t w_t |v_t|:
      weight_step W        the weights are rounded once
      lost sum_t |v_t|     ... and lose at most this much below the range of their type
      u_out |out|          the output is rounded once
      W (2 D 2^-24 A + 2^-20 + (L / 16) 2^-23)
                           scores: D products summed in fp32, each step off by at most 2^-24 of
                           A = scale sum_d |q_d k_d|, in numerator and weight sum; exp2, its
                           argument and the division a few fp32 steps; the sums over the
                           context, 16 tokens a step, numerator and weights."""
    n, Hq, D = q.shape
    Hkv = k.shape[1]
    g = Hq // Hkv
    out = torch.zeros((n, Hq, D), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    # (a masked value must not be touched: rows one by one unless everything is finite)
    whole = bool(torch.isfinite(k).all() and torch.isfinite(v).all())
    for h in range(Hkv):
        rows = [slice(0, n)] if whole else [slice(i, i + 1) for i in range(n)]
        for r in rows:
            keep = seen[r, h]
            kk, vv = k[:, h], v[:, h]
            if not whole:
                at = keep[0].nonzero()[:, 0]
                kk, vv, keep = kk[at], vv[at], keep[:, at]
            if keep.shape[-1] == 0:
                continue
            x = q[r, h * g:(h + 1) * g].double()
            hide = ~keep[:, None, :]
            y = (torch.einsum("nhd,td->nht", x, kk) * scale).masked_fill(hide, -math.inf)
            A = (torch.einsum("nhd,td->nht", x.abs(), kk.abs()) * abs(scale)).masked_fill(hide, 0).amax(-1)
            w = torch.softmax(y, -1).masked_fill(~keep.any(-1)[:, None, None], 0.0)
            o = torch.einsum("nht,td->nhd", w, vv)
            W = torch.einsum("nht,td->nhd", w, vv.abs())
            L = keep.shape[-1]
            t = weight_step * W + R.half_step(out_dtype) * o.abs()
            t += W * (2 * D * FP32 * A[..., None] + 2.0 ** -20 + L / 16 * 2 * FP32)
            t += lost * torch.einsum("nt,td->nd", keep.double(), vv.abs())[:, None]
            out[r, h * g:(h + 1) * g] = o
            tol[r, h * g:(h + 1) * g] = t
    return out, tol


def tree(q, kc, vc, tables, lens, starts, sees, scale, k_scale=1.0, v_scale=1.0):
    """sees[s]: bool [C, C], what each new token of sequence s sees of its own tree.  The weights
    enter as one term of the cache's 16-bit type (fp16 over 8 bits), fp16's 2^7 larger."""
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    pdt = torch.float16 if kc.dtype == torch.uint8 else q.dtype
    for s, L in enumerate(lens):
        a, b = int(starts[s]), int(starts[s + 1])
        n, L = b - a, int(L)
        if n == 0 or L == 0:
            continue
        seen = torch.ones((n, L), dtype=torch.bool, device=q.device)
        first = max(n - L, 0)                    # new tokens that the context does not hold
        own = sees[s].to(q.device).tril()
        seen[:, max(L - n, 0):] = own[:, first:]
        k, v = gather(kc, tables[s], L, k_scale), gather(vc, tables[s], L, v_scale)
        seen = seen[:, None].expand(n, kc.shape[1], L)
        o, t = attend(q[a:b], k, v, seen, scale, q.dtype, R.half_step(pdt),
                      2.0 ** -32 if pdt == torch.float16 else 0.0)
        out[a:b], tol[a:b] = o, t
    return out, tol


def masks(sees, words, device):
    """int32 [T, words] of the trees' bool matrices."""
    rows = []
    for m in sees:
        n = m.shape[0]
        wide = torch.zeros((n, 32 * words), dtype=torch.int64)
        wide[:, :min(n, 32 * words)] = m[:, :32 * words].long()
        rows.append((wide.view(n, words, 32) << torch.arange(32)).sum(-1))
    return torch.cat(rows).to(torch.int32).to(device) if rows else torch.zeros((0, words), dtype=torch.int32, device=device)


def paths(parents):
    """What a tree's nodes see: their ancestors and themselves."""
    n = len(parents)
    m = torch.zeros((n, n), dtype=torch.bool)
    for i, p in enumerate(parents):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def accept(parents, draft, target, most):
    """(path, next token) of one tree by the definition."""
    if not parents:
        return [], -1
    got = {0: [0]}
    for i in range(1, len(parents)):
        if parents[i] in got and draft[i] == target[parents[i]]:
            got[i] = got[parents[i]] + [i]
    path = max(got.values(), key=lambda p: (len(p), -p[-1]))[:most]
    return path, target[path[-1]]


def exponent(x):
    """floor(log2 x) of x > 0 (Python float)."""
    return math.frexp(x)[1] - 1


def bounds(k, largest):
    """(hi, lo, step) of rows k [n, D] (fp64): whole numbers and the step."""
    nan = torch.isnan(k)
    x = k.clamp(-largest, largest)
    m = float(torch.where(nan, torch.zeros_like(x), x).abs().max())
    e = min(max(exponent(m), -100), 96) if m > 0 else -100
    y = torch.round(x * 2.0 ** (6 - e)).clamp(-127, 127)
    none = nan.all(0)
    hi = torch.where(nan, torch.full_like(y, -1e9), y).amax(0)
    lo = torch.where(nan, torch.full_like(y, 1e9), y).amin(0)
    hi[none] = lo[none] = 0
    return hi, lo, math.nan if bool(nan.any()) else 2.0 ** (e - 6)


def scores(q, hi, lo, step, largest):
    """Scores [B] of the blocks' bounds hi, lo [B, D] (fp64) and steps [B] for a group's rows q
    [g, D] (fp64); a NaN step gives +inf."""
    q = torch.nan_to_num(q.clamp(-largest, largest), nan=0.0)
    m = float(q.abs().max())
    e = max(exponent(m), -100) if m > 0 else -100
    p = torch.round(q * 2.0 ** (5 - e))
    total = torch.zeros(hi.shape[0], dtype=torch.float64, device=q.device)
    for r in range(q.shape[0]):
        total += torch.maximum(p[r] * hi, p[r] * lo).sum(-1)
    return torch.where(torch.isnan(step), torch.full_like(total, math.inf), total * step.nan_to_num(0.0))


def select(score, blocks, keep, first, last):
    """The selection among `blocks` blocks with scores [>= blocks] (a list)."""
    if blocks <= keep:
        got = list(range(blocks))
    else:
        got = list(range(first)) + list(range(blocks - last, blocks))
        middle = sorted(range(first, blocks - last), key=lambda b: (-score[b], b))
        got = sorted(got + middle[:keep - len(got)])
    return got + [-1] * (keep - len(got))
