"""Plain 64-bit forms of the chunk operators, with the error each result may have.

A kernel's error is bounded by its roundings, each at most half a step of its type: u =
finfo(t).eps / 2 relative to the rounded value (2^-8 bf16, 2^-11 fp16, 2^-24 fp32).
"""
import math

import torch

FP32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def cache_values(pool, scale=1.0):
    if pool.dtype == torch.uint8:
        return pool.view(torch.float8_e4m3fn).double() * scale
    return pool.double()


def prefill(q, kc, vc, tables, lens, starts, scale, k_scale=1.0, v_scale=1.0):
    """(out, tolerance), both fp64 [T, Hq, D], of attention over the paged pools: per row and
    head, out = sum_t w_t v_t over the tokens it sees.

    Tolerance of a row, with W = sum_t w_t |v_t| and u the half step of the 16-bit type that
    holds the weights:
      u W                  the weights are rounded once;
      2^-32 sum_t |v_t|    ... and below fp16's normal range by up to 2^-25 each, while the
                           weights are relative to one of at least 2^7 (bf16 has fp32's range);
      u_out |out|          the output is rounded once;
      W (2 D 2^-24 A + 2^-20 + (L / 16) 2^-23)
                           scores: D products summed in fp32, each step of the sum off by at
                           most 2^-24 of A = scale sum_d |q_d k_d|, twice (numerator and weight
                           sum); exp2, its argument and the division a few fp32 steps; and the
                           sums over the context, 16 tokens a step, numerator and weights.
    """
    T, Hq, D = q.shape
    Hkv, bs = kc.shape[1], kc.shape[2]
    g = Hq // Hkv
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    pdt = torch.float16 if kc.dtype == torch.uint8 else q.dtype
    for s, L in enumerate(lens):
        a, b = int(starts[s]), int(starts[s + 1])
        n, L = b - a, int(L)
        if n == 0 or L == 0:
            continue
        ids = tables[s, :(L + bs - 1) // bs].long()
        k = cache_values(kc[ids], k_scale).transpose(1, 2).reshape(-1, Hkv, D)[:L]
        v = cache_values(vc[ids], v_scale).transpose(1, 2).reshape(-1, Hkv, D)[:L]
        # every new token at once; one by one where masked values must not be touched
        whole = bool(torch.isfinite(k).all() and torch.isfinite(v).all())
        for j0, j1 in [(0, n)] if whole else [(j, j + 1) for j in range(n)]:
            lim = L - n + 1 + torch.arange(j0, j1, device=q.device)
            seen = max(int(lim[-1]), 0) if not whole else L
            if seen == 0:
                continue
            kk, vv = k[:seen].repeat_interleave(g, 1), v[:seen].repeat_interleave(g, 1)
            x = q[a + j0:a + j1].double()
            hide = torch.arange(seen, device=q.device) >= lim[:, None]
            y = (torch.einsum("nhd,thd->hnt", x, kk) * scale).masked_fill(hide, -math.inf)
            A = (torch.einsum("nhd,thd->hnt", x.abs(), kk.abs()) * abs(scale)).masked_fill(hide, 0).amax(-1)
            w = torch.softmax(y, -1).masked_fill((lim <= 0)[None, :, None], 0.0)
            o = torch.einsum("hnt,thd->nhd", w, vv)
            W = torch.einsum("hnt,thd->nhd", w, vv.abs())
            out[a + j0:a + j1] = o
            t = half_step(pdt) * W + half_step(q.dtype) * o.abs()
            t += W * (2 * D * FP32 * A.t()[..., None] + 2.0 ** -20 + L / 16 * 2 * FP32)
            if pdt == torch.float16:
                t += 2.0 ** -32 * torch.einsum("nt,thd->nhd", (~hide).double(), vv.abs())
            tol[a + j0:a + j1] = t
    return out, tol


def rope(x, positions, inv_freq, pair_axes, interleaved):
    """x [T, H, D] rotated, fp64."""
    half = inv_freq.numel()
    axes = torch.as_tensor(pair_axes if pair_axes is not None else [0] * half, device=x.device)
    a = positions[axes].t().double() * inv_freq.double()       # [T, half]
    c, s = a.cos()[:, None], a.sin()[:, None]
    y = x.double().clone()
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    u, v = x.double()[..., first], x.double()[..., second]
    y[..., first], y[..., second] = u * c - v * s, u * s + v * c
    size = torch.zeros_like(y)                                 # |u| + |v| of each rotated pair
    size[..., first] = size[..., second] = u.abs() + v.abs()
    return y, size
