"""Shared by the INT4 cache tests: caches built by the oracle's quantiser, and the bounds that arithmetic
gives for decode over them.

Bounds of one output element (u = half a step of the output type relative to the value; everything else
fp32): with w_t the softmax weights, v_t the dequantised values,
    A  = sum_t w_t |v_t|,                 A' = sum_t w_t s_t (15 + |z_t|)   (code and zero-point parts apart)
    d  = 2^-19 * max_t scale * sum_d |q_d| s_t (15 + |z_t|)   the scores' rounding: under 16 accumulation
         steps of 2^-23 each, code and zero-point parts apart
|err| <= u |ref| + 2^-11 A (each weight times its V scale is rounded once to fp16, half a step 2^-11)
       + ((8 + L / 16) 2^-23 + L 2^-28) A' (fp32 accumulation over L / 16 steps; fp16 weights below 2^-14,
         whose spacing is 2^-24 against a largest of at least 2^3, half of it to each side)
       + 2 d (A + |ref|) + 2^-20 (A + |ref|) (scores and exp2 through numerator and denominator)
The log-sum-exp: d + 2^-20 + 2^-21 |lse|.
"""

from __future__ import annotations

import numpy as np
import torch

from oracle import kv_int4 as oq

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def empty_cache(NB, Hkv, bs, D, dtype, device="cuda"):
    c = torch.zeros((NB, Hkv, bs, D // 2), dtype=torch.uint8, device=device)
    p = torch.zeros((NB, Hkv, bs, D // 64, 2), dtype=dtype, device=device)
    return c, torch.zeros_like(c), p, torch.zeros_like(p)


def quantized_pool(x: torch.Tensor):
    """16-bit pool [NB, bs, Hkv, D] -> (codes uint8 [NB, Hkv, bs, D/2], params float32 [NB, Hkv, bs, n, 2])."""
    code, s, z = oq.quantize_rows(x.transpose(1, 2).contiguous())
    return oq.pack(code), np.stack([s, z], axis=-1).astype(np.float32)


def to_device(kc, vc, kp, vp, dtype, device="cuda"):
    f = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
    return f(kc), f(vc), f(kp).to(dtype), f(vp).to(dtype)


def reference(q, kc, vc, kp, vp, tables, lens, scale, rows=None, want_bound=True):
    """float64 decode over the stored cache for (sequence, head) pairs `rows` (all when None).
    Returns (rows, out [n, D], lse [n], bound [n, D], lse_bound [n])."""
    qf = q.double().numpy()
    B, Hq, D = qf.shape
    Hkv, bs = kc.shape[1], kc.shape[2]
    G = Hq // Hkv
    rows = [(b, h) for b in range(B) for h in range(Hq)] if rows is None else rows
    u = torch.finfo(q.dtype).eps / 2
    out, lse = np.zeros((len(rows), D)), np.full(len(rows), -np.inf)
    bound, lse_bound = np.zeros((len(rows), D)), np.zeros(len(rows))
    seen = {}
    for i, (b, h) in enumerate(rows):
        L = int(lens[b])
        if L == 0:
            continue
        key = (b, h // G)
        if key not in seen:
            seen.clear()  # rows come sorted: one (sequence, KV head) at a time
            blk = np.asarray(tables[b][: -(-L // bs)], dtype=np.int64)
            take = lambda a: a[blk, h // G].reshape(-1, *a.shape[3:])[:L]  # noqa: E731
            kpar, vpar = np.asarray(take(kp), dtype=np.float64), np.asarray(take(vp), dtype=np.float64)
            span = lambda par: np.repeat(np.abs(par[..., 0]) * (15 + np.abs(par[..., 1])), 64, axis=-1)  # noqa: E731
            seen[key] = (oq.values(take(kc), kpar), oq.values(take(vc), vpar), span(kpar), span(vpar))
        k, v, kspan, vspan = seen[key]
        x = (k @ qf[b, h]) * scale
        top = x.max()
        p = np.exp(x - top)
        lse[i] = top + np.log(p.sum())
        w = p / p.sum()
        out[i] = w @ v
        if want_bound:
            d = 2.0 ** -19 * scale * (kspan @ np.abs(qf[b, h])).max()
            A, A2 = w @ np.abs(v), w @ vspan
            r = np.abs(out[i])
            bound[i] = (u * r + 2.0 ** -11 * A + ((8 + L / 16) * 2.0 ** -23 + L * 2.0 ** -28) * A2
                        + (2 * d + 2.0 ** -20) * (A + r) + torch.finfo(q.dtype).tiny)
            lse_bound[i] = d + 2.0 ** -20 + 2.0 ** -21 * abs(lse[i])
    return rows, out, lse, bound, lse_bound


def assert_within(got, ref, bound, what=""):
    got = np.asarray(got, dtype=np.float64)
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; first at {i}: got {got[i]!r} ref {ref[i]!r} "
                             f"bound {bound[i]:.3e}; worst err/bound {np.nanmax(err / np.maximum(bound, 1e-300)):.3g}")
