"""INT4 KV cache: groups of 64 values with 4-bit codes, a scale and a zero point (oracle; test
infrastructure only).

KV-cache compression is listed among the tuning steps of "Nano-vLLM-Ascend: lightweight LLM inference
framework for Ascend NPU", section 4.3; no format is given.  Reading taken here: a row of D values (one
token, one KV head) is cut into D / 64 groups; a group stands for s * (code + z) with

    lo = min x, hi = max x                        (x: the 16-bit value, exact in fp32)
    s  = round16(fp32(hi / 15) - fp32(lo / 15))   round16: to nearest even in the 16-bit type of x
    z  = round16(fp32(lo / s))
    code = clip(rint(fp32(fp32(x * fp32(1 / s)) - z)), 0, 15)
    s < 2^-126:  s = |lo|, z = sign(lo), code = 0

min and max keep a NaN, so a group that holds one gets s and z NaN; one that holds an infinity gets s infinite or
NaN.  A code that is NaN before it is clipped is 0.

numpy's float32 arithmetic is IEEE, so a device kernel that takes the same steps reaches the same codes.
Stored: codes uint8 [NB, Hkv, bs, D/2]; 8 codes to a 4-byte word, lowest nibble first, word j of a row
holding values 8 * (j div n) .. + 7 of group j mod n (n = D / 64).  Parameters [NB, Hkv, bs, n, 2] = (s, z).
"""

from __future__ import annotations

import numpy as np
import torch

GROUP = 64


def _round16(a: np.ndarray, dtype) -> np.ndarray:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype).float().numpy()


def quantize_rows(x: torch.Tensor):
    """x [..., D], 16-bit.  Returns (codes uint8 [..., n, 64], s float32 [..., n], z float32 [..., n])."""
    xf = x.float().numpy()
    g = xf.reshape(*xf.shape[:-1], xf.shape[-1] // GROUP, GROUP)
    lo, hi = g.min(-1), g.max(-1)
    fifteen = np.float32(15)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        s = _round16(hi / fifteen - lo / fifteen, x.dtype)
        alike = s < np.float32(2.0 ** -126)  # not where s is NaN
        z = _round16(np.where(alike, np.sign(lo), lo / np.where(alike, np.float32(1), s)), x.dtype)
        inv = np.float32(1) / np.where(alike, np.float32(1), s)
        code = np.rint((g * inv[..., None]).astype(np.float32) - z[..., None])
    s = np.where(alike, np.abs(lo), s).astype(np.float32)
    code = np.where(alike[..., None] | np.isnan(code), 0, np.clip(code, 0, 15)).astype(np.uint8)
    return code, s, z


def pack(code: np.ndarray) -> np.ndarray:
    """Codes [..., n, 64] -> stored bytes [..., n * 32]."""
    n = code.shape[-2]
    out = np.zeros((*code.shape[:-2], n * 32), dtype=np.uint8)
    for d in range(64 * n):
        grp, within = divmod(d, GROUP)
        byte = ((within // 8) * n + grp) * 4 + (within % 8) // 2
        out[..., byte] |= code[..., grp, within] << (4 * (within % 2))
    return out


def unpack(rows: np.ndarray) -> np.ndarray:
    """Stored bytes [..., n * 32] -> codes [..., n, 64]."""
    n = rows.shape[-1] // 32
    code = np.zeros((*rows.shape[:-1], n, GROUP), dtype=np.uint8)
    for d in range(64 * n):
        grp, within = divmod(d, GROUP)
        byte = ((within // 8) * n + grp) * 4 + (within % 8) // 2
        code[..., grp, within] = (rows[..., byte] >> (4 * (within % 2))) & 15
    return code


def values(rows: np.ndarray, params: np.ndarray) -> np.ndarray:
    """The float64 values [..., D] of stored rows [..., D/2] with parameters [..., n, 2] (any float type)."""
    p = np.asarray(params, dtype=np.float64)
    v = p[..., 0:1] * (unpack(rows).astype(np.float64) + p[..., 1:2])
    return v.reshape(*v.shape[:-2], v.shape[-2] * GROUP)


def write_kv_int4(new: torch.Tensor, slot_mapping, codes: np.ndarray, params: np.ndarray) -> np.ndarray:
    """In place: quantise rows new [T, Hkv, D] into codes and params (float32 values of the 16-bit type) at
    their slots (-1: nothing).  Returns the float32 values s * (code + z) of every row [T, Hkv, D]."""
    bs = codes.shape[2]
    code, s, z = quantize_rows(new)
    packed = pack(code)
    for t, slot in enumerate(slot_mapping):
        if int(slot) < 0:
            continue
        blk, row = divmod(int(slot), bs)
        codes[blk, :, row] = packed[t]
        params[blk, :, row, :, 0] = s[t]
        params[blk, :, row, :, 1] = z[t]
    held = s[..., None] * (code.astype(np.float32) + z[..., None])
    return held.reshape(new.shape)


def cache_values(codes: np.ndarray, params: np.ndarray) -> np.ndarray:
    """The float64 cache [NB, bs, Hkv, D] that attention over the INT4 cache reads."""
    return values(codes, params).transpose(0, 2, 1, 3)
