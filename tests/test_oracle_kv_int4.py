"""The oracle's INT4 cache format: stored places, the error of a group, and mistakes planted in it."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv_int4 as oq

TYPES = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("n", [1, 2])
def test_pack_places_every_code(n):
    """unpack undoes pack, and one code alone lands in the nibble that the format names."""
    rng = np.random.default_rng(n)
    code = rng.integers(0, 16, (3, 5, n, 64)).astype(np.uint8)
    assert np.array_equal(oq.unpack(oq.pack(code)), code)
    for d in (0, 1, 7, 8, 63) + ((64, 71, 127) if n == 2 else ()):
        one = np.zeros((n, 64), np.uint8)
        one[d // 64, d % 64] = 13
        word = int.from_bytes(oq.pack(one).tobytes(), "little")
        j = (d % 64) // 8 * n + d // 64                     # word j: 8 values from 8 (j div n) of group j mod n
        assert word == 13 << (32 * j + 4 * (d % 8))


def _rows(dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(40, 3, 128, generator=g) * torch.exp(2 * torch.randn(40, 3, 1, generator=g))
    x[:10] += 5 * torch.randn(10, 3, 1, generator=g)
    return x.to(dtype)


def _errors(x, held, s, z):
    """|x - held| against half a step, the range lost to the roundings of s and z, and those of the arithmetic:
    s and z are off by at most u (half a step of the type) relative, so the ends of the codes' span lie up to
    15 u s + u |z| s away from lo and hi; x / s - z rounds to 2^-22 (|x / s| + |z|) of a step."""
    u = torch.finfo(x.dtype).eps / 2
    g = x.double().numpy().reshape(*x.shape[:-1], -1, 64)
    err = np.abs(g - held)
    step = s[..., None].astype(np.float64)
    zz = np.abs(z[..., None].astype(np.float64))
    return err, step * (0.5 + 15 * u + u * zz + 2.0 ** -22 * (np.abs(g) / np.maximum(step, 1e-300) + zz)) * (1 + 1e-12)


@pytest.mark.parametrize("dtype", TYPES)
def test_group_error_is_half_a_step(dtype):
    x = _rows(dtype, 1)
    code, s, z = oq.quantize_rows(x)
    err, bound = _errors(x, s[..., None].astype(np.float64) * (code + z[..., None].astype(np.float64)), s, z)
    assert (err <= bound).all()
    assert code.max() == 15 and code.min() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_groups_of_one_value_are_exact(dtype):
    x = torch.zeros(6, 1, 64, dtype=dtype)
    x[1], x[2], x[3] = 0.75, -3.0, torch.finfo(dtype).max
    x[4], x[5] = torch.finfo(dtype).min, torch.finfo(dtype).tiny
    code, s, z = oq.quantize_rows(x)
    held = s[..., None].astype(np.float64) * (code + z[..., None])
    assert np.array_equal(held.reshape(x.shape), x.double().numpy()) and (code == 0).all()


def test_largest_values_of_both_signs_do_not_overflow():
    for dtype in TYPES:
        x = torch.zeros(1, 1, 64, dtype=dtype)
        x[0, 0, 0], x[0, 0, 1] = torch.finfo(dtype).max, torch.finfo(dtype).min
        code, s, z = oq.quantize_rows(x)
        assert np.isfinite(s).all() and np.isfinite(z).all() and code[0, 0, 0, 0] == 15 and code[0, 0, 0, 1] == 0


@pytest.mark.parametrize("name", ["words in order", "high nibble first", "zero point dropped", "truncated codes"])
def test_planted_mistakes_are_caught(name):
    """Each mistake in the stored form moves a value further than the error of a group allows."""
    x = _rows(torch.bfloat16, 2)
    code, s, z = oq.quantize_rows(x)
    stored = oq.pack(code)
    params = np.stack([s, z], -1)
    if name == "words in order":
        stored = stored.reshape(*stored.shape[:-1], 8, 2, 4).swapaxes(-3, -2).reshape(stored.shape)
    elif name == "high nibble first":
        stored = (stored >> 4) | (stored << 4)
    elif name == "zero point dropped":
        params[..., 1] = -7.5
    else:
        g = x.float().numpy().reshape(*x.shape[:-1], -1, 64)
        stored = oq.pack(np.clip(np.floor(g / s[..., None] - z[..., None]), 0, 15).astype(np.uint8))
    held = oq.values(stored, params).reshape(*x.shape[:-1], -1, 64)
    err, bound = _errors(x, held, s, z)
    assert (err > bound).any()


@pytest.mark.parametrize("dtype", TYPES)
def test_a_nan_or_infinity_spoils_its_group(dtype):
    x = _rows(dtype, 5)
    bad = x.clone()
    bad[3, 1, 70], bad[5, 0, 2], bad[6, 2, 100], bad[7, 0, 64:] = float("nan"), float("inf"), float("-inf"), float("inf")
    (code, s, z), (c0, s0, z0) = oq.quantize_rows(bad), oq.quantize_rows(x)
    lost = np.zeros(s.shape, bool)
    lost[3, 1, 1] = lost[5, 0, 0] = lost[6, 2, 1] = lost[7, 0, 1] = True
    with np.errstate(invalid="ignore"):
        held = s[..., None] * (code + z[..., None])
    assert not np.isfinite(held[lost]).any() and not np.isfinite(s[lost]).any() and (code[lost] == 0).all()
    assert np.array_equal(code[~lost], c0[~lost]) and np.array_equal(s[~lost], s0[~lost])
    assert np.array_equal(z[~lost], z0[~lost])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset", [0, 30, 300, 1000])
def test_groups_far_from_zero_lose_what_the_rounding_shifts(dtype, offset):
    """Within u (15 + |z|) steps more than half a step (and the arithmetic's 2^-22 of |x / s| and |z|); bf16 groups far
    from zero do lose more than half a step at their ends, so the half step alone is no bound."""
    g = torch.Generator().manual_seed(offset)
    x = (offset + 3 * torch.randn(500, 1, 64, generator=g).clamp(-3, 3)).to(dtype)
    code, s, z = oq.quantize_rows(x)
    err, bound = _errors(x, s[..., None].astype(np.float64) * (code + z[..., None].astype(np.float64)), s, z)
    assert (err <= bound).all()
    if dtype == torch.bfloat16 and offset >= 300:
        assert (err > 0.6 * s[..., None]).any()
