"""Refusals of the INT4 cache calls, on the CPU: the C entries' status codes on addresses that are never used, and
the Python binding's messages with the device calls trapped (valid arguments stop at the device check only)."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_330_b200 as pa

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, -1, -2, -3, -4
FAKE, OFF8, NULL = 0x10000, 0x10008, None  # an aligned address, one 8 bytes further, none: never dereferenced


# ------------------------------------------------------------------------------------------ C entries
def _write(k=FAKE, v=FAKE, slots=FAKE, T=4, kc=FAKE, vc=FAKE, kp=FAKE, vp=FAKE, ko=NULL, vo=NULL, NB=8, bs=16, Hkv=2,
           D=128, dt=1):
    return pa.lib.pa_write_kv_int4(k, v, slots, T, kc, vc, kp, vp, ko, vo, NB, bs, Hkv, D, dt, NULL)


def _rope(q=FAKE, qo=FAKE, k=FAKE, v=FAKE, pos=FAKE, cos=FAKE, sin=FAKE, maxp=64, slots=FAKE, T=4, Hq=4, kc=FAKE,
          ko=NULL, NB=8, bs=16, Hkv=2, D=128, dt=1):
    return pa.lib.pa_rope_write_kv_int4(q, qo, k, v, pos, cos, sin, maxp, slots, T, Hq, kc, FAKE, FAKE, FAKE, ko, NULL,
                                        NB, bs, Hkv, D, dt, NULL)


def _decode(q=FAKE, kc=FAKE, kp=FAKE, bt=FAKE, mb=8, lens=FAKE, B=2, Hq=4, Hkv=2, D=128, bs=16, NB=16, maxL=100, dt=1,
            ws=FAKE, wsb=1 << 24, parts=0, out=FAKE, lse=NULL):
    return pa.lib.pa_decode_int4(q, kc, FAKE, kp, FAKE, bt, mb, lens, B, Hq, Hkv, D, bs, NB, maxL, 0.1, dt, ws, wsb,
                                 parts, out, lse, NULL)


def test_write_int4_refusals():
    assert _write(T=0) == OK
    assert _write(T=0, kc=NULL) == INVALID
    for bad in (dict(k=NULL), dict(v=NULL), dict(slots=NULL), dict(kc=NULL), dict(vp=NULL), dict(T=-1), dict(NB=-1),
                dict(Hkv=0), dict(D=0)):
        assert _write(**bad) == INVALID, bad
    for bad in (dict(D=96), dict(D=256), dict(bs=8), dict(bs=24), dict(dt=2), dict(dt=-1), dict(T=1 << 30),
                dict(Hkv=1 << 18, bs=256)):
        assert _write(**bad) == UNSUPPORTED, bad
    for bad in (dict(k=OFF8), dict(vc=OFF8), dict(kp=OFF8), dict(ko=OFF8), dict(vo=OFF8), dict(slots=FAKE + 4)):
        assert _write(**bad) == ALIGN, bad


def test_rope_write_int4_refusals():
    assert _rope(T=0) == OK
    for bad in (dict(q=NULL), dict(qo=NULL), dict(pos=NULL), dict(cos=NULL), dict(maxp=0), dict(Hq=0), dict(T=-1)):
        assert _rope(**bad) == INVALID, bad
    for bad in (dict(D=32), dict(bs=512), dict(dt=5), dict(T=1 << 27)):
        assert _rope(**bad) == UNSUPPORTED, bad
    for bad in (dict(q=OFF8), dict(qo=OFF8), dict(cos=OFF8), dict(sin=OFF8), dict(pos=FAKE + 4), dict(kc=OFF8),
                dict(ko=OFF8)):
        assert _rope(**bad) == ALIGN, bad


def test_copy_and_load_int4_refusals():
    def copy(pairs=FAKE, n=3, kc=FAKE, NB=8, bs=16, D=64):
        return pa.lib.pa_copy_blocks_int4(pairs, n, kc, FAKE, FAKE, FAKE, NB, bs, 2, D, NULL)

    def load(pairs=FAKE, n=3, kc=FAKE, NB=8, k=FAKE, v=FAKE, NB2=8, bs=16, D=64, dt=0):
        return pa.lib.pa_load_blocks_int4(pairs, n, kc, FAKE, FAKE, FAKE, NB, k, v, NB2, bs, 2, D, dt, NULL)

    for fn in (copy, load):
        assert fn(n=0) == OK
        assert fn(n=-1) == fn(pairs=NULL) == fn(kc=NULL) == fn(NB=-1) == INVALID
        assert fn(bs=20) == fn(D=72) == UNSUPPORTED
        assert fn(pairs=FAKE + 2) == fn(kc=OFF8) == ALIGN
    assert load(k=NULL) == load(NB2=-1) == INVALID
    assert load(dt=3) == UNSUPPORTED
    assert load(v=OFF8) == ALIGN


def test_decode_int4_refusals():
    assert _decode(B=0) == OK
    for bad in (dict(q=NULL), dict(kc=NULL), dict(kp=NULL), dict(bt=NULL), dict(lens=NULL), dict(out=NULL), dict(B=-1),
                dict(Hq=5), dict(maxL=-1), dict(parts=-1), dict(mb=4), dict(NB=0)):
        assert _decode(**bad) == INVALID, bad
    for bad in (dict(D=80), dict(bs=8), dict(dt=2), dict(Hq=6), dict(Hq=64), dict(NB=1 << 27), dict(mb=1 << 27)):
        assert _decode(**bad) == UNSUPPORTED, bad
    for bad in (dict(q=OFF8), dict(kc=OFF8), dict(kp=OFF8), dict(out=OFF8), dict(bt=FAKE + 2), dict(lse=FAKE + 2),
                dict(ws=FAKE + 16)):
        assert _decode(**bad) == ALIGN, bad
    assert _decode(ws=NULL) == _decode(wsb=64) == WORKSPACE


def test_decode_int4_plan():
    for B, Hq, Hkv, D, L in ((4, 4, 4, 64, 64), (128, 16, 8, 128, 1024), (64, 64, 8, 128, 8192), (1, 32, 2, 128, 100001)):
        grid, pieces, ws = pa.decode_int4_plan(B, Hq, Hkv, D, L)
        assert 1 <= grid and pieces == B * Hkv + grid
        assert ws >= 3 * 4 * 1024 + pieces * (Hq // Hkv) * (D + 2) * 4
        assert pa.lib.pa_decode_int4_workspace_size(B, Hq, Hkv, D, L, 0) == ws
    assert pa.decode_int4_plan(4, 8, 2, 128, 1000, num_partitions=7)[0] == 7
    assert pa.decode_int4_plan(4, 8, 2, 128, 1000, num_partitions=1 << 30) == pa.decode_int4_plan(
        4, 8, 2, 128, 1000, num_partitions=1024)
    # a small batch's grid is a multiple of its segments: contexts of one length are cut where CTAs meet, or not at all
    assert pa.decode_int4_plan(1, 16, 8, 128, 300)[0] % 8 == 0
    for bad in ((4, 8, 2, 96, 100), (4, 6, 4, 128, 100), (4, 64, 2, 128, 100), (-1, 8, 2, 128, 100), (4, 8, 2, 128, -1)):
        assert pa.lib.pa_decode_int4_workspace_size(*bad, 0) == 0
        with pytest.raises(pa.PagedAttnError):
            pa.decode_int4_plan(*bad)


# ------------------------------------------------------------------------------------------ Python binding
DEVICE_MSG = "device calls take CUDA tensors"


@pytest.fixture
def trapped():
    """The native half of the binding bound to entries that only note that they were reached."""
    reached = []
    note = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: reached.append(1) or 0)
    native = pa._native()
    native.bind(*[ctypes.cast(note, ctypes.c_void_p).value] * 5)
    yield
    native.bind(*(ctypes.cast(getattr(pa.lib, f), ctypes.c_void_p).value for f in pa._NATIVE_ENTRIES))
    assert not reached


def _raises(msg, fn, *a, **kw):
    with pytest.raises(ValueError, match=msg):
        fn(*a, **kw)


def _cache(NB=6, Hkv=2, bs=16, D=128, dt=torch.bfloat16):
    c, p = torch.zeros(NB, Hkv, bs, D // 2, dtype=torch.uint8), torch.zeros(NB, Hkv, bs, D // 64, 2, dtype=dt)
    return [c, c.clone(), p, p.clone()]


def _rows(T=5, H=2, D=128, dt=torch.bfloat16):
    return torch.zeros(T, H, D, dtype=dt)


def _bad_caches(call):
    """call(cache): every kind of wrong cache is named."""
    for i, x, msg in ((0, lambda t: t.to(torch.int8), "k_codes must be torch.uint8"),
                      (1, lambda t: t[:3].contiguous(), "v_codes must have shape"),
                      (2, lambda t: t.float(), "unsupported dtype"),
                      (2, lambda t: t[:, :, :, :1].contiguous(), "k_params must have shape"),
                      (3, lambda t: t.half(), "v_params must be"),
                      (3, lambda t: t[:, :1].contiguous(), "v_params must have shape"),
                      (0, lambda t: t.transpose(1, 2), "contiguous")):
        c = _cache()
        c[i] = x(c[i])
        _raises(msg, call, c)


def test_write_int4_binding(trapped):
    k, v, slots = _rows(), _rows(), torch.zeros(5, dtype=torch.int64)
    _raises(DEVICE_MSG, pa.write_kv_int4, k, v, slots, *_cache())
    _raises(DEVICE_MSG, pa.write_kv_int4, k, v, slots, *_cache(), k_out=k, v_out=v)
    _bad_caches(lambda c: pa.write_kv_int4(k, v, slots, *c))
    c = _cache()
    _raises("k must be", pa.write_kv_int4, k.half(), v, slots, *c)
    _raises("v must have shape", pa.write_kv_int4, k, v[:, :1].contiguous(), slots, *c)
    _raises("k must have shape", pa.write_kv_int4, torch.tensor(1.0, dtype=torch.bfloat16), v, slots, *c)
    _raises("slot_mapping must be torch.int64", pa.write_kv_int4, k, v, slots.int(), *c)
    _raises("slot_mapping must have shape", pa.write_kv_int4, k, v, slots[:4], *c)
    _raises("k_out must be", pa.write_kv_int4, k, v, slots, *c, k_out=k.float())
    _raises("v_out must have shape", pa.write_kv_int4, k, v, slots, *c, v_out=v[:4])
    _raises("contiguous", pa.write_kv_int4, k.transpose(0, 1), v, slots, *c)


def test_rope_write_int4_binding(trapped):
    q, k, v = _rows(H=4), _rows(), _rows()
    pos = slots = torch.zeros(5, dtype=torch.int64)
    cos = sin = torch.zeros(32, 64)
    good = (q, k, v, pos, cos, sin, slots)
    _raises(DEVICE_MSG, pa.rope_write_kv_int4, *good, *_cache())
    _raises(DEVICE_MSG, pa.rope_write_kv_int4, *good, *_cache(), q_out=q, k_out=k, v_out=v)
    _bad_caches(lambda c: pa.rope_write_kv_int4(*good, *c))
    c = _cache()
    _raises("q must be", pa.rope_write_kv_int4, q.half(), *good[1:], *c)
    _raises("q must have shape", pa.rope_write_kv_int4, q[:, :, :64].contiguous(), *good[1:], *c)
    _raises("k must have shape", pa.rope_write_kv_int4, q, k[:4], *good[2:], *c)
    _raises("positions must be torch.int64", pa.rope_write_kv_int4, q, k, v, pos.int(), cos, sin, slots, *c)
    _raises("cos_table must be", pa.rope_write_kv_int4, q, k, v, pos, cos.double(), sin, slots, *c)
    _raises("cos_table must have shape", pa.rope_write_kv_int4, q, k, v, pos, cos[:, :32].contiguous(), sin, slots, *c)
    _raises("sin_table must have shape", pa.rope_write_kv_int4, q, k, v, pos, cos, sin[:9], slots, *c)
    _raises("q_out must have shape", pa.rope_write_kv_int4, *good, *c, q_out=q[:3])


def test_copy_and_load_int4_binding(trapped):
    pairs = torch.zeros(2, 2, dtype=torch.int32)
    k16 = torch.zeros(3, 16, 2, 128, dtype=torch.bfloat16)
    _raises(DEVICE_MSG, pa.copy_blocks_int4, pairs, *_cache())
    _raises(DEVICE_MSG, pa.load_blocks_int4, pairs, *_cache(), k16, k16.clone())
    _bad_caches(lambda c: pa.copy_blocks_int4(pairs, *c))
    _bad_caches(lambda c: pa.load_blocks_int4(pairs, *c, k16, k16.clone()))
    c = _cache()
    for fn, more in ((pa.copy_blocks_int4, ()), (pa.load_blocks_int4, (k16, k16.clone()))):
        _raises("pairs must be torch.int32", fn, pairs.long(), *c, *more)
        _raises("pairs must have shape", fn, torch.zeros(2, 3, dtype=torch.int32), *c, *more)
        _raises("pairs must have 2 dimensions", fn, pairs[0], *c, *more)
    _raises("k_cache must be", pa.load_blocks_int4, pairs, *c, k16.half(), k16.half())
    _raises("k_cache must have shape", pa.load_blocks_int4, pairs, *c, k16[:, :8].contiguous(), k16[:, :8].contiguous())
    _raises("v_cache must have shape", pa.load_blocks_int4, pairs, *c, k16, k16[:2])


def test_decode_int4_binding(trapped):
    q, bt, lens = _rows(T=3, H=8), torch.zeros(3, 4, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    _raises(DEVICE_MSG, pa.decode_int4, q, *_cache(), bt, lens, 64, 0.1)
    _raises(DEVICE_MSG, pa.decode_int4, q, *_cache(), bt, lens, 64, 0.1, out=q.clone(), lse=torch.zeros(3, 8),
            workspace=torch.zeros(4096, dtype=torch.uint8))
    _bad_caches(lambda c: pa.decode_int4(q, *c, bt, lens, 64, 0.1))
    c = _cache()
    _raises("q must be", pa.decode_int4, q.half(), *c, bt, lens, 64, 0.1)
    _raises("q must have shape", pa.decode_int4, q[:, :, :64].contiguous(), *c, bt, lens, 64, 0.1)
    _raises("block_tables must be torch.int32", pa.decode_int4, q, *c, bt.long(), lens, 64, 0.1)
    _raises("block_tables must have shape", pa.decode_int4, q, *c, bt[:2], lens, 64, 0.1)
    _raises("context_lens must be torch.int32", pa.decode_int4, q, *c, bt, lens.long(), 64, 0.1)
    _raises("context_lens must have shape", pa.decode_int4, q, *c, bt, lens[:2], 64, 0.1)
    _raises("out must have shape", pa.decode_int4, q, *c, bt, lens, 64, 0.1, out=q[:2])
    _raises("lse must be torch.float32", pa.decode_int4, q, *c, bt, lens, 64, 0.1, lse=torch.zeros(3, 8).double())
    _raises("lse must have shape", pa.decode_int4, q, *c, bt, lens, 64, 0.1, lse=torch.zeros(3, 4))


def test_wrong_kinds_reach_no_library_call(trapped):
    """Arrays, numbers, None, sparse tensors and numbers out of range: a Python error, no call and no crash."""
    q, bt, lens = _rows(T=1, H=2), torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    errors = (AttributeError, TypeError, ValueError, RuntimeError)
    for x in (np.zeros((1, 2, 128)), 3, None, "q", q.to_sparse()):
        with pytest.raises(errors):
            pa.decode_int4(x, *_cache(), bt, lens, 16, 0.1)
        with pytest.raises(errors):
            pa.write_kv_int4(q, x, torch.zeros(1, dtype=torch.int64), *_cache())
        with pytest.raises(errors):
            pa.decode_int4(q, x, *_cache()[1:], bt, lens, 16, 0.1)
    for bad in (dict(max_context_len=1 << 40), dict(max_context_len="16"), dict(scale="x"), dict(num_partitions=1.5)):
        with pytest.raises(errors):
            pa.decode_int4(q, *_cache(), bt, lens, **{"max_context_len": 16, "scale": 0.1, **bad})
    for n in range(3):
        assert pa._native().write_kv_int4(*[q] * n) == pa._WRONG
