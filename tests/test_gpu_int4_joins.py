"""decode_int4 where segments are cut between CTAs: unequal long sequences, call after call."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.int4_common import DT, assert_within, reference

pytestmark = pytest.mark.gpu

pa = pytest.importorskip("paged_kv_cache_330_b200")

COUNTERS = 3 * 1024 * 4  # bytes of the counters, at the head of a workspace


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert pa.device_error() == 0, "a kernel recorded a device-side error"


def _context(lens, Hq, Hkv, D, bs, dtype, seed):
    """A used cache on the device with the lengths' blocks in random order: (q, cache, tables, lens, longest)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    held = [-(-n // bs) for n in lens]
    NB = sum(held) + 3
    order = torch.randperm(NB, generator=g, device="cuda").to(torch.int32)
    tables = torch.full((len(lens), max(1, max(held))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(held):
        tables[b, :n] = order[at : at + n]
        at += n
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    codes = [torch.randint(0, 256, (NB, Hkv, bs, D // 2), generator=g, device="cuda", dtype=torch.uint8) for _ in "kv"]
    par = [torch.stack([0.3 * torch.exp(0.3 * randn(NB, Hkv, bs, D // 64)), -7.5 + 1.5 * randn(NB, Hkv, bs, D // 64)],
                       dim=-1).to(dtype) for _ in "kv"]
    return (randn(len(lens), Hq, D).to(dtype), (*codes, *par), tables,
            torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens))


def _reference(q, cache, tables, lens, scale, rows):
    host = [x.cpu().numpy() if x.dtype == torch.uint8 else x.float().cpu().numpy() for x in cache]
    return reference(q.cpu(), *host, tables.cpu().numpy(), lens.cpu().numpy(), scale, rows)


def _check(got, lse, ref, what):
    rows, out, ref_lse, bound, lse_bound = ref
    at = np.asarray(rows)
    assert_within(got.double().cpu().numpy()[at[:, 0], at[:, 1]], out, bound, what)
    assert_within(lse.double().cpu().numpy()[at[:, 0], at[:, 1]], ref_lse, lse_bound, what + " lse")


@pytest.mark.parametrize("lens,Hq,Hkv,D,dtype", [
    ([32000, 16000], 16, 2, 128, "bf16"), ([100000, 3000], 16, 8, 128, "bf16"), ([64000, 1000], 8, 1, 128, "f16"),
    ([50000, 20000], 16, 1, 128, "f16"), ([8193, 30, 30], 16, 2, 64, "bf16")])
def test_decode_int4_unequal_long_sequences_call_after_call(lens, Hq, Hkv, D, dtype):
    """A CTA that ends one long segment and begins another may be the last of both to be counted, or of one, or of
    none: the order in which CTAs finish decides, so every one of many calls has to give the same bits, within the
    bounds, and to leave all counters at zero."""
    q, cache, tables, ln, top = _context(lens, Hq, Hkv, D, 64, DT[dtype], sum(lens))
    scale = D ** -0.5
    ws = torch.zeros(pa.decode_int4_plan(len(lens), Hq, Hkv, D, top)[2], dtype=torch.uint8, device="cuda")
    lse = torch.empty(len(lens), Hq, device="cuda")
    want = pa.decode_int4(q, *cache, tables, ln, top, scale, lse=lse, workspace=ws)
    assert ws[COUNTERS:].any()  # segments were cut: shares went through the workspace
    rows = [(b, h) for b in range(len(lens)) for h in (0, Hq // 2, Hq - 1)]
    _check(want, lse, _reference(q, cache, tables, ln, scale, rows), f"{lens}")
    lse0 = lse.clone()
    off = torch.zeros((), dtype=torch.int64, device="cuda")
    out = torch.empty_like(q)
    for _ in range(500):
        out.fill_(7.0)
        lse.fill_(7.0)
        pa.decode_int4(q, *cache, tables, ln, top, scale, out=out, lse=lse, workspace=ws)
        off += (out != want).sum() + (lse != lse0).sum()
    assert int(off) == 0
    assert not ws[:COUNTERS].any()
