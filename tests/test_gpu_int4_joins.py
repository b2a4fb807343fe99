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


# ------------------------------------------------------------------------------------------ graphs, streams, workspaces
CUT = [20000, 40, 9000]  # one KV head: 3 segments, the long ones cut between CTAs, the first by more than 16


def _cut_case(seed):
    q, cache, tables, ln, top = _context(CUT, 8, 1, 128, 16, torch.bfloat16, seed)
    need = pa.decode_int4_plan(len(CUT), 8, 1, 128, top)[2]
    return q, cache, tables, ln, top, 128 ** -0.5, lambda: torch.zeros(need, dtype=torch.uint8, device="cuda")


def _slots(tables, ln, bs):
    """The slot of every sequence's last token."""
    t = (ln - 1).long()
    return tables.gather(1, (t // bs)[:, None])[:, 0].long() * bs + t % bs


def test_decode_int4_cut_segments_in_two_graphs():
    """Write and decode of segments cut between CTAs, captured three times over in each of two graphs with a cache and a
    workspace of its own, replayed in turn and then side by side: the eager calls' bits, all counters at zero at the end, and shares
    in the workspaces."""
    q, cache, tables, ln, top, scale, ws_of = _cut_case(5)
    g = torch.Generator(device="cuda").manual_seed(6)
    kn, vn = (torch.randn(3, 1, 128, generator=g, device="cuda").to(q.dtype) for _ in "kv")
    slots = _slots(tables, ln, 16)
    side = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for s in side:
        ws, out, mine = ws_of(), torch.empty_like(q), [x.clone() for x in cache]
        pa.write_kv_int4(kn, vn, slots, *mine)
        pa.decode_int4(q, *mine, tables, ln, top, scale, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(3):
                pa.write_kv_int4(kn, vn, slots, *mine)
                pa.decode_int4(q, *mine, tables, ln, top, scale, out=out, workspace=ws)
        graphs.append((graph, ws, out, mine))
    for i in range(6):
        q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        kn.copy_(torch.randn(kn.shape, generator=g, device="cuda"))
        pa.write_kv_int4(kn, vn, slots, *cache)
        want = pa.decode_int4(q, *cache, tables, ln, top, scale, workspace=ws_of())
        for _, _, out, _ in graphs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        if i < 4:
            graphs[i % 2][0].replay()
        else:  # both at once
            for s, (graph, *_) in zip(side, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for j, (_, ws, out, _) in enumerate(graphs):
            if i >= 4 or j == i % 2:
                assert torch.equal(out, want), (i, j)
            assert not ws[:COUNTERS].any() and ws[COUNTERS:].any()


def test_decode_int4_cut_segments_on_two_streams():
    """Two decodes of different q at once, each with a workspace of its own, call after call."""
    q, cache, tables, ln, top, scale, ws_of = _cut_case(8)
    qs = [q, torch.randn(q.shape, device="cuda").to(q.dtype)]
    want = [pa.decode_int4(x, *cache, tables, ln, top, scale, workspace=ws_of()) for x in qs]
    assert not torch.equal(want[0], want[1])
    streams, ws = [torch.cuda.Stream() for _ in qs], [ws_of() for _ in qs]
    outs = [torch.empty(200, *q.shape, dtype=q.dtype, device="cuda") for _ in qs]
    torch.cuda.synchronize()
    for i in range(200):
        for s, x, o, w in zip(streams, qs, outs, ws):
            pa.decode_int4(x, *cache, tables, ln, top, scale, out=o[i], workspace=w, stream=s)
    torch.cuda.synchronize()
    for o, x, w in zip(outs, want, ws):
        assert (o == x).all() and not w[:COUNTERS].any() and w[COUNTERS:].any()


def test_decode_int4_captured_without_a_workspace():
    """A captured call that makes its workspace and its output itself: zero-filled at every replay."""
    q, cache, tables, ln, top, scale, ws_of = _cut_case(9)
    pa.decode_int4(q, *cache, tables, ln, top, scale)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pa.decode_int4(q, *cache, tables, ln, top, scale)
        again = pa.decode_int4(q, *cache, tables, ln, top, scale)
    for _ in range(3):
        q.copy_(torch.randn(q.shape, device="cuda"))
        want = pa.decode_int4(q, *cache, tables, ln, top, scale, workspace=ws_of())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(again, want)


def test_int4_calls_of_nothing():
    """No sequences, no tokens, no pairs: nothing is written, and an empty output comes back."""
    q, cache, tables, ln, top, scale, _ = _cut_case(10)
    before = [x.clone() for x in cache]
    out = pa.decode_int4(q[:0], *cache, tables[:0], ln[:0], top, scale, lse=torch.empty(0, 8, device="cuda"))
    assert out.shape == (0, 8, 128)
    rows, none = torch.empty(0, 1, 128, dtype=q.dtype, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    pa.write_kv_int4(rows, rows, none, *cache, k_out=rows.clone(), v_out=rows.clone())
    table = torch.ones(4, 64, device="cuda")
    assert pa.rope_write_kv_int4(q[:0], rows, rows, none, table, table, none, *cache).shape == (0, 8, 128)
    pairs = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    pa.copy_blocks_int4(pairs, *cache)
    k16 = torch.zeros(2, 16, 1, 128, dtype=q.dtype, device="cuda")
    pa.load_blocks_int4(pairs, *cache, k16, k16.clone())
    assert all(torch.equal(a, b) for a, b in zip(before, cache)) and not k16.any()


def test_int4_blocks_expanded_right_before_a_cascade_reads_them():
    """load_blocks_int4 lets the next kernel begin at its start: the cascade behind it on the stream, of two kernels of
    which the second begins early too, still reads expanded blocks only."""
    D, bs, Hq, Hkv, B, P = 128, 64, 16, 2, 24, 4096
    lens = [P + 17 * b for b in range(B)]
    q, cache, _, ln, top = _context(lens, Hq, Hkv, D, bs, torch.bfloat16, 11)
    held = [-(-n // bs) for n in lens]
    shared = P // bs
    tables = torch.full((B, max(held)), -1, dtype=torch.int32)
    at = shared
    for b, n in enumerate(held):
        tables[b, :shared] = torch.arange(shared)
        tables[b, shared:n] = torch.arange(at, at + n - shared)
        at += n - shared
    tables = tables.cuda()
    pairs = torch.arange(at, dtype=torch.int32, device="cuda")[:, None].expand(-1, 2).contiguous()
    k16 = torch.empty(at, bs, Hkv, D, dtype=q.dtype, device="cuda")
    v16 = torch.empty_like(k16)
    groups = torch.tensor([0, B], dtype=torch.int32, device="cuda")
    prefix = torch.full((B,), P, dtype=torch.int32, device="cuda")
    scale = D ** -0.5

    def cascade():
        return pa.decode_cascade(q, k16, v16, tables, ln, top, scale, groups, prefix, B, P)

    pa.load_blocks_int4(pairs, *cache, k16, v16)
    torch.cuda.synchronize()
    want = cascade()
    for _ in range(20):
        k16.fill_(float("nan"))
        v16.fill_(float("nan"))
        pa.load_blocks_int4(pairs, *cache, k16, v16)
        assert torch.equal(cascade(), want)
