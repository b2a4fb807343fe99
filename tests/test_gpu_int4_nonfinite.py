"""NaN and infinities in the INT4 cache: what they reach stays visible, what they do not reach stays right."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv_int4 as oq
from tests.int4_common import DT, assert_within, empty_cache, quantized_pool, reference, to_device
from workloads import make_custom, make_rope_case

pytestmark = pytest.mark.gpu

pa = pytest.importorskip("paged_kv_cache_330_b200")

NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert pa.device_error() == 0, "a kernel recorded a device-side error"


# ------------------------------------------------------------------------------------------ writes
def _spoil(x):
    """A NaN, infinities, both, a whole group of either, in groups of x [T, H, D]; returns which groups [T, H, D/64]."""
    T, H, D = x.shape
    n = D // 64
    lost = torch.zeros(T, H, n, dtype=torch.bool)
    kinds = [lambda v: v[17:18].fill_(NAN), lambda v: v[63:].fill_(INF), lambda v: v[:1].fill_(-INF),
             lambda v: (v[3:4].fill_(INF), v[40:41].fill_(-INF)), lambda v: (v[0:1].fill_(NAN), v[9:10].fill_(INF)),
             lambda v: v.fill_(NAN), lambda v: v.fill_(INF), lambda v: v.fill_(-INF),
             lambda v: (v.fill_(0.5), v[31:32].fill_(NAN)), lambda v: (v.zero_(), v[31:32].fill_(NAN))]
    for i, kind in enumerate(kinds):
        t, h, grp = 1 + i, i % H, i % n
        kind(x[t, h, 64 * grp : 64 * grp + 64])
        lost[t, h, grp] = True
    return lost


def _check_written(x, lost, out, codes, params, slots, bs):
    """Groups with a NaN or an infinity come back as nothing finite, in the rows handed back and in the parameters;
    the others are the oracle's, bit for bit."""
    code, s, z = oq.quantize_rows(x)
    with np.errstate(invalid="ignore"):
        held = (s[..., None] * (code.astype(np.float32) + z[..., None])).reshape(x.shape)
    wide = lost.repeat_interleave(64, dim=-1)
    got = out.cpu()
    assert not torch.isfinite(got[wide]).any()
    assert torch.equal(got[~wide], torch.from_numpy(held).to(x.dtype)[~wide])
    blk, row = slots // bs, slots % bs
    par = params.cpu()[blk, :, row].float()  # [T, H, n, 2]
    assert not torch.isfinite(par[..., 0][lost]).any()
    ref = torch.from_numpy(np.stack([s, z], -1))
    assert torch.equal(par[~lost], ref[~lost])
    assert torch.equal(torch.isnan(par), torch.isnan(ref))
    assert np.array_equal(codes.cpu()[blk, :, row].numpy(), oq.pack(code))


@pytest.mark.parametrize("D,dt", [(64, "f16"), (64, "bf16"), (128, "f16"), (128, "bf16")])
def test_write_int4_spoils_the_group_of_a_nan_or_infinity(D, dt):
    g = torch.Generator().manual_seed(D)
    T, H, bs = 21, 3, 16
    k, v = (torch.randn(T, H, D, generator=g).to(DT[dt]) for _ in "kv")
    lost_k = _spoil(k)
    lost_v = torch.zeros_like(lost_k)
    v[20, 2, 5], lost_v[20, 2, 0] = NAN, True
    slots = torch.randperm(32, generator=g)[:T]
    cache = empty_cache(2, H, bs, D, DT[dt])
    ko, vo = torch.zeros_like(k).cuda(), torch.zeros_like(v).cuda()
    pa.write_kv_int4(k.cuda(), v.cuda(), slots.cuda(), *cache, k_out=ko, v_out=vo)
    _check_written(k, lost_k, ko, cache[0], cache[2], slots, bs)
    _check_written(v, lost_v, vo, cache[1], cache[3], slots, bs)
    k16 = torch.zeros(2, bs, H, D, dtype=DT[dt], device="cuda")  # and expanded
    v16 = torch.zeros_like(k16)
    pa.load_blocks_int4(torch.tensor([[0, 0], [1, 1]], dtype=torch.int32, device="cuda"), *cache, k16, v16)
    for got, want in ((k16, ko), (v16, vo)):
        rows = got.view(-1, H, D)[slots.cuda()]
        assert torch.equal(torch.isfinite(rows), torch.isfinite(want))
        assert torch.equal(rows[torch.isfinite(rows)], want[torch.isfinite(want)])


@pytest.mark.parametrize("D,dt", [(64, "bf16"), (128, "f16")])
def test_rope_write_int4_spoils_the_groups_of_a_turned_nan(D, dt):
    """A NaN in a key turns into two (elements i and i + D/2), at D 128 in both groups; q rows keep theirs to themselves."""
    rc = make_rope_case(seed=D, num_tokens=9, num_q_heads=4, num_kv_heads=2, head_dim=D, block_size=16, num_blocks=1,
                        dtype=dt, max_position=64, skip_frac=0.0)
    slots = torch.arange(9)
    rc.k[3, 1, 7] = NAN
    rc.q[5, 2, 9] = NAN
    cache = empty_cache(1, 2, 16, D, DT[dt])
    ko = torch.zeros_like(rc.k).cuda()
    args = [x.cuda() for x in (rc.q, rc.k, rc.v, rc.positions, rc.cos, rc.sin, slots)]
    q_out = pa.rope_write_kv_int4(*args, *cache, k_out=ko)
    bad = torch.isnan(ko).cpu()
    assert bad[3, 1].all() and int(bad.sum()) == D and not torch.isinf(ko).any()
    assert int(torch.isnan(q_out).sum()) == 2 and torch.isnan(q_out[5, 2]).sum() == 2


# ------------------------------------------------------------------------------------------ decode
def _pool(wl):
    _, bt, lens, _, _ = pa.replay_ops(wl.ops, wl.num_blocks, wl.cfg["block_size"], wl.free_order, wl.batch)
    (kc, kp), (vc, vp) = quantized_pool(wl.k_cache0), quantized_pool(wl.v_cache0)
    return [kc, vc, kp, vp], bt, lens


LENS = [3000, 1, 40, 20000, 700]  # within a warp, between the warps of a CTA, between CTAs by one and by two rounds


def _workload(Hq, Hkv, D, dt, q_scale=1.0):
    return make_custom(seed=7 + D, lens=LENS, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, block_size=32, dtype=dt,
                       q_scale=q_scale)


@pytest.mark.parametrize("Hq,Hkv,D,dt", [(8, 2, 128, "bf16"), (16, 1, 64, "f16"), (2, 2, 128, "f16")])
def test_decode_int4_nan_in_a_key_reaches_its_heads(Hq, Hkv, D, dt):
    """One key's NaN among thousands: softmax over a NaN score is NaN, wherever the segment is cut; other KV heads and
    sequences keep their results."""
    wl = _workload(Hq, Hkv, D, dt)
    host, bt, lens = _pool(wl)
    rows, out, lse, bound, lse_bound = reference(wl.q, *host, bt, lens, wl.scale)
    G = Hq // Hkv
    bad = {(0, 0): 1700, (2, 0): 39, (3, Hkv - 1): 12345, (4, 0): 0}  # (sequence, KV head): token
    for (b, kvh), t in bad.items():
        host[2][bt[b][t // 32], kvh, t % 32, 0, 0] = NAN
    cache = to_device(*host, wl.q.dtype)
    lost = np.array([(b, h // G) in bad for b, h in rows])
    for ns in (0, 1, 7, 300):
        got_lse = torch.zeros(len(LENS), Hq, device="cuda")
        got = pa.decode_int4(wl.q.cuda(), *cache, torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda(), max(LENS),
                             wl.scale, lse=got_lse, num_partitions=ns)
        at = np.asarray(rows)
        o, l = (x.double().cpu().numpy()[at[:, 0], at[:, 1]] for x in (got, got_lse))
        assert np.isnan(o[lost]).all() and np.isnan(l[lost]).all(), ns
        assert_within(o[~lost], out[~lost], bound[~lost], f"beside a NaN key, partitions {ns}")
        assert_within(l[~lost], lse[~lost], lse_bound[~lost], f"beside a NaN key, partitions {ns}, lse")


@pytest.mark.parametrize("q_scale", [1.0, 30.0])
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("Hq,Hkv,dt", [(8, 2, "bf16"), (16, 1, "f16"), (2, 2, "f16")])
def test_decode_int4_nonfinite_value_reaches_its_group_alone(Hq, Hkv, dt, value, q_scale):
    """One value row's NaN or infinity (as the writes store a group with one: scale, or scale and zero point, not
    finite) takes its 64 columns; the other 64 of the head, the log-sum-exp and all else stay within the bounds."""
    D = 128
    wl = _workload(Hq, Hkv, D, dt, q_scale)
    host, bt, lens = _pool(wl)
    rows, out, lse, bound, lse_bound = reference(wl.q, *host, bt, lens, wl.scale)
    G = Hq // Hkv
    bad = {(0, 0): (1700, 1), (2, 0): (39, 0), (3, Hkv - 1): (12345, 0), (4, 0): (0, 1)}  # (token, group)
    for (b, kvh), (t, grp) in bad.items():
        host[3][bt[b][t // 32], kvh, t % 32, grp, 0] = value
        host[3][bt[b][t // 32], kvh, t % 32, grp, 1] = 0.0 if value == INF else NAN
        if value == INF:
            host[1][bt[b][t // 32], kvh, t % 32] = 0
    cache = to_device(*host, wl.q.dtype)
    lost = np.zeros(out.shape, dtype=bool)
    other = np.zeros(out.shape, dtype=bool)  # the spoilt row's other group: its codes were changed (an infinity's case)
    for i, (b, h) in enumerate(rows):
        if (b, h // G) in bad:
            grp = bad[b, h // G][1]
            lost[i, 64 * grp : 64 * grp + 64] = True
            other[i, 64 * (1 - grp) : 64 * (1 - grp) + 64] = True
    if value == INF:  # the reference of the other group, with the codes as they are now
        fine = [x.copy() for x in host]
        fine[3][~np.isfinite(fine[3])] = 0.0
        _, out2, _, bound2, _ = reference(wl.q, *fine, bt, lens, wl.scale)
        out, bound = np.where(other, out2, out), np.where(other, bound2, bound)
    for ns in (0, 1, 7, 300):
        got_lse = torch.zeros(len(LENS), Hq, device="cuda")
        got = pa.decode_int4(wl.q.cuda(), *cache, torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda(), max(LENS),
                             wl.scale, lse=got_lse, num_partitions=ns)
        at = np.asarray(rows)
        o, l = (x.double().cpu().numpy()[at[:, 0], at[:, 1]] for x in (got, got_lse))
        assert not np.isfinite(o[lost]).any(), ns
        assert_within(o[~lost], out[~lost], bound[~lost], f"beside {value} in V, partitions {ns}")
        assert_within(l, lse, lse_bound, f"beside {value} in V, partitions {ns}, lse")
