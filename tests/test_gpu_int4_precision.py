"""How near decode_int4 comes to the result that only the output's rounding keeps from the exact one."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv_int4 as oq
from tests.int4_common import assert_within, quantized_pool, reference, to_device
from workloads import make_custom

pytestmark = pytest.mark.gpu

pa = pytest.importorskip("paged_kv_cache_330_b200")


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert pa.device_error() == 0, "a kernel recorded a device-side error"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (6, 3), (8, 2), (16, 2), (32, 2)])
def test_decode_int4_error_is_the_outputs_rounding(Hq, Hkv, D, dtype):
    """The 2-norm of the error over 64 sequences of 1 to 64 tokens is at most 1.15 times that of the exact result
    rounded to the type.  One fp16 rounding of the softmax weights (half a step 2^-11, as large as that of an fp16
    output, and independent of it) would make it sqrt(2) times; two terms (2^-22) leave: sums of at most 8 steps of
    2^-23 of parts up to (15 + |z|) / |code + z| ~ 20 times the result, 2e-5; products of a code cut at 2^-14 of the
    largest weight in 16, relative to a result of at least that weight times 4 codes, under 16 of them 2e-5 on the
    mean; scores off by 2^-19 of their parts at worst, 2e-5.  Together 4e-5 beside the 2e-4 of an fp16 output's
    rounding (sqrt(1 + 0.04) = 1.02); bf16: one rounding of the weights 2e-4 beside 1.6e-3, 1.01."""
    lens = list(range(1, 65))
    wl = make_custom(seed=Hq * 7 + D, lens=lens, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, block_size=16, dtype=dtype)
    _, bt, ln, _, _ = pa.replay_ops(wl.ops, wl.num_blocks, 16, wl.free_order, wl.batch)
    (kc, kp), (vc, vp) = quantized_pool(wl.k_cache0), quantized_pool(wl.v_cache0)
    cache = to_device(kc, vc, kp, vp, wl.q.dtype)
    _, out, _, _, _ = reference(wl.q, kc, vc, kp, vp, bt, ln, wl.scale, want_bound=False)
    own = np.linalg.norm(torch.from_numpy(out).to(wl.q.dtype).double().numpy() - out)
    for ns in (0, 7):  # whole segments, and some of them cut
        got = pa.decode_int4(wl.q.cuda(), *cache, torch.from_numpy(bt).cuda(), torch.from_numpy(ln).cuda(), 64, wl.scale,
                             num_partitions=ns)
        err = np.linalg.norm(got.double().cpu().numpy().reshape(out.shape) - out)
        assert err <= 1.15 * own, (err / own, own / np.linalg.norm(out))


@pytest.mark.parametrize("D,Hq,Hkv,dtype", [(128, 8, 2, "bf16"), (64, 4, 4, "f16"), (128, 16, 1, "f16"), (64, 8, 4, "bf16")])
def test_decode_int4_small_q_elements_beside_an_outlier_count(D, Hq, Hkv, dtype):
    """One channel of q 2^8 times the others, K alike there for all tokens: what tells the tokens apart is what the
    small elements add.  The matrix unit cuts each of the 16 products of a step at 2^-18 of the largest |q| of the 16, per
    unit of a code: over D / 16 steps, of which one has the outlier, a score moves by at most
    d2 = 16 2^-18 (|outlier| + (D / 16 - 1) m) s scale, m the largest of the other elements and s the sequence's largest
    K scale.  On top of the bounds without outliers: 2 d2 (A + |ref|) for an element, d2 for a log-sum-exp.  Neither
    zeros nor the result that only the outlier decides lie within them."""
    wl = make_custom(seed=13, lens=[700, 33, 1024, 5, 3000], num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D,
                     block_size=16, dtype=dtype)
    wl.q[..., 5] = 2.0 ** 8
    wl.k_cache0[..., 5] = 1.0
    _, bt, lens, _, _ = pa.replay_ops(wl.ops, wl.num_blocks, 16, wl.free_order, wl.batch)
    (kc, kp), (vc, vp) = quantized_pool(wl.k_cache0), quantized_pool(wl.v_cache0)
    rows, out, lse, bound, lse_bound = reference(wl.q, kc, vc, kp, vp, bt, lens, wl.scale)
    only = torch.zeros_like(wl.q)
    only[..., 5] = wl.q[..., 5]
    _, dropped, _, _, _ = reference(only, kc, vc, kp, vp, bt, lens, wl.scale, want_bound=False)
    q = wl.q.double().numpy()
    for i, (b, h) in enumerate(rows):
        L = int(lens[b])
        blk, kvh = np.asarray(bt[b][: -(-L // 16)], dtype=np.int64), h // (Hq // Hkv)
        take = lambda a: a[blk, kvh].reshape(-1, *a.shape[3:])[:L].astype(a.dtype)  # noqa: E731
        k, v = oq.values(take(kc), take(kp)), oq.values(take(vc), take(vp))
        x = (k @ q[b, h]) * wl.scale
        w = np.exp(x - x.max())
        A = (w / w.sum()) @ np.abs(v)
        m = np.abs(np.delete(q[b, h], 5)).max()
        d2 = 16 * 2.0 ** -18 * (abs(q[b, h, 5]) + (D / 16 - 1) * m) * take(kp)[..., 0].max() * wl.scale
        bound[i] += 2 * d2 * (A + np.abs(out[i]))
        lse_bound[i] += d2
    many = np.array([lens[b] > 5 for b, _ in rows])
    for other in (np.zeros_like(out), dropped):
        assert (np.abs(other - out) > bound)[many].mean() > 0.5
    cache = to_device(kc, vc, kp, vp, wl.q.dtype)
    got_lse = torch.empty(len(lens), Hq, device="cuda")
    got = pa.decode_int4(wl.q.cuda(), *cache, torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda(), 3000, wl.scale,
                         lse=got_lse)
    assert_within(got.double().cpu().numpy().reshape(out.shape), out, bound, "outlier in q")
    assert_within(got_lse.double().cpu().numpy().reshape(-1), lse, lse_bound, "outlier in q, lse")


@pytest.mark.parametrize("shift", [8, 14, 20, 27])
@pytest.mark.parametrize("Hq,Hkv,small", [(8, 2, 0), (16, 1, 1), (2, 2, 1)])
def test_decode_int4_groups_of_v_with_scales_far_apart(Hq, Hkv, small, shift):
    """The values of one group 2^shift times smaller than those of the row's other group (bf16).  Both enter with one
    power of two per head, so a weight times its V scale counts down to 2^-28 of the head's largest, T: the columns of the
    small group are off by at most L 2^-28 T (15 + |z|) more than the usual bound.  The other group's columns, and the
    log-sum-exps, keep the usual bounds."""
    D, lens = 128, [700, 33, 1024, 5, 1]
    wl = make_custom(seed=31 + shift, lens=lens, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, block_size=16)
    wl.v_cache0[..., 64 * small : 64 * small + 64] *= 2.0 ** -shift
    _, bt, ln, _, _ = pa.replay_ops(wl.ops, wl.num_blocks, 16, wl.free_order, wl.batch)
    (kc, kp), (vc, vp) = quantized_pool(wl.k_cache0), quantized_pool(wl.v_cache0)
    rows, out, lse, bound, lse_bound = reference(wl.q, kc, vc, kp, vp, bt, ln, wl.scale)
    q = wl.q.double().numpy()
    for i, (b, h) in enumerate(rows):
        L = int(ln[b])
        blk, kvh = np.asarray(bt[b][: -(-L // 16)], dtype=np.int64), h // (Hq // Hkv)
        take = lambda a: a[blk, kvh].reshape(-1, *a.shape[3:])[:L]  # noqa: E731
        x = (oq.values(take(kc), take(kp)) @ q[b, h]) * wl.scale
        w = np.exp(x - x.max()) / np.exp(x - x.max()).sum()
        par = take(vp).astype(np.float64)
        T = (w[:, None] * par[..., 0]).max()
        bound[i, 64 * small : 64 * small + 64] += L * 2.0 ** -28 * T * (15 + np.abs(par[:, small, 1]).max())
    cache = to_device(kc, vc, kp, vp, wl.q.dtype)
    got_lse = torch.empty(len(lens), Hq, device="cuda")
    for ns in (0, 7):
        got = pa.decode_int4(wl.q.cuda(), *cache, torch.from_numpy(bt).cuda(), torch.from_numpy(ln).cuda(), 1024, wl.scale,
                             lse=got_lse, num_partitions=ns)
        assert_within(got.double().cpu().numpy().reshape(out.shape), out, bound, f"groups 2^{shift} apart")
        assert_within(got_lse.double().cpu().numpy().reshape(-1), lse, lse_bound, f"groups 2^{shift} apart, lse")
