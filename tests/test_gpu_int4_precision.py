"""How near decode_int4 comes to the result that only the output's rounding keeps from the exact one."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.int4_common import quantized_pool, reference, to_device
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
