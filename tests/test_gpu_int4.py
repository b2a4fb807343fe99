"""GPU parity of the INT4 KV cache: the quantising writes, the block copy and the expansion bit for bit against
the oracle, decode within bounds that arithmetic gives (tests/int4_common.py)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import kv_int4 as oq
from tests.gpu_common import assert_close
from tests.int4_common import DT, assert_within, empty_cache, quantized_pool, reference, to_device
from workloads import make_custom, make_prefix_groups, make_rope_case, make_workload, rope_tables

pytestmark = pytest.mark.gpu

pa = pytest.importorskip("paged_kv_cache_330_b200")


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert pa.device_error() == 0, "a kernel recorded a device-side error"


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


def _same_params(got, ref_f32, dtype):
    assert torch.equal(got.cpu().view(torch.int16), torch.from_numpy(ref_f32).to(dtype).view(torch.int16))


# ------------------------------------------------------------------------------------------ write
@pytest.mark.parametrize("Hkv,D,dt,bs", [(1, 64, "f16", 16), (8, 128, "bf16", 32), (3, 64, "bf16", 256),
                                         (5, 128, "f16", 64), (2, 128, "bf16", 128)])
@pytest.mark.parametrize("rows_back", [False, True])
def test_write_int4_bit_exact(Hkv, D, dt, bs, rows_back):
    """Codes and parameters bit for bit, untouched rows keep their bytes, slot -1 writes nothing (not k_out
    either), special rows: zeros, a constant, one non-zero value, the largest finite value of both signs, tiny
    values, groups far from zero and groups one unit in the last place wide."""
    dtype = DT[dt]
    g = torch.Generator().manual_seed(Hkv * 1000 + D + bs)
    NB, T = 7, 3 * bs + 5
    k = (torch.randn(T, Hkv, D, generator=g) * torch.exp(torch.randn(T, Hkv, 1, generator=g) * 3)).clamp(-6e4, 6e4)
    v = torch.randn(T, Hkv, D, generator=g)
    big = torch.finfo(dtype).max
    k[0] = 0
    k[1] = 0.75
    k[2] = 0
    k[2, :, D // 3] = -2.5
    k[3, :, 0], k[3, :, 1] = big, -big
    k[4] = 1e-5 if dt == "f16" else 1e-30
    k[5] = 1000.0
    k[5, :, ::3] = 1000.0 * (1 + 2.0 ** -7)
    k[6] = -3.0 + 0.01 * torch.randn(Hkv, D, generator=g)
    k[7] = torch.finfo(dtype).tiny * torch.randint(1, 4, (Hkv, D), generator=g)
    k, v = k.to(dtype), v.to(dtype)
    slots = torch.randperm(NB * bs, generator=g)[:T].to(torch.int64)
    slots[9::5] = -1
    kc0 = np.full((NB, Hkv, bs, D // 2), 0x5A, dtype=np.uint8)
    kp0 = np.full((NB, Hkv, bs, D // 64, 2), -7.25, dtype=np.float32)
    okc, ovc, okp, ovp = kc0.copy(), kc0.copy(), kp0.copy(), kp0.copy()
    kheld = oq.write_kv_int4(k, slots.numpy(), okc, okp)
    vheld = oq.write_kv_int4(v, slots.numpy(), ovc, ovp)
    cache = to_device(kc0, kc0, kp0, kp0, dtype)
    ko = torch.full((T, Hkv, D), 9.0, dtype=dtype, device="cuda") if rows_back else None
    vo = torch.full_like(ko, 9.0) if rows_back else None
    pa.write_kv_int4(k.cuda(), v.cuda(), slots.cuda(), *cache, k_out=ko, v_out=vo)
    assert np.array_equal(cache[0].cpu().numpy(), okc) and np.array_equal(cache[1].cpu().numpy(), ovc)
    _same_params(cache[2], okp, dtype)
    _same_params(cache[3], ovp, dtype)
    if rows_back:
        for got, held in ((ko, kheld), (vo, vheld)):
            want = torch.from_numpy(held).to(dtype)
            want[slots < 0] = 9.0
            assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("T", [1, 2, 3, 31, 129])
def test_write_int4_in_place_rows(T):
    """k_out = k and v_out = v: the rows are replaced by what the cache holds."""
    g = torch.Generator().manual_seed(T)
    k, v = (torch.randn(T, 3, 128, generator=g).to(torch.bfloat16) for _ in range(2))
    slots = torch.randperm(160, generator=g)[:T].to(torch.int64)
    a, b = empty_cache(10, 3, 16, 128, torch.bfloat16), empty_cache(10, 3, 16, 128, torch.bfloat16)
    kd, vd = k.cuda(), v.cuda()
    ko, vo = torch.empty_like(kd), torch.empty_like(vd)
    pa.write_kv_int4(kd, vd, slots.cuda(), *a, k_out=ko, v_out=vo)
    pa.write_kv_int4(kd, vd, slots.cuda(), *b, k_out=kd, v_out=vd)
    assert torch.equal(kd, ko) and torch.equal(vd, vo)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_write_int4_nonfinite_stays_in_its_group():
    """A NaN or an infinity spoils its own group of 64 only."""
    g = torch.Generator().manual_seed(4)
    k = torch.randn(6, 2, 128, generator=g).to(torch.bfloat16)
    bad = k.clone()
    bad[1, 0, 5], bad[2, 1, 100], bad[3, 0, 64] = float("nan"), float("inf"), float("-inf")
    slots = torch.arange(6)
    a, b = empty_cache(1, 2, 16, 128, torch.bfloat16), empty_cache(1, 2, 16, 128, torch.bfloat16)
    oa, ob = torch.zeros_like(k).cuda(), torch.zeros_like(k).cuda()
    pa.write_kv_int4(k.cuda(), k.cuda(), slots.cuda(), *a, k_out=oa)
    pa.write_kv_int4(bad.cuda(), k.cuda(), slots.cuda(), *b, k_out=ob)
    spoilt = torch.zeros(6, 2, 2, dtype=torch.bool)
    spoilt[1, 0, 0] = spoilt[2, 1, 1] = spoilt[3, 0, 1] = True
    fine = ~spoilt.repeat_interleave(64, dim=-1)
    assert torch.equal(oa.cpu()[fine], ob.cpu()[fine])


def test_write_int4_slot_out_of_range_sets_index_bit():
    k = torch.ones(2, 1, 64, dtype=torch.float16, device="cuda")
    cache = empty_cache(2, 1, 16, 64, torch.float16)
    pa.write_kv_int4(k, k, torch.tensor([32, 31], device="cuda"), *cache)
    assert pa.device_error() == 2
    assert (cache[2][1, 0, 15] != 0).any() and (cache[2].flatten()[:-2] == 0).all()


# ------------------------------------------------------------------------------------------ rotary + write
@pytest.mark.parametrize("T,Hq,Hkv,D,bs,dt", [(1, 4, 4, 64, 16, "f16"), (33, 12, 3, 64, 64, "bf16"),
                                              (130, 16, 8, 128, 16, "bf16"), (65, 20, 5, 128, 32, "f16"),
                                              (7, 16, 1, 128, 256, "bf16")])
def test_rope_write_int4_is_rope_then_write(T, Hq, Hkv, D, bs, dt):
    """Bit for bit the two calls it fuses: rope_write_kv into a 16-bit cache, its k rows through write_kv_int4."""
    NB = -(-T // bs) + 3
    rc = make_rope_case(seed=T + D, num_tokens=T, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, block_size=bs,
                        num_blocks=NB, dtype=dt, max_position=777, skip_frac=0.2, random_angles=True)
    dtype = DT[dt]
    dev = lambda x: x.cuda()  # noqa: E731
    every = torch.arange(T)  # the turned keys of every token, also of those without a slot
    NB2 = -(-T // bs)
    k16, v16 = (torch.zeros(NB2, bs, Hkv, D, dtype=dtype, device="cuda") for _ in range(2))
    q_ref = pa.rope_write_kv(dev(rc.q), dev(rc.k), dev(rc.v), dev(rc.positions), dev(rc.cos), dev(rc.sin),
                             dev(every), k16, v16)
    turned = k16.view(-1, Hkv, D)[:T].contiguous()
    a, b = empty_cache(NB, Hkv, bs, D, dtype), empty_cache(NB, Hkv, bs, D, dtype)
    ka, va, kb, vb = (torch.zeros(T, Hkv, D, dtype=dtype, device="cuda") for _ in range(4))
    pa.write_kv_int4(turned, dev(rc.v), dev(rc.slots), *a, k_out=ka, v_out=va)
    q = dev(rc.q)
    q_out = pa.rope_write_kv_int4(q, dev(rc.k), dev(rc.v), dev(rc.positions), dev(rc.cos), dev(rc.sin),
                                  dev(rc.slots), *b, k_out=kb, v_out=vb)
    assert np.array_equal(_bits(q_out), _bits(q_ref))
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))
    assert torch.equal(ka, kb) and torch.equal(va, vb)
    pa.rope_write_kv_int4(q, dev(rc.k), dev(rc.v), dev(rc.positions), dev(rc.cos), dev(rc.sin), dev(rc.slots), *b,
                          q_out=q)  # in place
    assert torch.equal(q, q_out)


def test_rope_write_int4_bad_position_leaves_token_alone():
    rc = make_rope_case(seed=1, num_tokens=3, num_q_heads=2, num_kv_heads=1, head_dim=64, block_size=16,
                        num_blocks=1, dtype="f16", max_position=16, skip_frac=0.0)
    pos = torch.tensor([0, 16, -1])
    cache = empty_cache(1, 1, 16, 64, torch.float16)
    q_out = torch.full_like(rc.q, 5.0).cuda()
    ko = torch.full_like(rc.k, 5.0).cuda()
    pa.rope_write_kv_int4(rc.q.cuda(), rc.k.cuda(), rc.v.cuda(), pos.cuda(), rc.cos.cuda(), rc.sin.cuda(),
                          torch.arange(3).cuda(), *cache, q_out=q_out, k_out=ko)
    assert pa.device_error() == 2
    assert (q_out[1:] == 5).all() and (ko[1:] == 5).all() and (q_out[0] != 5).any()
    assert (cache[2][0, 0, 1:] == 0).all() and (cache[3][0, 0, 1:] == 0).all() and (cache[2][0, 0, 0] != 0).any()


# ------------------------------------------------------------------------------------------ pages
def _random_cache(NB, Hkv, bs, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    codes = [torch.randint(0, 256, (NB, Hkv, bs, D // 2), generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    par = [torch.stack([0.3 * torch.exp(0.3 * torch.randn(NB, Hkv, bs, D // 64, generator=g)),
                        -7.5 + 2 * torch.randn(NB, Hkv, bs, D // 64, generator=g)], dim=-1).to(dtype).cuda()
           for _ in range(2)]
    return codes[0], codes[1], par[0], par[1]


@pytest.mark.parametrize("Hkv,bs,D", [(1, 16, 64), (3, 16, 128), (8, 32, 128), (5, 256, 64), (8, 256, 128)])
def test_copy_blocks_int4_bit_exact(Hkv, bs, D):
    """One source copied into several blocks, the first and last block of the pool, everything else untouched."""
    NB = 11
    cache = _random_cache(NB, Hkv, bs, D, torch.bfloat16, Hkv + bs)
    pairs = torch.tensor([[3, 7], [3, 10], [9, 0], [4, 1]], dtype=torch.int32)
    want = [x.clone() for x in cache]
    for s, t in pairs.tolist():
        for x in want:
            x[t] = x[s]
    pa.copy_blocks_int4(pairs.cuda(), *cache)
    assert all(torch.equal(x, y) for x, y in zip(cache, want))
    pa.copy_blocks_int4(pairs[:0].cuda(), *cache)
    assert all(torch.equal(x, y) for x, y in zip(cache, want))


def test_copy_and_load_out_of_range_pairs_are_skipped():
    cache = _random_cache(4, 2, 16, 64, torch.float16, 3)
    want = [x.clone() for x in cache]
    for x in want:
        x[2] = x[1]
    pa.copy_blocks_int4(torch.tensor([[0, 4], [-1, 0], [1, 2], [4, 3]], dtype=torch.int32, device="cuda"), *cache)
    assert pa.device_error() == 2
    assert all(torch.equal(x, y) for x, y in zip(cache, want))
    k16 = torch.full((3, 16, 2, 64), 5.0, dtype=torch.float16, device="cuda")
    v16 = k16.clone()
    pa.load_blocks_int4(torch.tensor([[0, 3], [4, 0], [1, 2], [0, -1]], dtype=torch.int32, device="cuda"), *cache,
                        k16, v16)
    assert pa.device_error() == 2
    assert (k16[:2] == 5).all() and (v16[:2] == 5).all() and (k16[2] != 5).any()


@pytest.mark.parametrize("Hkv,bs,D,dt", [(1, 16, 64, "f16"), (3, 16, 128, "bf16"), (8, 32, 128, "f16"),
                                         (5, 256, 64, "bf16")])
def test_load_blocks_int4_bit_exact(Hkv, bs, D, dt):
    """fp32 s * (code + z) rounded once to the type, in the 16-bit cache's layout; other blocks untouched."""
    dtype = DT[dt]
    NB, NB2 = 9, 5
    cache = _random_cache(NB, Hkv, bs, D, dtype, Hkv * bs)
    k16 = torch.full((NB2, bs, Hkv, D), 5.0, dtype=dtype, device="cuda")
    v16 = k16.clone()
    pairs = torch.tensor([[8, 0], [2, 4], [2, 1]], dtype=torch.int32)
    pa.load_blocks_int4(pairs.cuda(), *cache, k16, v16)
    for got, codes, par in ((k16, cache[0], cache[2]), (v16, cache[1], cache[3])):
        p = par.float().cpu().numpy()
        code = oq.unpack(codes.cpu().numpy()).astype(np.float32)
        vals = (p[..., 0:1] * (code + p[..., 1:2])).reshape(NB, Hkv, bs, D).transpose(0, 2, 1, 3)
        want = torch.full((NB2, bs, Hkv, D), 5.0, dtype=dtype)
        for s, t in pairs.tolist():
            want[t] = torch.from_numpy(vals[s].copy()).to(dtype)
        assert torch.equal(got.cpu(), want)


# ------------------------------------------------------------------------------------------ decode
def _pool_step(wl):
    """The workload's pool and new tokens in an INT4 cache: (numpy cache after the write, device cache, tables,
    lens); the new tokens go through write_kv_int4, the rest through the oracle's quantiser."""
    _, bt, lens, sm, _ = pa.replay_ops(wl.ops, wl.num_blocks, wl.cfg["block_size"], wl.free_order, wl.batch)
    (kc, kp), (vc, vp) = quantized_pool(wl.k_cache0), quantized_pool(wl.v_cache0)
    dtype = wl.q.dtype
    cache = to_device(kc, vc, kp, vp, dtype)
    pa.write_kv_int4(wl.k_new.cuda(), wl.v_new.cuda(), torch.from_numpy(sm).cuda(), *cache)
    oq.write_kv_int4(wl.k_new, sm, kc, kp)
    oq.write_kv_int4(wl.v_new, sm, vc, vp)
    assert np.array_equal(cache[0].cpu().numpy(), kc) and np.array_equal(cache[1].cpu().numpy(), vc)
    return (kc, vc, kp, vp), cache, bt, lens


def _check_decode(wl, cache, bt, lens, ref, what, **kw):
    rows, out, lse, bound, lse_bound = ref
    B, Hq, _ = wl.q.shape
    got_lse = torch.full((B, Hq), 7.0, dtype=torch.float32, device="cuda")
    got = pa.decode_int4(wl.q.cuda(), *cache, torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda(),
                         int(lens.max()), wl.scale, lse=got_lse, **kw)
    g, gl = got.double().cpu().numpy(), got_lse.double().cpu().numpy()
    at = np.asarray(rows)
    assert_within(g[at[:, 0], at[:, 1]], out, bound, what)
    live = np.isfinite(lse)
    assert_within(gl[at[:, 0], at[:, 1]][live], lse[live], lse_bound[live], what + " lse")
    assert (g[lens == 0] == 0).all() and np.isneginf(gl[lens == 0]).all()
    return got


RAGGED = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 777, 1000, 1500]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (6, 3), (8, 2), (16, 2), (16, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_decode_int4_ragged_shapes(D, Hq, Hkv, dtype):
    for bs, seed in ((16, 1), (64, 2), (256, 3)):
        wl = make_custom(seed=seed * 89 + Hq * 5 + D, lens=RAGGED, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D,
                         block_size=bs, dtype=dtype)
        host, cache, bt, lens = _pool_step(wl)
        ref = reference(wl.q, *host, bt, lens, wl.scale)
        for ns in (0, 1, 7, 64):
            _check_decode(wl, cache, bt, lens, ref, f"int4 D{D} G{Hq // Hkv} bs{bs} {dtype} partitions{ns}",
                          num_partitions=ns)


@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 0], [16], [5000], [1] * 40, [2048, 0, 1, 3000]])
def test_decode_int4_few_sequences(lens):
    wl = make_custom(seed=sum(lens) + len(lens), lens=lens, num_q_heads=8, num_kv_heads=1, head_dim=128, block_size=16)
    host, cache, bt, ln = _pool_step(wl)
    _check_decode(wl, cache, bt, ln, reference(wl.q, *host, bt, ln, wl.scale), f"int4 {lens[:4]}")


def test_decode_int4_qwen_batch():
    wl = make_workload("qwen_decode")
    host, cache, bt, lens = _pool_step(wl)
    rng = np.random.default_rng(0)
    rows = sorted({(int(b), int(h)) for b, h in zip(rng.integers(0, 128, 200), rng.integers(0, 16, 200))})
    ref = reference(wl.q, *host, bt, lens, wl.scale, rows)
    outs = [_check_decode(wl, cache, bt, lens, ref, f"int4 qwen partitions {ns}", num_partitions=ns)
            for ns in (0, 0, 1, 5, 1000)]
    assert torch.equal(outs[0], outs[1])  # the same plan twice: the same bits


@pytest.mark.parametrize("B", [257, 600, 1500])
def test_decode_int4_large_batches(B):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 120, B)
    lens[::89] = 0
    wl = make_custom(seed=B * 11, lens=lens.tolist(), num_q_heads=4, num_kv_heads=2, head_dim=64, block_size=16)
    host, cache, bt, ln = _pool_step(wl)
    ref = reference(wl.q, *host, bt, ln, wl.scale)
    for ns in (0, 7):
        _check_decode(wl, cache, bt, ln, ref, f"int4 B{B} partitions{ns}", num_partitions=ns)


@pytest.mark.parametrize("B,D", [(383, 128), (384, 128), (385, 128), (511, 64), (512, 64), (513, 64)])
def test_decode_int4_batches_about_the_threads_of_a_cta(B, D):
    """Where segments stop being dealt by length, and the counts that are and are not a multiple of four."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 150, B)
    lens[rng.integers(0, B, 5)] = 700
    wl = make_custom(seed=B, lens=lens.tolist(), num_q_heads=2, num_kv_heads=1, head_dim=D, block_size=16)
    host, cache, bt, ln = _pool_step(wl)
    ref = reference(wl.q, *host, bt, ln, wl.scale)
    for ns in (0, 3, 12, 16):  # 12 CTAs of 32 segments each at most
        _check_decode(wl, cache, bt, ln, ref, f"int4 B{B} partitions{ns}", num_partitions=ns)


@pytest.mark.parametrize("lens", [[2048] * 20, [1024] * 19, [8192, 8000, 64, 1], [8193, 30, 30], [4000, 100] * 10])
def test_decode_int4_dealt_and_cut(lens):
    """Equal and unequal lengths on both sides of the rule that deals segments whole, dealt and cut by the grid given."""
    wl = make_custom(seed=len(lens), lens=lens, num_q_heads=16, num_kv_heads=2, head_dim=64, block_size=32)
    host, cache, bt, ln = _pool_step(wl)
    rows = [(b, h) for b in range(0, len(lens), max(1, len(lens) // 4)) for h in (0, 7, 8, 15)]
    ref = reference(wl.q, *host, bt, ln, wl.scale, rows)
    for ns in (0, 2, 20, 38, 148):
        _check_decode(wl, cache, bt, ln, ref, f"int4 {lens[:3]} partitions{ns}", num_partitions=ns)


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(16, 1, 128, "bf16"), (4, 2, 64, "f16")])
def test_decode_int4_one_long_sequence(Hq, Hkv, D, dtype):
    wl = make_custom(seed=9, lens=[40001], num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, block_size=64, dtype=dtype)
    host, cache, bt, lens = _pool_step(wl)
    ref = reference(wl.q, *host, bt, lens, wl.scale)
    for ns in (0, 1, 2, 300):
        _check_decode(wl, cache, bt, lens, ref, f"int4 long partitions{ns}", num_partitions=ns)


def test_decode_int4_large_logits():
    wl = make_custom(seed=12, lens=[700, 33, 1024, 5], num_q_heads=16, num_kv_heads=8, head_dim=128, block_size=16,
                     q_scale=30.0)
    host, cache, bt, lens = _pool_step(wl)
    got = _check_decode(wl, cache, bt, lens, reference(wl.q, *host, bt, lens, wl.scale), "int4 q x30")
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("D,Hq,Hkv,dtype", [(128, 8, 2, "bf16"), (64, 4, 4, "f16"), (128, 16, 1, "f16")])
def test_decode_int4_outlier_channel_in_q(D, Hq, Hkv, dtype):
    """One channel of q 2^8 times the others, K alike there for all tokens: what tells the tokens apart is what the
    small q elements add.  A product of a code and a q element is cut at 2^-16 of the largest |q| of the row times the
    scale, at worst (24 bits below the largest product's exponent field, which is 2^-14 for any code of 2^-20 units):
    D such cuts move a score by at most D 2^-16 max|q| max s scale, on top of the bounds for q without outliers."""
    wl = make_custom(seed=13, lens=[700, 33, 1024, 5, 3000], num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D,
                     block_size=16, dtype=dtype)
    wl.q[..., 5] = 2.0 ** 8
    wl.k_cache0[..., 5] = 1.0
    wl.k_new[..., 5] = 1.0
    host, cache, bt, lens = _pool_step(wl)
    rows, out, lse, bound, lse_bound = reference(wl.q, *host, bt, lens, wl.scale)
    d2 = D * 2.0 ** -16 * wl.q.float().abs().max().item() * float(np.abs(host[2][..., 0]).max()) * wl.scale
    most = (np.abs(host[3][..., 0]) * (15 + np.abs(host[3][..., 1]))).max()  # of any |v|
    _check_decode(wl, cache, bt, lens, (rows, out, lse, bound + 2 * d2 * 2 * most, lse_bound + d2), "int4 outlier in q")


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 2, 128, "bf16"), (8, 1, 64, "f16"), (16, 1, 128, "bf16")])
def test_decode_int4_not_finite_q_spoils_its_own_head(Hq, Hkv, D, dtype):
    wl = make_custom(seed=14, lens=[70, 1, 2000, 33], num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, block_size=16,
                     dtype=dtype)
    host, cache, bt, lens = _pool_step(wl)
    rows, out, lse, bound, lse_bound = reference(wl.q, *host, bt, lens, wl.scale)
    q = wl.q.clone()
    q[0, 1, 7], q[1, 0, 0], q[2, 3, D - 1], q[2, 2, 1] = float("inf"), float("nan"), float("-inf"), float("nan")
    lost = {(0, 1), (1, 0), (2, 3), (2, 2)}
    wl.q = q
    keep = [i for i, r in enumerate(rows) if tuple(r) not in lost]
    _check_decode(wl, cache, bt, lens, ([rows[i] for i in keep], out[keep], lse[keep], bound[keep], lse_bound[keep]),
                  "int4 inf and nan in q")


@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
def test_decode_int4_logits_and_scales_moving_along_a_sequence(order):
    """Keys whose logits rise (or fall) by hundreds along the sequence and value rows scaled over 2^+-30: the
    running reference of the softmax and of the fp16 weights moves many times within one piece."""
    wl = make_custom(seed=21, lens=[3000, 1, 700, 2048, 65], num_q_heads=16, num_kv_heads=4, head_dim=128,
                     block_size=16)
    _, bt, lens, _, _ = pa.replay_ops(wl.ops, wl.num_blocks, 16, wl.free_order, wl.batch)
    g = torch.Generator().manual_seed(5)
    kf, vf = wl.k_cache0.float(), wl.v_cache0.float()
    for b, L in enumerate(lens):
        for j in range(-(-int(L) // 16)):
            x = j / max(1, -(-int(L) // 16))
            x = {"rising": x, "falling": 1 - x, "mixed": float(torch.rand((), generator=g))}[order]
            kf[bt[b][j]] *= 1 + 40 * x
            vf[bt[b][j]] *= 2.0 ** float(torch.randint(-30, 31, (), generator=g))
    wl.k_cache0, wl.v_cache0 = kf.to(wl.q.dtype), vf.to(wl.q.dtype)
    host, cache, bt, lens = _pool_step(wl)
    _check_decode(wl, cache, bt, lens, reference(wl.q, *host, bt, lens, wl.scale), f"int4 {order}")


def test_decode_int4_zero_and_tiny_value_rows():
    """Value rows of zeros (scale 0) first, rows of tiny values after them, then ordinary ones."""
    for tail in (0.0, 1e-6, 1.0):
        wl = make_custom(seed=23, lens=[400, 300, 17], num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16)
        _, bt, lens, _, _ = pa.replay_ops(wl.ops, wl.num_blocks, 16, wl.free_order, wl.batch)
        for b in range(3):
            for j in range(-(-int(lens[b]) // 16)):
                wl.v_cache0[bt[b][j]] *= 0.0 if j < 10 else tail
        wl.v_new *= tail
        host, cache, bt, lens = _pool_step(wl)
        got = _check_decode(wl, cache, bt, lens, reference(wl.q, *host, bt, lens, wl.scale), f"int4 zero rows {tail}")
        if tail == 0:
            assert (got == 0).all()


def test_decode_int4_masked_places_hold_anything():
    """NaN and infinite parameters in rows behind the last token of a block, in blocks no table names and in
    table entries past the context (-1): none of it is read into a result."""
    wl = make_custom(seed=31, lens=[1, 15, 17, 33, 50, 100], num_q_heads=4, num_kv_heads=2, head_dim=128, block_size=32)
    host, cache, bt, lens = _pool_step(wl)
    ref = reference(wl.q, *host, bt, lens, wl.scale)
    free = torch.ones(cache[2].shape[0], 32, dtype=torch.bool)
    for b, L in enumerate(lens):
        for t in range(int(L)):
            free[bt[b][t // 32], t % 32] = False
    hole = free.cuda()[:, None, :, None, None].expand_as(cache[2])
    for par, x in ((cache[2], float("nan")), (cache[3], float("inf"))):
        par[hole] = x
    for par, x in ((cache[2], float("-inf")), (cache[3], float("nan"))):
        par[..., 1][hole[..., 1]] = x
    wide = np.full((bt.shape[0], bt.shape[1] + 3), -1, dtype=np.int32)
    wide[:, : bt.shape[1]] = bt
    for ns in (0, 1, 3):
        _check_decode(wl, cache, wide, lens, ref, f"int4 masked partitions {ns}", num_partitions=ns)


def test_decode_int4_bad_block_sets_index_bit():
    wl = make_custom(seed=2, lens=[40, 20], num_q_heads=2, num_kv_heads=1, head_dim=64, block_size=16)
    _, cache, bt, lens = _pool_step(wl)
    bad = bt.copy()
    bad[0, 1] = wl.num_blocks
    pa.decode_int4(wl.q.cuda(), *cache, torch.from_numpy(bad).cuda(), torch.from_numpy(lens).cuda(), 40, wl.scale)
    assert pa.device_error() == 2


def test_int4_cache_of_more_than_32_bits_of_bytes():
    """Blocks on both sides of byte 2^32 of the codes (40000 blocks of 128 KiB): write, copy, decode and expansion give
    what a cache of a few blocks gives, bit for bit."""
    Hkv, bs, D, NB, dt = 8, 256, 128, 40000, torch.bfloat16
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of free device memory")
    far = [3, 32767, 32768, NB - 2, NB - 1]
    gen = torch.Generator(device="cuda").manual_seed(3)
    T = 4 * bs
    k, v = (torch.randn(T, Hkv, D, generator=gen, device="cuda").to(dt) for _ in "kv")
    q = torch.randn(2, 16, D, generator=gen, device="cuda").to(dt)
    lens = torch.tensor([3 * bs + 17, 2 * bs], dtype=torch.int32, device="cuda")
    got = []
    for blocks, n in ((far, NB), ([0, 1, 2, 3, 4], 5)):
        cache = empty_cache(n, Hkv, bs, D, dt)
        slots = torch.cat([torch.arange(bs) + b * bs for b in blocks[:4]]).cuda()
        pa.write_kv_int4(k, v, slots, *cache)
        pa.copy_blocks_int4(torch.tensor([[blocks[3], blocks[4]]], dtype=torch.int32, device="cuda"), *cache)
        tables = torch.tensor([[blocks[1], blocks[0], blocks[2], blocks[4]], [blocks[3], blocks[2], -1, -1]],
                              dtype=torch.int32, device="cuda")
        out = pa.decode_int4(q, *cache, tables, lens, 4 * bs, D ** -0.5)
        k16 = torch.zeros(2, bs, Hkv, D, dtype=dt, device="cuda")
        v16 = torch.zeros_like(k16)
        pa.load_blocks_int4(torch.tensor([[blocks[4], 0], [blocks[1], 1]], dtype=torch.int32, device="cuda"), *cache, k16, v16)
        got.append((out, k16, v16))
        del cache
    assert pa.device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(*got)) and got[0][1].any()


# ------------------------------------------------------------------------------------------ streams, graphs, workspaces
def test_decode_int4_one_workspace_for_calls_of_all_sizes():
    """A workspace zero-filled once and used by calls of other batches, heads, dimensions and work splits in turn, each
    with segments cut between CTAs: every call's result is that of a fresh workspace, bit for bit."""
    calls = []
    for seed, (lens, Hq, Hkv, D, ns) in enumerate([
            ([9000, 40], 8, 1, 128, 0), ([700] * 40, 16, 8, 64, 37), ([20000], 16, 1, 64, 300),
            ([3000, 0, 5, 1200] * 30, 8, 4, 128, 0), ([2000] * 3, 4, 2, 64, 1000), ([9000, 40], 8, 1, 128, 0)]):
        wl = make_custom(seed=50 + seed, lens=lens, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, block_size=16)
        _, cache, bt, ln = _pool_step(wl)
        dev = torch.from_numpy(bt).cuda(), torch.from_numpy(ln).cuda()
        calls.append((wl.q.cuda(), cache, *dev, int(ln.max()), wl.scale, ns,
                      pa.decode_int4_plan(len(lens), Hq, Hkv, D, int(ln.max()), ns)[2]))
    ws = torch.zeros(max(c[-1] for c in calls), dtype=torch.uint8, device="cuda")
    for again in range(2):
        for i, (q, cache, bt, ln, top, scale, ns, need) in enumerate(calls):
            got, got_lse, want, want_lse = (torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"),
                                            torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"))
            pa.decode_int4(q, *cache, bt, ln, top, scale, out=got, lse=got_lse, workspace=ws, num_partitions=ns)
            pa.decode_int4(q, *cache, bt, ln, top, scale, out=want, lse=want_lse, num_partitions=ns)
            assert torch.equal(got, want) and torch.equal(got_lse, want_lse), (again, i)


def test_decode_int4_graph_replay_and_side_stream():
    """Write and decode captured once on a side stream and replayed with new inputs: the eager calls' bits; the
    workspace ends zeroed; two graphs with a workspace each, replayed in turn."""
    wl = make_custom(seed=41, lens=[300, 1, 77, 1200, 16], num_q_heads=16, num_kv_heads=8, head_dim=128, block_size=16)
    _, cache, bt, lens = _pool_step(wl)
    dev = dict(bt=torch.from_numpy(bt).cuda(), lens=torch.from_numpy(lens).cuda())
    q = wl.q.cuda()
    kn, vn = wl.k_new.cuda(), wl.v_new.cuda()
    _, _, _, sm, _ = pa.replay_ops(wl.ops, wl.num_blocks, 16, wl.free_order, wl.batch)
    slots = torch.from_numpy(sm).cuda()
    need = pa.decode_int4_plan(5, 16, 8, 128, 1200)[2]
    graphs = []
    side = torch.cuda.Stream()
    for _ in range(2):
        ws, out = torch.zeros(need, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            pa.decode_int4(q, *cache, dev["bt"], dev["lens"], 1200, wl.scale, out=out, workspace=ws)  # warm
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for _ in range(3):
                pa.write_kv_int4(kn, vn, slots, *cache)
                pa.decode_int4(q, *cache, dev["bt"], dev["lens"], 1200, wl.scale, out=out, workspace=ws)
        graphs.append((graph, ws, out))
    g = torch.Generator().manual_seed(3)
    for i in range(4):
        q.copy_(torch.randn(q.shape, generator=g).to(q.dtype))
        kn.copy_(torch.randn(kn.shape, generator=g).to(q.dtype))
        want_cache = [x.clone() for x in cache]
        pa.write_kv_int4(kn, vn, slots, *want_cache)
        want = pa.decode_int4(q, *want_cache, dev["bt"], dev["lens"], 1200, wl.scale)
        graph, ws, out = graphs[i % 2]
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert (ws[: 4 * 5 * 8] == 0).all()  # the counters of 5 sequences x 8 KV heads


def test_decode_int4_given_stream_without_workspace_while_the_current_one_is_behind():
    """What a call makes itself (out, the zero-filled workspace, q_out) follows the stream it is given: the current
    stream is busy, and memory of the workspace's size that it has just freed holds no zeros."""
    wl = make_custom(seed=43, lens=[9000, 1, 4000], num_q_heads=8, num_kv_heads=1, head_dim=128, block_size=16)
    host, cache, bt, lens = _pool_step(wl)
    dev = torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda()
    q = wl.q.cuda()
    want = pa.decode_int4(q, *cache, *dev, 9000, wl.scale)
    need = pa.decode_int4_plan(3, 8, 1, 128, 9000)[2]
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        junk = [torch.full((need,), 1, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # 10 ms of the current stream
        del junk
        got = pa.decode_int4(q, *cache, *dev, 9000, wl.scale, stream=side)
        side.synchronize()
        assert torch.equal(got.cpu(), want.cpu())
    x = torch.randn(5, 8, 128, device="cuda").to(q.dtype)
    kv = torch.randn(2, 5, 1, 128, device="cuda").to(q.dtype)
    pos, slots = torch.arange(5, device="cuda"), torch.full((5,), -1, dtype=torch.int64, device="cuda")
    angle = torch.rand(16, 64, device="cuda")
    args = (x, kv[0], kv[1], pos, angle.cos(), angle.sin(), slots, *cache)
    want = pa.rope_write_kv_int4(*args)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    got = pa.rope_write_kv_int4(*args, stream=side)
    side.synchronize()
    assert torch.equal(got.cpu(), want.cpu())


def test_decode_int4_two_streams_two_workspaces():
    wl = make_custom(seed=43, lens=[900] * 24, num_q_heads=16, num_kv_heads=8, head_dim=128, block_size=16)
    _, cache, bt, lens = _pool_step(wl)
    args = (*cache, torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda(), 900, wl.scale)
    q = wl.q.cuda()
    want = pa.decode_int4(q, *args)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q) for _ in streams]
    ws = [torch.zeros(pa.decode_int4_plan(24, 16, 8, 128, 900)[2], dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o, w in zip(streams, outs, ws):
            pa.decode_int4(q, *args, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


# ------------------------------------------------------------------------------------------ together
def test_int4_serving_run_fork_copy_write_decode():
    """A prompt written, two sequences forked from it in the middle of a block (copy-on-write), decode steps of
    rotary write + attention: every step against the oracle's attention over the oracle's own cache."""
    Hq, Hkv, D, bs, NB, dtype = 8, 4, 128, 16, 40, torch.bfloat16
    g = torch.Generator().manual_seed(77)
    cos, sin = rope_tables(256, D)
    cache = empty_cache(NB, Hkv, bs, D, dtype)
    host = [np.zeros((NB, Hkv, bs, D // 2), np.uint8) for _ in range(2)] + \
           [np.zeros((NB, Hkv, bs, D // 64, 2), np.float32) for _ in range(2)]
    pool = pa.BlockPool(NB, bs)

    def step(seqs, counts):
        slots, pairs = pool.append_batch(seqs, counts)
        T = len(slots)
        q = torch.randn(T, Hq, D, generator=g).to(dtype)
        k, v = (torch.randn(T, Hkv, D, generator=g).to(dtype) for _ in range(2))
        pos = torch.cat([torch.arange(pool.info(s)[0] - n, pool.info(s)[0]) for s, n in zip(seqs, counts)])
        if pairs:
            pa.copy_blocks_int4(torch.tensor(pairs, dtype=torch.int32, device="cuda"), *cache)
            for s, t in pairs:
                for x in host:
                    x[t] = x[s]
        sl = torch.from_numpy(slots)
        # the turned keys as a 16-bit cache would hold them
        k16 = torch.zeros(-(-T // bs), bs, Hkv, D, dtype=dtype, device="cuda")
        v16 = torch.zeros_like(k16)
        qr = pa.rope_write_kv(q.cuda(), k.cuda(), v.cuda(), pos.cuda(), cos.cuda(), sin.cuda(),
                              torch.arange(T).cuda(), k16, v16)
        q_out = pa.rope_write_kv_int4(q.cuda(), k.cuda(), v.cuda(), pos.cuda(), cos.cuda(), sin.cuda(), sl.cuda(),
                                      *cache)
        assert torch.equal(q_out, qr)
        oq.write_kv_int4(k16.view(-1, Hkv, D)[:T].cpu(), slots, host[0], host[2])
        oq.write_kv_int4(v, slots, host[1], host[3])
        return q_out, pairs

    pool.alloc(0, 0)
    step([0], [45])                      # the prompt
    pool.fork(0, 1, 45)
    pool.fork(0, 2, 40)
    copies = 0
    for _ in range(9):
        q, pairs = step([0, 1, 2], [1, 1, 1])
        copies += len(pairs)
        bt, lens = pool.block_table([0, 1, 2], 8)
        got = pa.decode_int4(q, *cache, torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda(), int(lens.max()),
                             D ** -0.5)
        _, out, _, bound, _ = reference(q.cpu(), *host, bt, lens, D ** -0.5)
        assert_within(got.double().cpu().numpy().reshape(-1, D), out, bound, "serving run")
    assert copies == 2
    assert np.array_equal(cache[0].cpu().numpy(), host[0])


def test_int4_context_expanded_for_a_prefill_chunk():
    """A context held in 4 bits, expanded into a 16-bit cache, and a chunk's causal attention over it: the
    oracle's attention over the values the 4-bit cache holds."""
    wl = make_custom(seed=13, lens=[40, 150, 333], chunk_lens=[40, 100, 64], kind="prefill", num_q_heads=8,
                     num_kv_heads=2, head_dim=128, block_size=32)
    host, cache, bt, lens = _pool_step(wl)
    k16 = torch.zeros_like(wl.k_cache0).cuda()
    v16 = torch.zeros_like(k16)
    used = sorted({int(x) for x in bt.flatten() if x >= 0})
    pairs = torch.tensor([[b, b] for b in used], dtype=torch.int32, device="cuda")
    pa.load_blocks_int4(pairs, *cache, k16, v16)
    qsl = torch.from_numpy(wl.query_start_loc).cuda()
    got = pa.prefill_chunk(wl.q.cuda(), qsl, k16, v16, torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda(), 100,
                           wl.scale)
    kv = [oq.cache_values(host[0], host[2]), oq.cache_values(host[1], host[3])]
    kd, vd = (torch.from_numpy(x).to(wl.q.dtype) for x in kv)
    ref = oatt.prefill_attention(wl.q, wl.query_start_loc, kd, vd, [list(r) for r in bt], lens, wl.scale)
    for (b, h), r in ref.items():
        rows = slice(wl.query_start_loc[b], wl.query_start_loc[b + 1])
        assert_close(got[rows, h].float().cpu().numpy(), r, f"prefill over int4 seq{b} head{h}")


def test_int4_forked_prefix_equals_copied_prefix():
    """Sequences that share their prefix blocks decode to the bits of sequences with blocks of their own."""
    wl = make_prefix_groups(seed=8, group_sizes=[3, 2], prefix_lens=[64, 32], suffix_lo=0, suffix_hi=40,
                            num_q_heads=4, num_kv_heads=2, head_dim=128, block_size=16)
    _, cache, bt, lens = _pool_step(wl)
    B, MB = bt.shape
    NB = cache[0].shape[0]
    big = [torch.zeros((NB + B * MB, *x.shape[1:]), dtype=x.dtype, device="cuda") for x in cache]
    for x, y in zip(big, cache):
        x[:NB] = y
    own = bt.copy()
    pairs = []
    for b in range(B):
        for j in range(MB):
            if bt[b, j] >= 0:
                own[b, j] = NB + b * MB + j
                pairs.append([int(bt[b, j]), int(own[b, j])])
    pa.copy_blocks_int4(torch.tensor(pairs, dtype=torch.int32, device="cuda"), *big)
    ln = torch.from_numpy(lens).cuda()
    a = pa.decode_int4(wl.q.cuda(), *cache, torch.from_numpy(bt).cuda(), ln, int(lens.max()), wl.scale)
    b = pa.decode_int4(wl.q.cuda(), *big, torch.from_numpy(own).cuda(), ln, int(lens.max()), wl.scale)
    assert torch.equal(a, b)


def test_int4_split_context_merges():
    """Two halves of every context decoded apart (with their log-sum-exps) and merged: the whole context's result."""
    wl = make_custom(seed=19, lens=[700, 1, 64, 129], num_q_heads=8, num_kv_heads=2, head_dim=64, block_size=16,
                     dtype="f16")
    host, cache, bt, lens = _pool_step(wl)
    parts, lses = [], []
    for r in range(2):
        half = lens // 2 // 16 * 16
        t = np.full_like(bt, -1)
        ln = half if r == 0 else lens - half
        for b in range(len(lens)):
            src = bt[b, half[b] // 16:] if r else bt[b, : half[b] // 16]
            t[b, : len(src)] = src
        lse = torch.empty(4, 8, device="cuda")
        parts.append(pa.decode_int4(wl.q.cuda(), *cache, torch.from_numpy(t).cuda(),
                                    torch.from_numpy(ln.astype(np.int32)).cuda(), int(ln.max()), wl.scale, lse=lse))
        lses.append(lse)
    got = pa.merge_attn_states(torch.stack(parts), torch.stack(lses))
    _, out, _, bound, _ = reference(wl.q, *host, bt, lens, wl.scale)
    # each part is rounded to the type before the merge, and the merge once more: two steps more
    extra = torch.finfo(wl.q.dtype).eps * 4
    assert_within(got.double().cpu().numpy().reshape(-1, 64), out, 2 * bound + extra, "merged halves")
