"""decode_int4's numbers: what is refused is named, on the CPU and ahead of the device check."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_kv_cache_330_b200 as pa


def _args(dt=torch.bfloat16):
    codes, par = torch.zeros(2, 1, 16, 64, dtype=torch.uint8), torch.zeros(2, 1, 16, 2, 2, dtype=dt)
    return (torch.zeros(1, 2, 128, dtype=dt), codes, codes.clone(), par, par.clone(),
            torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32))


@pytest.mark.parametrize("bad,error,msg", [
    (dict(max_context_len=16.0), TypeError, "max_context_len must be an integer, got 16.0"),
    (dict(max_context_len="16"), TypeError, "max_context_len must be an integer, got '16'"),
    (dict(max_context_len=np.float32(16)), TypeError, "max_context_len must be an integer"),
    (dict(max_context_len=None), TypeError, "max_context_len must be an integer"),
    (dict(max_context_len=1 << 31), ValueError, "max_context_len must fit in 32 bits"),
    (dict(num_partitions=1.5), TypeError, "num_partitions must be an integer, got 1.5"),
    (dict(num_partitions="2"), TypeError, "num_partitions must be an integer"),
    (dict(num_partitions=-(1 << 40)), ValueError, "num_partitions must fit in 32 bits"),
    (dict(scale="0.1"), TypeError, "scale must be a number, got '0.1'"),
    (dict(scale=None), TypeError, "scale must be a number"),
    (dict(scale=1j), TypeError, "scale must be a number")])
def test_a_wrong_number_is_named(bad, error, msg):
    with pytest.raises(error, match=msg):
        pa.decode_int4(*_args(), **{"max_context_len": 16, "scale": 0.1, **bad})


@pytest.mark.parametrize("good", [dict(max_context_len=np.int64(16)), dict(max_context_len=torch.tensor(16)),
                                  dict(scale=np.float32(0.1)), dict(scale=1), dict(num_partitions=np.int32(3))])
def test_numbers_of_other_kinds_reach_the_device_check(good):
    with pytest.raises(ValueError, match="device calls take CUDA tensors"):
        pa.decode_int4(*_args(), **{"max_context_len": 16, "scale": 0.1, **good})


def test_a_refusal_without_a_known_reason_is_an_error_of_the_arguments():
    with pytest.raises(ValueError, match="not as this call takes it"):
        pa._refuse(None, ())


def test_tables_of_nearly_2_to_the_31_tokens_are_refused():
    """The kernel counts tokens in 32 bits, some hundreds past a sequence's end."""
    def call(mb, bs):  # addresses that are never used; without a workspace the last check refuses what is left
        at = 0x10000
        return pa.lib.pa_decode_int4(at, at, at, at, at, at, mb, at, 2, 4, 2, 128, bs, 16, 100, 0.1, 1, None, 0, 0, at,
                                     None, None)

    for bs in (16, 256):
        most = ((1 << 31) - 1024) // bs
        assert call(most, bs) == -4       # PA_ERR_WORKSPACE
        assert call(most + 1, bs) == -2   # PA_ERR_UNSUPPORTED
        assert call((1 << 31) // bs - 1, bs) == -2
