"""Calls of the 4-bit operators and the code scoring on the GPU: empty batches,
tensors that the library cannot read, streams, captured first calls."""
import numpy as np
import pytest

import four_bit_ref as ref
import synth

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def ads():
    import torch
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import ar_decode_step_gb300.build as b
    b.build()
    import ar_decode_step_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("V,top", [(1026, 5), (1026, 0), (40000, 3)])
def test_code_logprobs_of_an_empty_batch(ads, V, top):
    import torch
    lp, ent, at, at_lp = ads.code_logprobs(torch.empty((0, 2 * V), device="cuda"),
                                           torch.empty((0, 2), dtype=torch.int32, device="cuda"), V, top=top)
    assert lp.shape == ent.shape == (0, 2) and at.shape == at_lp.shape == (0, 2, top)
    assert at.dtype == torch.int32 and lp.dtype == torch.float32
