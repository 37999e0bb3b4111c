"""The prompt prologue's E4M3 codes under scales of every size: V is only divided by its scale, so that its codes are those
of the quotient in fp32. A quotient of 0 / 0, of two infinities or with a NaN is the NaN code; what is too large saturates."""
import math

import numpy as np
import pytest
import torch

from oracle import fp8 as OF
from tests.test_gpu_prompt_prologue import make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from load_balanced_split_step_b200 import binding
    return binding


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -149, 1e-39, 2.0 ** -128, 2.0 ** -127, 2.0 ** -126, 3 * 2.0 ** -110, 2.0 ** -100,
                                   1.5 * 2.0 ** -100, -0.37, 2.0 ** 100, 1.75 * 2.0 ** 100, 2.0 ** 126, 3e38, math.inf, math.nan])
def test_codes_are_those_of_the_quotient(B, scale):
    n, Hkv, D, P = 128, 2, 128, 64
    g = torch.Generator().manual_seed(5)
    bits = torch.randint(0, 65536, (n, 3 * Hkv, D), generator=g, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    # values whose quotients are of the codes' size, where bf16 has such, and zeros
    near = (torch.randn((n, 3 * Hkv, D), generator=g).double() * (scale if 0 < abs(scale) < math.inf else 1.0)).to(torch.bfloat16)
    near[::7] = 0
    c = make((n,), (0,), Hkv, Hkv, D, P, "e4m3", "NHD", seed=2)
    c["vs"] = torch.tensor([scale, 0.37])
    for x in (bits, near):
        c["qkv"] = x
        d, _, _, st = run(B, c, Hkv, Hkv, "e4m3", "NHD")
        assert st == 0
        y = x[:, 2 * Hkv:].float().numpy() / c["vs"].numpy()[:, None]
        got = d["v"].cpu()[c["table"][0, :n // P].long()].reshape(n, Hkv, D).numpy()
        nan = np.isnan(y)
        assert np.array_equal((got & 127) == 127, nan)
        codes = OF.encode_array(np.clip(np.nan_to_num(y.astype(np.float64), nan=0.0, posinf=1e9, neginf=-1e9), -448, 448))
        assert np.array_equal(got[~nan], codes.astype(np.uint8)[~nan])
