"""Rotation bases below 1 (append_kv): what is refused (no GPU needed) and what holds of the others."""
import numpy as np
import pytest
import torch

import bit_quantized_token_gb300 as bq
from test_serve_args import append


@pytest.fixture(scope="module", autouse=True)
def library():
    bq.build()


@pytest.mark.parametrize("theta", [9.7e-4, 1e-6, 1e-200, 1e-310, 5e-324])
def test_turns_of_which_nothing_is_known(theta):
    with pytest.raises(bq.LlmError, match="rope_theta is below 2"):
        append(rope_theta=theta)


@pytest.mark.gpu
@pytest.mark.parametrize("theta", [2.0 ** -10, 0.03, 0.5, 1.0])
def test_small_bases(theta):
    """Against the formula in 64 bits, as test_gpu_kv_rows; the turn's table is off by 2^-50 of the turn, which is up to
    1 / (2 pi theta) here, and so is the reference's own power (2 2^-53 of it)."""
    from test_gpu_kv_rows import gen, make_cache, reference, tolerance
    torch.cuda.set_device(0)
    T, hd, g = 40, 128, gen(1)
    x = torch.randn(T, 1, hd, device="cuda", generator=g)
    cache = make_cache(1, 1, T, hd, "bf16", g)
    pos = torch.from_numpy(np.random.default_rng(0).integers(0, 1 << 16, T)).to(torch.int32).cuda()
    rows, out = torch.arange(T, dtype=torch.int32, device="cuda"), torch.empty_like(x)
    bq.append_kv(x, x, bq.KVView(*cache), torch.zeros_like(rows), rows, q=x, q_out=out, positions=pos, rope_theta=theta,
                 rope_neox=True)
    want, size = reference(x, None, pos, theta, True)
    far = pos.double()[:, None, None] * (1 / theta) * (2.0 ** -50 + 2.0 ** -52)
    assert ((out.double() - want).abs() <= tolerance(size, want, pos, hd, torch.float32) + size * far).all()
