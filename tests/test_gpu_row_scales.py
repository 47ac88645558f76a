"""e4m3 rows whose largest value is so small that its 448th part is zero in fp32."""
import pytest
import torch

import mla_latent_kv_42_b200 as M
from mla_latent_kv_42_b200 import build, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    M.load_library()
    M.read_device_status()


@pytest.mark.parametrize("d", [synth.PRODUCTION, synth.RUNNING], ids=["production", "running"])
def test_scale_that_fp32_holds_as_zero(d):
    """c' = x / sqrt(eps) gain = 2^-100 2^10 2^-57 = 2^-147 where x is not zero (x^2 is far below eps):
    2^-147 / 448 rounds to zero in fp32 (half its smallest value is 2^-150). No e4m3 scale holds such a
    part, so it reads back as zeros, not as a quotient by zero; the same for the rotated part."""
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    x = torch.zeros((2, d.D), dtype=torch.bfloat16, device="cuda")
    x[0, 1::3] = 2.0 ** -100
    x[1] = 1
    gc = torch.full((d.d_c,), 2.0 ** -57, dtype=torch.bfloat16, device="cuda")
    gr = torch.full((d.d_rope,), 2.0 ** -57, dtype=torch.bfloat16, device="cuda")
    pool = torch.full((1, M.fp8_page_bytes(d)), 0x55, dtype=torch.uint8, device="cuda")
    M.norm_append_kv_fp8(d, x, i32(0, 0), i32(0, 1), i32(0)[None], pool, gain_c=gc, gain_r=gr, eps=2.0 ** -20)
    got = M.read_kv_fp8(d, pool, i32(0, 0), i32(0, 1), i32(0)[None])
    assert M.read_device_status() == 0
    n = d.page_size * d.D
    scales = pool[:, n:].contiguous().view(torch.float32).view(d.page_size, 2)[:2]
    assert bool((scales[0] == 1).all())
    assert not bool(got[0].any())
    assert bool((got[1, :d.d_c].float() - 2.0 ** -57).abs().max() <= 2.0 ** -57 * 2.0 ** -7)
