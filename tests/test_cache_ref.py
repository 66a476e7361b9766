"""The 64-bit forms of the 8-bit cache that the GPU tests use, against independent ones."""
import torch

import cache_ref as C


def test_codes_are_the_librarys():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    want, got = codes.double(), C.code_values()
    assert torch.equal(torch.isnan(want), torch.isnan(got))
    assert torch.equal(want[~torch.isnan(want)], got[~torch.isnan(got)])


def test_rounding_is_the_librarys():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(500, 64, generator=g, dtype=torch.float64).float()
    codes, scale = C.quantize(x)
    power = C.powers()[scale.long()][:, None]
    assert torch.equal((x.double() / power).float().to(torch.float8_e4m3fn).view(torch.uint8), codes.view(torch.uint8))
    top = x.double().abs().amax(-1)
    assert bool((top <= 448 * power[:, 0]).all()) and bool((top > 224 * power[:, 0]).all())
    err = (C.numbers(codes, scale) - x.double()).abs()
    assert bool((err <= C.half_step(x.double(), scale[:, None])).all())


def test_rows_at_the_edges():
    x = torch.zeros(8, 16, dtype=torch.float64)
    x[1, 3] = 448.0
    x[2, 3] = 448.0000001
    x[3, 3] = float("inf")
    x[4, 3] = float("nan")
    x[5, 3] = 3.3e38
    x[6, 3] = 1e-40
    x[7] = torch.linspace(-1, 1, 16, dtype=torch.float64)
    codes, scale = C.quantize(x)
    assert scale.tolist()[:7] == [10, 127, 128, 255, 255, 246, 10]
    y = C.numbers(codes, scale)
    assert y[1, 3] == 448 and y[2, 3] == 448 and bool(torch.isnan(y[3:5]).all()) and y[5, 3] == 448 * 2.0 ** 119
    # a row's numbers are numbers of bf16
    rest = torch.isfinite(y)
    assert torch.equal(y[rest].to(torch.bfloat16).double(), y[rest])


def test_norm_against_a_library_routine():
    g = torch.Generator().manual_seed(2)
    x, w = torch.randn(3, 5, 64, generator=g, dtype=torch.float64), torch.rand(64, generator=g, dtype=torch.float64)
    want = torch.nn.functional.rms_norm(x, (64,), w, 1e-5)
    y, t = C.norm_rotate(x, w, 1e-5, None, None, False)
    assert torch.allclose(y, want, atol=1e-12) and bool((t > 0).any())
