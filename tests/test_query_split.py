"""How the dense pass over an 8-bit prefix splits a query row into 8-bit parts
(csrc/dense_quant.cu), on the CPU with torch's e4m3 and e5m2: what losa.h says of it."""
import numpy as np
import torch

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


def scaled(x, row_max):
    """Rows are scaled by a power of two to a maximum in [128, 256)."""
    return x.double() * 2.0 ** (7 - np.floor(np.log2(row_max)))


def test_torch_rounds_to_nearest_even():
    x = torch.tensor([1.0625, 1.1875, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])
    assert x.to(E4).tolist() == [1.0, 1.25, 16.0, 20.0, 0.0, 2.0 ** -8]
    y = torch.tensor([1.125, 1.375, 2.0 ** -17, 3 * 2.0 ** -17])
    assert y.to(E5).tolist() == [1.0, 1.5, 0.0, 2.0 ** -15]


def test_a_bf16_element_in_two_parts():
    """Exact down to 2^-13 of the row's largest element, within 2^-21 of that below."""
    bits = torch.arange(0, 0x7f80, dtype=torch.int32)
    all_bf16 = bits.to(torch.int16).view(torch.bfloat16)
    for row_max in (1.0, 1.5, 1.9921875):
        x = all_bf16[(all_bf16.float() <= row_max) & (all_bf16.float() >= 2.0 ** -60)]
        s = scaled(x, row_max)
        hi = s.float().to(E4)
        lo = (s - hi.double()).float().to(E5)
        err = (s - hi.double() - lo.double()).abs() * (row_max / scaled(torch.tensor(row_max), row_max))
        exact = x.double() >= 2.0 ** -13 * row_max
        assert exact.sum() > 1000 and (err[exact] == 0).all()
        assert err.max() <= 2.0 ** -21 * row_max and err.max() > 2.0 ** -23 * row_max


def test_an_fp32_element_in_six_parts():
    """Within 2^-29 of the row's largest element (the last three parts 2^12 times larger)."""
    g = torch.Generator().manual_seed(1)
    for row_max in (1.0, 1.5, 1.9999999):
        x = torch.cat([(torch.rand(20000, generator=g) * row_max * 2.0 ** -e) for e in range(0, 40, 3)])
        s = scaled(x, row_max)
        unit = row_max / scaled(torch.tensor(row_max, dtype=torch.float64), row_max)
        rest, total = s.float(), torch.zeros_like(s)
        for p in range(6):
            part = rest.to(E4).float()
            total += part.double() / (4096.0 if p >= 3 else 1.0)
            rest = (rest - part) * (4096.0 if p == 2 else 1.0)
        assert ((s - total).abs() * unit).max() <= 2.0 ** -29 * row_max
