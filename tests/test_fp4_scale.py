"""The scale of a 4-bit group: bf16(float32(max |x| * r)), r the float32 number nearest to 1/6, beside bf16(max |x| / 6) (on
the CPU; every significand, so every magnitude that float32 holds as a normal number)."""
import torch

R = torch.tensor(float.fromhex("0x1.555556p-3"), dtype=torch.float32)


def _scales(x):
    return (x * R).bfloat16(), (x / torch.tensor(6.0)).bfloat16()


def test_r_is_the_number_nearest_to_a_sixth():
    assert torch.tensor(1.0 / 6.0, dtype=torch.float64).float() == R


def test_where_the_product_and_the_quotient_differ():
    """In 21 of the 2^23 significands of float32, by one step of bfloat16, the product above; for no bfloat16 or float16
    magnitude."""
    x = (torch.arange(1 << 23, dtype=torch.int32) | 127 << 23).view(torch.float32)
    product, quotient = _scales(x)
    at = (product != quotient).nonzero().flatten()
    assert len(at) == 21
    assert torch.equal(product[at].view(torch.int16), quotient[at].view(torch.int16) + 1)
    for t in (torch.bfloat16, torch.float16):
        x = torch.arange(1 << 15, dtype=torch.int16).view(t)
        x = x[torch.isfinite(x)].float()
        product, quotient = _scales(x)
        assert torch.equal(product, quotient)
