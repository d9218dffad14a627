"""The plain 4-bit definitions against torch's casts and values by hand."""
import torch

from tests import nvfp4_ref as N


def test_e4m3_codes_are_torch_s():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.isnan(N.E4M3), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.equal(N.E4M3[fine], want[fine])


def test_scales_round_like_torch_s_cast():
    x = torch.cat([torch.linspace(0, 448, 20001), torch.linspace(0, 0.1, 20001)]).float()
    want = x.to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(N.nearest_even(x.double(), N.E4M3[:0x7f]).to(torch.uint8), want)


def test_codes_by_hand():
    x = torch.tensor([6.0, 5.0, 5.01, 4.99, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.26, -0.24, -0.75, -5.0, 0.0, -6.0])
    codes, scales = N.quantise(x[None].bfloat16().double().bfloat16(), 1.0)
    assert scales.tolist() == [[0x38]]                      # 1.0
    # 5.01 and 4.99 are 5 in bf16; ties go to the even code
    nibbles = [7, 6, 6, 6, 6, 4, 4, 2, 2, 0, 1, 8, 10, 14, 0, 15]
    assert codes.tolist() == [[nibbles[i] | nibbles[i + 1] << 4 for i in range(0, 16, 2)]]
    back = N.values(codes, scales, 0.5)
    assert back[0, :4].tolist() == [3.0, 2.0, 2.0, 2.0] and back[0, 12].item() == -0.5


def test_a_group_that_is_not_finite():
    x = torch.ones((1, 32)).bfloat16()
    x[0, 3] = float("inf")
    codes, scales = N.quantise(x, 1.0)
    assert scales[0, 0] == 0x7f and (codes[0, :8] == 0).all() and torch.isnan(N.values(codes, scales, 1.0)[0, :16]).all()
    assert torch.isfinite(N.values(codes, scales, 1.0)[0, 16:]).all()
