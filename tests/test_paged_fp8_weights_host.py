"""The arithmetic of the attention over a paged cache in 8 bits that the kernels rely on, on the CPU."""

import numpy as np
import torch


def e5m2(x):
    """fp16 numbers rounded to E5M2, as fp64."""
    return torch.from_numpy(x).to(torch.float16).to(torch.float8_e5m2).double().numpy()


def test_three_e5m2_numbers_hold_an_fp16_weight():
    """Every fp16 number p from 0 to 2^14 is p1 + 2^-4 p2 + 2^-8 p3 with E5M2 numbers; what is carried on between them is an
    fp16 number each time, and no part passes E5M2's largest number."""
    bits = np.arange(0x0000, 0x7401, dtype=np.uint16)  # 0x7400 is 2^14
    p = bits.view(np.float16).astype(np.float64)
    assert p[-1] == 2.0 ** 14 and p[1] == 2.0 ** -24
    rest, total = p, np.zeros_like(p)
    for k in range(3):
        assert np.array_equal(rest, rest.astype(np.float16).astype(np.float64))
        assert np.abs(rest).max() <= 57344
        part = e5m2(rest)
        total = total + part * 2.0 ** (-4 * k)
        left = rest - part
        assert np.array_equal(left, left.astype(np.float16).astype(np.float64))
        rest = left * 16
    assert np.array_equal(total, p)
    # the upper byte of an fp16 number whose lower byte is 0 is the E5M2 number of its value
    codes = torch.arange(256, dtype=torch.uint8)
    as_half = (codes.to(torch.int32) << 8).to(torch.int16).view(torch.float16)
    assert torch.equal(codes.view(torch.float8_e5m2).float().nan_to_num(7.0), as_half.float().nan_to_num(7.0))


def test_rows_left_out_of_a_block_do_not_cut_it():
    """The oracle's append takes the stored rows of a block together: one scale from all of them, earlier tokens rounded
    anew once, tokens that stand between them as they were."""
    from oracle import kda_paged_fp8_oracle as fp8
    rng = np.random.default_rng(6)
    codes = rng.integers(0, 0x70, (1, 16, 1, 4)).astype(np.uint8)
    x = rng.normal(size=(8, 1, 4)) * np.array([1, 1, 1, 1, 1, 1, 1, 1000.0])[:, None, None]
    slots = [5, 6, -1, 8, -1, -1, 11, 12]
    got, scales, _, kind = fp8.write_side(x, slots, codes, np.full((1, 1, 1), 2.0 ** -30))
    need = 2.0 ** fp8.scale_exponent(np.abs(x[[0, 1, 3, 6, 7]]).max())
    assert scales[0, 0, 0] == need
    assert kind[0, :, 0].tolist() == [1] * 5 + [2, 2, 0, 2, 0, 0, 2, 2] + [0] * 3
    assert np.array_equal(got[0, [7, 9, 10, 13, 14, 15]], codes[0, [7, 9, 10, 13, 14, 15]])
