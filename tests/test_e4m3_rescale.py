"""What a page's codes keep when its scale grows: every value of at least 2^-13 of the largest that the scale is for.  (The largest is
more than 224 of the new scale, a value of 2^-13 of it more than 2^-6 of it: the format's normal range, where dividing by a power of
two is exact.  One below 2^-6 of the scale, up to 2^-13.8 of the largest, may lose bits.)"""
import torch

import attention_model as am


def test_values_of_2_13_of_the_largest_are_kept():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    codes = codes[torch.isfinite(codes)]
    lost = 0.0
    for up in range(1, 18):
        for largest in (225.0, 240.0, 300.0, 448.0):
            new = largest * 2.0 ** up  # (a largest value that needs this scale, for codes of scale 1)
            s = am.scale_of(new)
            assert s == 2.0 ** up
            kept = am.e4m3(codes / s) * s == codes
            assert bool(kept[codes.abs() >= new * 2.0 ** -13].all())
            if not kept.all():
                lost = max(lost, float(codes[~kept].abs().max() / new))
    assert 2.0 ** -14 < lost < 2.0 ** -13
