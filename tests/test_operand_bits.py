"""What two fp16 parts (and one) hold of a value, as the layer's gradients use them: the bounds of the
interface, checked on the CPU over all magnitudes.  A tensor's largest value is scaled into [2^13, 2^14)."""
import torch

import layer_ref as R


def parts(v, exponent):
    """hi + lo of v 2^exponent, taken back (all in 64 bits but the two roundings)."""
    s = v.float() * 2.0 ** exponent
    hi = s.half()
    lo = (s - hi.float()).half()
    return (hi.double() + lo.double()) * 2.0 ** -exponent


def magnitudes(top):
    """fp32 values of every exponent down to 2^-60 of `top`, 24 bits each."""
    f = 1 + torch.rand(61, 4000, generator=R.gen(1), dtype=torch.float64)
    return (top / 2 * f * 2.0 ** -torch.arange(61.0, dtype=torch.float64).view(-1, 1)).float()


def test_two_parts_hold_22_bits_down_to_2_to_the_minus_16():
    # the largest anywhere in the binade it is scaled to
    for top in (1.0, 1.25, 1.9999):
        v = magnitudes(top)
        err = (parts(v, 13) - v.double()).abs()
        near = v >= 2.0 ** -16 * top
        assert bool((err[near] <= 2.0 ** -22 * v.double()[near]).all())
        assert float(err[~near].max()) <= 2.0 ** -38 * top
        # further down the bits go: the bound is not loose by more than a binade
        assert float((err / v.double())[v < 2.0 ** -18 * top].max()) > 2.0 ** -22
        assert float((err / v.double())[v < 2.0 ** -23 * top].max()) > 2.0 ** -16


def test_one_part_holds_bf16_values_down_to_2_to_the_minus_30():
    for top in (1.0, 1.25, 1.984375):
        v = magnitudes(top).bfloat16()
        s = (v.float() * 2.0 ** 13).half()
        err = (s.double() * 2.0 ** -13 - v.double()).abs()
        near = v.double() >= 2.0 ** -30 * top
        assert float(err[near].max()) == 0.0
        assert 0.0 < float(err[~near].max()) <= 2.0 ** -38 * top
