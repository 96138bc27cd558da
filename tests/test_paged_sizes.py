"""Sizes that the C calls take as 32-bit numbers are not cut to 32 bits, nor
to whole numbers, on their way there.  Host only, but for the last test."""
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from sparse_head_latent_absorbed_b200 import build
    build.build()
    import sparse_head_latent_absorbed_b200._lib as m
    return m


BAD = [2 ** 32 + 700, -2 ** 32 + 700, 2 ** 31, 700.5, float("nan"), float("inf")]


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("at", range(3))
def test_workspace_bytes(L, at, bad):
    args = [3, 2, 700]
    args[at] = bad
    with pytest.raises(L.MLAError):
        L.mla_attend_paged_workspace_bytes(*args, 16)


def test_whole_numbers_of_any_type(L):
    f = L.mla_attend_paged_workspace_bytes
    assert f(3, 2, 700, 16) == f(3.0, torch.tensor(2), torch.tensor([700]).max(), 16) > 0
    assert f(3, 2, 2 ** 24 + 1, 16) == 0  # refused, as by the C call


@pytest.mark.gpu
def test_a_bound_past_32_bits_is_refused():
    import paged_ref as R
    import sparse_head_latent_absorbed_b200 as shla
    w = R.make([2], [40], 16, 16, 73)
    for bad in BAD:
        with pytest.raises(shla.MLAError):
            shla.mla_attend_paged(**{**w, "max_kv": bad})
    got = shla.mla_attend_paged(**{**w, "max_kv": 40.0})
    assert torch.equal(got, shla.mla_attend_paged(**w))
