"""The form that MLA_FORM_AUTO takes: never one whose workspace is out of
proportion where the other form would serve the call.  Host only."""
import pytest


@pytest.fixture(scope="module")
def size():
    from sparse_head_latent_absorbed_b200 import build
    build.build()
    import sparse_head_latent_absorbed_b200._lib as m
    return m.mla_attend_paged_workspace_bytes


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("S,bound", [(256, 131072), (64, 1 << 20), (17, 131072), (1, (1 << 21) + 1)])
def test_a_wide_bound_takes_the_absorbed_form(size, S, bound, bits):
    # (the expanded form is not refused, but would need from 11 GB up to twice a GPU's memory)
    N = min(65535, 256 * S)
    assert size(N, S, bound, bits, "expanded") >= 11e9
    assert 0 < size(N, S, bound, bits) == size(N, S, bound, bits, "absorbed") < 36e9


@pytest.mark.parametrize("S,bound", [(16, 131072), (1, 1 << 21), (1, 6000), (256, 8192)])
def test_up_to_two_million_positions_it_expands(size, S, bound):
    N = 255 * S
    assert 0 < size(N, S, bound, 16) == size(N, S, bound, 16, "expanded") < 11.1e9


def test_where_the_absorbed_form_is_refused_it_expands(size):
    # more than 2^30 tiles of a token and 128 positions
    N, S, bound = 60000, 2, 1 << 22
    assert size(N, S, bound, 16, "absorbed") == 0
    assert 0 < size(N, S, bound, 16) == size(N, S, bound, 16, "expanded")
