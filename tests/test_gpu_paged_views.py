"""Pages of one row whose row stride says nothing: torch gives a dimension of
size one whatever stride the view came by."""
import pytest
import torch

import paged_ref as R
from test_gpu_paged import FORMS, check, ref_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def shla():
    import sparse_head_latent_absorbed_b200 as m
    return m


def views(pages):
    """[P, 1, width] pages as views that hold the same rows."""
    P, _, width = pages.shape
    more = 16 if pages.dtype == torch.uint8 else 8
    wide = torch.zeros(P, 3, width + more, dtype=pages.dtype, device=pages.device)
    wide[:, 1, :width] = pages[:, 0]
    yield "transposed", pages.view(1, P, width).clone().transpose(0, 1)
    yield "row of a page", wide[:, 1:2, :width]
    yield "column", wide.clone()[:, 2, :width].copy_(pages[:, 0])[:, None]
    yield "stride 0", pages[:, 0].clone().as_strided((P, 1, width), (width, 0, 1))


@pytest.mark.parametrize("bits", [16, 8])
def test_pages_of_one_row(shla, bits):
    w = R.make([2, 130], [90, 260], bits, 1, 70, poison=False)
    want = ref_of(w)
    flat = w["pages"].view(w["pages"].shape[0], -1)
    slots = torch.randperm(len(flat), device="cuda").int()
    rows = R.cache_rows(len(flat), 71, "cuda")
    stored = R.row8(rows) if bits == 8 else rows
    for name, pages in views(w["pages"]):
        assert pages.shape == w["pages"].shape, name
        for form in FORMS:
            check(shla.mla_attend_paged(**{**w, "pages": pages}, form=form), want)
        back = shla.mla_page_read(pages, slots)
        assert torch.equal(back.double(), R.values(flat)[slots.long()]), name
        shla.mla_page_write(rows, slots, pages)
        assert torch.equal(pages[slots.long(), 0], stored), name


@pytest.mark.parametrize("bits", [16, 8])
def test_a_single_row(shla, bits):
    rows = R.cache_rows(1, 72, "cuda")
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    stored = R.row8(rows) if bits == 8 else rows
    pages = torch.zeros_like(stored).as_strided((1, 1, stored.shape[1]), (7, 5, 1))
    shla.mla_page_write(rows, slot, pages)
    assert torch.equal(pages[0], stored)
    assert torch.equal(shla.mla_page_read(pages, slot).double(), R.values(stored))
