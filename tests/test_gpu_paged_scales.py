"""8-bit rows written by other means, whose scales are not powers of two (the
same 656 bytes with the scale max / 448 are common): a value is code * scale in
fp32, rounded once more to bf16, wherever the rows are read."""
import pytest
import torch

import paged_ref as R
from test_gpu_paged import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def shla():
    import sparse_head_latent_absorbed_b200 as m
    return m


def foreign_rows(rows):
    """bf16 [N, 576] -> uint8 [N, 656] with scales max / 448, and the values they stand for."""
    x = rows[:, :512].float().view(-1, 4, 128)
    scale = x.abs().amax(-1) / 448.0
    codes = (x / scale[..., None]).to(torch.float8_e4m3fn)
    stored = torch.cat([codes.view(-1, 512).view(torch.uint8), scale.view(torch.uint8),
                        rows[:, 512:].contiguous().view(torch.uint8)], 1)
    val = (codes.float() * scale[..., None]).view(-1, 512).to(torch.bfloat16)
    return stored, torch.cat([val, rows[:, 512:]], 1)


def test_read(shla):
    rows = R.cache_rows(3000, 80, "cuda", 2.0)
    rows[:, :128] *= 2.0 ** 20  # a scale above 2^7
    rows[:, 128:256] *= 2.0 ** -80
    stored, want = foreign_rows(rows)
    slots = torch.randperm(3008, device="cuda")[:3000].int()
    pages = torch.zeros(47, 64, 656, dtype=torch.uint8, device="cuda")
    pages.view(-1, 656)[slots.long()] = stored
    assert torch.equal(shla.mla_page_read(pages, slots), want)


# absorbed without and with conversion to bf16 rows first, and expanded
@pytest.mark.parametrize("form,q,kv", [("absorbed", [1] * 5, [3, 1, 64, 129, 1000]),
                                       ("absorbed", [40, 30], [9000, 700]),
                                       ("expanded", [2, 130], [300, 260])])
def test_attention(shla, form, q, kv):
    w = R.make(q, kv, 16, 16, 81, poison=False)
    stored, val = foreign_rows(w["pages"].view(-1, 576))
    shape = w["pages"].shape
    args = ("q_nope", "q_pe", "wkv_b", "pages", "page_table", "cu_q", "kv_len", "scale")
    want = R.attend(*({**w, "pages": val.view(shape)}[k] for k in args))
    w["pages"] = stored.view(shape[0], shape[1], 656)
    check(shla.mla_attend_paged(**w, form=form), want)
    # the same bits as over pages that hold those values in 16 bits
    if form == "expanded":
        w16 = {**w, "pages": val.view(shape)}
        assert torch.equal(shla.mla_attend_paged(**w, form=form),
                           shla.mla_attend_paged(**w16, form=form))


@pytest.mark.parametrize("foreign", [False, True])
@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("q,kv,page", [([1, 2, 1], [70, 129, 1], 16), ([1, 1], [200, 65], 7),
                                       ([130], [150], 64)])
def test_bytes_that_no_row_uses(shla, form, q, kv, page, foreign):
    # every byte of free rows is 0xff: NaN codes under NaN scales, the pool's first row
    # among them
    w = R.make(q, kv, 16, page, 82, poison=False)
    P = w["pages"].shape[0]
    rows = w["pages"].view(-1, 576)
    stored, val = foreign_rows(rows) if foreign else (R.row8(rows), rows)
    if not foreign:
        val = R.values(stored).to(torch.bfloat16)
    used = torch.zeros(P * page, dtype=torch.bool, device="cuda")
    for s, n in enumerate(kv):
        j = torch.arange(n, device="cuda")
        used[w["page_table"][s].long()[j // page] * page + j % page] = True
    # a page more, at the front
    stored = torch.where(used[:, None], stored, torch.full_like(stored, 255))
    w["pages"] = torch.cat([torch.full_like(stored[:page], 255), stored]).view(P + 1, page, 656)
    w["page_table"] = w["page_table"] + 1
    ref = torch.cat([torch.zeros_like(val[:page]), torch.where(used[:, None], val, 0.0)])
    args = ("q_nope", "q_pe", "wkv_b", "pages", "page_table", "cu_q", "kv_len", "scale")
    want = R.attend(*({**w, "pages": ref.view(P + 1, page, 576)}[k] for k in args))
    check(shla.mla_attend_paged(**w, form=form), want)
