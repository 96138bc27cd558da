"""Paged latent cache and the attention over it, against the 64-bit forms of
paged_ref.

Writing and reading are exact: a code is one defined rounding and a code times
its power-of-two scale is a bf16 value.

Attention: every rounding to bf16 is off by at most half a step, 2^-8 of the
value, so by 2^-8 / sqrt(3) = 2.3e-3 in the mean square at worst.  The absorbed
form rounds q~ (a relative error of the scores, which have a spread of about 1,
so the same relative error of the weights), the weights, the mixed latent (a
split token's twice) and the output: sqrt(5) * 2.3e-3 = 5.0e-3 of the output's
norm.  The expanded form rounds keys, weights, values, output and, where work
is split, partial outputs: as many.  REL allows twice that.  One element's error is a sum of many, so close to
normal with 5e-3 of its row's mean square as deviation: over 10^6 elements 6
deviations, 3e-2, plus its own rounding; ELEM allows 4e-2.  Where a scale
factor f > 1 widens the scores' spread to f, q~'s share grows f-fold.
"""
import pytest
import torch

import mla_inputs as mi
import paged_ref as R

pytestmark = pytest.mark.gpu

REL, ELEM = 1e-2, 4e-2
FORMS = ["absorbed", "expanded"]
REF = ("q_nope", "q_pe", "wkv_b", "pages", "page_table", "cu_q", "kv_len", "scale")


@pytest.fixture(scope="module")
def shla():
    import sparse_head_latent_absorbed_b200 as m
    return m


def ref_of(w):
    return R.attend(*(w[k] for k in REF))


def check(out, want, spread=1.0):
    got = out.double()
    assert torch.isfinite(got).all()
    err = got - want
    assert err.norm() <= REL * spread * want.norm() + 1e-30
    rms = want.square().mean(-1, keepdim=True).sqrt()
    assert (err.abs() <= 2.0 ** -8 * want.abs() + ELEM * spread * rms).all()


# ---------------------------------------------------------------------------
# writing and reading
# ---------------------------------------------------------------------------

def odd_rows(n, seed):
    rows = R.cache_rows(n, seed, "cuda", 2.0)
    if n >= 8:
        rows[0] = 0
        rows[1, :512] *= 1e-33
        rows[2, :512] = (rows[2, :512].float() * 1e36).clamp(-3.38e38, 3.38e38).to(torch.bfloat16)
        rows[3, 5], rows[3, 130], rows[3, 300] = float("nan"), float("inf"), -float("inf")
        rows[4, :128] = float("nan")
        rows[5, :512] = 448.0  # the largest code at scale 1, and just above it
        rows[6, :512] = 450.0
        rows[7, 575] = float("nan")
    return rows


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("n,page", [(1, 1), (7, 3), (8, 16), (333, 64), (5000, 48)])
def test_write_and_read_are_exact(shla, bits, n, page):
    rows = odd_rows(n, n)
    P = n // page + 3
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(P * page, generator=g)[:n].to(torch.int32).cuda()
    width, dtype = (656, torch.uint8) if bits == 8 else (576, torch.bfloat16)
    pages = torch.full((P, page, width), 7, dtype=dtype, device="cuda")
    want = pages.clone().view(P * page, width)
    want[slots.long()] = R.row8(rows) if bits == 8 else rows
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    shla.mla_page_write(rows, slots, pages, status=status)
    assert torch.equal(pages.view(P * page, width).view(torch.uint8), want.view(torch.uint8))
    back = shla.mla_page_read(pages, slots, status=status)
    val = R.values(want[slots.long()])
    assert torch.equal(torch.isnan(back), torch.isnan(val))
    assert torch.equal(torch.nan_to_num(back.double()), torch.nan_to_num(val))
    assert status.tolist() == [0, 0]


@pytest.mark.parametrize("bits", [8, 16])
def test_skipped_and_bad_slots(shla, bits):
    rows = R.cache_rows(40, 3, "cuda")
    width, dtype = (656, torch.uint8) if bits == 8 else (576, torch.bfloat16)
    pages = torch.zeros(2, 8, width, dtype=dtype, device="cuda")
    slots = torch.full((40,), -1, dtype=torch.int32, device="cuda")
    slots[3], slots[9], slots[10], slots[11], slots[12] = 15, 16, -2, 2 ** 31 - 1, -2 ** 31
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    shla.mla_page_write(rows, slots, pages, status=status)
    assert status.tolist() == [0, 4]
    want = torch.zeros(16, width, dtype=dtype, device="cuda")
    want[15] = (R.row8(rows[3:4]) if bits == 8 else rows[3:4])[0]
    assert torch.equal(pages.view(16, width).view(torch.uint8), want.view(torch.uint8))
    back = shla.mla_page_read(pages, slots, status=status)
    assert status.tolist() == [0, 8]
    assert (back[[i for i in range(40) if i != 3]] == 0).all()
    assert torch.equal(back[3].double(), R.values(want[15:16])[0])


@pytest.mark.parametrize("bits", [8, 16])
def test_strided_rows_and_pages(shla, bits):
    # rows inside wider ones, pages inside a wider and longer pool
    wide = R.cache_rows(50, 4, "cuda").repeat(1, 2)
    rows = wide[:, 576:]
    width, dtype, more = (656, torch.uint8, 16) if bits == 8 else (576, torch.bfloat16, 8)
    big = torch.full((6, 20, width + more), 9, dtype=dtype, device="cuda")
    pages = big[1:5, 2:18, :width]
    slots = torch.arange(50, dtype=torch.int32, device="cuda") + 7
    want = big.clone()
    flat = R.row8(rows) if bits == 8 else rows
    for i in range(50):
        want[1 + (i + 7) // 16, 2 + (i + 7) % 16, :width] = flat[i]
    shla.mla_page_write(rows, slots, pages)
    assert torch.equal(big.view(torch.uint8), want.view(torch.uint8))
    out = torch.full((50, 600), 3.0, dtype=torch.bfloat16, device="cuda")
    shla.mla_page_read(pages, slots, out=out[:, :576])
    assert torch.equal(out[:, :576].double(), R.values(flat)) and (out[:, 576:] == 3).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

SHAPES = [  # new tokens, cached positions, page size
    ([1], [1], 16),
    ([1], [64], 64),
    ([1], [65], 16),
    ([1], [700], 7),
    ([1], [700], 1),
    ([1] * 5, [3, 1, 64, 129, 1000], 64),
    ([4, 1, 7], [300, 1, 7], 48),
    ([3, 0, 40], [5, 9, 500], 32),
    ([1] * 40, [100 + 37 * i for i in range(40)], 64),
    ([1], [20000], 64),
    ([128], [128], 64),
    ([129, 1], [129, 300], 16),
    ([200, 1, 257], [900, 300, 257], 64),
    ([300, 130, 1], [300, 1500, 5], 20),
]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_attention(shla, form, bits, case):
    q, kv, page = SHAPES[case]
    # what the call must not use (free pages, rows behind a sequence's end,
    # padding tokens) holds NaN
    w = R.make(q, kv, bits, page, 100 + case, pad_tokens=case % 3)
    out = torch.full_like(w["q_nope"], 7.0)
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    got = shla.mla_attend_paged(**w, form=form, out=out, status=status)
    assert got is out and status.tolist() == [0, 0]
    n = sum(q)
    check(out[:n], ref_of(w)[:n])
    assert (out[n:] == 7).all()
    again = shla.mla_attend_paged(**w, form=form)
    assert torch.equal(again[:n], out[:n])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
def test_tokens_that_see_nothing(shla, form, bits):
    # more new tokens than positions: the first ones see none of them
    w = R.make([5, 2, 1, 150], [2, 0, 0, 20], bits, 16, 7)
    got = shla.mla_attend_paged(**w, form=form)
    want = ref_of(w)
    assert (got[want.abs().amax((1, 2)) == 0] == 0).all()
    check(got, want)


@pytest.mark.parametrize("form", FORMS)
def test_nothing_to_do(shla, form):
    w = R.make([0, 0], [5, 9], 16, 16, 8, pad_tokens=4)
    out = torch.full_like(w["q_nope"], 3.0)
    shla.mla_attend_paged(**w, form=form, out=out)
    torch.cuda.synchronize()
    assert (out == 3).all()
    w["q_nope"], w["q_pe"] = w["q_nope"][:0], w["q_pe"][:0]
    assert shla.mla_attend_paged(**w, form=form).shape == (0, 128, 128)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
def test_pages_outside_the_pool_read_as_zeros(shla, form, bits):
    w = R.make([3, 200], [100, 300], bits, 16, 9)
    P = w["pages"].shape[0]
    w["page_table"][0, 0], w["page_table"][0, 6] = -1, P
    w["page_table"][1, 3], w["page_table"][1, 18] = 2 ** 31 - 1, -2 ** 31
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    got = shla.mla_attend_paged(**w, form=form, status=status)
    assert status.tolist() == [0, 4]
    check(got, ref_of(w))


@pytest.mark.parametrize("form", FORMS)
def test_lengths_are_cut_to_the_bound_and_the_table(shla, form):
    w = R.make([2, 130], [70, 200], 16, 16, 10)
    kept = w["kv_len"].clone()
    w["kv_len"] = w["kv_len"] + torch.tensor([0, 2 ** 30], dtype=torch.int32, device="cuda")
    w["max_kv"] = 200
    a = shla.mla_attend_paged(**w, form=form)
    w["kv_len"] = kept
    assert torch.equal(a, shla.mla_attend_paged(**w, form=form))
    w["max_kv"] = 5000  # the table reaches 208 positions
    w["pages"][w["page_table"][1, 12].long(), 8:] = R.cache_rows(8, 11, "cuda")
    w["kv_len"] = torch.tensor([70, 3000], dtype=torch.int32, device="cuda")
    got = shla.mla_attend_paged(**w, form=form)
    w["kv_len"] = torch.tensor([70, 208], dtype=torch.int32, device="cuda")
    check(got, ref_of(w))


@pytest.mark.parametrize("page", [64, 48, 1])
def test_8_bit_pages_that_several_tokens_read(shla, page):
    # (the absorbed form reads them once for all tokens of a call of this size)
    q, kv = [5, 1, 0, 3, 60], [7000, 129, 50, 2, 640]
    w = R.make(q, kv, 8, page, 20, pad_tokens=1)
    w["page_table"][1, 0] = -1
    out = torch.full_like(w["q_nope"], 7.0)
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    shla.mla_attend_paged(**w, form="absorbed", out=out, status=status)
    assert status.tolist() == [0, 1] and (out[69:] == 7).all()
    check(out[:69], ref_of(w)[:69])
    # lengths beyond a table that is shorter than the bound
    keep = 6720 // page
    w["page_table"] = w["page_table"][:, :keep].contiguous()
    w["max_kv"] = 9000
    got = shla.mla_attend_paged(**w, form="absorbed")
    w["kv_len"] = w["kv_len"].clamp(max=keep * page)
    check(got[:69], ref_of(w)[:69])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("q,kv", [([1] * 3, [700, 64, 130]), ([2, 130], [300, 260])])
def test_scales_of_every_size(shla, form, q, kv):
    # groups whose scales lie near 2^20, 2^-100, 1 and 2^9: wkv_b makes up for
    # the width, so that the scores stay as they are
    w = R.make(q, kv, 8, 16, 21, poison=False)
    flat = R.values(w["pages"].view(-1, 656))
    wide = torch.tensor([2.0 ** 20, 2.0 ** -100, 1.0, 2.0 ** 9], dtype=torch.float64,
                        device="cuda").repeat_interleave(128)
    flat[:, :512] *= wide
    w["pages"] = R.row8(flat.to(torch.bfloat16)).view(w["pages"].shape)
    w["wkv_b"] = (w["wkv_b"].double() / wide).to(torch.bfloat16)
    check(shla.mla_attend_paged(**w, form=form), ref_of(w))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("factor", [10.0, 0.01])
def test_wide_and_narrow_scores(shla, form, factor):
    w = R.make([3, 150], [400, 260], 16, 64, 12, scale=mi.softmax_scale() * factor)
    check(shla.mla_attend_paged(**w, form=form), ref_of(w), max(1.0, factor))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("where", [0, 77, 250])
def test_one_key_far_above_the_rest(shla, form, where):
    # the maximum jumps by about 40 at one position, in the first, a middle
    # and the last tile
    w = R.make([1, 130], [300, 300], 16, 64, 13)
    w["q_pe"][..., 0] = 8.0
    for s in range(2):
        page = int(w["page_table"][s, where // 64])
        w["pages"][page, where % 64, 512] = 5.0 * 192 ** 0.5
    check(shla.mla_attend_paged(**w, form=form), ref_of(w))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
def test_pages_past_four_gigabytes(shla, form, bits):
    # the sequence's pages lie at the end of a pool of over 2^32 bytes
    w = R.make([2, 129], [150, 200], bits, 64, 14, poison=False)
    small = w["pages"]
    row = 656 if bits == 8 else 1152
    P = (2 ** 32 + 2 ** 28) // (64 * row)
    pool = torch.empty(P, 64, small.shape[2], dtype=small.dtype, device="cuda")
    pool[P - small.shape[0]:] = small
    want = ref_of(w)
    w["pages"] = pool
    w["page_table"] += P - small.shape[0]
    check(shla.mla_attend_paged(**w, form=form), want)
    slots = torch.tensor([P * 64 - 1, P * 64 - 70], dtype=torch.int32, device="cuda")
    rows = R.cache_rows(2, 15, "cuda")
    shla.mla_page_write(rows, slots, pool)
    want = R.values(R.row8(rows)) if bits == 8 else rows.double()
    assert torch.equal(shla.mla_page_read(pool, slots).double(), want)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
def test_strided_pool(shla, form, bits):
    w = R.make([2, 140], [90, 260], bits, 16, 16)
    want = ref_of(w)
    P, ps, width = w["pages"].shape
    more = 16 if bits == 8 else 8
    big = torch.zeros(P, ps + 3, width + more, dtype=w["pages"].dtype, device="cuda")
    view = big[:, :ps, :width]
    view.copy_(w["pages"])
    w["pages"] = view
    check(shla.mla_attend_paged(**w, form=form), want)


@pytest.mark.parametrize("form", FORMS)
def test_captured_call_follows_its_inputs(shla, form):
    # one graph, replayed for other lengths, tokens and pages
    a = R.make([2, 140, 1], [90, 260, 700], 8, 16, 17, pad_tokens=40)
    b = R.make([1, 150, 32], [300, 180, 32], 8, 16, 18)
    b["pages"] = torch.cat([b["pages"], b["pages"][:1].expand(a["pages"].shape[0], -1, -1)])
    keep = {k: a[k].clone() for k in ("q_nope", "q_pe", "page_table", "cu_q", "kv_len", "pages")}
    N, S = a["q_nope"].shape[0], 3
    a["max_kv"] = 700
    ws = torch.empty(shla.mla_attend_paged_workspace_bytes(N, S, 700, 8, form), dtype=torch.uint8,
                     device="cuda")
    out = torch.full_like(a["q_nope"], 7.0)
    shla.mla_attend_paged(**a, form=form, out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        shla.mla_attend_paged(**a, form=form, out=out, ws=ws)
    for w in (b, keep, b):
        n = w["q_nope"].shape[0]
        a["q_nope"][:n], a["q_pe"][:n] = w["q_nope"], w["q_pe"]
        a["page_table"][:, :w["page_table"].shape[1]] = w["page_table"]
        a["cu_q"].copy_(w["cu_q"])
        a["kv_len"].copy_(w["kv_len"])
        a["pages"].copy_(w["pages"][:a["pages"].shape[0]])
        out.fill_(7.0)
        ws.fill_(255)  # nothing is kept there between calls
        graph.replay()
        torch.cuda.synchronize()
        ref = dict(a)
        used = int(a["cu_q"][-1])
        check(out[:used], ref_of(ref)[:used])
        assert (out[used:] == 7).all()


def test_captured_call_that_converts_its_pages(shla):
    # as above, of the absorbed form that converts 8-bit pages first; lengths grow
    # from call to call, and the workspace holds what another call left
    w = R.make([4, 0, 30], [1500, 900, 1800], 8, 64, 24, pad_tokens=3)
    N = w["q_nope"].shape[0]
    full, w["max_kv"] = w["kv_len"].clone(), 9000
    need = [shla.mla_attend_paged_workspace_bytes(N, 3, 9000, b, "absorbed") for b in (8, 16)]
    assert need[0] > need[1]
    ws = torch.empty(need[0], dtype=torch.uint8, device="cuda")
    out = torch.full_like(w["q_nope"], 7.0)
    shla.mla_attend_paged(**w, form="absorbed", out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        shla.mla_attend_paged(**w, form="absorbed", out=out, ws=ws)
    for cut in (1400, 3, 0):
        w["kv_len"].copy_((full - cut).clamp(min=0))
        out.fill_(7.0)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        check(out[:34], ref_of(w)[:34])
        assert (out[34:] == 7).all()


def test_captured_expanded_call_with_split_work(shla):
    # long enough that several pairs share an item and their outputs are joined
    w = R.make([300, 40, 0], [2500, 1300, 70], 16, 64, 28, pad_tokens=2)
    N, full, w["max_kv"] = w["q_nope"].shape[0], w["kv_len"].clone(), 4000
    ws = torch.empty(shla.mla_attend_paged_workspace_bytes(N, 3, 4000, 16, "expanded"),
                     dtype=torch.uint8, device="cuda")
    out = torch.full_like(w["q_nope"], 7.0)
    shla.mla_attend_paged(**w, form="expanded", out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        shla.mla_attend_paged(**w, form="expanded", out=out, ws=ws)
    for cut in (1200, 0, 77):
        w["kv_len"].copy_((full - cut).clamp(min=0))
        out.fill_(7.0)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        check(out[:340], ref_of(w)[:340])
        assert (out[340:] == 7).all()
        assert torch.equal(shla.mla_attend_paged(**w, form="expanded")[:340], out[:340])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
def test_sequences_that_share_pages(shla, form, bits):
    # a common prefix: the second sequence's first pages are the first one's
    w = R.make([3, 140, 1], [700, 400, 500], bits, 16, 25)
    w["page_table"][1, :12] = w["page_table"][0, :12]
    w["page_table"][2] = w["page_table"][0]
    check(shla.mla_attend_paged(**w, form=form), ref_of(w))


def test_more_positions_than_one_group_of_heads_holds(shla):
    # the expanded form in groups of 64 heads; checked for six of the 128
    w = R.make([257, 130], [35000, 34000], 16, 64, 26)
    got = shla.mla_attend_paged(**w, form="expanded")
    heads = [0, 1, 63, 64, 65, 127]
    some = {k: w[k][:, heads] for k in ("q_nope", "q_pe")}
    want = R.attend(*({**w, **some, "wkv_b": w["wkv_b"][heads]}[k] for k in REF))
    check(got[:, heads], want)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("column", [5, 500, 560])
def test_nan_stays_with_the_tokens_that_see_it(shla, form, bits, column):
    # in a latent or a rotary value of position 1037 of the first sequence, which
    # all its new tokens see; the others keep their results
    w = R.make([2, 130, 1], [1500, 260, 70], bits, 16, 27)
    good = shla.mla_attend_paged(**w, form=form)
    page, o = int(w["page_table"][0, 1037 // 16]), 1037 % 16
    if bits == 16:
        w["pages"][page, o, column] = float("nan")
    elif column < 512:
        w["pages"][page, o, 512:528].view(torch.float32)[column // 128] = float("nan")
    else:
        w["pages"][page, o, 528:].view(torch.bfloat16)[column - 512] = float("nan")
    got = shla.mla_attend_paged(**w, form=form)
    assert torch.isnan(got[:2]).all()
    assert torch.equal(got[2:], good[2:])


@pytest.mark.parametrize("form", FORMS)
def test_two_streams_at_once(shla, form):
    ws = [R.make([3, 140], [900, 500], 8, 16, 19), R.make([1, 160], [1200, 400], 16, 64, 20)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(shla.mla_attend_paged(**ws[i], form=form))
    torch.cuda.synchronize()
    for i in range(2):
        check(outs[i][0], ref_of(ws[i]))
        assert all(torch.equal(o, outs[i][0]) for o in outs[i])


def test_the_step_as_a_server_runs_it(shla):
    """Query path, cache write, paging, attention and output projection of a
    decode step, against the same steps in 64 bits from the stored rows."""
    import oracle as orc
    S, page, have = 3, 16, [37, 0, 200]
    w = R.make([1] * S, [n + 1 for n in have], 8, page, 21, poison=False)
    g = torch.Generator(device="cuda").manual_seed(22)
    rn = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    x = rn(S, 7168)
    wq_a, wq_b = rn(1536, 7168, std=7168 ** -0.5), rn(24576, 1536, std=1536 ** -0.5)
    w_kva, w_o = rn(7168, 576, std=7168 ** -0.5), rn(7168, 16384, std=16384 ** -0.5)
    one, norm = torch.ones(1536, dtype=torch.bfloat16, device="cuda"), rn(512, std=0.3)
    table = mi.rope_table(256).cuda()
    pos = torch.tensor(have, dtype=torch.int32, device="cuda")
    w["q_nope"], w["q_pe"] = shla.mla_query_proj(x, wq_a, one, 1e-6, wq_b, table, pos)
    # the new positions' rows (one batch row of S tokens, each with its own
    # position's coefficients), then into their pages
    rows = torch.zeros(1, S, 576, dtype=torch.bfloat16, device="cuda")
    shla.mla_cache_write(x[None], w_kva, norm, 1e-6, table[pos.long()].contiguous(), 0, rows)
    at = torch.tensor([int(w["page_table"][s, n // page]) * page + n % page
                       for s, n in enumerate(have)], dtype=torch.int32, device="cuda")
    shla.mla_page_write(rows[0], at, w["pages"])
    assert torch.equal(w["pages"].view(-1, 656)[at.long()], R.row8(rows[0]))
    o = shla.mla_attend_paged(**w)
    check(o, ref_of(w))
    delta = shla.mla_out_proj(o, w_o).double()
    want = o.double().flatten(1) @ w_o.double().T
    assert (delta - want).norm() <= 2.0 ** -8 * want.norm()
    kv = mi.f64(x) @ mi.f64(w_kva)
    lat = orc.rmsnorm(kv[:, :512], mi.f64(norm), 1e-6)
    assert (abs(mi.f64(rows[0])[:, :512] - lat) <= 2.0 ** -7 * abs(lat) + 1e-4).all()


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def test_refusals(shla):
    w = R.make([2], [40], 16, 16, 23)
    call = lambda **k: shla.mla_attend_paged(**{**w, **k})  # noqa: E731
    bad = [dict(q_nope=w["q_nope"].float()), dict(q_nope=w["q_nope"][:, :64]),
           dict(q_nope=w["q_nope"].transpose(0, 1)), dict(q_pe=w["q_pe"][:1]),
           dict(wkv_b=w["wkv_b"][:64]), dict(pages=w["pages"].float()),
           dict(pages=w["pages"][..., :512]), dict(pages=w["pages"].transpose(0, 1)[:, :, :570]),
           dict(page_table=w["page_table"].long()), dict(page_table=w["page_table"][:0]),
           dict(cu_q=w["cu_q"][:1]), dict(kv_len=w["kv_len"].cpu()), dict(max_kv=0),
           dict(max_kv=2 ** 24 + 1), dict(form="both"), dict(out=w["q_nope"][:1]),
           dict(ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
           dict(ws=torch.empty(1 << 20, dtype=torch.float32, device="cuda")),
           dict(ws=torch.empty(1 << 24, dtype=torch.uint8)),
           dict(status=torch.zeros(1, dtype=torch.int32, device="cuda")),
           dict(pages=torch.empty(40 * 577, dtype=torch.bfloat16, device="cuda")[1:].as_strided(
               (2, 16, 576), (16 * 576, 576, 1)))]
    for k in bad:
        with pytest.raises(shla.MLAError):
            call(**k)
    rows, slots = w["pages"].view(-1, 576)[:3], torch.zeros(3, dtype=torch.int32, device="cuda")
    for args in ((rows.float(), slots, w["pages"]), (rows[:, :512], slots, w["pages"]),
                 (rows, slots[:2], w["pages"]), (rows, slots.long(), w["pages"]),
                 (rows, slots, w["pages"].cpu()), (rows, slots, w["pages"][0])):
        with pytest.raises(shla.MLAError):
            shla.mla_page_write(*args)
    with pytest.raises(shla.MLAError):
        shla.mla_page_read(w["pages"], slots, out=rows[:2])
