"""Attention over millions of cached positions.

All positions hold the same latent c, under rotary keys that give them unequal
weights: whatever the weights, O = W_UV c.  An accumulator that adds with
truncation falls short of it in proportion to the additions: 2^-23 at most for
each product of 16 positions, 2^-10 for the 2^17 positions of a run, and the
runs are added to nearest.  So <O, W_UV c> / |W_UV c|^2 may be off by 2^-10,
and by what the roundings to bf16 leave on average over 16384 outputs, which is
2^-9 / sqrt(3) / 128 < 1e-5 each."""
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE, POOL = 64, 1 << 18  # positions of the pool: a table names each page many times


@pytest.fixture(scope="module")
def shla():
    import sparse_head_latent_absorbed_b200 as m
    return m


def call(shla, form, bits, q_lens, kv_lens, seed, page=PAGE):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rows = torch.empty(POOL, 576, dtype=torch.bfloat16, device="cuda")
    c = rn(512)
    # (values that the 8-bit pages hold too: four significant bits)
    m, e = torch.frexp(c)
    c = torch.ldexp((m * 16).round() / 16, e.clamp(min=-3))
    rows[:, :512], rows[:, 512:] = c, rn(POOL, 64)
    if bits == 16:
        pages = rows.view(-1, page, 576)
    else:
        pages = torch.empty(POOL // page, page, 656, dtype=torch.uint8, device="cuda")
        slots = torch.arange(POOL, dtype=torch.int32, device="cuda")
        shla.mla_page_write(rows, slots, pages)
        assert torch.equal(shla.mla_page_read(pages, slots), rows)
    N, S = sum(q_lens), len(q_lens)
    wide = -(-max(kv_lens) // page)
    table = torch.randint(POOL // page, (S, wide), generator=g, device="cuda").int()
    w = (rn(128, 256, 512) * 512 ** -0.5).to(torch.bfloat16)
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = shla.mla_attend_paged(
        (rn(N, 128, 128) * 0.1).to(torch.bfloat16), (rn(N, 128, 64) * 1.5).to(torch.bfloat16), w,
        pages, table, torch.tensor([0] + q_lens).cumsum(0).int().cuda(),
        torch.tensor(kv_lens, dtype=torch.int32, device="cuda"), 192 ** -0.5, max(kv_lens),
        form=form, status=status)
    want = torch.einsum("hdc,c->hd", w[:, 128:].double(), c.double())
    assert status.tolist() == [0, 0]
    for a in range(0, N, 1024):
        got = out[a:a + 1024].double()
        short = 1 - (got * want).sum((1, 2)) / want.square().sum()
        assert short.abs().max() <= 2.0 ** -10 + 4e-5
        assert (got - want).norm(dim=(1, 2)).max() <= 1e-2 * want.norm()


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("q,kv", [
    ([148], [1 << 22]),              # a pair holds whole tokens
    ([1] * 150, [1 << 20] * 75 + [(1 << 20) - 9000] * 75),
    ([1, 2], [1 << 22, 130]),        # all share a token
    ([3, 80, 70], [(1 << 17) + 128 * 1024, (1 << 17) + 1, 1 << 17]),  # runs that just end
])
def test_absorbed(shla, q, kv, bits):
    call(shla, "absorbed", bits, q, kv, 1)


@pytest.mark.parametrize("q,kv", [
    ([8192], [1 << 20]),             # a pair holds whole items
    ([1000], [(1 << 18) + 77]),
    ([300], [1 << 22]),              # all share an item
])
def test_expanded(shla, q, kv):
    call(shla, "expanded", 16, q, kv, 2)


def test_the_longest_sequence_in_the_smallest_pages(shla):
    # 2^24 positions under 148 tokens: a pair's second token waits 0.6 s for the first
    # one's queries to be done with
    call(shla, "absorbed", 16, [148], [1 << 24], 3, page=1)
