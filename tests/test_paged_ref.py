"""The plain 64-bit forms that the paged-cache kernels are held to: quantised
rows against exhaustive search, attention against the oracle's decode."""
import numpy as np
import pytest
import torch

import mla_inputs as mi
import oracle as orc
import paged_ref as R


def test_codes_are_the_nearest_values():
    rows = R.cache_rows(40, 1, "cpu", 2.0)
    rows[3] = 0
    rows[4, :512] *= 1e-30
    rows[5, 0] = 3.0e38
    rows[6, 7], rows[6, 8], rows[6, 9] = float("inf"), float("nan"), -float("inf")
    flat = R.row8(rows)
    got = R.values(flat)
    x = rows[:, :512].double()
    s = R.scales(rows[:, :512]).repeat_interleave(128, 1)
    fin = torch.isfinite(s)
    assert torch.isnan(got[:, :512][~fin]).all() and (~fin).sum() == 128 and not fin[6, 0]
    # no value of the grid (all magnitudes times the scale) is nearer
    best = (x.abs()[..., None] - R.E4M3 * s[..., None]).abs().amin(-1)
    assert torch.equal((got[:, :512] - x).abs()[fin], best[fin])
    # a half step of four significant bits, 2^-4 of the value, at most; below
    # the normal range 2^-10 of the scale
    lim = torch.maximum(x.abs() * 2.0 ** -4, s * 2.0 ** -10)
    assert ((got[:, :512] - x).abs() <= lim)[fin & (x.abs() < 448 * s)].all()
    assert torch.equal(flat[:, 528:].contiguous().view(torch.bfloat16), rows[:, 512:])


def test_code_values_are_exact_in_bf16():
    rows = R.cache_rows(20, 2, "cpu", 3.0)
    rows[1, :512] = (rows[1, :512].float() * 1e-36).to(torch.bfloat16)
    rows[2, :512] = (rows[2, :512].float() * 1e35).to(torch.bfloat16)
    v = R.values(R.row8(rows))
    assert torch.equal(v.to(torch.bfloat16).double(), v)


@pytest.mark.parametrize("bits", [16, 8])
def test_attention_is_the_oracles_decode(bits):
    # token i of a sequence is a decode over the positions it sees
    w = R.make([2, 1, 3], [9, 4, 3], bits, 4, 5, device="cpu")
    got = R.attend(*(w[k] for k in ("q_nope", "q_pe", "wkv_b", "pages", "page_table", "cu_q",
                                    "kv_len", "scale")))
    val = R.values(w["pages"].reshape(-1, w["pages"].shape[-1])).numpy()
    r = 0
    for s, (n, kv) in enumerate(((2, 9), (1, 4), (3, 3))):
        slot = [int(w["page_table"][s, t // 4]) * 4 + t % 4 for t in range(kv)]
        c = val[slot][None]
        for i in range(n):
            lim = kv - n + i + 1
            want = orc.decode_absorbed(mi.f64(w["q_nope"][r:r + 1]), mi.f64(w["q_pe"][r:r + 1]),
                                       mi.f64(w["wkv_b"]), c[..., :512], c[..., 512:],
                                       np.arange(lim)[None], np.array([lim]), w["scale"])
            assert np.allclose(got[r].numpy(), want[0], rtol=0, atol=1e-12)
            r += 1


def test_tokens_without_keys_give_zeros_and_padding_is_left():
    w = R.make([3, 0, 2], [1, 0, 0], 16, 4, 6, device="cpu", pad_tokens=2)
    out = torch.full((7, 128, 128), 5.0, dtype=torch.float64)
    R.attend(*(w[k] for k in ("q_nope", "q_pe", "wkv_b", "pages", "page_table", "cu_q", "kv_len",
                              "scale")), out=out)
    assert (out[[0, 1, 3, 4]] == 0).all() and (out[2] != 0).any() and (out[5:] == 5).all()
