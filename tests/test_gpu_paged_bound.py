"""Attention over a paged cache where the host's bound on the lengths lies far
above them.  The expanded form then takes eight heads at a time, and a group's
work is less than one unit for each CTA pair: some pairs have nothing.

Tolerances: those of test_gpu_paged (the same roundings)."""
import random

import pytest
import torch

import paged_ref as R
from test_gpu_paged import check, ref_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def shla():
    import sparse_head_latent_absorbed_b200 as m
    return m


def same_whatever_the_workspace_held(shla, w, form):
    N, S = w["q_nope"].shape[0], w["kv_len"].shape[0]
    bits = 8 if w["pages"].dtype == torch.uint8 else 16
    need = shla.mla_attend_paged_workspace_bytes(N, S, w["max_kv"], bits, form)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = []
    for fill in (255, 0):
        ws.fill_(fill)
        status = torch.zeros(2, dtype=torch.int32, device="cuda")
        outs.append(shla.mla_attend_paged(**w, form=form, ws=ws, status=status))
        assert status.tolist() == [0, 0]
    check(outs[0], ref_of(w))
    assert torch.equal(outs[0], outs[1])


# one block of up to 256 tokens; two, of which one alone is long enough to be cut
CASES = [([256], [1500], 600000), ([208], [1024], 600000), ([256], [2048], 530000),
         ([230], [1281], 600000), ([1], [1100], 600000), ([1, 1], [1152, 896], 300000),
         ([3, 200], [128, 1500], 300000), ([300], [1400], 1000000), ([256], [900], 140000)]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("q,kv,bound", CASES)
def test_expanded_form_with_fewer_units_of_work_than_pairs(shla, q, kv, bound, bits):
    w = R.make(q, kv, bits, 64, 40 + len(kv))
    w["max_kv"] = bound
    same_whatever_the_workspace_held(shla, w, "expanded")


@pytest.mark.parametrize("n,kv", [(256, 1500), (208, 1024), (231, 2047)])
def test_auto_form_under_a_wide_bound(shla, n, kv):
    w = R.make([n], [kv], 16, 64, 50)
    w["max_kv"] = 600000
    same_whatever_the_workspace_held(shla, w, "auto")


@pytest.mark.parametrize("seed", range(8))
def test_random_short_work_under_a_wide_bound(shla, seed):
    rng = random.Random(seed)
    S = rng.randint(1, 4)
    q = [rng.choice((0, 1, rng.randint(1, 40), rng.randint(100, 520))) for _ in range(S)]
    q[0] = max(q[0], 1)
    kv = [rng.randint(1, 2300) for _ in range(S)]
    w = R.make(q, kv, rng.choice((8, 16)), 16, 60 + seed)
    w["max_kv"] = rng.choice((150000, 300000, 600000)) // S
    same_whatever_the_workspace_held(shla, w, "expanded")
