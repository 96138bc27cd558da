"""mla_attend_paged refuses outputs or a workspace that share memory with what
the call reads: kernels still read queries while others store outputs.  Host
only; the addresses are never used."""
import ctypes

import pytest

N, S, MP = 300, 3, 8
SIZES = {"q": N * 128 * 128 * 2, "qp": N * 128 * 64 * 2, "w": 128 * 256 * 512 * 2,
         "table": S * MP * 4, "cu": (S + 1) * 4, "kv": S * 4, "O": N * 128 * 128 * 2}
INPUTS = ("q", "qp", "w", "table", "cu", "kv")


@pytest.fixture(scope="module")
def L():
    from sparse_head_latent_absorbed_b200 import build
    build.build()
    import sparse_head_latent_absorbed_b200._lib as m
    return m


def places():
    at, place = 1 << 40, {}
    for name, size in SIZES.items():
        place[name] = at
        at += (size + 4095) // 4096 * 4096
    place["pool"], place["ws"] = 1 << 42, 1 << 43
    return place


def call(L, place, form=0):
    p = {k: ctypes.c_void_p(v) for k, v in place.items()}
    # (a workspace of no bytes: refused even where there is a device)
    return L.LIB.mla_attend_paged(p["q"], p["qp"], p["w"], p["pool"], 0, 4, 64, 64 * 1152, 1152,
                                  p["table"], MP, p["cu"], p["kv"], S, N, 512, 1.0, form, p["O"],
                                  p["ws"], 0, None, None)


@pytest.mark.parametrize("form", [0, 1, 2])
def test_overlaps_are_refused(L, form):
    overlap = -7
    assert L.status_string(overlap) not in ("unknown status code", "")
    assert call(L, places(), form) in (-4, -6)  # apart: as far as the workspace or the device
    for name in INPUTS:
        size, base = SIZES[name], places()[name]
        # the output's first bytes on the input's last, and its last on the first
        for at in (base, (base + size - 1) // 16 * 16, (base - SIZES["O"]) // 16 * 16 + 16):
            assert call(L, {**places(), "O": at}, form) == overlap, (name, at - base)
        assert call(L, {**places(), "ws": base // 256 * 256}, form) == overlap, name
    assert call(L, {**places(), "ws": places()["O"]}, form) == overlap
    # next to each other is apart
    p = places()
    p["O"] = p["q"] - SIZES["O"]
    assert call(L, p, form) in (-4, -6)
