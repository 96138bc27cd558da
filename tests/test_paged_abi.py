"""Host-side checks of the paged-cache entry points: every refusal comes
before any CUDA call."""
import ctypes

import pytest

vp = ctypes.c_void_p
D, ODD = vp(4096), vp(4096 + 8)


@pytest.fixture(scope="module")
def L():
    from sparse_head_latent_absorbed_b200 import build
    build.build()
    import sparse_head_latent_absorbed_b200._lib as m
    return m


def _write(L, rows=D, rstride=576, slots=D, N=4, pool=D, kind=0, P=4, ps=16, page=16 * 1152,
           row=1152):
    return L.LIB.mla_page_write(rows, rstride, slots, N, pool, kind, P, ps, page, row, None, None)


def _read(L, rows=D, rstride=576, slots=D, N=4, pool=D, kind=0, P=4, ps=16, page=16 * 1152,
          row=1152):
    return L.LIB.mla_page_read(pool, kind, P, ps, page, row, slots, N, rows, rstride, None, None)


@pytest.mark.parametrize("call", [_write, _read])
def test_page_calls(L, call):
    assert call(L, rows=None) == call(L, slots=None) == call(L, pool=None) == -1
    for bad in (dict(N=-1), dict(rstride=575), dict(kind=2), dict(kind=-1), dict(P=0), dict(ps=0),
                dict(row=1136), dict(kind=1, row=640), dict(page=-16 * 1152),
                dict(page=15 * 1152), dict(page=16 * 1152 + 16), dict(P=2 ** 27 + 1),
                dict(page=2 ** 31 * 1152)):
        assert call(L, **bad) == -2, bad
    for bad in (dict(rows=ODD), dict(pool=ODD), dict(rstride=577), dict(slots=vp(4098)),
                dict(kind=1, row=664, page=16 * 664), dict(row=1160, page=16 * 1160)):
        assert call(L, **bad) == -3, bad
    assert call(L, N=0) == 0


def _attend(L, q=D, qp=D, w=D, pool=D, kind=0, P=4, ps=16, page=16 * 1152, row=1152, table=D,
            mp=4, cu=D, kv=D, S=2, N=8, max_kv=64, form=0, O=D, ws=D, wsb=1 << 40):
    return L.LIB.mla_attend_paged(q, qp, w, pool, kind, P, ps, page, row, table, mp, cu, kv, S, N,
                                  max_kv, 1.0, form, O, ws, wsb, None, None)


def test_attend(L):
    for k in ("q", "qp", "w", "pool", "table", "cu", "kv", "O"):
        assert _attend(L, **{k: None}) == -1, k
    for bad in (dict(S=0), dict(N=0), dict(N=65536), dict(S=65536), dict(max_kv=0),
                dict(max_kv=2 ** 24 + 1), dict(form=3), dict(form=-1), dict(mp=0), dict(P=0),
                dict(N=65535, max_kv=2 ** 24, form=1), dict(S=2048, max_kv=65536, form=2)):
        assert _attend(L, **bad) == -2, bad
    for k in ("q", "qp", "w", "O", "pool"):
        assert _attend(L, **{k: ODD}) == -3, k
    assert _attend(L, ws=None) == _attend(L, ws=vp(4096 + 16)) == -4


def test_workspace_sizes(L):
    f = L.mla_attend_paged_workspace_bytes
    assert f(0, 1, 10, 16) == f(1, 0, 10, 16) == f(1, 1, 0, 16) == 0
    # q~ and the mixed latents of each token, two partial ones for each SM pair
    own = f(16, 16, 100, 16, "absorbed")
    assert own >= 2 * 16 * 128 * 512 * 2 + 2 * 128 * 512 * 2
    # 8-bit pages that several tokens a sequence read are staged as bf16 rows
    assert f(16, 16, 100, 8, "absorbed") == own == f(16, 5, 100, 8, "absorbed")
    assert f(16, 5, 16384, 8, "absorbed") >= own + 5 * 16384 * 1152
    assert own == f(16, 6, 16384, 8, "absorbed") == f(16, 5, 16383, 8, "absorbed")
    assert own == f(16, 5, 16384, 16, "absorbed") == f(16, 5, 1 << 20, 8, "absorbed")
    # keys and values of 128 heads, of fewer where they would pass 4 GiB
    assert f(128, 1, 128, 8) >= 256 * (1152 + 128 * 512)
    assert f(512, 1, 2 ** 17, 16) < 2 ** 17 * 1152 + 2 ** 32 + 21 * 2 ** 20
    # the form that "auto" takes
    for n, kv in ((112, 1024), (160, 1025), (160, 4096), (208, 4097)):
        assert f(n - 1, 1, kv, 16) == f(n - 1, 1, kv, 16, "absorbed")
        assert f(n, 1, kv, 16) == f(n, 1, kv, 16, "expanded") != f(n, 1, kv, 16, "absorbed")
    # not the expanded form where it is refused
    assert f(60000, 200, 2 ** 20, 16) == f(60000, 200, 2 ** 20, 16, "absorbed") > 0
    assert f(60000, 200, 2 ** 20, 16, "expanded") == 0
    for bad in (dict(form="other"), dict(bits=4)):
        with pytest.raises(L.MLAError):
            f(1, 1, 10, **{"bits": 16, **bad})


def test_scale(L):
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert L.LIB.mla_attend_paged(D, D, D, D, 0, 4, 16, 16 * 1152, 1152, D, 4, D, D, 1, 1, 64,
                                      s, 0, D, D, 1 << 40, None, None) == -2
