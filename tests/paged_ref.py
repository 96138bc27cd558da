"""Plain 64-bit forms of the paged-cache operators (torch, any device), and
seeded inputs for their tests.  Shares nothing with the CUDA library."""
import math

import torch

import mla_inputs as mi

# every finite e4m3 magnitude, by its code: exponent field 0 is subnormal
# (mantissa * 2^-9), others (1 + mantissa / 8) * 2^(field - 7); code 127 is NaN
E4M3 = torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7)
                     for c in range(127)], dtype=torch.float64)


def scales(lat):
    """[N, 512] -> scale of each group of 128: the least 2^n, n in [-117, 119],
    with max |x| <= 448 * 2^n; NaN for a group with a NaN or an infinity."""
    x = lat.double().reshape(-1, 4, 128)
    top = x.abs().amax(-1)
    n = torch.full_like(top, -117.0)
    for k in range(-117, 119):
        n += (top > 448.0 * 2.0 ** k).double()
    s = torch.pow(2.0, n.cpu()).to(lat.device)
    return torch.where(torch.isfinite(x).all(-1), s, torch.nan)


def codes(lat, scale):
    """Nearest e4m3 code of each value over its group's scale, ties to the even
    code, by search in the table; 0 where the scale is NaN."""
    table = E4M3.to(lat.device)
    y = (lat.double().reshape(-1, 4, 128) / scale[..., None]).reshape(lat.shape[0], -1)
    fin = torch.isfinite(y)
    a = torch.where(fin, y.abs(), 0.0).clamp(max=448.0)
    hi = torch.searchsorted(table, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - table[lo], table[hi] - a
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = torch.where(fin, pick | torch.where(torch.signbit(y), 128, 0), 0)
    return c.to(torch.uint8)


def row8(rows):
    """bf16 [N, 576] -> uint8 [N, 656]."""
    s = scales(rows[:, :512])
    return torch.cat([codes(rows[:, :512], s), s.float().view(torch.uint8),
                      rows[:, 512:].contiguous().view(torch.uint8)], 1)


def values(flat):
    """Rows of a pool of either kind (flattened to [slots, width]) in 64 bits."""
    if flat.dtype == torch.bfloat16:
        return flat.double()
    c = flat[:, :512].long()
    m = torch.cat([E4M3, E4M3.new_full((1,), math.nan)]).to(flat.device)[c & 127]
    v = torch.where(c >= 128, -m, m)
    s = flat[:, 512:528].contiguous().view(torch.float32).double()
    lat = (v.view(-1, 4, 128) * s[..., None]).view(-1, 512)
    return torch.cat([lat, flat[:, 528:].contiguous().view(torch.bfloat16).double()], 1)


def attend(q_nope, q_pe, wkv_b, pages, table, cu_q, kv_len, scale, out=None):
    """Expanded form by the definition, in 64 bits, one sequence at a time."""
    P, ps, _ = pages.shape
    val = values(pages.reshape(P * ps, -1))
    out = torch.zeros(q_nope.shape, dtype=torch.float64, device=q_nope.device) if out is None else out
    w_k, w_v = wkv_b[:, :128].double(), wkv_b[:, 128:].double()
    cu, kv = cu_q.tolist(), kv_len.tolist()
    for s, n_kv in enumerate(kv):
        a, n = cu[s], cu[s + 1] - cu[s]
        if n == 0:
            continue
        out[a:a + n] = 0
        if n_kv == 0:
            continue
        j = torch.arange(n_kv, device=val.device)
        page = table[s].long()[j // ps]
        ok = (page >= 0) & (page < P)
        row = torch.where(ok[:, None], val[torch.where(ok, page, 0) * ps + j % ps], 0.0)
        k = torch.einsum("tc,hdc->htd", row[:, :512], w_k)
        v = torch.einsum("tc,hdc->htd", row[:, :512], w_v)
        z = torch.einsum("qhd,htd->hqt", q_nope[a:a + n].double(), k)
        z += torch.einsum("qhr,tr->hqt", q_pe[a:a + n].double(), row[:, 512:])
        lim = n_kv - n + 1 + torch.arange(n, device=val.device)
        hide = j[None, :] >= lim[:, None]
        p = torch.softmax((z * scale).masked_fill(hide, -math.inf), -1)
        o = torch.einsum("hqt,htd->qhd", torch.where(hide, 0.0, p), v)
        out[a:a + n] = torch.where((lim > 0)[:, None, None], o, 0.0)
    return out


def cache_rows(n, seed, device, spread=1.0):
    g = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn(n, 576, generator=g, device=device)
    x[:, :512] *= torch.exp2(spread * torch.randn(512, generator=g, device=device))
    return x.to(torch.bfloat16)


def make(q_lens, kv_lens, bits, page, seed, device="cuda", extra_pages=3, pad_tokens=0,
         poison=True, scale=None):
    """A filled pool, its table in shuffled page order, and queries.  Everything
    the call must not use (free pages, rows behind a sequence's end, padding
    tokens) is NaN with `poison`."""
    g = torch.Generator(device=device).manual_seed(seed)
    used = [-(-n // page) for n in kv_lens]
    P = sum(used) + extra_pages
    order = torch.randperm(P, generator=g, device=device)
    table = torch.full((len(kv_lens), max(used + [1])), -7, dtype=torch.int32, device=device)
    bad = float("nan") if poison else 0.0
    rows = torch.full((P * page, 576), bad, dtype=torch.bfloat16, device=device)
    at = 0
    for s, n in enumerate(kv_lens):
        table[s, :used[s]] = order[at:at + used[s]].int()
        at += used[s]
        j = torch.arange(n, device=device)
        slot = table[s].long()[j // page] * page + j % page
        rows[slot] = cache_rows(n, seed * 1000 + s, device, 0.5)
    if bits == 8:
        pages = row8(rows).view(P, page, 656)
    else:
        pages = rows.view(P, page, 576)
    N = sum(q_lens) + pad_tokens
    q_nope = torch.randn(N, 128, 128, generator=g, device=device).to(torch.bfloat16)
    q_pe = torch.randn(N, 128, 64, generator=g, device=device).to(torch.bfloat16)
    if pad_tokens and poison:
        q_nope[sum(q_lens):] = bad
        q_pe[sum(q_lens):] = bad
    wkv_b = (torch.randn(128, 256, 512, generator=g, device=device) * 512 ** -0.5).to(torch.bfloat16)
    cu = torch.tensor([0] + q_lens).cumsum(0).to(torch.int32).to(device)
    kv = torch.tensor(kv_lens, dtype=torch.int32, device=device)
    return dict(q_nope=q_nope, q_pe=q_pe, wkv_b=wkv_b, pages=pages, page_table=table, cu_q=cu,
                kv_len=kv, scale=mi.softmax_scale() if scale is None else scale,
                max_kv=max(kv_lens + [1]))
