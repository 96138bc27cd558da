"""The paged-cache operators as they are measured: cases, inputs, plain forms and 64-bit values.

Three operators work on one paged latent cache (576 values a position: a
512-wide latent and a 64-wide rotary key):

  write    new positions' rows into their slots, in 8 bits with a power-of-two
           scale for each 128 latent values, or unchanged in 16 bits
  read     rows at given slots back as bf16
  attend   the new tokens of each sequence against all of its cached positions
           (causal among the new ones), 128 heads, from one token a sequence to
           chunks of thousands

``run`` computes them from elementary torch operations, or, where ``own`` is
true, through this repository's entry points.
"""
import math

import torch

own = False

H, C, R, D = 128, 512, 64, 128     # heads, latent, rotary key, per-head key / value width
ROW16, ROW8 = C + R, C + 16 + 2 * R  # elements of a 16-bit row, bytes of an 8-bit one
SCALE = (D + R) ** -0.5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _write(rows, bits, page, **more):
    return dict(op="write", rows=rows, bits=bits, page=page, **more)


def _read(rows, bits, page, **more):
    return dict(op="read", rows=rows, bits=bits, page=page, **more)


def _attend(seqs, q_lo, q_hi, kv_lo, kv_hi, bits, page, **more):
    return dict(op="attend", seqs=seqs, q_lo=q_lo, q_hi=q_hi, kv_lo=kv_lo, kv_hi=kv_hi, bits=bits,
                page=page, **more)


def listed():
    return [
        # a decode step's new positions, one for each of 128 sequences
        _write(128, 8, 64, name="write8_step"),
        # the positions of one large prefill batch
        _write(16384, 8, 64, name="write8_prefill"),
        # a short prefix read back, and a whole long context
        _read(500, 8, 64, name="read8_prefix"),
        _read(32768, 8, 64, name="read8_context"),
        # one user, one new token, a short conversation: latency
        _attend(1, 1, 1, 700, 700, 16, 16, name="attend16_one"),
        # a decode step of 64 sequences of mixed length, 16-bit pages
        _attend(64, 1, 1, 1000, 8000, 16, 64, name="attend16_step"),
        # the same for 128 sequences up to 16k positions, 8-bit pages
        _attend(128, 1, 1, 1000, 16000, 8, 64, name="attend8_step"),
        # a step with three drafted tokens a sequence to be verified
        _attend(32, 4, 4, 2000, 6000, 8, 64, name="attend8_draft"),
        # three fresh prompts of odd lengths: every key is also a new token
        _attend(3, 700, 2000, 0, 0, 16, 64, name="attend16_prompts"),
        # one prefill chunk in the middle of a prompt
        _attend(1, 512, 512, 6000, 6000, 16, 64, name="attend16_chunk"),
        # a large chunk at the end of a long 8-bit context
        _attend(1, 1024, 1024, 32768, 32768, 8, 64, name="attend8_chunk_long"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("write", "read", "step", "step", "draft", "chunk", "chunk", "prompts"))
    bits, page = rng.choice((8, 16)), rng.choice((16, 32, 48, 64, 64, 128))
    if kind == "write":
        return _write(_log(rng, 1, 20000), bits, page)
    if kind == "read":
        return _read(_log(rng, 1, 40000), bits, page)
    if kind == "step":
        seqs, kv = _log(rng, 1, 128), _log(rng, 16, 16000)
        return _attend(seqs, 1, 1, max(1, kv // rng.choice((1, 2, 8))), kv, bits, page)
    if kind == "draft":
        q = rng.randint(2, 24)
        seqs, kv = _log(rng, 1, 32), _log(rng, 64, 8000)
        return _attend(seqs, rng.choice((1, q)), q, max(q, kv // 3), max(q, kv), bits, page)
    if kind == "chunk":
        q = _log(rng, 130, 1024)
        kv = q + _log(rng, 1, 30000)
        return _attend(rng.choice((1, 1, 2)) if kv < 12000 else 1, q, q, max(q, kv // 2), kv, bits, page)
    q = _log(rng, 130, 2000)
    return _attend(rng.randint(1, 4), max(1, q // 3), q, 0, 0, bits, page)


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi] in a fixed mixed order, hi among them."""
    return [hi - int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _lengths(case):
    """New tokens and cached positions (the new ones included) of each sequence."""
    q = _spread(case["seqs"], case["q_lo"], case["q_hi"])
    kv = _spread(case["seqs"], case["kv_lo"], case["kv_hi"])
    return q, [max(a, b) for a, b in zip(q, kv)]


def work(case):
    row = ROW8 if case["bits"] == 8 else 2 * ROW16
    if case["op"] != "attend":
        return {"bytes": case["rows"] * (row + 2 * ROW16 + 4), "flops": case["rows"] * C}
    q, kv = _lengths(case)
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(q, kv))
    up = 2 * H * 2 * D * C  # keys and values of one position, or the fold and the value product of one token
    absorbed = sum(q) * up + pairs * 2 * H * (C + R + C)
    expanded = sum(kv) * up + pairs * 2 * H * (D + R + D)
    moved = sum(kv) * row + sum(q) * 2 * H * (D + R + D) + 2 * H * 2 * D * C
    return {"bytes": moved, "flops": min(absorbed, expanded)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(torch.bfloat16)


def _rows(n, gen):
    """Cache rows: normalised latents under a per-feature weight, rotary keys of unit variance."""
    weight = torch.exp2(torch.randn(C, generator=gen, device="cuda") * 0.5)
    x = torch.randn(n, ROW16, generator=gen, device="cuda")
    x[:, :C] *= weight / weight.square().mean().sqrt()
    return x.to(torch.bfloat16)


def _pool(case, positions):
    """Pages of a pool that holds a few more than the positions need, and their order in it."""
    need = -(-positions // case["page"])
    return need + need // 8 + 2


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ps = case["page"]
    if case["op"] != "attend":
        n = case["rows"]
        pool = _pool(case, n)
        order = torch.randperm(pool, generator=gen, device="cuda")
        i = torch.arange(n, device="cuda")
        slots = (order[i // ps] * ps + i % ps).to(torch.int32)
        rows = _rows(n, gen)
        width, dtype = (ROW8, torch.uint8) if case["bits"] == 8 else (ROW16, torch.bfloat16)
        pages = torch.zeros(pool, ps, width, dtype=dtype, device="cuda")
        if case["op"] == "read":
            _put(pages, rows, slots)
        return dict(case=case, rows=rows, slots=slots, pages=pages)
    q, kv = _lengths(case)
    most = max(-(-n // ps) for n in kv)
    pool = _pool(case, sum(-(-n // ps) * ps for n in kv))
    order = torch.randperm(pool, generator=gen, device="cuda")
    table = torch.zeros(len(kv), most, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(kv):
        np_ = -(-n // ps)
        table[s, :np_] = order[at:at + np_]
        at += np_
    if case["bits"] == 8:
        pages = torch.zeros(pool, ps, ROW8, dtype=torch.uint8, device="cuda")
        _put(pages, _rows(pool * ps, gen), torch.arange(pool * ps, device="cuda", dtype=torch.int32))
    else:
        pages = _rows(pool * ps, gen).view(pool, ps, ROW16)
    cu = torch.tensor([0] + q).cumsum(0).to(torch.int32).cuda()
    return dict(case=case, pages=pages, table=table, cu_q=cu, q_max=max(q), max_kv=max(kv),
                kv_len=torch.tensor(kv, dtype=torch.int32, device="cuda"),
                q_nope=_normal((sum(q), H, D), gen), q_pe=_normal((sum(q), H, R), gen),
                wkv_b=_normal((H, 2 * D, C), gen, C ** -0.5))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _values(pages):
    """What a pool of either kind holds, as views."""
    if pages.dtype == torch.bfloat16:
        return pages
    return {"latent": pages[..., :C].view(torch.float8_e4m3fn),
            "scale": pages[..., C:C + 16].view(torch.float32),
            "rotary": pages[..., C + 16:].view(torch.bfloat16)}


def run(state):
    op = state["case"]["op"]
    if own:
        import sparse_head_latent_absorbed_b200 as shla
        if op == "write":
            shla.mla_page_write(state["rows"], state["slots"], state["pages"])
            return _values(state["pages"])
        if op == "read":
            return shla.mla_page_read(state["pages"], state["slots"])
        return shla.mla_attend_paged(state["q_nope"], state["q_pe"], state["wkv_b"],
                                     state["pages"], state["table"], state["cu_q"],
                                     state["kv_len"], SCALE, state["max_kv"])
    if op == "write":
        _put(state["pages"], state["rows"], state["slots"])
        return _values(state["pages"])
    if op == "read":
        return _get(state["pages"], state["slots"])
    return _attend_plain(state)


def _two_to(n):
    """2^n in 32 bits from its exponent field (exp2 rounds), n in [-126, 127]."""
    return ((n.to(torch.int32) + 127) << 23).view(torch.float32)


def _put(pages, rows, slots):
    flat = pages.view(-1, pages.shape[-1])
    if pages.dtype == torch.bfloat16:
        flat.index_copy_(0, slots.long(), rows)
        return
    x = rows[:, :C].float().view(-1, 4, 128)
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1)
    n = (e - 9 + (m > 0.875)).clamp(-117, 119)
    n = torch.where(top > 0, n, -117)
    scale = _two_to(n)
    code = (x * _two_to(-n)[..., None]).to(torch.float8_e4m3fn).view(-1, C)
    flat.index_copy_(0, slots.long(), torch.cat([code.view(torch.uint8), scale.view(torch.uint8),
                                                 rows[:, C:].contiguous().view(torch.uint8)], 1))


def _get(pages, slots):
    got = pages.view(-1, pages.shape[-1])[slots.long()]
    if pages.dtype == torch.bfloat16:
        return got
    x = got[:, :C].contiguous().view(torch.float8_e4m3fn).float().view(-1, 4, 128)
    x = x * got[:, C:C + 16].contiguous().view(torch.float32)[..., None]
    return torch.cat([x.view(-1, C).to(torch.bfloat16),
                      got[:, C + 16:].contiguous().view(torch.bfloat16)], 1)


def _attend_plain(state):
    """Padded over sequences: keys [S, K, 576], queries [S, Q, 128, .], one masked softmax."""
    ps = state["case"]["page"]
    S, K, Q = state["kv_len"].shape[0], state["max_kv"], state["q_max"]
    j = torch.arange(K, device="cuda")
    there = j < state["kv_len"][:, None]
    slots = torch.where(there, state["table"].long()[:, j // ps] * ps + j % ps, 0)
    keys = _get(state["pages"], slots.view(-1)).view(S, K, ROW16).float() * there[..., None]
    start, n = state["cu_q"][:-1].long(), state["cu_q"].diff()
    i = torch.arange(Q, device="cuda")
    mine = i < n[:, None]
    at = torch.where(mine, start[:, None] + i, 0)
    lim = (state["kv_len"] - n)[:, None] + i + 1
    q, qr = state["q_nope"][at].float(), state["q_pe"][at].float()  # [S, Q, H, .]
    w_k, w_v = state["wkv_b"][:, :D].float(), state["wkv_b"][:, D:].float()
    lat, rot = keys[..., :C], keys[..., C:]
    if Q < D:  # few tokens a sequence: the queries go into the latent space, the values come out of it
        q = torch.einsum("sqhd,hdc->shqc", q, w_k)
        s = torch.matmul(q.reshape(S, H * Q, C), lat.transpose(1, 2))
    else:  # many: keys and values of every head
        k = torch.einsum("skc,hdc->shkd", lat, w_k)
        s = torch.matmul(q.transpose(1, 2), k.transpose(2, 3)).view(S, H * Q, K)
    s += torch.matmul(qr.transpose(1, 2).reshape(S, H * Q, R), rot.transpose(1, 2))
    s = s.mul_(SCALE).view(S, H, Q, K)
    s.masked_fill_((j >= lim[..., None])[:, None], float("-inf"))
    s.sub_(s.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    total = s.sum(-1, keepdim=True)
    if Q < D:
        o = torch.matmul(s.view(S, H * Q, K), lat).view(S, H, Q, C) / total.clamp_min(1e-30)
        o = torch.einsum("shqc,hdc->sqhd", o, w_v)
    else:
        v = torch.einsum("skc,hdc->shkd", lat, w_v)
        o = (torch.matmul(s, v) / total.clamp_min(1e-30)).transpose(1, 2)
    out = torch.zeros_like(state["q_nope"], dtype=torch.bfloat16)
    return out.index_put_((at[mine],), o[mine].to(torch.bfloat16))


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------

def _power(n):
    """2^n in 64 bits, exactly."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _quantised(x):
    """Rounds each group of 128 to four significant bits under a power-of-two scale, by the definition."""
    x = x.double().view(-1, 4, 128)
    top = x.abs().amax(-1, keepdim=True)
    # (a bf16 value that is not 448 2^n is off it by 2^-8 of it, the logarithm by far less)
    n = torch.ceil(torch.log2(top.clamp_min(1e-300) / 448.0) - 1e-6).clamp(-117, 119)
    scale = _power(n)
    y = (x / scale).abs()
    step = _power(torch.floor(torch.log2(y.clamp_min(2.0 ** -6)) + 1e-6) - 3.0)
    return torch.copysign(torch.round(y / step) * step, x).view(-1, C), scale.view(-1, 4)


def exact(case, seed):
    state = prepare(case, seed)
    pages, ps = state["pages"], case["page"]
    if case["op"] == "write":
        flat, slots, rows = pages.view(-1, pages.shape[-1]), state["slots"].long(), state["rows"]
        if case["bits"] == 16:
            want = flat.double()
            want[slots] = rows.double()
            return want.view(pages.shape)
        lat = torch.zeros(flat.shape[0], C, dtype=torch.float64, device="cuda")
        scale = torch.zeros(flat.shape[0], 4, dtype=torch.float64, device="cuda")
        rot = torch.zeros(flat.shape[0], R, dtype=torch.float64, device="cuda")
        lat[slots], scale[slots] = _quantised(rows[:, :C])
        rot[slots] = rows[:, C:].double()
        return {"latent": lat.view(-1, ps, C), "scale": scale.view(-1, ps, 4),
                "rotary": rot.view(-1, ps, R)}
    if case["op"] == "read":
        rows = state["rows"].double()
        if case["bits"] == 8:
            lat, scale = _quantised(state["rows"][:, :C])
            rows[:, :C] = (lat.view(-1, 4, 128) * scale[..., None]).view(-1, C)
        return rows
    q_len, kv_len = _lengths(case)
    if work(case)["flops"] > 2e13:
        return None
    w_k, w_v = state["wkv_b"][:, :D].double(), state["wkv_b"][:, D:].double()
    out = torch.zeros(sum(q_len), H, D, dtype=torch.float64, device="cuda")
    at = 0
    for s, (n, m) in enumerate(zip(q_len, kv_len)):
        row = pages[state["table"][s, :-(-m // ps)].long()].flatten(0, 1)[:m]
        if case["bits"] == 8:
            lat = row[:, :C].contiguous().view(torch.float8_e4m3fn).double()
            lat = (lat.view(m, 4, 128) * row[:, C:C + 16].contiguous().view(torch.float32).double()[..., None]).view(m, C)
            rot = row[:, C + 16:].contiguous().view(torch.bfloat16).double()
        else:
            lat, rot = row[:, :C].double(), row[:, C:].double()
        q, qr = state["q_nope"][at:at + n].double(), state["q_pe"][at:at + n].double()
        seen = torch.arange(m, device="cuda") <= torch.arange(m - n, m, device="cuda")[:, None]
        for h in range(0, H, 16):  # sixteen heads at a time: keys and values of every position
            k = torch.einsum("kc,hdc->hkd", lat, w_k[h:h + 16])
            v = torch.einsum("kc,hdc->hkd", lat, w_v[h:h + 16])
            z = torch.einsum("qhd,hkd->hqk", q[:, h:h + 16], k)
            z += torch.einsum("qhr,kr->hqk", qr[:, h:h + 16], rot)
            z = (z * SCALE).masked_fill_(~seen, float("-inf"))
            out[at:at + n, h:h + 16] = torch.einsum("hqk,hkd->qhd", torch.softmax(z, -1), v)
        at += n
    return out
