"""The operators around a paged key/value cache: their plain forms, the calls a
program makes of them, and the cases they are measured on.

  plan      hga_paged_plan: block tables, slot map and positions of a step,
            built on the GPU from the requests' lengths.
  rope      hga_qk_norm_rope: per-head RMS norms of q and k and the position
            rotation in one pass over a fused QKV buffer, into dense tensors
            or into the pages of a cache.
  rope_bwd  hga_qk_norm_rope_backward: the gradients of the fused buffer and
            of the norm weights.
  decode    hga_paged_decode: attention of one new token per sequence over
            its pages, with an optional window and first tokens that stay
            visible.

Head shapes are those of this repository's workloads (32/4 heads of 128, 8/8
of 64, 2/1 of 64) and a few generic ones.
"""
from __future__ import annotations

import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases --

def listed():
    qwen = dict(Hq=32, Hkv=4, D=128)
    small = dict(Hq=8, Hkv=8, D=64)
    return [
        # one decode step of a full serving batch: one new token a request,
        # a sixteenth of the rows ended and taken by new requests
        dict(name="plan_step_256", op="plan", B=256, ctx=32768, new_max=1, tokens=0, page=16,
             pad=0, release=True),
        # the prompts of 32 requests laid out at once, ragged
        dict(name="plan_prompts_32", op="plan", B=32, ctx=0, new_max=0, tokens=500001, page=64,
             pad=777, release=False),
        # the new tokens of a 16-sequence decode step, written to their pages
        dict(name="rope_step_16", op="rope", N=16, **qwen, dtype="bf16", layout="half", R=128,
             theta=1e6, scaling="none", factor=1.0, L0=0, norm=True, pages=True, page=16, pad=0,
             far=65536),
        # a 32K prompt into pages, scaled for four times its trained length
        dict(name="rope_prompt_32k", op="rope", N=32768, **qwen, dtype="bf16", layout="half",
             R=128, theta=1e6, scaling="yarn", factor=4.0, L0=32768, norm=True, pages=True,
             page=64, pad=0, far=0),
        # dense fp32 outputs of an odd length, part of the head rotated, positions halved
        dict(name="rope_f32_4097", op="rope", N=4097, **small, dtype="f32", layout="interleaved",
             R=32, theta=1e4, scaling="linear", factor=2.0, L0=0, norm=True, pages=False, page=0,
             pad=0, far=0),
        # training: gradients of a 32K sequence as the attention backward gives them (fp32)
        dict(name="rope_bwd_32k", op="rope_bwd", N=32768, **qwen, dtype="bf16", grad="f32",
             layout="half", R=128, theta=1e6, scaling="none", factor=1.0, L0=0, norm=True, far=0),
        # a short odd micro-batch with part of the head rotated
        dict(name="rope_bwd_999", op="rope_bwd", N=999, **small, dtype="bf16", grad="bf16",
             layout="interleaved", R=32, theta=1e4, scaling="none", factor=1.0, L0=0, norm=True,
             far=0),
        # one chat over a long document: few rows, the length split over the card
        dict(name="decode_1x32k", op="decode", B=1, ctx=32768, spread=1.0, **qwen, dtype="bf16",
             page=16, window=0, sinks=0),
        # the repository's decode workload's shape, every key read
        dict(name="decode_16x64k", op="decode", B=16, ctx=65536, spread=1.0, **qwen,
             dtype="bf16", page=64, window=0, sinks=0),
        # a serving batch of ragged short requests, one of them empty, MHA
        dict(name="decode_64_ragged", op="decode", B=64, ctx=6001, spread=60.0, **small,
             dtype="bf16", page=16, window=0, sinks=0),
        # a window of eight chunks and two sink chunks over long caches
        dict(name="decode_96_window", op="decode", B=96, ctx=16384, spread=8.0, **qwen,
             dtype="bf16", page=32, window=512, sinks=128),
        # fp32 cache, a small group of heads
        dict(name="decode_f32_5x2k", op="decode", B=5, ctx=2049, spread=3.0, Hq=12, Hkv=4, D=64,
             dtype="f32", page=16, window=0, sinks=0),
    ]


HEADS = [(32, 4, 128), (8, 8, 64), (2, 1, 64), (12, 4, 64), (20, 4, 128), (32, 8, 128),
         (16, 1, 64), (24, 1, 64), (4, 4, 128)]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope_bwd", "decode", "decode"])
    Hq, Hkv, D = rng.choice(HEADS)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _log(rng, 1, 1500)
        steps = rng.random() < 0.5
        return dict(op=op, B=B, ctx=_log(rng, 1, 32768) if steps else 0,
                    new_max=rng.choice([1, 1, 4]) if steps else 0,
                    tokens=0 if steps else _log(rng, 2, 500001), page=page, pad=rng.choice([0, 3, 64, 501]), release=rng.random() < 0.5)
    if op in ("rope", "rope_bwd"):
        c = dict(op=op, N=_log(rng, 1, 32768 * 36 // (Hq + 2 * Hkv) * 64 // D), Hq=Hq, Hkv=Hkv,
                 D=D, dtype=dtype)
        c["N"] = min(c["N"], 32768)
        if op == "rope_bwd":
            c["grad"] = "f32" if dtype == "f32" else rng.choice(["f32", "bf16"])
        scaling = rng.choice(["none", "linear", "yarn"])
        c.update(layout=rng.choice(["half", "interleaved"]),
                 R=rng.choice([0, 16, 32, 48, 64] + ([96, 128] if D == 128 else [])),
                 theta=rng.choice([1e4, 5e5, 1e6]), scaling=scaling,
                 factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 7.5]),
                 L0=4096 if scaling == "yarn" else 0, norm=rng.random() < 0.8)
        if op == "rope":
            pages = rng.random() < 0.5
            c.update(pages=pages, page=page if pages else 0,
                     pad=rng.choice([0, 1, 5]) if pages and c["N"] > 8 else 0)
        c["far"] = rng.choice([0, 0, 1000000])
        return c
    row = Hkv * D * (4 if dtype == "f32" else 2)
    most = (1 << 30) // row                       # keys of all sequences together
    B = _log(rng, 1, 128)
    window = rng.choice([0, 0, 64, 300, 1024])
    return dict(op=op, B=B, ctx=_log(rng, 1, min(65536, max(2, most // B))),
                spread=rng.choice([1.0, 2.0, 30.0]), Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, page=page,
                window=window, sinks=rng.choice([0, 4, 100]) if window else 0)


# --------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _ints(g, lo, hi, n):
    """n whole numbers of [lo, hi]."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "plan":
        _prepare_plan(case, g, s)
    elif case["op"] == "decode":
        _prepare_decode(case, g, s)
    else:
        _prepare_rope(case, g, s)
    return s


def _prepare_plan(c, g, s):
    """Requests with ctx tokens at most, on shuffled pages; free pages for
    about 97 of 100 of those that the step asks for, so that some have to
    wait.  tokens: the prompts' lengths together (0: up to new_max each)."""
    B, p = c["B"], c["page"]
    lens = _ints(g, 0, c["ctx"], B)
    if c["tokens"]:
        u = torch.rand(B, generator=g, device="cuda", dtype=torch.float64) + 0.05
        new = torch.floor(u / u.sum() * c["tokens"]).to(torch.int32)
        new[0] += c["tokens"] - new.sum()
        M = -(-(c["ctx"] + c["tokens"]) // p)
        P = B * (c["ctx"] // p + 1) + -(-c["tokens"] // p) + B
    else:
        new = _ints(g, 0 if c["new_max"] > 1 else 1, c["new_max"], B)
        M = -(-(c["ctx"] + c["new_max"]) // p)
        P = B * M
    held = (lens + p - 1) // p
    used, want = int(held.sum()), int(((lens + new + p - 1) // p - held).sum())
    free = max(1, want * 97 // 100)
    ids = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    j = torch.arange(M, device="cuda", dtype=torch.int32)
    table[j[None] < held[:, None]] = ids[:used]
    s["free_pages"] = torch.full((P,), -1, dtype=torch.int32, device="cuda")
    s["free_pages"][:free] = ids[used:used + free]
    s.update(lens=lens, new=new, table=table, n_slots=(c["tokens"] or B * c["new_max"]) + c["pad"],
             free_count=torch.tensor([free], dtype=torch.int32, device="cuda"), release=None)
    if c["release"]:
        s["release"] = (_ints(g, 0, 15, B) == 0).to(torch.int32)


def _prepare_rope(c, g, s):
    N, Hq, Hkv, D, t = c["N"], c["Hq"], c["Hkv"], c["D"], DT[c["dtype"]]
    W = (Hq + 2 * Hkv) * D
    chan = torch.exp(0.5 * torch.randn(W, generator=g, device="cuda"))
    s["qkv"] = (torch.randn(N, W, generator=g, device="cuda") * chan).to(t)
    for name in ("qw", "kw"):
        w = 1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")
        s[name] = w.to(t) if c["norm"] else None
    if c["far"]:
        s["pos"] = _ints(g, 0, c["far"], N)
    else:
        s["pos"] = torch.arange(N, device="cuda", dtype=torch.int32) + _ints(g, 0, 3, 1)
    s["rope"] = dict(rotary_dim=c["R"], theta=c["theta"], layout=c["layout"],
                     scaling=c["scaling"], factor=c["factor"], original_len=c["L0"])
    if c["op"] == "rope_bwd":
        gt = DT[c["grad"]]
        for name, h in (("d_q", Hq), ("d_k", Hkv), ("d_v", Hkv)):
            s[name] = torch.randn(N, h, D, generator=g, device="cuda").to(gt)
    elif c["pages"]:
        real, p = N - c["pad"], c["page"]
        P = -(-real // p) + 2
        for name in ("k_pages", "v_pages"):
            s[name] = torch.randn(P, p, Hkv, D, generator=g, device="cuda").to(t)
        at = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
        i = torch.arange(N, device="cuda", dtype=torch.int32)
        slot = at[(i // p).clamp(max=P - 1).long()] * p + i % p
        s["slot"] = torch.where(i < real, slot, torch.full_like(slot, -1))


def _prepare_decode(c, g, s):
    B, Hq, Hkv, D, p, t = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"], DT[c["dtype"]]
    M = -(-c["ctx"] // p)
    low = math.log(max(1.0, c["ctx"] / c["spread"]))
    u = torch.rand(B, generator=g, device="cuda")
    lens = torch.exp(low + u * (math.log(c["ctx"]) - low)).round().to(torch.int32)
    if c["spread"] > 1 and B > 4:
        lens[B // 2] = 0                            # a row of the batch that nobody holds
    lens[0] = c["ctx"]
    held = (lens + p - 1) // p
    used = int(held.sum())
    P = used + 1
    ids = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(M, device="cuda")[None] < held[:, None]] = ids[:used]
    s.update(lens=lens, table=table)
    s["q"] = torch.randn(B, Hq, D, generator=g, device="cuda").to(t)
    # keys of a trained head: a few directions carry the scores
    s["k_pages"] = torch.randn(P, p, Hkv, D, generator=g, device="cuda", dtype=t).mul_(1.5)
    s["v_pages"] = torch.randn(P, p, Hkv, D, generator=g, device="cuda", dtype=t)


# ------------------------------------------------------------------ run --

def run(state):
    c = state["case"]
    if c["op"] == "plan":
        return _run_plan(state)
    if c["op"] == "rope":
        return _run_rope(state)
    if c["op"] == "rope_bwd":
        return _run_rope_bwd(state)
    return _run_decode(state)


def _split(s):
    """q, k and v as views of the fused buffer."""
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    x = s["qkv"].view(-1, Hq + 2 * Hkv, D)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _run_plan(s):
    table, free_pages = s["table"], s["free_pages"]
    if s["release"] is not None:                  # released rows change the table and the stack
        table, free_pages = table.clone(), free_pages.clone()
    if own:
        import hierarchical_kv_routing_b200 as hga
        r = hga.hga_paged_plan(s["lens"], s["new"], free_pages, s["free_count"], table,
                               s["case"]["page"], s["n_slots"], release=s["release"])
    else:
        r = plan_plain(s["lens"], s["new"], free_pages, s["free_count"], table,
                       s["case"]["page"], s["n_slots"], s["release"])
    return dict(r, block_table=table, free_pages=free_pages)


def _run_rope(s):
    c = s["case"]
    q, k, v = _split(s)
    if own:
        import hierarchical_kv_routing_b200 as hga
        rope = hga.HGARope(**s["rope"])
        if not c["pages"]:
            return hga.hga_qk_norm_rope(q, k, v, s["pos"], rope, q_weight=s["qw"],
                                        k_weight=s["kw"])
        q_out, _, _ = hga.hga_qk_norm_rope(q, k, v, s["pos"], rope, q_weight=s["qw"],
                                           k_weight=s["kw"], k_pages=s["k_pages"],
                                           v_pages=s["v_pages"], slot=s["slot"])
        return q_out, s["k_pages"], s["v_pages"]
    cos, sin = angles_plain(s["pos"], s["rope"])
    q_out = rope_plain(q, s["qw"], cos, sin, s["rope"])
    k_out = rope_plain(k, s["kw"], cos, sin, s["rope"])
    if not c["pages"]:
        return q_out, k_out, v.contiguous()
    real = c["N"] - c["pad"]                      # the padded tokens come last
    at = s["slot"][:real].long()
    s["k_pages"].view(-1, c["Hkv"], c["D"])[at] = k_out[:real]
    s["v_pages"].view(-1, c["Hkv"], c["D"])[at] = v[:real]
    return q_out, s["k_pages"], s["v_pages"]


def _run_rope_bwd(s):
    c = s["case"]
    q, k, _ = _split(s)
    d = torch.empty_like(s["qkv"])
    dq, dk, dv = _split(dict(s, qkv=d))
    if own:
        import hierarchical_kv_routing_b200 as hga
        _, _, _, dqw, dkw = hga.hga_qk_norm_rope_backward(
            q, k, s["d_q"], s["d_k"], s["pos"], hga.HGARope(**s["rope"]), q_weight=s["qw"],
            k_weight=s["kw"], d_v=s["d_v"], dq=dq, dk=dk, dv=dv)
        return [d] if dqw is None else [d, dqw, dkw]
    cos, sin = angles_plain(s["pos"], s["rope"])
    gq, dqw = rope_bwd_plain(q, s["d_q"], s["qw"], cos, sin, s["rope"])
    gk, dkw = rope_bwd_plain(k, s["d_k"], s["kw"], cos, sin, s["rope"])
    dq.copy_(gq)
    dk.copy_(gk)
    dv.copy_(s["d_v"])
    return [d] if dqw is None else [d, dqw, dkw]


def _run_decode(s):
    c = s["case"]
    if own:
        import hierarchical_kv_routing_b200 as hga
        return hga.hga_paged_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                    window=c["window"], sinks=c["sinks"], want_lse=True)
    return decode_plain(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], c["window"],
                        c["sinks"])


# ---------------------------------------------------------- plain forms --

def plan_plain(lens, new, free_pages, free_count, table, page, n_slots, release):
    """Writes table and free_pages in place; the rest comes back."""
    B, M = table.shape
    P = free_pages.numel()
    dev = lens.device
    j = torch.arange(M, device=dev)[None]
    n0, lens0, new = free_count.long(), lens.long(), new.long()
    if release is not None:
        gone = (release != 0)
        give = (j < ((lens0 + page - 1) // page)[:, None]) & gone[:, None]
        at = torch.where(give, n0 + torch.cumsum(give.reshape(-1), 0).view(B, M) - 1, P)
        more = torch.cat([free_pages, free_pages.new_zeros(1)])
        more.scatter_(0, at.reshape(-1), table.reshape(-1))
        free_pages.copy_(more[:P])
        n0 = n0 + give.sum()
        lens0 = torch.where(gone, 0, lens0)
    held = (lens0 + page - 1) // page
    end = torch.cumsum(new, 0)
    cu = torch.cat([end.new_zeros(1), end])
    fits = (lens0 + new <= M * page) & (end <= n_slots)
    need = torch.where(fits, (lens0 + new + page - 1) // page - held, 0)
    cum = torch.cumsum(need, 0)
    ok = fits & ((need == 0) | (cum <= n0))
    need = torch.where(ok, need, 0)
    granted = torch.where(ok, new, 0)
    i = j - held[:, None]                         # which of the row's new pages
    mine = (i >= 0) & (i < need[:, None])
    at = (n0 - 1 - (cum - need)[:, None] - i).clamp(0, P - 1)
    table.copy_(torch.where(mine, free_pages[at], table))
    t = torch.arange(n_slots, device=dev)
    b = torch.searchsorted(end, t, right=True)
    real = b < B
    b = b.clamp(max=B - 1)
    pos = lens0[b] + t - cu[b]
    pg = table[b, (pos // page).clamp(0, M - 1)].long()
    slot = torch.where(real & (granted[b] > 0) & (pg >= 0), pg * page + pos % page, -1)
    to = dict(dtype=torch.int32)
    return dict(lens=(lens0 + granted).to(**to), free_count=(n0 - need.sum()).to(**to),
                cu_tokens=cu.to(**to), granted=granted.to(**to), slot=slot.to(**to),
                pos=torch.where(real, pos, 0).to(**to))


def omega_plain(r):
    """The turn rates of the R / 2 pairs (64 bits, host) and the magnitude."""
    R, f = r["rotary_dim"], r["factor"]
    w = [r["theta"] ** (-2.0 * i / R) for i in range(R // 2)]
    if r["scaling"] == "linear":
        return [x / f for x in w], 1.0
    if r["scaling"] == "yarn":
        def dim(turns):
            return R * math.log(r["original_len"] / (2 * math.pi * turns)) / (2 * math.log(r["theta"]))
        low, high = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), R - 1)
        span = high - low if high != low else 0.001
        ramp = [min(1.0, max(0.0, (i - low) / span)) for i in range(R // 2)]
        return [x * (1 - g) + x / f * g for x, g in zip(w, ramp)], 0.1 * math.log(f) + 1.0
    return w, 1.0


def angles_plain(pos, r):
    """cos and sin [N, 1, R / 2] in 32 bits, of angles formed in 64."""
    w, m = omega_plain(r)
    a = pos.double()[:, None, None] * torch.tensor(w, dtype=torch.float64, device=pos.device)
    return (torch.cos(a) * m).float(), (torch.sin(a) * m).float()


def _pairs(x, r):
    """(first, second) of every pair of the rotated part, and the rest."""
    R = r["rotary_dim"]
    if r["layout"] == "half":
        return x[..., :R // 2], x[..., R // 2:R], x[..., R:]
    return x[..., 0:R:2], x[..., 1:R:2], x[..., R:]


def _joined(a, b, rest, r):
    if r["layout"] != "half":
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def rope_plain(x, w, cos, sin, r):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    if r["rotary_dim"]:
        a, b, rest = _pairs(y, r)
        y = _joined(a * cos - b * sin, b * cos + a * sin, rest, r)
    return y.to(x.dtype)


def rope_bwd_plain(x, dy, w, cos, sin, r):
    g = dy.float()
    if r["rotary_dim"]:
        a, b, rest = _pairs(g, r)
        g = _joined(a * cos + b * sin, b * cos - a * sin, rest, r)
    if w is None:
        return g, None
    y = x.float()
    rs = torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)
    n = y * rs
    dw = (g * n).sum((0, 1), dtype=torch.float64).float()
    u = g * w.float()
    return rs * (u - n * (u * n).mean(-1, keepdim=True)), dw


def _visible(lens, cap, window, sinks):
    """Token of every visible key [B, n] (n from the cache's width) and which are real."""
    n = min(cap, window + sinks) if window else cap
    lo = (lens - window).clamp(min=0) if window else torch.zeros_like(lens)
    s = lo.clamp(max=sinks)
    i = torch.arange(n, device=lens.device)[None]
    tok = torch.where(i < s[:, None], i, i - s[:, None] + lo[:, None])
    return tok, i < (s + lens - lo)[:, None]


def decode_plain(q, k_pages, v_pages, table, lens, window, sinks):
    B, Hq, D = q.shape
    page, Hkv = k_pages.shape[1], k_pages.shape[2]
    tok, real = _visible(lens.long(), table.shape[1] * page, window, sinks)
    pg = torch.gather(table.long(), 1, torch.where(real, tok // page, 0))
    row = torch.where(real, pg * page + tok % page, 0)
    k = k_pages.view(-1, Hkv, D)[row].float()     # [B, n, Hkv, D]
    v = v_pages.view(-1, Hkv, D)[row].float()
    qg = q.float().view(B, Hkv, Hq // Hkv, D)
    x = torch.einsum("bhgd,bnhd->bhgn", qg, k) / math.sqrt(D)
    x = x.masked_fill(~real[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(x - top)
    z = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgn,bnhd->bhgd", p, v) / torch.where(z == 0, 1.0, z)
    lse = top + torch.log(z)
    return o.reshape(B, Hq, D).to(q.dtype), lse.reshape(B, Hq)


# ---------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None                               # whole numbers only
    if case["op"] == "decode":
        return _exact_decode(s)
    c = case
    q, k, v = (x.double() for x in _split(s))
    w, m = omega_plain(s["rope"])
    R, half = c["R"], c["layout"] == "half"
    a = s["pos"].double()[:, None] * torch.tensor(w, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(a, m), a)[:, None]        # [N, 1, R / 2]

    def turned(x, t):
        """The pairs of x as complex numbers, times t."""
        if not R:
            return x
        z = torch.complex(*((x[..., :R // 2], x[..., R // 2:R]) if half
                            else (x[..., 0:R:2], x[..., 1:R:2]))) * t
        y = x.clone()
        if half:
            y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
        else:
            y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
        return y

    if c["op"] == "rope":
        def out(x, wt):
            if wt is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["D"] + 1e-6) * wt.double()
            return turned(x, turn)
        qo, ko = out(q, s["qw"]), out(k, s["kw"])
        if not c["pages"]:
            return qo, ko, v
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        put = s["slot"] >= 0
        at = s["slot"][put].long()
        kp.view(-1, c["Hkv"], c["D"])[at] = ko[put]
        vp.view(-1, c["Hkv"], c["D"])[at] = v[put]
        return qo, kp, vp

    def back(x, dy, wt):
        gr = turned(dy.double(), turn.conj())     # the magnitude m stays in both directions
        if wt is None:
            return gr, None
        ms = (x * x).sum(-1, keepdim=True) / c["D"] + 1e-6
        u = gr * wt.double()
        dx = u / torch.sqrt(ms) - x * (u * x).sum(-1, keepdim=True) / (c["D"] * ms * torch.sqrt(ms))
        return dx, (gr * x / torch.sqrt(ms)).sum((0, 1))
    dq, dqw = back(q, s["d_q"], s["qw"])
    dk, dkw = back(k, s["d_k"], s["kw"])
    d = torch.cat([dq, dk, s["d_v"].double()], 1).reshape(c["N"], -1)
    return [d] if dqw is None else [d, dqw, dkw]


def _exact_decode(s):
    c = s["case"]
    B, Hq, Hkv, D, p = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
    o = torch.zeros(B, Hkv, Hq // Hkv, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hkv, Hq // Hkv), float("-inf"), dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        keep = torch.arange(n, device="cuda")
        if c["window"]:
            keep = keep[(keep < c["sinks"]) | (keep >= n - c["window"])]
        pg = s["table"][b][keep // p].long()
        k = s["k_pages"][pg, keep % p].double()
        v = s["v_pages"][pg, keep % p].double()
        x = torch.einsum("hgd,nhd->hgn", s["q"][b].double().view(Hkv, -1, D), k) * D ** -0.5
        lse[b] = torch.logsumexp(x, -1)
        o[b] = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), v)
    return o.view(B, Hq, D), lse.view(B, Hq)


# ----------------------------------------------------------------- work --

def work(case):
    c = case
    if c["op"] == "plan":
        tokens = c["tokens"] or c["B"] * c["new_max"]
        pages = tokens / c["page"] / (1 if c["tokens"] or c["new_max"] == 1 else 2)
        if c["release"]:
            pages += c["B"] * c["ctx"] / 2 / c["page"] / 16
        return dict(bytes=c["B"] * 24 + (tokens + c["pad"]) * 8 + pages * 8, flops=0)
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("rope", "rope_bwd"):
        rows = c["N"] * (c["Hq"] + 2 * c["Hkv"])
        if c["op"] == "rope":
            return dict(bytes=2 * rows * c["D"] * e, flops=rows * c["D"] * 8)
        ge = 4 if c["grad"] == "f32" else 2
        read = c["N"] * (c["Hq"] + c["Hkv"]) if c["norm"] else 0
        return dict(bytes=(read * e + rows * (e + ge)) * c["D"], flops=rows * c["D"] * 14)
    # lengths are spread evenly over the logarithm of [ctx / spread, ctx]
    lo = max(1.0, c["ctx"] / c["spread"])
    mean = c["ctx"] if c["ctx"] / lo < 1.001 else (c["ctx"] - lo) / math.log(c["ctx"] / lo)
    keys = min(mean, c["window"] + c["sinks"]) if c["window"] else mean
    n = c["B"] * keys
    return dict(bytes=n * c["Hkv"] * c["D"] * 2 * e + 2 * c["B"] * c["Hq"] * c["D"] * e,
                flops=4 * n * c["Hq"] * c["D"])
