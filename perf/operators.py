"""Measured cases of the operators over a paged key-value cache: appending keys and values with the
position rotation, attention of new tokens over the cache (all pages, or listed ones) and the choice
of pages by a score from per-channel key bounds.

Every case is one pass of one operator.  `run` computes it in a plain form (elementary torch
operations in fp32, fp64 for the page scores) or, where `own` is set, by this package's calls.
"""
import math

import torch

own = False

GOLDEN = 0.6180339887498949


# --------------------------------------------------------------------------- cases
def _append(name, **kw):
    c = dict(name=name, op="append", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, page=64, new=1, old=0,
             spread="even", rot=128, interleaved=False, bounds=True)
    c.update(kw)
    return c


def _decode(name, **kw):
    c = dict(name=name, op="decode", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, page=64, Sq=1,
             length=4096, spread="even", pre=-1, sel=0)
    c.update(kw)
    return c


def _select(name, **kw):
    c = dict(name=name, op="select", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, page=64, Sq=1,
             length=4096, spread="even", sel=16)
    c.update(kw)
    return c


def listed():
    return [
        # one request's next token: the smallest call, all latency
        _append("append_step_b1", old=517),
        # a full decoding batch's next tokens; fp16, one KV head per query head, small pages,
        # pairs side by side, half of the head rotated, no page bounds
        _append("append_step_b128", dtype="fp16", B=128, Hq=16, Hkv=16, D=64, page=16, old=2048,
                spread="ragged", rot=32, interleaved=True, bounds=False),
        # four prompts of the ragged batch's lengths into an empty cache
        _append("append_prompts", B=4, new=4096, spread="4096,3001,517,14"),
        # one short request: all latency
        _decode("decode_b1_517", length=517),
        # the ragged batch's lengths
        _decode("decode_ragged", B=4, spread="4096,3001,517,14"),
        # an ordinary decoding batch of mixed lengths
        _decode("decode_batch", B=64, length=8192, spread="ragged"),
        # fp16, one KV head per query head, small pages, odd lengths
        _decode("decode_mha_d64", dtype="fp16", B=8, Hq=16, Hkv=16, D=64, page=16, length=2047,
                spread="ragged"),
        # five draft tokens checked at once, sliding window, large pages
        _decode("decode_draft_window", B=16, page=128, Sq=5, length=16384, spread="ragged", pre=4095),
        # long contexts: the largest
        _decode("decode_long", B=8, length=131072),
        # the same contexts through 64 listed pages per KV head
        _decode("decode_selected", B=8, length=131072, sel=64),
        # the choice of those pages
        _select("select_long", B=8, length=131072, sel=64),
        # and for one short request, fp16, small pages
        _select("select_b1", dtype="fp16", Hq=16, Hkv=4, D=64, page=16, length=2048, sel=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "decode", "select"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), Hq=Hkv * G, Hkv=Hkv, D=D,
             page=rng.choice([16, 32, 64, 128, 256]), spread=rng.choice(["even", "ragged"]))
    if op == "append":
        new = _log(rng, 1, 4096)
        B = _log(rng, 1, max(1, min(128, 8192 // new)))
        c.update(B=B, new=new, old=_log(rng, 1, min(4096, 65536 // B)) - 1,
                 rot=rng.choice([D, D // 2, 0]), interleaved=rng.choice([False, True]),
                 bounds=rng.choice([False, True]))
        return c
    # a choice needs more pages than it takes
    length = _log(rng, 32 * c["page"] if op == "select" else 1, 131072)
    most = 8 * 131072 * 8 * 128 // (length * Hkv * D)       # the largest listed case's keys
    c.update(B=_log(rng, 1, max(1, min(64, most // 2))), length=length, Sq=rng.choice([1, 1, 1, 2, 5]))
    pages = -(-length // c["page"])
    if op == "select":
        c["sel"] = _log(rng, 4, min(512, pages // 2))
    else:
        listed_pages = rng.choice([False, False, True])
        c["sel"] = _log(rng, 1, min(128, pages)) if listed_pages else 0
        c["pre"] = _log(rng, 1, 8192) - 1 if not listed_pages and rng.random() < 0.3 else -1
    return c


def _lens(case, most):
    """Per-sequence lengths of a case: all `most`, spread over [1, most], or given."""
    B, how = case["B"], case["spread"]
    if how == "even":
        return [most] * B
    if how == "ragged":
        return [most if b == 0 else 1 + int((b * GOLDEN % 1.0) * most) for b in range(B)]
    return [int(x) for x in how.split(",")]


def _old_new(case):
    """Tokens in the cache before the append, and new ones, of each sequence."""
    if "," in case["spread"]:
        return [case["old"]] * case["B"], _lens(case, case["new"])
    if case["new"] == 1:
        return [n - 1 for n in _lens(case, case["old"] + 1)], [1] * case["B"]
    return [case["old"]] * case["B"], _lens(case, case["new"])


# --------------------------------------------------------------------------- inputs
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _paged(case, cap, g):
    """Pools of N(0, 1) values (keys with an offset per channel, as rotated keys have), pages in
    random order, table entries past a sequence's pages -1."""
    page, Hkv, D, B = case["page"], case["Hkv"], case["D"], case["B"]
    need = [-(-n // page) for n in cap]
    num = sum(need) + 8
    k = torch.randn(num, Hkv, page, D, generator=g, device="cuda", dtype=_dt(case))
    v = torch.randn(num, Hkv, page, D, generator=g, device="cuda", dtype=_dt(case))
    k += torch.randn(1, Hkv, 1, D, generator=g, device="cuda", dtype=_dt(case))
    order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    wide = max(max(need), 1)
    n = torch.tensor(need, device="cuda")
    at = torch.arange(wide, device="cuda")[None]
    start = (torch.cumsum(n, 0) - n)[:, None]
    table = torch.where(at < n[:, None], order[(start + at).clamp(max=num - 1)], -1)
    return k, v, table.to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    s = dict(case)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=_dt(case))

    if case["op"] == "append":
        old, new = _old_new(case)
        most = max(o + n for o, n in zip(old, new))
        s["k"], s["v"], s["table"] = _paged(case, [o + n for o, n in zip(old, new)], g)
        s["lens"] = torch.tensor(old, dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        # q, k, v side by side, as one projection leaves them: [B, new, Hq + 2 Hkv, D]
        x = rand(B, case["new"], Hq + 2 * Hkv, D).transpose(1, 2)
        s["q"], s["kn"], s["vn"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        if case["rot"]:
            f = 10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
            a = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * f
            s["cos"], s["sin"] = a.cos().float(), a.sin().float()
        else:
            s["cos"] = s["sin"] = None
        s["q_out"] = torch.zeros(B, Hq, case["new"], D, device="cuda", dtype=_dt(case))
    else:
        lens = _lens(case, case["length"])
        s["k"], s["v"], s["table"] = _paged(case, lens, g)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = rand(B, Hq, case["Sq"], D)
        if case["op"] == "decode" and case["sel"]:
            # distinct pages of each KV head in ascending order, the newest among them
            n = -(-s["lens"] // case["page"])
            at = torch.arange(s["table"].shape[1], device="cuda")
            r = torch.rand(B, Hkv, at.numel(), generator=g, device="cuda")
            r = torch.where(at == n[:, None, None] - 1, 2.0, torch.where(at < n[:, None, None], r, -1.0))
            val, idx = r.topk(min(case["sel"], at.numel()), dim=-1)
            idx = torch.where(val >= 0, idx, at.numel()).sort(dim=-1).values
            s["idx"] = torch.where(idx < at.numel(), idx, -1).to(torch.int32).contiguous()
    if case["op"] == "select" or case.get("bounds"):
        s["kmin"], s["kmax"] = s["k"].amin(2).contiguous(), s["k"].amax(2).contiguous()
    if own:
        import attention_forward_fa_gb300 as fa
        s["fa"] = fa
        s["cache"] = fa.PagedKV(s["k"], s["v"], s["table"], s.get("kmin"), s.get("kmax"))
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return {"append": _plain_append, "decode": _plain_decode, "select": _plain_select}[s["op"]](s)


def _own(s):
    fa = s["fa"]
    if s["op"] == "append":
        fa.paged_kv_append(s["cache"], s["lens"], s["kn"], s["vn"], new_lens=s["new_lens"], q=s["q"],
                           q_out=s["q_out"], cos=s["cos"], sin=s["sin"], interleaved=s["interleaved"])
        return _append_out(s)
    if s["op"] == "select":
        return fa.select_kv_pages(s["q"], s["cache"], s["lens"], s["sel"])
    o, lse = fa.flash_attention_decode(s["q"], s["cache"], s["lens"], page_idx=s.get("idx"),
                                       pre_tokens=s["pre"] if s["pre"] >= 0 else None)
    return {"o": o, "lse": lse}


def _append_out(s):
    out = {"k": s["k"], "v": s["v"], "q": s["q_out"]}
    if s["bounds"]:
        out["kmin"], out["kmax"] = s["kmin"], s["kmax"]
    return out


def _rotated(x, cos, sin, interleaved):
    """x [B, H, S, D] fp32, cos / sin [B, 1, S, r / 2]: the first r channels rotated."""
    h = cos.shape[-1]
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if interleaved else (x[..., :h], x[..., h:2 * h])
    a, b = a * cos - b * sin, a * sin + b * cos
    y = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((y, x[..., 2 * h:]), -1)


def _plain_append(s):
    page, new = s["page"], s["new"]
    at = torch.arange(new, device="cuda")
    pos = s["lens"][:, None] + at
    live = at < s["new_lens"][:, None]
    k, q = s["kn"].float(), s["q"].float()
    if s["cos"] is not None:
        p = pos.clamp(max=s["cos"].shape[0] - 1)
        c, d = s["cos"][p][:, None], s["sin"][p][:, None]
        k, q = _rotated(k, c, d, s["interleaved"]), _rotated(q, c, d, s["interleaved"])
    k = k.to(s["k"].dtype).transpose(1, 2)[live]                       # [tokens, Hkv, D]
    v = s["vn"].transpose(1, 2)[live]
    where = s["table"].gather(1, (pos // page).clamp(max=s["table"].shape[1] - 1).long())[live].long()
    slot = (pos % page)[live].long()
    s["k"][where, :, slot] = k
    s["v"][where, :, slot] = v
    s["q_out"].copy_(torch.where(live[:, None, :, None], q.to(s["q_out"].dtype), s["q_out"]))
    if s["bounds"]:
        # one line for each (sequence, page that it touches)
        first = s["lens"] // page
        lines = (new + page - 2) // page + 1
        line = (torch.arange(s["B"], device="cuda")[:, None] * lines + pos // page - first[:, None])[live].long()
        shape = (s["B"] * lines,) + k.shape[1:]
        lo = torch.full(shape, math.inf, device="cuda").index_reduce_(0, line, k.float(), "amin")
        hi = torch.full(shape, -math.inf, device="cuda").index_reduce_(0, line, k.float(), "amax")
        pages = first[:, None] + torch.arange(lines, device="cuda")
        used = (pages * page < (s["lens"] + s["new_lens"])[:, None]).flatten()
        ids = s["table"].gather(1, pages.clamp(max=s["table"].shape[1] - 1).long()).flatten()[used].long()
        kept = (pages * page < s["lens"][:, None]).flatten()[used][:, None, None]   # had keys before
        lo, hi = lo[used], hi[used]
        s["kmin"][ids] = torch.where(kept, torch.minimum(lo, s["kmin"][ids].float()), lo).to(k.dtype)
        s["kmax"][ids] = torch.where(kept, torch.maximum(hi, s["kmax"][ids].float()), hi).to(k.dtype)
    return _append_out(s)


def _plain_decode(s):
    B, Hq, Sq, D = s["q"].shape
    Hkv, page = s["Hkv"], s["page"]
    G = Hq // Hkv
    slots = torch.arange(page, device="cuda")
    n_pages = -(-s["lens"] // page)
    if s["sel"]:
        idx = s["idx"].long()                                             # [B, Hkv, M]
        good = (idx >= 0) & (idx < n_pages[:, None, None])
        ids = s["table"][:, None].expand(-1, Hkv, -1).gather(2, idx.clamp(min=0)).clamp(min=0).long()
        heads = torch.arange(Hkv, device="cuda")[None, :, None]
        k, v = s["k"][ids, heads], s["v"][ids, heads]                     # [B, Hkv, M, page, D]
        pos = (idx[..., None] * page + slots).flatten(2)
        good = good[..., None].expand(-1, -1, -1, page).flatten(2)
    else:
        ids = s["table"].clamp(min=0).long()
        k, v = s["k"][ids].transpose(1, 2), s["v"][ids].transpose(1, 2)
        pos = torch.arange(ids.shape[1] * page, device="cuda")[None, None].expand(B, Hkv, -1)
        good = torch.ones_like(pos, dtype=torch.bool)
    last = (s["lens"][:, None] - Sq + torch.arange(Sq, device="cuda"))[:, None, :, None]
    low = last - s["pre"] if s["pre"] >= 0 else torch.zeros_like(last)
    p = pos[:, :, None]
    see = good[:, :, None] & (p <= last) & (p >= low)                     # [B, Hkv, Sq, keys]
    k, v = k.flatten(2, 3).float(), v.flatten(2, 3).float()
    v = torch.where(see.any(2)[..., None], v, 0.0)
    q = s["q"].float().view(B, Hkv, G * Sq, D) / math.sqrt(D)
    x = (q @ k.transpose(-1, -2)).view(B, Hkv, G, Sq, -1).masked_fill(~see[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    e = torch.exp(x - m)
    t = e.sum(-1, keepdim=True)
    o = (e.view(B, Hkv, G * Sq, -1) @ v).view(B, Hkv, G, Sq, D) / torch.where(t > 0, t, 1.0)
    lse = torch.where(t > 0, m + torch.log(t), math.inf)
    return {"o": o.view(B, Hq, Sq, D).to(s["q"].dtype), "lse": lse.view(B, Hq, Sq)}


def _plain_select(s):
    B, Hq, Sq, D = s["q"].shape
    Hkv, M = s["Hkv"], s["sel"]
    ids = s["table"].clamp(min=0).long()
    lo, hi = s["kmin"][ids].transpose(1, 2).double(), s["kmax"][ids].transpose(1, 2).double()
    q = s["q"].double().view(B, Hkv, -1, D)                               # all rows of a KV head
    x = q.clamp(min=0) @ hi.transpose(-1, -2) + q.clamp(max=0) @ lo.transpose(-1, -2)
    x = x.amax(2)                                                         # [B, Hkv, pages]
    n = (-(-s["lens"] // s["page"]))[:, None, None]
    at = torch.arange(ids.shape[1], device="cuda")
    x = torch.where((at < 1) | (at == n - 1), math.inf, x)                # first and newest page: always
    x = torch.where(at < n, x, -math.inf)
    idx = x.sort(dim=-1, descending=True, stable=True).indices[..., :M]
    idx = torch.where(idx < n, idx, at.numel()).sort(dim=-1).values
    idx = torch.where(idx < at.numel(), idx, -1)
    pad = M - idx.shape[-1]
    if pad:
        idx = torch.cat((idx, idx.new_full((B, Hkv, pad), -1)), -1)
    return idx.to(torch.int32)


# --------------------------------------------------------------------------- work
def work(case):
    B, Hq, Hkv, D, page = case["B"], case["Hq"], case["Hkv"], case["D"], case["page"]
    if case["op"] == "append":
        old, new = _old_new(case)
        tokens = sum(new)
        angles = min(tokens, max(o + n for o, n in zip(old, new)))          # rows of the tables
        rot = case["rot"]
        touched = sum(-(-(o + n) // page) - o // page for o, n in zip(old, new))
        kept = sum(1 for o in old if o % page)
        b = 2 * 2 * tokens * (Hq + 2 * Hkv) * D + 4 * rot * angles + 4 * (touched + 2 * B)
        if case["bounds"]:
            b += 2 * 2 * Hkv * D * (touched + kept)
        return {"bytes": b, "flops": 3 * tokens * (Hq + Hkv) * rot}
    lens, Sq = _lens(case, case["length"]), case["Sq"]
    if case["op"] == "select":
        pages = sum(-(-n // page) for n in lens)
        return {"bytes": 2 * 2 * pages * Hkv * D + 4 * pages + 2 * B * Hq * Sq * D + 4 * B * Hkv * case["sel"],
                "flops": 4 * pages * Hq * Sq * D}
    if case["sel"]:
        read = [min(n, (min(case["sel"], -(-n // page)) - 1) * page + (n - 1) % page + 1) for n in lens]
    elif case["pre"] >= 0:
        read = [min(n, case["pre"] + Sq) for n in lens]
    else:
        read = lens
    keys = sum(read)
    return {"bytes": 2 * 2 * keys * Hkv * D + 4 * -(-keys // page) + 2 * 2 * B * Hq * Sq * D + 4 * B * Hq * Sq,
            "flops": 4 * keys * Hq * Sq * D}


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "decode": _exact_decode, "select": _exact_select}[case["op"]](s)


def _exact_turn(x, pos, r, interleaved):
    """Complex rotation by the angles of the tables, taken anew in 64 bits."""
    if not r:
        return x
    j = torch.arange(r // 2, device=x.device, dtype=torch.float64)
    turn = torch.polar(torch.ones((), device=x.device, dtype=torch.float64), pos.double()[:, None] * 10000.0 ** (-2 * j / r))
    if interleaved:
        z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2).contiguous()) * turn
        y = torch.view_as_real(z).reshape(*x.shape[:-1], r)
    else:
        z = torch.complex(x[..., : r // 2], x[..., r // 2: r]) * turn
        y = torch.cat((z.real, z.imag), dim=-1)
    return torch.cat((y, x[..., r:]), dim=-1)


def _exact_append(s):
    k, v, q_out, page = s["k"].double(), s["v"].double(), s["q_out"].double(), s["page"]
    lo, hi = (s["kmin"].double(), s["kmax"].double()) if s["bounds"] else (None, None)
    for b, (o, n) in enumerate(zip(s["lens"].tolist(), s["new_lens"].tolist())):
        pos = torch.arange(o, o + n, device="cuda")
        kn = _exact_turn(s["kn"][b, :, :n].double(), pos, s["rot"], s["interleaved"])
        q_out[b, :, :n] = _exact_turn(s["q"][b, :, :n].double(), pos, s["rot"], s["interleaved"])
        for p in range(o // page, -(-(o + n) // page)):
            a, z = max(p * page, o), min((p + 1) * page, o + n)
            i = int(s["table"][b, p])
            k[i, :, a - p * page: z - p * page] = kn[:, a - o: z - o]
            v[i, :, a - p * page: z - p * page] = s["vn"][b, :, a - o: z - o].double()
            if s["bounds"]:
                l, h = kn[:, a - o: z - o].amin(1), kn[:, a - o: z - o].amax(1)
                lo[i], hi[i] = (l, h) if a == p * page else (torch.minimum(l, lo[i]), torch.maximum(h, hi[i]))
    out = {"k": k, "v": v, "q": q_out}
    if s["bounds"]:
        out["kmin"], out["kmax"] = lo, hi
    return out


def _exact_decode(s):
    B, Hq, Sq, D = s["q"].shape
    page, G = s["page"], Hq // s["Hkv"]
    o = torch.zeros(B, Hq, Sq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Sq), math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        every = torch.arange(-(-n // page), device="cuda")
        for h in range(s["Hkv"]):
            pages = every
            if s["sel"]:
                pages = s["idx"][b, h][s["idx"][b, h] >= 0].long()
            at = (pages[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)
            keep = at < n
            ids = s["table"][b][pages].long()
            k = s["k"][ids, h].reshape(-1, D)[keep].double()
            v = s["v"][ids, h].reshape(-1, D)[keep].double()
            at = at[keep]
            for i in range(Sq):
                tok = n - Sq + i
                see = at <= tok
                if s["pre"] >= 0:
                    see &= at >= tok - s["pre"]
                if not bool(see.any()):
                    continue
                x = (s["q"][b, h * G:(h + 1) * G, i].double() @ k[see].T) * D ** -0.5
                lse[b, h * G:(h + 1) * G, i] = torch.logsumexp(x, -1)
                o[b, h * G:(h + 1) * G, i] = torch.softmax(x, -1) @ v[see]
    return {"o": o, "lse": lse}


def _exact_select(s):
    B, Hq, Sq, D = s["q"].shape
    Hkv, M = s["Hkv"], s["sel"]
    out = torch.full((B, Hkv, M), -1, dtype=torch.int32)
    for b, n in enumerate(s["lens"].tolist()):
        n = -(-n // s["page"])
        ids = s["table"][b, :n].long()
        for h in range(Hkv):
            lo, hi = s["kmin"][ids, h].double(), s["kmax"][ids, h].double()
            rows = s["q"][b, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)].reshape(-1, D).double()
            best = torch.stack([torch.maximum(r * lo, r * hi).sum(-1) for r in rows]).amax(0)
            best[0] = best[n - 1] = math.inf
            chosen = torch.argsort(best, descending=True, stable=True)[:M].sort().values
            out[b, h, : chosen.numel()] = chosen.to(device="cpu", dtype=torch.int32)
    return out
