"""Measured cases of the operators over a paged key-value cache held in 8 bits, and of drafting over
either kind of cache: appending keys and values as they are quantised, attention of new tokens over
the 8-bit cache, reading a cache back into dense 16-bit tensors, attention of a tree of drafted
tokens, and keeping the drafts that were accepted.

Every case is one pass of one operator.  `run` computes it in a plain form (elementary torch
operations in fp32, fp64 where values next to a rounding border matter) or, where `own` is set, by
this package's calls.

An 8-bit cache holds each row of D channels of one token and KV head as e4m3 or e5m2 codes and one
scale 2^e, e the least integer >= -80 at which no code exceeds the format's largest value, kept as
the byte e + 127 (a float8_e8m0fnu number).
"""
import math

import torch

own = False

GOLDEN = 0.6180339887498949
LEAST = -80         # of a scale's exponent
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 9, "e5m2": 16}    # the largest value is 0.875 * 2^TOP


# --------------------------------------------------------------------------- cases
def _case(name, op, **kw):
    c = dict(name=name, op=op, dtype="bf16", fmt="e4m3", B=1, Hq=32, Hkv=8, D=128, page=64, spread="even")
    c.update(kw)
    return c


def _append(name, **kw):
    return _case(name, "append", **{**dict(new=1, old=0, rot=128, interleaved=False, bounds=True, tree=False), **kw})


def _decode(name, **kw):
    return _case(name, "decode", **{**dict(Sq=1, length=4096, pre=-1, sel=0), **kw})


def _tree(name, **kw):
    return _case(name, "tree", **{**dict(fmt="", Sq=8, length=4096), **kw})


def _read(name, **kw):
    return _case(name, "read", **{**dict(length=4096, start=0), **kw})


def _keep(name, **kw):
    return _case(name, "keep", **{**dict(fmt="", old=4096, Sq=16, most=4, bounds=True), **kw})


def listed():
    return [
        # a serving batch's drafts of one step, each sequence's a tree: positions given, no page bounds
        _append("append8_drafts", B=64, new=8, old=2048, spread="ragged", bounds=False, tree=True),
        # four prompts of the ragged batch's lengths into an empty cache
        _append("append8_prompts", B=4, new=4096, spread="4096,3001,517,14"),
        # one short request's next token: the smallest call, all latency
        _decode("decode8_b1_517", length=517),
        # an ordinary decoding batch of mixed lengths; e5m2, fp16, small pages
        _decode("decode8_batch", B=64, length=8192, spread="ragged", fmt="e5m2", dtype="fp16", page=16),
        # long contexts: the largest
        _decode("decode8_long", B=8, length=131072),
        # a prompt's prefix out of the 8-bit cache, for a prefill of what follows it
        _read("read8_prompts", B=4, spread="4096,3001,517,14"),
        # a long 16-bit cache out of its pages (fp16, odd start)
        _read("read16_long", dtype="fp16", fmt="", B=2, Hq=16, Hkv=16, D=64, page=16, length=65535, start=1001),
        # one request's few drafts: latency
        _tree("tree_b1", Sq=8, length=517),
        # a batch of small trees of uneven sizes
        _tree("tree_batch", B=16, Sq=12, length=8192, spread="ragged"),
        # large trees over an 8-bit cache
        _tree("tree8_wide", B=4, Sq=64, length=16384, spread="ragged", fmt="e4m3"),
        # one request's accepted path
        _keep("keep_b1", Sq=8, most=4, old=517),
        # a batch's accepted paths, out of large trees, in an 8-bit cache
        _keep("keep8_batch", B=64, Sq=64, most=12, old=8192, spread="ragged", fmt="e4m3"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "read", "tree", "tree", "keep"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    eight = op in ("append", "decode") or rng.random() < 0.5
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), fmt=rng.choice(["e4m3", "e4m3", "e5m2"]) if eight else "",
             Hq=Hkv * G, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128, 256]), spread=rng.choice(["even", "ragged"]))
    if op == "append":
        new = _log(rng, 1, 4096)
        B = _log(rng, 1, max(1, min(128, 8192 // new)))
        c.update(B=B, new=new, old=_log(rng, 1, min(4096, 65536 // B)) - 1,
                 rot=rng.choice([D, D // 2, 0]), interleaved=rng.choice([False, True]),
                 bounds=rng.choice([False, True]), tree=new <= 64 and rng.random() < 0.5)
        return c
    if op == "keep":
        S = _log(rng, 2, 64)
        c.update(B=_log(rng, 1, 64), old=_log(rng, 1, 8192), Sq=S, most=_log(rng, 1, min(S - 1, 16)),
                 bounds=rng.choice([False, True]))
        return c
    if op == "read":
        length = _log(rng, 1, 65536)
        most = 2 * 65536 * 16 * 64 // (length * Hkv * D)
        c.update(B=_log(rng, 1, max(1, min(64, most))), length=length, start=rng.choice([0, _log(rng, 1, 2048)]))
        return c
    if op == "tree":
        S = _log(rng, 1, 64)
        length = _log(rng, S, 65536)
        rows = 32 * 64 * 16384 * 2 * 128 // (Hkv * G * S * length * D)       # half the listed largest's work
        c.update(B=_log(rng, 1, max(1, min(64, rows))), length=length, Sq=S)
        if rows < 1:
            c["length"] = max(S, length // 8)
        return c
    length = _log(rng, 1, 131072)
    most = 8 * 131072 * 8 * 128 // (length * Hkv * D)                        # the largest listed case's keys
    c.update(B=_log(rng, 1, max(1, min(64, most // 2))), length=length, Sq=rng.choice([1, 1, 1, 2, 5]))
    listed_pages = rng.choice([False, False, True])
    c["sel"] = _log(rng, 1, min(128, -(-length // c["page"]))) if listed_pages else 0
    c["pre"] = _log(rng, 1, 8192) - 1 if not listed_pages and rng.random() < 0.3 else -1
    return c


def _lens(case, most, least=1):
    """Per-sequence lengths of a case: all `most`, spread over [least, most], or given."""
    B, how = case["B"], case["spread"]
    if how == "even":
        return [most] * B
    if how == "ragged":
        return [most if b == 0 else least + int((b * GOLDEN % 1.0) * (most - least + 1)) for b in range(B)]
    return [int(x) for x in how.split(",")]


def _drafts(case):
    """How many of a case's Sq drafts each sequence has (of a ragged batch between half and all)."""
    S = case["Sq"]
    return [S] * case["B"] if case["spread"] == "even" else [S - int((b * GOLDEN % 1.0) * (S // 2)) for b in range(case["B"])]


def _old_new(case):
    """Tokens in the cache before the append, and new ones, of each sequence."""
    if "," in case["spread"]:
        return [case["old"]] * case["B"], _lens(case, case["new"])
    if case["new"] <= 64:
        return [n - 1 for n in _lens(case, case["old"] + 1)], [case["new"]] * case["B"]
    return [case["old"]] * case["B"], _lens(case, case["new"])


def _kept(case):
    """Tokens in the cache before the drafts, and accepted drafts, of each sequence."""
    return _lens(case, case["old"]), _lens(case, case["most"])


# --------------------------------------------------------------------------- inputs
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _exponent(amax, fmt):
    """The least e >= LEAST with amax <= (largest value) * 2^e."""
    m, x = torch.frexp(amax)
    e = x - TOP[fmt] + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, LEAST).clamp(min=LEAST)


def _quantise(x, fmt):
    """Codes and scale bytes of rows x [..., D]."""
    e = _exponent(x.abs().amax(-1), fmt)
    return torch.ldexp(x, -e[..., None]).float().to(FP8[fmt]), (e + 127).to(torch.uint8)


def _values(codes, scale, fmt):
    """What uint8 codes [..., D] and scale bytes stand for, in fp32."""
    return torch.ldexp(codes.view(FP8[fmt]).float(), scale.int()[..., None] - 127)


def _paged(s, case, cap, g):
    """Pools of N(0, 1) values (keys with an offset per channel, as rotated keys have), pages in
    random order, table entries past a sequence's pages -1."""
    page, Hkv, D, B = case["page"], case["Hkv"], case["D"], case["B"]
    need = [-(-n // page) for n in cap]
    num = sum(need) + 8
    for x in ("k", "v"):
        t = torch.randn(num, Hkv, page, D, generator=g, device="cuda", dtype=_dt(case))
        if x == "k":
            t += torch.randn(1, Hkv, 1, D, generator=g, device="cuda", dtype=_dt(case))
        if case["fmt"]:
            codes = torch.empty(num, Hkv, page, D, device="cuda", dtype=FP8[case["fmt"]])
            scale = torch.empty(num, Hkv, page, device="cuda", dtype=torch.uint8)
            for a in range(0, num, 1024):        # (a long cache's fp32 copy by parts)
                codes[a: a + 1024], scale[a: a + 1024] = _quantise(t[a: a + 1024].float(), case["fmt"])
            s[x], s[x + "_scale"] = codes, scale.view(torch.float8_e8m0fnu)
            if x == "k" and case.get("bounds"):
                t = _values(codes, scale, case["fmt"])
        else:
            s[x] = t
        if x == "k" and case.get("bounds"):
            s["kmin"], s["kmax"] = t.amin(2).to(_dt(case)), t.amax(2).to(_dt(case))
        del t
    order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    wide = max(max(need), 1)
    n = torch.tensor(need, device="cuda")
    at = torch.arange(wide, device="cuda")[None]
    start = (torch.cumsum(n, 0) - n)[:, None]
    table = torch.where(at < n[:, None], order[(start + at).clamp(max=num - 1)], -1)
    s["table"] = table.to(torch.int32).contiguous()


def _ancestors(B, S, g):
    """Random trees: bool [B, S, S], row i the drafts on the way from the root to draft i, itself
    included, and the depths [B, S]."""
    r = torch.rand(B, S, generator=g, device="cuda").cpu()
    # a draft's parent is one of the four before it, or the last token of the text
    parent = (torch.arange(S) - 1 - (r * 4).long()).clamp(min=-1)
    anc = torch.zeros(B, S, S, dtype=torch.bool)
    seq = torch.arange(B)
    for i in range(S):
        up = parent[:, i]
        anc[:, i] = anc[seq, up.clamp(min=0)] & (up >= 0)[:, None]
        anc[:, i, i] = True
    return anc.cuda(), (anc.sum(-1) - 1).to(torch.int32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, Hq, Hkv, D, op = case["B"], case["Hq"], case["Hkv"], case["D"], case["op"]
    s = dict(case)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=_dt(case))

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    if op == "append":
        old, new = _old_new(case)
        _paged(s, case, [o + n for o, n in zip(old, new)], g)
        s["lens"], s["new_lens"] = ints(old), ints(new)
        # q, k, v side by side, as one projection leaves them: [B, new, Hq + 2 Hkv, D]
        x = rand(B, case["new"], Hq + 2 * Hkv, D).transpose(1, 2)
        s["q"], s["kn"], s["vn"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        s["pos"] = None
        if case["tree"]:
            s["pos"] = s["lens"][:, None] + _ancestors(B, case["new"], g)[1]
        if case["rot"]:
            f = 10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
            a = torch.arange(max(o + n for o, n in zip(old, new)), device="cuda", dtype=torch.float64)[:, None] * f
            s["cos"], s["sin"] = a.cos().float(), a.sin().float()
        else:
            s["cos"] = s["sin"] = None
        s["q_out"] = torch.zeros(B, Hq, case["new"], D, device="cuda", dtype=_dt(case))
    elif op == "keep":
        old, kept = _kept(case)
        _paged(s, case, [o + case["Sq"] for o in old], g)
        s["lens"], s["keep_lens"] = ints(old), ints(kept)
        # accepted drafts in ascending order, none of them in its place already
        r = torch.rand(B, case["Sq"] - 1, generator=g, device="cuda")
        first = r.argsort(-1)[:, : case["most"]] + 1
        live = torch.arange(case["most"], device="cuda") < s["keep_lens"][:, None]
        first = torch.where(live, first, case["Sq"]).sort(-1).values
        s["idx"] = torch.where(live, first, -1).to(torch.int32).contiguous()
    elif op == "read":
        lens = _lens(case, case["length"])
        _paged(s, case, [case["start"] + n for n in lens], g)
        s["lens"], s["starts"] = ints(lens), ints([case["start"]] * B)
        s["k_out"], s["v_out"] = (torch.zeros(B, Hkv, max(lens), D, device="cuda", dtype=_dt(case)) for _ in range(2))
    else:
        lens = _lens(case, case["length"], case["Sq"] if op == "tree" else 1)
        _paged(s, case, lens, g)
        s["lens"] = ints(lens)
        s["q"] = rand(B, Hq, case["Sq"], D)
        if op == "tree":
            s["anc"] = _ancestors(B, case["Sq"], g)[0]
            s["new_lens"] = ints(_drafts(case))
        elif case["sel"]:
            # distinct pages of each KV head in ascending order, the newest among them
            n = -(-s["lens"] // case["page"])
            at = torch.arange(s["table"].shape[1], device="cuda")
            r = torch.rand(B, Hkv, at.numel(), generator=g, device="cuda")
            r = torch.where(at == n[:, None, None] - 1, 2.0, torch.where(at < n[:, None, None], r, -1.0))
            val, idx = r.topk(min(case["sel"], at.numel()), dim=-1)
            idx = torch.where(val >= 0, idx, at.numel()).sort(dim=-1).values
            s["idx"] = torch.where(idx < at.numel(), idx, -1).to(torch.int32).contiguous()
    if own:
        import attention_forward_fa_gb300 as fa
        s["fa"] = fa
        eight = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], dtype=_dt(case)) if case["fmt"] else {}
        s["cache"] = fa.PagedKV(s["k"], s["v"], s["table"], s.get("kmin"), s.get("kmax"), **eight)
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return {"append": _plain_append, "decode": _plain_decode, "tree": _plain_decode, "read": _plain_read,
            "keep": _plain_keep}[s["op"]](s)


def _own(s):
    fa, op = s["fa"], s["op"]
    if op == "append":
        fa.paged_kv_append(s["cache"], s["lens"], s["kn"], s["vn"], new_lens=s["new_lens"], q=s["q"],
                           q_out=s["q_out"], cos=s["cos"], sin=s["sin"], interleaved=s["interleaved"],
                           positions=s["pos"])
        return _pools(s)
    if op == "keep":
        fa.paged_kv_keep(s["cache"], s["lens"], s["idx"], s["keep_lens"])
        return _pools(s)
    if op == "read":
        fa.paged_kv_read(s["cache"], s["lens"], starts=s["starts"], k_out=s["k_out"], v_out=s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "tree":
        o, lse = fa.flash_attention_decode_tree(s["q"], s["cache"], s["lens"], s["anc"], new_lens=s["new_lens"])
    else:
        o, lse = fa.flash_attention_decode(s["q"], s["cache"], s["lens"], page_idx=s.get("idx"),
                                           pre_tokens=s["pre"] if s["pre"] >= 0 else None)
    return {"o": o, "lse": lse}


def _pools(s):
    names = ["k", "v"] + (["k_scale", "v_scale"] if s["fmt"] else []) + (["q_out"] if s["op"] == "append" else [])
    return {x: s[x] for x in names + (["kmin", "kmax"] if s["bounds"] else [])}


def _bytes(t):
    """A pool as what may be indexed: 8-bit codes and scales by their bits."""
    return t.view(torch.uint8) if t.element_size() == 1 else t


def _rotated(x, cos, sin, interleaved):
    """x [B, H, S, D], cos / sin [B, 1, S, r / 2]: the first r channels rotated."""
    h = cos.shape[-1]
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if interleaved else (x[..., :h], x[..., h:2 * h])
    a, b = a * cos - b * sin, a * sin + b * cos
    y = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((y, x[..., 2 * h:]), -1)


def _plain_append(s):
    page, new, fmt = s["page"], s["new"], s["fmt"]
    at = torch.arange(new, device="cuda")
    pos = s["lens"][:, None] + at
    live = at < s["new_lens"][:, None]
    k, q = s["kn"].double(), s["q"].float()
    if s["cos"] is not None:
        p = (pos if s["pos"] is None else s["pos"]).clamp(max=s["cos"].shape[0] - 1)
        c, d = s["cos"][p][:, None], s["sin"][p][:, None]
        k, q = _rotated(k, c.double(), d.double(), s["interleaved"]), _rotated(q, c, d, s["interleaved"])
    k, ke = _quantise(k.transpose(1, 2)[live], fmt)                    # [tokens, Hkv, D]
    v, ve = _quantise(s["vn"].transpose(1, 2)[live].float(), fmt)
    where = s["table"].gather(1, (pos // page).clamp(max=s["table"].shape[1] - 1).long())[live].long()
    slot = (pos % page)[live].long()
    for x, y in (("k", k), ("v", v), ("k_scale", ke), ("v_scale", ve)):
        _bytes(s[x])[where, :, slot] = _bytes(y)
    s["q_out"].copy_(torch.where(live[:, None, :, None], q.to(s["q_out"].dtype), s["q_out"]))
    if s["bounds"]:
        _plain_bounds(s, _values(_bytes(k), ke, fmt), pos, live, live)
    return _pools(s)


def _plain_bounds(s, k, pos, live, written):
    """The bounds of the pages in which keys k [tokens, Hkv, D] were written, those at `written` of
    positions pos [B, n], of which the ones at `live` count: anew where slot 0 was written."""
    page, B = s["page"], s["B"]
    first = pos[:, :1] // page
    lines = (pos.shape[1] + page - 2) // page + 1                      # pages that a sequence may touch
    line = (torch.arange(B, device="cuda")[:, None] * lines + pos // page - first)[live & written].long()
    shape = (B * lines,) + k.shape[1:]
    lo = torch.full(shape, math.inf, device="cuda").index_reduce_(0, line, k, "amin")
    hi = torch.full(shape, -math.inf, device="cuda").index_reduce_(0, line, k, "amax")
    anew = torch.zeros(B * lines, device="cuda").index_reduce_(0, line, (pos % page == 0)[live & written].float(), "amax")
    used = torch.zeros(B * lines, device="cuda").index_fill_(0, line, 1.0) > 0
    pages = first + torch.arange(lines, device="cuda")
    ids = s["table"].gather(1, pages.clamp(max=s["table"].shape[1] - 1).long()).flatten().long()
    used &= ids >= 0
    at = torch.where(used, ids, s["kmin"].shape[0])                    # (a row behind the last takes what is none)
    for x, new, of in (("kmin", lo, torch.minimum), ("kmax", hi, torch.maximum)):
        was = torch.cat((s[x], torch.zeros_like(s[x][:1])))
        got = torch.where(anew[:, None, None] > 0, new, of(new, was[at].float()))
        was[at] = got.to(was.dtype)
        s[x].copy_(was[:-1])


def _plain_keep(s):
    page, M = s["page"], s["most"]
    at = torch.arange(M, device="cuda")
    live = at < s["keep_lens"][:, None]
    src, dst = s["lens"][:, None] + s["idx"].clamp(min=0), (s["lens"][:, None] + at)
    cols = s["table"].shape[1] - 1
    from_page = s["table"].gather(1, (src // page).clamp(max=cols).long())[live].long()
    to_page = s["table"].gather(1, (dst // page).clamp(max=cols).long())[live].long()
    from_slot, to_slot = (src % page)[live].long(), (dst % page)[live].long()
    for x in ("k", "v") + (("k_scale", "v_scale") if s["fmt"] else ()):
        pool = _bytes(s[x])
        pool[to_page, :, to_slot] = pool[from_page, :, from_slot]
    if s["bounds"]:
        k = _bytes(s["k"])[to_page, :, to_slot]
        k = _values(k, _bytes(s["k_scale"])[to_page, :, to_slot], s["fmt"]) if s["fmt"] else k.float()
        moved = src > dst
        _plain_bounds(s, k[moved[live]], dst, live, moved)
    return _pools(s)


def _plain_read(s):
    page, S = s["page"], s["k_out"].shape[2]
    at = torch.arange(S, device="cuda")
    live = (at < s["lens"][:, None])[:, None, :, None]
    pos = s["starts"][:, None] + at
    ids = s["table"].gather(1, (pos // page).clamp(max=s["table"].shape[1] - 1).long()).clamp(min=0).long()
    slot = (pos % page).long()
    for x in ("k", "v"):
        rows = _bytes(s[x])[ids, :, slot]                              # [B, S, Hkv, D]
        if s["fmt"]:
            rows = _values(rows, _bytes(s[x + "_scale"])[ids, :, slot], s["fmt"])
        out = s[x + "_out"]
        out.copy_(torch.where(live, rows.transpose(1, 2).to(out.dtype), out))
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_decode(s):
    B, Hq, Sq, D = s["q"].shape
    Hkv, page = s["Hkv"], s["page"]
    G = Hq // Hkv
    slots = torch.arange(page, device="cuda")
    n_pages = -(-s["lens"] // page)
    if s.get("sel"):
        idx = s["idx"].long()                                             # [B, Hkv, M]
        good = (idx >= 0) & (idx < n_pages[:, None, None])
        ids = s["table"][:, None].expand(-1, Hkv, -1).gather(2, idx.clamp(min=0)).clamp(min=0).long()
        heads = torch.arange(Hkv, device="cuda")[None, :, None]
        at = (ids, heads)                                                 # [B, Hkv, M, page, D]
        pos = (idx[..., None] * page + slots).flatten(2)
        good = good[..., None].expand(-1, -1, -1, page).flatten(2)
    else:
        at = (s["table"].clamp(min=0).long()[:, None], torch.arange(Hkv, device="cuda")[None, :, None])
        pos = torch.arange(s["table"].shape[1] * page, device="cuda")[None, None].expand(B, Hkv, -1)
        good = torch.ones_like(pos, dtype=torch.bool)
    k, v = ((_values(_bytes(s[x])[at], _bytes(s[x + "_scale"])[at], s["fmt"]) if s["fmt"] else s[x][at].float()).flatten(2, 3)
            for x in ("k", "v"))
    p = pos[:, :, None]
    if s["op"] == "tree":
        base = (s["lens"] - s["new_lens"])[:, None, None, None]
        row = torch.arange(Sq, device="cuda")[None, None, :, None]
        draft = (p - base).clamp(0, Sq - 1).expand(B, Hkv, Sq, -1)
        on = s["anc"][:, None].expand(-1, Hkv, -1, -1).gather(3, draft)
        on = on & (row < s["new_lens"][:, None, None, None]) & (p < s["lens"][:, None, None, None])
        see = good[:, :, None] & ((p < base) | on)
    else:
        last = (s["lens"][:, None] - Sq + torch.arange(Sq, device="cuda"))[:, None, :, None]
        low = last - s["pre"] if s["pre"] >= 0 else torch.zeros_like(last)
        see = good[:, :, None] & (p <= last) & (p >= low)                 # [B, Hkv, Sq, keys]
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


# --------------------------------------------------------------------------- work
def work(case):
    B, Hq, Hkv, D, page, op = case["B"], case["Hq"], case["Hkv"], case["D"], case["page"], case["op"]
    row = D + 1 if case["fmt"] else 2 * D        # bytes of a cached row
    if op == "append":
        old, new = _old_new(case)
        tokens, rot = sum(new), case["rot"]
        angles = min(tokens, max(o + n for o, n in zip(old, new)))          # rows of the tables
        touched = sum(-(-(o + n) // page) - o // page for o, n in zip(old, new))
        kept = sum(1 for o in old if o % page)
        b = (2 * 2 * Hq * D + 2 * Hkv * (2 * D + row)) * tokens + 4 * rot * angles + 4 * (touched + 2 * B)
        b += 4 * tokens if case["tree"] else 0
        if case["bounds"]:
            b += 2 * 2 * Hkv * D * (touched + kept)
        return {"bytes": b, "flops": 3 * tokens * (Hq + Hkv) * rot + 2 * 2 * tokens * Hkv * D}
    if op == "keep":
        old, kept = _kept(case)
        tokens = sum(kept)
        b = 2 * 2 * tokens * Hkv * row + 4 * (tokens + 4 * B)
        if case["bounds"]:
            b += 2 * 2 * 2 * Hkv * D * B
        return {"bytes": b, "flops": 0}
    if op == "read":
        tokens = sum(_lens(case, case["length"]))
        return {"bytes": 2 * tokens * Hkv * (row + 2 * D) + 4 * -(-tokens // page) + 8 * B, "flops": 0}
    Sq = case["Sq"]
    lens = _lens(case, case["length"], Sq if op == "tree" else 1)
    if case.get("sel"):
        read = [min(n, (min(case["sel"], -(-n // page)) - 1) * page + (n - 1) % page + 1) for n in lens]
    elif case.get("pre", -1) >= 0:
        read = [min(n, case["pre"] + Sq) for n in lens]
    else:
        read = lens
    keys = sum(read)
    b = 2 * keys * Hkv * row + 4 * -(-keys // page) + 2 * 2 * B * Hq * Sq * D + 4 * B * Hq * Sq
    return {"bytes": b + (B * Sq * Sq if op == "tree" else 0), "flops": 4 * keys * Hq * Sq * D}


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "decode": _exact_attention, "tree": _exact_attention, "read": _exact_read,
            "keep": _exact_keep}[case["op"]](s)


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


def _exact_scale(x, fmt):
    """The scale 2^e of rows x: the power of two, by logarithms and a correction."""
    top = 0.875 * 2.0 ** TOP[fmt]
    a = x.abs().amax(-1) / top
    e = torch.ceil(torch.log2(a.clamp(min=2.0 ** LEAST)))
    e = torch.where(2.0 ** (e - 1) >= a, e - 1, torch.where(2.0 ** e < a, e + 1, e)).clamp(min=LEAST)
    return 2.0 ** e


def _exact_stored(y, f, fmt):
    """Rows y as codes of scales f hold them: the nearest number of the format, ties to even."""
    digits, least = (3, -9) if fmt == "e4m3" else (2, -16)
    z = y / f[..., None]
    step = 2.0 ** (torch.floor(torch.log2(z.abs().clamp(min=2.0 ** (least + digits)))) - digits)
    return torch.round(z / step) * step * f[..., None]


def _exact_append(s):
    """Codes are the scaled values themselves, unrounded; bounds are those of the keys as stored."""
    page, fmt = s["page"], s["fmt"]
    out = {x: _bytes(s[x]).view(FP8[fmt]).double() for x in ("k", "v")}
    out |= {x: 2.0 ** (_bytes(s[x]).double() - 127) for x in ("k_scale", "v_scale")}
    out["q_out"] = s["q_out"].double()
    if s["bounds"]:
        out["kmin"], out["kmax"] = s["kmin"].double(), s["kmax"].double()
    for b, (o, n) in enumerate(zip(s["lens"].tolist(), s["new_lens"].tolist())):
        pos = torch.arange(o, o + n, device="cuda")
        turn = pos if s["pos"] is None else s["pos"][b, :n]
        kn = _exact_turn(s["kn"][b, :, :n].double(), turn, s["rot"], s["interleaved"])
        vn = s["vn"][b, :, :n].double()
        out["q_out"][b, :, :n] = _exact_turn(s["q"][b, :, :n].double(), turn, s["rot"], s["interleaved"])
        ids, slot = s["table"][b].long()[pos // page], pos % page
        for x, y in (("k", kn), ("v", vn)):
            f = _exact_scale(y, fmt)
            out[x][ids, :, slot] = (y / f[..., None]).transpose(0, 1)
            out[x + "_scale"][ids, :, slot] = f.transpose(0, 1)
        if s["bounds"]:
            for p in range(o // page, -(-(o + n) // page)):
                a, z = max(p * page, o), min((p + 1) * page, o + n)
                i = int(s["table"][b, p])
                key = _exact_stored(kn[:, a - o: z - o], _exact_scale(kn[:, a - o: z - o], fmt), fmt)
                l, h = key.amin(1), key.amax(1)
                out["kmin"][i], out["kmax"][i] = (l, h) if a == p * page else (torch.minimum(l, out["kmin"][i]), torch.maximum(h, out["kmax"][i]))
    return out


def _exact_keep(s):
    page, fmt = s["page"], s["fmt"]
    out = {x: _bytes(s[x]).clone() for x in ("k", "v")}
    if fmt:
        out |= {x: _bytes(s[x]).clone() for x in ("k_scale", "v_scale")}
    lo, hi = (s["kmin"].double(), s["kmax"].double()) if s["bounds"] else (None, None)
    for b, (o, n) in enumerate(zip(s["lens"].tolist(), s["keep_lens"].tolist())):
        for i, j in enumerate(s["idx"][b, :n].tolist()):
            if i == j:
                continue
            to, slot = int(s["table"][b, (o + i) // page]), (o + i) % page
            src, at = int(s["table"][b, (o + j) // page]), (o + j) % page
            for x in out:
                out[x][to, :, slot] = out[x][src, :, at]
            if s["bounds"]:
                key = out["k"][to, :, slot]
                key = key.view(FP8[fmt]).double() * 2.0 ** (out["k_scale"][to, :, slot].double()[:, None] - 127) if fmt else key.double()
                lo[to], hi[to] = (key, key) if slot == 0 else (torch.minimum(lo[to], key), torch.maximum(hi[to], key))
    out = {x: (2.0 ** (y.double() - 127) if x.endswith("scale") else y.view(FP8[fmt]).double() if fmt else y.double())
           for x, y in out.items()}
    if s["bounds"]:
        out["kmin"], out["kmax"] = lo, hi
    return out


def _exact_rows(s, x, b, h, pos):
    """Rows of the cache at positions pos of sequence b and KV head h, in 64 bits."""
    ids, slot = s["table"][b].long()[pos // s["page"]], pos % s["page"]
    if not s["fmt"]:
        return s[x][ids, h, slot].double()
    f = 2.0 ** (_bytes(s[x + "_scale"])[ids, h, slot].double() - 127)
    return _bytes(s[x])[ids, h, slot].view(FP8[s["fmt"]]).double() * f[:, None]


def _exact_read(s):
    out = {x: s[x + "_out"].double() for x in ("k", "v")}
    for b, n in enumerate(s["lens"].tolist()):
        pos = torch.arange(n, device="cuda") + s["start"]
        for h in range(s["Hkv"]):
            for x in out:
                out[x][b, h, :n] = _exact_rows(s, x, b, h, pos)
    return out


def _exact_attention(s):
    B, Hq, Sq, D = s["q"].shape
    page, G = s["page"], Hq // s["Hkv"]
    o = torch.zeros(B, Hq, Sq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Sq), math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        every = torch.arange(-(-n // page), device="cuda")
        drafts = int(s["new_lens"][b]) if s["op"] == "tree" else 0
        for h in range(s["Hkv"]):
            pages = every
            if s.get("sel"):
                pages = s["idx"][b, h][s["idx"][b, h] >= 0].long()
            at = (pages[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)
            at = at[at < n]
            k, v = (_exact_rows(s, x, b, h, at) for x in ("k", "v"))
            heads = slice(h * G, (h + 1) * G)
            see = torch.zeros(Sq, at.numel(), dtype=torch.bool, device="cuda")
            for i in range(Sq):
                if s["op"] == "tree":
                    see[i, : n - drafts] = True
                    if i < drafts:
                        see[i, n - drafts:] = s["anc"][b, i, :drafts]
                else:
                    see[i] = at <= n - Sq + i
                    if s["pre"] >= 0:
                        see[i] &= at >= n - Sq + i - s["pre"]
            x = (s["q"][b, heads].double() @ k.T) * D ** -0.5
            x = x.masked_fill(~see, -math.inf)
            some = see.any(-1)
            total = torch.logsumexp(x, -1)
            lse[b, heads] = torch.where(some, total, math.inf)
            w = torch.exp(x - torch.where(some, total, 0.0)[..., None])
            o[b, heads] = w @ v
    return {"o": o, "lse": lse}
