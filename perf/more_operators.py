"""Timed cases of the calls around a softmax layer's paged key/value cache.

Four operators, each with a plain form in elementary torch operations and the
library's own calls:

    rotate  ssd_attn_qk_norm_rope: the norm of every query and key head and the
            position rotation, over packed prompts or one token per sequence
    write   ssd_attn_paged_append: new tokens' queries and keys normed and rotated,
            keys and values appended to the pages of their sequences.  Pages in 4
            bits are read back (ssd_attn_paged_gather) as the values they stand for:
            the rows that the next part of a prompt attends
    step    ssd_attn_paged_append of one token per sequence, then
            ssd_attn_paged_decode_step over the pages, which hold the input type
    step4   ssd_attn_paged_decode_step over pages in 4 bits

A case says which operator it is ("op"), its sizes and its type ("io").  Pages are
[pages, key heads, rows of a page, head width], those of a sequence in any order;
4-bit pages hold two codes to a byte and, for every 64 values of a row, a step and
a least value in half precision: value = code step + least.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6
_GROUP = 64          # values that share a step and a least value


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one user's next token
        dict(name="rotate_1", op="rotate", io="bf16", lens="1", prefix="9000", hq=32, hkv=8, d=128, rot=128,
             pairs="half", norm=True, fused=True),
        # long documents in front of softmax prefill
        dict(name="rotate_32768", op="rotate", io="bf16", lens="8192,8192,8192,8192", prefix="0,0,0,0", hq=32,
             hkv=8, d=128, rot=128, pairs="half", norm=True, fused=True),
        # a small full-precision model that rotates a quarter of each head, neighbours paired, no norm
        dict(name="rotate_f32", op="rotate", io="f32", lens="1,200,65,17,1130", prefix="0,0,7,131000,0", hq=8,
             hkv=2, d=64, rot=16, pairs="next", norm=False, fused=False),
        # a serving batch of mixed prompts, some on cached prefixes
        dict(name="write_packed", op="write", io="bf16", bits=16, lens="8192,4097,3000,2048,1500,1024,777,512",
             prefix="0,0,1000,0,0,4096,0,77", page=64, hq=32, hkv=8, d=128, rot=128, pairs="half", norm=True),
        # the same batch into pages in 4 bits, read back for the prompts' own attention
        dict(name="write4_packed", op="write", io="bf16", bits=4, lens="8192,4097,3000,2048,1500,1024,777,512",
             prefix="0,0,1000,0,0,4096,0,77", page=64, hq=32, hkv=8, d=128, rot=128, pairs="half", norm=True),
        # short requests into pages in 4 bits
        dict(name="write4_short", op="write", io="bf16", bits=4, lens="1,33,5,17", prefix="64,0,15,130", page=16,
             hq=8, hkv=2, d=64, rot=64, pairs="half", norm=False),
        # generation: one user at a long context, a batch at mixed lengths, a small full-precision
        # model whose table is far wider than its sequences are long
        dict(name="step_long", op="step", io="bf16", batch=1, longest=131000, shortest=131000, room=131072,
             page=64, hq=32, hkv=8, d=128, rot=128, pairs="half", norm=True),
        dict(name="step_64", op="step", io="bf16", batch=64, longest=8190, shortest=100, room=8192, page=16,
             hq=32, hkv=8, d=128, rot=128, pairs="half", norm=True),
        dict(name="step_f32", op="step", io="f32", batch=3, longest=1000, shortest=5, room=16384, page=32, hq=8,
             hkv=8, d=64, rot=64, pairs="half", norm=False),
        # the same over pages in 4 bits
        dict(name="step4_long", op="step4", io="bf16", batch=1, longest=131000, shortest=131000, room=131072,
             page=64, hq=32, hkv=8, d=128),
        dict(name="step4_64", op="step4", io="bf16", batch=64, longest=8190, shortest=100, room=8192, page=16,
             hq=32, hkv=8, d=128),
        dict(name="step4_short", op="step4", io="f32", batch=5, longest=300, shortest=0, room=2048, page=128, hq=6,
             hkv=2, d=256),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, total, count):
    """`count` lengths of very different sizes, `total` tokens at most."""
    w = [math.exp(rng.uniform(0.0, 3.0)) for _ in range(count)]
    return [max(1, int(total * x / sum(w))) for x in w]


def draw(rng):
    op = rng.choice(["rotate", "write", "write", "step", "step4"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    g = rng.choice([1, 2, 3, 4, 6, 8, 16, 20])
    while hkv * g > 64:
        g //= 2
    heads = dict(hq=hkv * g, hkv=hkv, d=d)
    rot = rng.choice([0, d // 4, d // 2, d, d, d])
    turn = dict(rot=rot, pairs=rng.choice(["half", "half", "next"]), norm=rot == 0 or rng.random() < 0.7)
    if op in ("rotate", "write"):
        # bounded by the largest listed cases: 32768 and 21150 tokens of 40 and 48 heads of 128
        room = 21150 * 48 * 128 // ((g + 2) * hkv * d) // (2 if io == "f32" else 1)
        total = _logint(rng, 1, max(2, min(room, 32768)))
        lens = _lens(rng, total, rng.randint(1, 12))
        prefix = [rng.choice([0, 0, rng.randint(1, 200), _logint(rng, 1, 2000 if op == "write" else 500000)])
                  for _ in lens]
        case = dict(op=op, io=io, lens=",".join(map(str, lens)), prefix=",".join(map(str, prefix)), **heads, **turn)
        if op == "rotate":
            return dict(case, fused=rng.random() < 0.5)
        # (values that 4-bit codes stand for are compared in bf16: a value next to the
        # border of two codes may take either)
        bits = 16 if io == "f32" else rng.choice([4, 16])
        return dict(case, bits=bits, page=rng.choice([16, 32, 64, 128]))
    room = 64 * 8192 * 8 * 128 // (hkv * d) // (4 if io == "f32" else 1) // (1 if g <= 8 else 2)
    batch = _logint(rng, 1, 64)
    room = _logint(rng, 16, max(17, min(room // batch, 131072)))
    longest = rng.randint(1, max(1, room - 1))
    case = dict(op=op, io=io, batch=batch, longest=longest, shortest=rng.randint(0, longest), room=room,
                page=rng.choice([16, 32, 64, 128, 256]), **heads)
    return dict(case, **turn) if op == "step" else case


def _ints(text):
    return [int(x) for x in text.split(",")]


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _projection(gen, tokens, heads, d, dt, fused):
    """[tokens, heads_i, d] each, its own tensor or slices of one projection."""
    x = torch.randn(tokens, sum(heads) * d, generator=gen, device="cuda").to(dt)
    parts = torch.split(x, [h * d for h in heads], dim=-1)
    return [(p if fused else p.contiguous()).unflatten(-1, (h, d)) for p, h in zip(parts, heads)]


def _quantise(x):
    """Codes and (step, least) of x [.., D], one pair for each 64 values."""
    x = x.float().unflatten(-1, (-1, _GROUP))
    lo, hi = x.amin(dim=-1, keepdim=True), x.amax(dim=-1, keepdim=True)
    least = lo.clamp(-65504, 65504).half()
    step = ((hi - lo) / 15).clamp(max=65504).half()
    code = torch.round((x - least.float()) / step.float()).clamp(0, 15)
    code = torch.where(step > 0, code, 0).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.cat([step, least], dim=-1)


def _values(codes, scales):
    """What codes [.., D / 2] with scales [.., D / 64, 2] stand for, in fp32."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float().unflatten(-1, (-1, _GROUP))
    return (c * scales[..., :1].float() + scales[..., 1:].float()).flatten(-2)


def _pages(gen, case, rows, dt, fill):
    """Pages for sequences of up to rows[b] rows and their table, entries past the
    last page -1.  Pages of a sequence lie anywhere."""
    page, hkv, d = case["page"], case["hkv"], case["d"]
    need = -(-np.array(rows) // page)
    width = max(int(need.max()), -(-case.get("room", 1) // page))
    n = 3 + (len(rows) * -(-(case["longest"] + 1) // page) if "room" in case else int(need.sum()))
    order = torch.randperm(n, generator=gen, device="cuda").int()
    table = torch.full((len(rows), width), -1, dtype=torch.int32, device="cuda")
    at = np.arange(width) < need[:, None]
    table[torch.from_numpy(at).cuda()] = order[:int(need.sum())]
    st = dict(table=table)
    for x in ("k", "v"):
        if fill == 4:
            codes = torch.empty(n, hkv, page, d // 2, dtype=torch.uint8, device="cuda")
            scales = torch.empty(n, hkv, page, d // _GROUP, 2, dtype=torch.half, device="cuda")
            for i in range(0, n, 1024):
                codes[i:i + 1024], scales[i:i + 1024] = _quantise(
                    torch.randn(codes[i:i + 1024].shape[:-1] + (d,), generator=gen, device="cuda"))
            st[x + "_pages"], st[x + "_scales"] = codes, scales
        else:
            st[x + "_pages"] = torch.randn(n, hkv, page, d, generator=gen, device="cuda", dtype=dt)
            st[x + "_scales"] = None
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["io"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    st = dict(case=case)
    if "rot" in case:
        i = torch.arange(case["rot"] // 2, dtype=torch.float64)
        st["inv_freq"] = (1e6 ** (-2 * i / case["rot"])).float().cuda() if case["rot"] else None
        for x in ("q", "k"):
            st[x + "_weight"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda") if case["norm"] else None
    if case["op"] in ("rotate", "write"):
        lens, pre = _ints(case["lens"]), _ints(case["prefix"])
        fused = case.get("fused", True)
        st["q"], st["k"], st["v"] = _projection(gen, sum(lens), [hq, hkv, hkv], d, dt, fused)
        if case["op"] == "rotate":
            st["positions"] = torch.from_numpy(np.concatenate([p + np.arange(n) for n, p in zip(lens, pre)])).int().cuda()
            return st
        st["cu"] = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        st["cu_all"] = np.concatenate([[0], np.cumsum(np.add(lens, pre))]).astype(np.int64)
        st["lengths"] = torch.tensor(pre, dtype=torch.int32, device="cuda")
        st |= _pages(gen, case, np.add(lens, pre), dt, case["bits"])
        return st
    B, lo, hi = case["batch"], case["shortest"], case["longest"]
    u = torch.rand(B, generator=gen, device="cuda")
    st["lengths"] = (lo + (u * (hi - lo + 1)).floor().clamp_(max=hi - lo)).int()
    st["q"], st["k"], st["v"] = _projection(gen, B, [hq, hkv, hkv], d, dt, case["op"] == "step")
    st |= _pages(gen, case, st["lengths"].cpu().numpy() + 1, dt, 4 if case["op"] == "step4" else 16)
    return st


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import state_space_model_mamba_amd as ssd
        pages = (st.get("k_pages"), st.get("v_pages"), st.get("table"))
        turn = {x: st.get(x) for x in ("inv_freq", "q_weight", "k_weight")}
        turn |= dict(eps=_EPS, interleaved=case.get("pairs") == "next")
        if op == "rotate":
            q, k = ssd.ssd_attn_qk_norm_rope(st["q"], st["k"], st["positions"], **turn)
            return {"q": q, "k": k}
        if op == "write":
            scales = dict(k_scales=st["k_scales"], v_scales=st["v_scales"])
            q = ssd.ssd_attn_paged_append(st["q"], st["k"], st["v"], *pages, st["lengths"], cu_seqlens=st["cu"],
                                          **scales, **turn)
            if case["bits"] == 16:
                return {"q": q, "k": st["k_pages"], "v": st["v_pages"]}
            k, v = ssd.ssd_attn_paged_gather(*pages, st["cu_all"], **scales)
            return {"q": q, "k": k, "v": v}
        if op == "step":
            q = ssd.ssd_attn_paged_append(st["q"], st["k"], st["v"], *pages, st["lengths"], **turn)
            o = ssd.ssd_attn_paged_decode_step(q, *pages, st["lengths"])
            return {"o": o, "k": st["k_pages"], "v": st["v_pages"]}
        return {"o": ssd.ssd_attn_paged_decode_step(st["q"], *pages, st["lengths"], k_scales=st["k_scales"],
                                                    v_scales=st["v_scales"])}
    if op == "rotate":
        cos, sin = _plain_angles(st, st["positions"])
        return {x: _plain_turn(st, x, cos, sin).to(st[x].dtype) for x in ("q", "k")}
    if op == "write":
        return _plain_write(st)
    if op == "step":
        row = st["lengths"].long()
        cos, sin = _plain_angles(st, row)
        q = _plain_turn(st, "q", cos, sin).to(st["q"].dtype)
        _plain_store(st, torch.arange(len(row), device=row.device), row, _plain_turn(st, "k", cos, sin))
        return {"o": _plain_attend(st, q), "k": st["k_pages"], "v": st["v_pages"]}
    return {"o": _plain_attend(st, st["q"])}


def _plain_angles(st, positions):
    if st["inv_freq"] is None:
        return None, None
    a = positions.double()[:, None] * st["inv_freq"].double()
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]      # [T, 1, rot / 2]


def _plain_turn(st, name, cos, sin):
    """The normed and rotated queries or keys in fp32."""
    x, w, r = st[name].float(), st[name + "_weight"], st["case"]["rot"]
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + _EPS) * w
    if r == 0:
        return x
    head, rest = x[..., :r], x[..., r:]
    if st["case"]["pairs"] == "half":
        a, b = head[..., :r // 2], head[..., r // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], dim=-1)
    a, b = head[..., 0::2], head[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2), rest], dim=-1)


def _plain_store(st, seq, row, k):
    """Rows `row` of sequences `seq` become k (fp32) and the tokens' v."""
    page, size = st["table"][seq, row // st["case"]["page"]].long(), st["case"]["page"]
    for name, x in (("k", k), ("v", st["v"])):
        if st[name + "_scales"] is not None:
            codes, scales = _quantise(x)
            st[name + "_pages"][page, :, row % size] = codes
            st[name + "_scales"][page, :, row % size] = scales
        else:
            st[name + "_pages"][page, :, row % size] = x.to(st[name + "_pages"].dtype)


def _rows(cu, first, dev):
    """Sequence and row of every packed token; sequence b starts at row first[b]."""
    n = np.diff(cu)
    seq = torch.from_numpy(np.repeat(np.arange(len(n)), n)).to(dev)
    at = torch.arange(int(cu[-1]), device=dev) - torch.from_numpy(np.repeat(cu[:-1], n)).to(dev)
    return seq, at + first.long()[seq]


def _plain_write(st):
    dev = st["q"].device
    seq, row = _rows(st["cu"], st["lengths"], dev)
    cos, sin = _plain_angles(st, row)
    q = _plain_turn(st, "q", cos, sin).to(st["q"].dtype)
    _plain_store(st, seq, row, _plain_turn(st, "k", cos, sin))
    if st["case"]["bits"] == 16:
        return {"q": q, "k": st["k_pages"], "v": st["v_pages"]}
    seq, row = _rows(st["cu_all"], torch.zeros_like(st["lengths"]), dev)
    size = st["case"]["page"]
    page = st["table"][seq, row // size].long()
    k, v = (_values(st[x + "_pages"][page, :, row % size], st[x + "_scales"][page, :, row % size]).to(q.dtype)
            for x in ("k", "v"))
    return {"q": q, "k": k, "v": v}


def _plain_attend(st, q):
    case = st["case"]
    hkv, at = case["hkv"], st["lengths"].long()
    table = st["table"].long().clamp(min=0)

    def rows(x):                                                     # [B, hkv, rows, D] in fp32
        p = st[x + "_pages"][table].transpose(1, 2).flatten(2, 3)
        if st[x + "_scales"] is None:
            return p.float()
        return _values(p, st[x + "_scales"][table].transpose(1, 2).flatten(2, 3))

    k = rows("k").transpose(-1, -2).contiguous()
    s = torch.matmul(q.float().unflatten(1, (hkv, -1)), k) * case["d"] ** -0.5
    see = torch.arange(s.shape[-1], device=at.device) <= at[:, None]
    s = s.masked_fill_(~see[:, None, None], -math.inf)
    s = torch.exp(s - s.amax(dim=-1, keepdim=True))
    o = torch.matmul(s, rows("v").contiguous()) / s.sum(dim=-1, keepdim=True)
    return o.flatten(1, 2).to(q.dtype)


# --------------------------------------------------------------------------
# The bytes and operations a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    esz = 2 if case["io"] == "bf16" else 4
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    row4 = hkv * (d // 2 + 4 * (d // _GROUP))                        # bytes of one row of 4-bit keys or values
    turn = 8 if case.get("norm") or case.get("rot") else 0           # operations for each value
    if case["op"] in ("rotate", "write"):
        tokens = sum(_ints(case["lens"]))
        if case["op"] == "rotate":
            return {"bytes": 2 * esz * tokens * (hq + hkv) * d, "flops": turn * tokens * (hq + hkv) * d}
        read = esz * tokens * (hq + 2 * hkv) * d
        if case["bits"] == 16:
            return {"bytes": 2 * read, "flops": turn * tokens * (hq + hkv) * d}
        rows = tokens + sum(_ints(case["prefix"]))
        # the new rows need not be read back from memory; the cached ones must be
        return {"bytes": read + esz * tokens * hq * d + 2 * rows * row4 + 2 * esz * rows * hkv * d,
                "flops": tokens * (turn * (hq + hkv) + 16 * hkv) * d + 4 * rows * hkv * d}
    rows = case["batch"] * ((case["shortest"] + case["longest"]) // 2 + 1)
    if case["op"] == "step4":
        return {"bytes": 2 * rows * row4 + 2 * esz * case["batch"] * hq * d, "flops": 4 * rows * hq * d + 4 * rows * hkv * d}
    return {"bytes": 2 * esz * rows * hkv * d + esz * case["batch"] * (2 * hq + 2 * hkv) * d,
            "flops": 4 * rows * hq * d + turn * case["batch"] * (hq + hkv) * d}


# --------------------------------------------------------------------------
# The definition in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotate":
        return {x: _exact_turn(case, st, x, st["positions"]) for x in ("q", "k")}
    if case["op"] == "write":
        lens, pre = _ints(case["lens"]), _ints(case["prefix"])
        row = torch.cat([p + torch.arange(n) for n, p in zip(lens, pre)]).cuda()
        out = {"q": _exact_turn(case, st, "q", row), "k": [], "v": []}
        new = {"k": _exact_turn(case, st, "k", row), "v": st["v"].double()}
        if case["bits"] == 16:
            for x in new:
                out[x] = st[x + "_pages"].double()
                t = 0
                for b, (n, p) in enumerate(zip(lens, pre)):
                    r = torch.arange(p, p + n, device="cuda")
                    out[x][st["table"][b].long()[r // case["page"]], :, r % case["page"]] = new[x][t:t + n]
                    t += n
            return out
        t = 0
        for b, (n, p) in enumerate(zip(lens, pre)):
            for x in new:
                out[x] += [_exact_cached(case, st, x, b, p), _exact_4bit(new[x][t:t + n])]
            t += n
        return {x: out[x] if x == "q" else torch.cat(out[x]) for x in out}
    dt = _DT[case["io"]]
    q, o = st["q"].double(), torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "step":          # the queries and the cache hold numbers of the input type
        q = _exact_turn(case, st, "q", st["lengths"]).to(dt).double()
        new = {"k": _exact_turn(case, st, "k", st["lengths"]).to(dt).double(), "v": st["v"].double()}
    for b, n in enumerate(st["lengths"].tolist()):
        if case["op"] == "step":
            k, v = (torch.cat([_exact_cached(case, st, x, b, n), new[x][b:b + 1]]) for x in ("k", "v"))
        else:
            k, v = (_exact_cached(case, st, x, b, n + 1) for x in ("k", "v"))
        for h in range(case["hq"]):
            j = h // (case["hq"] // case["hkv"])
            o[b, h] = torch.softmax((k[:, j] * q[b, h]).sum(dim=-1) / math.sqrt(case["d"]), dim=0) @ v[:, j]
    return {"o": o} if case["op"] == "step4" else {"o": o, "k": None, "v": None}   # (the pages hold copies)


def _exact_turn(case, st, name, positions):
    x, w, r = st[name].double(), st[name + "_weight"], case["rot"]
    if w is not None:
        x = x / torch.sqrt((x * x).sum(dim=-1, keepdim=True) / case["d"] + _EPS) * w.double()
    if r:
        a = positions.double()[:, None] * st["inv_freq"].double()
        turn = torch.polar(torch.ones_like(a), a)[:, None]           # as complex numbers
        i = torch.arange(r // 2, device="cuda")
        one, two = (i, i + r // 2) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
        z = torch.complex(x[..., one], x[..., two]) * turn
        x = x.clone()
        x[..., one], x[..., two] = z.real, z.imag
    return x


def _exact_cached(case, st, name, b, n):
    """The first n cached rows of sequence b: [n, hkv, D]."""
    page = case["page"]
    of = st["table"][b, :-(-n // page)].long()
    p = st[name + "_pages"][of]
    if st[name + "_scales"] is not None:
        codes = torch.empty(p.shape[:-1] + (case["d"],), dtype=torch.float64, device="cuda")
        codes[..., 0::2], codes[..., 1::2] = (p % 16).double(), (p // 16).double()
        s = st[name + "_scales"][of].double().repeat_interleave(_GROUP, dim=-2)
        p = codes * s[..., 0] + s[..., 1]
    return p.double().transpose(1, 2).flatten(0, 1)[:n]


def _exact_4bit(x):
    """Values [T, hkv, D] as 4-bit codes would give them back."""
    y = torch.empty_like(x)
    for g in range(0, x.shape[-1], _GROUP):
        part = x[..., g:g + _GROUP]
        lo, hi = part.min(dim=-1, keepdim=True).values, part.max(dim=-1, keepdim=True).values
        least, step = lo.half().double(), ((hi - lo) / 15).half().double()
        code = ((part - least) / torch.where(step > 0, step, 1.0)).round().clamp(0, 15)
        y[..., g:g + _GROUP] = code * step + least
    return y
