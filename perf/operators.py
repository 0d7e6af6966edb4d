"""Timed cases of the linear-attention and softmax-attention operators.

Four operators, each with a plain form in elementary torch operations and the
library's own call:

    lin_scan     ssd_linattn_chunk_scan(_varlen): linear attention with one decay per
                 head over whole prompts (batched or packed), with the end states
    lin_step     ssd_linattn_decode_step: one token per sequence, state updated in place
    attn_prefill ssd_attn_prefill: causal softmax attention over packed prompts,
                 grouped heads, optionally on top of keys already in a cache
    attn_step    ssd_attn_decode_step: one token per sequence, appended to a padded
                 key/value cache of which each sequence has filled its own length

A case says which operator it is ("op"), its sizes and its type ("io"); "lens"
lists the lengths of packed sequences.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one short chat prompt: a single odd-sized segment, where launch latency counts
        dict(name="lin_scan_short", op="lin_scan", io="bf16", batch=1, lens="77", hk=16, hv=32,
             dk=128, dv=128, init=False, fused=False),
        # a training-like batch at the small layer's shape (24 heads of 64 values, 128 keys)
        dict(name="lin_scan_8x2048", op="lin_scan", io="bf16", batch=8, lens="2048", hk=8, hv=24,
             dk=128, dv=64, init=False, fused=False),
        # long documents at the Gated DeltaNet layer's shape, q/k/v sliced from one projection
        dict(name="lin_scan_4x8192", op="lin_scan", io="bf16", batch=4, lens="8192", hk=16, hv=32,
             dk=128, dv=128, init=False, fused=True),
        # a serving batch of mixed prompts, continuing from cached states
        dict(name="lin_scan_packed", op="lin_scan", io="bf16", batch=0,
             lens="8192,4097,3000,2048,1500,1024,777,512", hk=16, hv=32, dk=128, dv=128,
             init=True, fused=False),
        # full precision (checks, small research models)
        dict(name="lin_scan_f32", op="lin_scan", io="f32", batch=2, lens="1000", hk=4, hv=8,
             dk=64, dv=64, init=True, fused=False),
        # generation for one user, and for a full serving batch (the state exceeds every cache)
        dict(name="lin_step_1", op="lin_step", io="bf16", batch=1, hk=16, hv=32, dk=128, dv=128),
        dict(name="lin_step_256", op="lin_step", io="bf16", batch=256, hk=16, hv=32, dk=128, dv=128),
        # one long document through a softmax layer
        dict(name="attn_prefill_8192", op="attn_prefill", io="bf16", lens="8192", prefix="0",
             hq=32, hkv=8, d=128, fused=False),
        # the same serving batch of mixed prompts as lin_scan_packed, some on cached prefixes
        dict(name="attn_prefill_packed", op="attn_prefill", io="bf16",
             lens="8192,4097,3000,2048,1500,1024,777,512", prefix="0,0,1000,0,0,4096,0,77",
             hq=32, hkv=8, d=128, fused=True),
        # short requests, full precision, small heads
        dict(name="attn_prefill_f32", op="attn_prefill", io="f32", lens="1,200,65,17,130",
             prefix="0,0,0,0,0", hq=8, hkv=2, d=64, fused=False),
        # generation at a long context for one user, and for a batch at mixed lengths
        dict(name="attn_step_long", op="attn_step", io="bf16", batch=1, cap=131072, longest=131000,
             shortest=131000, hq=32, hkv=8, d=128),
        dict(name="attn_step_64", op="attn_step", io="bf16", batch=64, cap=8192, longest=8190,
             shortest=100, hq=32, hkv=8, d=128),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, total, count):
    """`count` lengths of very different sizes, `total` tokens at most."""
    w = [math.exp(rng.uniform(0.0, 3.0)) for _ in range(count)]
    return [max(1, int(total * x / sum(w))) for x in w]


def draw(rng):
    op = rng.choice(["lin_scan", "lin_scan", "lin_step", "attn_prefill", "attn_prefill", "attn_step"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "lin_scan":
        dk, dv = rng.choice([64, 128, 256]), rng.choice([64, 128, 256])
        r = rng.choice([1, 2, 2, 3, 4])
        hk = rng.choice([1, 3, 4, 8, 16])
        # bounded by the largest listed case: 32768 tokens of 32 heads of 128 x 128
        room = 32768 * 32 * 128 * 128 // (hk * r * dk * dv) // (8 if io == "f32" else 1)
        total = _logint(rng, 1, max(2, min(room, 65536)))
        if rng.random() < 0.5:
            batch = min(rng.choice([1, 2, 4, 7]), total)
            lens = str(total // batch)
        else:
            batch = 0
            lens = ",".join(str(n) for n in _lens(rng, total, rng.randint(1, 12)))
        return dict(op=op, io=io, batch=batch, lens=lens, hk=hk, hv=hk * r, dk=dk, dv=dv,
                    init=rng.random() < 0.5, fused=rng.random() < 0.5)
    if op == "lin_step":
        dk, dv = rng.choice([64, 128, 256]), rng.choice([64, 128, 256])
        r = rng.choice([1, 2, 3, 4])
        hk = rng.choice([1, 3, 4, 8, 16])
        most = 256 * 32 * 128 * 128 // (hk * r * dk * dv)
        return dict(op=op, io=io, batch=_logint(rng, 1, max(2, min(most, 300))), hk=hk, hv=hk * r,
                    dk=dk, dv=dv)
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 8])
    if op == "attn_prefill":
        # query-key pairs bounded by the largest listed case (8192 causal tokens, 32 heads of 128)
        pairs = 8192 * 8192 // 2 * 32 * 128 // (hkv * g * d) // (16 if io == "f32" else 1)
        total = _logint(rng, 1, min(8192, int(math.sqrt(pairs))))
        lens = _lens(rng, total, rng.randint(1, 10))
        prefix = [rng.choice([0, 0, 0, _logint(rng, 1, 1000)]) for _ in lens]
        if sum(n * (n / 2 + p) for n, p in zip(lens, prefix)) > pairs:
            prefix = [0 for _ in lens]
        return dict(op=op, io=io, lens=",".join(map(str, lens)), prefix=",".join(map(str, prefix)),
                    hq=hkv * g, hkv=hkv, d=d, fused=rng.random() < 0.5)
    room = 64 * 8192 * 8 * 128 // (hkv * d) // (4 if io == "f32" else 1)
    batch = _logint(rng, 1, 64)
    cap = _logint(rng, 16, max(17, min(room // batch, 131072)))
    longest = rng.randint(1, cap - 1)
    return dict(op=op, io=io, batch=batch, cap=cap, longest=longest,
                shortest=rng.randint(0, longest), hq=hkv * g, hkv=hkv, d=d)


def _ints(text):
    return [int(x) for x in text.split(",")]


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _projection(gen, tokens, heads, dt, fused):
    """q, k, v [tokens, heads_i, dim_i], each its own tensor or slices of one projection."""
    widths = [h * d for h, d, _ in heads]
    if fused:
        x = torch.randn(*tokens, sum(widths), generator=gen, device="cuda")
        parts = torch.split(x, widths, dim=-1)
        for p, (_, _, s) in zip(parts, heads):
            p.mul_(s)
        parts = torch.split(x.to(dt), widths, dim=-1)
    else:
        parts = [(torch.randn(*tokens, w, generator=gen, device="cuda") * s).to(dt)
                 for w, (_, _, s) in zip(widths, heads)]
    return [p.unflatten(-1, (h, d)) for p, (h, d, _) in zip(parts, heads)]


def _log_decay(hv):
    """Geometric slopes over the heads, the slowest forgetting over some 256 tokens."""
    h = torch.arange(1, hv + 1, dtype=torch.float64)
    return (-torch.exp2(-8.0 * h / hv)).float().cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["io"]]
    st = dict(case=case)
    if case["op"] in ("lin_scan", "lin_step"):
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        heads = [(hk, dk, dk ** -0.5), (hk, dk, dk ** -0.5), (hv, dv, 1.0)]
        st["g"] = _log_decay(hv)
        st["scale"] = 1.0
        if case["op"] == "lin_step":
            st["q"], st["k"], st["v"] = _projection(gen, (case["batch"],), heads, dt, False)
            st["state"] = torch.randn(case["batch"], hv, dk, dv, generator=gen, device="cuda")
            return st
        lens = _ints(case["lens"])
        if case["batch"]:
            tokens, nseq = (case["batch"], lens[0]), case["batch"]
        else:
            tokens, nseq = (sum(lens),), len(lens)
            st["cu"] = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        st["q"], st["k"], st["v"] = _projection(gen, tokens, heads, dt, case["fused"])
        st["init"] = (torch.randn(nseq, hv, dk, dv, generator=gen, device="cuda") * dk ** -0.5
                      if case["init"] else None)
        return st
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    st["scale"] = d ** -0.5
    if case["op"] == "attn_prefill":
        lens, pre = _ints(case["lens"]), _ints(case["prefix"])
        st["cu"] = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        if any(pre):   # keys of the prompt follow the sequence's cached ones
            kl = np.array(lens) + np.array(pre)
            st["kv_lens"] = kl.astype(np.int64)
            st["kv_starts"] = np.concatenate([[0], np.cumsum(kl)[:-1]]).astype(np.int64)
            q, = _projection(gen, (sum(lens),), [(hq, d, 1.0)], dt, False)
            k, v = _projection(gen, (int(kl.sum()),), [(hkv, d, 1.0), (hkv, d, 1.0)], dt, case["fused"])
        else:
            st["kv_lens"] = st["kv_starts"] = None
            q, k, v = _projection(gen, (sum(lens),), [(hq, d, 1.0), (hkv, d, 1.0), (hkv, d, 1.0)], dt,
                                  case["fused"])
        st["q"], st["k"], st["v"] = q, k, v
        return st
    B, M = case["batch"], case["cap"]
    st["q"], st["k"], st["v"] = _projection(gen, (B,), [(hq, d, 1.0), (hkv, d, 1.0), (hkv, d, 1.0)], dt, False)
    st["k_cache"] = torch.randn(B, M, hkv, d, generator=gen, device="cuda", dtype=dt)
    st["v_cache"] = torch.randn(B, M, hkv, d, generator=gen, device="cuda", dtype=dt)
    u = torch.rand(B, generator=gen, device="cuda")
    lo, hi = case["shortest"], case["longest"]
    st["lengths"] = (lo + (u * (hi - lo + 1)).floor().clamp_(max=hi - lo)).to(torch.int32)
    return st


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if own:
        import state_space_model_mamba_amd as ssd
        if op == "lin_scan":
            if st["case"]["batch"]:
                o, fin = ssd.ssd_linattn_chunk_scan(st["q"], st["k"], st["v"], st["g"],
                                                    initial_state=st["init"], scale=st["scale"])
            else:
                o, fin = ssd.ssd_linattn_chunk_scan_varlen(st["q"], st["k"], st["v"], st["g"], st["cu"],
                                                           initial_states=st["init"], scale=st["scale"])
            return {"o": o, "state": fin}
        if op == "lin_step":
            o = ssd.ssd_linattn_decode_step(st["q"], st["k"], st["v"], st["g"], st["state"],
                                            scale=st["scale"])
            return {"o": o, "state": st["state"]}
        if op == "attn_prefill":
            return {"o": ssd.ssd_attn_prefill(st["q"], st["k"], st["v"], st["cu"],
                                              kv_starts=st["kv_starts"], kv_lens=st["kv_lens"],
                                              scale=st["scale"])}
        o = ssd.ssd_attn_decode_step(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"],
                                     st["lengths"], scale=st["scale"])
        return {"o": o, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    if op == "lin_scan":
        return _plain_lin_scan(st)
    if op == "lin_step":
        return _plain_lin_step(st)
    if op == "attn_prefill":
        return _plain_attn_prefill(st)
    return _plain_attn_step(st)


def _plain_lin_scan(st):
    """Chunks of 128 tokens: the masked product inside a chunk, the chunk's end
    state from zero, and every chunk's entering state (and the end states) as one
    product of decays with those."""
    case, C = st["case"], 128
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    r, dev = hv // hk, st["q"].device
    lens = _ints(case["lens"]) if not case["batch"] else [_ints(case["lens"])[0]] * case["batch"]
    lens = np.array(lens)
    base = np.cumsum(lens) - lens
    per = -(-lens // C)
    seq = np.repeat(np.arange(len(lens)), per)                       # the chunk's sequence
    at = (np.arange(per.sum()) - np.repeat(np.cumsum(per) - per, per)) * C   # its first token there
    n = np.minimum(C, lens[seq] - at)                                # its tokens
    seq, at, n, base, lens = (torch.from_numpy(np.ascontiguousarray(a)).to(dev)
                              for a in (seq, at, n, base, lens))
    t = torch.arange(C, device=dev)
    ok = t < n[:, None]
    idx = torch.where(ok, (base[seq] + at)[:, None] + t, 0)
    g = st["g"].double()

    def tokens(x, heads, dim):   # [chunks, heads, C, dim], zero past the end
        x = x.reshape(-1, heads, dim)[idx].float()
        return (x * ok[:, :, None, None]).transpose(1, 2).contiguous()

    q, k, v = tokens(st["q"], hk, dk), tokens(st["k"], hk, dk), tokens(st["v"], hv, dv)
    v = v.unflatten(1, (hk, r))
    gap = (t[:, None] - t).clamp(min=0)
    mask = torch.where(t[:, None] >= t, torch.exp(g[:, None, None] * gap), 0).float()
    p = torch.matmul(q, k.transpose(-1, -2).contiguous())[:, :, None] * mask.unflatten(0, (hk, r))
    o = torch.matmul(p, v)
    w = torch.exp(g[:, None] * (n[:, None, None] - 1 - t).clamp(min=0)).float()   # [chunks, hv, C]
    kw = k[:, :, None] * w.unflatten(1, (hk, r))[..., None]
    z = torch.matmul(kw.transpose(-1, -2).contiguous(), v)           # [chunks, hk, r, dk, dv]
    z = z.flatten(1, 2).transpose(0, 1).reshape(hv, len(n), dk * dv)
    # rows: every chunk's entering state, then every sequence's end state
    row_seq = torch.cat([seq, torch.arange(len(lens), device=dev)])
    row_at = torch.cat([at, lens])
    dist = row_at[:, None] - (at + n)
    m = torch.where((row_seq[:, None] == seq) & (dist >= 0),
                    torch.exp(g[:, None, None] * dist.clamp(min=0)), 0).float()
    s = torch.matmul(m, z)                                           # [hv, rows, dk dv]
    if st["init"] is not None:
        first = torch.exp(g[:, None] * row_at).float()
        s = s + first[:, :, None] * st["init"].flatten(2).transpose(0, 1)[:, row_seq]
    s = s.reshape(hk, r, len(row_at), dk, dv)
    into = s[:, :, :len(n)].permute(2, 0, 1, 3, 4).contiguous()
    qd = q[:, :, None] * torch.exp(g[:, None] * (t + 1)).float().unflatten(0, (hk, r))[..., None]
    o = (o + torch.matmul(qd, into)) * st["scale"]
    out = torch.empty(st["v"].shape, dtype=st["v"].dtype, device=dev)
    o = o.flatten(1, 2).transpose(1, 2)                              # [chunks, C, hv, dv]
    out.view(-1, hv, dv)[idx[ok]] = o[ok].to(out.dtype)
    end = s[:, :, len(n):].flatten(0, 1).transpose(0, 1).contiguous()
    return {"o": out, "state": end}


def _plain_lin_step(st):
    case = st["case"]
    r = case["hv"] // case["hk"]
    q, k = (st[x].float().repeat_interleave(r, dim=1) for x in ("q", "k"))
    s = st["state"]
    s.mul_(torch.exp(st["g"].double()).float()[:, None, None]).add_(k[..., None] * st["v"].float()[:, :, None])
    o = (s * q[..., None]).sum(dim=2) * st["scale"]
    return {"o": o.to(st["v"].dtype), "state": s}


def _plain_attn_prefill(st):
    """Sequences of about one length together (padded to the longest of them)."""
    case, dev = st["case"], st["q"].device
    hkv, d = case["hkv"], case["d"]
    grp = case["hq"] // hkv
    lq = np.diff(st["cu"])
    qs = st["cu"][:-1]
    lk = lq if st["kv_lens"] is None else st["kv_lens"]
    ks = qs if st["kv_starts"] is None else st["kv_starts"]
    out = torch.empty_like(st["q"], memory_format=torch.contiguous_format)
    size = np.ceil(2 * np.log2(lq)).astype(int) * 64 + np.ceil(2 * np.log2(lk)).astype(int)
    for b in np.unique(size):
        of = np.nonzero(size == b)[0]
        nq, nk, q0, k0 = (torch.from_numpy(np.ascontiguousarray(a[of])).to(dev) for a in (lq, lk, qs, ks))
        i = torch.arange(int(lq[of].max()), device=dev)
        j = torch.arange(int(lk[of].max()), device=dev)
        okq, okk = i < nq[:, None], j < nk[:, None]
        q = st["q"][torch.where(okq, q0[:, None] + i, 0)].float()
        k = st["k"][torch.where(okk, k0[:, None] + j, 0)].float()
        v = st["v"][torch.where(okk, k0[:, None] + j, 0)].float() * okk[..., None, None]
        q = q.unflatten(2, (hkv, grp)).permute(0, 2, 3, 1, 4).contiguous()      # [n, hkv, grp, i, d]
        k = k.permute(0, 2, 3, 1).contiguous()                                  # [n, hkv, d, j]
        v = v.permute(0, 2, 1, 3).contiguous()                                  # [n, hkv, j, d]
        s = torch.matmul(q.flatten(2, 3), k).mul_(st["scale"]).unflatten(2, (grp, len(i)))
        see = j <= (nk - nq)[:, None, None] + i[:, None]                        # [n, i, j]
        see = (see & okk[:, None])[:, None, None]
        s = s.masked_fill_(~see, -math.inf)
        top = s.amax(dim=-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
        s = s.sub_(top).exp_()
        den = s.sum(dim=-1, keepdim=True)
        o = torch.matmul(s.flatten(2, 3), v).unflatten(2, (grp, len(i)))
        o = torch.where(den > 0, o / den, 0).permute(0, 3, 1, 2, 4).flatten(2, 3)
        out[(q0[:, None] + i)[okq]] = o[okq].to(out.dtype)
    return {"o": out}


def _plain_attn_step(st):
    case = st["case"]
    hkv, d = case["hkv"], case["d"]
    grp = case["hq"] // hkv
    at = st["lengths"].long()
    b = torch.arange(len(at), device=at.device)
    st["k_cache"][b, at] = st["k"]
    st["v_cache"][b, at] = st["v"]
    q = st["q"].float().unflatten(1, (hkv, grp))
    k = st["k_cache"].permute(0, 2, 3, 1).float().contiguous()      # [B, hkv, d, M]
    s = torch.matmul(q, k) * st["scale"]
    see = torch.arange(case["cap"], device=at.device) <= at[:, None]
    s = s.masked_fill_(~see[:, None, None], -math.inf)
    s = torch.exp(s - s.amax(dim=-1, keepdim=True))
    v = st["v_cache"].permute(0, 2, 1, 3).float().contiguous()
    o = torch.matmul(s, v) / s.sum(dim=-1, keepdim=True)
    return {"o": o.flatten(1, 2).to(st["q"].dtype), "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


# --------------------------------------------------------------------------
# The bytes and operations a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    esz = 2 if case["io"] == "bf16" else 4
    if case["op"] in ("lin_scan", "lin_step"):
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        state = 4 * hv * dk * dv
        if case["op"] == "lin_step":
            tokens, states = case["batch"], 2 * case["batch"]
        else:
            lens = _ints(case["lens"])
            nseq = case["batch"] or len(lens)
            tokens = sum(lens) if not case["batch"] else case["batch"] * lens[0]
            states = nseq * (2 if case["init"] else 1)
        return {"bytes": tokens * esz * 2 * (hk * dk + hv * dv) + states * state + 4 * hv,
                "flops": 4 * tokens * hv * dk * dv}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "attn_prefill":
        lens, pre = _ints(case["lens"]), _ints(case["prefix"])
        pairs = sum(n * (n + 1) // 2 + n * p for n, p in zip(lens, pre))
        tokens, keys = sum(lens), sum(lens) + sum(pre)
    else:
        tokens = case["batch"]
        pairs = keys = tokens * ((case["shortest"] + case["longest"]) // 2 + 1)
    return {"bytes": esz * d * 2 * (tokens * hq + keys * hkv), "flops": 4 * pairs * hq * d}


# --------------------------------------------------------------------------
# The definition in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "lin_scan":
        return _exact_lin_scan(case, st)
    if case["op"] == "lin_step":
        hk, hv = case["hk"], case["hv"]
        s = st["state"].double() * st["g"].double().exp()[:, None, None]
        o = torch.empty(case["batch"], hv, case["dv"], dtype=torch.float64, device="cuda")
        for j in range(hv):
            k, q = st["k"][:, j // (hv // hk)].double(), st["q"][:, j // (hv // hk)].double()
            s[:, j] += k[:, :, None] * st["v"][:, j].double()[:, None, :]
            o[:, j] = (q[:, None, :] @ s[:, j])[:, 0] * st["scale"]
        return {"o": o, "state": s}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "attn_prefill":
        o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        for b in range(len(st["cu"]) - 1):
            q0, q1 = int(st["cu"][b]), int(st["cu"][b + 1])
            k0 = q0 if st["kv_starts"] is None else int(st["kv_starts"][b])
            nk = q1 - q0 if st["kv_lens"] is None else int(st["kv_lens"][b])
            pos = torch.arange(q1 - q0, device="cuda") + nk - (q1 - q0)
            hide = torch.arange(nk, device="cuda") > pos[:, None]
            for h in range(hq):
                k, v = (st[x][k0:k0 + nk, h // (hq // hkv)].double() for x in ("k", "v"))
                a = (st["q"][q0:q1, h].double() @ k.T.contiguous()) * st["scale"]
                o[q0:q1, h] = torch.softmax(a.masked_fill(hide, -math.inf), dim=-1) @ v
        return {"o": o}
    o = torch.zeros(case["batch"], hq, d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lengths"].tolist()):
        k, v = (torch.cat([st[x + "_cache"][b, :n], st[x][b:b + 1]]).double().transpose(0, 1).contiguous()
                for x in ("k", "v"))                                # [hkv, n + 1, d]
        q = st["q"][b].double().unflatten(0, (hkv, hq // hkv))
        a = (q @ k.transpose(1, 2).contiguous()) * st["scale"]
        o[b] = (torch.softmax(a, dim=-1) @ v).flatten(0, 1)
    return {"o": o, "k_cache": None, "v_cache": None}   # (the caches hold copies)


def _exact_lin_scan(case, st):
    """Every output as the sum over all earlier tokens, one head of one sequence at a time."""
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    lens = _ints(case["lens"]) if not case["batch"] else [_ints(case["lens"])[0]] * case["batch"]
    q, k, v = (st[x].reshape(-1, h, e) for x, h, e in (("q", hk, dk), ("k", hk, dk), ("v", hv, dv)))
    o = torch.empty(v.shape, dtype=torch.float64, device="cuda")
    end = torch.empty(len(lens), hv, dk, dv, dtype=torch.float64, device="cuda")
    g = st["g"].double()
    t0 = 0
    for b, n in enumerate(lens):
        t = torch.arange(n, dtype=torch.float64, device="cuda")
        for j in range(hv):
            qj, kj = (x[t0:t0 + n, j // (hv // hk)].double() for x in (q, k))
            vj = v[t0:t0 + n, j].double()
            s0 = torch.zeros(dk, dv, dtype=torch.float64, device="cuda") if st["init"] is None else st["init"][b, j].double()
            end[b, j] = (kj * torch.exp(g[j] * (n - 1 - t))[:, None]).T.contiguous() @ vj + torch.exp(g[j] * n) * s0
            for i in range(0, n, 8192):
                rows = slice(i, min(n, i + 8192))
                gap = t[rows, None] - t[None, :rows.stop]
                a = (qj[rows] @ kj[:rows.stop].T.contiguous()) * torch.exp(g[j] * gap.clamp(min=0)) * (gap >= 0)
                y = a @ vj[:rows.stop] + torch.exp(g[j] * (t[rows, None] + 1)) * (qj[rows] @ s0)
                o[t0 + i:t0 + rows.stop, j] = y * st["scale"]
        t0 += n
    return {"o": o.view(st["v"].shape), "state": end}
