"""Cases that time attention with shaped scores (tanh cap, distance bias, document,
prefix and window masks), its gradients, its decode over a key/value cache with
accumulated attention weights, and the eviction of cache slots by those weights.

``own = False`` computes each operator from its formula with elementary torch
operations in 32 bits; ``own = True`` calls the package.
"""
import math
import random

import torch

own = False

# ------------------------------------------------------------------- cases ---
#
# "fwd":    one forward pass (inference prefill).
# "step":   forward and backward, as a training step runs them.
# "decode": the newest q_len tokens of each sequence against its cache.
# "evict":  each (sequence, kv head) keeps `keep` slots of its cache.
# mask: "none", "docs" (documents packed in one row), "prefix" (keys of the prompt
# visible to all), "window" (the last `window` keys).


def _train(name, op, dtype, B, N, H, H_kv, D, causal=True, cap=0.0, alibi=False, mask="none",
           arg=0, mult=1.0):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "N": N, "H": H, "H_kv": H_kv, "D": D,
            "causal": causal, "cap": cap, "alibi": alibi, "mask": mask, "arg": arg, "mult": mult}


def _dec(name, B, lo, hi, q_len, H, H_kv, D, page=0, cap=0.0, alibi=False, window=0,
         weights=True):
    return {"name": name, "op": "decode", "B": B, "lo": lo, "hi": hi, "q_len": q_len, "H": H,
            "H_kv": H_kv, "D": D, "page": page, "cap": cap, "alibi": alibi, "window": window,
            "weights": weights}


def _ev(name, B, lo, hi, H_kv, D, keep, recent, page=0):
    return {"name": name, "op": "evict", "B": B, "lo": lo, "hi": hi, "H_kv": H_kv, "D": D,
            "keep": keep, "recent": recent, "page": page}


def listed():
    return [
        # The small float32 configuration: launch latency.
        _train("fwd_f32_b1_h2_n128_d64", "fwd", "f32", 1, 128, 2, 2, 64, cap=30.0, alibi=True),
        # Half-width heads with a distance bias: prefill of a small model.
        _train("fwd_b4_h16_n2048_d64_alibi", "fwd", "bf16", 4, 2048, 16, 16, 64, alibi=True),
        # Long causal prefill with capped scores (logits of standard deviation 4).
        _train("fwd_b2_h16_n8192_d128_cap", "fwd", "bf16", 2, 8192, 16, 16, 128, cap=50.0,
               mult=2.0),
        # Prefix mask, grouped heads, an odd length: prompt read both ways, answer causal.
        _train("fwd_b2_h16_kv4_n4001_d128_prefix", "fwd", "bf16", 2, 4001, 16, 4, 128,
               causal=False, cap=50.0, mask="prefix", arg=1500, mult=2.0),
        # Training step, long causal sequence, capped scores, grouped heads.
        _train("step_b1_h16_kv4_n8192_d128_cap", "step", "bf16", 1, 8192, 16, 4, 128, cap=50.0,
               mult=2.0),
        # Training step on packed documents with a distance bias, half-width heads, odd length.
        _train("step_b2_h8_n1537_d64_docs_alibi", "step", "bf16", 2, 1537, 8, 8, 64, alibi=True,
               mask="docs", arg=5),
        # Small float32 step with a window: gradient checks and tests of a trainer.
        _train("step_f32_b1_h4_kv2_n200_d64_window", "step", "f32", 1, 200, 4, 2, 64, cap=30.0,
               mask="window", arg=48),
        # One request, short cache: latency of a decode step.
        _dec("decode_b1_h16_kv2_len700_d64", 1, 700, 700, 1, 16, 2, 64, cap=30.0),
        # A serving batch over pages of 64 rows.
        _dec("decode_b16_h32_kv8_d128_paged64", 16, 4096, 32768, 1, 32, 8, 128, page=64,
             cap=50.0),
        # Eight new tokens a sequence (a verify step), distance bias, last 4096 keys.
        _dec("decode_b16_h32_kv8_d128_q8_window", 16, 4096, 32768, 8, 32, 8, 128, alibi=True,
             window=4096),
        # One request drops to 512 slots.
        _ev("evict_b1_kv8_len1500_d128", 1, 1500, 1500, 8, 128, 512, 32),
        # A serving batch drops to 2048 slots, from pages of 64 rows.
        _ev("evict_b16_kv8_d128_paged64", 16, 4096, 32768, 8, 128, 2048, 64, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "step", "step", "decode", "decode", "evict"])
    H_kv = rng.choice([1, 2, 3, 4, 8])
    if op in ("fwd", "step"):
        # A query with one key has a gradient of zero: a step of such queries alone has
        # rounding errors for dQ and dK, which no two computations share.
        least = 1 if op == "fwd" else 24
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        H = H_kv * rng.choice([1, 2, 4])
        if dtype == "f32":   # the float32 path: small, any head size
            H_kv = min(H_kv, 4)
            H, D, B = H_kv * rng.choice([1, 2]), rng.choice([16, 40, 64, 128]), rng.choice([1, 2])
            N = _log(rng, least, 400)
        else:
            D, B = rng.choice([64, 128]), rng.choice([1, 2, 3, 4])
            N = _log(rng, least, 8192)
            while B * H * N * N > 1.0e9:
                N = N * 2 // 3
        mask = rng.choice(["none", "docs", "prefix", "window"])
        arg = {"none": 0, "docs": rng.randint(1, 9), "prefix": rng.randint(0, N),
               "window": _log(rng, (least + 2) // 3, max(least, N))}[mask]
        cap = rng.choice([0.0, 20.0, 50.0])
        c = _train("", op, dtype, B, N, H, H_kv, D, mask != "prefix", cap,
                   cap == 0.0 or rng.random() < 0.3, mask, arg, 2.0 if cap else 1.0)
    elif op == "decode":
        H = H_kv * rng.choice([1, 2, 4, 7, 8])
        lo, B = _log(rng, 1, 8000), _log(rng, 1, 24)
        cap = rng.choice([0.0, 30.0, 50.0])
        c = _dec("", B, lo, lo * rng.choice([1, 2, 4]), rng.choice([1, 1, 2, 5, 8]), H, H_kv,
                 rng.choice([64, 128]), rng.choice([0, 0, 16, 64, 128, 256]), cap,
                 cap == 0.0 or rng.random() < 0.3, rng.choice([0, 0, _log(rng, 1, 5000)]),
                 rng.random() < 0.6)
    else:
        lo = _log(rng, 1, 8000)
        hi = lo * rng.choice([1, 2, 4])
        keep = _log(rng, 1, max(2, hi // 2))
        c = _ev("", _log(rng, 1, 24), lo, hi, H_kv, rng.choice([64, 128]), keep,
                rng.randint(0, keep), rng.choice([0, 0, 16, 64, 128, 256]))
    del c["name"]
    return c


# The layout of a case that is no random input: document borders, cache lengths.


def _plan(case):
    return random.Random("%(B)d %(H_kv)d %(D)d" % case + str(case.get("N", case.get("hi"))))


def _ranges(case):
    """Per sequence, per query: first visible key, and one past the last."""
    r, N = _plan(case), case["N"]
    out = []
    for _ in range(case["B"]):
        lo, hi = [0] * N, [N] * N
        if case["mask"] == "docs":
            cuts = [0] + sorted(r.randint(0, N) for _ in range(case["arg"] - 1)) + [N]
            for a, b in zip(cuts, cuts[1:]):
                lo[a:b], hi[a:b] = [a] * (b - a), [b] * (b - a)
        elif case["mask"] == "prefix":
            hi = [max(i + 1, case["arg"]) for i in range(N)]
        elif case["mask"] == "window":
            lo = [max(0, i + 1 - case["arg"]) for i in range(N)]
        out.append((lo, hi))
    return out


def _lengths(case):
    r = _plan(case)
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


# ------------------------------------------------------------------- state ---


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _slopes(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    if case["op"] in ("fwd", "step"):
        B, N, H, H_kv, D = (case[k] for k in ("B", "N", "H", "H_kv", "D"))
        s["q"], s["k"] = normal(B, N, H, D) * case["mult"], normal(B, N, H_kv, D) * case["mult"]
        s["v"] = normal(B, N, H_kv, D)
        if case["op"] == "step":
            s["dout"] = normal(B, N, H, D)
        s["slopes"] = _slopes(H) if case["alibi"] else None
        s["begin"] = s["end"] = None
        if case["mask"] != "none":
            lo, hi = zip(*_ranges(case))
            s["begin"] = torch.tensor(lo, dtype=torch.int32, device="cuda")
            s["end"] = torch.tensor(hi, dtype=torch.int32, device="cuda")
        return s
    B, H_kv, D, page = case["B"], case["H_kv"], case["D"], case["page"]
    lens = _lengths(case)
    s["max_len"] = max(lens)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if page:
        n_pages = -(-max(lens) // page)
        table = torch.full((B, n_pages), -1, dtype=torch.int32)
        order = list(range(sum(-(-n // page) for n in lens) + 3))
        random.Random(seed).shuffle(order)
        rows = len(order) * page
        for b, n in enumerate(lens):
            for i in range(-(-n // page)):
                table[b, i] = order.pop()
        s["table"], s["page_size"] = table.cuda(), page
    else:
        rows, s["table"], s["page_size"] = B * max(lens), None, max(lens)
    s["k"], s["v"] = normal(rows, H_kv, D), normal(rows, H_kv, D)
    # Weights that earlier steps have accumulated, equal ones among them.
    w = torch.rand(B, H_kv, max(lens), generator=g, device="cuda")
    s["w"] = torch.floor(torch.log(w + 1e-6).square() * 512) / 512
    s["w"] *= torch.arange(max(lens), device="cuda") < s["lens"][:, None, None]
    if case["op"] == "decode":
        s["q"] = normal(B * case["q_len"], case["H"], D) * (3.0 if case["cap"] else 1.0)
        s["slopes"] = _slopes(case["H"]) if case["alibi"] else None
    else:
        s["k_out"], s["v_out"] = (torch.zeros(B * case["keep"], H_kv, D, device="cuda", dtype=dt)
                                  for _ in range(2))
    return s


# --------------------------------------------------------------- one pass ---


def run(s):
    return {"fwd": _fwd, "step": _step, "decode": _decode, "evict": _evict}[s["op"]](s)


def _fwd(s):
    if own:
        import exact_io_aware_tmem_b200 as fa
        return fa.fwd(s["q"], s["k"], s["v"], causal=s["causal"], softcap=s["cap"] or None,
                      alibi_slopes=s["slopes"], key_begin=s["begin"], key_end=s["end"])
    z, _ = _logits(s)
    p, lse = _softmax(z)
    v = s["v"].float().permute(0, 2, 1, 3)[:, :, None]
    return _tokens(p @ v).to(s["q"].dtype), lse.flatten(1, 2)


def _step(s):
    if own:
        import exact_io_aware_tmem_b200 as fa
        kw = dict(causal=s["causal"], softcap=s["cap"] or None, alibi_slopes=s["slopes"],
                  key_begin=s["begin"], key_end=s["end"])
        o, lse = fa.fwd(s["q"], s["k"], s["v"], **kw)
        return (o, lse) + tuple(fa.bwd(s["dout"], s["q"], s["k"], s["v"], o, lse, **kw))
    B, N, H, D = s["q"].shape
    z, slope = _logits(s)
    p, lse = _softmax(z)
    del z
    q, do = (_grouped(s[n], s["H_kv"]) for n in ("q", "dout"))
    k, v = (s[n].float().permute(0, 2, 1, 3)[:, :, None] for n in ("k", "v"))
    o = p @ v
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = do @ v.transpose(-1, -2)
    ds -= (o * do).sum(-1, keepdim=True)
    ds *= p
    if slope is not None:
        ds *= slope
    ds *= 1.0 / math.sqrt(D)
    dq, dk = ds @ k, (ds.transpose(-1, -2) @ q).sum(2)
    dt = s["q"].dtype
    return (_tokens(o).to(dt), lse.flatten(1, 2), _tokens(dq).to(dt),
            dk.permute(0, 2, 1, 3).to(dt).contiguous(), dv.permute(0, 2, 1, 3).to(dt).contiguous())


def _grouped(x, H_kv):
    """[B, N, H, D] -> float32 [B, H_kv, H / H_kv, N, D]."""
    B, N, H, D = x.shape
    return x.float().view(B, N, H_kv, H // H_kv, D).permute(0, 2, 3, 1, 4)


def _tokens(x):
    """[B, H_kv, g, N, D] -> [B, N, H, D]."""
    B, H_kv, g, N, D = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(B, N, H_kv * g, D)


def _logits(s):
    """Shaped scores, -inf where hidden, and the cap's derivative (None: no cap)."""
    B, N, H, D = s["q"].shape
    q, k = _grouped(s["q"], s["H_kv"]), s["k"].float().permute(0, 2, 1, 3)[:, :, None]
    z = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    slope = None
    if s["cap"]:
        z = torch.tanh(z / s["cap"])
        if s["op"] == "step":
            slope = 1.0 - z * z
        z *= s["cap"]
    pos = torch.arange(N, device="cuda")
    if s["slopes"] is not None:
        dist = (pos[:, None] - pos[None, :]).abs().float()
        z -= s["slopes"].view(s["H_kv"], -1, 1, 1) * dist
    hidden = torch.zeros(1, N, N, dtype=torch.bool, device="cuda")
    if s["causal"]:
        hidden = hidden | (pos[None, :] > pos[:, None])
    if s["begin"] is not None:
        hidden = hidden | (pos < s["begin"][:, :, None]) | (pos >= s["end"][:, :, None])
    return z.masked_fill_(hidden[:, None, None], -math.inf), slope


def _softmax(z):
    """Rows that see no key give zeros and a log-sum-exp of -inf."""
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(l, -math.inf))
    p /= torch.where(l > 0, l, torch.ones_like(l))
    return p, lse.squeeze(-1)


def _cache_rows(s):
    """Row of every position of every sequence; positions past the end give row 0."""
    j = torch.arange(s["max_len"], device="cuda")
    if s["table"] is None:
        r = torch.arange(s["B"], device="cuda")[:, None] * s["page_size"] + j
    else:
        r = s["table"].long()[:, j // s["page_size"]] * s["page_size"] + j % s["page_size"]
    return torch.where(j < s["lens"][:, None], r, torch.zeros_like(r))


def _decode(s):
    w = s["w"] if s["weights"] else None
    if own:
        import exact_io_aware_tmem_b200 as fa
        o, lse = fa.decode(s["q"], s["k"], s["v"], s["lens"], q_len=s["q_len"],
                           max_seqlen_k=s["max_len"], block_table=s["table"],
                           page_size=s["page_size"], softcap=s["cap"] or None,
                           alibi_slopes=s["slopes"], window=s["window"] or None, key_weights=w)
        return (o, lse) if w is None else (o, lse, w)
    B, Q, H, H_kv, D = (s[n] for n in ("B", "q_len", "H", "H_kv", "D"))
    rows = _cache_rows(s)
    k, v = (s[n][rows].permute(0, 2, 1, 3)[:, :, None].float() for n in ("k", "v"))
    q = s["q"].float().view(B, Q, H_kv, H // H_kv, D).permute(0, 2, 3, 1, 4)
    z = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    if s["cap"]:
        z = torch.tanh(z / s["cap"]) * s["cap"]
    j = torch.arange(s["max_len"], device="cuda")
    i = s["lens"][:, None] - Q + torch.arange(Q, device="cuda")
    dist = i[:, :, None] - j
    if s["slopes"] is not None:
        z -= s["slopes"].view(H_kv, -1, 1, 1) * dist[:, None, None].abs().float()
    hidden = dist < 0
    if s["window"]:
        hidden = hidden | (dist >= s["window"])
    p, lse = _softmax(z.masked_fill_(hidden[:, None, None], -math.inf))
    o = (p @ v).permute(0, 3, 1, 2, 4).reshape(B * Q, H, D).to(s["q"].dtype)
    lse = lse.permute(0, 3, 1, 2).reshape(B * Q, H)
    if w is None:
        return o, lse
    w += p.sum((2, 3))
    return o, lse, w


def _evict(s):
    keep, recent = s["keep"], s["recent"]
    if own:
        import exact_io_aware_tmem_b200 as fa
        return fa.evict(s["k"], s["v"], s["lens"], s["w"], keep=keep, recent=recent,
                        max_seqlen_k=s["max_len"], block_table=s["table"],
                        page_size=s["page_size"], k_out=s["k_out"], v_out=s["v_out"])
    B, H_kv, D = s["B"], s["H_kv"], s["D"]
    lens = s["lens"].long()[:, None, None]
    new = lens.clamp(max=keep)
    j = torch.arange(s["max_len"], device="cuda")
    # The recent slots go first, then the others by weight, then what is no slot.
    score = s["w"].masked_fill(j >= lens - recent, math.inf).masked_fill(j >= lens, -math.inf)
    n = min(keep, s["max_len"])
    first = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :n]
    at = torch.arange(n, device="cuda")
    slots = torch.sort(first.masked_fill(at >= new, 1 << 40), -1).values
    live = slots < (1 << 40)
    slots = slots.masked_fill(~live, 0)
    b, hk = torch.arange(B, device="cuda")[:, None, None], torch.arange(H_kv, device="cuda")[:, None]
    src = _cache_rows(s)[b, slots]
    for a, c in (("k", "k_out"), ("v", "v_out")):
        dst = s[c].view(B, keep, H_kv, D)[:, :n]
        moved = s[a][src, hk].permute(0, 2, 1, 3)
        dst.copy_(torch.where(live.permute(0, 2, 1)[..., None], moved, dst))
    w = s["w"].new_zeros(B, H_kv, keep)
    w[..., :n] = s["w"].gather(-1, slots).masked_fill(~live, 0.0)
    pos = torch.full((B, H_kv, keep), -1, dtype=torch.int32, device="cuda")
    pos[..., :n] = slots.masked_fill(~live, -1).int()
    return s["k_out"], s["v_out"], new.view(B).int(), w, pos


# -------------------------------------------------------------------- work ---


def _pairs(case):
    """Visible (query, key) pairs of one head over the batch."""
    n = 0
    for lo, hi in _ranges(case):
        n += sum(max(0, (min(b, i + 1) if case["causal"] else b) - a)
                 for i, (a, b) in enumerate(zip(lo, hi)))
    return n


def work(case):
    if case["op"] in ("fwd", "step"):
        B, N, H, H_kv, D = (case[k] for k in ("B", "N", "H", "H_kv", "D"))
        e = 4 if case["dtype"] == "f32" else 2
        q, kv, lse = B * N * H * D * e, B * N * H_kv * D * e, B * N * H * 4
        f = 4.0 * D * _pairs(case) * H
        if case["op"] == "fwd":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": f}
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 3.5 * f}
    H_kv, D, lens = case["H_kv"], case["D"], _lengths(case)
    if case["op"] == "decode":
        Q, H = case["q_len"], case["H"]
        seen = [min(n, case["window"] + Q - 1) if case["window"] else n for n in lens]
        rows = case["B"] * Q * H
        return {"bytes": sum(seen) * H_kv * (4 * D + (8 if case["weights"] else 0)) +
                rows * (4 * D + 4), "flops": 4.0 * D * Q * H * sum(seen)}
    kept = sum(min(n, case["keep"]) for n in lens) * H_kv
    return {"bytes": kept * (8 * D + 8) + sum(lens) * H_kv * 4, "flops": 0.0}


# ----------------------------------------------------- results in 64 bits ---


def exact(case, seed):
    s = prepare(case, seed)
    return {"fwd": _exact_train, "step": _exact_train, "decode": _exact_decode,
            "evict": _exact_evict}[case["op"]](case, s)


def _exact_train(case, s):
    """One kv head of one sequence at a time; the gradients by differentiating the loss."""
    B, N, H, H_kv, D = (case[k] for k in ("B", "N", "H", "H_kv", "D"))
    g = H // H_kv
    step = case["op"] == "step"
    new = lambda h: torch.zeros(B, N, h, D, dtype=torch.float64, device="cuda")  # noqa: E731
    o, lse = new(H), torch.zeros(B, H, N, dtype=torch.float64, device="cuda")
    dq, dk, dv = (new(H), new(H_kv), new(H_kv)) if step else (None, None, None)
    i = torch.arange(N, device="cuda", dtype=torch.float64)
    bounds = _ranges(case)
    for b in range(B):
        lo, hi = (torch.tensor(x, device="cuda")[:, None] for x in bounds[b])
        see = (i >= lo) & (i < hi)
        if case["causal"]:
            see = see & (i[:, None] >= i)
        for c in range(H_kv):
            q, k, v = (s["q"][b, :, c * g:(c + 1) * g].double(), s["k"][b, :, c].double(),
                       s["v"][b, :, c].double())
            leaves = [x.requires_grad_(step) for x in (q, k, v)]
            for h in range(g):
                x = torch.matmul(q[:, h], k.T) / D ** 0.5
                if case["cap"]:
                    x = x.div(case["cap"]).tanh().mul(case["cap"])
                if case["alibi"]:
                    x = x - 2.0 ** (-8.0 * (c * g + h + 1) / H) * torch.cdist(i[:, None], i[:, None], p=1)
                x = torch.where(see, x, torch.tensor(-math.inf, device="cuda", dtype=torch.float64))
                any_key = see.any(1)
                y = torch.where(any_key, torch.logsumexp(x, 1), torch.zeros_like(i))
                out = torch.where(see, (x - y[:, None]).exp(), torch.zeros_like(x)) @ v
                o[b, :, c * g + h] = out.detach()
                lse[b, c * g + h] = torch.where(any_key, y, torch.full_like(y, -math.inf)).detach()
                if step:
                    (out * s["dout"][b, :, c * g + h].double()).sum().backward()
                del x, y, out
            if step:
                dq[b, :, c * g:(c + 1) * g], dk[b, :, c], dv[b, :, c] = (x.grad for x in leaves)
    return (o, lse, dq, dk, dv) if step else (o, lse)


def _exact_decode(case, s):
    B, Q, H, H_kv, D = (case[k] for k in ("B", "q_len", "H", "H_kv", "D"))
    g, lens = H // H_kv, _lengths(case)
    o = torch.zeros(B, Q, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Q, H), -math.inf, dtype=torch.float64, device="cuda")
    w = s["w"].double()
    for b, n in enumerate(lens):
        if s["table"] is None:
            at = torch.arange(n, device="cuda") + b * s["page_size"]
        else:
            pages = s["table"][b].long()[:, None] * case["page"]
            at = (pages + torch.arange(case["page"], device="cuda")).reshape(-1)[:n]
        keys, values = s["k"][at].double(), s["v"][at].double()
        j = torch.arange(n, device="cuda")
        for t in range(Q):
            here = n - Q + t
            see = j <= here
            if case["window"]:
                see = see & (j > here - case["window"])
            if here < 0 or not n:
                continue
            for h in range(H):
                x = keys[see, h // g] @ s["q"][b * Q + t, h].double() / math.sqrt(D)
                if case["cap"]:
                    x = case["cap"] * torch.tanh(x / case["cap"])
                if case["alibi"]:
                    x = x - 2.0 ** (-8.0 * (h + 1) / H) * (here - j[see]).double()
                lse[b, t, h] = torch.logsumexp(x, 0)
                p = torch.exp(x - lse[b, t, h])
                o[b, t, h] = p @ values[see, h // g]
                w[b, h // g, :n][see] += p
    out = (o.view(B * Q, H, D), lse.view(B * Q, H))
    return out + (w,) if case["weights"] else out


def _exact_evict(case, s):
    B, H_kv, keep = case["B"], case["H_kv"], case["keep"]
    k, v = (torch.zeros_like(s[n], dtype=torch.float64) for n in ("k_out", "v_out"))
    w = torch.zeros(B, H_kv, keep, dtype=torch.float64)
    pos = torch.full((B, H_kv, keep), -1, dtype=torch.int32)
    weights = s["w"].cpu().tolist()
    table = None if s["table"] is None else s["table"].cpu().tolist()
    lens = _lengths(case)
    for b, n in enumerate(lens):
        for c in range(H_kv):
            old = max(0, n - case["recent"])
            best = sorted(range(old), key=lambda j: (-weights[b][c][j], j))
            slots = sorted(best[:max(0, min(n, keep) - (n - old))] +
                           list(range(old, n)))[-min(n, keep):]
            at = [b * s["page_size"] + j if table is None else
                  table[b][j // case["page"]] * case["page"] + j % case["page"] for j in slots]
            at, m = torch.tensor(at, device="cuda", dtype=torch.long), len(slots)
            k[b * keep:b * keep + m, c], v[b * keep:b * keep + m, c] = \
                s["k"][at, c].double(), s["v"][at, c].double()
            w[b, c, :m] = torch.tensor([weights[b][c][j] for j in slots], dtype=torch.float64)
            pos[b, c, :m] = torch.tensor(slots, dtype=torch.int32)
    return k, v, torch.tensor([min(n, keep) for n in lens], dtype=torch.int32), w, pos
