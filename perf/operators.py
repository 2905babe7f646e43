"""Cases that measure the paged-cache operators: append (with the rotation of K), gather and
decode, on bf16 and on 4-bit caches, in their plain form and through the library.

A cache is a pool of pages [num_pages, Hkv, page, d] for K and one for V and a table of page
numbers per sequence (row p of a sequence is slot p % page of its page p // page). The 4-bit
pool holds, per row, d/2 bytes of codes (code + 8 in a nibble) and d/32 bf16 scales; the order
of the codes in a row is given by _place().
"""
import math
import random

import torch

own = False

GROUP = 32


def _case(name, op, q4, B, Hkv, d, page, mix, **more):
    c = {"name": name, "op": op, "q4": q4, "B": B, "Hkv": Hkv, "d": d, "page": page, "mix": mix,
         "theta": 500000.0, "rope": True}
    c.update(more)
    return c


def listed():
    return [
        # one user's next token enters the cache: latency alone
        _case("append-one", "append", False, 1, 8, 128, 16, 1, N=1, lo=1, start_lo=517, start_hi=517),
        # a padded batch of prompts of unequal lengths is written after its prefill
        _case("append-prompts", "append", False, 8, 8, 128, 64, 2, N=4096, lo=300, start_lo=0, start_hi=0),
        # one user's next token is decoded from a short context
        _case("decode-one", "decode", False, 1, 8, 128, 16, 3, Hq=32, lo=517, hi=517, window=0, alibi=False),
        # a serving batch in mid-flight: every sequence has its own length
        _case("decode-batch", "decode", False, 64, 8, 128, 64, 4, Hq=32, lo=1, hi=4096, window=0, alibi=False),
        # the dense decode benchmark's shape (Hq=64, Hkv=8, 32k keys, 8 sequences) in pages
        _case("decode-long", "decode", False, 8, 8, 128, 128, 5, Hq=64, lo=32768, hi=32768, window=0, alibi=False),
        # head dim 64, no grouping, window and ALiBi, pages of 48, some sequences still empty
        _case("decode-window-alibi", "decode", False, 24, 16, 64, 48, 6, Hq=16, lo=0, hi=6001, window=1024, alibi=True,
              rope=False),
        # a serving batch's next tokens enter a 4-bit cache, and the values it now holds are read
        _case("append4-batch", "append", True, 64, 8, 128, 16, 7, N=1, lo=1, start_lo=3, start_hi=4000),
        # prompts enter a 4-bit cache and are read back as the values that later tokens attend to
        _case("append4-prompts", "append", True, 4, 8, 128, 64, 8, N=4096, lo=2000, start_lo=0, start_hi=77),
        # as decode-one, from a 4-bit cache
        _case("decode4-one", "decode", True, 1, 8, 128, 16, 9, Hq=32, lo=517, hi=517, window=0, alibi=False),
        # as decode-batch, from a 4-bit cache, contexts twice as long
        _case("decode4-batch", "decode", True, 64, 8, 128, 64, 10, Hq=32, lo=1, hi=8192, window=0, alibi=False),
        # as decode-long, from a 4-bit cache
        _case("decode4-long", "decode", True, 8, 8, 128, 128, 11, Hq=64, lo=32768, hi=32768, window=0, alibi=False),
        # sequences leave the pool as one dense padded batch
        _case("gather", "gather", False, 16, 16, 64, 32, 12, N=2048, lo=0, start_lo=0, start_hi=1000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "gather"])
    q4 = rng.random() < 0.5
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 48, 64, 80, 128, 256])
    mix = rng.randrange(1 << 30)
    if op == "decode":
        Hkv = rng.choice([1, 2, 4, 8, 8, 12])
        g = rng.choice([1, 2, 3, 4, 7, 8, 8, 16, 20])
        hi = _log_int(rng, 1, 32768)
        # keys times heads at most those of the largest listed case, scores too
        most = min(8 * 8 * 32768 // (Hkv * hi), 8 * 64 * 32768 // (Hkv * g * hi), 256)
        B = _log_int(rng, 1, max(1, most))
        lo = rng.choice([0, 1, hi // 2, hi])
        c = _case("", op, q4, B, Hkv, d, page, mix, Hq=Hkv * g, lo=lo, hi=hi,
                  window=rng.choice([0, 0, _log_int(rng, 1, hi)]), alibi=rng.random() < 0.25)
        c["rope"] = rng.random() < 0.75
    else:
        Hkv = rng.choice([1, 2, 4, 8, 8, 12, 16])
        N = rng.choice([1, _log_int(rng, 1, 4096)])
        B = _log_int(rng, 1, max(1, min(256, 16 * 1024 * 8 // (Hkv * N))))
        hi = _log_int(rng, 1, 4000)
        c = _case("", op, q4, B, Hkv, d, page, mix, N=N, lo=rng.choice([0, 1, N // 2, N]),
                  start_lo=rng.choice([0, hi // 2, hi]), start_hi=hi)
    c["theta"] = rng.choice([10000.0, 500000.0])
    del c["name"]
    return c


def _lengths(case):
    """(start, count) per sequence: where rows begin and how many there are. Decode: (0, length)."""
    r = random.Random(case["mix"])
    B = case["B"]
    if case["op"] == "decode":
        return [0] * B, [r.randint(case["lo"], case["hi"]) for _ in range(B)]
    start = [r.randint(case["start_lo"], case["start_hi"]) for _ in range(B)]
    count = [r.randint(case["lo"], case["N"]) for _ in range(B)]
    return start, count


def _place(d, page, device):
    """[page, d/2, 2] int64: for each slot and byte of its row, the elements whose codes are the
    byte's low nibble and its high nibble."""
    G = d // GROUP
    slot = torch.arange(page, device=device)[:, None]
    byte = torch.arange(d // 2, device=device)[None, :]
    chunk = byte // (2 * G)  # 8 chunks of G halfwords
    if d == 128:
        chunk = chunk ^ (4 * ((slot >> 1) & 1))
    half = (byte % (2 * G)) // 2
    first = GROUP * half + 4 * chunk + 2 * (byte % 2) + 0 * slot
    return torch.stack((first, first + 1), -1)


def _pack(codes):
    """Codes -7..7 [pages, Hkv, page, d] (int8) -> the bytes of the pool's rows."""
    P, H, S, d = codes.shape
    at = _place(d, S, codes.device)
    n = (codes + 8).to(torch.uint8)
    lo = torch.gather(n, 3, at[..., 0].expand(P, H, S, d // 2))
    hi = torch.gather(n, 3, at[..., 1].expand(P, H, S, d // 2))
    return lo | (hi << 4)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(int(seed))
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    start, count = _lengths(case)
    pages = [-(-(s + n) // page) for s, n in zip(start, count)]
    P, wide = sum(pages) + 3, max(pages) + 1
    order = torch.randperm(P, generator=gen, device=dev).to(torch.int32)
    table = torch.full((B, wide), -1, dtype=torch.int32)
    at, i = [], 0
    for b, n in enumerate(pages):
        at += [b * wide + j for j in range(n)]
    flat = table.view(-1).to(dev)
    if at:
        flat[torch.tensor(at, device=dev)] = order[:len(at)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    s = {"case": case, "table": flat.view(B, wide), "start": i32(start), "count": i32(count)}
    randn = lambda *shape: torch.randn(*shape, generator=gen, device=dev)  # noqa: E731
    if case["op"] == "append":
        if case["q4"]:
            for n in "kv":
                s[n + "_pages"] = torch.zeros(P, Hkv, page, d // 2, dtype=torch.uint8, device=dev)
                s[n + "_scales"] = torch.zeros(P, Hkv, page, d // GROUP, dtype=torch.bfloat16, device=dev)
        else:
            for n in "kv":
                s[n + "_pages"] = torch.zeros(P, Hkv, page, d, dtype=torch.bfloat16, device=dev)
        for n in "kv":
            s[n] = randn(B, Hkv, case["N"], d).bfloat16()
    else:
        for n in "kv":
            if case["q4"]:
                codes = randn(P, Hkv, page, d).mul_(3.2).round_().clamp_(-7, 7).to(torch.int8)
                s[n + "_pages"] = _pack(codes)
                s[n + "_scales"] = (0.31 * torch.exp(0.2 * randn(P, Hkv, page, d // GROUP))).bfloat16()
            else:
                s[n + "_pages"] = randn(P, Hkv, page, d).bfloat16()
    if case["op"] == "decode":
        s["q"] = randn(B, case["Hq"], d).bfloat16()
        if case["alibi"]:
            Hq = case["Hq"]
            s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device=dev)
    return s


def _cos_sin(pos, d, theta):
    """(cos, sin) of pos * theta^(-2i/d) in 64 bits: pos [...] -> [..., d/2]."""
    i = torch.arange(d // 2, device=pos.device, dtype=torch.float64)
    angle = pos.double()[..., None] * torch.pow(torch.tensor(theta, dtype=torch.float64, device=pos.device), -2.0 * i / d)
    return torch.cos(angle), torch.sin(angle)


def _rotate(x, cos, sin):
    lo, hi = x.chunk(2, -1)
    return torch.cat((lo * cos - hi * sin, hi * cos + lo * sin), -1)


def _rows(s, pos, n):
    """Rows `pos` [B, L] of every sequence's K or V as fp32 [B, L, Hkv, d] (any valid slot where
    the table has no page: the caller masks those)."""
    case = s["case"]
    page, d = case["page"], case["d"]
    at = (pos // page).clamp(max=s["table"].shape[1] - 1)
    which = torch.gather(s["table"].long(), 1, at).clamp(min=0)
    slot = pos % page
    rows = s[n + "_pages"][which, :, slot]
    if not case["q4"]:
        return rows.float()
    scales = s[n + "_scales"][which, :, slot].float()
    place = _place(d, page, pos.device).flatten(1)  # [page, d]: the element of each nibble
    back = torch.argsort(place, 1)[slot]  # [B, L, d]: the nibble of each element
    nib = torch.stack((rows & 15, rows >> 4), -1).flatten(3)
    codes = torch.gather(nib, 3, back[:, :, None].expand_as(nib))
    return (codes.float() - 8.0) * scales.repeat_interleave(GROUP, -1)


def _quantise(x):
    """x fp32 (bf16 values) [..., d] -> (codes int8, scales bf16)."""
    g = x.unflatten(-1, (-1, GROUP))
    a = g.abs().amax(-1)
    s = (a / 7).bfloat16()
    s = torch.where(a < 2.0 ** -96, torch.zeros_like(s), s)
    s = torch.where(torch.isfinite(a), s, torch.full_like(s, math.nan))
    ok = torch.isfinite(s) & (s > 0)
    div = torch.where(ok, s, torch.ones_like(s)).double()[..., None]
    c = torch.sign(g) * torch.floor(g.abs().double() / div + 0.5).clamp(max=7)
    c = torch.where(ok[..., None], c, torch.zeros_like(c))
    return c.to(torch.int8).flatten(-2), s


def _append(s):
    case = s["case"]
    B, N, page, d = case["B"], case["N"], case["page"], case["d"]
    n = torch.arange(N, device=s["k"].device)
    pos = s["start"].long()[:, None] + n
    k = s["k"].double()
    if case["rope"]:
        cos, sin = _cos_sin(pos, d, case["theta"])
        k = _rotate(k, cos[:, None], sin[:, None])
    k = k.float().bfloat16()
    live = n < s["count"][:, None]
    b, r = live.nonzero(as_tuple=True)
    p = pos[b, r]
    which, slot = s["table"].long()[b, p // page], p % page
    rows = {"k": k[b, :, r], "v": s["v"][b, :, r]}  # [rows, Hkv, d]
    if not case["q4"]:
        s["k_pages"][which, :, slot] = rows["k"]
        s["v_pages"][which, :, slot] = rows["v"]
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    place = _place(d, page, p.device)[slot]  # [rows, d/2, 2]
    kc, ks = _quantise(rows["k"].float())
    vc, vs = _quantise(rows["v"].float())
    for_k = torch.gather(kc, 2, place.flatten(1)[:, None].expand_as(kc)).unflatten(-1, (-1, 2))
    for_v = torch.gather(vc, 2, place.flatten(1)[:, None].expand_as(vc)).unflatten(-1, (-1, 2))
    byte = lambda c: (c[..., 0] + 8).to(torch.uint8) | ((c[..., 1] + 8).to(torch.uint8) << 4)  # noqa: E731
    s["k_pages"][which, :, slot] = byte(for_k)
    s["v_pages"][which, :, slot] = byte(for_v)
    s["k_scales"][which, :, slot] = ks
    s["v_scales"][which, :, slot] = vs
    return _gather(s)


def _gather(s):
    case = s["case"]
    n = torch.arange(case["N"], device=s["table"].device)
    pos = s["start"].long()[:, None] + n
    live = (n < s["count"][:, None])[:, :, None, None]
    zero = torch.zeros((), device=n.device)
    k = torch.where(live, _rows(s, pos, "k"), zero).bfloat16().transpose(1, 2).contiguous()
    v = torch.where(live, _rows(s, pos, "v"), zero).bfloat16().transpose(1, 2).contiguous()
    return {"k": k, "v": v}


def _decode(s):
    case = s["case"]
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    lens = s["count"].long()
    dev = lens.device
    q = s["q"].float()
    if case["rope"]:
        cos, sin = _cos_sin((lens - 1).clamp(min=0), d, case["theta"])
        q = _rotate(q, cos[:, None].float(), sin[:, None].float())
    q = q.view(B, Hkv, Hq // Hkv, d)
    n = torch.arange(max(1, case["hi"]), device=dev)
    pos = n.expand(B, -1)
    live = n < lens[:, None]
    if case["window"]:
        live = live & (n >= lens[:, None] - case["window"])
    keep = live[:, :, None, None]
    k = torch.where(keep, _rows(s, pos, "k"), torch.zeros((), device=dev))
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * d ** -0.5  # [B, Hkv, g, L]
    del k
    if case["alibi"]:
        x = x + s["slopes"].view(Hkv, -1, 1) * (n - (lens[:, None] - 1)).float()[:, None, None]
    x = x.masked_fill(~live[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    base = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(x - base)
    total = p.sum(-1, keepdim=True)
    v = torch.where(keep, _rows(s, pos, "v"), torch.zeros((), device=dev))
    o = torch.matmul(p, v.transpose(1, 2))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (base + torch.log(total)).view(B, Hq)
    return {"out": o.reshape(B, Hq, d).bfloat16(), "lse": lse}


def _own(s):
    import attention_attn_fwd_bwd_gb300 as af

    case = s["case"]
    cache = af.PagedCache(s["k_pages"], s["v_pages"], s["table"], k_scales=s.get("k_scales"),
                          v_scales=s.get("v_scales"))
    mode = af.ROPE_FUSED if case["rope"] else af.ROPE_NONE
    if case["op"] == "decode":
        out, lse = af.paged_decode(s["q"], cache, s["count"], rope_theta=case["theta"], rope_mode=mode,
                                   window=case["window"], alibi_slopes=s.get("slopes"))
        return {"out": out, "lse": lse}
    if case["op"] == "append":
        af.paged_append(cache, s["k"], s["v"], s["start"], s["count"], rope_theta=case["theta"], rope_mode=mode)
        if not case["q4"]:
            return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    k, v = af.paged_gather(cache, s["start"], s["count"], case["N"])
    return {"k": k, "v": v}


def run(state):
    if own:
        return _own(state)
    return {"append": _append, "gather": _gather, "decode": _decode}[state["case"]["op"]](state)


def work(case):
    start, count = _lengths(case)
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    row = 2 * Hkv * (d // 2 + d // 16 if case["q4"] else 2 * d)  # K and V of one position in the cache
    dense = 2 * Hkv * 2 * d
    if case["op"] == "decode":
        seen = sum(min(n, case["window"] or n) for n in count)
        tables = 4 * (B + sum(-(-n // case["page"]) for n in count))
        return {"bytes": seen * row + B * case["Hq"] * (4 * d + 4) + tables, "flops": 4 * seen * case["Hq"] * d}
    rows = sum(count)
    tables = 4 * sum(2 + -(-n // case["page"]) for n in count)
    if case["op"] == "gather":
        return {"bytes": rows * row + B * case["N"] * dense + tables, "flops": rows * Hkv * d * 2 if case["q4"] else 0}
    back = B * case["N"] * dense if case["q4"] else 0  # the values, read back
    return {"bytes": rows * (dense + row) + back + tables, "flops": rows * Hkv * d * (3 + (8 if case["q4"] else 0))}


# --- the operators' definitions in 64 bits, one sequence at a time ---------------------------

def _exact_rows(s, b, first, n, name):
    """Rows first .. first+n-1 of sequence b in 64 bits, [Hkv, n, d], from the pool's bytes."""
    case = s["case"]
    page, d, H = case["page"], case["d"], case["Hkv"]
    p = torch.arange(first, first + n, device=s["table"].device)
    which = s["table"][b, p.div(page, rounding_mode="floor")].long()
    raw = s[name + "_pages"][which, :, p.remainder(page)]  # [n, Hkv, bytes]
    if not case["q4"]:
        return raw.double().transpose(0, 1)
    G = d // GROUP
    half = raw.contiguous().view(torch.int16).to(torch.int64).bitwise_and(0xFFFF).view(n, H, 8, G)
    if d == 128:  # slots with bit 1 set hold their two halves of the row swapped
        swapped = (p.remainder(page).bitwise_and(2) > 0)[:, None, None, None]
        half = torch.where(swapped, half.roll(4, 2), half)
    nib = torch.stack([half.bitwise_right_shift(4 * i).bitwise_and(15) for i in range(4)], -1)
    codes = nib.permute(0, 1, 3, 2, 4).reshape(n, H, G, GROUP).double() - 8
    value = codes * s[name + "_scales"][which, :, p.remainder(page)].double()[..., None]
    return value.reshape(n, H, d).transpose(0, 1)


def _exact_turn(x, pos, theta):
    """x [..., n, d] in 64 bits, row j turned by the angles of position pos[j]: as complex numbers."""
    h = x.shape[-1] // 2
    i = torch.arange(h, dtype=torch.float64, device=x.device)
    freq = torch.exp(-math.log(theta) * i / h)
    z = torch.complex(x[..., :h].contiguous(), x[..., h:].contiguous())
    z = z * torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos.double()[:, None] * freq)
    return torch.cat((z.real, z.imag), -1)


def exact(case, seed):
    s = prepare(case, seed)
    start, count = _lengths(case)
    B, d = case["B"], case["d"]
    dev = s["table"].device
    f64 = dict(dtype=torch.float64, device=dev)
    if case["op"] == "decode":
        Hq, Hkv = case["Hq"], case["Hkv"]
        out, lse = torch.zeros(B, Hq, d, **f64), torch.full((B, Hq), -math.inf, **f64)
        for b, L in enumerate(count):
            if not L:
                continue
            first = max(0, L - case["window"]) if case["window"] else 0
            n = torch.arange(first, L, device=dev)
            q = s["q"][b].double()
            if case["rope"]:
                q = _exact_turn(q[:, None], torch.tensor([L - 1], device=dev), case["theta"])[:, 0]
            x = torch.einsum("hgc,hnc->hgn", q.view(Hkv, -1, d), _exact_rows(s, b, first, L - first, "k")) / math.sqrt(d)
            if case["alibi"]:
                x = x + s["slopes"].double().view(Hkv, -1, 1) * (n - (L - 1))
            l = torch.logsumexp(x, -1)
            lse[b] = l.view(-1)
            out[b] = torch.einsum("hgn,hnc->hgc", torch.exp(x - l[..., None]), _exact_rows(s, b, first, L - first, "v")).reshape(Hq, d)
        return {"out": out, "lse": lse}
    if case["op"] == "append":
        k64 = {"k": s["k"].double(), "v": s["v"].double()}
        if case["rope"]:
            for b in range(B):
                k64["k"][b] = _exact_turn(k64["k"][b], start[b] + torch.arange(case["N"], device=dev), case["theta"])
        if case["q4"]:
            done = {}
            for n, x in k64.items():
                # what the cache of 16-bit values would hold, then the nearest multiple of the group's step
                g = x.float().bfloat16().double().reshape(*x.shape[:-1], -1, GROUP)
                step = (g.abs().amax(-1, keepdim=True).float() / 7).bfloat16().double()
                v = torch.where(step > 0, torch.trunc(g / step + 0.5 * g.sign()).clamp(-7, 7) * step, torch.zeros_like(g))
                done[n] = v.reshape(x.shape)
                for b in range(B):
                    done[n][b, :, count[b]:] = 0
            return done
        pools = {}
        for n, x in k64.items():
            pool = torch.zeros(s[n + "_pages"].shape, **f64)
            for b in range(B):
                p = start[b] + torch.arange(count[b], device=dev)
                pool[s["table"][b, p // case["page"]].long(), :, p % case["page"]] = x[b, :, :count[b]].transpose(0, 1)
            pools[n + "_pages"] = pool
        return pools
    done = {n: torch.zeros(B, case["Hkv"], case["N"], d, **f64) for n in "kv"}
    for n, x in done.items():
        for b in range(B):
            x[b, :, :count[b]] = _exact_rows(s, b, start[b], count[b], n)
    return done
