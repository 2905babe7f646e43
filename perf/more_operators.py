"""Cases that measure the attention of a chunk of new tokens over a paged cache (paged_attend, bf16
and 4-bit caches) and rotary positions with several axes (rope_axes, forward and gradient), in their
plain form and through the library.

A cache is a pool of pages [num_pages, Hkv, page, d] for K and one for V and a table of page
numbers per sequence (row p of a sequence is slot p % page of its page p // page). The 4-bit
pool holds, per row, d/2 bytes of codes (code + 8 in a nibble) and d/32 bf16 steps; the order
of the codes in a row is given by _place().
"""
import math
import random

import torch

own = False

GROUP = 32


def _sections(case):
    return [int(n) for n in case["sections"].split(",")]


def _attend(name, q4, B, Hq, Hkv, d, page, N, mix, **more):
    c = {"name": name, "op": "attend", "q4": q4, "B": B, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "N": N, "mix": mix,
         "lo": N, "ones": False, "start_lo": 0, "start_hi": 0, "window": 0, "alibi": False, "rope": True,
         "theta": 500000.0, "token_major": False}
    c.update(more)
    return c


def _rope(name, B, Hq, Hk, d, N, sections, **more):
    c = {"name": name, "op": "rope", "B": B, "Hq": Hq, "Hk": Hk, "d": d, "N": N, "sections": ",".join(map(str, sections)),
         "interleaved": False, "own_spectrum": False, "inverse": False, "theta": 500000.0, "far": 4096, "packed": False}
    c.update(more)
    return c


def listed():
    return [
        # four drafted tokens of one user are verified against a short context: latency alone
        _attend("attend-few", False, 1, 32, 8, 128, 16, 4, 1, start_lo=517, start_hi=517),
        # a serving step that mixes chunks of prompts with single tokens of other users, padded
        _attend("attend-mixed", False, 32, 32, 8, 128, 64, 512, 2, lo=1, ones=True, start_lo=0, start_hi=4096,
                token_major=True),
        # chunks of prompts of unequal length behind contexts of unequal length
        _attend("attend-chunks", False, 4, 32, 8, 128, 64, 2048, 3, lo=1500, start_lo=0, start_hi=6144),
        # a long prompt's last chunk; its rows come rotated
        _attend("attend-long", False, 1, 32, 8, 128, 128, 4096, 4, start_lo=28672, start_hi=28672, rope=False,
                token_major=True),
        # head dim 64, no grouping, window and ALiBi, pages of 48, sequences without new tokens among them
        _attend("attend-window-alibi", False, 24, 16, 16, 64, 48, 300, 5, lo=0, start_lo=0, start_hi=6001, window=1024,
                alibi=True, rope=False),
        # drafted tokens of a batch are verified against long contexts in a 4-bit cache
        _attend("attend4-verify", True, 16, 64, 8, 128, 64, 8, 6, lo=1, start_lo=1, start_hi=16384),
        # chunks of prompts over a 4-bit cache
        _attend("attend4-chunks", True, 4, 32, 8, 128, 64, 1024, 7, lo=700, start_lo=0, start_hi=8192),
        # one new token for each user of a batch: positions on three axes
        _rope("rope-step", 64, 32, 8, 128, 1, (16, 24, 24)),
        # prompts with video frames: time, height and width, from one fused projection
        _rope("rope-video", 2, 32, 8, 128, 8000, (16, 24, 24), packed=True),
        # images, rows and columns, every axis with a spectrum of its own, axes in turn
        _rope("rope-image", 24, 16, 16, 64, 1025, (16, 16), interleaved=True, own_spectrum=True, theta=10000.0, far=64),
        # the gradients of a training step's q and k
        _rope("rope-gradient", 4, 32, 8, 128, 4096, (24, 20, 20), interleaved=True, inverse=True, theta=5000000.0, far=100000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    if rng.random() < 0.35:
        d = rng.choice([64, 128, 128])
        axes = rng.choice([1, 2, 3, 3, 4])
        cut = sorted(rng.sample(range(1, d // 2), axes - 1))
        sections = [b - a for a, b in zip([0] + cut, cut + [d // 2])]
        Hq = rng.choice([1, 4, 12, 16, 32, 40])
        Hk = rng.choice([0, 1, 2, 4, 8, 16])
        N = rng.choice([1, _log_int(rng, 1, 16000), _log_int(rng, 100, 16000)])
        B = _log_int(rng, 1, max(1, min(64, 2 * 40 * 8000 // (N * (Hq + Hk)))))
        c = _rope("", B, Hq, Hk, d, N, sections, interleaved=rng.random() < 0.5, own_spectrum=rng.random() < 0.3,
                  inverse=rng.random() < 0.4, theta=rng.choice([10000.0, 500000.0, 5000000.0]),
                  far=_log_int(rng, 16, 1 << 22), packed=Hk > 0 and rng.random() < 0.5)
    else:
        d = rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 4, 8, 8, 12])
        g = rng.choice([1, 2, 3, 4, 4, 7, 8, 8, 20])
        N = rng.choice([1, _log_int(rng, 1, 32), _log_int(rng, 16, 4096), _log_int(rng, 16, 4096)])
        hi = _log_int(rng, 1, 28672)
        # pairs of a query head and a key at most those of the largest listed case, rows of the cache too
        most = min(32 * 4096 * 32768 // (Hkv * g * N * (hi + N)), 8 * 8 * 32768 // (Hkv * (hi + N)), 64)
        B = _log_int(rng, 1, max(1, most))
        c = _attend("", rng.random() < 0.4, B, Hkv * g, Hkv, d, rng.choice([16, 32, 48, 64, 80, 128, 256]), N,
                    rng.randrange(1 << 30), lo=rng.choice([0, 1, N // 2, N]), ones=rng.random() < 0.2,
                    start_lo=rng.choice([0, hi // 2, hi]), start_hi=hi,
                    window=rng.choice([0, 0, _log_int(rng, 1, hi + N)]), alibi=rng.random() < 0.25,
                    rope=rng.random() < 0.6, theta=rng.choice([10000.0, 500000.0]), token_major=rng.random() < 0.5)
    del c["name"]
    return c


def _lengths(case):
    """(start, count) per sequence: the position of its first new row, and how many there are."""
    r = random.Random(case["mix"])
    B, N = case["B"], case["N"]
    start = [r.randint(case["start_lo"], case["start_hi"]) for _ in range(B)]
    count = [r.randint(min(case["lo"], N), N) for _ in range(B)]
    if case["ones"]:
        count = [1 if b % 2 else n for b, n in enumerate(count)]
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
    randn = lambda *shape: torch.randn(*shape, generator=gen, device=dev)  # noqa: E731
    B, N, d = case["B"], case["N"], case["d"]
    if case["op"] == "rope":
        Hq, Hk = case["Hq"], case["Hk"]
        if case["packed"]:  # q, k and v as one projection leaves them: [B, N, Hq + 2 Hk, d]
            qkv = randn(B, N, Hq + 2 * Hk, d).bfloat16().transpose(1, 2)
            q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        else:
            q = randn(B, Hq, N, d).bfloat16()
            k = randn(B, Hk, N, d).bfloat16() if Hk else None
        pos = torch.randint(0, case["far"], (len(_sections(case)), B, N), generator=gen, device=dev, dtype=torch.int32)
        return {"case": case, "q": q, "k": k, "pos": pos}
    Hq, Hkv, page = case["Hq"], case["Hkv"], case["page"]
    start, count = _lengths(case)
    pages = [-(-(s + n) // page) for s, n in zip(start, count)]
    P, wide = sum(pages) + 3, max(pages) + 1
    order = torch.randperm(P, generator=gen, device=dev).to(torch.int32)
    at = [b * wide + j for b, n in enumerate(pages) for j in range(n)]
    flat = torch.full((B * wide,), -1, dtype=torch.int32, device=dev)
    if at:
        flat[torch.tensor(at, device=dev)] = order[:len(at)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    s = {"case": case, "table": flat.view(B, wide), "start": i32(start), "count": i32(count)}
    for n in "kv":
        if case["q4"]:
            codes = randn(P, Hkv, page, d).mul_(3.2).round_().clamp_(-7, 7).to(torch.int8)
            s[n + "_pages"] = _pack(codes)
            s[n + "_scales"] = (0.31 * torch.exp(0.2 * randn(P, Hkv, page, d // GROUP))).bfloat16()
        else:
            s[n + "_pages"] = randn(P, Hkv, page, d).bfloat16()
    s["q"] = randn(B, N, Hq, d).bfloat16().transpose(1, 2) if case["token_major"] else randn(B, Hq, N, d).bfloat16()
    if case["alibi"]:
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device=dev)
    return s


def _turn(x, angle):
    """Pairs (x_i, x_{i + d/2}) turned by the angles [..., d/2] (64 bits)."""
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    lo, hi = x.float().chunk(2, -1)
    return torch.cat((lo * cos - hi * sin, hi * cos + lo * sin), -1)


def _pairs(case):
    """Axis and exponent of theta for each pair: lists of d/2."""
    sections, half = _sections(case), case["d"] // 2
    if case["interleaved"]:  # dealt in turn; an axis that has all of its pairs is passed over
        left, axis = list(sections), []
        while len(axis) < half:
            for a in range(len(sections)):
                if left[a]:
                    left[a] -= 1
                    axis.append(a)
    else:
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
    if not case["own_spectrum"]:
        return axis, [-i / half for i in range(half)]
    seen, power = [0] * len(sections), []
    for a in axis:
        power.append(-seen[a] / sections[a])
        seen[a] += 1
    return axis, power


def _rope_plain(s):
    case = s["case"]
    axis, power = _pairs(case)
    dev = s["q"].device
    freq = torch.pow(torch.tensor(case["theta"], dtype=torch.float64, device=dev),
                     torch.tensor(power, dtype=torch.float64, device=dev))
    pos = s["pos"][torch.tensor(axis, device=dev)].permute(1, 2, 0).double()  # [B, N, d/2]
    angle = (pos * freq * (-1 if case["inverse"] else 1))[:, None]
    out = {"q": _turn(s["q"], angle).bfloat16()}
    if s["k"] is not None:
        out["k"] = _turn(s["k"], angle).bfloat16()
    return out


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
    steps = s[n + "_scales"][which, :, slot].float()
    place = _place(d, page, pos.device).flatten(1)  # [page, d]: the element of each nibble
    back = torch.argsort(place, 1)[slot]  # [B, L, d]: the nibble of each element
    nib = torch.stack((rows & 15, rows >> 4), -1).flatten(3)
    codes = torch.gather(nib, 3, back[:, :, None].expand_as(nib))
    return (codes.float() - 8.0) * steps.repeat_interleave(GROUP, -1)


def _attend_plain(s):
    case = s["case"]
    B, Hq, Hkv, N, d = case["B"], case["Hq"], case["Hkv"], case["N"], case["d"]
    start, count = s["start"].long()[:, None], s["count"].long()[:, None]
    dev = start.device
    n = torch.arange(N, device=dev)
    pos = start + n  # [B, N]
    q = s["q"].float()
    if case["rope"]:
        i = torch.arange(d // 2, device=dev, dtype=torch.float64)
        freq = torch.pow(torch.tensor(case["theta"], dtype=torch.float64, device=dev), -2.0 * i / d)
        q = _turn(q, (pos.double()[..., None] * freq)[:, None])
    q = q.reshape(B, Hkv, -1, d)  # the heads of a group, one after the other
    m = torch.arange(max(1, max(a + b for a, b in zip(*_lengths(case)))), device=dev)
    end = start + count
    keep = (m < end)[:, :, None, None]  # [B, L, 1, 1]
    k = torch.where(keep, _rows(s, m.expand(B, -1), "k"), torch.zeros((), device=dev))
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(d ** -0.5).view(B, Hkv, Hq // Hkv, N, -1)
    del k
    off = m - pos[..., None]  # [B, N, L]
    if case["alibi"]:
        x = x + s["slopes"].view(Hkv, -1, 1, 1) * off.float()[:, None, None]
    seen = (off <= 0) & (n < count)[..., None]
    if case["window"]:
        seen = seen & (off > -case["window"])
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    base = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = x.sub_(base).exp_()
    total = p.sum(-1, keepdim=True)
    v = torch.where(keep, _rows(s, m.expand(B, -1), "v"), torch.zeros((), device=dev))
    o = torch.matmul(p.view(B, Hkv, -1, m.numel()), v.transpose(1, 2)).view(B, Hkv, -1, N, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (base + torch.log(total)).view(B, Hq, N)
    return {"out": o.reshape(B, Hq, N, d).bfloat16(), "lse": lse}


def _own(s):
    import attention_attn_fwd_bwd_gb300 as af

    case = s["case"]
    if case["op"] == "rope":
        q, k = af.rope_axes(s["q"], s["k"], s["pos"], _sections(case), rope_theta=case["theta"],
                            interleaved=case["interleaved"], own_spectrum=case["own_spectrum"], inverse=case["inverse"])
        return {"q": q} if k is None else {"q": q, "k": k}
    cache = af.PagedCache(s["k_pages"], s["v_pages"], s["table"], k_scales=s.get("k_scales"),
                          v_scales=s.get("v_scales"))
    out, lse = af.paged_attend(s["q"], cache, s["start"], s["count"], rope_theta=case["theta"],
                               rope_mode=af.ROPE_FUSED if case["rope"] else af.ROPE_NONE, window=case["window"],
                               alibi_slopes=s.get("slopes"))
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"attend": _attend_plain, "rope": _rope_plain}[state["case"]["op"]](state)


def work(case):
    B, N, d = case["B"], case["N"], case["d"]
    if case["op"] == "rope":
        values = B * N * (case["Hq"] + case["Hk"]) * d
        return {"bytes": 4 * values + 4 * len(_sections(case)) * B * N, "flops": 3 * values}
    start, count = _lengths(case)
    Hq, W = case["Hq"], case["window"]
    row = 2 * case["Hkv"] * (d // 2 + d // 16 if case["q4"] else 2 * d)  # K and V of one position in the cache
    pairs = rows = tables = 0
    for s, n in zip(start, count):
        if not n:
            continue
        first = max(0, s - W + 1) if W else 0
        rows += s + n - first
        tables += -(-(s + n) // case["page"]) - first // case["page"]
        pairs += sum(min(s + i + 1, W) for i in range(n)) if W else n * s + n * (n + 1) // 2
    dense = sum(count) * Hq * 2 * d + B * N * Hq * (2 * d + 4)  # q of the live rows; out and lse of all
    return {"bytes": rows * row + dense + 4 * (2 * B + tables), "flops": 4 * pairs * Hq * d}


# --- the operators' definitions in 64 bits ---------------------------------------------------

def _exact_turn(x, angle):
    """x [..., d] in 64 bits, turned by angle [..., d/2]: as complex numbers."""
    h = x.shape[-1] // 2
    z = torch.complex(x[..., :h].contiguous(), x[..., h:].contiguous())
    z = z * torch.polar(torch.ones_like(angle), angle)
    return torch.cat((z.real, z.imag), -1)


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


def _exact_rope(case, s):
    """One pair at a time, from its axis' positions."""
    sections, half = _sections(case), case["d"] // 2
    turn = -1.0 if case["inverse"] else 1.0
    whose = {}  # pair -> (axis, its number within the axis)
    if case["interleaved"]:
        order = sorted((j, a) for a, n in enumerate(sections) for j in range(n))
    else:
        order = [(j, a) for a, n in enumerate(sections) for j in range(n)]
    for i, (j, a) in enumerate(order):
        whose[i] = (a, j)
    done = {}
    for name in "qk":
        if s[name] is None:
            continue
        x = s[name].double()
        y = torch.empty_like(x)
        for i in range(half):
            a, j = whose[i]
            f = math.exp(-math.log(case["theta"]) * (j / sections[a] if case["own_spectrum"] else i / half))
            angle = (s["pos"][a].double() * (turn * f))[:, None]
            c, w = torch.cos(angle), torch.sin(angle)
            y[..., i] = x[..., i] * c - x[..., i + half] * w
            y[..., i + half] = x[..., i] * w + x[..., i + half] * c
        done[name] = y
    return done


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    start, count = _lengths(case)
    B, Hq, Hkv, N, d = case["B"], case["Hq"], case["Hkv"], case["N"], case["d"]
    g, W = Hq // Hkv, case["window"]
    dev = s["table"].device
    f64 = dict(dtype=torch.float64, device=dev)
    out, lse = torch.zeros(B, Hq, N, d, **f64), torch.full((B, Hq, N), -math.inf, **f64)
    for b in range(B):
        if not count[b]:
            continue
        end = start[b] + count[b]
        first = max(0, start[b] - W + 1) if W else 0
        p, m = torch.arange(start[b], end, device=dev)[:, None], torch.arange(first, end, device=dev)
        hidden = m > p
        if W:
            hidden = hidden | (p - m >= W)
        q = s["q"][b, :, :count[b]].double()
        if case["rope"]:
            f = torch.exp(-math.log(case["theta"]) * torch.arange(d // 2, **f64) / (d // 2))
            q = _exact_turn(q, (p.double() * f).expand(Hq, -1, -1))
        k, v = (_exact_rows(s, b, first, end - first, n) for n in "kv")
        for h in range(Hq):
            x = q[h] @ k[h // g].T / math.sqrt(d)
            if case["alibi"]:
                x = x + s["slopes"][h].double() * (m - p)
            x = x.masked_fill(hidden, -math.inf)
            l = torch.logsumexp(x, -1)
            lse[b, h, :count[b]] = l
            out[b, h, :count[b]] = torch.exp(x - l[:, None]) @ v[h // g]
    return {"out": out, "lse": lse}
