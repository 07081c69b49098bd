"""Measured cases of the serving and training operators around attention.

Four operators, each in its plain form (elementary torch operations, 32-bit sums, one rounding
at the end) and, where ``own`` is true, through the library's public calls:

* rotary positions on queries and keys, forward and backward;
* a paged key/value cache written (rotated, quantised to 8 bits with a power-of-two scale per
  row) and read back to dense 16-bit rows;
* one decode step over such a cache with grouped heads, the new token's row written first;
* one decode step of a batch whose sequences share a long prefix.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges.
"""
import math

import torch

own = False

PAGE = 16          # tokens per page of the cache
E4M3_MAX = 448.0   # largest finite e4m3 value
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # One token for each of 256 sequences in a continuous batch: launch latency.
        dict(name="rotary_decode_B256", kind="rotary", B=256, Hq=32, Hk=8, L=1, D=128, rd=128,
             inter=False, scaling="none", factor=1.0, maxpos=4096, dtype="bf16", grad=False,
             packed=False),
        # The training shape of the benchmark: 8 x 4096 tokens, 32 heads, both directions.
        dict(name="rotary_train_B8_L4096", kind="rotary", B=8, Hq=32, Hk=32, L=4096, D=128,
             rd=128, inter=False, scaling="none", factor=1.0, maxpos=4096, dtype="bf16",
             grad=True, packed=False),
        # A long context past the trained length: interleaved pairs, part of the head, scaled
        # frequencies, read in place from packed [B, L, 3, H, D].
        dict(name="rotary_long_L16384_D64", kind="rotary", B=1, Hq=16, Hk=16, L=16384, D=64,
             rd=32, inter=True, scaling="yarn", factor=16.0, maxpos=262144, dtype="fp16",
             grad=True, packed=True),
        # Prefill of 8 prompts of up to 2048 tokens into an 8-bit cache, then read back whole.
        dict(name="cache_prefill_B8_L2048", kind="cache", B=8, H=32, D=128, start=0, new=2048,
             rd=128, inter=False, quant=True, dtype="bf16"),
        # A chunk of a prompt behind tokens that are cached already; odd lengths, half the head
        # rotated, 64-wide heads.
        dict(name="cache_chunk_B16_D64", kind="cache", B=16, H=8, D=64, start=1501, new=333,
             rd=32, inter=True, quant=True, dtype="fp16"),
        # One sequence, short: the smallest serving step (write one row, attend), latency.
        dict(name="step_B1_short", kind="decode", B=1, Hq=32, Hk=8, D=128, lo=333, hi=333,
             quant=True, append=True, dtype="bf16"),
        # The serving batch of the benchmark (256 sequences of 1..4096 tokens, 32 heads of
        # 128) on an 8-bit cache, the new token written first.
        dict(name="step_B256_H32", kind="decode", B=256, Hq=32, Hk=32, D=128, lo=1, hi=4096,
             quant=True, append=True, dtype="bf16"),
        # Long contexts with 8 query heads per cache head.
        dict(name="decode_gqa8_L16384", kind="decode", B=48, Hq=64, Hk=8, D=128, lo=1, hi=16384,
             quant=True, append=False, dtype="bf16"),
        # Grouped heads on a 16-bit cache, 64-wide, odd lengths.
        dict(name="decode_gqa4_16bit_D64", kind="decode", B=17, Hq=16, Hk=4, D=64, lo=77,
             hi=4001, quant=False, append=False, dtype="fp16"),
        # A few questions about one short document: latency.
        dict(name="prefix_B4_P517_D64", kind="prefix", B=4, Hq=16, Hk=4, D=64, prefix=517, lo=0,
             hi=45, dtype="fp16"),
        # A system prompt of 4096 tokens before 64 conversations.
        dict(name="prefix_B64_P4096", kind="prefix", B=64, Hq=32, Hk=8, D=128, prefix=4096, lo=1,
             hi=512, dtype="bf16"),
        # A long document shared by the whole serving batch, 32 heads of 128.
        dict(name="prefix_B256_P16384", kind="prefix", B=256, Hq=32, Hk=32, D=128, prefix=16384,
             lo=1, hi=255, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rotary", "cache", "decode", "prefix"])
    D = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    if kind == "rotary":
        Hk = rng.choice([1, 2, 4, 8, 16, 32])
        packed = rng.random() < 0.3
        Hq = Hk if packed else Hk * rng.choice([1, 2, 4] if Hk < 32 else [1])
        grad = rng.random() < 0.5
        B = _spread(rng, 1, 256)
        L = 1 if rng.random() < 0.25 else _spread(rng, 1, 16384)
        while B * L * (Hq + Hk) * D > 8 * 4096 * 64 * 128:
            B, L = max(1, B // 2), max(1, L // 2)
        return dict(kind=kind, B=B, Hq=Hq, Hk=Hk, L=L, D=D, rd=rng.choice([D, D // 2, D // 4]),
                    inter=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    factor=rng.choice([2.0, 4.0, 16.0]), maxpos=max(L, _spread(rng, 256, 262144)),
                    dtype=dtype, grad=grad, packed=packed)
    if kind == "cache":
        H, B = rng.choice([1, 4, 8, 32]), _spread(rng, 1, 64)
        start, new = rng.choice([0, _spread(rng, 1, 4096)]), _spread(rng, 1, 2048)
        while B * (start + new) * H * D > 8 * 1400 * 32 * 128:
            B, start, new = max(1, B // 2), start // 2, max(1, new // 2)
        return dict(kind=kind, B=B, H=H, D=D, start=start, new=new,
                    rd=rng.choice([0, D, D // 2]), inter=rng.random() < 0.5,
                    quant=rng.random() < 0.7, dtype=dtype)
    Hk = rng.choice([1, 2, 4, 8, 32])
    Hq = Hk * rng.choice([1, 2, 4, 8] if Hk < 32 else [1])
    B = _spread(rng, 1, 256)
    if kind == "decode":
        hi = _spread(rng, 16, 16384)
        quant = rng.random() < 0.6
        while B * hi * Hk * D * (1 if quant else 2) > 256 * 1024 * 32 * 128:
            B, hi = max(1, B // 2), max(16, hi // 2)
        return dict(kind=kind, B=B, Hq=Hq, Hk=Hk, D=D, lo=rng.randint(1, hi), hi=hi,
                    quant=quant, append=rng.random() < 0.5, dtype=dtype)
    prefix, hi = _spread(rng, 64, 16384), _spread(rng, 1, 512)
    while (B * hi + prefix) * Hk * D > 256 * 255 * 32 * 128 or B * Hq * prefix > 256 * 32 * 16384:
        B, prefix, hi = max(1, B // 2), max(64, prefix // 2), max(1, hi // 2)
    return dict(kind=kind, B=B, Hq=Hq, Hk=Hk, D=D, prefix=prefix, lo=rng.randint(0, hi), hi=hi,
                dtype=dtype)


def _lens(lo, hi, n):
    """n whole numbers spread evenly from lo to hi."""
    return [lo + (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _new_lens(c):
    return _lens(max(1, c["new"] // 2), c["new"], c["B"])


def work(case):
    """Each input read once, each output written once; products and sums of the attention."""
    c, D = case, case["D"]
    if c["kind"] == "rotary":
        n = c["B"] * c["L"] * (c["Hq"] + c["Hk"]) * D
        passes = 2 if c["grad"] else 1
        return {"bytes": passes * n * 4 + c["B"] * c["L"] * 4, "flops": passes * n * 3}
    if c["kind"] == "cache":
        new, el = sum(_new_lens(c)), 1 if c["quant"] else 2
        cached = sum(_lens(0, c["start"], c["B"])) + new
        row = D * el + (1 if c["quant"] else 0)
        return {"bytes": 2 * c["H"] * (new * (D * 2 + row) + cached * row +
                                       c["B"] * (c["start"] + c["new"]) * D * 2),
                "flops": 2 * c["H"] * (new + cached) * D}
    if c["kind"] == "decode":
        n, row = sum(_lens(c["lo"], c["hi"], c["B"])), D + 1 if c["quant"] else 2 * D
        extra = c["B"] * c["Hk"] * 2 * (2 * D + row) if c["append"] else 0
        return {"bytes": 2 * n * c["Hk"] * row + c["B"] * c["Hq"] * (4 * D + 4) + extra,
                "flops": 4 * n * c["Hq"] * D}
    n = sum(_lens(c["lo"], c["hi"], c["B"]))
    return {"bytes": 4 * (n + c["prefix"]) * c["Hk"] * D + c["B"] * c["Hq"] * (4 * D + 4),
            "flops": 4 * (n + c["B"] * c["prefix"]) * c["Hq"] * D}


# ---------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------
def _thetas(c):
    """Radians per position of each pair, and the factor on cos and sin (lists of floats).

    none: base^(-2i/r); linear: divided by the factor; ntk: the base grows so that the lowest
    frequency is divided by the factor; yarn: frequencies that turn at least 32 times within the
    trained 4096 positions stay, those that turn once or less are divided by the factor, a ramp
    between, and cos and sin times 0.1 ln(factor) + 1."""
    r, base, f = c["rd"], 10000.0, c.get("factor", 1.0)
    scaling = c.get("scaling", "none")
    if scaling == "ntk":
        base *= f ** (r / (r - 2))
    th = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if scaling == "linear":
        th = [t / f for t in th]
    if scaling == "yarn":
        ramp = [min(1.0, max(0.0, (4096 * t / (2 * math.pi) - 1.0) / 31.0)) for t in th]
        th = [t * g + t / f * (1.0 - g) for t, g in zip(th, ramp)]
    return th, (0.1 * math.log(f) + 1.0 if scaling == "yarn" else 1.0)


def _freqs(c):
    """The frequency table that a program keeps for the library's calls."""
    import tiled_attention_08_gb300 as fa
    return fa.rotary_freqs(c["rd"], 10000.0, c.get("scaling", "none"), c.get("factor", 1.0),
                           original_len=4096, device="cuda")


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _permuted(g, values):
    v = torch.tensor(values, dtype=torch.int32, device="cuda")
    return v[torch.randperm(len(values), generator=g, device="cuda")]


def _tables(g, capacity, spare):
    """A block table with `capacity[b]` tokens of room per sequence, pages in shuffled order, and
    the number of pages; entries past a sequence's pages are 0."""
    pages = [(n + PAGE - 1) // PAGE for n in capacity]
    total = sum(pages) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    p = torch.tensor(pages, device="cuda")
    first = torch.cumsum(p, 0) - p
    col = torch.arange(max(1, max(pages)), device="cuda")
    at = (first[:, None] + col[None]).clamp(max=total - 1)
    return torch.where(col[None] < p[:, None], order[at], 0).to(torch.int32), total


def _e4m3_cache(g, pages, H, D):
    """A cache of quantised N(0, 1) rows: e4m3 values [pages, H, 16, D], exponents [pages, H, 16]."""
    val = torch.empty((pages, H, PAGE, D), device="cuda", dtype=torch.float8_e4m3fn)
    ex = torch.empty((pages, H, PAGE), device="cuda", dtype=torch.uint8)
    step = max(1, (1 << 28) // (H * PAGE * D))
    for i in range(0, pages, step):
        x = _randn(g, (min(step, pages - i), H, PAGE, D), torch.float16)
        v, e = _quantise(x.float())
        val[i:i + step], ex[i:i + step] = v, e
    return val, ex


def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    B, D = c["B"], c["D"]
    s = {"c": c, "dtype": dt, "scale": 1.0 / math.sqrt(D)}
    if c.get("rd"):
        th, s["mscale"] = _thetas(c)
        s["theta"] = torch.tensor(th, dtype=torch.float64, device="cuda")
        if own:
            s["freqs"] = _freqs(c)[0]
    if c["kind"] == "rotary":
        L = c["L"]
        if c["packed"]:
            x = _randn(g, (B, L, 3, c["Hq"], D), dt)
            s["q"], s["k"] = x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2)
        else:
            s["q"], s["k"] = _randn(g, (B, c["Hq"], L, D), dt), _randn(g, (B, c["Hk"], L, D), dt)
        at = _permuted(g, _lens(0, c["maxpos"] - L, B))
        s["pos"] = at[:, None] + torch.arange(L, dtype=torch.int32, device="cuda")[None]
        if c["grad"]:
            s["gq"], s["gk"] = _randn(g, s["q"].shape, dt), _randn(g, s["k"].shape, dt)
            s["q"].requires_grad_(), s["k"].requires_grad_()
        return s
    if c["kind"] == "cache":
        start, new = _permuted(g, _lens(0, c["start"], B)), _permuted(g, _new_lens(c))
        s["new_lens"], s["lens"], s["H"] = new, start + new, c["H"]
        s["tables"], pages = _tables(g, s["lens"].tolist(), 5)
        s["k"], s["v"] = _randn(g, (B, c["H"], c["new"], D), dt), _randn(g, (B, c["H"], c["new"], D), dt)
    elif c["kind"] == "decode":
        s["lens"], s["H"] = _permuted(g, _lens(c["lo"], c["hi"], B)), c["Hk"]
        s["tables"], pages = _tables(g, s["lens"].tolist(), 5)
        s["q"] = _randn(g, (B, c["Hq"], D), dt)
        if c["append"]:
            s["k"], s["v"] = _randn(g, (B, c["Hk"], 1, D), dt), _randn(g, (B, c["Hk"], 1, D), dt)
    else:
        s["lens"], s["H"] = _permuted(g, _lens(c["lo"], c["hi"], B)), c["Hk"]
        room = [c["prefix"]] + s["lens"].tolist()
        tables, pages = _tables(g, room, 5)
        s["prefix_table"] = tables[0, :(c["prefix"] + PAGE - 1) // PAGE].contiguous()
        s["tables"] = tables[1:, :max(1, (max(room[1:]) + PAGE - 1) // PAGE)].contiguous()
        s["q"] = _randn(g, (B, c["Hq"], D), dt)
    if c.get("quant"):
        s["kc"], s["ke"] = _e4m3_cache(g, pages, s["H"], D)
        s["vc"], s["ve"] = _e4m3_cache(g, pages, s["H"], D)
    else:
        s["kc"], s["vc"] = (_randn(g, (pages, s["H"], PAGE, D), dt) for _ in range(2))
        s["ke"] = s["ve"] = None
    return s


# ---------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _with_cache(s, o, lse):
    """The step's answer; where it wrote a token, with the cache that it wrote into."""
    return (o, lse, s["kc"], s["vc"], s["ke"], s["ve"]) if s["c"].get("append") else (o, lse)


def _run_own(s):
    import tiled_attention_08_gb300 as fa
    c = s["c"]
    if c["kind"] == "rotary":
        q, k = fa.rotary(s["q"], s["k"], s["pos"], s["freqs"], s["mscale"], c["inter"])
        if not c["grad"]:
            return q, k
        dq, dk = torch.autograd.grad((q, k), (s["q"], s["k"]), (s["gq"], s["gk"]))
        return q.detach(), k.detach(), dq, dk
    if c["kind"] == "cache":
        rot = dict(freqs=s["freqs"], mscale=s["mscale"], interleaved=c["inter"]) if c["rd"] else {}
        fa.cache_append(s["k"], s["v"], s["kc"], s["vc"], s["tables"], s["lens"], s["new_lens"],
                        k_exp=s["ke"], v_exp=s["ve"], **rot)
        return fa.cache_read(s["kc"], s["vc"], s["tables"], s["lens"], c["start"] + c["new"],
                             k_exp=s["ke"], v_exp=s["ve"], dtype=s["dtype"])
    if c["kind"] == "decode":
        if c["append"]:
            fa.cache_append(s["k"], s["v"], s["kc"], s["vc"], s["tables"], s["lens"],
                            k_exp=s["ke"], v_exp=s["ve"])
        o, lse = fa.decode_paged(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["scale"],
                                 k_exp=s["ke"], v_exp=s["ve"])
        return _with_cache(s, o, lse)
    return fa.decode_shared_prefix(s["q"], s["kc"], s["vc"], s["prefix_table"], c["prefix"],
                                   s["tables"], s["lens"], s["scale"])


def _rotate(x, pos, theta, mscale, inter):
    """x [B, H, L, D] in 32 bits, rotated by pos [B, L] times theta [r/2] (angles in 64)."""
    ang = pos.double()[:, None, :, None] * theta
    cos, sin = (torch.cos(ang) * mscale).float(), (torch.sin(ang) * mscale).float()
    r = 2 * theta.numel()
    rot, rest = x[..., :r], x[..., r:]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if inter else (rot[..., :r // 2], rot[..., r // 2:])
    u, w = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((u, w), -1).flatten(-2) if inter else torch.cat((u, w), -1)
    return torch.cat((y, rest), -1)


def _quantise(x):
    """e4m3 values and biased exponents of rows: the smallest power of two that brings the row's
    largest magnitude to at most 448, rounded to the nearest (ties to even)."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-127, 127)
    e = torch.where(amax == 0, -127, e)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _dense(cache, ex, tables):
    """The rows of the tables' pages as [B, H, tokens, D] in 32 bits."""
    t = tables.long()
    x = cache.view(torch.uint8)[t].view(torch.float8_e4m3fn).float() if ex is not None else cache[t].float()
    if ex is not None:
        x = torch.ldexp(x, ex[t].int()[..., None] - 127)
    B, n, H, page, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, n * page, D)


def _append(s, k, v, new_lens):
    """Rows t < new_lens[b] of k, v [B, H, L, D] (32 bits) into the last slots of each sequence."""
    t = torch.arange(k.shape[2], device="cuda")[None]
    at = (s["lens"] - new_lens)[:, None] + t
    b, t = torch.nonzero(t < new_lens[:, None], as_tuple=True)
    at = at[b, t].long()
    page, slot = s["tables"][b, at // PAGE].long(), at % PAGE
    for x, cache, ex in ((k, s["kc"], s["ke"]), (v, s["vc"], s["ve"])):
        rows = x.transpose(1, 2)[b, t]  # [tokens, H, D]
        if ex is None:
            cache[page, :, slot] = rows.to(cache.dtype)
        else:
            val, e = _quantise(rows)
            cache.view(torch.uint8)[page, :, slot] = val.view(torch.uint8)
            ex[page, :, slot] = e


def _scores(q, k, scale):
    """q [B, Hk, G, D] . k [B, Hk, n, D] * scale in 32 bits."""
    return (q @ k.transpose(-1, -2)) * scale


def _run_plain(s):
    c, dt = s["c"], s["dtype"]
    if c["kind"] == "rotary":
        with torch.no_grad():
            rot = lambda x, sign: _rotate(x.float(), s["pos"], sign * s["theta"], s["mscale"], c["inter"]).to(dt)  # noqa: E731
            out = rot(s["q"], 1), rot(s["k"], 1)
            return out + (rot(s["gq"], -1), rot(s["gk"], -1)) if c["grad"] else out
    if c["kind"] == "cache":
        k = s["k"].float()
        if c["rd"]:
            pos = (s["lens"] - s["new_lens"])[:, None] + torch.arange(c["new"], device="cuda")[None]
            k = _rotate(k, pos, s["theta"], s["mscale"], c["inter"])
        _append(s, k, s["v"].float(), s["new_lens"])
        n = c["start"] + c["new"]
        live = torch.arange(n, device="cuda")[None, None, :, None] < s["lens"][:, None, None, None]
        out = []
        for x in (_dense(s["kc"], s["ke"], s["tables"]), _dense(s["vc"], s["ve"], s["tables"])):
            x = torch.nn.functional.pad(x, (0, 0, 0, max(0, n - x.shape[2])))[:, :, :n]
            out.append(torch.where(live, x, 0.0).to(dt))
        return tuple(out)
    if c["kind"] == "decode" and c["append"]:
        _append(s, s["k"].float(), s["v"].float(), torch.ones_like(s["lens"]))
    B, H, D = c["B"], c["Hk"], c["D"]
    q = s["q"].float().view(B, H, -1, D)
    k, v = _dense(s["kc"], s["ke"], s["tables"]), _dense(s["vc"], s["ve"], s["tables"])
    y = _scores(q, k, s["scale"])
    dead = torch.arange(k.shape[2], device="cuda")[None] >= s["lens"][:, None]
    y = y.masked_fill(dead[:, None, None], -math.inf)
    v = v.masked_fill(dead[:, None, :, None], 0.0)
    if c["kind"] == "prefix":
        G = q.shape[2]
        kp, vp = (_dense(x, None, s["prefix_table"][None])[0, :, :c["prefix"]] for x in (s["kc"], s["vc"]))
        qh = q.transpose(0, 1).reshape(H, B * G, D)
        yp = ((qh @ kp.transpose(-1, -2)) * s["scale"]).view(H, B, G, -1).transpose(0, 1)
        top = torch.maximum(y.amax(-1), yp.amax(-1))[..., None]
        p, pp = torch.exp(y - top), torch.exp(yp - top)
        total = p.sum(-1) + pp.sum(-1)
        o = p @ v + (pp.transpose(0, 1).reshape(H, B * G, -1) @ vp).view(H, B, G, D).transpose(0, 1)
    else:
        top = y.amax(-1, keepdim=True)
        p = torch.exp(y - top)
        total = p.sum(-1)
        o = p @ v
    o = o / total[..., None]
    lse = top[..., 0] + torch.log(total)
    return _with_cache(s, o.reshape(B, -1, D).to(dt), lse.reshape(B, -1))


# ---------------------------------------------------------------------------------------
# The same results from the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _turned(x, pos, theta, mscale, inter):
    """Pairs of x as complex numbers times mscale * exp(i pos theta), in 64 bits."""
    x = x.double().clone()
    r = 2 * len(theta)
    z = torch.polar(torch.full((), float(mscale), dtype=torch.float64, device="cuda"),
                    pos.double().unsqueeze(-1) * theta).unsqueeze(1)
    first, second = (slice(0, r, 2), slice(1, r, 2)) if inter else (slice(0, r // 2), slice(r // 2, r))
    y = torch.complex(x[..., first], x[..., second]) * z
    x[..., first], x[..., second] = y.real, y.imag
    return x


def _held(x):
    """What rows of x (64 bits) stand for once held as e4m3 times a power of two per row."""
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, 1.0) / E4M3_MAX))
    e = torch.where(amax > torch.exp2(e) * E4M3_MAX, e + 1, e)
    e = torch.where(amax <= torch.exp2(e - 1) * E4M3_MAX, e - 1, e).clamp(-127, 127)
    y = x / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * torch.exp2(e)


def _row64(cache, ex, table, n):
    """The first n tokens of one table's pages, [H, n, D] in 64 bits."""
    t = table[:(n + PAGE - 1) // PAGE].long()
    if ex is None:
        x = cache[t].double()
    else:
        x = cache.view(torch.uint8)[t].view(torch.float8_e4m3fn).double() * torch.exp2(ex[t].double() - 127)[..., None]
    return x.transpose(0, 1).reshape(cache.shape[1], -1, cache.shape[3])[:, :n]


def exact(case, seed):
    s = prepare(case, seed)
    c, dt = case, DTYPES[case["dtype"]]
    if c["kind"] == "rotary":
        if c["B"] * c["L"] * (c["Hq"] + c["Hk"]) * c["D"] > 1 << 29:
            return None
        with torch.no_grad():
            f = [_turned(s[n], s["pos"], s["theta"], s["mscale"], c["inter"]) for n in ("q", "k")]
            if c["grad"]:
                f += [_turned(s[n], -s["pos"], s["theta"], s["mscale"], c["inter"]) for n in ("gq", "gk")]
        return tuple(f)
    lens = s["lens"].tolist()
    if c["kind"] == "cache":
        n = c["start"] + c["new"]
        k, v = s["k"].double(), s["v"].double()
        if c["rd"]:
            pos = (s["lens"] - s["new_lens"])[:, None] + torch.arange(c["new"], device="cuda")[None]
            k = _turned(k, pos, s["theta"], s["mscale"], c["inter"])
        out = [torch.zeros((c["B"], c["H"], n, c["D"]), dtype=torch.float64, device="cuda") for _ in range(2)]
        for b, new in enumerate(s["new_lens"].tolist()):
            old = lens[b] - new
            for o, x, cache, ex in ((out[0], k, s["kc"], s["ke"]), (out[1], v, s["vc"], s["ve"])):
                if old:
                    o[b, :, :old] = _row64(cache, ex, s["tables"][b], old)
                rows = x[b, :, :new]
                o[b, :, old:lens[b]] = _held(rows) if c["quant"] else rows.to(dt).double()
        return tuple(out)
    H, D = c["Hk"], c["D"]
    if c["kind"] == "prefix":
        kp, vp = (_row64(x, None, s["prefix_table"], c["prefix"]) for x in (s["kc"], s["vc"]))
    o, lse = [], []
    for b, n in enumerate(lens):
        k, v = _row64(s["kc"], s["ke"], s["tables"][b], n), _row64(s["vc"], s["ve"], s["tables"][b], n)
        if c.get("append"):
            new = [_held(s[x][b].double()) if c["quant"] else s[x][b].double() for x in ("k", "v")]
            k, v = torch.cat((k[:, :n - 1], new[0]), 1), torch.cat((v[:, :n - 1], new[1]), 1)
        if c["kind"] == "prefix":
            k, v = torch.cat((kp, k), 1), torch.cat((vp, v), 1)
        y = s["q"][b].double().view(H, -1, D) @ k.mT * s["scale"]
        lse.append(torch.logsumexp(y, -1).reshape(-1))
        o.append((torch.softmax(y, -1) @ v).reshape(-1, D))
    out = torch.stack(o), torch.stack(lse)
    return out + (None,) * 4 if c.get("append") else out
