"""Measured cases of attention with a sliding window, dense and over a paged cache.

Three operators, each in its plain form (elementary torch operations, 32-bit sums, one rounding at
the end) and, where ``own`` is true, through the library's public calls:

* attention in which a token sees the ``window`` tokens up to its own and the first ``sinks`` of the
  sequence, with grouped heads, forward and backward;
* attention of a chunk of new tokens of every sequence over a paged cache (16-bit or e4m3), with or
  without such a window;
* one decode step over a paged cache with such a window.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges.
"""
import math

import torch

own = False

PAGE = 16  # tokens per page of the cache
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # A training step's layer at a long context: 32 query heads on 8, window of a quarter.
        dict(name="window_train_L16384_W4096", kind="dense", B=1, Hq=32, Hk=8, Lq=16384, Lk=16384,
             D=128, window=4096, sinks=4, dtype="bf16", grad=True, blhd=False),
        # The training shape of the benchmark (8 x 4096 tokens, 32 heads of 128) with a window.
        dict(name="window_train_B8_L4096_W1024", kind="dense", B=8, Hq=32, Hk=32, Lq=4096, Lk=4096,
             D=128, window=1024, sinks=0, dtype="bf16", grad=True, blhd=False),
        # 64-wide heads, odd lengths and window, more first tokens than a tile, [B, L, H, D] memory.
        dict(name="window_train_odd_D64", kind="dense", B=3, Hq=16, Hk=4, Lq=5001, Lk=5001, D=64,
             window=777, sinks=131, dtype="fp16", grad=True, blhd=True),
        # The last tokens of a short prompt behind earlier ones, forward only: latency.
        dict(name="window_tail_L200", kind="dense", B=1, Hq=32, Hk=8, Lq=200, Lk=1500, D=128,
             window=512, sinks=16, dtype="fp16", grad=False, blhd=False),
        # One short turn of one conversation behind a short history, 8-bit cache: latency.
        dict(name="chunk_B1_L16", kind="chunk", B=1, Hq=32, Hk=8, D=128, new=16, lo=517, hi=517,
             window=0, sinks=0, quant=True, dtype="bf16"),
        # Chunked prefill of 8 prompts behind up to 16384 cached tokens, 8 query heads per cache
        # head, 8-bit cache.
        dict(name="chunk_B8_L512_e4m3", kind="chunk", B=8, Hq=64, Hk=8, D=128, new=512, lo=512,
             hi=16384, window=0, sinks=0, quant=True, dtype="bf16"),
        # Large chunks of long documents with a window, 16-bit cache.
        dict(name="chunk_B4_L2048_W4096", kind="chunk", B=4, Hq=32, Hk=8, D=128, new=2048, lo=2048,
             hi=32768, window=4096, sinks=16, quant=False, dtype="bf16"),
        # Two whole prompts of 4096 tokens through the cache, 32 equal heads of 128.
        dict(name="chunk_prompt_B2_L4096", kind="chunk", B=2, Hq=32, Hk=32, D=128, new=4096, lo=0,
             hi=0, window=0, sinks=0, quant=False, dtype="bf16"),
        # 64-wide heads, odd lengths, chunks of different sizes in a padded batch.
        dict(name="chunk_B17_L127_D64", kind="chunk", B=17, Hq=16, Hk=4, D=64, new=127, lo=77,
             hi=4001, window=0, sinks=0, quant=False, dtype="fp16"),
        # A continuous batch of 256 sequences of 1..16384 tokens, a window of 4096.
        dict(name="decode_window_B256_W4096", kind="decode", B=256, Hq=32, Hk=8, D=128, lo=1,
             hi=16384, window=4096, sinks=4, quant=False, dtype="bf16"),
        # Long conversations, a short window, 8 query heads per cache head, 8-bit cache.
        dict(name="decode_window_B48_W1024", kind="decode", B=48, Hq=64, Hk=8, D=128, lo=777,
             hi=32768, window=1024, sinks=64, quant=True, dtype="bf16"),
        # One sequence: the smallest serving step.
        dict(name="decode_window_B1", kind="decode", B=1, Hq=32, Hk=8, D=128, lo=5000, hi=5000,
             window=512, sinks=16, quant=True, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["dense", "chunk", "decode"])
    D = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 8, 32])
    c = dict(kind=kind, B=1, Hq=Hk * rng.choice([1, 2, 3, 4, 8] if Hk < 32 else [1]), Hk=Hk, D=D,
             window=0, sinks=rng.choice([0, rng.randint(1, 16), rng.randint(1, 200)]),
             dtype=rng.choice(["bf16", "fp16"]))
    if kind == "dense":
        grad = rng.random() < 0.7
        c["B"], c["Lk"] = _spread(rng, 1, 16), _spread(rng, 16, 16384)
        c["Lq"] = c["Lk"] if grad or rng.random() < 0.5 else rng.randint(1, c["Lk"])
        c["window"] = _spread(rng, 8, 4096)
        c["grad"], c["blhd"] = grad, rng.random() < 0.5
        while work(c)["flops"] > 3.3e12:
            c["B"], c["Lk"], c["Lq"] = max(1, c["B"] // 2), c["Lk"] // 2, max(1, c["Lq"] // 2)
        return c
    c["quant"] = rng.random() < 0.5
    if kind == "chunk":
        c["B"], c["new"], c["hi"] = _spread(rng, 1, 32), _spread(rng, 2, 4096), _spread(rng, 16, 32768)
        c["lo"] = rng.randint(0, c["hi"])
        if rng.random() < 0.5:
            c["window"] = _spread(rng, 16, 8192)
        while work(c)["flops"] > 9.0e11 or c["B"] * (c["hi"] + c["new"]) * Hk * D > 1 << 29:
            c["B"], c["new"] = max(1, c["B"] // 2), max(2, c["new"] // 2)
            c["lo"], c["hi"] = c["lo"] // 2, max(16, c["hi"] // 2)
        return c
    c["B"], c["hi"] = _spread(rng, 1, 256), _spread(rng, 16, 32768)
    c["lo"], c["window"] = rng.randint(1, c["hi"]), _spread(rng, 16, 4096)
    while work(c)["bytes"] > 3.0e9 or c["B"] * c["hi"] * Hk * D > 1 << 32:
        c["B"], c["lo"], c["hi"] = max(1, c["B"] // 2), max(1, c["lo"] // 2), max(16, c["hi"] // 2)
    return c


def _lens(lo, hi, n):
    """n whole numbers spread evenly from lo to hi."""
    return [lo + (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _new_lens(c):
    return _lens(max(1, c["new"] // 2), c["new"], c["B"])


def _seen(t, window, sinks):
    """Tokens that a query at position t >= 0 sees (window 0: all up to its own)."""
    if window == 0 or t < window:
        return t + 1
    return window + min(sinks, t + 1 - window)


def work(case):
    """Each input read once (of a cache the rows that some query sees), each output written once;
    products and sums of the attention, two and a half times as many backward."""
    c, D, w, s = case, case["D"], case["window"], case["sinks"]
    if c["kind"] == "dense":
        pairs = sum(_seen(t, w, s) for t in range(max(0, c["Lk"] - c["Lq"]), c["Lk"]))
        q, k = c["B"] * c["Hq"] * c["Lq"], c["B"] * c["Hk"] * c["Lk"]
        fwd = 4 * q * D + 4 * k * D + 4 * q
        bwd = 8 * q * D + 8 * k * D + 4 * q
        return {"bytes": fwd + (bwd if c["grad"] else 0),
                "flops": c["B"] * c["Hq"] * D * pairs * (14 if c["grad"] else 4)}
    row = 2 * (D + 1 if c["quant"] else 2 * D)
    rows = pairs = queries = 0
    if c["kind"] == "decode":
        for n in _lens(c["lo"], c["hi"], c["B"]):
            rows, pairs = rows + _seen(n - 1, w, s), pairs + _seen(n - 1, w, s)
        queries = c["B"]
    else:
        for old, new in zip(_lens(c["lo"], c["hi"], c["B"]), _new_lens(c)):
            rows += new - 1 + _seen(old, w, s)
            pairs += sum(_seen(t, w, s) for t in range(old, old + new))
            queries += c["new"]
    return {"bytes": rows * c["Hk"] * row + queries * c["Hq"] * (4 * D + 4),
            "flops": 4 * pairs * c["Hq"] * D}


# ---------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------
def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _permuted(g, values):
    v = torch.tensor(values, dtype=torch.int32, device="cuda")
    return v[torch.randperm(len(values), generator=g, device="cuda")]


def _tables(g, room, spare):
    """A block table with room for `room[b]` tokens of each sequence, pages in shuffled order, and
    the number of pages; entries behind a sequence's pages are 0."""
    pages = torch.tensor([(n + PAGE - 1) // PAGE for n in room], device="cuda")
    total = int(pages.sum()) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    first = torch.cumsum(pages, 0) - pages
    col = torch.arange(max(1, int(pages.max())), device="cuda")
    at = (first[:, None] + col[None]).clamp(max=total - 1)
    return torch.where(col[None] < pages[:, None], order[at], 0).to(torch.int32), total


def _e4m3_cache(g, pages, H, D):
    """Rows of N(0, 1) as e4m3 values times a power of two each: values [pages, H, 16, D] and
    exponents + 127 [pages, H, 16].  The power of two is the smallest that brings the row's largest
    magnitude to at most 448."""
    val = torch.empty((pages, H, PAGE, D), device="cuda", dtype=torch.float8_e4m3fn)
    ex = torch.empty((pages, H, PAGE), device="cuda", dtype=torch.uint8)
    step = max(1, (1 << 28) // (H * PAGE * D))
    for i in range(0, pages, step):
        x = _randn(g, (min(step, pages - i), H, PAGE, D), torch.float16).float()
        m, e = torch.frexp(x.abs().amax(-1))  # m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
        e = torch.where(m > 0.875, e - 8, e - 9)
        val[i:i + step] = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
        ex[i:i + step] = (e + 127).to(torch.uint8)
    return val, ex


def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    B, D = c["B"], c["D"]
    s = {"c": c, "dtype": dt, "scale": 1.0 / math.sqrt(D)}
    if c["kind"] == "dense":
        def operand(H, L):
            if c["blhd"]:
                return _randn(g, (B, L, H, D), dt).transpose(1, 2)
            return _randn(g, (B, H, L, D), dt)
        s["q"], s["k"], s["v"] = operand(c["Hq"], c["Lq"]), operand(c["Hk"], c["Lk"]), operand(c["Hk"], c["Lk"])
        if c["grad"]:
            s["do"] = operand(c["Hq"], c["Lq"])
            for x in ("q", "k", "v"):
                s[x].requires_grad_()
        return s
    lens = _permuted(g, _lens(c["lo"], c["hi"], B))
    if c["kind"] == "chunk":
        s["new_lens"] = _permuted(g, _new_lens(c))
        s["lens"] = lens + s["new_lens"]
        s["q"] = _randn(g, (B, c["Hq"], c["new"], D), dt)
    else:
        s["lens"] = lens
        s["q"] = _randn(g, (B, c["Hq"], D), dt)
    s["lens_list"] = s["lens"].tolist()  # a scheduler knows them on the host, too
    s["new_list"] = s["new_lens"].tolist() if c["kind"] == "chunk" else None
    s["tables"], pages = _tables(g, s["lens_list"], 5)
    if c["quant"]:
        s["kc"], s["ke"] = _e4m3_cache(g, pages, c["Hk"], D)
        s["vc"], s["ve"] = _e4m3_cache(g, pages, c["Hk"], D)
    else:
        s["kc"], s["vc"] = (_randn(g, (pages, c["Hk"], PAGE, D), dt) for _ in range(2))
        s["ke"] = s["ve"] = None
    return s


# ---------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    with torch.no_grad():
        return {"dense": _plain_dense, "chunk": _plain_chunk, "decode": _plain_decode}[state["c"]["kind"]](state)


def _run_own(s):
    import tiled_attention_08_gb300 as fa
    c = s["c"]
    if c["kind"] == "dense":
        o = fa.attention_window(s["q"], s["k"], s["v"], c["window"], c["sinks"], s["scale"])
        if not c["grad"]:
            return o
        grads = torch.autograd.grad(o, (s["q"], s["k"], s["v"]), s["do"])
        return (o.detach(), *grads)
    kw = dict(scale=s["scale"], k_exp=s["ke"], v_exp=s["ve"])
    if c["window"]:
        kw.update(window=c["window"], sinks=c["sinks"])
    if c["kind"] == "chunk":
        return fa.attention_paged(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["new_lens"], **kw)
    return fa.decode_paged(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], **kw)


def _hidden(t, j, window, sinks):
    """Whether queries at positions t [n, 1] do not see keys j [1, m]."""
    far = j > t
    return far | ((j <= t - window) & (j >= sinks)) if window else far


def _keys(first, last, window, sinks):
    """Indices of the keys that queries at positions first .. last can see between them."""
    lo = max(0, first - window + 1) if window else 0
    lead = torch.arange(min(sinks, lo), device="cuda")
    return torch.cat((lead, torch.arange(lo, last + 1, device="cuda")))


def _weights(y, hidden):
    """exp(y - top) with zeros where hidden, its sums and log-sum-exp; rows that see nothing: zeros
    and -inf."""
    y = y.masked_fill(hidden, -math.inf)
    top = y.amax(-1, keepdim=True)
    p = torch.exp(y - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return p, total, (top + torch.log(total))[..., 0]


def _plain_dense(s):
    c, dt = s["c"], s["dtype"]
    B, Hq, Hk, Lq, Lk, D = (c[x] for x in ("B", "Hq", "Hk", "Lq", "Lk", "D"))
    w, sinks, G, step = c["window"], c["sinks"], Hq // Hk, 1024
    group = lambda x: x.detach().float().reshape(B, Hk, G, Lq, D)  # noqa: E731
    q, k, v = group(s["q"]), s["k"].detach().float(), s["v"].detach().float()
    o = torch.zeros_like(q)
    if c["grad"]:
        do = group(s["do"])
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b in range(B):
        for r in range(0, Lq, step):
            rows = slice(r, min(r + step, Lq))
            t = torch.arange(rows.start, rows.stop, device="cuda")[:, None] + (Lk - Lq)
            at = _keys(rows.start + Lk - Lq, rows.stop - 1 + Lk - Lq, w, sinks)
            kb, vb = k[b][:, at][:, None], v[b][:, at][:, None]
            p, total, _ = _weights((q[b][:, :, rows] @ kb.mT) * s["scale"], _hidden(t, at[None], w, sinks))
            p = p / torch.where(total > 0, total, 1.0)
            o[b][:, :, rows] = p @ vb
            if c["grad"]:
                g = do[b][:, :, rows]
                dp = g @ vb.mT
                delta = (g * o[b][:, :, rows]).sum(-1, keepdim=True)
                ds = p * (dp - delta) * s["scale"]
                dq[b][:, :, rows] = ds @ kb
                dk[b].index_add_(1, at, (ds.mT @ q[b][:, :, rows]).sum(1))
                dv[b].index_add_(1, at, (p.mT @ g).sum(1))
    o = o.reshape(B, Hq, Lq, D).to(dt)
    return (o, dq.reshape(B, Hq, Lq, D).to(dt), dk.to(dt), dv.to(dt)) if c["grad"] else o


def _cached(s, which, b, at):
    """Rows of tokens `at` of sequence b, [Hk, n, D] in 32 bits."""
    cache, ex = (s["kc"], s["ke"]) if which == "k" else (s["vc"], s["ve"])
    page, slot = s["tables"][b, at // PAGE].long(), at % PAGE
    if ex is None:
        return cache[page, :, slot].float().transpose(0, 1)
    x = cache.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float()
    return torch.ldexp(x, ex[page, :, slot].int()[..., None] - 127).transpose(0, 1)


def _plain_chunk(s):
    c, dt = s["c"], s["dtype"]
    Hk, D, w, sinks, step = c["Hk"], c["D"], c["window"], c["sinks"], 256
    q = s["q"].float().view(c["B"], Hk, -1, c["new"], D)
    o, lse = torch.zeros_like(q), torch.full(q.shape[:-1], -math.inf, device="cuda")
    for b, (n, new) in enumerate(zip(s["lens_list"], s["new_list"])):
        for r in range(0, new, step):
            rows = slice(r, min(r + step, new))
            t = torch.arange(rows.start, rows.stop, device="cuda")[:, None] + (n - new)
            at = _keys(rows.start + n - new, rows.stop - 1 + n - new, w, sinks)
            y = (q[b][:, :, rows] @ _cached(s, "k", b, at)[:, None].mT) * s["scale"]
            p, total, lse[b][:, :, rows] = _weights(y, _hidden(t, at[None], w, sinks))
            o[b][:, :, rows] = (p @ _cached(s, "v", b, at)[:, None]) / total
    return o.view(s["q"].shape).to(dt), lse.view(s["q"].shape[:-1])


def _plain_decode(s):
    c, dt = s["c"], s["dtype"]
    B, Hk, D, w, sinks = c["B"], c["Hk"], c["D"], c["window"], c["sinks"]
    n = s["lens"].long()[:, None]
    lo = (n - w).clamp(min=0)  # the window's first token
    lead = torch.arange(sinks, device="cuda")[None]
    rest = torch.arange(w, device="cuda")[None] + lo
    at = torch.cat((lead.expand(B, -1), rest), 1)
    hidden = torch.cat((lead >= lo, rest >= n), 1)
    at = at.masked_fill(hidden, 0)
    page, slot = torch.gather(s["tables"].long(), 1, at // PAGE), at % PAGE

    def dense(cache, ex):
        if ex is None:
            return cache[page, :, slot].float().transpose(1, 2)
        x = cache.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float()
        return torch.ldexp(x, ex[page, :, slot].int()[..., None] - 127).transpose(1, 2)

    y = (s["q"].float().view(B, Hk, -1, D) @ dense(s["kc"], s["ke"]).mT) * s["scale"]
    p, total, lse = _weights(y, hidden[:, None, None])
    o = (p @ dense(s["vc"], s["ve"])) / total
    return o.reshape(B, -1, D).to(dt), lse.reshape(B, -1)


# ---------------------------------------------------------------------------------------
# The same results from the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _attend64(q, k, v, first, w, sinks, scale):
    """Queries q [.., n, D] at positions first .. first + n - 1 on keys 0 .. of [H, 1, m, D]."""
    n, m = q.shape[-2], k.shape[-2]
    back = (torch.arange(n, device="cuda") + first)[:, None] - torch.arange(m, device="cuda")[None]
    sees = back >= 0
    if w:
        sees &= (back < w) | (torch.arange(m, device="cuda")[None] < sinks)
    y = torch.where(sees, q @ k.mT * scale, -math.inf)
    return torch.softmax(y, -1) @ v, torch.logsumexp(y, -1)


def _row64(cache, ex, table, n):
    """The first n tokens of one table's pages, [H, n, D] in 64 bits."""
    t = table[:(n + PAGE - 1) // PAGE].long()
    if ex is None:
        x = cache[t].double()
    else:
        x = cache.view(torch.uint8)[t].view(torch.float8_e4m3fn).double() * torch.exp2(ex[t].double() - 127)[..., None]
    return x.transpose(0, 1).reshape(cache.shape[1], -1, cache.shape[3])[:, :n]


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    B, Hk, D, w, sinks = c["B"], c["Hk"], c["D"], c["window"], c["sinks"]
    if c["kind"] == "dense":
        G, Lq, Lk = c["Hq"] // Hk, c["Lq"], c["Lk"]
        out = [torch.empty((B, H, L, D), dtype=torch.float64, device="cuda")
               for H, L in ((c["Hq"], Lq), (c["Hq"], Lq), (Hk, Lk), (Hk, Lk))]
        for b in range(B):
            for h in range(Hk):
                heads = slice(h * G, h * G + G)
                k, v = (s[x].detach()[b, h].double().requires_grad_(c["grad"]) for x in ("k", "v"))
                for r in range(0, Lq, 512):  # rows r .. of the group's heads
                    n, first = min(512, Lq - r), r + Lk - Lq
                    q = s["q"].detach()[b, heads, r:r + n].double().requires_grad_(c["grad"])
                    a = max(0, first + 1 - w)  # keys a .. and the sinks before them
                    e = min(sinks, a)
                    kk, vv = (torch.cat((x[:e], x[a:first + n])) for x in (k, v))
                    # The lead's keys stand right before the window's: shift their distance.
                    back = (torch.arange(n, device="cuda") + first)[:, None] - torch.cat(
                        (torch.arange(e, device="cuda"), torch.arange(a, first + n, device="cuda")))[None]
                    sink = torch.arange(kk.shape[0], device="cuda")[None] < e
                    if a < sinks:
                        sink = sink | (torch.arange(kk.shape[0], device="cuda")[None] < sinks)
                    y = torch.where((back >= 0) & ((back < w) | sink), q @ kk.mT * s["scale"], -math.inf)
                    o = torch.softmax(y, -1) @ vv
                    out[0][b, heads, r:r + n] = o.detach()
                    if c["grad"]:
                        o.backward(s["do"][b, heads, r:r + n].double())
                        out[1][b, heads, r:r + n] = q.grad
                if c["grad"]:
                    out[2][b, h], out[3][b, h] = k.grad, v.grad
        return tuple(out) if c["grad"] else out[0]
    lens, news = s["lens_list"], s["new_list"] or [1] * B
    most = c["new"] if c["kind"] == "chunk" else 1
    q = s["q"].view(B, Hk, -1, most, D).double()
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, new) in enumerate(zip(lens, news)):
        k, v = _row64(s["kc"], s["ke"], s["tables"][b], n), _row64(s["vc"], s["ve"], s["tables"][b], n)
        for r in range(0, new, 128):
            e = min(128, new - r)
            out[b, :, :, r:r + e], lse[b, :, :, r:r + e] = _attend64(
                q[b, :, :, r:r + e], k[:, None], v[:, None], n - new + r, w, sinks, s["scale"])
    return out.view(s["q"].shape), lse.view(s["q"].shape[:-1])
