"""The operators around speculative sampling of several continuations of one prompt as they are measured: RMS norm with the
residual's addition, attention of a batch over a shared prefix and each request's own pages, and verification of drafted tokens
by sampling. Each case is one pass through one operator, either in its plain form (elementary torch operations) or, where
``own`` is true, through the package's entry points."""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}


def listed():
    return [
        # one token between two blocks of the 5120 wide stack
        {"name": "norm one token", "op": "norm", "rows": 1, "width": 5120, "dtype": "bf16", "out": "bf16", "group": 0},
        # 64 sequences of 8-row verify blocks, 8-bit inputs of the next products with a scale for 128 columns
        {"name": "norm verify e4m3", "op": "norm", "rows": 512, "width": 7168, "dtype": "bf16", "out": "e4m3", "group": 128},
        # an odd prompt chunk, a scale for each token
        {"name": "norm prompt e4m3", "op": "norm", "rows": 8191, "width": 6144, "dtype": "f16", "out": "e4m3", "group": 6144},
        # a residual stream held in fp32
        {"name": "norm prompt f32", "op": "norm", "rows": 4000, "width": 5120, "dtype": "f32", "out": "f32", "group": 0},
        # a few short continuations of a short prompt, small heads
        {"name": "prefix short", "op": "prefix", "batch": 3, "rows": 1, "hq": 4, "hkv": 1, "d": 64, "prefix": 130, "lo": 0,
         "hi": 40, "page": 16, "dtype": "f16", "cache": "f16"},
        # four samples of one 4096-token prompt, 24 / 4 x 256
        {"name": "prefix four samples", "op": "prefix", "batch": 4, "rows": 1, "hq": 24, "hkv": 4, "d": 256, "prefix": 4096,
         "lo": 1, "hi": 64, "page": 64, "dtype": "bf16", "cache": "bf16"},
        # 64 requests behind one long document, 48 / 8 x 128, answers of up to 2000 tokens
        {"name": "prefix document", "op": "prefix", "batch": 64, "rows": 1, "hq": 48, "hkv": 8, "d": 128, "prefix": 32768,
         "lo": 1, "hi": 2000, "page": 64, "dtype": "bf16", "cache": "bf16"},
        # 32 requests verify 8 rows each behind an instruction of an odd length
        {"name": "prefix verify", "op": "prefix", "batch": 32, "rows": 8, "hq": 48, "hkv": 8, "d": 128, "prefix": 8191,
         "lo": 8, "hi": 1000, "page": 16, "dtype": "bf16", "cache": "bf16"},
        # a full server behind a long document in an e4m3 cache
        {"name": "prefix document e4m3", "op": "prefix", "batch": 64, "rows": 1, "hq": 48, "hkv": 8, "d": 128, "prefix": 65536,
         "lo": 1, "hi": 500, "page": 32, "dtype": "bf16", "cache": "e4m3"},
        # one user, an anchor and seven drafts
        {"name": "drafts one user", "op": "drafts", "batch": 1, "rows": 8, "vocab": 151936, "dtype": "f32", "draft": True},
        # 64 users, an anchor and three drafts
        {"name": "drafts 64 users", "op": "drafts", "batch": 64, "rows": 4, "vocab": 202048, "dtype": "f32", "draft": True},
        # sampling without drafts from bf16 logits of an odd vocabulary
        {"name": "sample 128 bf16", "op": "drafts", "batch": 128, "rows": 1, "vocab": 163841, "dtype": "bf16", "draft": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "prefix", "prefix", "drafts"])
    if op == "norm":
        width = 128 * rng.randint(2, 128) if rng.random() < 0.6 else 16 * rng.randint(4, 1000)
        dtype, out = rng.choice(["bf16", "f16", "f32"]), rng.choice(["same", "e4m3"])
        group = 0 if out == "same" else rng.choice([128, width]) if width % 128 == 0 else width
        return {"op": op, "rows": _log_int(rng, 1, min(8000, int(4e7 / width))), "width": width, "dtype": dtype,
                "out": dtype if out == "same" else out, "group": group}
    if op == "prefix":
        hkv = rng.choice([1, 2, 4, 8])
        d = rng.choice([64, 96, 128, 128, 256])
        group, rows = rng.choice([1, 4, 6, 7, 8, 12]), rng.choice([1, 1, 1, 2, 5, 8])
        prefix = _log_int(rng, 1, 60000)
        # the products over the prefix, and the cache that is read, are bounded by those of the largest listed cases
        most = max(1, min(int(1.2e10 / (prefix * hkv * group * rows * d)), 200))
        batch = _log_int(rng, 1, most)
        hi = _log_int(rng, 1, max(2, min(4000, int(1e8 / (batch * hkv * d)))))
        dtype = rng.choice(["bf16", "f16"])
        return {"op": op, "batch": batch, "rows": rows, "hq": hkv * group, "hkv": hkv, "d": d, "prefix": prefix,
                "lo": rng.randint(0, hi), "hi": hi, "page": rng.choice([1, 16, 24, 32, 64, 256]), "dtype": dtype,
                "cache": rng.choice([dtype, dtype, "e4m3"])}
    rows, vocab = rng.choice([1, 2, 3, 5, 8]), _log_int(rng, 1000, 240000)
    return {"op": op, "batch": _log_int(rng, 1, max(1, min(256, int(8e7 / (rows * vocab))))), "rows": rows, "vocab": vocab,
            "dtype": rng.choice(["f32", "bf16", "f16"]), "draft": rows > 1 and rng.random() < 0.7}


# ---- inputs -----------------------------------------------------------------------------------------------------

def _spread(lo, hi, n, g=None):
    """n whole numbers evenly spaced over [lo, hi] (their sum does not depend on the seed), in an order that does."""
    v = torch.tensor([lo + (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)], dtype=torch.int32)
    return v if g is None else v[torch.randperm(n, generator=g)]


def _pages(tokens, page):
    return (tokens + page - 1) // page


def prepare(case, seed):
    g = torch.Generator()
    g.manual_seed(int(seed))
    dev = torch.device("cuda")
    gd = torch.Generator(device=dev)
    gd.manual_seed(int(seed) + 1)
    return {"norm": _prepare_norm, "prefix": _prepare_prefix, "drafts": _prepare_drafts}[case["op"]](case, g, gd, dev)


def _prepare_norm(case, g, gd, dev):
    n, width, dt, out = case["rows"], case["width"], DTYPES[case["dtype"]], DTYPES[case["out"]]
    # a residual stream with a few columns far above the others, and a block's output
    residual = torch.randn((n, width), generator=gd, device=dev)
    residual[:, torch.randperm(width, generator=g)[:3].to(dev)] *= 20.0
    x = torch.randn((n, width), generator=gd, device=dev).mul_(0.5)
    gain = (1 + 0.2 * torch.randn((width,), generator=gd, device=dev)).to(dt)
    groups = width // case["group"] if case["group"] else 0
    return {"op": "norm", "x": x.to(dt), "residual": residual.to(dt), "gain": gain, "eps": 1e-6,
            "residual_out": torch.empty((n, width), dtype=dt, device=dev), "out": torch.empty((n, width), dtype=out, device=dev),
            "scales": torch.empty((n, groups), device=dev) if groups else None}


def _own_lengths(case, g=None):
    return _spread(case["lo"], case["hi"], case["batch"], g)


def _prepare_prefix(case, g, gd, dev):
    b, r, hq, hkv, d, page, prefix = (case[k] for k in ("batch", "rows", "hq", "hkv", "d", "page", "prefix"))
    dt, ct = DTYPES[case["dtype"]], DTYPES[case["cache"]]
    lens = _own_lengths(case, g)
    own_pages, prefix_pages = _pages(lens, page).to(torch.int64), _pages(prefix, page)
    n_pages = int(own_pages.sum()) + prefix_pages + 3
    ids = torch.randperm(n_pages, generator=g).to(torch.int32)
    at = torch.cumsum(own_pages, 0) - own_pages
    k = torch.arange(max(1, int(own_pages.max())))
    table = torch.where(k[None, :] < own_pages[:, None], ids[(at[:, None] + k[None, :]).clamp(max=n_pages - 1)],
                        torch.tensor(-1, dtype=torch.int32))
    # normalised queries and keys; a shared direction gives the scores the peaks that trained heads have
    q = torch.randn((b, r, hq, d), generator=gd, device=dev)
    common = torch.randn((d,), generator=gd, device=dev)
    q.add_(common, alpha=0.7)
    kv = []
    for add in (0.5, 0.0):
        x = torch.randn((n_pages, hkv, page, d), generator=gd, device=dev, dtype=torch.bfloat16)
        kv.append(x.add_(common.to(x.dtype), alpha=add))
    scales = None
    if case["cache"] == "e4m3":
        scales = 0.02 + 0.03 * torch.rand((2, hkv), generator=gd, device=dev)
        kv = [x.div_(s[None, :, None, None]) for x, s in zip(kv, scales)]
    return {"op": "prefix", "q": q.to(dt), "k_pages": kv[0].to(ct), "v_pages": kv[1].to(ct),
            "prefix_table": ids[n_pages - 3 - prefix_pages:n_pages - 3].to(dev),
            "prefix_len": torch.tensor([prefix], dtype=torch.int32, device=dev), "table": table.to(dev),
            "lens": lens.to(dev), "scale": d ** -0.5, "k_scale": None if scales is None else scales[0],
            "v_scale": None if scales is None else scales[1], "out": torch.empty((b, r, hq, d), dtype=dt, device=dev),
            "lse": torch.empty((b, r, hq), device=dev)}


def _prepare_drafts(case, g, gd, dev):
    b, r, vocab, dt = case["batch"], case["rows"], case["vocab"], DTYPES[case["dtype"]]
    logits = torch.randn((b, r, vocab), generator=gd, device=dev).mul_(3.0)
    f = lambda *shape: torch.rand(shape, generator=gd, device=dev)  # noqa: E731
    temperature = 0.6 + 0.6 * f(b)
    temperature[3::8] = 0.0  # some users ask for greedy decoding
    race = lambda *shape: torch.empty(shape, device=dev).exponential_(generator=gd)  # noqa: E731
    draft_logits = tokens = None
    if case["draft"]:
        draft_logits = (logits[:, :r - 1] + 0.8 * torch.randn((b, r - 1, vocab), generator=gd, device=dev)).to(dt)
        t = temperature.clamp(min=0.05)[:, None, None]
        chosen = (draft_logits.float() / t - race(b, r - 1, vocab).log_()).argmax(-1)
    else:  # drafts from elsewhere: likely tokens
        chosen = logits[:, :r - 1].argmax(-1)
    tokens = torch.cat([torch.randint(0, vocab, (b, 1), generator=gd, device=dev), chosen], 1).to(torch.int32)
    n_drafts = torch.full((b,), r - 1, dtype=torch.int32)
    n_drafts[4::5] //= 2  # some requests had fewer drafts
    return {"op": "drafts", "logits": logits.to(dt).view(b * r, vocab), "tokens": tokens,
            "draft_logits": None if draft_logits is None else draft_logits.view(-1, vocab),
            "n_drafts": n_drafts.to(dev), "temperature": temperature, "uniforms": f(b, r - 1), "noise": race(b, vocab),
            "positions": torch.randint(1, 9000, (b,), generator=g).to(torch.int32).to(dev),
            "accept_out": torch.empty((3, b), dtype=torch.int32, device=dev), "logprobs": torch.empty((b, r), device=dev)}


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(state):
    if own:
        return {"norm": _own_norm, "prefix": _own_prefix, "drafts": _own_drafts}[state["op"]](state)
    return {"norm": _plain_norm, "prefix": _plain_prefix, "drafts": _plain_drafts}[state["op"]](state)


def _own_norm(s):
    from decode_megakernel_04_gb300 import rms_norm
    rms_norm(s["x"], s["out"], gain=s["gain"], residual=s["residual"], residual_out=s["residual_out"], eps=s["eps"],
             scales=s["scales"])
    return {"out": s["out"], "residual_out": s["residual_out"], "scales": s["scales"]}


def _plain_norm(s):
    h = s["x"].float() + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + s["eps"]) * s["gain"].float()
    scales = None
    if s["scales"] is not None:
        n, groups = s["scales"].shape
        y = y.view(n, groups, -1)
        scales = y.abs().amax(-1) / 448.0
        y = torch.where(scales[..., None] > 0, y / scales[..., None], 0.0).clamp(-448.0, 448.0).view(n, -1)
    return {"out": y.to(s["out"].dtype), "residual_out": h.to(s["x"].dtype), "scales": scales}


def _own_prefix(s):
    from decode_megakernel_04_gb300 import prefix_attention
    prefix_attention(s["q"], s["k_pages"], s["v_pages"], s["prefix_table"], s["prefix_len"], s["table"], s["lens"], s["out"],
                     scale=s["scale"], lse=s["lse"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_gather(pages, table, scale):
    """[rows of the table, kv heads, table width x page, width] in 32 bits."""
    b, n = table.shape
    x = pages[table.long().clamp(min=0)].float()
    if scale is not None:
        x = x * scale[:, None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(b, pages.shape[1], n * pages.shape[2], pages.shape[3])


def _plain_prefix(s):
    q, lens = s["q"], s["lens"]
    b, r, hq, d = q.shape
    hkv = s["k_pages"].shape[1]
    g = hq // hkv
    qf = q.float().view(b, r, hkv, g, d).mul(s["scale"])
    # the prefix once for all rows of a kv head; [hkv, b r g, keys]
    table = s["prefix_table"][None]
    k = _plain_gather(s["k_pages"], table, s["k_scale"])[0]
    shared = torch.matmul(qf.permute(2, 0, 1, 3, 4).reshape(hkv, -1, d), k.transpose(-1, -2))
    shared.masked_fill_(torch.arange(k.shape[1], device=q.device) >= s["prefix_len"], -math.inf)
    top_shared = shared.amax(-1).view(hkv, b, r, g).permute(1, 0, 2, 3)
    # each request's own keys; [b, hkv, r, g, keys]
    k = _plain_gather(s["k_pages"], s["table"], s["k_scale"])
    score = torch.matmul(qf.transpose(1, 2).reshape(b, hkv, -1, d), k.transpose(-1, -2)).view(b, hkv, r, g, -1)
    del k
    seen = lens[:, None] - (r - 1 - torch.arange(r, device=q.device))
    hidden = torch.arange(score.shape[-1], device=q.device) >= seen[..., None]
    score.masked_fill_(hidden[:, None, :, None], -math.inf)
    top = torch.maximum(top_shared, score.amax(-1)).clamp(min=-1e30)
    shared.sub_(top.permute(1, 0, 2, 3).reshape(hkv, -1, 1)).exp_()
    score.sub_(top[..., None]).exp_()
    total = shared.sum(-1).view(hkv, b, r, g).permute(1, 0, 2, 3) + score.sum(-1)
    v = _plain_gather(s["v_pages"], table, s["v_scale"])[0]
    o = torch.matmul(shared, v).view(hkv, b, r, g, d).permute(1, 0, 2, 3, 4)
    v = _plain_gather(s["v_pages"], s["table"], s["v_scale"])
    o = o + torch.matmul(score.view(b, hkv, r * g, -1), v).view(b, hkv, r, g, d)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    lse = torch.where(total > 0, top + total.log(), -math.inf)
    return {"out": o.transpose(1, 2).reshape(b, r, hq, d).to(q.dtype), "lse": lse.transpose(1, 2).reshape(b, r, hq)}


def _own_drafts(s):
    from decode_megakernel_04_gb300 import verify_drafts
    verify_drafts(s["logits"], s["tokens"], s["noise"], s["uniforms"], s["accept_out"], draft_logits=s["draft_logits"],
                  n_drafts=s["n_drafts"], temperature=s["temperature"], positions=s["positions"], logprobs=s["logprobs"])
    return {"accept_out": s["accept_out"], "logprobs": s["logprobs"]}


def _plain_probabilities(logits, b, temperature):
    """softmax(logits / temperature) in 64 bits, one for the first largest token where the temperature is 0; [b, rows, vocab]."""
    z = logits.view(b, -1, logits.shape[-1]).double()
    t = temperature.double()[:, None, None]
    top, at = z.max(-1, keepdim=True)
    w = z.sub_(top).div_(torch.where(t > 0, t, 1.0)).exp_()
    w = w.div_(w.sum(-1, keepdim=True))
    first = torch.arange(w.shape[-1], device=w.device) == at
    return torch.where(t > 0, w, first.to(w.dtype))


def _plain_drafts(s):
    tokens, n_drafts = s["tokens"].long(), s["n_drafts"].long()
    b, r = tokens.shape
    dev = tokens.device
    p = _plain_probabilities(s["logits"], b, s["temperature"])
    vocab = p.shape[-1]
    places = torch.arange(r, device=dev)
    q = None if s["draft_logits"] is None else _plain_probabilities(s["draft_logits"], b, s["temperature"])
    drafted = tokens[:, 1:, None]
    px = p[:, :r - 1].gather(-1, drafted)[..., 0]
    qx = torch.ones_like(px) if q is None else q.gather(-1, drafted)[..., 0]
    good = (s["uniforms"].double() * qx < px) & (places[:r - 1] < n_drafts[:, None])
    a = good.long().cumprod(-1).sum(-1)
    row = p.gather(1, a[:, None, None].expand(b, 1, vocab))[:, 0]
    if r > 1:
        at = a.clamp(max=r - 2)
        x = tokens.gather(1, at[:, None] + 1)
        other = torch.zeros_like(row).scatter_(1, x, 1.0) if q is None else q.gather(1, at[:, None, None].expand(b, 1, vocab))[:, 0]
        rest = (row - other).clamp(min=0.0)
        rest = torch.where((rest.sum(-1, keepdim=True) > 0) & (a < n_drafts)[:, None], rest, row)
    else:
        rest = row
    token = (rest / s["noise"].double()).argmax(-1)
    logprobs = torch.where(places[:r - 1] < a[:, None], px.log(), 0.0)
    logprobs = torch.cat([logprobs, torch.zeros_like(row[:, :1])], 1)
    logprobs = logprobs.scatter(1, a[:, None], row.gather(1, token[:, None]).log())
    return {"accept_out": torch.stack([a + 1, token, s["positions"].long() + a + 1]).to(torch.int32),
            "logprobs": logprobs.float()}


# ---- what a pass cannot do without ----------------------------------------------------------------------------------

def work(case):
    if case["op"] == "norm":
        n, width, size, to = case["rows"], case["width"], SIZES[case["dtype"]], SIZES[case["out"]]
        groups = width // case["group"] if case["group"] else 0
        return {"bytes": n * (width * (3 * size + to) + 4 * groups) + width * size, "flops": 6 * n * width}
    if case["op"] == "prefix":
        b, r, hq, hkv, d = (case[k] for k in ("batch", "rows", "hq", "hkv", "d"))
        mine, prefix = int(_own_lengths(case).sum()), case["prefix"]
        return {"bytes": 2 * (prefix + mine) * hkv * d * SIZES[case["cache"]] + b * r * hq * (4 * d + 4) +
                4 * (mine + prefix) // case["page"], "flops": 4 * (mine + prefix * b) * r * hq * d}
    b, r, vocab = case["batch"], case["rows"], case["vocab"]
    rows = r + (r - 1 if case["draft"] else 0)
    return {"bytes": b * vocab * (rows * SIZES[case["dtype"]] + 4) + b * r * 12, "flops": 4 * b * (rows + 1) * vocab}


# ---- the definitions in 64 bits, for measuring errors ---------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "prefix": _exact_prefix, "drafts": _exact_drafts}[s["op"]](s)


def _exact_norm(s):
    h = s["x"].double() + s["residual"].double()
    width = h.shape[-1]
    y = h / (h.pow(2).sum(-1, keepdim=True) / width + s["eps"]).sqrt() * s["gain"].double()
    if s["scales"] is None:
        return {"out": y, "residual_out": h, "scales": None}
    n, groups = s["scales"].shape
    blocks = y.reshape(n, groups, width // groups)
    scales = blocks.abs().max(-1).values / 448
    return {"out": (blocks / scales[:, :, None].clip(min=1e-300)).reshape(n, width), "residual_out": h, "scales": scales}


def _exact_prefix(s):
    q = s["q"].double()
    b, r, hq, d = q.shape
    hkv, page = s["k_pages"].shape[1:3]

    def cached(pages, table, n, scale):
        x = pages[table[:-(-n // page)].long()].transpose(0, 1).reshape(hkv, -1, d)[:, :n].double()
        return x if scale is None else x * scale.double()[:, None, None]

    n0 = int(s["prefix_len"])
    k0, v0 = (cached(s[x + "_pages"], s["prefix_table"], n0, s[x + "_scale"]) for x in "kv")
    out, lse = torch.zeros_like(q), torch.full((b, r, hq), -math.inf, dtype=torch.float64, device=q.device)
    for i, n in enumerate(s["lens"].tolist()):
        k, v = (torch.cat([x0, cached(s[x + "_pages"], s["table"][i], n, s[x + "_scale"])], 1) for x, x0 in (("k", k0), ("v", v0)))
        for j in range(r):
            m = n0 + max(0, n - (r - 1 - j))
            if m == 0:
                continue
            z = torch.einsum("hgd,hnd->hgn", q[i, j].view(hkv, -1, d), k[:, :m]) * s["scale"]
            lse[i, j] = torch.logsumexp(z, -1).reshape(-1)
            out[i, j] = torch.einsum("hgn,hnd->hgd", torch.softmax(z, -1), v[:, :m]).reshape(hq, d)
    return {"out": out, "lse": lse}


def _exact_drafts(s):
    b, r = s["tokens"].shape
    logits = s["logits"].view(b, r, -1)
    draft = None if s["draft_logits"] is None else s["draft_logits"].view(b, r - 1, -1)
    tokens, uniforms, count = s["tokens"].tolist(), s["uniforms"].tolist(), s["n_drafts"].tolist()
    accept, logprobs = np.zeros((3, b), np.int32), np.zeros((b, r))

    def log_p(z, t):
        z = z.double()
        if t > 0:
            return torch.log_softmax(z / t, -1)
        y = torch.full_like(z, -math.inf)
        y[int((z == z.max()).nonzero()[0])] = 0.0
        return y

    for i, t in enumerate(s["temperature"].tolist()):
        a = 0
        while True:
            p = log_p(logits[i, a], t)
            if a == count[i]:
                rest = p.exp()
                break
            x = tokens[i][a + 1]
            q = torch.zeros_like(p) if draft is None else log_p(draft[i, a], t).exp()
            if draft is None:
                q[x] = 1.0
            if uniforms[i][a] * float(q[x]) < math.exp(float(p[x])):
                logprobs[i, a] = float(p[x])
                a += 1
                continue
            rest = (p.exp() - q).clip(min=0)
            if not float(rest.sum()) > 0:
                rest = p.exp()
            break
        token = int((rest / s["noise"][i].double()).argmax())
        logprobs[i, a] = float(p[token])
        accept[:, i] = a + 1, token, int(s["positions"][i]) + a + 1
    return {"accept_out": accept, "logprobs": logprobs}
