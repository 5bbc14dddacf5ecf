"""The serving operators as they are measured: page tables, query / key norms with rotation and cache append,
attention over a paged cache, and logit controls. Each case is one pass through one operator, either in its plain
form (elementary torch operations) or, where ``own`` is true, through the package's entry points."""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def listed():
    return [
        # one user's next token at a 4096-token context: the bookkeeping of a single decode step
        {"name": "tables one token", "op": "tables", "batch": 1, "page": 64, "held_lo": 4096, "held_hi": 4096,
         "decode": 1, "chunk": 1, "max_pages": 128},
        # a full server's step: 200 decodes, 48 prompt chunks of 1 to 4096 tokens, 8 finished requests
        {"name": "tables mixed 256", "op": "tables", "batch": 256, "page": 16, "held_lo": 1, "held_hi": 8192,
         "decode": 200, "chunk": 4096, "max_pages": 1024},
        # one token of the 48 / 8 x 128 attention, one position of a bf16 cache written
        {"name": "norm rope one token", "op": "qk", "tokens": 1, "hq": 48, "hkv": 8, "d": 128, "rope": 128,
         "dtype": "bf16", "cache": "bf16", "page": 16, "far": 8192},
        # a 64-sequence 8-row verify block of the 24 / 4 x 256 attention into an e4m3 cache, quarter rotation
        {"name": "norm rope verify e4m3", "op": "qk", "tokens": 512, "hq": 24, "hkv": 4, "d": 256, "rope": 64,
         "dtype": "bf16", "cache": "e4m3", "page": 64, "far": 1000000},
        # a prompt chunk of 8190 tokens, far positions, fp16
        {"name": "norm rope prompt", "op": "qk", "tokens": 8190, "hq": 48, "hkv": 8, "d": 128, "rope": 128,
         "dtype": "f16", "cache": "f16", "page": 16, "far": 131072},
        # the headline decode: batch 1 at 4096 positions, 24 / 4 x 256
        {"name": "attend one 4096", "op": "attend", "batch": 1, "rows": 1, "hq": 24, "hkv": 4, "d": 256,
         "lo": 4096, "hi": 4096, "page": 64, "dtype": "bf16", "cache": "bf16"},
        # short ragged requests, an idle entry among them, fp16, 4 / 1 x 64
        {"name": "attend short ragged", "op": "attend", "batch": 129, "rows": 1, "hq": 4, "hkv": 1, "d": 64,
         "lo": 0, "hi": 700, "page": 16, "dtype": "f16", "cache": "f16"},
        # 8 sequences verify 8 rows each at 8192 positions, 48 / 8 x 128
        {"name": "attend verify 8192", "op": "attend", "batch": 8, "rows": 8, "hq": 48, "hkv": 8, "d": 128,
         "lo": 8192, "hi": 8192, "page": 16, "dtype": "bf16", "cache": "bf16"},
        # a full server: 64 requests between 1 and 16384 positions over an e4m3 cache
        {"name": "attend ragged e4m3", "op": "attend", "batch": 64, "rows": 1, "hq": 48, "hkv": 8, "d": 128,
         "lo": 1, "hi": 16384, "page": 32, "dtype": "bf16", "cache": "e4m3"},
        # one user's logits, 512 tokens of history, every control
        {"name": "logits one", "op": "logits", "rows": 1, "vocab": 151936, "history": 512, "biases": 16,
         "dtype": "f32", "mask": True},
        # 64 rows, long histories, grammar masks
        {"name": "logits 64", "op": "logits", "rows": 64, "vocab": 202048, "history": 8192, "biases": 300,
         "dtype": "f32", "mask": True},
        # a large batch of bf16 logits, penalties and biases only, an odd vocabulary
        {"name": "logits 256 bf16", "op": "logits", "rows": 256, "vocab": 163841, "history": 1500, "biases": 8,
         "dtype": "bf16", "mask": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "qk", "attend", "attend", "logits"])
    if op == "tables":
        batch = _log_int(rng, 1, 250)
        page = rng.choice([1, 8, 16, 24, 64, 128])
        hi = _log_int(rng, 1, 8000)
        chunk = _log_int(rng, 1, 4000)
        return {"op": op, "batch": batch, "page": page, "held_lo": rng.randint(0, hi), "held_hi": hi,
                "decode": rng.randint(int(0.8 * batch), batch), "chunk": chunk,
                "max_pages": -(-(hi + chunk) // page) + rng.randint(0, 9)}
    if op == "qk":
        hkv = rng.choice([1, 2, 4, 8])
        d = rng.choice([64, 128, 256])
        dtype = rng.choice(["bf16", "f16"])
        return {"op": op, "tokens": _log_int(rng, 1, 3000), "hq": hkv * rng.choice([1, 3, 4, 6]), "hkv": hkv, "d": d,
                "rope": rng.choice([d, d // 2, d // 4]), "dtype": dtype, "cache": rng.choice([dtype, "e4m3"]),
                "page": rng.choice([1, 16, 24, 64]), "far": _log_int(rng, 1000, 2000000)}
    if op == "attend":
        hkv = rng.choice([1, 2, 4, 8])
        d = rng.choice([64, 128, 256])
        hi = _log_int(rng, 1, 40000)
        rows, group = rng.choice([1, 1, 1, 2, 5, 8]), rng.choice([1, 4, 6, 7, 8, 12])
        # the cache read and the products over it are bounded: at most what the largest listed cases have
        most = max(1, int(2.5e8 // (hi * hkv * d * max(1.0, rows * group / 24))))
        dtype = rng.choice(["bf16", "f16"])
        return {"op": op, "batch": _log_int(rng, 1, min(200, most)), "rows": rows,
                "hq": hkv * group, "hkv": hkv, "d": d, "lo": rng.randint(0, hi), "hi": hi,
                "page": rng.choice([1, 16, 24, 32, 64, 256]), "dtype": dtype, "cache": rng.choice([dtype, "e4m3"])}
    return {"op": op, "rows": _log_int(rng, 1, 128), "vocab": _log_int(rng, 1000, 240000),
            "history": _log_int(rng, 1, 8000), "biases": _log_int(rng, 1, 300),
            "dtype": rng.choice(["f32", "bf16", "f16"]), "mask": rng.random() < 0.7}


# ---- inputs -----------------------------------------------------------------------------------------------------

def _spread(lo, hi, n, g=None):
    """n whole numbers evenly spaced over [lo, hi] (their sum does not depend on the seed), in an order that does."""
    v = torch.tensor([lo + (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)], dtype=torch.int32)
    return v if g is None else v[torch.randperm(n, generator=g)]


def _table_lengths(case, g=None):
    """(held, start, count): decodes that drop up to 3 rejected tokens, prompt chunks, and finished requests."""
    n, dec = case["batch"], case["decode"]
    chunks = (n - dec) * 6 // 7
    held = _spread(case["held_lo"], case["held_hi"], n, g)
    drop = torch.tensor([i % 4 for i in range(n)], dtype=torch.int32) if n > 1 else torch.zeros(1, dtype=torch.int32)
    start = torch.clamp(held - drop, min=0)
    count = torch.ones(n, dtype=torch.int32)
    if chunks:
        start[dec:dec + chunks] = held[dec:dec + chunks]
        count[dec:dec + chunks] = _spread(1, case["chunk"], chunks, g)
    start[dec + chunks:] = 0
    count[dec + chunks:] = 0
    most = case["max_pages"] * case["page"]
    count = torch.minimum(count, most - start)
    return held, start, count


def _pages(tokens, page):
    return torch.div(tokens + page - 1, page, rounding_mode="floor")


def _attend_lengths(case, g=None):
    return _spread(case["lo"], case["hi"], case["batch"], g)


def prepare(case, seed):
    g = torch.Generator()
    g.manual_seed(int(seed))
    dev = torch.device("cuda")
    gd = torch.Generator(device=dev)
    gd.manual_seed(int(seed) + 1)
    return {"tables": _prepare_tables, "qk": _prepare_qk, "attend": _prepare_attend,
            "logits": _prepare_logits}[case["op"]](case, g, gd, dev)


def _prepare_tables(case, g, gd, dev):
    held, start, count = _table_lengths(case, g)
    n, page, max_pages = case["batch"], case["page"], case["max_pages"]
    hp = _pages(held, page).to(torch.int64)
    used = int(hp.sum())
    n_pages = used + int(_pages(count, page).sum()) + n + 5
    ids = torch.randperm(n_pages, generator=g).to(torch.int32)
    at = torch.cumsum(hp, 0) - hp
    k = torch.arange(max_pages)
    mine = k[None, :] < hp[:, None]
    table = torch.where(mine, ids[(at[:, None] + k[None, :]).clamp(max=n_pages - 1)], torch.tensor(-1, dtype=torch.int32))
    head = int(torch.randint(0, n_pages, (1,), generator=g))
    free = n_pages - used
    ring = torch.full((n_pages,), -1, dtype=torch.int32)
    ring[(head + torch.arange(free)) % n_pages] = ids[used:]
    cap = int(count.sum()) + n % 3  # a padded tail on some batches
    i32 = dict(dtype=torch.int32, device=dev)
    return {"op": "tables", "page": page, "n_pages": n_pages, "held": held.to(dev), "start": start.to(dev),
            "count": count.to(dev), "table": table.to(dev), "ring": ring.to(dev),
            "ring_state": torch.tensor([head, free], **i32), "ring_state_out": torch.zeros(2, **i32),
            "slots": torch.empty(cap, dtype=torch.int64, device=dev), "positions": torch.empty(cap, **i32),
            "owners": torch.empty(cap, **i32), "starts": torch.empty(n + 1, **i32), "lens": torch.empty(n, **i32),
            "status": torch.zeros(1, **i32)}


def _prepare_qk(case, g, gd, dev):
    n, hq, hkv, d, page = case["tokens"], case["hq"], case["hkv"], case["d"], case["page"]
    dt, ct = DTYPES[case["dtype"]], DTYPES[case["cache"]]
    # q, k and v side by side, as a fused projection writes them
    qkv = torch.randn((n, hq + 2 * hkv, d), generator=gd, device=dev).mul_(1.5).to(dt)
    gains = (1 + 0.2 * torch.randn((2, d), generator=gd, device=dev)).to(dt)
    pos = torch.randint(0, case["far"], (n,), generator=g).to(torch.int32)
    n_pages = -(-n // page) + 2
    slots = torch.randperm(n_pages * page, generator=g)[:n]
    slots[n - n // 16:] = -1  # the padded tail of a batch is not stored
    pages = torch.zeros((2, n_pages, hkv, page, d), device=dev).to(ct)
    scales = 0.02 + 0.03 * torch.rand((2, hkv), generator=gd, device=dev) if case["cache"] == "e4m3" else None
    inv = 10000.0 ** (-torch.arange(0, case["rope"], 2, dtype=torch.float64) / case["rope"])
    return {"op": "qk", "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:], "q_gain": gains[0],
            "k_gain": gains[1], "eps": 1e-6, "inv_freq": inv.to(dev), "positions": pos.to(dev), "slots": slots.to(dev),
            "k_pages": pages[0], "v_pages": pages[1], "k_scale": None if scales is None else scales[0],
            "v_scale": None if scales is None else scales[1], "q_out": torch.empty((n, hq, d), dtype=dt, device=dev)}


def _prepare_attend(case, g, gd, dev):
    b, r, hq, hkv, d, page = (case[k] for k in ("batch", "rows", "hq", "hkv", "d", "page"))
    dt, ct = DTYPES[case["dtype"]], DTYPES[case["cache"]]
    lens = _attend_lengths(case, g)
    np_ = _pages(lens, page).to(torch.int64)
    n_pages = int(np_.sum()) + 3
    ids = torch.randperm(n_pages, generator=g).to(torch.int32)
    at = torch.cumsum(np_, 0) - np_
    k = torch.arange(max(1, int(np_.max())))
    table = torch.where(k[None, :] < np_[:, None], ids[(at[:, None] + k[None, :]).clamp(max=n_pages - 1)],
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
    return {"op": "attend", "q": q.to(dt), "k_pages": kv[0].to(ct), "v_pages": kv[1].to(ct), "table": table.to(dev),
            "lens": lens.to(dev), "scale": d ** -0.5, "k_scale": None if scales is None else scales[0],
            "v_scale": None if scales is None else scales[1], "out": torch.empty((b, r, hq, d), dtype=dt, device=dev),
            "lse": torch.empty((b, r, hq), device=dev)}


def _prepare_logits(case, g, gd, dev):
    n, vocab, hist, nb = case["rows"], case["vocab"], case["history"], case["biases"]
    logits = torch.randn((n, vocab), generator=gd, device=dev).mul_(3.0).to(DTYPES[case["dtype"]])
    # a text repeats itself: ids crowd towards the low end
    u = torch.rand((n, hist), generator=gd, device=dev)
    history = (u.pow(3) * vocab).to(torch.int32).clamp_(max=vocab - 1)
    total = _spread(max(1, hist // 2), hist, n, g)
    prompt = total // 3
    f = lambda lo, hi: lo + (hi - lo) * torch.rand((n,), generator=gd, device=dev)  # noqa: E731
    ids = torch.randint(0, vocab, (n, nb), generator=gd, device=dev).to(torch.int32)
    ids[:, nb - nb // 4:] = -1  # rows list different numbers of biases
    vals = 4 * torch.randn((n, nb), generator=gd, device=dev)
    allowed = None
    if case["mask"]:
        words = -(-vocab // 32)
        a = torch.randint(0, 1 << 32, (n, words), generator=gd, device=dev)
        b = torch.randint(0, 1 << 32, (n, words), generator=gd, device=dev)
        allowed = (a & b).to(torch.int64)
        allowed = torch.where(allowed >= 1 << 31, allowed - (1 << 32), allowed).to(torch.int32)
    return {"op": "logits", "logits": logits, "history": history, "prompt": prompt.to(dev), "total": total.to(dev),
            "repetition": f(1.0, 1.5), "presence": f(0.0, 1.0), "frequency": f(0.0, 0.5), "bias_ids": ids,
            "bias_vals": vals, "allowed": allowed, "out": torch.empty((n, vocab), device=dev),
            "token": torch.empty((n,), dtype=torch.int32, device=dev)}


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(state):
    if own:
        return {"tables": _own_tables, "qk": _own_qk, "attend": _own_attend, "logits": _own_logits}[state["op"]](state)
    return {"tables": _plain_tables, "qk": _plain_qk, "attend": _plain_attend, "logits": _plain_logits}[state["op"]](state)


def _own_tables(s):
    from decode_megakernel_04_gb300 import page_tables
    page_tables(s["table"], s["held"], s["start"], s["count"], s["ring"], s["ring_state"], s["page"], s["n_pages"],
                slots=s["slots"], positions=s["positions"], owners=s["owners"], starts=s["starts"], lens=s["lens"],
                ring_state_out=s["ring_state_out"], status=s["status"])
    return {k: s[k] for k in ("table", "ring", "ring_state_out", "slots", "positions", "owners", "starts", "lens", "status")}


def _plain_tables(s):
    page, table, ring = s["page"], s["table"], s["ring"]
    cap_ring, cap = ring.numel(), s["slots"].numel()
    n, max_pages = table.shape
    dev = table.device
    held, start, count = s["held"].long(), s["start"].long(), s["count"].long()
    lens = start + count
    have, need = (held + page - 1) // page, (lens + page - 1) // page
    grow, shrink = (need - have).clamp(min=0), (have - need).clamp(min=0)
    starts = torch.cat([count.new_zeros(1), torch.cumsum(count, 0)])
    pop_at, push_at = torch.cumsum(grow, 0) - grow, torch.cumsum(shrink, 0) - shrink
    head, free = s["ring_state"].long().unbind()
    k = torch.arange(max_pages, device=dev)
    popped = ring[(head + pop_at[:, None] + k - have[:, None]) % cap_ring]
    fresh = (k >= have[:, None]) & (k < need[:, None])
    gone = (k >= need[:, None]) & (k < have[:, None])
    to = torch.where(gone, (head + free + push_at[:, None] + k - need[:, None]) % cap_ring, cap_ring)
    ring_out = torch.cat([ring, ring.new_zeros(1)]).scatter(0, to.reshape(-1), table.reshape(-1))[:cap_ring]
    table_out = torch.where(fresh, popped, table)
    state = torch.stack([(head + grow.sum()) % cap_ring, free - grow.sum() + shrink.sum()])
    t = torch.arange(cap, device=dev)
    owner = torch.searchsorted(starts, t, right=True) - 1
    real = t < starts[-1]
    b = owner.clamp(max=n - 1)
    pos = start[b] + t - starts[b]
    slot = table_out[b, (pos // page).clamp(0, max_pages - 1)].long() * page + pos % page
    i32 = torch.int32
    return {"table": table_out, "ring": ring_out, "ring_state_out": state.to(i32),
            "slots": torch.where(real, slot, -1), "positions": torch.where(real, pos, 0).to(i32),
            "owners": torch.where(real, b, -1).to(i32), "starts": starts.to(i32), "lens": lens.to(i32),
            "status": torch.zeros_like(s["status"])}


def _own_qk(s):
    from decode_megakernel_04_gb300 import qk_norm_rope
    qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_out"], v=s["v"], q_gain=s["q_gain"],
                 k_gain=s["k_gain"], eps=s["eps"], k_pages=s["k_pages"], v_pages=s["v_pages"], slots=s["slots"],
                 k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {k: s[k] for k in ("q_out", "k_pages", "v_pages")}


def _plain_norm_rope(x, gain, eps, cos, sin):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * gain.float()
    h = cos.shape[-1]
    a, b = y[..., :h], y[..., h:2 * h]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., 2 * h:]], -1)


def _plain_store(pages, slots, x, scale):
    """Rows of `x` with a slot >= 0 go to their slots; the others fall on a spare row that is cut off."""
    n_pages, hkv, page, d = pages.shape
    if scale is not None:
        x = (x / scale[None, :, None]).clamp(-448.0, 448.0)
    to = torch.where(slots >= 0, slots, n_pages * page)
    flat = torch.empty((n_pages * page + 1, hkv, d), device=x.device)
    flat[:-1] = pages.float().transpose(1, 2).reshape(-1, hkv, d)
    flat[to] = x
    return flat[:-1].view(n_pages, page, hkv, d).transpose(1, 2).to(pages.dtype).contiguous()


def _plain_qk(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _plain_norm_rope(s["q"], s["q_gain"], s["eps"], cos, sin)
    k = _plain_norm_rope(s["k"], s["k_gain"], s["eps"], cos, sin)
    return {"q_out": q.to(s["q"].dtype), "k_pages": _plain_store(s["k_pages"], s["slots"], k, s["k_scale"]),
            "v_pages": _plain_store(s["v_pages"], s["slots"], s["v"].float(), s["v_scale"])}


def _own_attend(s):
    from decode_megakernel_04_gb300 import paged_attention
    paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["out"], scale=s["scale"],
                    lse=s["lse"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_gather(pages, table, scale):
    """[batch, kv heads, table width x page, width] in 32 bits."""
    b, n = table.shape
    x = pages[table.long().clamp(min=0)].float()
    if scale is not None:
        x = x * scale[:, None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(b, pages.shape[1], n * pages.shape[2], pages.shape[3])


def _plain_attend(s):
    q, lens = s["q"], s["lens"]
    b, r, hq, d = q.shape
    hkv = s["k_pages"].shape[1]
    k = _plain_gather(s["k_pages"], s["table"], s["k_scale"])
    qg = q.float().view(b, r, hkv, hq // hkv, d).transpose(1, 2).reshape(b, hkv, -1, d)
    score = (torch.matmul(qg, k.transpose(-1, -2)) * s["scale"]).view(b, hkv, r, hq // hkv, -1)
    del k
    seen = lens[:, None] - (r - 1 - torch.arange(r, device=q.device))
    hidden = torch.arange(score.shape[-1], device=q.device) >= seen[..., None]
    score.masked_fill_(hidden[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = _plain_gather(s["v_pages"], s["table"], s["v_scale"])
    o = torch.matmul(p.view(b, hkv, -1, p.shape[-1]), v).view(b, hkv, r, hq // hkv, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = torch.where(total > 0, top + total.log(), -math.inf)[..., 0]
    return {"out": o.transpose(1, 2).reshape(b, r, hq, d).to(q.dtype), "lse": lse.transpose(1, 2).reshape(b, r, hq)}


def _own_logits(s):
    from decode_megakernel_04_gb300 import logit_controls
    logit_controls(s["logits"], s["out"], history=s["history"], prompt_len=s["prompt"], total_len=s["total"],
                   repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"], bias_ids=s["bias_ids"],
                   bias_vals=s["bias_vals"], allowed=s["allowed"], token=s["token"])
    return {"out": s["out"], "token": s["token"]}


def _plain_logits(s):
    z = s["logits"].float()
    n, vocab = z.shape
    dev = z.device
    history, at = s["history"].long(), torch.arange(s["history"].shape[1], device=dev)
    valid = (at < s["total"][:, None]) & (history >= 0) & (history < vocab)
    said = valid & (at >= s["prompt"][:, None])
    bucket = lambda ok: torch.where(ok, history, vocab)  # noqa: E731
    spare = z.new_zeros((n, vocab + 1))
    seen = spare.scatter(1, bucket(valid), 1.0)[:, :vocab] > 0
    count = spare.scatter_add(1, bucket(said), torch.ones_like(history, dtype=torch.float32))[:, :vocab]
    rep = s["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = torch.where(count > 0, z - s["frequency"][:, None] * count, z)
    z = torch.where(count > 0, z - s["presence"][:, None], z)
    ids = s["bias_ids"].long()
    listed_ = torch.where((ids >= 0) & (ids < vocab), ids, vocab)
    entry = torch.arange(ids.shape[1], device=dev).expand_as(ids)
    last = torch.full((n, vocab + 1), -1, device=dev, dtype=torch.int64)
    last = last.scatter_reduce(1, listed_, entry, "amax")[:, :vocab]
    z = torch.where(last >= 0, z + s["bias_vals"].gather(1, last.clamp(min=0)), z)
    if s["allowed"] is not None:
        v = torch.arange(vocab, device=dev)
        z = torch.where((s["allowed"][:, v >> 5] >> (v & 31)) & 1 == 1, z, -math.inf)
    rank = torch.where(torch.isnan(z), -math.inf, z)
    top = rank.amax(-1, keepdim=True)
    first = torch.where((rank == top) & (top > -math.inf), torch.arange(vocab, device=dev), vocab).amin(-1)
    return {"out": z, "token": torch.where(first < vocab, first, -1).to(torch.int32)}


# ---- what a pass cannot do without ----------------------------------------------------------------------------------

def work(case):
    if case["op"] == "tables":
        held, start, count = _table_lengths(case)
        n, page, tokens = case["batch"], case["page"], int(count.sum())
        have, need = _pages(held, page), _pages(start + count, page)
        fresh, gone = int((need - have).clamp(min=0).sum()), int((have - need).clamp(min=0).sum())
        touched = int((need - torch.div(start, page, rounding_mode="floor"))[count > 0].sum())
        # lengths in; popped, pushed and looked-up page ids; a slot, a position and an owner for each token
        return {"bytes": 20 * n + 8 * fresh + 8 * gone + 4 * touched + 16 * tokens, "flops": 4 * tokens}
    if case["op"] == "qk":
        n, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        cache = 1 if case["cache"] == "e4m3" else 2
        return {"bytes": n * (4 * hq * d + 2 * hkv * d * (2 + cache) + 12), "flops": 8 * n * (hq + hkv) * d}
    if case["op"] == "attend":
        b, r, hq, hkv, d = (case[k] for k in ("batch", "rows", "hq", "hkv", "d"))
        total = int(_attend_lengths(case).sum())
        cache = 1 if case["cache"] == "e4m3" else 2
        return {"bytes": 2 * total * hkv * d * cache + b * r * hq * (4 * d + 4) + 4 * total // case["page"],
                "flops": 4 * total * r * hq * d}
    n, vocab = case["rows"], case["vocab"]
    size = 4 if case["dtype"] == "f32" else 2
    tokens = int(_spread(max(1, case["history"] // 2), case["history"], n).sum())
    return {"bytes": n * (vocab * (size + 4) + (vocab // 8 if case["mask"] else 0) + 8 * case["biases"]) + 4 * tokens,
            "flops": 2 * n * vocab + 4 * tokens}


# ---- the definitions in 64 bits, for measuring errors ---------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "qk": _exact_qk, "attend": _exact_attend, "logits": _exact_logits}[s["op"]](s)


def _exact_tables(s):
    page, cap = s["page"], s["slots"].numel()
    held, start, count = (s[k].tolist() for k in ("held", "start", "count"))
    table, ring = s["table"].cpu().numpy().copy(), s["ring"].cpu().numpy().copy()
    head, free = s["ring_state"].tolist()
    tail, size = head + free, ring.size
    pops = pushes = 0
    slots, positions, owners = np.full(cap, -1, np.int64), np.zeros(cap, np.int32), np.full(cap, -1, np.int32)
    starts = [0]
    for b, (h, s0, c) in enumerate(zip(held, start, count)):
        have, need = -(-h // page), -(-(s0 + c) // page)
        for k in range(have, need):
            table[b, k] = ring[(head + pops) % size]
            pops += 1
        for k in range(need, have):
            ring[(tail + pushes) % size] = table[b, k]
            pushes += 1
        p = np.arange(s0, s0 + c)
        at = slice(starts[-1], starts[-1] + c)
        slots[at] = table[b, p // page].astype(np.int64) * page + p % page
        positions[at], owners[at] = p, b
        starts.append(starts[-1] + c)
    i = lambda v: np.array(v, np.int32)  # noqa: E731
    return {"table": table, "ring": ring, "ring_state_out": i([(head + pops) % size, free - pops + pushes]),
            "slots": slots, "positions": positions, "owners": owners, "starts": i(starts),
            "lens": i([a + c for a, c in zip(start, count)]), "status": i([0])}


def _exact_qk(s):
    phase = torch.polar(torch.ones((), dtype=torch.float64, device=s["q"].device),
                        s["positions"].double().outer(s["inv_freq"]))[:, None]
    half = phase.shape[-1]

    def turned(x, gain):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt() * gain.double()
        z = torch.complex(x[..., :half], x[..., half:2 * half]) * phase
        return torch.cat([z.real, z.imag, x[..., 2 * half:]], -1)

    def stored(pages, x, scale):
        p = pages.double()
        if scale is not None:
            x = (x / scale.double()[:, None]).clip(-448, 448)
        keep = s["slots"] >= 0
        at = s["slots"][keep]
        p[at // p.shape[2], :, at % p.shape[2]] = x[keep]
        return p

    return {"q_out": turned(s["q"], s["q_gain"]),
            "k_pages": stored(s["k_pages"], turned(s["k"], s["k_gain"]), s["k_scale"]),
            "v_pages": stored(s["v_pages"], s["v"].double(), s["v_scale"])}


def _exact_attend(s):
    q = s["q"].double()
    b, r, hq, d = q.shape
    hkv, page = s["k_pages"].shape[1:3]
    out, lse = torch.zeros_like(q), torch.full((b, r, hq), -math.inf, dtype=torch.float64, device=q.device)
    for i, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        ids = s["table"][i, :-(-n // page)].long()
        k, v = (x[ids].transpose(0, 1).reshape(hkv, -1, d)[:, :n].double() for x in (s["k_pages"], s["v_pages"]))
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"].double()[:, None, None], v * s["v_scale"].double()[:, None, None]
        for j in range(r):
            m = n - (r - 1 - j)
            if m <= 0:
                continue
            z = torch.einsum("hgd,hnd->hgn", q[i, j].view(hkv, -1, d), k[:, :m]) * s["scale"]
            lse[i, j] = torch.logsumexp(z, -1).reshape(-1)
            out[i, j] = torch.einsum("hgn,hnd->hgd", torch.softmax(z, -1), v[:, :m]).reshape(hq, d)
    return {"out": out, "lse": lse}


def _exact_logits(s):
    z = s["logits"].double()
    n, vocab = z.shape
    history, prompt, total = s["history"].cpu().numpy(), s["prompt"].tolist(), s["total"].tolist()
    ids, vals = s["bias_ids"].cpu().numpy(), s["bias_vals"].double().cpu().numpy()
    token = []
    for i in range(n):
        seen = torch.from_numpy(np.unique(history[i, :total[i]])).long().to(z.device)
        x = z[i, seen]
        rep = s["repetition"][i].double()
        z[i, seen] = torch.where(x > 0, x / rep, x * rep)
        said, times = (torch.from_numpy(t.astype(np.int64)).to(z.device)
                       for t in np.unique(history[i, prompt[i]:total[i]], return_counts=True))
        z[i, said] -= s["frequency"][i].double() * times + s["presence"][i].double()
        chosen = {int(t): v for t, v in zip(ids[i], vals[i]) if 0 <= t < vocab}
        at = torch.tensor(list(chosen), dtype=torch.int64, device=z.device)
        z[i, at] += torch.tensor(list(chosen.values()), dtype=torch.float64, device=z.device)
    if s["allowed"] is not None:
        bits = np.unpackbits(s["allowed"].cpu().numpy().view(np.uint8), axis=-1, bitorder="little")[:, :vocab]
        z[torch.from_numpy(bits == 0).to(z.device)] = -math.inf
    for row in z.unbind():
        top = row.max()
        token.append(int((row == top).nonzero()[0]) if top > -math.inf else -1)
    return {"out": z, "token": np.array(token, np.int32)}
