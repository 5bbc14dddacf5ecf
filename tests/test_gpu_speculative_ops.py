"""GPU: RMS norm, attention over a shared prefix and verification of drafts against plain implementations in 64 bits.

Tolerances are derived, not fitted (see test_gpu_serving_ops.py): a value that is rounded once to type t is off by at most half
a step; what the kernels compute in fp32 before that is bounded from the number and size of its terms, at each check."""
import math
import threading

import numpy as np
import pytest
import torch

from test_gpu_serving_ops import BF16, DEV, E4M3, F16, F32, attention_inputs, check_rounded, gen, half_step, i32, qk_slack, rotate, stepless

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from decode_megakernel_04_gb300 import _build
    _build.build()


def rounded(got, want, dtype, what, slack):
    if dtype is F32:
        bound = slack + (want.abs() + slack) * 2.0 ** -24 + 2.0 ** -150
        worst = ((got.double() - want).abs() / bound).max().item() if got.numel() else 0.0
        assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"
    else:
        check_rounded(got, want, dtype, what, slack)


# ---- RMS norm ---------------------------------------------------------------------------------------------------------

def norm_inputs(rows, width, dtype, seed=0, pad=0):
    g = gen(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    x, r = ((rn(rows, width + pad) * s).to(dtype)[:, :width] for s in (0.7, 3.0))
    return x, r, (1 + 0.3 * rn(width)).to(dtype)


def check_norm(x, r, gain, eps, out, h_out, scales):
    """The sum h is one fp32 rounding (2^-24) off before its own. The mean square: products 2^-24, at most 64 sums in a
    thread and 12 across the block, 2^-24 each, the division: relative 80 2^-24, half of it in the root; rsqrt 2 units, two
    products: y is off by less than 2^-18 of itself (with h's part). A scale is a largest y and a division."""
    h = x.double() if r is None else x.double() + r.double()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    if gain is not None:
        y = y * gain.double()
    if h_out is not None:
        rounded(h_out, h, x.dtype, "residual_out", h.abs() * 2.0 ** -24)
    if scales is None:
        rounded(out, y, x.dtype, "out", y.abs() * 2.0 ** -18)
        return
    n, groups = scales.shape
    width = y.shape[1]
    top = y.view(n, groups, width // groups).abs().amax(-1)
    assert ((scales.double() - top / 448).abs() <= top / 448 * 2.0 ** -17 + 2.0 ** -149).all()
    s = scales.double().repeat_interleave(width // groups, 1)
    want = torch.where(s > 0, y / s.clamp(min=2.0 ** -149), 0.0)
    check_rounded(out.float(), want.clamp(-448, 448), E4M3, "codes", want.abs() * 2.0 ** -17)


CASES_NORM = [  # rows, width, dtype, group (0: no codes), padding of a row
    (1, 8, BF16, 0, 0), (1, 8, F32, 8, 0), (3, 16, F16, 16, 8), (1, 5120, BF16, 0, 0), (2, 264, F16, 264, 0), (5, 256, BF16, 256, 8),
    (17, 7168, BF16, 128, 0), (7, 6144, F16, 6144, 16), (33, 5120, F32, 0, 8), (4, 1000, F32, 1000, 0), (3, 2048, F32, 32, 0),
    (2, 8192, BF16, 64, 0), (2, 8200, F16, 0, 0), (3, 16384, BF16, 128, 0), (2, 16392, BF16, 16392, 8), (2, 32768, F32, 256, 0),
    (2, 32760, F16, 0, 0), (1, 32768, BF16, 32768, 0), (600, 2560, BF16, 128, 0), (2000, 1024, F32, 8, 0), (4000, 320, F16, 64, 0),
    (700, 6144, BF16, 6144, 0), (1500, 5120, F32, 0, 0)]


@pytest.mark.parametrize("with_residual", [True, False])
@pytest.mark.parametrize("case", CASES_NORM, ids=str)
def test_rms_norm(case, with_residual):
    from decode_megakernel_04_gb300 import rms_norm
    rows, width, dtype, group, pad = case
    x, r, gain = norm_inputs(rows, width, dtype, pad=pad)
    if not with_residual:
        r = gain = None
    wide = torch.full((rows + 1, width + 16), 7.0, device=DEV).to(E4M3 if group else dtype)
    hs = torch.full((rows + 1, width + 8), 7.0, device=DEV).to(dtype)
    scales = torch.full((rows + 1, (width // group if group else 1) + 1), 7.0, device=DEV)
    sc = scales[:rows, :-1] if group else None
    rms_norm(x, wide[:rows, :width], gain=gain, residual=r, residual_out=hs[:rows, :width], eps=1e-5, scales=sc)
    torch.cuda.synchronize()
    check_norm(x, r, gain, 1e-5, wide[:rows, :width], hs[:rows, :width], sc)
    for t in (wide.float(), hs.float(), scales):  # rows behind the last one and padding stay
        assert (t[rows:] == 7).all() and (t[:, -1] == 7).all()


@pytest.mark.parametrize("width", [256, 5120, 20000])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_rms_norm_in_place(width, dtype):
    from decode_megakernel_04_gb300 import rms_norm
    x, r, gain = norm_inputs(9, width, dtype)
    want, h = torch.empty_like(x), torch.empty_like(x)
    rms_norm(x, want, gain=gain, residual=r, residual_out=h)
    for out_over, h_over in (("x", "r"), ("r", "x"), ("x", None), (None, "x"), (None, "r")):
        t = dict(x=x.clone(), r=r.clone())
        out = t[out_over] if out_over else torch.empty_like(x)
        hh = t[h_over] if h_over else torch.empty_like(x)
        rms_norm(t["x"], out, gain=gain, residual=t["r"], residual_out=hh)
        assert torch.equal(out, want) and torch.equal(hh, h)


def test_rms_norm_special_rows():
    from decode_megakernel_04_gb300 import rms_norm
    for dtype in (BF16, F16, F32):
        x = torch.randn(6, 512, generator=gen(1), device=DEV).to(dtype)
        x[1] = 0
        x[2, 5] = float("nan")
        x[3, 5] = float("inf")
        x[4] *= 2.0 ** -14
        out = torch.empty_like(x)
        rms_norm(x, out, eps=0.0)
        assert out[1].isnan().all()  # 0 / 0, as the formula has it
        assert out[2].isnan().all() and out[3, 5].isnan() and (out[3, 6:] == 0).all()
        check_norm(x[[0, 4, 5]], None, None, 0.0, out[[0, 4, 5]], None, None)
        for group in (64, 512):
            codes, scales = torch.empty(6, 512, device=DEV).to(E4M3), torch.empty(6, 512 // group, device=DEV)
            rms_norm(x, codes, scales=scales)
            assert (codes[1].float() == 0).all() and (scales[1] == 0).all()
            for bad in (2, 3):
                assert codes[bad].float().isnan().all() and scales[bad].isnan().all()
            check_norm(x[[0, 4, 5]], None, None, 1e-6, codes[[0, 4, 5]], None, scales[[0, 4, 5]])


def test_rms_norm_gains_that_are_not_finite():
    """They are their column's alone; among codes they make their group's codes and scale NaN, also where the rest of it is 0."""
    from decode_megakernel_04_gb300 import rms_norm
    for dtype in (BF16, F16, F32):
        x = 1 + torch.rand(3, 512, generator=gen(2), device=DEV).to(dtype)
        gain = torch.ones(512, dtype=dtype, device=DEV)
        gain[5], gain[200] = float("nan"), float("inf")
        out = torch.empty_like(x)
        rms_norm(x, out, gain=gain)
        at = torch.ones(512, dtype=torch.bool, device=DEV)
        at[[5, 200]] = False
        assert out[:, 5].isnan().all() and (out[:, 200] == math.inf).all()
        check_norm(x, None, None, 1e-6, torch.where(at, out, (x.double() / (x.double() ** 2).mean(-1, keepdim=True).add(1e-6).sqrt()).to(dtype)), None, None)
        plain, ps = torch.empty(3, 512, device=DEV).to(E4M3), torch.empty(3, 8, device=DEV)
        rms_norm(x, plain, gain=gain.nan_to_num(nan=0.0, posinf=1.0), scales=ps)
        codes, scales = torch.empty_like(plain), torch.empty_like(ps)
        rms_norm(x, codes, gain=gain, scales=scales)
        f = codes.float()
        at[:64] = at[192:256] = False
        assert f[:, ~at].isnan().all() and scales[:, [0, 3]].isnan().all()
        assert torch.equal(f[:, at], plain.float()[:, at]) and torch.equal(scales[:, [1, 2, 4, 5, 6, 7]], ps[:, [1, 2, 4, 5, 6, 7]])
        one = torch.empty(3, 1, device=DEV)
        gain[:] = 0
        gain[5] = float("nan")
        for sc in (one, scales):
            rms_norm(x, codes, gain=gain, scales=sc)
            assert codes.float()[:, :64].isnan().all() and sc[:, 0].isnan().all()
            assert codes.float()[:, 64:].isnan().all() if sc is one else (codes.float()[:, 64:] == 0).all() and (sc[:, 1:] == 0).all()
            rms_norm(torch.zeros_like(x), codes, eps=0.0, scales=sc)  # 0 / 0, as with 16-bit results
            assert codes.float().isnan().all() and sc.isnan().all()


def test_rms_norm_groups_of_zeros_and_of_the_smallest_values():
    """A group without a value gets scale 0 and codes 0; one whose scale is subnormal keeps its codes."""
    from decode_megakernel_04_gb300 import rms_norm
    x = torch.ones(1, 256, device=DEV)
    gain = torch.ones(256, device=DEV)
    gain[64:128] = 0
    gain[128:192] = 2.0 ** -140 * torch.arange(1, 65, device=DEV)
    codes, scales = torch.empty(1, 256, device=DEV).to(E4M3), torch.empty(1, 4, device=DEV)
    rms_norm(x, codes, gain=gain, scales=scales, eps=0.0)
    assert scales[0, 1] == 0 and (codes[0, 64:128].float() == 0).all()
    want = gain[128:192].double() / scales[0, 2].double()
    assert scales[0, 2] > 0
    check_rounded(codes[0, 128:192].float(), want.clamp(max=448), E4M3, "codes", want * 2.0 ** -17)


def test_rms_norm_offsets_beyond_32_bits():
    from decode_megakernel_04_gb300 import rms_norm
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 26 GB")
    stride = 2 ** 30 + 8
    buf = [torch.empty(4 * stride, dtype=BF16, device=DEV) for _ in range(3)]
    x, r, out = (b.as_strided((4, 512), (stride, 1)) for b in buf)
    a, c, gain = norm_inputs(4, 512, BF16, seed=5)
    x.copy_(a), r.copy_(c)
    rms_norm(x, out, gain=gain, residual=r, residual_out=x)
    check_norm(a, c, gain, 1e-6, out, x, None)


# ---- verification of drafts ---------------------------------------------------------------------------------------------

def as_counted(z):
    """A row of logits in fp64 as the definition counts it: NaN is -infinity, +infinity takes all."""
    z = z.double().clone()
    z[z.isnan()] = -math.inf
    return z


def probabilities(z, t):
    z = as_counted(z)
    p = torch.zeros_like(z)
    t = min(max(t, 2.0 ** -100), 2.0 ** 100) if t > 0 else 0
    top = z.max()
    if top == -math.inf:
        return p
    if not t > 0:
        p[int((z == top).nonzero()[0])] = 1
        return p
    if top == math.inf:
        p[z == top] = 1
    else:
        p = torch.exp((z - top) / t)
    return p / p.sum()


def drafts_reference(s, b):
    """(rows accepted, token, log-probabilities, how near the nearest decision was: a relative distance)."""
    rows = s["tokens"].shape[1]
    t = 1.0 if s.get("temperature") is None else s["temperature"][b].item()
    n = rows - 1 if s.get("n_drafts") is None else min(max(s["n_drafts"][b].item(), 0), rows - 1)
    vocab = s["logits"].shape[1]
    lp, near, a = [0.0] * rows, math.inf, 0
    log = lambda x: math.log(x) if x > 0 else -math.inf  # noqa: E731
    while True:
        p = probabilities(s["logits"][b * rows + a], t)
        if a == n:
            w = p
            break
        x = s["tokens"][b, a + 1].item()
        q = torch.zeros_like(p)
        if s.get("draft_logits") is not None:
            q = probabilities(s["draft_logits"][b * (rows - 1) + a], t)
        elif 0 <= x < vocab:
            q[x] = 1
        if 0 <= x < vocab:
            left, right = s["uniforms"][b, a].item() * q[x].item(), p[x].item()
            if right > 0 or left > 0:
                near = min(near, abs(left - right) / max(left, right))
            if left < right:
                lp[a] = log(right)
                a += 1
                continue
        w = (p - q).clamp(min=0)
        if not (w > 0).any():
            w = p
        break
    e = s["noise"][b].double()
    score = torch.where(w > 0, w / e, 0.0)
    score[score.isnan() | (score < 0)] = 0
    token = int(score.argmax()) if (score > 0).any() else -1
    if token >= 0:
        token = int((score == score.max()).nonzero()[0])
        others = score.clone()
        others[token] = 0
        if score.max() < math.inf:
            near = min(near, 1 - (others.max() / score[token]).item())
    lp[a] = log(p[token].item()) if token >= 0 else -math.inf
    return a + 1, token, lp, near


def draft_inputs(batch, rows, vocab, dtype, draft=True, seed=0, pad=0, spread=3.0, away=0.8):
    g = gen(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    z = rn(batch * rows, vocab + pad) * spread
    race = lambda *s: torch.empty(s, device=DEV).exponential_(generator=g)  # noqa: E731
    t = 0.5 + torch.rand(batch, generator=g, device=DEV)
    t[2::5] = 0
    s = dict(logits=z.to(dtype)[:, :vocab], temperature=t, noise=race(batch, vocab + pad)[:, :vocab],
             uniforms=torch.rand(batch, rows - 1, generator=g, device=DEV))
    zz = z.view(batch, rows, -1)[:, :rows - 1, :vocab]
    if draft and rows > 1:
        y = (zz + away * rn(batch, rows - 1, vocab)).to(dtype)
        chosen = (y.float() / t.clamp(min=0.02)[:, None, None] - race(batch, rows - 1, vocab).log()).argmax(-1)
        wide = torch.empty(batch * (rows - 1), vocab + 2 * pad, dtype=dtype, device=DEV)
        wide[:, :vocab] = y.view(-1, vocab)
        s["draft_logits"] = wide[:, :vocab]
    else:
        chosen = zz.argmax(-1)
    s["tokens"] = torch.cat([torch.full((batch, 1), -5, device=DEV), chosen], 1).to(torch.int32)
    n = torch.full((batch,), rows - 1, dtype=torch.int32, device=DEV)
    n[1::3] //= 2
    s["n_drafts"] = n
    s["positions"] = torch.arange(batch, dtype=torch.int32, device=DEV) * 3 + 1
    return s


def run_drafts(s, **kw):
    from decode_megakernel_04_gb300 import verify_drafts
    b, rows = s["tokens"].shape
    accept = i32([[-9] * b] * 4)  # a row behind the three stays
    lp = torch.full((b + 1, rows), 7.0, device=DEV)
    args = {k: s.get(k) for k in ("draft_logits", "n_drafts", "temperature", "positions")}
    verify_drafts(s["logits"], s["tokens"], s["noise"], s.get("uniforms"), accept[:3], logprobs=lp[:b], **args, **kw)
    torch.cuda.synchronize()
    assert (accept[3] == -9).all() and (lp[b] == 7).all()
    return accept[:3], lp[:b]


def check_drafts(s, accept, lp, undecided=0):
    """Weights are off by 2^-19 relative: a row's exponent is at most 2^-22 of its size (under 60 for a weight that counts)
    off from log2(e) / T in fp32, its product and difference, exp2 2^-22, sums 2^-20. So decisions nearer than 2^-17 may go
    either way; these cases have at most `undecided` of them. A log-probability takes the sum's 2^-20 and 2^-22 of its size."""
    b, rows = s["tokens"].shape
    at = s.get("positions")
    skipped = 0
    for i in range(b):
        a, token, want, near = drafts_reference(s, i)
        if near < 2.0 ** -17:
            skipped += 1
            continue
        got = accept[:, i].tolist()
        assert got == [a, token, (0 if at is None else at[i].item()) + a], (i, got, a, token, near)
        for r, w in enumerate(want):
            x = lp[i, r].item()
            assert x == w if math.isinf(w) or w == 0 else abs(x - w) <= 2.0 ** -20 + abs(w) * 2.0 ** -21, (i, r, x, w)
    assert skipped <= undecided, skipped


CASES_DRAFTS = [  # batch, rows, vocab, dtype, draft logits, padding of a row
    (1, 1, 1, F32, False, 0), (2, 1, 7, F16, False, 1), (1, 2, 2, F32, True, 0), (3, 4, 33, BF16, True, 3), (5, 8, 1000, F32, True, 0),
    (4, 3, 1001, F16, False, 0), (1, 8, 151936, F32, True, 0), (7, 2, 32001, BF16, True, 5), (33, 5, 1024, F32, True, 1),
    (2, 64, 300, F32, True, 0), (3, 1, 202048, BF16, False, 0), (130, 3, 500, F16, True, 2), (2, 4, 163841, BF16, True, 0),
    (300, 1, 4097, F32, False, 0), (1, 3, 1 << 20, F16, True, 0), (16, 8, 50257, F32, False, 0)]


@pytest.mark.parametrize("case", CASES_DRAFTS, ids=str)
def test_verify_drafts(case):
    batch, rows, vocab, dtype, draft, pad = case
    s = draft_inputs(batch, rows, vocab, dtype, draft, seed=batch + rows, pad=pad)
    status = i32([0])
    accept, lp = run_drafts(s, status=status)
    check_drafts(s, accept, lp)
    assert status.item() == 0
    again = run_drafts(s)
    assert torch.equal(again[0], accept) and torch.equal(again[1], lp)


def test_verify_drafts_first_token_is_distributed_as_the_target():
    """40000 requests of the same logits: the first emitted token (the draft if it was accepted, else the bonus token) follows
    the target's row 0, whatever the drafts' distribution; within 5 standard deviations for each token."""
    g = gen(3)
    n, vocab = 40000, 9
    z = torch.randn(2, vocab, generator=g, device=DEV) * 1.5
    y = torch.randn(1, vocab, generator=g, device=DEV) * 1.5
    race = lambda *s: torch.empty(s, device=DEV).exponential_(generator=g)  # noqa: E731
    for with_draft in (True, False):
        chosen = (y - race(n, vocab).log()).argmax(-1) if with_draft else torch.full((n,), 4, device=DEV)
        s = dict(logits=z.repeat(n, 1), tokens=torch.stack([chosen, chosen], 1).to(torch.int32), noise=race(n, vocab),
                 uniforms=torch.rand(n, 1, generator=g, device=DEV), temperature=torch.full((n,), 0.8, device=DEV))
        if with_draft:
            s["draft_logits"] = (y * 0.8).repeat(n, 1)  # drafts are drawn at the same temperature
        accept, _ = run_drafts(s)
        first = torch.where(accept[0] == 2, chosen, accept[1].long())
        p = probabilities(z[0], 0.8).cpu().numpy()
        got = np.bincount(first.cpu().numpy(), minlength=vocab)
        assert (np.abs(got - n * p) <= 5 * np.sqrt(n * p * (1 - p)) + 1).all(), (with_draft, got, n * p)
        kept = accept[1][accept[0] == 2].cpu().numpy()  # and the token behind an accepted draft the target's row 1
        p = probabilities(z[1], 0.8).cpu().numpy()
        assert (np.abs(np.bincount(kept, minlength=vocab) - kept.size * p) <= 5 * np.sqrt(kept.size * p * (1 - p)) + 1).all()


def test_verify_drafts_special_logits():
    inf, nan = float("inf"), float("nan")
    z = torch.randn(10, 3, 40, generator=gen(8), device=DEV) * 2
    y = z[:, :2] + 0.3 * torch.randn(10, 2, 40, generator=gen(9), device=DEV)
    z[1] = -inf                                     # nothing is allowed
    z[2, 0] = nan
    z[3, :, ::2] = -inf
    z[4, :, 5] = nan
    z[5, :, [7, 30]] = inf                          # two tokens share everything
    z[6] = torch.finfo(F32).min                     # a mask of the lowest value everywhere: all alike
    z[7, :, 1:] = torch.finfo(F32).min
    y[8] = -inf                                     # a draft model that allowed nothing
    y[9, :, 3] = inf
    g = gen(10)
    for temperature in (1.0, 0.0, 1e-38, 3e38, nan, -1.0):
        s = dict(logits=z.view(30, 40), draft_logits=y.reshape(20, 40), temperature=torch.full((10,), temperature, device=DEV),
                 tokens=torch.randint(0, 40, (10, 3), generator=g, device=DEV).to(torch.int32),
                 noise=torch.empty(10, 40, device=DEV).exponential_(generator=g), uniforms=torch.rand(10, 2, generator=g, device=DEV))
        s["tokens"][5, 1:], s["tokens"][7, 1:], s["tokens"][9, 1:] = 7, 0, 3
        accept, lp = run_drafts(s)
        check_drafts(s, accept, lp)
        assert accept[:, 1].tolist() == [1, -1, 1] and lp[1].tolist() == [-inf, 0, 0]
        assert accept[1, 2].item() == -1
        s["draft_logits"] = None
        check_drafts(s, *run_drafts(s))


def test_verify_drafts_ties_and_greedy():
    """Temperature 0: drafts are kept while they are the first largest token."""
    z = torch.zeros(4 * 3, 5000, device=DEV)
    z[:, 4000] = z[:, 4999] = 2
    z[4, 77] = 2
    tokens = i32([[0, 4000, 4000], [0, 4999, 4000], [0, 4000, 4999], [0, 4000, 4000]])
    tokens[1, 1] = 4000
    s = dict(logits=z, tokens=tokens, noise=torch.rand(4, 5000, generator=gen(1), device=DEV) + 0.1, uniforms=torch.zeros(4, 2, device=DEV),
             temperature=torch.zeros(4, device=DEV), n_drafts=i32([2, 2, 2, 1]))
    accept, lp = run_drafts(s)
    assert accept.tolist() == [[3, 2, 2, 2], [4000, 77, 4000, 4000], [3, 2, 2, 2]] and (lp == 0).all()
    # equal quotients: the lowest index wins, across CTAs and lanes
    s = dict(logits=torch.zeros(2, 30000, device=DEV), tokens=i32([[0], [0]]), noise=torch.full((2, 30000), 3.0, device=DEV))
    s["noise"][1, [29999, 20001, 20000]] = 2.0
    assert run_drafts(s)[0][1].tolist() == [0, 20000]
    s["noise"][1, [25000, 25003]] = 0.0             # before all others
    s["noise"][0, :29998] = float("nan")
    s["noise"][0, 29998] = -1.0
    assert run_drafts(s)[0][1].tolist() == [29999, 25000]


def test_verify_drafts_tokens_and_counts_out_of_range():
    s = draft_inputs(6, 4, 300, F32, seed=4)
    s["temperature"].fill_(1.0)
    s["tokens"][0, 1], s["tokens"][1, 2], s["tokens"][2, 3] = -1, 300, 2 ** 30
    s["n_drafts"] = i32([3, 3, 3, 9, -2, 3])
    status = i32([0])
    accept, lp = run_drafts(s, status=status)
    assert status.item() & 32 and status.item() & 2
    check_drafts(s, accept, lp)
    # the drafts' own distribution leaves nothing where the two are the same: then the target's
    s["draft_logits"] = s["logits"].view(6, 4, 300)[:, :3].reshape(18, 300).clone()
    accept, lp = run_drafts(s)
    check_drafts(s, accept, lp)
    assert accept[0, 0].item() == 1 and accept[1, 0].item() >= 0
    for same in (3, 5):  # every draft that may be drawn is kept
        assert accept[0, same].item() == 4


def test_verify_drafts_refused_where_draft_and_target_agree():
    """Long rows, raced in many shares: the draft's own distribution leaves nothing, so the token comes from the target's."""
    s = draft_inputs(5, 2, 30011, F32, seed=21)
    s["draft_logits"] = s["logits"].view(5, 2, -1)[:, 0].clone()
    s["tokens"][:, 1] = -1
    s["n_drafts"] = i32([1] * 5)
    accept, lp = run_drafts(s, status=i32([0]))
    check_drafts(s, accept, lp)
    assert (accept[0] == 1).all() and (accept[1] >= 0).all()


def refused_drafts(batch, vocab, away, seed, dtype=F32, temperature=1.0):
    """Two rows a request whose draft is the token that the draft model favours most against the target, with a uniform number
    next to 1: refused in every request."""
    s = draft_inputs(batch, 2, vocab, dtype, seed=seed, away=away)
    s["temperature"].fill_(temperature)
    s["n_drafts"].fill_(1)
    s["uniforms"].fill_(1 - 2.0 ** -24)
    s["draft_logits"][:, 0] = s["logits"].view(batch, 2, -1)[:, 0, 0] + 1  # (of these it is likely enough)
    s["tokens"][:, 1] = (s["draft_logits"].double() - s["logits"].view(batch, 2, -1)[:, 0].double()).argmax(-1)
    return s


@pytest.mark.parametrize("vocab", [40, 30011])
def test_verify_drafts_signs_of_noise_behind_a_refusal(vocab):
    """Where the draft's probability is the larger one a token's weight is 0, whatever its noise; -0 is 0."""
    s = refused_drafts(5, vocab, 0.8, seed=41)
    z = s["logits"].view(5, 2, -1)[:, 0]
    p, q = (torch.softmax(x.double(), -1) for x in (z, s["draft_logits"]))
    for b, bad in enumerate((-1.0, -0.0, float("nan"), -1e-30, 0.0)):
        s["noise"][b, q[b] > p[b]] = bad
    accept, lp = run_drafts(s)
    check_drafts(s, accept, lp)
    assert (accept[0] == 1).all() and (p > q).gather(1, accept[1].long()[:, None]).all()
    at = torch.where(p > 1.5 * q, p, 0.0).argsort(-1, descending=True)[:, 3]  # some token with a weight
    s["noise"].scatter_(1, at[:, None], -0.0)
    accept, _ = run_drafts(s)
    assert torch.equal(accept[1].long(), at)
    s = dict(logits=z.contiguous(), tokens=i32([[0]] * 5), noise=s["noise"])
    assert torch.equal(run_drafts(s)[0][1, :1].long(), at[:1])  # (behind a row without drafts too; other rows have zeros elsewhere)


@pytest.mark.parametrize("vocab", [40, 30011])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_drafts_noise_that_draws_none_of_the_weights(vocab, draft):
    """Behind a refusal some tokens have a weight, but no noise that draws: -1, not a token without a weight."""
    s = refused_drafts(5, vocab, 0.8, seed=43)
    z = s["logits"].view(5, 2, -1)[:, 0]
    p, q = (torch.softmax(x.double(), -1) for x in (z, s["draft_logits"]))
    if draft:
        weight = p > q * (1 - 2.0 ** -15)  # (all that may have one in fp32)
    else:  # (a draft that the target does not want: every other token has a weight)
        s["draft_logits"] = None
        weight = torch.ones_like(p, dtype=torch.bool).scatter_(1, s["tokens"][:, 1:].long(), False)
        z.scatter_(1, s["tokens"][:, 1:].long(), -20.0)
    for b, bad in enumerate((-1.0, float("inf"), float("nan"), 3e38)):
        s["noise"][b, weight[b]] = bad
    accept, lp = run_drafts(s)
    assert accept[0].tolist() == [1] * 5 and accept[1, :4].tolist() == [-1] * 4 and accept[1, 4].item() >= 0
    assert (lp[:4, 0] == -math.inf).all() and lp[4, 0].isfinite() and (lp[:, 1] == 0).all()
    s["noise"][s["noise"] > 2.0 ** 126] = float("inf")  # (as they count)
    check_drafts(s, accept, lp)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab, batch", [(4000, 1000), (151936, 20)])
@pytest.mark.parametrize("away", [1e-1, 1e-2, 1e-3, 1e-5])
def test_verify_drafts_refused_from_a_draft_model_near_the_target(away, vocab, batch, dtype):
    """w = p - q is a difference of two fp32 numbers, so its error goes by p + q. A weight e^-x of the largest is off by 2^-22 x for
    its exponent (the difference, the constant, its quotient and the product 2^-24 each), 2^-22 for exp2 and 2^-23 for two
    products; the sum by that of its terms (the mean of their x is at most ln(vocab) < 12: 2^-18.4), 63 additions in a thread and
    two roundings at each of 17 joins (97 x 2^-24 = 2^-17.4) and what the joins' factors are off by (17 x 2^-22 = 2^-17.9). In all less than
    2^-16, and 2^-22 x. The token may be any whose quotient with that much more weight (and a quotient's 2^-22) is not under
    the largest that is sure."""
    s = draft_inputs(batch, 2, vocab, dtype, seed=vocab + batch, away=away)
    t = s["temperature"] = 0.5 + torch.rand(batch, generator=gen(5), device=DEV)
    s["n_drafts"].fill_(1)
    s["uniforms"].fill_(1 - 2.0 ** -24)
    z, y = s["logits"].view(batch, 2, -1)[:, 0].double(), s["draft_logits"].double()
    x = (y - z).argmax(-1)
    s["tokens"][:, 1] = x
    accept, lp = run_drafts(s)
    down = [(v.amax(-1, keepdim=True) - v) / t.double()[:, None] for v in (z, y)]
    p, q = (torch.softmax(-v, -1) for v in down)
    dp, dq = (w * (2.0 ** -16 + v * 2.0 ** -22) for w, v in zip((p, q), down))
    of = lambda v, i: v.gather(1, i[:, None])[:, 0]  # noqa: E731
    refused = accept[0] == 1
    assert not (~refused & ((1 - 2.0 ** -24) * of(q - dq, x) >= of(p + dp, x))).any()
    assert away < 1e-4 or refused.float().mean() > 0.9
    sure = ((p - q - dp - dq) / s["noise"].double()).amax(-1)
    token = accept[1].long()
    assert (token[refused] >= 0).all() and (token < vocab).all()
    token = token.clamp(min=0)
    most = of(p - q + dp + dq, token) / of(s["noise"].double(), token)
    assert (most >= sure * (1 - 2.0 ** -21))[refused].all()
    assert (most > 0)[refused & (sure > 0)].all()
    want = of(p, token).log()
    assert ((lp[:, 0].double() - want).abs() <= 2.0 ** -16 + want.abs() * 2.0 ** -21)[refused].all()


def test_verify_drafts_workspace_of_the_largest_call_fits_all():
    """One buffer of any contents for calls of all shapes, one after another."""
    from decode_megakernel_04_gb300 import verify_drafts_workspace
    shapes = [(1, 1, 1), (1, 8, 20000), (3, 8, 20000), (33, 2, 20000), (36, 2, 20000), (64, 2, 20000), (64, 8, 20000), (64, 8, 40000)]
    last = 0
    for batch, rows, vocab in shapes:  # each at least as large as the one before
        size = verify_drafts_workspace(torch.empty(batch * rows, vocab, device=DEV), torch.empty(batch, rows, dtype=torch.int32, device=DEV))
        assert size >= last
        last = size
    ws = torch.full((last + 16,), 255, dtype=torch.uint8, device=DEV)
    for k in (7, 1, 3, 0, 6, 2, 1):
        s = draft_inputs(*shapes[k], F32, seed=30 + k)
        accept, lp = run_drafts(s, workspace=ws[:last])
        check_drafts(s, accept, lp)
        again = run_drafts(s)
        assert torch.equal(again[0], accept) and torch.equal(again[1], lp)
    assert (ws[last:] == 255).all()


def test_verify_drafts_defaults():
    s = draft_inputs(5, 3, 777, F32, seed=6)
    for k in ("temperature", "n_drafts", "positions"):
        del s[k]
    check_drafts(s, *run_drafts(s))


def test_verify_drafts_offsets_beyond_32_bits():
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 22 GB")
    from decode_megakernel_04_gb300 import verify_drafts
    s = draft_inputs(2, 2, 1000, BF16, seed=12)
    stride = 2 ** 30 + 3
    big = torch.empty(4 * stride, dtype=BF16, device=DEV).as_strided((4, 1000), (stride, 1))
    y = torch.empty(2 * stride, dtype=BF16, device=DEV).as_strided((2, 1000), (stride, 1))
    e = torch.empty(2 * stride, device=DEV).as_strided((2, 1000), (stride, 1))
    big.copy_(s["logits"]), y.copy_(s["draft_logits"]), e.copy_(s["noise"])
    s.update(logits=big, draft_logits=y, noise=e)
    check_drafts(s, *run_drafts(s))


def test_verify_drafts_of_most_rows():
    """A million rows, and the longest rows."""
    from decode_megakernel_04_gb300 import verify_drafts
    n = 1 << 20
    z = torch.randn(n, 8, generator=gen(2), device=DEV)
    e = torch.empty(n, 8, device=DEV).exponential_(generator=gen(3))
    accept, lp = i32([[0]]).expand(3, n).contiguous(), torch.empty(n, 1, device=DEV)
    verify_drafts(z, torch.zeros(n, 1, dtype=torch.int32, device=DEV), e, None, accept, logprobs=lp)
    p = torch.softmax(z.double(), -1)
    score = p / e.double()
    top2 = score.topk(2, -1).values
    sure = (top2[:, 1] < top2[:, 0] * (1 - 2.0 ** -17))
    assert sure.sum() > n - 100 and (accept[1].long() == score.argmax(-1))[sure].all() and (accept[0] == 1).all()
    want = p.gather(1, accept[1].long()[:, None]).log()
    assert ((lp.double() - want).abs() <= 2.0 ** -20 + want.abs() * 2.0 ** -21).all()
    check_drafts(*(lambda s: (s, *run_drafts(s)))(draft_inputs(2, 2, 1 << 24, BF16, seed=5)))


# ---- attention over a shared prefix -------------------------------------------------------------------------------------

def prefix_inputs(prefix, lens, R, hq, hkv, d, page, dtype, cache, layout="head", seed=0, poison=True, max_pages=None, prefix_pages=None):
    """attention_inputs with the prefix as one more request, taken apart again."""
    s = attention_inputs(list(lens) + [prefix], R, hq, hkv, d, page, dtype, cache, seed=seed, layout=layout, poison=poison)
    own = max(1, max(-(-max(0, n) // page) for n in lens))
    n = -(-max(0, prefix) // page)
    table = torch.full((len(lens), (max_pages or own) + 2), 2 ** 30, dtype=torch.int32, device=DEV)
    table[:, :own] = s["table"][:-1, :own]
    pt = torch.full((prefix_pages or max(1, n),), 2 ** 30, dtype=torch.int32, device=DEV)
    pt[:n] = s["table"][-1, :n]
    return dict(s, q=s["q"][:-1], table=table[:, :max_pages or own], lens=s["lens"][:-1].clone(), prefix_table=pt, prefix_len=i32([prefix]))


def prefix_reference(s, scale):
    q = s["q"].double()
    B, R, hq, d = q.shape
    hkv, page = s["k"].shape[1], s["page"]
    G = hq // hkv

    def cached(x, table, n, sc):
        x = x[table[:-(-n // page)].long()].double().transpose(0, 1).reshape(hkv, -1, d)[:, :n]
        return x if sc is None else x * sc.double()[:, None, None]

    P = max(0, s["prefix_len"].item())
    kp, vp = cached(s["k"], s["prefix_table"], P, s["ks"]), cached(s["v"], s["prefix_table"], P, s["vs"])
    out, av = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((B, R, hq), -math.inf, dtype=torch.float64, device=DEV)
    qk = torch.zeros((B, R, hq), dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        n = max(0, n)
        k = torch.cat([kp, cached(s["k"], s["table"][b], n, s["ks"])], 1)
        v = torch.cat([vp, cached(s["v"], s["table"][b], n, s["vs"])], 1)
        for r in range(R):
            m = P + max(0, n - (R - 1 - r))
            if m == 0:
                continue
            x = q[b, r].view(hkv, G, d)
            z = torch.matmul(x, k[:, :m].transpose(1, 2)) * scale
            p = torch.softmax(z, -1)
            out[b, r] = torch.matmul(p, v[:, :m]).view(hq, d)
            av[b, r] = torch.matmul(p, v[:, :m].abs()).view(hq, d)
            lse[b, r] = torch.logsumexp(z, -1).view(hq)
            qk[b, r] = (torch.matmul(x.abs(), k[:, :m].abs().transpose(1, 2)).amax(-1) * abs(scale)).view(hq)
    return out, lse, av, qk


def run_prefix(s, scale=None, **kw):
    from decode_megakernel_04_gb300 import prefix_attention
    B, R, hq, d = s["q"].shape
    out = torch.full((B, R, hq, d + 8), 7.0, dtype=s["q"].dtype, device=DEV)
    lse = torch.full((B, R, hq), 7.0, device=DEV)
    prefix_attention(s["q"], s["k"], s["v"], s["prefix_table"], s["prefix_len"], s["table"], s["lens"], out[..., :d], scale=scale,
                     lse=lse, k_scale=s["ks"], v_scale=s["vs"], **kw)
    torch.cuda.synchronize()
    assert (out[..., d:] == 7).all()
    return out[..., :d], lse


def check_prefix(s, got, lse, scale, what=""):
    """check_attention's bounds (test_gpu_serving_ops.py), with a probability rounded once to 16 bits: bf16 half a step 2^-8, fp16
    and e4m3 2^-11; fp16 ones against a largest of 2^14, so off by another 2^-25 / 2^14 = 2^-39 of the largest where they are
    subnormal."""
    d = s["q"].shape[-1]
    out, l64, av, qk = prefix_reference(s, scale)
    n = (s["lens"].clamp(min=0) + s["prefix_len"].clamp(min=0)).double()[:, None, None]
    e4 = s["ks"] is not None
    ds = qk * ((d + 4) * 2.0 ** -23 + (2.0 ** -20 if e4 else 0))
    rel = 2 * (ds + 2.0 ** -21 + n * 2.0 ** -23) + (2.0 ** -11 if e4 or s["q"].dtype is F16 else 2.0 ** -8)
    v_max = s["v"].float().nan_to_num().abs().amax((0, 2, 3))
    v_max = (v_max if s["vs"] is None else v_max * s["vs"]).max().double()
    slack = rel[..., None] * av + (n * 2.0 ** -39)[..., None] * v_max
    assert not got.isnan().any(), what
    empty = l64 == -math.inf
    assert (got[empty] == 0).all() and (lse[empty] == -math.inf).all(), what
    check_rounded(got, out, s["q"].dtype, what + " out", slack)
    err = (lse.double() - l64).abs()[~empty]
    bound = (ds + 2.0 ** -20 + n * 2.0 ** -23 + l64.abs() * 2.0 ** -22)[~empty]
    assert err.numel() == 0 or (err <= bound).all(), f"{what} lse {(err / bound).max().item()}"


CASES_PREFIX = [  # prefix, lens, R, hq, hkv, d, page, dtype, cache, layout
    (0, [0, 1, 5], 1, 4, 1, 64, 16, F16, F16, "head"),
    (1, [0, 1, 5], 1, 4, 1, 64, 16, F16, F16, "head"),
    (130, [0, 20, 40], 1, 4, 1, 64, 16, F16, F16, "head"),
    (128, [3], 1, 1, 1, 128, 16, BF16, BF16, "head"),
    (129, [17, 0], 1, 6, 1, 128, 16, BF16, BF16, "place"),
    (127, [1, 2, 3, 4], 1, 24, 4, 256, 64, BF16, BF16, "padded"),
    (4096, [1, 22, 43, 64], 1, 24, 4, 256, 64, BF16, BF16, "head"),
    (1000, [9, 8, 100], 8, 6, 1, 128, 16, BF16, BF16, "head"),
    (777, [0, 3, 5, 9], 5, 8, 2, 128, 1, F16, F16, "place"),            # lengths under the rows: padding rows
    (2500, [i * 7 % 300 for i in range(33)], 1, 48, 8, 128, 32, BF16, BF16, "head"),   # 198 rows of a kv head
    (600, [i * 5 % 90 for i in range(70)], 1, 14, 2, 64, 24, F16, F16, "padded"),      # 490 rows
    (900, [i * 11 % 200 for i in range(45)], 1, 12, 2, 256, 16, F16, F16, "head"),     # 270 rows
    (300, [40] * 22, 2, 18, 3, 128, 256, BF16, BF16, "head"),           # 264 rows: a block of two and one of one tile
    (5000, [100] * 3, 1, 1, 1, 128, 16, F16, F16, "head"),
    (20000, [500, 3], 1, 12, 2, 128, 64, BF16, BF16, "head"),
    (700, [3, 64, 100], 1, 6, 2, 16, 16, BF16, BF16, "head"),           # narrow and odd widths
    (700, [3, 64, 100], 2, 6, 2, 80, 16, F16, F16, "padded"),
    (333, [3, 64, 100], 1, 6, 2, 192, 16, BF16, BF16, "head"),
    (1200, [90, 0, 200], 1, 6, 2, 48, 8, BF16, E4M3, "head"),
    (1200, [90, 0, 200], 4, 6, 2, 240, 16, F16, E4M3, "head"),
    (1000, [3, 64, 1000, 0, 127], 1, 48, 8, 128, 32, BF16, E4M3, "head"),
    (130, [3, 64, 10, 0, 127], 1, 4, 1, 64, 16, F16, E4M3, "place"),
    (3000, [i * 13 % 150 for i in range(40)], 1, 48, 8, 128, 16, BF16, E4M3, "padded"),
    (2000, [10, 20, 30], 8, 24, 4, 256, 64, BF16, E4M3, "head"),
    (900, [30] * 30, 1, 20, 2, 256, 64, F16, E4M3, "head"),
]


@pytest.mark.parametrize("wide", [False, True], ids=["", "wide"])
@pytest.mark.parametrize("case", CASES_PREFIX, ids=lambda c: f"{c[0]}+{len(c[1])}x{max(c[1])}-" + "-".join(str(x) for x in c[2:]))
def test_prefix_attention(case, wide):
    """Each case with tables as wide as what is in them, and with wide ones."""
    prefix, lens, R, hq, hkv, d, page, dtype, cache, layout = case
    extra = dict(max_pages=(1 << 20) // page, prefix_pages=(1 << 21) // page) if wide else {}
    s = prefix_inputs(prefix, lens, R, hq, hkv, d, page, dtype, cache, layout, seed=prefix, **extra)
    status = i32([0])
    got, lse = run_prefix(s, status=status)
    check_prefix(s, got, lse, d ** -0.5)
    assert status.item() == 0
    again = run_prefix(s)
    assert torch.equal(again[0], got) and torch.equal(again[1], lse)


def test_prefix_attention_is_attention_over_the_whole():
    """The same requests through mk_paged_attention with tables that begin with the prefix's pages (a prefix of whole pages)."""
    from decode_megakernel_04_gb300 import paged_attention
    s = prefix_inputs(1024, [5, 77, 300], 2, 12, 2, 128, 16, F16, F16)
    got, lse = run_prefix(s)
    whole = torch.cat([s["prefix_table"][None].expand(3, -1), s["table"]], 1).contiguous()
    out, l2 = torch.empty_like(got), torch.empty_like(lse)
    paged_attention(s["q"], s["k"], s["v"], whole, s["lens"] + 1024, out, lse=l2)
    check_prefix(s, got, lse, 128 ** -0.5)
    check_prefix(s, out, l2, 128 ** -0.5)


@pytest.mark.parametrize("dtype, cache, d", [(BF16, BF16, 128), (F16, F16, 64), (F16, F16, 256), (BF16, E4M3, 128), (F16, E4M3, 128)])
def test_prefix_scores_that_grow_and_that_begin_at_minus_infinity(dtype, cache, d):
    """Keys in ascending order (every tile moves every maximum), large and small scores, a first tile of -infinity."""
    s = prefix_inputs(1500, [40, 0, 300], 1, 12, 2, d, 16, dtype, cache, seed=2, poison=False)
    if cache is E4M3:
        s["ks"].fill_(0.5), s["vs"].fill_(0.5)
    s["q"][..., 0] = 4.0
    pages = s["prefix_table"].long()
    grow = torch.linspace(-30, 30, pages.numel() * 16, device=DEV).view(-1, 1, 16)
    for scale_up in (1.0, 4.0):
        k0 = s["k"][pages].float()
        k0[..., 0] = grow * scale_up
        s["k"][pages] = k0.to(cache)
        got, lse = run_prefix(s, scale=0.25)
        check_prefix(s, got, lse, 0.25, "growing")
    if cache is E4M3:
        return
    k0 = s["k"][pages].float()
    k0[:20] = 0
    k0[:20, ..., 0] = -math.inf
    s["k"][pages] = k0.to(cache)
    got, lse = run_prefix(s, scale=0.25)
    k0[:20] = 0  # for the reference: far below what counts (0 * infinity elsewhere)
    s2 = dict(s, k=s["k"].clone())
    s2["k"][pages[:20]] = 0
    s2["k"][pages[:20], ..., 0] = -1e4
    check_prefix(s2, got, lse, 0.25, "after -infinity")


@pytest.mark.parametrize("dtype, cache, d", [(F16, F16, 64), (F16, F16, 128), (F16, F16, 256), (F16, E4M3, 128), (BF16, E4M3, 128), (BF16, BF16, 256)])
@pytest.mark.parametrize("first", [True, False])
def test_prefix_many_weak_keys_behind_a_strong_one(dtype, cache, d, first):
    """One key of the prefix 14 to 18 above the others with a value of zero: the others' small probabilities are the result."""
    s = prefix_inputs(4000, [7, 300, 64], 1, 24, 8, d, 16, dtype, cache, seed=4, poison=False)
    if cache is E4M3:
        s["ks"].fill_(1.0), s["vs"].fill_(0.5)
    s["q"].mul_(0.125)
    s["q"][..., 0] = 4.0
    s["k"][..., 0] = 0.0
    s["v"].copy_((s["v"].float() * 0.25 + 1.0).to(cache))
    at = s["prefix_table"][0 if first else 130].long()
    s["k"][at, :, 3] = 0.0
    s["k"][at, :, 3, 0] = (14.0 + torch.arange(8, device=DEV) % 5).to(cache)
    s["v"][at, :, 3] = 0.0
    got, lse = run_prefix(s, scale=0.25)
    check_prefix(s, got, lse, 0.25)


def test_prefix_scores_of_any_size():
    """Scores of some hundred: one key takes all, and the bases of prefix and own positions are far apart."""
    for own in (False, True):
        s = prefix_inputs(300, [50, 3], 1, 6, 1, 128, 16, BF16, BF16, seed=7, poison=False)
        s["q"].mul_(20)
        if own:
            s["k"][s["table"][0, 0].long()] *= 8
        got, lse = run_prefix(s, scale=1.0)
        check_prefix(s, got, lse, 1.0)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-30])
@pytest.mark.parametrize("dtype, cache, d", [(BF16, BF16, 128), (F16, F16, 64), (BF16, BF16, 256), (BF16, E4M3, 128), (F16, E4M3, 64)])
def test_prefix_scales_of_any_sign(dtype, cache, d, scale):
    """Also e4m3 caches whose heads' scales have different signs."""
    s = prefix_inputs(300, [40, 3, 200], 3, 12, 2, d, 16, dtype, cache, seed=17)
    if s["ks"] is not None:
        s["ks"][1] *= -1
    check_prefix(s, *run_prefix(s, scale=scale), scale)


@pytest.mark.parametrize("dtype, cache, d", [(BF16, BF16, 128), (F16, F16, 64), (BF16, BF16, 256), (BF16, E4M3, 128), (F16, E4M3, 64)])
def test_prefix_scales_that_are_nan_reach_their_rows(dtype, cache, d):
    """A scale of NaN gives NaN, as in mk_paged_attention; rows that see nothing are 0 all the same."""
    from decode_megakernel_04_gb300 import paged_attention
    for prefix in (200, 0):
        s = prefix_inputs(prefix, [40, 1, 200], 3, 12, 2, d, 16, dtype, cache, seed=18)
        nan = float("nan")
        scale = d ** -0.5
        if cache is E4M3:
            s["ks"][1] = nan
        else:
            scale = nan
        got, lse = run_prefix(s, scale=scale)
        seen = torch.ones(3, 3, 12, dtype=torch.bool, device=DEV)
        if prefix == 0:
            seen[1, :2] = False  # (one position: the newest row's)
        bad = seen.clone()
        if cache is E4M3:
            bad[..., :6] = False
        assert got[bad].isnan().all() and lse[bad].isnan().all()
        assert (got[~seen] == 0).all() and (lse[~seen] == -math.inf).all()
        assert not got[~bad].isnan().any() and not lse[~bad].isnan().any()
        if prefix == 0:  # the same call without the prefix
            out, l2 = torch.empty_like(s["q"]), torch.empty_like(lse)
            paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], out, scale=scale, lse=l2, k_scale=s["ks"], v_scale=s["vs"])
            assert torch.equal(out.isnan(), got.isnan()) and torch.equal(l2.isnan(), lse.isnan())


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_prefix_hidden_values_do_not_leak(cache):
    """NaN and infinities behind the prefix's end in its last page, and in the places of later rows of a verify block."""
    s = prefix_inputs(133, [70, 64, 9], 8, 6, 1, 128, 16, BF16, cache, seed=3)  # (unseen places are NaN)
    got, lse = run_prefix(s)
    check_prefix(s, got, lse, 128 ** -0.5)
    bad = dict(s, k=s["k"].clone(), v=s["v"].clone())
    for b, n in enumerate((70, 64, 9)):  # the newest key and value of each request
        p = n - 1
        at = s["table"][b, p // 16].long()
        bad["k"][at, :, p % 16] = float("nan")
        bad["v"][at, :, p % 16] = float("nan")
    got2, lse2 = run_prefix(bad)
    assert got2[:, 7].isnan().all() and lse2[:, 7].isnan().all()
    # The other rows are what they were, within the same bounds (values beside those that are left out of a product are added to
    # its sums in fp32, in another order and unrounded, so not bit for bit).
    got2[:, 7], lse2[:, 7] = got[:, 7], lse[:, 7]
    check_prefix(s, got2, lse2, 128 ** -0.5, "beside hidden values")


def test_prefix_values_that_are_not_finite_reach_their_rows():
    s = prefix_inputs(300, [5, 9], 1, 4, 1, 128, 16, BF16, BF16, seed=5, poison=False)
    at = s["prefix_table"][2].long()
    s["v"][at, 0, 7, 11] = float("inf")
    got, _ = run_prefix(s)
    assert (~got[..., 11].isfinite()).all() and got[..., :11].isfinite().all() and got[..., 12:].isfinite().all()
    s["v"][at, 0, 7, 11] = 0
    s["k"][at, 0, 7] = float("nan")
    got, lse = run_prefix(s)
    assert got.isnan().all() and lse.isnan().all()


def test_prefix_lengths_and_pages_out_of_range():
    s = prefix_inputs(96, [20, 33], 1, 4, 2, 64, 16, F16, F16, seed=6, poison=False)
    status = i32([0])
    s["prefix_len"].fill_(5000)  # counts as all the table holds
    got, lse = run_prefix(s, status=status)
    assert status.item() == 2
    s["prefix_len"].fill_(96)
    check_prefix(s, got, lse, 64 ** -0.5)
    s["prefix_len"].fill_(-3)
    status.zero_()
    got, lse = run_prefix(s, status=status)
    assert status.item() == 2
    check_prefix(s, got, lse, 64 ** -0.5)
    s["prefix_len"].fill_(96)
    for bad in (-1, s["k"].shape[0], 2 ** 31 - 1, -2 ** 31):
        status.zero_()
        t = s["prefix_table"].clone()
        t[3] = bad
        got, lse = run_prefix(dict(s, prefix_table=t), status=status)
        assert status.item() == 1
        z = dict(s, k=torch.cat([s["k"], torch.zeros_like(s["k"][:1])]), v=torch.cat([s["v"], torch.zeros_like(s["v"][:1])]))
        t[3] = s["k"].shape[0]  # a page of zeros
        check_prefix(dict(z, prefix_table=t), got, lse, 64 ** -0.5)


def test_prefix_offsets_beyond_32_bits():
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 18 GB")
    s = prefix_inputs(200, [20, 33], 1, 4, 2, 128, 16, BF16, BF16, seed=8, poison=False)
    n, hkv, page, d = s["k"].shape
    stride = 2 ** 33 // (n + 2)
    stride -= stride % 8
    big = torch.empty(n * stride, dtype=BF16, device=DEV).as_strided((n, hkv, page, d), (stride, page * d, d, 1))
    big.copy_(s["k"])
    got, lse = run_prefix(dict(s, k=big))
    check_prefix(s, got, lse, d ** -0.5)


def test_prefix_most_heads_and_many_requests():
    s = prefix_inputs(50, [3] * 2, 1, 4096, 4096, 16, 16, BF16, BF16, seed=9)
    check_prefix(s, *run_prefix(s), 0.25)
    s = prefix_inputs(200, [i % 5 for i in range(2000)], 1, 2, 1, 64, 16, F16, F16, seed=10)
    check_prefix(s, *run_prefix(s), 0.125)
    s = prefix_inputs(100, [520, 513], 512, 4, 2, 64, 16, BF16, BF16, seed=11)
    check_prefix(s, *run_prefix(s), 0.125)


def test_prefix_workspace_of_the_largest_call_fits_all():
    from decode_megakernel_04_gb300 import prefix_attention, prefix_attention_workspace
    s = prefix_inputs(700, [40] * 40, 1, 12, 2, 128, 16, BF16, BF16)
    wide = torch.zeros(40, 5000, dtype=torch.int32, device=DEV)
    last = 0
    for b in (1, 2, 5, 11, 12, 22, 23, 40):
        for t in (s["table"][:b], wide[:b]):
            size = prefix_attention_workspace(s["q"][:b], s["k"], s["prefix_table"], t)
            assert size > 0 and size <= prefix_attention_workspace(s["q"], s["k"], s["prefix_table"], wide)
        assert size >= last
        last = size
    ws = torch.full((last + 16,), 255, dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(s["q"]), torch.empty(40, 1, 12, device=DEV)
    for b in (40, 3, 17):
        prefix_attention(s["q"][:b], s["k"], s["v"], s["prefix_table"], s["prefix_len"], s["table"][:b], s["lens"][:b], out[:b],
                         lse=lse[:b], workspace=ws[:last])
        part = dict(s, q=s["q"][:b], table=s["table"][:b], lens=s["lens"][:b])
        check_prefix(part, out[:b], lse[:b], 128 ** -0.5)
    assert (ws[last:] == 255).all()
    from decode_megakernel_04_gb300 import MKError
    with pytest.raises(MKError):
        prefix_attention(s["q"], s["k"], s["v"], s["prefix_table"], s["prefix_len"], s["table"], s["lens"], out,
                         workspace=ws[:prefix_attention_workspace(s["q"], s["k"], s["prefix_table"], s["table"]) - 16])


@pytest.mark.parametrize("at", [16, 32, 48, 240])
@pytest.mark.parametrize("case", [(700, 1, BF16, BF16, 128), (300, 2, F16, F16, 64), (900, 1, BF16, BF16, 256), (500, 1, BF16, E4M3, 128)], ids=str)
def test_prefix_workspace_that_begins_between_32_byte_boundaries(case, at):
    """A part of a larger buffer, on 16 bytes as documented: the result is that of any other workspace, and nothing is written
    outside of it."""
    from decode_megakernel_04_gb300 import prefix_attention_workspace
    prefix, R, dtype, cache, d = case
    s = prefix_inputs(prefix, [40, 3, 0, 150], R, 12, 2, d, 16, dtype, cache, seed=at)
    size = prefix_attention_workspace(s["q"], s["k"], s["prefix_table"], s["table"])
    ws = torch.full((size + 512,), 255, dtype=torch.uint8, device=DEV)
    got, lse = run_prefix(s, workspace=ws[at:at + size])
    check_prefix(s, got, lse, d ** -0.5)
    want, lse2 = run_prefix(s)
    assert torch.equal(got, want) and torch.equal(lse, lse2)
    assert (ws[:at] == 255).all() and (ws[at + size:] == 255).all()


# ---- streams, graphs, threads, steps ------------------------------------------------------------------------------------

def operator_calls(seed=0):
    """One call of each operator: (call(stream), check())."""
    from decode_megakernel_04_gb300 import prefix_attention, rms_norm, verify_drafts
    x, r, gain = norm_inputs(200, 7168, BF16, seed=seed)
    codes, scales, h = torch.empty(200, 7168, device=DEV).to(E4M3), torch.empty(200, 56, device=DEV), torch.empty_like(x)
    p = prefix_inputs(3000, [i * 7 % 300 for i in range(40)], 1, 48, 8, 128, 32, BF16, BF16, seed=seed)
    out, lse = torch.empty_like(p["q"]), torch.empty(40, 1, 48, device=DEV)
    s = draft_inputs(9, 4, 30000, F32, seed=seed + 1)
    accept, lp = i32([[0] * 9] * 3), torch.empty(9, 4, device=DEV)

    def wipe():
        for t in (codes.view(torch.uint8), scales, h, out, lse, accept, lp):
            t.fill_(99)

    def call(stream=None):
        rms_norm(x, codes, gain=gain, residual=r, residual_out=h, scales=scales, stream=stream)
        prefix_attention(p["q"], p["k"], p["v"], p["prefix_table"], p["prefix_len"], p["table"], p["lens"], out, lse=lse, stream=stream)
        verify_drafts(s["logits"], s["tokens"], s["noise"], s["uniforms"], accept, draft_logits=s["draft_logits"],
                      n_drafts=s["n_drafts"], temperature=s["temperature"], positions=s["positions"], logprobs=lp, stream=stream)

    def check():
        check_norm(x, r, gain, 1e-6, codes, h, scales)
        check_prefix(p, out, lse, 128 ** -0.5)
        check_drafts(s, accept, lp)

    return call, check, wipe, (p, s)


def test_operators_captured_and_on_streams():
    """Two graphs of the operators replayed at the same time on two streams beside an eager call, with lengths that changed
    since the capture."""
    sets = [operator_calls(seed) for seed in (0, 3)]
    graphs = []
    for call, check, wipe, _ in sets:
        call()
        torch.cuda.synchronize()
        check()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    third = operator_calls(7)
    for call, check, wipe, (p, s) in sets:
        wipe()
        p["prefix_len"].fill_(1777)
        p["lens"].clamp_(max=131)
        s["uniforms"].copy_(torch.rand(s["uniforms"].shape, generator=gen(21), device=DEV))
    third[2]()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        third[0](streams[2].cuda_stream)
    torch.cuda.synchronize()
    for _, check, _, _ in sets + [third]:
        check()


def test_operators_from_several_threads():
    sets = [operator_calls(seed) for seed in range(4)]
    for _, _, wipe, _ in sets:
        wipe()
    torch.cuda.synchronize()
    errors = []

    def work(call):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(6):
                    call()
            st.synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c[0],)) for c in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for _, check, _, _ in sets:
        check()


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_a_speculative_step_of_forked_samples(cache):
    """A layer's attention block and the end of a step as a serving program runs them, captured once: norm with the residual,
    projection, per-head norms and rotation with the append, attention over the shared prompt and own pages, norm, logits,
    verification; against fp64 of the same chain, each operator from what it was given."""
    from decode_megakernel_04_gb300 import prefix_attention, qk_norm_rope, rms_norm, verify_drafts
    B, R, hq, hkv, d, width, vocab, page, prompt = 6, 3, 12, 2, 128, 512, 999, 16, 300
    g = gen(31)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    s = prefix_inputs(prompt, [page * 4] * B, R, hq, hkv, d, page, BF16, cache, seed=12, poison=False)
    ks, vs = (torch.full((hkv,), 0.03, device=DEV) for _ in range(2)) if cache is E4M3 else (None, None)
    s["ks"], s["vs"] = ks, vs
    lens = i32([R + 2 * b for b in range(B)])  # own positions, the new rows' included
    slots = torch.empty(B, R, dtype=torch.int64, device=DEV)
    x, res = rn(B * R, width).to(BF16), (2 * rn(B * R, width)).to(BF16)
    gain, wq = (1 + 0.1 * rn(width)).to(BF16), (rn((hq + 2 * hkv) * d, width) * 0.05).to(BF16)
    wo, head = (rn(width, hq * d) * 0.03).to(BF16), (rn(vocab, width) * 0.3).to(BF16)
    inv = (1e4 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).to(DEV)
    dr = draft_inputs(B, R, vocab, F32, seed=13)
    t = {}

    def step():
        p = lens[:, None].long() - R + torch.arange(R, device=DEV)
        slots.copy_(s["table"].long().gather(1, p // page) * page + p % page)
        pos = (prompt + p).to(torch.int32).view(-1)
        t.update(h=torch.empty_like(x), n1=torch.empty_like(x), out=torch.empty(B, R, hq, d, dtype=BF16, device=DEV),
                 lse=torch.empty(B, R, hq, device=DEV), h2=torch.empty_like(x), n2=torch.empty_like(x), pos=pos,
                 accept=torch.empty(3, B, dtype=torch.int32, device=DEV), lp=torch.empty(B, R, device=DEV))
        rms_norm(x, t["n1"], gain=gain, residual=res, residual_out=t["h"])
        qkv = (t["n1"] @ wq.t()).view(B * R, -1, d)
        t["qkv"], q = qkv, torch.empty(B * R, hq, d, dtype=BF16, device=DEV)
        qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], pos, inv, q, v=qkv[:, hq + hkv:], k_pages=s["k"], v_pages=s["v"],
                     slots=slots.view(-1), k_scale=ks, v_scale=vs)
        t["q"] = q.view(B, R, hq, d)
        prefix_attention(t["q"], s["k"], s["v"], s["prefix_table"], s["prefix_len"], s["table"], lens, t["out"], lse=t["lse"],
                         k_scale=ks, v_scale=vs)
        t["y"] = t["out"].view(B * R, -1) @ wo.t()
        rms_norm(t["y"], t["n2"], gain=gain, residual=t["h"], residual_out=t["h2"])
        t["logits"] = (t["n2"] @ head.t()).float()
        verify_drafts(t["logits"], dr["tokens"], dr["noise"], dr["uniforms"], t["accept"], n_drafts=dr["n_drafts"],
                      temperature=dr["temperature"], positions=t["pos"].view(B, R)[:, 0].contiguous(), logprobs=t["lp"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(3):
        before = s["k"].clone()
        graph.replay()
        torch.cuda.synchronize()
        check_norm(x, res, gain, 1e-6, t["n1"], t["h"], None)
        p = lens[:, None].long() - R + torch.arange(R, device=DEV)
        want = rotate(t["qkv"][:, hq:hq + hkv], None, 0, t["pos"], inv)
        got = s["k"].transpose(1, 2).reshape(-1, hkv, d)[slots.view(-1)].float()
        check_rounded(got, want if ks is None else (want / ks.double()[:, None]).clamp(-448, 448), cache, "cache", qk_slack(want if ks is None else want / 0.03))
        assert torch.equal(before[s["prefix_table"].long()].float(), s["k"][s["prefix_table"].long()].float())
        check_prefix(dict(s, q=t["q"], lens=lens), t["out"], t["lse"], d ** -0.5)
        check_norm(t["y"], t["h"], gain, 1e-6, t["n2"], t["h2"], None)
        check_drafts(dict(dr, logits=t["logits"], draft_logits=None, positions=t["pos"].view(B, R)[:, 0]), t["accept"], t["lp"])
        lens.add_(t["accept"][0])  # the accepted rows are kept; the next block begins behind them
        x.copy_(rn(B * R, width).to(BF16))


def test_verify_with_sampling():
    """Megakernel.verify(sampling=...) is a step with logits followed by verify_drafts, and commits what it accepted."""
    from decode_megakernel_04_gb300 import Megakernel
    from synthetic import config, make_tokens, make_weights
    cfg = config("tiny_dense")
    w = make_weights(cfg, seed=0, device=torch.device(DEV))
    ctx = make_tokens(0, "ctx", (2, 48), cfg.vocab, device=torch.device(DEV))
    a, b = (Megakernel(cfg, w, max_batch=2, max_rows=4, max_ctx=96) for _ in range(2))
    a.prefill(ctx), b.prefill(ctx)
    g = gen(17)
    tokens, pos = i32([[3, 1, 2, 9], [7, 5, 5, 5]]), i32([48, 48])
    for R, nxt in ((4, 4), (4, 1), (1, 2), (2, 1)):
        logits, plain = torch.empty(2 * R, cfg.vocab, device=DEV), torch.empty(2 * R, cfg.vocab, device=DEV)
        s = dict(noise=torch.empty(2, cfg.vocab, device=DEV).exponential_(generator=g), uniforms=torch.rand(2, R - 1, generator=g, device=DEV),
                 temperature=torch.tensor([0.7, 1.3], device=DEV), logprobs=torch.empty(2, R, device=DEV))
        accept, argmax = i32([[0, 0]] * 3), i32([0] * 2 * R)
        a.verify(tokens, pos, accept, logits=logits, argmax=argmax, sampling=s)
        assert a.status() == 0
        b.step(tokens, pos, plain)
        assert b.status() == 0 and torch.equal(logits, plain)
        assert torch.equal(argmax.long(), logits.argmax(-1))
        check_drafts(dict(s, logits=logits, tokens=tokens, positions=pos), accept, s["logprobs"])
        pos = accept[2].contiguous()
        tokens = torch.cat([accept[1][:, None], torch.randint(0, cfg.vocab, (2, nxt - 1), generator=g, device=DEV, dtype=torch.int32)], 1).contiguous()
    a.close(), b.close()


@pytest.mark.parametrize("model", ["hybrid", "moe"])
def test_verify_with_sampling_over_recurrent_states(model):
    """Stacks whose layers carry a state from row to row: the rows that sampling refused are not in the state that the next block
    begins with. Logits against the oracle, which takes the same blocks at the positions that the device decided."""
    from decode_megakernel_04_gb300 import Megakernel
    from gpu_harness import Report, compare_logits
    from oracle import Oracle
    from synthetic import make_tokens, make_weights
    from test_gpu_steps import TOL, _hybrid, _moe
    cfg = _hybrid() if model == "hybrid" else _moe()
    dev = torch.device(DEV)
    w = make_weights(cfg, seed=6, device=dev)
    B, T, g, rep = 2, 19, gen(23), Report()
    ctx = make_tokens(6, "ctx", (B, T), cfg.vocab, device=dev).contiguous()
    m = Megakernel(cfg, w, max_batch=B, max_rows=4, max_ctx=64)
    m.prefill(ctx)
    orc = Oracle(cfg, w, B, 64)
    orc.prefill(ctx.cpu().numpy())
    token, pos = make_tokens(6, "first", (B, 1), cfg.vocab, device=dev), torch.full((B,), T, dtype=torch.int32, device=dev)
    # drafts up to the first number of 1 are kept (any token has some probability), that one is refused
    for turn, (R, keep) in enumerate(((4, (1, 3)), (4, (0, 2)), (3, (2, 0)), (1, (0, 0)), (2, (0, 1)))):
        drafted = torch.randint(0, cfg.vocab, (B, R - 1), generator=g, device=DEV, dtype=torch.int32)
        tokens = torch.cat([token.view(B, 1).to(torch.int32), drafted], 1).contiguous()
        u = torch.ones(B, R - 1, device=DEV)
        for b in range(B):
            u[b, :keep[b]] = 0
        logits, accept = torch.empty(B * R, cfg.vocab, device=DEV), i32([[0] * B] * 3)
        s = dict(noise=torch.empty(B, cfg.vocab, device=DEV).exponential_(generator=g), uniforms=u, logprobs=torch.empty(B, R, device=DEV))
        m.verify(tokens, pos, accept, logits, sampling=s)
        assert m.status() == 0
        ref = orc.step(tokens.cpu().numpy().astype(np.int64), pos.cpu().numpy().astype(np.int64))
        compare_logits(logits.cpu().numpy().reshape(B, R, -1), ref, TOL, rep, f"block {turn}")
        check_drafts(dict(s, logits=logits, tokens=tokens, positions=pos), accept, s["logprobs"])
        assert accept[0].tolist() == [k + 1 for k in keep]
        token, pos = accept[1].clone(), accept[2].clone()
    m.close()


def test_sampling_that_the_library_refuses_is_refused_before_the_step():
    from decode_megakernel_04_gb300 import MKError
    m, vocab = stepless()[0], 8
    tok, z = i32([[1, 2], [3, 4]]), torch.zeros(4, vocab, device=DEV)
    noise, u, accept = torch.ones(2, vocab, device=DEV), torch.zeros(2, 1, device=DEV), i32([[0, 0]] * 3)
    odd = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    for bad in (dict(noise=noise, uniforms=u, workspace=odd[:8]), dict(noise=noise, uniforms=u, workspace=odd[1:])):
        with pytest.raises(MKError):
            m.verify(tok, i32([0, 0]), accept, z, sampling=bad)
    for bad in (dict(noise=noise), dict(uniforms=u), dict(noise=noise[:, :-1], uniforms=u), dict(noise=noise, uniforms=u[:1]),
                dict(noise=noise, uniforms=u, draft_logits=z), dict(noise=noise, uniforms=u, temperature=u[:1, 0])):
        with pytest.raises(ValueError):
            m.verify(tok, i32([0, 0]), accept, z, sampling=bad)
    with pytest.raises(ValueError):
        m.verify(tok, i32([0, 0]), accept, torch.zeros(4, vocab + 1, device=DEV)[:, :vocab], sampling=dict(noise=noise, uniforms=u))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_sampling_of_16_bit_logits_is_refused_before_the_step(dtype):
    """The step writes fp32 rows; verify_drafts alone takes these."""
    m, vocab = stepless()[0], 8
    tok, z, accept = i32([[1, 2], [3, 4]]), torch.zeros(4, vocab, dtype=dtype, device=DEV), i32([[0, 0]] * 3)
    with pytest.raises(ValueError):
        m.verify(tok, i32([0, 0]), accept, z, sampling=dict(noise=torch.ones(2, vocab, device=DEV), uniforms=torch.zeros(2, 1, device=DEV)))


def test_wrappers_refuse():
    import decode_megakernel_04_gb300 as mk
    x = torch.zeros(4, 256, dtype=BF16, device=DEV)
    for bad in (dict(out=torch.zeros(4, 128, dtype=BF16, device=DEV)), dict(out=torch.zeros(3, 256, dtype=BF16, device=DEV)),
                dict(out=x.clone(), residual=x[:, :128]), dict(out=x.clone(), gain=x[0, :128]), dict(out=x.clone(), residual=x.float()),
                dict(out=x.to(E4M3)), dict(out=x.to(E4M3), scales=torch.zeros(4, 3, device=DEV)), dict(out=x.clone(), scales=torch.zeros(4, 2, device=DEV)),
                dict(out=x.clone(), residual_out=x.t().contiguous().t()), dict(out=x.long())):
        with pytest.raises((ValueError, mk.MKError)):
            mk.rms_norm(x, **bad)
    s = prefix_inputs(100, [5, 6], 1, 4, 2, 64, 16, F16, F16)
    good = dict(q=s["q"], k_pages=s["k"], v_pages=s["v"], prefix_table=s["prefix_table"], prefix_len=s["prefix_len"], table=s["table"],
                lens=s["lens"], out=torch.empty_like(s["q"]))
    mk.prefix_attention(**good)
    for bad in (dict(prefix_len=s["prefix_len"].long()), dict(prefix_len=i32([1, 2])), dict(prefix_table=s["prefix_table"].cpu()),
                dict(prefix_table=s["prefix_table"][:0]), dict(out=torch.empty_like(s["q"]).bfloat16()), dict(lens=s["lens"][:1]),
                dict(prefix_table=s["prefix_table"][::2]), dict(k_pages=s["k"].bfloat16())):
        with pytest.raises((ValueError, mk.MKError)):
            mk.prefix_attention(**dict(good, **bad))
    d = draft_inputs(2, 3, 50, F32)
    good = dict(logits=d["logits"], tokens=d["tokens"], noise=d["noise"], uniforms=d["uniforms"], accept_out=i32([[0, 0]] * 3))
    mk.verify_drafts(**good)
    for bad in (dict(logits=d["logits"][:5]), dict(tokens=d["tokens"].long()), dict(noise=d["noise"][:, :49]), dict(uniforms=None),
                dict(uniforms=d["uniforms"][:, :1]), dict(accept_out=i32([[0, 0]] * 2)), dict(draft_logits=d["logits"]),
                dict(logits=d["logits"].double()), dict(draft_logits=d["draft_logits"].half()), dict(logprobs=torch.zeros(2, 2, device=DEV))):
        with pytest.raises((ValueError, mk.MKError)):
            mk.verify_drafts(**dict(good, **bad))
