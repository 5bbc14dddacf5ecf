"""GPU: the serving operators against plain implementations in 64 bits.

Tolerances are derived, not fitted. A value that is rounded once to type t is off by at most half a step: eps_t / 2 of
its size (bf16 2^-8, fp16 2^-11, e4m3 2^-4), or half of the smallest subnormal. What the kernels compute in fp32
before that is bounded from the number and size of its terms (written at each check)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from decode_megakernel_04_gb300 import _build
    _build.build()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def half_step(dtype, x):
    """Half a step of dtype at the sizes |x| (fp64)."""
    if dtype is E4M3:
        return torch.clamp(x.abs() * 2.0 ** -4, min=2.0 ** -10)
    tiny = {BF16: 2.0 ** -134, F16: 2.0 ** -25}[dtype]  # half of the smallest subnormal
    return torch.clamp(x.abs() * (torch.finfo(dtype).eps / 2), min=tiny)


# ---- page tables ----------------------------------------------------------------------------------------------------

def tables_reference(table, held, start, count, ring, state, page, n_pages, places):
    """The definition, request by request. Returns a dict, or the status when the step is refused."""
    B, max_pages = table.shape
    most = max_pages * page
    head, free = state
    bad = not (0 <= head < ring.size and 0 <= free <= ring.size)
    for h, s, c in zip(held, start, count):
        bad |= h < 0 or h > most or s < 0 or s > h or c < 0 or s + c > most
    if bad:
        return 2
    have = [-(-h // page) for h in held]
    need = [-(-(s + c) // page) for s, c in zip(start, count)]
    pops = sum(max(0, n - h) for h, n in zip(have, need))
    pushes = sum(max(0, h - n) for h, n in zip(have, need))
    why = (4 if pops > free else 0) | (8 if sum(count) > places else 0) | (2 if free + pushes > ring.size else 0)
    if why:
        return why
    table, out_ring = table.copy(), ring.copy()
    slots, pos, own = np.full(places, -1, np.int64), np.zeros(places, np.int32), np.full(places, -1, np.int32)
    starts, status, t, p, q = [0], 0, 0, 0, 0
    for b in range(B):
        for k in range(have[b], need[b]):
            table[b, k] = ring[(head + p) % ring.size]
            p += 1
        for k in range(need[b], have[b]):
            out_ring[(head + free + q) % ring.size] = table[b, k]
            q += 1
        for x in range(start[b], start[b] + count[b]):
            pg = table[b, x // page]
            if 0 <= pg < n_pages:
                slots[t] = int(pg) * page + x % page
            else:
                status |= 1
            pos[t], own[t] = x, b
            t += 1
        starts.append(t)
    return dict(table=table, ring=out_ring, ring_state_out=np.array([(head + p) % ring.size, free - p + q]), slots=slots,
                positions=pos, owners=own, starts=np.array(starts), lens=np.array(start) + np.array(count),
                status=np.array([status]))


def run_tables(table, held, start, count, ring, state, page, n_pages, places, in_place=False, stream=None):
    from decode_megakernel_04_gb300 import page_tables
    B = len(held)
    wide = torch.full((B, table.shape[1] + 3), -7, dtype=torch.int32, device=DEV)  # rows inside a wider table
    t = wide[:, :table.shape[1]]
    t.copy_(torch.from_numpy(table))
    o = dict(table=t, ring=torch.from_numpy(ring).to(DEV), slots=torch.full((places,), 99, dtype=torch.int64, device=DEV),
             positions=i32([99] * places), owners=i32([99] * places), starts=i32([99] * (B + 1)), status=i32([0]))
    h, st = i32(held), i32(state)
    o["lens"] = h if in_place else i32([99] * B)
    o["ring_state_out"] = st if in_place else i32([99, 99])
    page_tables(t, h, i32(start), i32(count), o["ring"], st, page, n_pages, slots=o["slots"], positions=o["positions"],
                owners=o["owners"], starts=o["starts"], lens=o["lens"],
                ring_state_out=None if in_place else o["ring_state_out"], status=o["status"], stream=stream)
    torch.cuda.synchronize()
    assert (wide[:, table.shape[1]:] == -7).all()
    return {k: v.cpu().numpy() for k, v in o.items()}


def draw_tables(rng, B, page, max_pages, kind):
    most = max_pages * page
    held, start, count = [], [], []
    for b in range(B):
        h = int(rng.integers(0, most + 1))
        what = rng.integers(0, 4) if kind == "mixed" else {"decode": 0, "end": 2}[kind]
        if what == 0:
            s, c = h - min(h, int(rng.integers(0, 5))), 1
        elif what == 1:
            s, c = h, int(rng.integers(0, most + 1))
        elif what == 2:
            s, c = 0, 0
        else:
            s, c = h, 0
        held.append(h), start.append(s), count.append(min(c, most - s))
    return held, start, count


def make_pool(rng, held, page, max_pages, n_pages, extra):
    B = len(held)
    ids = rng.permutation(n_pages).astype(np.int32)
    table, at = np.full((B, max_pages), -1, np.int32), 0
    for b, h in enumerate(held):
        n = -(-h // page)
        table[b, :n] = ids[at:at + n]
        at += n
    size = n_pages + extra
    head = int(rng.integers(0, size))
    ring = np.full(size, -1, np.int32)
    free = n_pages - at
    ring[(head + np.arange(free)) % size] = ids[at:]
    return table, ring, [head, free]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B, page, max_pages, kind", [
    (1, 64, 4, "decode"), (1, 1, 5, "mixed"), (3, 16, 9, "mixed"), (37, 7, 12, "mixed"), (513, 4, 6, "mixed"),
    (64, 16, 40, "end"), (1100, 3, 3, "mixed"), (4096, 2, 3, "mixed"), (9, 128, 30, "mixed")])
def test_page_tables(B, page, max_pages, kind, in_place):
    rng = np.random.default_rng(B * 1000 + page)
    held, start, count = draw_tables(rng, B, page, max_pages, kind)
    n_pages = 2 * B * max_pages + 3
    table, ring, state = make_pool(rng, held, page, max_pages, n_pages, int(rng.integers(0, 4)))
    places = sum(count) + (B % 3)
    want = tables_reference(table, held, start, count, ring, state, page, n_pages, places)
    got = run_tables(table, held, start, count, ring, state, page, n_pages, places, in_place)
    for k, v in want.items():
        assert np.array_equal(got[k], v), k


@pytest.mark.parametrize("change, why", [
    (dict(held=[5, -1, 9]), 2), (dict(start=[5, 5, 9]), 2), (dict(count=[1, -1, 0]), 2), (dict(count=[1, 100, 0]), 2),
    (dict(held=[5, 3, 33]), 2), (dict(state=[0, 0]), 4), (dict(places=3), 8), (dict(state=[99, 3]), 2),
    (dict(state=[0, -1]), 2), (dict(state=[0, 40]), 2), (dict(start=[0, 0, 0], count=[0, 0, 0], state=[0, 20]), 2),
    (dict(state=[0, 0], places=1), 12)])
def test_page_tables_refused_step_changes_nothing(change, why):
    a = dict(held=[5, 3, 9], start=[5, 3, 9], count=[4, 14, 1], state=[2, 8], places=20, page=8)
    a.update(change)
    ring = np.arange(20, dtype=np.int32)
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    n_pages = 20
    assert tables_reference(table, a["held"], a["start"], a["count"], ring, a["state"], 8, n_pages, a["places"]) == why
    for in_place in (False, True):
        got = run_tables(table, a["held"], a["start"], a["count"], ring, a["state"], 8, n_pages, a["places"], in_place)
        assert got["status"][0] == why
        assert np.array_equal(got["table"], table) and np.array_equal(got["ring"], ring)
        assert np.array_equal(got["ring_state_out"], a["state"]) and np.array_equal(got["lens"], a["held"])
        assert (got["slots"] == -1).all() and (got["positions"] == 0).all() and (got["owners"] == -1).all()
        assert (got["starts"] == 0).all()


def test_page_tables_with_the_most_places():
    """2^31 - 1 places (17 GB of slots), in a step that is taken and in one that is refused."""
    from decode_megakernel_04_gb300 import page_tables
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 20 GB")
    slots = torch.empty(2 ** 31 - 1, dtype=torch.int64, device=DEV)
    for count, why, first in ((3, 0, [0, 1, 2, -1]), (-1, 2, [-1] * 4)):
        slots.fill_(7)
        t, status, starts = i32([[-1, -1]]), i32([0]), i32([9, 9])
        page_tables(t, i32([0]), i32([0]), i32([count]), i32([0, 1, 2, 3]), i32([0, 4]), 4, 4, slots=slots, starts=starts, status=status)
        assert status.item() == why and slots[:4].tolist() == first and starts.tolist() == [0, max(0, count)]
        for part in slots[4:].split(1 << 28):
            assert (part == -1).all()
    with pytest.raises(ValueError):
        page_tables(t, i32([0]), i32([0]), i32([0]), i32([0, 1, 2, 3]), i32([0, 4]), 4, 4, slots=slots[:1].expand(2 ** 31))


def test_page_tables_bad_page_ids():
    table = np.array([[3, 77, -1], [4, 5, -1]], np.int32)
    ring = np.array([6, -2, 8, 9, 10, 11, 12, 13], np.int32)
    args = (table, [9, 8], [7, 8], [2, 3], ring, [1, 4], 4, 8, 8)  # request 0's page 1 and the first free page are bad
    want, got = tables_reference(*args), run_tables(*args)
    assert want["status"][0] == 1 and (want["slots"] == -1).sum() > 3
    for k, v in want.items():
        assert np.array_equal(got[k], v), k


def test_page_tables_optional_outputs():
    from decode_megakernel_04_gb300 import page_tables
    t, st = i32([[0, -1], [1, -1]]), i32([0, 2])
    slots = torch.full((3,), 9, dtype=torch.int64, device=DEV)
    page_tables(t, i32([4, 2]), i32([4, 2]), i32([1, 2]), i32([2, 3, 0, 0]), st, 4, 4, slots=slots)
    assert slots.tolist() == [8, 6, 7] and t.tolist() == [[0, 2], [1, -1]] and st.tolist() == [1, 1]


# ---- per-head norm, rotation, append ---------------------------------------------------------------------------------

def rotate(x, gain, eps, pos, inv):
    """fp64: norm (gain None: none) and rotate-half."""
    x = x.double()
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gain.double()
    if inv is None:
        return x
    a = pos.double()[:, None, None] * inv
    h = inv.numel()
    u, v = x[..., :h], x[..., h:2 * h]
    return torch.cat([u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin(), x[..., 2 * h:]], -1)


def check_rounded(got, want, dtype, what, slack):
    """got is `want` rounded once to dtype after an error of at most `slack`."""
    err = (got.double() - want).abs()
    bound = slack + half_step(dtype, want.abs() + slack)
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"


def qk_slack(want):
    """The fp32 part: the mean square (relative 16 x 2^-24), root, reciprocal and products (6 x 2^-24), sine and cosine
    (absolute 2^-21: their own error and 2^-32 turns of angle), two products and a sum; of the head's largest value."""
    return 2.0 ** -19 * want.abs().amax(-1, keepdim=True).clamp(min=1e-30)


CASES_QK = [  # tokens, hq, hkv, d, rope, dtype, cache, page, gains
    (1, 48, 8, 128, 128, BF16, BF16, 16, True), (1, 1, 1, 16, 16, F16, F16, 1, True), (7, 24, 4, 256, 64, BF16, E4M3, 64, True),
    (33, 4, 1, 64, 64, F16, E4M3, 16, True), (5, 6, 2, 80, 40, BF16, BF16, 24, True), (130, 5, 5, 192, 192, F16, F16, 7, True),
    (3, 8, 2, 128, 0, BF16, BF16, 16, True), (17, 3, 1, 128, 32, BF16, None, 1, False), (2, 4, 4, 112, 112, BF16, E4M3, 5, False),
    (700, 24, 4, 256, 256, BF16, BF16, 64, True), (2600, 48, 8, 128, 128, F16, F16, 16, True), (9, 2, 1, 48, 8, F16, F16, 3, True),
    (64, 9, 3, 240, 120, BF16, E4M3, 16, True)]


def qk_inputs(n, hq, hkv, d, rope, dtype, cache, page, gains, seed=0):
    g = gen(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    qkv = (2 * rn(n, hq + 2 * hkv, d)).to(dtype)
    s = dict(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], pos=torch.randint(0, 2 ** 31 - 1, (n,), generator=g, device=DEV).to(torch.int32))
    s["pos"][0] = 0
    s["inv"] = None if rope == 0 else (1e4 ** (-torch.arange(0, rope, 2, dtype=torch.float64) / rope)).to(DEV)
    s["qg"], s["kg"] = ((1 + 0.3 * rn(d)).to(dtype), (1 + 0.3 * rn(d)).to(dtype)) if gains else (None, None)
    if cache is not None:
        n_pages = -(-n // page) + 2
        perm = torch.randperm(n_pages * page, generator=g, device=DEV)
        s["slots"] = perm[:n].clone()
        s["slots"][::5] = -1
        s["untouched"] = torch.ones(n_pages * page, dtype=torch.bool, device=DEV)
        s["untouched"][s["slots"][s["slots"] >= 0]] = False
        # [page][place][head] in memory, padded: the strides are not those of a contiguous cache
        raw = rn(2, n_pages, page, hkv, d + 16).to(cache)
        s["pages"] = [r[..., :d].transpose(1, 2) for r in raw]
        s["before"] = [p.float().clone() for p in s["pages"]]
        s["scales"] = [0.01 + 0.05 * torch.rand(hkv, generator=g, device=DEV) for _ in range(2)] if cache is E4M3 else [None, None]
    return s


@pytest.mark.parametrize("case", CASES_QK, ids=str)
def test_qk_norm_rope(case):
    from decode_megakernel_04_gb300 import qk_norm_rope
    n, hq, hkv, d, rope, dtype, cache, page, gains = case
    s = qk_inputs(*case)
    q_out = torch.empty(n, hq + 1, d, dtype=dtype, device=DEV)[:, 1:]  # padded token stride
    k_out = torch.empty(n, hkv, d, dtype=dtype, device=DEV)
    status = i32([0])
    kw = {} if cache is None else dict(v=s["v"], k_pages=s["pages"][0], v_pages=s["pages"][1], slots=s["slots"],
                                      k_scale=s["scales"][0], v_scale=s["scales"][1])
    qk_norm_rope(s["q"], s["k"], s["pos"], s["inv"], q_out, k_out=k_out, q_gain=s["qg"], k_gain=s["kg"], eps=1e-5,
                 status=status, **kw)
    torch.cuda.synchronize()
    wq, wk = rotate(s["q"], s["qg"], 1e-5, s["pos"], s["inv"]), rotate(s["k"], s["kg"], 1e-5, s["pos"], s["inv"])
    check_rounded(q_out, wq, dtype, "q", qk_slack(wq))
    check_rounded(k_out, wk, dtype, "k", qk_slack(wk))
    assert status.item() == 0
    if cache is None:
        return
    keep = s["slots"] >= 0
    for pages, before, scale, want in zip(s["pages"], s["before"], s["scales"], (wk, s["v"].double())):
        flat = pages.float().transpose(1, 2).reshape(-1, hkv, d)
        assert torch.equal(flat[s["untouched"]], before.transpose(1, 2).reshape(-1, hkv, d)[s["untouched"]])
        if cache is E4M3:
            want = (want / scale.double()[:, None]).clamp(-448, 448)
        slack = qk_slack(want) if want.shape == wk.shape else 0
        check_rounded(flat[s["slots"][keep]], want[keep], cache, "cache", slack[keep])


@pytest.mark.parametrize("case", [c for c in CASES_QK if c[6] is not None], ids=str)
def test_qk_cached_values_are_exact(case):
    """Values are not normed or turned: a 16-bit cache holds them bit for bit, an e4m3 cache the code of the fp32 quotient."""
    from decode_megakernel_04_gb300 import qk_norm_rope
    n, hq, hkv, d, rope, dtype, cache, page, gains = case
    s = qk_inputs(*case, seed=1)
    qk_norm_rope(s["q"], s["k"], s["pos"], s["inv"], torch.empty(n, hq, d, dtype=dtype, device=DEV), q_gain=s["qg"], k_gain=s["kg"],
                 v=s["v"], k_pages=s["pages"][0], v_pages=s["pages"][1], slots=s["slots"], k_scale=s["scales"][0], v_scale=s["scales"][1])
    keep = (s["slots"] >= 0).cpu()
    got = s["pages"][1].float().cpu().transpose(1, 2).reshape(-1, hkv, d)[s["slots"].cpu()[keep]]
    want = s["v"].float().cpu()[keep]
    if cache is E4M3:
        want = (want / s["scales"][1].cpu()[:, None]).clamp(-448, 448).to(E4M3).float()
    assert torch.equal(got, want)


def test_qk_e4m3_values_halfway_between_two_codes():
    """value / scale exactly between two e4m3 codes goes to the even one. (17 .. 31) / 16 x 2^e are such, for odd numerators,
    and their products with 3, 5 and 7 are bf16 values."""
    from decode_megakernel_04_gb300 import qk_norm_rope
    half = torch.tensor([(m if e % 2 else -m) / 16 * 2.0 ** e for e in range(-5, 8) for m in range(17, 32, 2)])
    n, hkv, d = -(-half.numel() // 16), 3, 16
    half = torch.cat([half, half.new_ones(n * d - half.numel())]).view(n, 1, d)
    scale = torch.tensor([3.0, 5.0, 7.0]) / 64
    v = (half * scale[:, None]).to(BF16)
    assert torch.equal(v.double(), half.double() * scale.double()[:, None])
    kp, vp = (torch.zeros(n, hkv, 1, d, device=DEV).to(E4M3) for _ in range(2))
    q = torch.zeros(n, 1, d, dtype=BF16, device=DEV)
    qk_norm_rope(q, v.to(DEV), None, None, q, v=v.to(DEV), k_pages=kp, v_pages=vp, slots=torch.arange(n, device=DEV),
                 k_scale=scale.to(DEV), v_scale=scale.to(DEV))
    want = half.expand(n, hkv, d).to(E4M3).float()
    for got in (kp, vp):  # (without norm and rotation keys are stored as they come too)
        assert torch.equal(got[:, :, 0].float().cpu(), want)


@pytest.mark.parametrize("scale", [1e-30, 1e-44, 3e-5, 0.7, 1e25, -2.0])
def test_qk_e4m3_scales_and_values_of_any_size(scale):
    """Quotients of every size: past 448 (infinite ones too) 448, NaN NaN, down to 0; scales that fp32 has no reciprocal of."""
    from decode_megakernel_04_gb300 import qk_norm_rope
    x = torch.tensor([0.0, -0.0, 1.0, -1.0, 447.0, 448.0, 463.0, 465.0, -480.0, 511.0, 512.0, 1e4, 3e38, float("inf"), float("-inf"),
                      float("nan"), 2.0 ** -6, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -10, 2.0 ** -11, 1e-20, 1e-38, 1e-40])
    x = torch.cat([x, x * 0.3, x * 1e-3, x * scale, x * scale * 0.7, (x.double() * scale * 1.1).float()]).to(BF16)
    n, d = x.numel() // 16, 16
    v = x.view(n, 1, d)
    kp, vp = (torch.zeros(n, 1, 1, d, device=DEV).to(E4M3) for _ in range(2))
    q, sc = torch.zeros(n, 1, d, dtype=BF16, device=DEV), torch.tensor([scale])
    qk_norm_rope(q, v.to(DEV), None, None, q, v=v.to(DEV), k_pages=kp, v_pages=vp, slots=torch.arange(n, device=DEV),
                 k_scale=sc.to(DEV), v_scale=sc.to(DEV))
    want = (v.float() / sc[:, None]).clamp(-448, 448).to(E4M3).float()
    for got in (kp, vp):
        assert torch.equal(got[:, :, 0].float().cpu().nan_to_num(1000.0), want.nan_to_num(1000.0))


def test_qk_in_place_and_streams():
    from decode_megakernel_04_gb300 import qk_norm_rope
    s = qk_inputs(300, 24, 4, 128, 128, BF16, None, 1, True)
    q, k = s["q"].clone(), s["k"].clone()
    a, b = torch.empty_like(q), torch.empty_like(k)
    qk_norm_rope(s["q"], s["k"], s["pos"], s["inv"], a, k_out=b, q_gain=s["qg"], k_gain=s["kg"])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    qk_norm_rope(q, k, s["pos"], s["inv"], q, k_out=k, q_gain=s["qg"], k_gain=s["kg"], stream=st.cuda_stream)
    st.synchronize()
    assert torch.equal(a, q) and torch.equal(b, k)


def test_qk_bad_slots_are_flagged_and_not_stored():
    from decode_megakernel_04_gb300 import qk_norm_rope
    s = qk_inputs(4, 2, 2, 64, 64, BF16, BF16, 4, True)
    n_slots = s["pages"][0].shape[0] * 4
    slots = torch.tensor([n_slots, -5, 2 ** 40, n_slots - 1], device=DEV)
    status = i32([0])
    qk_norm_rope(s["q"], s["k"], s["pos"], s["inv"], torch.empty_like(s["q"].contiguous()), v=s["v"], k_pages=s["pages"][0],
                 v_pages=s["pages"][1], slots=slots, status=status)
    assert status.item() == 1
    for pages, before in zip(s["pages"], s["before"]):
        same = (pages.float() == before).transpose(1, 2).reshape(n_slots, -1).all(1)
        assert same[:-1].all() and not same[-1]


def test_qk_special_values_stay_in_their_head():
    from decode_megakernel_04_gb300 import qk_norm_rope
    s = qk_inputs(3, 4, 2, 128, 128, BF16, None, 1, True)
    q = s["q"].clone()
    q[1, 2, 5] = float("nan")
    q[2, 0] = 0
    out = torch.empty_like(q)
    qk_norm_rope(q, s["k"], s["pos"], s["inv"], out, q_gain=s["qg"], k_gain=s["kg"])
    assert out[1, 2].isnan().all() and (out[2, 0] == 0).all()
    out[1, 2] = 0
    assert out.isfinite().all()


# ---- paged attention ---------------------------------------------------------------------------------------------------

def attention_inputs(lens, R, hq, hkv, d, page, dtype, cache, seed=0, layout="head", poison=True, max_pages=None):
    g = gen(seed)
    B = len(lens)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    used = [-(-max(0, n) // page) for n in lens]
    n_pages = sum(used) + 3
    ids = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    mp = max_pages or max(1, max(used))
    table = torch.full((B, mp + 2), 2 ** 30, dtype=torch.int32, device=DEV)[:, :mp]  # unused entries are no pages
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = ids[at:at + n]
        at += n
    shape = {"head": (n_pages, hkv, page, d), "place": (n_pages, page, hkv, d), "padded": (n_pages, hkv, page + 1, d + 16)}[layout]
    kv = [(rn(*shape) * 1.5).to(cache) for _ in range(2)]
    if layout == "place":
        kv = [x.transpose(1, 2) for x in kv]
    if layout == "padded":
        kv = [x[:, :, :page, :d] for x in kv]
    if poison:  # everything no request sees: other pages, places behind the length
        seen = torch.zeros(n_pages, page, dtype=torch.bool, device=DEV)
        for b, n in enumerate(lens):
            p = torch.arange(max(0, n), device=DEV)
            seen[table[b].long()[p // page], p % page] = True
        for x in kv:
            f = x.float()
            f[(~seen)[:, None, :, None].expand_as(x)] = float("nan")
            x.copy_(f.to(cache))
    q = (rn(B, R + 1, hq, d)).to(dtype)[:, 1:]  # a batch stride of its own
    scales = [0.2 + rn(hkv).abs() for _ in range(2)] if cache is E4M3 else [None, None]
    return dict(q=q, k=kv[0], v=kv[1], table=table, lens=i32(lens), ks=scales[0], vs=scales[1], page=page)


def attention_reference(s, scale):
    """fp64, row by row. Returns out, lse and the sum of p |v| (for the bounds) with the largest sum |q k| of a row."""
    q = s["q"].double()
    B, R, hq, d = q.shape
    hkv, page = s["k"].shape[1], s["page"]
    G = hq // hkv
    out, av = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((B, R, hq), -math.inf, dtype=torch.float64, device=DEV)
    qk = torch.zeros((B, R, hq), dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        n = max(0, n)
        pages = s["table"][b, :-(-n // page)].long()
        k = s["k"][pages].double().transpose(0, 1).reshape(hkv, -1, d)[:, :n]
        v = s["v"][pages].double().transpose(0, 1).reshape(hkv, -1, d)[:, :n]
        if s["ks"] is not None:
            k, v = k * s["ks"].double()[:, None, None], v * s["vs"].double()[:, None, None]
        for r in range(R):
            m = n - (R - 1 - r)
            if m <= 0:
                continue
            x = q[b, r].view(hkv, G, d)
            z = torch.matmul(x, k[:, :m].transpose(1, 2)) * scale
            p = torch.softmax(z, -1)
            out[b, r] = torch.matmul(p, v[:, :m]).view(hq, d)
            av[b, r] = torch.matmul(p, v[:, :m].abs()).view(hq, d)
            lse[b, r] = torch.logsumexp(z, -1).view(hq)
            qk[b, r] = (torch.matmul(x.abs(), k[:, :m].abs().transpose(1, 2)).amax(-1) * abs(scale)).view(hq)
    return out, lse, av, qk


def run_attention(s, scale=None, status=None, **kw):
    from decode_megakernel_04_gb300 import paged_attention
    B, R, hq, d = s["q"].shape
    out = torch.full((B, R, hq, d + 8), 7.0, dtype=s["q"].dtype, device=DEV)
    lse = torch.full((B, R, hq), 7.0, device=DEV)
    paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], out[..., :d], scale=scale, lse=lse, k_scale=s["ks"],
                    v_scale=s["vs"], status=status, **kw)
    torch.cuda.synchronize()
    assert (out[..., d:] == 7).all()
    return out[..., :d], lse


def check_attention(s, got, lse, scale, what=""):
    """Bounds. A score is a sum of D products in fp32: off by (D + 4) 2^-23 of sum |q k| (natural units; e4m3: another
    2^-20 of it for queries rounded to fp16 against their row's largest). That moves a probability by that share,
    exp2 and its argument by 2^-21; probabilities enter the product off by 2^-16 (two 16-bit values; bf16 pairs leave
    2^-18, fp16 pairs less) or, e4m3, 2^-11 and 2^-25 absolute against a largest of 1. Numerator and denominator each
    take it, the sums over n keys n 2^-23 more, and the result is rounded once."""
    d = s["q"].shape[-1]
    out, l64, av, qk = attention_reference(s, scale)
    n = s["lens"].clamp(min=0).double()[:, None, None]
    e4 = s["ks"] is not None
    ds = qk * ((d + 4) * 2.0 ** -23 + (2.0 ** -20 if e4 else 0))
    rel = 2 * (ds + 2.0 ** -21 + n * 2.0 ** -23) + (2.0 ** -11 if e4 else 2.0 ** -16)
    slack = rel[..., None] * av
    if e4:
        v_max = s["v"].float().nan_to_num().abs().amax((0, 2, 3)).mul(s["vs"]).max().double()
        slack = slack + (n * 2.0 ** -25)[..., None] * v_max
    assert not got.isnan().any(), what
    empty = l64 == -math.inf
    assert (got[empty] == 0).all() and (lse[empty] == -math.inf).all(), what
    check_rounded(got, out, s["q"].dtype, what + " out", slack)
    err = (lse.double() - l64).abs()[~empty]
    bound = (ds + 2.0 ** -20 + n * 2.0 ** -23 + l64.abs() * 2.0 ** -22)[~empty]
    assert err.numel() == 0 or (err <= bound).all(), f"{what} lse {(err / bound).max().item()}"


CASES_ATT = [  # lens, R, hq, hkv, d, page, dtype, cache, layout
    ([1], 1, 1, 1, 64, 16, BF16, BF16, "head"),
    ([0, 1, 63, 64, 65, 128, 129], 1, 6, 1, 128, 16, BF16, BF16, "head"),
    ([300, 0, 17], 1, 4, 1, 64, 16, F16, F16, "place"),
    ([5, 700, 33], 1, 24, 4, 256, 64, BF16, BF16, "padded"),
    ([1500, 3, 64], 1, 8, 8, 128, 1, F16, F16, "head"),
    ([2000], 1, 16, 1, 128, 24, BF16, BF16, "place"),
    ([4096], 1, 24, 4, 256, 64, BF16, BF16, "head"),
    ([777, 1023, 5], 1, 36, 2, 128, 32, BF16, BF16, "head"),     # 18 rows of a kv head: two 16-row tiles
    ([900, 2], 1, 40, 1, 64, 256, F16, F16, "head"),             # 40 rows
    ([500, 70], 1, 72, 1, 128, 16, BF16, BF16, "head"),          # 72 rows: two blocks
    ([900, 128, 5], 1, 32, 1, 64, 16, BF16, BF16, "place"),      # 64 wide, 32 and 64 rows
    ([600, 129], 4, 16, 1, 64, 16, F16, F16, "head"),
    ([500, 70], 1, 100, 1, 256, 16, BF16, BF16, "head"),         # 100 rows, 256 wide
    ([8, 1, 64, 71, 0, 3, 1000], 8, 6, 1, 128, 16, BF16, BF16, "head"),
    ([9, 130, 64, 2], 5, 24, 4, 256, 64, BF16, BF16, "place"),
    ([65, 66, 67, 129], 3, 4, 1, 64, 16, F16, F16, "padded"),
    ([300, 12], 2, 48, 8, 128, 16, BF16, BF16, "head"),
    ([100], 20, 2, 1, 128, 16, BF16, BF16, "head"),              # a longer block of rows
    ([3, 64, 1000, 0, 127], 1, 48, 8, 128, 32, BF16, E4M3, "head"),
    ([3, 64, 1000, 0, 127], 1, 4, 1, 64, 16, F16, E4M3, "place"),
    ([700, 33], 1, 24, 4, 256, 64, BF16, E4M3, "padded"),
    ([8, 1, 70, 600], 8, 6, 1, 128, 16, BF16, E4M3, "head"),
    ([9, 140], 8, 12, 2, 256, 24, F16, E4M3, "head"),
    ([130, 260], 3, 40, 2, 64, 16, BF16, E4M3, "place"),
    ([1, 200], 1, 3, 1, 16, 16, BF16, BF16, "head"),             # narrow and odd widths
    ([90, 200], 2, 6, 2, 80, 16, F16, F16, "padded"),
    ([90, 200], 1, 6, 2, 112, 8, BF16, E4M3, "head"),
    ([90, 200], 2, 6, 2, 48, 8, BF16, E4M3, "head"),
    ([90, 333], 1, 6, 2, 192, 16, BF16, BF16, "head"),
    ([90, 333], 4, 6, 2, 240, 16, F16, E4M3, "head"),
    ([20000, 1], 1, 8, 1, 128, 64, BF16, BF16, "head"),          # cut into many parts
    ([9000, 100, 0, 2500], 8, 12, 2, 128, 16, BF16, BF16, "head"),
    ([30000], 1, 2, 1, 64, 16, F16, F16, "head"),
    ([12000, 50], 1, 6, 1, 256, 32, F16, E4M3, "head"),
    ([i * 7 % 400 for i in range(300)], 1, 4, 1, 64, 16, F16, F16, "head"),
    # keys that only some rows see on both sides of a tile's end
    ([128, 129, 131, 135, 136, 255, 256, 257, 260, 1025], 8, 6, 1, 128, 16, BF16, BF16, "head"),
    ([128, 129, 133, 256, 258, 7], 8, 3, 1, 256, 64, F16, F16, "place"),
    ([140, 128, 143, 15, 16, 17, 300], 16, 2, 1, 128, 16, BF16, BF16, "head"),   # 32 rows of 16 new tokens
    ([140, 33], 17, 2, 1, 128, 16, F16, F16, "head"),
    ([2300, 700], 4, 16, 1, 256, 32, BF16, BF16, "head"),        # 64 rows, 256 wide
    ([i * 37 % 900 for i in range(90)], 2, 24, 4, 128, 16, BF16, BF16, "place"),
]


@pytest.mark.parametrize("wide", [False, True], ids=["", "wide"])
@pytest.mark.parametrize("case", CASES_ATT, ids=lambda c: f"{len(c[0])}x{max(c[0])}-" + "-".join(str(x) for x in c[1:]))
def test_paged_attention(case, wide):
    """Each case with a table as wide as its longest request (small calls: clusters) and with one for long requests (the
    line of tiles cut into pieces, joined by a second launch)."""
    from decode_megakernel_04_gb300 import paged_attention_workspace
    lens, R, hq, hkv, d, page, dtype, cache, layout = case
    s = attention_inputs(lens, R, hq, hkv, d, page, dtype, cache, layout=layout, max_pages=1 << 20 >> (page.bit_length() - 1) if wide else None)
    assert not wide or paged_attention_workspace(s["q"], s["k"], s["table"]) > 0
    status = i32([0])
    got, lse = run_attention(s, status=status)
    check_attention(s, got, lse, d ** -0.5)
    assert status.item() == 0


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_attention_hidden_rows_do_not_leak(cache):
    """A verify block whose later rows' keys and values are NaN and infinite: earlier rows do not see them."""
    lens, R = [70, 64, 9, 130], 8
    s = attention_inputs(lens, R, 6, 1, 128, 16, BF16, cache, seed=3)
    clean, cl = run_attention(s, scale=0.1)
    for b, n in enumerate(lens):
        for back, bad in ((1, float("nan")), (2, float("inf")), (4, -448.0 if cache is E4M3 else float("-inf"))):
            p = n - back
            for x in (s["k"], s["v"]):
                f = x[s["table"][b, p // 16].long(), :, p % 16].float().fill_(bad)
                x[s["table"][b, p // 16].long(), :, p % 16] = f.to(cache)
    got, lse = run_attention(s, scale=0.1)
    free = [r for r in range(R) if R - 1 - r >= 4]  # rows that end before every bad key
    assert torch.equal(got[:, free], clean[:, free]) and torch.equal(lse[:, free], cl[:, free])
    assert got[:, -1].isnan().all()


def test_attention_scores_of_any_size():
    """Large scores (a softmax of one key), and the lowest values of the type as keys."""
    s = attention_inputs([200, 65], 1, 4, 1, 128, 16, BF16, BF16, seed=5)
    got, lse = run_attention(s, scale=30.0)
    check_attention(s, got, lse, 30.0)
    s["k"].fill_(torch.finfo(BF16).min)
    s["q"].zero_()
    s["q"][..., 0] = 1.0
    got, lse = run_attention(s, scale=1e-3)  # equal scores of -3.4e35: the mean of the values
    out, _, av, _ = attention_reference(s, 1e-3)
    check_rounded(got, out, BF16, "equal scores", (300 * 2.0 ** -23 + 2.0 ** -16) * av)


@pytest.mark.parametrize("width", [None, 50000])
@pytest.mark.parametrize("cache, d", [(BF16, 128), (BF16, 256), (F16, 64), (E4M3, 128)])
def test_attention_scores_that_grow_and_that_begin_at_minus_infinity(cache, d, width):
    """A maximum that moves with every tile; and requests whose first keys give every row -infinity."""
    s = attention_inputs([1500, 300, 1], 2, 6, 1, d, 16, F16 if cache is F16 else BF16, cache, seed=21, poison=False, max_pages=width)
    for b, n in enumerate([1500, 300, 1]):
        p = torch.arange(n, device=DEV)
        at = s["table"][b].long()[p // 16], slice(None), p % 16
        s["k"][at] = (s["k"][at].float() * (p / 400)[:, None, None]).to(cache)
    got, lse = run_attention(s, scale=0.5)
    check_attention(s, got, lse, 0.5, "growing")
    if cache is E4M3:
        return  # no infinity in that type
    s["q"][..., 0] = 1.0
    at = s["table"][0].long()[torch.arange(400, device=DEV) // 16], slice(None), torch.arange(400, device=DEV) % 16, 0
    s["k"][at] = float("-inf")
    s["k"][s["table"][2, 0].long(), :, 0, 0] = float("-inf")  # the request of one key: nothing is left of it
    got, lse = run_attention(s, scale=0.5)
    assert (got[2] == 0).all() and (lse[2] == -math.inf).all()
    out, l64, av, _ = attention_reference(s, 0.5)
    check_rounded(got[:2], out[:2], s["q"].dtype, "minus infinity", 2.0 ** -10 * av[:2])
    assert (lse[:2].double() - l64[:2]).abs().max() < 2.0 ** -9


@pytest.mark.parametrize("width", [None, 50000])
@pytest.mark.parametrize("dtype, d", [(BF16, 128), (F16, 128), (BF16, 256)])
def test_attention_whole_tiles_of_minus_infinity_before_the_first_score(dtype, d, width):
    """Tiles whose keys give every row -infinity, with the only finite scores behind them."""
    s = attention_inputs([512, 256, 200], 2, 12, 2, d, 16, dtype, dtype, seed=31, poison=False, max_pages=width)
    s["q"][..., 0] = 1.0
    qk = attention_reference(s, 0.1)[3]  # at least that of the keys that are left
    for b, tiles in enumerate([(0, 2), (0,), (0,)]):
        for t in tiles:
            p = 128 * t + torch.arange(128, device=DEV)
            s["k"][s["table"][b].long()[p // 16], :, p % 16, 0] = -math.inf
    got, lse = run_attention(s, scale=0.1)
    out, l64, av, _ = attention_reference(s, 0.1)
    ds = qk * (d + 4) * 2.0 ** -23  # the bounds of check_attention
    check_rounded(got, out, dtype, "out", (2 * (ds + 2.0 ** -21 + 512 * 2.0 ** -23) + 2.0 ** -16)[..., None] * av)
    assert ((lse.double() - l64).abs() <= ds + 2.0 ** -20 + 512 * 2.0 ** -23 + l64.abs() * 2.0 ** -22).all()


@pytest.mark.parametrize("width", [None, 50000])
def test_attention_of_the_lowest_scores(width):
    """Equal scores of -3.4e35 in long and short calls: the mean of the values."""
    s = attention_inputs([300, 65], 2, 6, 1, 128, 16, BF16, BF16, seed=33, poison=False, max_pages=width)
    s["k"].fill_(torch.finfo(BF16).min)
    s["q"].zero_()
    s["q"][..., 0] = 1.0
    got, _ = run_attention(s, scale=1e-3)
    out, _, av, _ = attention_reference(s, 1e-3)
    check_rounded(got, out, BF16, "equal scores", (300 * 2.0 ** -23 + 2.0 ** -16) * av)


def sink_inputs(lens, hq, hkv, d, dtype, cache, max_pages, seed=41):
    """One key 14 to 18 above all the others of its request (natural units), with a value of zero: the result is what
    the others' small probabilities give. It comes first, or in the middle."""
    s = attention_inputs(lens, 1, hq, hkv, d, 16, dtype, cache, seed=seed, poison=False, max_pages=max_pages)
    if cache is E4M3:
        s["ks"].fill_(1.0), s["vs"].fill_(0.5)
    s["q"].mul_(0.125)
    s["q"][..., 0] = 4.0
    s["k"][..., 0] = 0.0
    s["v"].copy_((s["v"].float() * 0.25 + 1.0).to(cache))
    for b, n in enumerate(lens):
        p = n // 2 if b % 2 else 0
        at = s["table"][b, p // 16].long()
        s["k"][at, :, p % 16] = 0.0
        s["k"][at, :, p % 16, 0] = 14.0 + b % 5
        s["v"][at, :, p % 16] = 0.0
    return s


@pytest.mark.parametrize("lens, width", [([1500, 300, 1000, 700, 1301], None), ([4000] * 40 + [1300], 50000)], ids=["short", "long"])
@pytest.mark.parametrize("dtype, cache, d", [(F16, F16, 64), (F16, F16, 128), (F16, F16, 256), (F16, E4M3, 64), (BF16, E4M3, 128),
                                             (F16, E4M3, 128), (BF16, E4M3, 256), (BF16, BF16, 128)])
def test_attention_of_many_weak_keys_behind_a_strong_one(dtype, cache, d, lens, width):
    """Probabilities far below the largest count. The bound is check_attention's, without its absolute share for e4m3: a
    probability is off by a relative 2^-16 (e4m3: 2^-11) or by 2^-40 of the largest one."""
    s = sink_inputs(lens, 24, 8, d, dtype, cache, width)
    got, lse = run_attention(s, scale=0.25)
    out, l64, av, qk = attention_reference(s, 0.25)
    n = s["lens"].double()[:, None, None]
    e4 = cache is E4M3
    ds = qk * ((d + 4) * 2.0 ** -23 + (2.0 ** -20 if e4 else 0))
    rel = 2 * (ds + 2.0 ** -21 + n * 2.0 ** -23) + (2.0 ** -11 if e4 else 2.0 ** -16)
    v_max = s["v"].float().abs().max().double() * (0.5 if e4 else 1.0)
    check_rounded(got, out, dtype, "weak keys", rel[..., None] * av + (n * 2.0 ** -40)[..., None] * v_max)
    assert ((lse.double() - l64).abs() <= ds + 2.0 ** -20 + n * 2.0 ** -23 + l64.abs() * 2.0 ** -22).all()


@pytest.mark.parametrize("width", [None, 50000])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("R, hq", [(1, 24), (6, 48)])
def test_attention_over_e4m3_with_fp16_results_is_rounded_once(R, hq, d, width):
    """Scores of one exact product each, so that what is left is the rounding of the probabilities: a pair of fp16 values
    (2^-22), not one (2^-11, as much as the result's own). Scores, exponentials and sums as in check_attention."""
    lens = [1, 2, 3, 7, 12, 20, 33, 40, 130, 200]
    s = attention_inputs(lens, R, hq, 8, d, 16, F16, E4M3, seed=45, max_pages=width)
    s["ks"].fill_(1.0)
    one = torch.zeros_like(s["q"])
    one[..., 3] = s["q"][..., 3]
    s["q"].copy_(one)
    got, _ = run_attention(s, scale=0.5)
    out, l64, av, qk = attention_reference(s, 0.5)
    n = s["lens"].double()[:, None, None]
    rel = 2 * (qk * 2.0 ** -21 + 2.0 ** -21 + n * 2.0 ** -23) + 2.0 ** -22
    check_rounded(got, out, F16, "out", rel[..., None] * av)


def test_attention_lengths_and_pages_out_of_range():
    s = attention_inputs([40, 30, 20, 10], 1, 4, 2, 64, 8, BF16, BF16, seed=6, max_pages=5, poison=False)
    good, gl = run_attention(s)
    t = dict(s)
    t["lens"] = i32([40, -3, 400, 10])     # -3 counts as 0, 400 as 40 (5 pages of 8)
    t["table"] = s["table"].clone()
    t["table"][2, 3:] = t["table"][0, :2]
    u = dict(t)
    u["lens"] = i32([40, 0, 40, 10])
    status = i32([0])
    got, lse = run_attention(t, status=status)
    want, wl = run_attention(u)
    assert status.item() == 2 and torch.equal(got, want) and torch.equal(lse, wl)
    assert torch.equal(got[0], good[0]) and (got[1] == 0).all()
    # pages that do not exist: flagged, other requests untouched, keys and values read as zeros
    t = dict(s)
    t["table"] = s["table"].clone()
    t["table"][1, 0], t["table"][1, 1] = -1, 2 ** 31 - 1
    status = i32([0])
    got, lse = run_attention(t, status=status)
    assert status.item() == 1 and torch.equal(got[[0, 2, 3]], good[[0, 2, 3]]) and got.isfinite().all()


@pytest.mark.parametrize("width", [None, 50000])
def test_attention_repeats_bit_for_bit(width):
    s = attention_inputs([5000, 1, 800], 1, 12, 2, 128, 16, BF16, BF16, seed=7, max_pages=width)
    a, b = run_attention(s), run_attention(s)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # the same page listed twice is read twice
    t = dict(s)
    t["table"] = s["table"].clone()
    t["table"][0, 1] = t["table"][0, 0]
    got, lse = run_attention(t)
    check_attention(t, got, lse, 128 ** -0.5)


def test_attention_offsets_beyond_32_bits():
    """A cache whose pages lie more than 2^31 elements apart."""
    d, page = 128, 16
    stride = (2 ** 31 + 2 ** 20) // 2
    raw = torch.empty(2 * stride + 4 * page * d, dtype=BF16, device=DEV)
    k = raw.as_strided((3, 1, page, d), (stride, page * d, d, 1))
    v = raw.as_strided((3, 1, page, d), (stride, page * d, d, 1), 2 * page * d)
    g = gen(8)
    for x in (k, v):
        x.copy_(torch.randn(3, 1, page, d, generator=g, device=DEV).to(BF16))
    s = dict(q=torch.randn(1, 1, 4, d, generator=g, device=DEV).to(BF16), k=k, v=v, table=i32([[2, 0, 1]]), lens=i32([45]),
             ks=None, vs=None, page=page)
    got, lse = run_attention(s)
    check_attention(s, got, lse, d ** -0.5)


@pytest.mark.parametrize("width", [None, 50000])
def test_attention_in_graphs_and_on_streams(width):
    """Two captured graphs without a workspace of their own replay at the same time; each is right after its inputs
    change; and calls on a side stream, by torch's current stream or by the argument."""
    from decode_megakernel_04_gb300 import paged_attention, paged_attention_workspace
    sets = [attention_inputs([3000 + 500 * i, 40], 1, 8, 1, 128, 16, BF16, BF16, seed=9 + i, poison=False, max_pages=width) for i in range(2)]
    outs, graphs = [], []
    for s in sets:
        run_attention(s)  # the first call sets the kernel up
        o, l = torch.empty_like(s["q"].contiguous()), torch.empty(s["q"].shape[:3], device=DEV)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], o, lse=l)
        outs.append((o, l))
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in sets]
    for turn in range(3):
        for s in sets:
            s["q"].mul_(0.7)
            s["lens"].copy_(i32([2000 + turn, 41 - turn]))
        want = [run_attention(s) for s in sets]
        torch.cuda.synchronize()
        for _ in range(5):
            for st, gr in zip(streams, graphs):
                with torch.cuda.stream(st):
                    gr.replay()
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(outs, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)
    s = sets[0]
    ws = torch.empty(max(64, paged_attention_workspace(s["q"], s["k"], s["table"])), dtype=torch.uint8, device=DEV).fill_(255)
    for kw in (dict(stream=streams[1].cuda_stream), dict(stream=streams[1].cuda_stream, workspace=ws), dict(workspace=ws), dict(stream=0)):
        got = run_attention(s, **kw)
        assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[0][1])
    with torch.cuda.stream(streams[0]):
        got = run_attention(s)
    assert torch.equal(got[0], want[0][0])


@pytest.mark.parametrize("rows, hq, hkv, d, dtype, cache", [
    (1, 32, 8, 128, 0, 0), (8, 48, 8, 128, 0, 0), (1, 24, 4, 256, 1, 1), (1, 32, 8, 64, 0, 0), (1, 48, 8, 128, 0, 3), (1, 2, 1, 128, 1, 1), (17, 4, 2, 256, 0, 0)])
def test_attention_workspace_of_the_largest_call_fits_all(rows, hq, hkv, d, dtype, cache):
    """0 or one size for the heads, rows and types; more requests or a wider table never need less."""
    import ctypes as C

    from decode_megakernel_04_gb300 import binding
    lib = binding.load()

    def size(batch, pages):
        a = binding.PagedAttentionArgs(batch=batch, rows=rows, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, n_pages=1 << 20,
                                       page_size=16, max_pages=pages, dtype=dtype, cache_dtype=cache)
        n = C.c_uint64(0)
        assert lib.mk_paged_attention_workspace(C.byref(a), 0, C.byref(n)) == 0
        return n.value

    got = np.array([[size(b, w) for w in (1, 4, 16, 32, 60, 94, 128, 300, 5000, 1 << 20, (1 << 27) - 64)]
                    for b in (1, 2, 7, 16, 30, 40, 60, 150, 400, 5000, 1 << 20)], np.int64)
    assert len(np.unique(got[got > 0])) == 1
    assert (np.diff(got, axis=0) >= 0).all() and (np.diff(got, axis=1) >= 0).all()


def test_attention_of_fewer_requests_in_the_largest_calls_workspace():
    from decode_megakernel_04_gb300 import paged_attention_workspace
    s = attention_inputs([7 + 10 * i for i in range(150)], 1, 32, 8, 128, 16, BF16, BF16, seed=13, poison=False)
    ws = torch.empty(paged_attention_workspace(s["q"], s["k"], s["table"]), dtype=torch.uint8, device=DEV)
    for n in (150, 60, 40, 30, 22, 5, 1):
        t = dict(s, q=s["q"][-n:], table=s["table"][-n:], lens=s["lens"][-n:].contiguous())
        got, lse = run_attention(t, workspace=ws)
        check_attention(t, got, lse, 128 ** -0.5)


def test_attention_refuses():
    from decode_megakernel_04_gb300 import MKError, paged_attention
    s = attention_inputs([20], 1, 4, 2, 64, 16, BF16, BF16)
    out = torch.empty_like(s["q"].contiguous())
    ok = dict(q=s["q"], k_pages=s["k"], v_pages=s["v"], table=s["table"], lens=s["lens"], out=out)
    wide = torch.empty(1, 1, 4, 66, dtype=BF16, device=DEV)
    for change in (dict(lens=s["lens"].long()), dict(lens=i32([1, 2])), dict(table=s["table"].repeat(2, 1)), dict(out=out.float()),
                   dict(v_pages=s["v"][:-1]), dict(k_pages=s["k"].half()), dict(q=s["q"].transpose(2, 3)), dict(lens=s["lens"].cpu())):
        with pytest.raises(ValueError):
            paged_attention(**{**ok, **change})
    for change in (dict(q=wide[..., 1:65]), dict(k_pages=s["k"].to(E4M3), v_pages=s["v"].to(E4M3)), dict(table=s["table"].repeat(1, 20000), workspace=torch.empty(64, dtype=torch.uint8, device=DEV)),
                   dict(q=s["q"].repeat(1, 1, 3, 1)[:, :, :3], out=out[:, :, :3])):
        with pytest.raises(MKError):
            paged_attention(**{**ok, **change})


def test_workspaces_for_another_stream_are_not_the_current_streams_memory():
    """What torch holds free for the current stream may still be read and written by work enqueued there."""
    from decode_megakernel_04_gb300 import serving
    size = 3 << 20
    dev = torch.device(DEV, 0)
    side = torch.cuda.Stream()

    def fresh(current, stream):
        torch.cuda.empty_cache()
        with torch.cuda.stream(current):
            x = torch.empty(size, dtype=torch.uint8, device=dev)
            at = x.data_ptr()
            del x  # free for `current` from here on
            w = serving._workspace(size, dev, 0, stream)
            same = w.data_ptr() == at
            del w
            return not same, serving._workspace(size, dev, 0, stream).data_ptr()

    main = torch.cuda.default_stream()
    for current, stream in ((main, side.cuda_stream), (side, 0)):
        own, at = fresh(current, stream)
        assert own
        with torch.cuda.stream(torch.cuda.ExternalStream(stream) if stream else main):  # it goes back to its stream
            assert torch.empty(size, dtype=torch.uint8, device=dev).data_ptr() == at
    for current, stream in ((main, 0), (main, None), (side, side.cuda_stream), (side, None)):
        assert not fresh(current, stream)[0]


# ---- logit controls ---------------------------------------------------------------------------------------------------

def controls_reference(z, history, prompt, total, rep, pres, freq, ids, vals, allowed):
    """Each step in fp64, rounded to fp32 (exact: a product, quotient or sum of fp32 values rounds the same through 53
    bits). Returns (z fp32, token)."""
    z = z.float().cpu().numpy()
    n, V = z.shape
    r32 = lambda x: x.astype(np.float64).astype(np.float32)  # noqa: E731
    out, token = np.empty_like(z), []
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(n):
            x = z[i].copy()
            if history is not None:
                h = history[i].cpu().numpy()
                T = h.size if total is None else min(max(int(total[i]), 0), h.size)
                P = 0 if prompt is None else min(max(int(prompt[i]), 0), T)
                ok = (h >= 0) & (h < V)
                seen = np.zeros(V, bool)
                seen[h[:T][ok[:T]]] = True
                cnt = np.bincount(h[P:T][ok[P:T]], minlength=V)
                if rep is not None:
                    f = np.float64(rep[i].item())
                    x = np.where(seen, np.where(x > 0, r32(x.astype(np.float64) / f), r32(x.astype(np.float64) * f)), x)
                if freq is not None:
                    part = r32(np.float64(freq[i].item()) * cnt.astype(np.float64))
                    x = np.where(cnt > 0, r32(x.astype(np.float64) - part.astype(np.float64)), x)
                if pres is not None:
                    x = np.where(cnt > 0, r32(x.astype(np.float64) - np.float64(pres[i].item())), x)
            if ids is not None:
                for t, v in {int(t): v for t, v in zip(ids[i].tolist(), vals[i].cpu().numpy()) if 0 <= t < V}.items():
                    x[t] = np.float32(np.float64(x[t]) + np.float64(v))
            if allowed is not None:
                bits = np.unpackbits(allowed[i].cpu().numpy().view(np.uint8), bitorder="little")[:V]
                x = np.where(bits == 1, x, np.float32(-np.inf))
            out[i] = x
            rank = np.where(np.isnan(x), -np.inf, x)
            token.append(int(rank.argmax()) if rank.max() > -np.inf else -1)
    return out, np.array(token)


CASES_LOGITS = [  # rows, vocab, history, biases, dtype, mask, row padding
    (1, 1, 3, 1, F32, True, 0), (2, 3, 5, 2, F32, True, 1), (3, 31, 8, 0, BF16, True, 0), (2, 33, 0, 3, F32, True, 2),
    (4, 1000, 64, 5, F32, True, 0), (3, 1001, 700, 17, BF16, True, 0), (5, 4097, 33, 0, F16, False, 3), (2, 32000, 2000, 300, F32, True, 4),
    (1, 151936, 5000, 40, F32, True, 0), (2, 163841, 300, 2047, BF16, True, 0), (1, 229121, 900, 9, F32, True, 1),
    (1, 262145, 3000, 50, F16, True, 0), (2, 500001, 100, 5, BF16, False, 0), (700, 130, 9, 4, F32, True, 0), (40, 5003, 50, 0, F32, False, 0),
    # long histories of many rows: a row's named tokens over 4, 2 and 1 CTAs
    (30, 5000, 3000, 20, F32, True, 0), (60, 9001, 1500, 2047, BF16, True, 1), (33, 40000, 12000, 40, F32, False, 0),
    (90, 3001, 2000, 3, F16, True, 0)]


def logit_inputs(rows, vocab, hist, biases, dtype, mask, pad, seed=0):
    g = gen(seed)
    z = (3 * torch.randn(rows, vocab + pad, generator=g, device=DEV)).to(dtype)[:, :vocab]
    kw = {}
    if hist:
        h = (torch.rand(rows, hist + pad, generator=g, device=DEV) ** 4 * (vocab + 2)).to(torch.int32) - 1  # some outside
        kw = dict(history=h[:, :hist], total_len=torch.randint(-1, hist + 3, (rows,), generator=g, device=DEV).to(torch.int32),
                  prompt_len=torch.randint(-1, hist + 2, (rows,), generator=g, device=DEV).to(torch.int32))
        for k in ("repetition", "presence", "frequency"):
            kw[k] = 0.5 + torch.rand(rows, generator=g, device=DEV)
    if biases:
        kw["bias_ids"] = torch.randint(-2, vocab + 2, (rows, biases), generator=g, device=DEV).to(torch.int32)
        kw["bias_vals"] = 5 * torch.randn(rows, biases, generator=g, device=DEV)
        if biases > 2:
            kw["bias_ids"][:, -1] = kw["bias_ids"][:, 0]  # named twice: the last entry counts
    if mask:
        w = -(-vocab // 32)
        kw["allowed"] = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows, w + pad), generator=g, device=DEV).to(torch.int32)[:, :w]
    return z, kw


def check_controls(z, kw, in_place=False, **call):
    from decode_megakernel_04_gb300 import logit_controls
    rows, vocab = z.shape
    want, token = controls_reference(z, *(kw.get(k) for k in ("history", "prompt_len", "total_len", "repetition", "presence",
                                                             "frequency", "bias_ids", "bias_vals", "allowed")))
    wide = torch.full((rows, vocab + 5), 7.0, device=DEV)
    out = z if in_place else wide[:, 1:vocab + 1]
    tok = i32([-9] * rows)
    logit_controls(z, out, token=tok, **kw, **call)
    torch.cuda.synchronize()
    got = out.cpu().numpy()
    assert np.array_equal(got.view(np.int32), want.view(np.int32)) or np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(tok.cpu().numpy(), token)
    if not in_place:
        assert (wide[:, 0] == 7).all() and (wide[:, vocab + 1:] == 7).all()


def many(z, kw, times=24):
    """The rows over again (more than a cluster per row is used for), each copy with its own penalties."""
    z = z.repeat(times, 1)
    kw = {k: v.repeat(times, *[1] * (v.dim() - 1)) for k, v in kw.items()}
    for k in ("repetition", "presence", "frequency"):
        if k in kw:
            kw[k] = kw[k] * torch.linspace(0.5, 1.5, kw[k].numel(), device=DEV)
    return z, kw


@pytest.mark.parametrize("rows", ["few", "many"])
@pytest.mark.parametrize("case", CASES_LOGITS, ids=str)
def test_logit_controls(case, rows):
    """Few rows: clusters. Many: the plain pass and the second kernel (a history of over 12 thousand tokens: clusters)."""
    z, kw = logit_inputs(*case)
    if rows == "many":
        if z.shape[0] >= 20 or z.shape[1] > 200000:
            pytest.skip("the same form as few, or long")
        z, kw = many(z, kw)
    check_controls(z, kw)
    if case[4] is F32:
        check_controls(z, kw, in_place=True)


@pytest.mark.parametrize("keep", [(), ("allowed",), ("bias_ids", "bias_vals"), ("history", "repetition"), ("history", "presence"),
                                  ("history", "frequency", "total_len"), ("history", "repetition", "prompt_len", "allowed"), ("history",)])
def test_logit_controls_each_alone(keep):
    z, kw = logit_inputs(3, 2050, 90, 12, F32, True, 0, seed=4)
    check_controls(z, {k: kw[k] for k in keep})
    check_controls(*many(z, {k: kw[k] for k in keep}))


def test_logit_controls_special_values():
    V = 5000
    z = torch.zeros(6, V, device=DEV)
    z[0] = float("-inf")
    z[1, 7], z[1, 9] = float("nan"), 3.0
    z[2, 4000], z[2, 4001] = float("inf"), float("inf")
    z[3] = -0.0
    z[4] = float("nan")
    z[5] = torch.finfo(F32).min
    check_controls(z, {})
    check_controls(*many(z, {}))
    allowed = torch.zeros(6, -(-V // 32), dtype=torch.int32, device=DEV)   # row 0..4: nothing is allowed
    allowed[5, 100] = 1 << 5
    check_controls(z, dict(allowed=allowed))
    check_controls(*many(z, dict(allowed=allowed)))
    allowed[1] = -1
    check_controls(z, dict(allowed=allowed))
    check_controls(*many(z, dict(allowed=allowed)))
    # every token of the row is in the history, and every token but one
    z = torch.randn(2, 300, generator=gen(3), device=DEV)
    kw = dict(history=torch.arange(300, device=DEV).to(torch.int32).repeat(2, 1), total_len=i32([300, 299]), repetition=torch.tensor([2.0, 0.5], device=DEV))
    check_controls(z, kw)
    check_controls(*many(z, kw))


@pytest.mark.parametrize("n, repeats", [(30, 1), (30, 6), (50, 6)])
def test_logit_controls_largest_logits_are_in_the_history(n, repeats):
    """The chunks' largest logits are mostly named tokens, so that the join has to look for others."""
    V = 20011
    z = torch.randn(n, V, generator=gen(5), device=DEV)
    top = z.topk(200, dim=1).indices.to(torch.int32).repeat(1, repeats)
    for pen in (1.0, 1.02, 5.0):
        kw = dict(history=top, total_len=i32([7 * i for i in range(n)]), frequency=torch.full((n,), pen, device=DEV))
        check_controls(z, kw)
        check_controls(z.clone(), kw, in_place=True)
        kw["allowed"] = torch.randint(-2 ** 31, 2 ** 31 - 1, (n, -(-V // 32)), generator=gen(6), device=DEV).to(torch.int32)
        check_controls(z, kw)


def test_logit_controls_ties_take_the_lowest_index_of_the_whole_row():
    for V in (64, 1000, 100003):
        z = torch.zeros(4, V, device=DEV)
        z[0, V // 2] = z[0, V - 1] = 2.0
        z[1, 3:] = 1.0
        z[2, :] = 5.0
        check_controls(z, {})
        check_controls(*many(z, {}))


def test_logit_controls_empty_lists():
    """A history of length 0 with penalties, biases of width 0, and a history longer than one pass of slices holds."""
    z, kw = logit_inputs(2, 777, 5, 3, F32, True, 0, seed=6)
    kw["history"], kw["total_len"], kw["prompt_len"] = kw["history"][:, :0], None, None
    check_controls(z, {k: v for k, v in kw.items() if v is not None and not k.startswith("bias")})
    kw["bias_ids"], kw["bias_vals"] = kw["bias_ids"][:, :0], kw["bias_vals"][:, :0]
    check_controls(z, {k: v for k, v in kw.items() if v is not None})
    check_controls(*many(z, {k: v for k, v in kw.items() if v is not None}))
    z, kw = logit_inputs(2, 300007, 60000, 3, BF16, True, 0, seed=7)
    kw["history"] = torch.randint(0, 300007, (2, 60000), generator=gen(8), device=DEV).to(torch.int32)
    check_controls(z, kw)
    check_controls(*many(z[:, :3000], {**kw, "allowed": kw["allowed"][:, :94]}, times=12))


def test_logit_controls_one_token_repeated():
    V, n = 4000, 20000
    z = torch.full((2, V), 1.0, device=DEV)
    kw = dict(history=torch.full((2, n), 17, dtype=torch.int32, device=DEV), total_len=i32([n, n]), prompt_len=i32([0, n - 3]),
              frequency=torch.tensor([0.5, 2.0], device=DEV), repetition=torch.tensor([2.0, 4.0], device=DEV))
    check_controls(z, kw)
    kw["history"], kw["total_len"], kw["prompt_len"] = kw["history"][:, :9000], i32([9000, 9000]), i32([0, 8998])
    check_controls(*many(z, kw))


@pytest.mark.parametrize("n", [3, 40])
def test_logit_controls_captured(n):
    from decode_megakernel_04_gb300 import logit_controls
    z, kw = logit_inputs(n, 30011, 200, 9, F32, True, 0)
    out, tok = torch.empty_like(z), i32([0] * n)
    logit_controls(z, out, token=tok, **kw)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        logit_controls(z, out, token=tok, **kw)
    z.mul_(-0.5)
    kw["history"].add_(1)
    gr.replay()
    torch.cuda.synchronize()
    want, token = controls_reference(z, *(kw.get(k) for k in ("history", "prompt_len", "total_len", "repetition", "presence",
                                                             "frequency", "bias_ids", "bias_vals", "allowed")))
    assert np.array_equal(out.cpu().numpy(), want) and np.array_equal(tok.cpu().numpy(), token)


# ---- together, and with the rest of the framework -----------------------------------------------------------------------

@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_serving_steps_together(cache):
    """Requests of different ages through page tables, norm + rotation + append and attention, several steps with
    prompts, rejected tokens and finished requests, all of it captured once and replayed; against contiguous fp64
    caches kept by the test."""
    from decode_megakernel_04_gb300 import page_tables, paged_attention, qk_norm_rope
    B, hq, hkv, d, page, n_pages, max_pages, places = 5, 12, 2, 128, 16, 64, 12, 160
    g = gen(11)
    t = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
    ring = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    state, lens, status = i32([0, n_pages]), i32([0] * B), i32([0])
    start, count = i32([0] * B), i32([0] * B)
    slots = torch.empty(places, dtype=torch.int64, device=DEV)
    pos, own, starts = i32([0] * places), i32([0] * places), i32([0] * (B + 1))
    qkv = torch.empty(places, hq + 2 * hkv, d, dtype=BF16, device=DEV)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    gains = (1 + 0.1 * torch.randn(2, d, generator=g, device=DEV)).to(BF16)
    inv = (1e4 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).to(DEV)
    kp, vp = (torch.zeros(n_pages, hkv, page, d, device=DEV).to(cache) for _ in range(2))
    ks, vs = (torch.full((hkv,), 0.03, device=DEV) for _ in range(2)) if cache is E4M3 else (None, None)
    q_out = torch.empty(places, hq, d, dtype=BF16, device=DEV)
    newest = torch.empty(B, 1, hq, d, dtype=BF16, device=DEV)
    out, lse = torch.empty_like(newest), torch.empty(B, 1, hq, device=DEV)

    def step():
        page_tables(t, lens, start, count, ring, state, page, n_pages, slots=slots, positions=pos, owners=own, starts=starts,
                    lens=lens, status=status)
        qk_norm_rope(q, k, pos, inv, q_out, v=v, q_gain=gains[0], k_gain=gains[1], k_pages=kp, v_pages=vp, slots=slots,
                     k_scale=ks, v_scale=vs, status=status)
        newest.copy_(q_out[(starts[1:] - 1).clamp(min=0).long()][:, None])  # each request's last new token
        paged_attention(newest, kp, vp, t, lens, out, lse=lse, k_scale=ks, v_scale=vs, status=status)

    qkv.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # count 0 everywhere: nothing but a warm-up
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    steps = [([0] * 5, [40, 1, 0, 17, 100]), (None, [1, 1, 9, 1, 1]), ([39, 2, 9, 16, 101], [3, 1, 1, 2, 1]),
             ([42, 0, 8, 18, 90], [1, 0, 1, 1, 60]), ([43, 0, 9, 0, 150], [1, 20, 1, 0, 1]), (None, [1, 1, 1, 5, 1])]
    K, V = [torch.zeros(0, hkv, d, dtype=torch.float64, device=DEV) for _ in range(B)], [torch.zeros(0, hkv, d, dtype=torch.float64, device=DEV) for _ in range(B)]
    for s0, c0 in steps:
        s0 = [x.shape[0] for x in K] if s0 is None else s0
        start.copy_(i32(s0)), count.copy_(i32(c0))
        qkv.copy_(torch.randn(qkv.shape, generator=g, device=DEV).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        assert status.item() == 0 and lens.tolist() == [a + b for a, b in zip(s0, c0)]
        at = 0
        used = set()
        for b in range(B):
            K[b], V[b] = K[b][:s0[b]], V[b][:s0[b]]
            new = slice(at, at + c0[b])
            p = torch.arange(s0[b], s0[b] + c0[b], device=DEV)
            assert torch.equal(pos[new].long(), p) and (own[new] == b).all()
            K[b] = torch.cat([K[b], rotate(k[new], gains[1], 1e-6, p, inv)])
            V[b] = torch.cat([V[b], v[new].double()])
            at += c0[b]
            n = K[b].shape[0]
            pages = t[b, :-(-n // page)].long()
            assert not used & set(pages.tolist())
            used |= set(pages.tolist())
            if not n:
                assert (out[b] == 0).all()
                continue
            # the cache holds the request, rounded once
            for mine, paged, sc in ((K[b], kp, ks), (V[b], vp, vs)):
                flat = paged[pages].transpose(1, 2).reshape(-1, hkv, d)[:n]
                want = mine if sc is None else (mine / sc.double()[:, None]).clamp(-448, 448)
                check_rounded(flat.float(), want, cache, "cache", qk_slack(want))
        free = {int(ring[(int(state[0]) + i) % n_pages]) for i in range(int(state[1]))}
        assert len(free) == int(state[1]) and not free & used and len(free) + len(used) == n_pages
        s = dict(q=newest, k=kp, v=vp, table=t, lens=lens, ks=ks, vs=vs, page=page)
        check_attention(s, out, lse, d ** -0.5, f"step {s0}")


def test_attention_reads_contiguous_caches_as_pages():
    """Caches of mk_decode_step_static's layout (one layer) are a paged cache with a fixed table."""
    B, hkv, ctx, d, page = 3, 4, 96, 128, 32
    g = gen(12)
    k, v = (torch.randn(B, hkv, ctx, d, generator=g, device=DEV).to(BF16) for _ in range(2))
    per = ctx // page
    view = lambda x: x.as_strided(((B - 1) * hkv * per + per, hkv, page, d), (page * d, ctx * d, d, 1))  # noqa: E731
    table = (torch.arange(B)[:, None] * hkv * per + torch.arange(per)).to(torch.int32).to(DEV)
    s = dict(q=torch.randn(B, 2, 24, d, generator=g, device=DEV).to(BF16), k=view(k), v=view(v), table=table, lens=i32([96, 5, 33]),
             ks=None, vs=None, page=page)
    got, lse = run_attention(s)
    check_attention(s, got, lse, d ** -0.5)
    # the same, straight from the contiguous caches
    x = s["q"][1, 1].double().view(hkv, 6, d)
    p = torch.softmax(torch.matmul(x, k[1, :, :5].double().transpose(1, 2)) * d ** -0.5, -1)
    want = torch.matmul(p, v[1, :, :5].double()).view(24, d)
    check_rounded(got[1, 1], want, BF16, "static cache", 2.0 ** -12 * want.abs().amax())


def test_step_with_controls():
    """Megakernel.step with controls: the plain step's logits, controlled, and the greedy token of what is left."""
    from decode_megakernel_04_gb300 import Megakernel
    from synthetic import config, make_tokens, make_weights
    cfg = config("tiny_dense")
    w = make_weights(cfg, seed=5, device=torch.device(DEV))
    B, R, T = 2, 3, 20
    ctx = make_tokens(5, "ctx", (B, T), cfg.vocab, device=DEV).contiguous()
    tok = make_tokens(5, "t", (B, R), cfg.vocab, device=DEV).contiguous()
    pos = i32([T, T])
    plain, got = torch.empty(B * R, cfg.vocab, device=DEV), torch.empty(B * R, cfg.vocab, device=DEV)
    am = i32([0] * (B * R))
    _, kw = logit_inputs(B * R, cfg.vocab, 50, 6, F32, True, 0)
    mks = [Megakernel(cfg, w, max_batch=B, max_rows=8, max_ctx=64) for _ in range(2)]
    for m in mks:
        m.prefill(ctx)
    mks[0].step(tok, pos, plain)
    mks[1].step(tok, pos, got, am, controls=kw)
    assert mks[0].status() == 0 and mks[1].status() == 0
    want, token = controls_reference(plain, *(kw.get(k) for k in ("history", "prompt_len", "total_len", "repetition", "presence",
                                                                 "frequency", "bias_ids", "bias_vals", "allowed")))
    assert np.array_equal(got.cpu().numpy(), want) and np.array_equal(am.cpu().numpy(), token)
    with pytest.raises(ValueError):
        mks[1].step(tok, pos, None, am, controls=kw)
    for m in mks:
        m.close()


def stepless():
    """A Megakernel of 2 sequences and 8 tokens of vocabulary whose step must not run, and its tokens and positions."""
    from decode_megakernel_04_gb300 import binding

    class Lib:
        def mk_decode_step(self, *args):
            raise AssertionError("the step ran")

    m = binding.Megakernel.__new__(binding.Megakernel)
    m.lib, m.device, m.h = Lib(), 0, None
    m.cfg = type("Cfg", (), {"vocab": 8})
    return m, i32([[1], [2]]), i32([0, 0])


def test_controls_that_the_library_refuses_are_refused_before_the_step():
    """Strides, alignment, list lengths and the workspace: what only the library checks."""
    from decode_megakernel_04_gb300 import MKError
    m, tok, pos = stepless()
    z = torch.zeros(2, 8, device=DEV)
    ids = i32([[1, 2]] * 2)
    pen = torch.ones(2, device=DEV)
    spare = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    many = torch.zeros(400, 8, device=DEV)
    for kw in (dict(allowed=i32([[-1]]).expand(2, -1)), dict(history=i32([[1, 2]]).expand(2, -1), repetition=pen),
               dict(bias_ids=ids.repeat(1, 1024), bias_vals=torch.zeros(2, 2048, device=DEV), workspace=spare)):
        with pytest.raises(MKError):
            m.step(tok, pos, z, controls=kw)
    # many rows need a workspace: one that is too short, and one that is not aligned
    for ws in (spare[:8], spare[1:]):
        with pytest.raises(MKError):
            m.step(i32([[1]] * 400), i32([0] * 400), many, controls=dict(bias_ids=i32([[1]] * 400), bias_vals=torch.zeros(400, 1, device=DEV), workspace=ws))


def test_controls_refuse_logits_with_gaps_between_rows():
    """The step writes contiguous rows, so controls at another row stride would work on the wrong values."""
    m, tok, pos = stepless()
    for z in (torch.zeros(2, 12, device=DEV)[:, :8], torch.zeros(4, 8, device=DEV)[::2], torch.zeros(2, 1, 9, device=DEV)[..., :8],
              torch.zeros(1, 8, device=DEV).expand(2, 8)):
        with pytest.raises(ValueError):
            m.step(tok, pos, z, controls=dict(bias_ids=i32([[1], [2]]), bias_vals=torch.ones(2, 1, device=DEV)))


def test_a_failed_call_leaves_nothing_for_the_next_one():
    """A device that is not there is an error of that call alone: the operators and the step after it succeed."""
    import ctypes as C

    from decode_megakernel_04_gb300 import Megakernel, binding, logit_controls, page_tables, paged_attention, qk_norm_rope
    from synthetic import config, make_tokens, make_weights
    lib = binding.load()
    cfg = config("tiny_dense")
    m = Megakernel(cfg, make_weights(cfg, seed=5, device=torch.device(DEV)), max_batch=1, max_rows=8, max_ctx=64)
    m.prefill(make_tokens(5, "ctx", (1, 20), cfg.vocab, device=DEV).contiguous())
    tok, z = make_tokens(5, "t", (1, 1), cfg.vocab, device=DEV).contiguous(), torch.empty(1, cfg.vocab, device=DEV)
    few, many = torch.zeros(2, 50, device=DEV), torch.zeros(500, 50, device=DEV)
    s = attention_inputs([40, 30], 1, 4, 2, 128, 16, BF16, BF16, seed=6, poison=False)
    wide = dict(s, table=s["table"].repeat(1, 4000))
    out = torch.empty_like(s["q"].contiguous())
    x = torch.zeros(3, 2, 64, dtype=BF16, device=DEV)
    t = i32([[0, -1], [1, -1]])
    args = binding.LogitControlsArgs(logits=few.data_ptr(), out=few.data_ptr(), logits_stride=50, out_stride=50, rows=2, vocab=50, dtype=2)
    calls = [lambda: page_tables(t, i32([4, 2]), i32([4, 2]), i32([0, 0]), i32([2, 3, 0, 0]), i32([0, 2]), 4, 4, slots=torch.empty(3, dtype=torch.int64, device=DEV)),
             lambda: qk_norm_rope(x, x, None, None, x), lambda: logit_controls(few, few), lambda: logit_controls(many, many),
             lambda: paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], out),
             lambda: paged_attention(wide["q"], wide["k"], wide["v"], wide["table"], wide["lens"], out), lambda: m.step(tok, i32([20]), z)]
    for call in calls:
        call()
        assert lib.mk_logit_controls(C.byref(args), 63, None) == 4  # MK_ERR_CUDA
        call()
    torch.cuda.synchronize()
    assert m.status() == 0
    m.close()


# ---- the ends of the documented ranges ------------------------------------------------------------------------------------

@pytest.mark.parametrize("lens, R, hq, hkv, d, dtype, cache", [
    ([70, 200, 64, 3], 64, 6, 1, 128, BF16, BF16), ([65, 130], 65, 4, 2, 64, F16, F16), ([1000, 1500, 999], 1000, 4, 2, 128, BF16, BF16),
    ([4096], 4096, 2, 1, 64, BF16, BF16), ([300], 100, 8, 1, 256, F16, F16), ([500, 90], 100, 6, 2, 128, BF16, E4M3),
    ([700], 65, 4, 1, 256, F16, E4M3)])
@pytest.mark.parametrize("width", [None, 50000])
def test_attention_of_many_new_tokens(lens, R, hq, hkv, d, dtype, cache, width):
    """A prompt's tokens at once; then the newest two keys become NaN, which the rows before them do not see."""
    s = attention_inputs(lens, R, hq, hkv, d, 16, dtype, cache, seed=51, max_pages=width)
    got, lse = run_attention(s)
    check_attention(s, got, lse, d ** -0.5)
    for x in (s["k"], s["v"]):  # the newest two keys of each request: every row before them as it was
        for b, n in enumerate(lens):
            for p in (n - 1, n - 2):
                at = s["table"][b, p // 16].long()
                x[at, :, p % 16] = torch.full((hkv, d), float("nan"), device=DEV).to(cache)
    bad, bl = run_attention(s)
    assert torch.equal(bad[:, :R - 2], got[:, :R - 2]) and torch.equal(bl[:, :R - 2], lse[:, :R - 2])
    assert bad[:, -1].isnan().all()


def test_attention_of_more_requests_than_a_cta_has_threads():
    for d, cache in ((128, BF16), (64, BF16), (128, E4M3)):
        s = attention_inputs([i * 11 % 90 for i in range(1300)], 1, 4, 1, d, 16, BF16, cache, seed=52, max_pages=50000)
        got, lse = run_attention(s)
        check_attention(s, got, lse, d ** -0.5)


def test_attention_of_one_very_long_request():
    """Positions, tiles and pieces of 3 million keys; all scores equal, so that the result is the mean of the values."""
    n, page, d = 3_000_001, 256, 64
    pages = -(-n // page)
    g = gen(53)
    k = torch.zeros(pages, 1, page, d, dtype=F16, device=DEV)
    v = torch.randint(0, 3, (pages, 1, page, d), generator=g, device=DEV).to(F16)
    s = dict(q=torch.ones(1, 2, 4, d, dtype=F16, device=DEV), k=k, v=v, table=torch.randperm(pages, generator=g, device=DEV).to(torch.int32)[None],
             lens=i32([n]), ks=None, vs=None, page=page)
    v[s["table"][0, -1].long(), :, n % page:] = float("nan")
    got, lse = run_attention(s)
    x = v[s["table"][0].long()].reshape(-1, d)
    for r in range(2):
        m = n - 1 + r
        # sums of whole numbers times a power of two: exact in fp32 within a piece while below 2^24; joined in 1 rounding each
        want = x[:m].double().mean(0)
        check_rounded(got[0, r], want.expand(4, d), F16, "mean", 2.0 ** -16 * want)
        assert (lse[0, r].double() - math.log(m)).abs().max() < 2.0 ** -18


def test_logit_controls_of_a_million_rows_and_of_the_longest_rows():
    from decode_megakernel_04_gb300 import logit_controls
    g = gen(54)
    for rows, vocab in ((1 << 20, 5), (1, 1 << 24), (40, 1 << 24), (3, (1 << 24) - 5)):
        z = torch.randn(rows, vocab, generator=g, device=DEV)
        bits = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows, -(-vocab // 32)), generator=g, device=DEV).to(torch.int32)
        hist = torch.randint(0, vocab, (rows, 3), generator=g, device=DEV).to(torch.int32)
        pen = 0.5 + torch.rand(rows, generator=g, device=DEV)
        out, tok = torch.empty_like(z), torch.empty(rows, dtype=torch.int32, device=DEV)
        logit_controls(z, out, history=hist, presence=pen, allowed=bits, token=tok)
        ids = hist.long()
        z.scatter_(1, ids, z.gather(1, ids) - pen[:, None])  # (an id named twice: both write the same)
        v = torch.arange(vocab, device=DEV)
        for r0 in range(0, rows, 1 << 18 if vocab < 100 else 4):
            part = slice(r0, r0 + (1 << 18 if vocab < 100 else 4))
            ok = (bits[part][:, v >> 5] >> (v & 31)) & 1 == 1
            want = torch.where(ok, z[part], -math.inf)
            assert torch.equal(out[part], want)
            first = torch.where(want == want.amax(1, keepdim=True), v, vocab).amin(1)
            assert torch.equal(tok[part].long(), torch.where(ok.any(1), first, -1))


def test_logit_controls_longest_history():
    """2^20 - 1 entries of one token: the count fills its bits; with the most biases."""
    V, n = 1000, 2 ** 20 - 1
    z = torch.full((2, V), 2.0, device=DEV)
    kw = dict(history=torch.full((2, n), 17, dtype=torch.int32, device=DEV), prompt_len=i32([0, 1]), repetition=torch.tensor([2.0, 4.0], device=DEV),
              frequency=torch.tensor([0.5, 2.0], device=DEV), bias_ids=i32([[17] * 2047] * 2), bias_vals=torch.arange(4094, device=DEV).view(2, 2047).float())
    check_controls(z, kw)


def test_qk_most_heads_and_any_position():
    from decode_megakernel_04_gb300 import qk_norm_rope
    g = gen(55)
    n, hq, hkv, d = 5, 4096, 4096, 16
    q, k = (torch.randn(n, h, d, generator=g, device=DEV).to(BF16) for h in (hq, hkv))
    pos = i32([-2 ** 31, -1, 0, 2 ** 31 - 1, -12345678])
    inv = (1e4 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).to(DEV)
    gain = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(BF16)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    qk_norm_rope(q, k, pos, inv, qo, k_out=ko, q_gain=gain, k_gain=gain)
    for x, y in ((q, qo), (k, ko)):
        want = rotate(x, gain, 1e-6, pos, inv)
        check_rounded(y, want, BF16, "heads", qk_slack(want))


@pytest.mark.parametrize("over", ["held", "start", "count"])
@pytest.mark.parametrize("chunk", [3, 2000])
def test_page_tables_lens_over_each_of_the_lengths(over, chunk):
    """lens may be held, start or count itself, for a step that is taken and one that is refused, of one CTA and of more."""
    from decode_megakernel_04_gb300 import page_tables
    rng = np.random.default_rng(5)
    B, page, max_pages = 20, 16, 400
    held = [int(x) for x in rng.integers(0, 4000, B)]
    start = [max(0, h - i % 3) for i, h in enumerate(held)]
    count = [1 + (chunk if i % 7 == 0 else 0) for i in range(B)]
    n_pages = 2 * B * max_pages
    table, ring, state = make_pool(rng, held, page, max_pages, n_pages, 0)
    for bad in (False, True):
        places = sum(count) - bad
        t = dict(held=i32(held), start=i32(start), count=i32(count))
        tab, rg = torch.from_numpy(table).to(DEV), torch.from_numpy(ring).to(DEV)
        st, slots, status = i32(state), torch.empty(places, dtype=torch.int64, device=DEV), i32([0])
        page_tables(tab, t["held"], t["start"], t["count"], rg, st, page, n_pages, slots=slots, lens=t[over], status=status)
        want = tables_reference(table, held, start, count, ring, state, page, n_pages, places)
        if bad:
            assert want == 8 == status.item() and t[over].tolist() == held and st.tolist() == state
        else:
            assert t[over].tolist() == want["lens"].tolist() and np.array_equal(slots.cpu().numpy(), want["slots"])
            assert st.tolist() == want["ring_state_out"].tolist() and np.array_equal(tab.cpu().numpy(), want["table"])


def test_calls_without_rows():
    from decode_megakernel_04_gb300 import logit_controls, paged_attention, qk_norm_rope
    x = torch.empty(0, 2, 64, dtype=BF16, device=DEV)
    qk_norm_rope(x, x, i32([]), torch.ones(32, dtype=torch.float64, device=DEV), x)
    kv = torch.zeros(3, 2, 16, 64, dtype=BF16, device=DEV)
    qk_norm_rope(x, x, None, None, x, v=x, k_pages=kv, v_pages=kv, slots=torch.empty(0, dtype=torch.int64, device=DEV))
    q = torch.empty(0, 1, 4, 64, dtype=BF16, device=DEV)
    paged_attention(q, kv, kv, torch.empty(0, 5, dtype=torch.int32, device=DEV), i32([]), q)
    z = torch.empty(0, 9, device=DEV)
    logit_controls(z, z, token=i32([]))
    torch.cuda.synchronize()


FIRST_CALL = """
import torch
from decode_megakernel_04_gb300 import logit_controls, page_tables, paged_attention, qk_norm_rope
D = "cuda"
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=D)
t, h, st, ring, slots = i32([[0, -1], [1, -1]]), i32([4, 2]), i32([0, 2]), i32([2, 3, 0, 0]), torch.empty(3, dtype=torch.int64, device=D)
one, so, lens = i32([1, 1]), i32([0, 0]), i32([0, 0])
x = torch.randn(2, 4, 128, device=D).bfloat16()
xo = torch.empty_like(x)
kv = torch.randn(4, 2, 16, 128, device=D).bfloat16()
q = torch.randn(2, 1, 4, 128, device=D).bfloat16()
tab, wide, al = i32([[0, 1], [2, 3]]), i32([[0, 1] + [0] * 5000, [2, 3] + [0] * 5000]), i32([20, 31])
o1, o2 = torch.zeros_like(q), torch.zeros_like(q)
few, many = torch.randn(2, 70, device=D), torch.randn(400, 70, device=D)
f2, m2 = torch.zeros_like(few), torch.zeros_like(many)
ids, vals = i32([[5]] * 400), torch.ones(400, 1, device=D)
def calls():
    page_tables(t, h, h, one, ring, st, 4, 4, slots=slots, lens=lens, ring_state_out=so)
    qk_norm_rope(x, x, None, None, xo)
    paged_attention(q, kv, kv, tab, al, o1)
    paged_attention(q, kv, kv, wide, al, o2)
    logit_controls(few, f2)
    logit_controls(many, m2, bias_ids=ids, bias_vals=vals)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    calls()
g.replay()
torch.cuda.synchronize()
got = [v.clone() for v in (slots, lens, so, xo, o1, o2, f2, m2)]
t.copy_(i32([[0, -1], [1, -1]])), o1.zero_(), o2.zero_(), f2.zero_(), m2.zero_(), xo.zero_()
calls()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (slots, lens, so, xo, o1, o2, f2, m2)))
assert torch.equal(xo, x) and torch.equal(f2, few) and o1.abs().sum() > 0 and (o1.float() - o2.float()).abs().max() < 0.02
print("same")
"""


def test_a_process_first_calls_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


def test_calls_from_several_threads_at_once():
    """Each thread on a stream of its own, scratch from torch's allocator: every result as alone."""
    from concurrent.futures import ThreadPoolExecutor

    from decode_megakernel_04_gb300 import logit_controls, paged_attention, qk_norm_rope
    sets = [attention_inputs([2000 + 77 * i, 40, 900], 1 + i % 2, 8, 2, 128, 16, BF16, BF16, seed=60 + i, poison=False,
                             max_pages=50000 if i % 3 else None) for i in range(6)]
    logits = [logit_inputs(100, 5003, 300, 9, F32, True, 0, seed=60 + i) for i in range(6)]
    norms = [qk_inputs(50 + i, 12, 2, 128, 128, BF16, None, 1, True, seed=60 + i) for i in range(6)]

    def work(i, stream):
        with torch.cuda.stream(stream):
            s, (z, kw), n = sets[i], logits[i], norms[i]
            outs = []
            for _ in range(20):
                o, l, y = torch.empty_like(s["q"].contiguous()), torch.empty(s["q"].shape[:3], device=DEV), torch.empty_like(z)
                tok, qo = i32([0] * 100), torch.empty_like(n["q"].contiguous())
                paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], o, lse=l)
                logit_controls(z, y, token=tok, **kw)
                qk_norm_rope(n["q"], n["k"], n["pos"], n["inv"], qo, q_gain=n["qg"], k_gain=n["kg"])
                outs.append((o, l, y, tok, qo))
            stream.synchronize()
        return outs

    torch.cuda.synchronize()
    want = [work(i, torch.cuda.current_stream())[0] for i in range(6)]
    streams = [torch.cuda.Stream() for _ in range(6)]
    torch.cuda.synchronize()
    with ThreadPoolExecutor(6) as pool:
        got = list(pool.map(work, range(6), streams))
    for w, outs in zip(want, got):
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(w, o))


def test_captured_calls_on_a_forked_stream_and_with_rows_over_several_ctas():
    """Inside one capture: attention with scratch of its own on a second stream, and logit controls whose rows take 1, 2 and 4
    CTAs; replayed with other inputs, twice."""
    from decode_megakernel_04_gb300 import logit_controls, paged_attention
    s = attention_inputs([3000, 40, 700], 2, 8, 1, 128, 16, BF16, BF16, seed=71, poison=False, max_pages=50000)
    sets = [logit_inputs(*case, seed=72) for case in ((30, 5000, 3000, 20, F32, True, 0), (60, 9001, 1500, 40, F32, True, 1), (90, 3001, 2000, 3, F32, True, 0))]
    outs = [torch.empty_like(z) for z, _ in sets]
    toks = [i32([0] * z.shape[0]) for z, _ in sets]
    o, l = torch.empty_like(s["q"].contiguous()), torch.empty(s["q"].shape[:3], device=DEV)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], o, lse=l, stream=side.cuda_stream)
        for (z, kw), out, tok in zip(sets, outs, toks):
            logit_controls(z, out, token=tok, **kw)
        main.wait_stream(side)
    for turn in range(2):
        s["q"].mul_(0.8)
        for z, kw in sets:
            z.mul_(-0.7)
            kw["history"].add_(1)
        graph.replay()
        want, wl = run_attention(s)
        assert torch.equal(o, want) and torch.equal(l, wl)
        for (z, kw), out, tok in zip(sets, outs, toks):
            y, token = controls_reference(z, *(kw.get(k) for k in ("history", "prompt_len", "total_len", "repetition", "presence",
                                                                  "frequency", "bias_ids", "bias_vals", "allowed")))
            assert np.array_equal(out.cpu().numpy(), y) and np.array_equal(tok.cpu().numpy(), token)
