"""RMS norm, attention over a shared prefix and verification of drafts without a GPU: the argument structs' layout and every
refusal of the C entry points (each returned before any CUDA call; the addresses are never read)."""
import ctypes as C
import os
import subprocess
import tempfile

import pytest
import torch

import decode_megakernel_04_gb300 as mk
from decode_megakernel_04_gb300 import _build, binding, serving

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, UNSUPPORTED = 1, 2
P = 0x10000  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


def _with(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def norm(**kw):
    return _with(binding.RmsNormArgs(x=P, residual=2 * P, gain=P, residual_out=3 * P, out=4 * P, scales=P, x_stride=256,
                                     residual_stride=256, residual_out_stride=256, out_stride=256, scales_stride=2, rows=4,
                                     width=256, group=128, eps=1e-6), kw)


def prefix(**kw):
    return _with(binding.PrefixAttentionArgs(
        q=P, k_pages=P, v_pages=P, prefix_table=P, prefix_len=P, table=P, lens=P, out=P, workspace=P, workspace_bytes=1 << 40,
        table_stride=8, q_stride=(512, 512, 128), out_stride=(512, 512, 128), k_page_stride=(4096, 2048, 128),
        v_page_stride=(4096, 2048, 128), batch=2, rows=1, n_q_heads=4, n_kv_heads=2, head_dim=128, n_pages=32, page_size=16,
        max_pages=8, max_prefix_pages=8, scale=1), kw)


def drafts(**kw):
    return _with(binding.VerifyDraftsArgs(logits=P, draft_logits=P, tokens=P, uniforms=P, noise=P, accept_out=P, workspace=P,
                                          workspace_bytes=1 << 30, logits_stride=100, draft_stride=100, noise_stride=100, batch=3,
                                          rows=4, vocab=100, dtype=2), kw)


REFUSALS = [
    ("mk_rms_norm", norm, BAD, [
        dict(x=0), dict(out=0), dict(out_dtype=3, scales=0), dict(rows=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(x=P + 8),
        dict(residual=P + 2), dict(gain=P + 4), dict(residual_out=P + 2), dict(out=P + 8), dict(scales=P + 2),
        dict(x_stride=260), dict(residual_stride=257), dict(residual_out_stride=1), dict(out_stride=252), dict(residual_out=4 * P),
        dict(out_dtype=3, out=P), dict(out_dtype=3, out=2 * P), dict(x_stride=248), dict(residual_stride=0), dict(out_stride=128),
        dict(residual_out_stride=8), dict(out_dtype=3, scales_stride=1), dict(residual_out=P, residual_out_stride=264),
        dict(residual_out=2 * P, residual_out_stride=264), dict(out=P, out_stride=264), dict(out=2 * P, out_stride=264)]),
    ("mk_rms_norm", norm, UNSUPPORTED, [
        dict(width=0), dict(width=4), dict(width=260), dict(width=32776), dict(dtype=3), dict(dtype=4), dict(out_dtype=1),
        dict(dtype=2), dict(out_dtype=3, group=0), dict(out_dtype=3, group=96), dict(out_dtype=3, group=512),
        dict(out_dtype=3, group=4), dict(width=264, out_dtype=3)]),
    ("mk_prefix_attention", prefix, BAD, [
        dict(q=0), dict(k_pages=0), dict(v_pages=0), dict(prefix_table=0), dict(prefix_len=0), dict(table=0), dict(lens=0),
        dict(out=0), dict(cache_dtype=3), dict(batch=-1), dict(rows=0), dict(n_q_heads=0), dict(n_kv_heads=0),
        dict(n_kv_heads=3), dict(n_pages=0), dict(page_size=0), dict(max_pages=0), dict(max_prefix_pages=0),
        dict(table_stride=7), dict(q=P + 8), dict(out=P + 2), dict(workspace=P + 4), dict(q_stride=(512, 512, 4)),
        dict(out_stride=(4, 512, 128)), dict(k_page_stride=(4096, 2048, 100)),
        dict(v_page_stride=(4096, 8, 128), cache_dtype=3, k_scale=P, v_scale=P), dict(table=P + 2), dict(prefix_table=P + 1),
        dict(prefix_len=P + 2), dict(lens=P + 1), dict(lse=P + 2), dict(status=P + 2),
        dict(cache_dtype=3, k_scale=P, v_scale=P + 1)]),
    ("mk_prefix_attention", prefix, UNSUPPORTED, [
        dict(head_dim=8), dict(head_dim=100), dict(head_dim=288), dict(dtype=2), dict(cache_dtype=1), dict(cache_dtype=2),
        dict(max_pages=1 << 20, page_size=1 << 11, table_stride=1 << 20), dict(max_prefix_pages=1 << 27),
        dict(k_page_stride=(-4096, 2048, 128)), dict(v_page_stride=(1 << 35, 2048, 128)), dict(batch=1 << 20, rows=64)]),
    ("mk_verify_drafts", drafts, BAD, [
        dict(logits=0), dict(tokens=0), dict(noise=0), dict(accept_out=0), dict(uniforms=0), dict(workspace=0), dict(batch=-1),
        dict(rows=0), dict(rows=65), dict(batch=1 << 19), dict(vocab=0),
        dict(vocab=(1 << 24) + 1, logits_stride=1 << 25, draft_stride=1 << 25, noise_stride=1 << 25), dict(logits_stride=99),
        dict(draft_stride=99), dict(noise_stride=99), dict(workspace_bytes=64), dict(workspace_bytes=-1), dict(logits=P + 2),
        dict(draft_logits=P + 1), dict(logits=P + 1, dtype=0), dict(tokens=P + 2), dict(n_drafts=P + 1), dict(positions=P + 2),
        dict(temperature=P + 1), dict(uniforms=P + 2), dict(noise=P + 2), dict(accept_out=P + 2), dict(logprobs=P + 1),
        dict(workspace=P + 8), dict(status=P + 2)]),
    ("mk_verify_drafts", drafts, UNSUPPORTED, [dict(dtype=3), dict(dtype=-1)]),
]


@pytest.mark.parametrize("name, make, code, change", [(n, m, c, k) for n, m, c, ks in REFUSALS for k in ks])
def test_refusals(lib, name, make, code, change):
    assert getattr(lib, name)(C.byref(make(**change)), 0, None) == code


@pytest.mark.parametrize("field", ["k_page_stride", "v_page_stride"])
@pytest.mark.parametrize("strides", [(0, 2048, 128), (4096, 0, 128), (4096, 2048, 0)])
def test_caches_expanded_over_a_dimension(lib, field, strides):
    """Refused by mk_prefix_attention, except where the dimension has one element."""
    counts = dict(n_pages=32, n_kv_heads=2, page_size=16)
    assert lib.mk_prefix_attention(C.byref(prefix(**{field: strides})), 0, None) == UNSUPPORTED
    one = [k for k, x in zip(counts, strides) if x == 0][0]
    shape = {one: 1, **({"n_q_heads": 1} if one == "n_kv_heads" else {})}
    assert lib.mk_prefix_attention(C.byref(prefix(**{field: strides}, **shape, batch=0)), 0, None) == 0


@pytest.mark.parametrize("name, make", [("mk_rms_norm", norm), ("mk_prefix_attention", prefix), ("mk_verify_drafts", drafts)])
def test_null_arguments_and_devices(lib, name, make):
    fn = getattr(lib, name)
    assert fn(None, 0, None) == BAD
    assert fn(C.byref(make()), -1, None) == BAD
    assert fn(C.byref(make()), 64, None) == BAD


def test_nothing_to_do(lib):
    """Calls without rows succeed and touch nothing (no device is needed)."""
    assert lib.mk_rms_norm(C.byref(norm(rows=0)), 0, None) == 0
    assert lib.mk_prefix_attention(C.byref(prefix(batch=0)), 0, None) == 0
    assert lib.mk_verify_drafts(C.byref(drafts(batch=0)), 0, None) == 0


def test_workspaces(lib):
    n = C.c_uint64(0)
    fn = lib.mk_verify_drafts_workspace
    assert fn(None, 0, C.byref(n)) == BAD and fn(C.byref(drafts()), 0, None) == BAD
    assert fn(C.byref(drafts(dtype=3)), 0, C.byref(n)) == UNSUPPORTED and fn(C.byref(drafts()), 64, C.byref(n)) == BAD
    sizes = []
    for change in (dict(), dict(batch=4), dict(batch=4, rows=5), dict(batch=4, rows=5, vocab=200000), dict(batch=4, rows=64, vocab=1 << 24)):
        assert fn(C.byref(drafts(**change)), 0, C.byref(n)) == 0
        sizes.append(n.value)
    assert sizes == sorted(sizes) and sizes[0] > 0
    # what it says is enough, one byte less is not
    assert lib.mk_verify_drafts_check(C.byref(drafts(workspace_bytes=sizes[0])), 0) == 0
    assert lib.mk_verify_drafts_check(C.byref(drafts(workspace_bytes=sizes[0] - 1)), 0) == BAD
    fn = lib.mk_prefix_attention_workspace
    assert fn(None, 0, C.byref(n)) == BAD and fn(C.byref(prefix()), 0, None) == BAD
    assert fn(C.byref(prefix(head_dim=100)), 0, C.byref(n)) == UNSUPPORTED and fn(C.byref(prefix()), 64, C.byref(n)) == BAD
    assert fn(C.byref(prefix(batch=1 << 20, rows=64)), 0, C.byref(n)) == UNSUPPORTED


@pytest.mark.parametrize("code, change", [(c, k) for n, m, c, ks in REFUSALS if n == "mk_verify_drafts" for k in ks])
def test_verify_drafts_check_refuses_what_the_call_refuses(lib, code, change):
    assert lib.mk_verify_drafts_check(C.byref(drafts(**change)), 0) == code


def test_verify_drafts_check_without_rows_arguments_or_a_device(lib):
    fn = lib.mk_verify_drafts_check
    assert fn(None, 0) == BAD and fn(C.byref(drafts()), -1) == BAD and fn(C.byref(drafts()), 64) == BAD
    assert fn(C.byref(drafts(batch=0)), 0) == 0 and fn(C.byref(drafts()), 0) == 0


def test_struct_layouts_match_the_header():
    structs = {"mk_rms_norm_args": binding.RmsNormArgs, "mk_prefix_attention_args": binding.PrefixAttentionArgs,
               "mk_verify_drafts_args": binding.VerifyDraftsArgs}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "mk.h"', 'int main(void) {']
    for name, cls in structs.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    lines.append('return 0; }')
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(src, "w").write("\n".join(lines))
        subprocess.run(["gcc", "-std=c99", "-I" + os.path.join(ROOT, "include"), src, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    for line in out.splitlines():
        key, off = line.split()
        name, _, f = key.partition(".")
        assert (getattr(structs[name], f).offset if f else C.sizeof(structs[name])) == int(off), key


@pytest.mark.parametrize("pack, a", [(serving._pack_norm, norm(dtype=1, out_dtype=3)),
                                     (serving._pack_prefix, prefix(k_scale=5, v_scale=6, lse=7, status=8, dtype=1, cache_dtype=3)),
                                     (serving._pack_drafts, drafts(n_drafts=5, positions=6, temperature=7, logprobs=8, status=9))])
def test_packed_arguments_are_the_structs(pack, a):
    vals = []
    for f, _ in a._fields_:
        v = getattr(a, f)
        vals += list(v) if hasattr(v, "__len__") else [v or 0]
    assert pack(*vals) == bytes(a)


def test_sampling_that_does_not_fit_is_refused_before_the_step():
    """A step cannot be taken back, so nothing of it is enqueued when its sampling is wrong."""
    class Lib:
        def mk_decode_step(self, *args):
            raise AssertionError("the step ran")

        mk_verify_step = mk_decode_step

    m = binding.Megakernel.__new__(binding.Megakernel)
    m.lib, m.device, m.h = Lib(), -1, None
    m.cfg = type("Cfg", (), {"vocab": 8})
    tok = torch.zeros(2, 1, dtype=torch.int32)
    accept = torch.zeros(3, 2, dtype=torch.int32)
    for z in (None, torch.zeros(3, 8), torch.zeros(2, 8)):  # none, another number of rows, not on a GPU
        with pytest.raises(ValueError):
            m.verify(tok, tok[:, 0], accept, z, sampling=dict(noise=torch.ones(2, 8)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float64, torch.int32])
def test_sampling_of_logits_that_are_not_fp32_is_refused_before_the_step(monkeypatch, dtype):
    """The step writes fp32 rows, so a buffer of another type is not one for it, whatever the operator takes."""
    class Lib:
        def mk_decode_step(self, *args):
            raise AssertionError("the step ran")

    monkeypatch.setattr(serving, "prepare_verify_drafts", lambda *args, **kw: ((), None))
    monkeypatch.setattr(serving, "check_verify_drafts", lambda call: None)
    m = binding.Megakernel.__new__(binding.Megakernel)
    m.lib, m.device, m.h = Lib(), -1, None
    m.cfg = type("Cfg", (), {"vocab": 8})
    tok = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        m.verify(tok, tok[:, 0], torch.zeros(3, 2, dtype=torch.int32), torch.zeros(4, 8, dtype=dtype), sampling={})


def test_wrappers_refuse_cpu_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mk.rms_norm(x[:, 0], x[:, 0])
    with pytest.raises(ValueError):
        mk.prefix_attention(x[:, None], x[None], x[None], i, i[:1], i[:, None], i, x[:, None])
    with pytest.raises(ValueError):
        mk.prefix_attention_workspace(x[:, None], x[None], i, i[:, None])
    with pytest.raises(ValueError):
        mk.verify_drafts(torch.zeros(2, 8), i[:, None], torch.ones(2, 8), None, torch.zeros(3, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        mk.verify_drafts_workspace(torch.zeros(2, 8), i[:, None])
