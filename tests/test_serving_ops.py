"""The serving operators without a GPU: the argument structs' layout and every refusal of the C entry points (each
returned before any CUDA call; the addresses are never read). No call here is valid as a whole."""
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


def tables(**kw):
    a = binding.PageTablesArgs(table=P, table_stride=8, held=P, start=P, count=P, ring=P, ring_state=P, ring_state_out=P,
                               slots=P, batch=4, max_pages=8, page_size=16, n_pages=32, ring_size=32, n_tokens=4)
    return _with(a, kw)


def qk(**kw):
    a = binding.QkNormRopeArgs(q=P, k=P, v=P, q_out=P, inv_freq=P, positions=P, slots=P, k_pages=P, v_pages=P,
                               q_stride=(512, 128), k_stride=(512, 128), v_stride=(512, 128), q_out_stride=(512, 128),
                               k_page_stride=(4096, 2048, 128), v_page_stride=(4096, 2048, 128), n_tokens=2, n_q_heads=4,
                               n_kv_heads=2, head_dim=128, rope_dim=128, n_pages=4, page_size=16, eps=1e-6)
    return _with(a, kw)


def attention(**kw):
    a = binding.PagedAttentionArgs(q=P, k_pages=P, v_pages=P, table=P, lens=P, out=P, workspace=P, workspace_bytes=1 << 40,
                                   table_stride=8, q_stride=(512, 512, 128), out_stride=(512, 512, 128),
                                   k_page_stride=(4096, 2048, 128), v_page_stride=(4096, 2048, 128), batch=2, rows=1,
                                   n_q_heads=4, n_kv_heads=2, head_dim=128, n_pages=32, page_size=16, max_pages=8, scale=1)
    return _with(a, kw)


def logits(**kw):
    a = binding.LogitControlsArgs(logits=P, out=2 * P, history=P, repetition=P, bias_ids=P, bias_vals=P, allowed=P,
                                  logits_stride=100, out_stride=100, history_stride=10, bias_stride=3, allowed_stride=4,
                                  rows=2, vocab=100, max_history=10, n_biases=3, dtype=2)
    return _with(a, kw)


def _with(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


REFUSALS = [
    ("mk_page_tables", tables, BAD, [
        dict(table=0), dict(held=0), dict(start=0), dict(count=0), dict(ring=0), dict(ring_state=0), dict(ring_state_out=0),
        dict(slots=0), dict(batch=0), dict(batch=4097), dict(max_pages=0), dict(page_size=0), dict(n_pages=0),
        dict(n_tokens=-1), dict(table_stride=7), dict(ring_size=31), dict(table=P + 2), dict(held=P + 1), dict(slots=P + 4),
        dict(starts=P + 2), dict(ring_state_out=P + 2), dict(status=P + 1)]),
    ("mk_page_tables", tables, UNSUPPORTED, [
        dict(max_pages=1 << 20, page_size=1 << 11, table_stride=1 << 20), dict(n_pages=1 << 20, page_size=1 << 11, ring_size=1 << 20)]),
    ("mk_qk_norm_rope", qk, BAD, [
        dict(q=0), dict(k=0), dict(q_out=0), dict(inv_freq=0), dict(positions=0), dict(v=0), dict(slots=0), dict(k_pages=0),
        dict(v_pages=0), dict(cache_dtype=3), dict(n_tokens=-1), dict(n_q_heads=0), dict(n_kv_heads=0), dict(n_pages=0),
        dict(page_size=0), dict(eps=-1.0), dict(eps=float("nan")), dict(q=P + 8), dict(k_out=P + 2), dict(q_gain=P + 4),
        dict(q_stride=(512, 124)), dict(k_stride=(508, 128)), dict(v_stride=(512, 4)), dict(q_out_stride=(512, 127)),
        dict(k_out=P, k_out_stride=(512, 1)), dict(k_page_stride=(4096, 2048, 132)),
        dict(v_page_stride=(4096, 2048, 136), cache_dtype=3, k_scale=P, v_scale=P), dict(positions=P + 2), dict(slots=P + 4),
        dict(inv_freq=P + 4), dict(status=P + 2), dict(cache_dtype=3, k_scale=P + 2, v_scale=P)]),
    ("mk_qk_norm_rope", qk, UNSUPPORTED, [
        dict(head_dim=8), dict(head_dim=72), dict(head_dim=272), dict(rope_dim=136), dict(rope_dim=12), dict(rope_dim=-8),
        dict(dtype=2), dict(dtype=3), dict(cache_dtype=1), dict(cache_dtype=2), dict(n_pages=1 << 20, page_size=1 << 11)]),
    ("mk_paged_attention", attention, BAD, [
        dict(q=0), dict(k_pages=0), dict(v_pages=0), dict(table=0), dict(lens=0), dict(out=0),
        dict(cache_dtype=3), dict(batch=-1), dict(rows=0), dict(n_q_heads=0), dict(n_kv_heads=0), dict(n_kv_heads=3),
        dict(n_pages=0), dict(page_size=0), dict(max_pages=0), dict(table_stride=7), dict(q=P + 8), dict(out=P + 2),
        dict(workspace=P + 4), dict(q_stride=(512, 512, 4)), dict(out_stride=(4, 512, 128)),
        dict(k_page_stride=(4096, 2048, 100)), dict(v_page_stride=(4096, 8, 128), cache_dtype=3, k_scale=P, v_scale=P),
        dict(table=P + 2), dict(lens=P + 1), dict(lse=P + 2), dict(status=P + 2), dict(cache_dtype=3, k_scale=P, v_scale=P + 1)]),
    ("mk_paged_attention", attention, UNSUPPORTED, [
        dict(head_dim=8), dict(head_dim=100), dict(head_dim=288), dict(dtype=2), dict(cache_dtype=1), dict(cache_dtype=2),
        dict(max_pages=1 << 20, page_size=1 << 11, table_stride=1 << 20), dict(k_page_stride=(-4096, 2048, 128)),
        dict(v_page_stride=(4096, 2048, -128)), dict(v_page_stride=(1 << 35, 2048, 128)),
        dict(k_page_stride=(1 << 36, 2048, 128), cache_dtype=3, k_scale=P, v_scale=P)]),
    ("mk_logit_controls", logits, BAD, [
        dict(logits=0), dict(out=0), dict(history=0), dict(bias_ids=0), dict(bias_vals=0), dict(rows=-1), dict(vocab=0), dict(rows=(1 << 20) + 1),
        dict(vocab=(1 << 24) + 1, logits_stride=1 << 25, out_stride=1 << 25, allowed_stride=1 << 20),
        dict(logits_stride=99), dict(out_stride=99), dict(history_stride=9), dict(bias_stride=2), dict(allowed_stride=3),
        dict(out=P, out_stride=104), dict(out=P, dtype=0), dict(logits=P + 2), dict(out=P + 1),
        dict(history=P + 2), dict(token=P + 1), dict(bias_vals=P + 2), dict(total_len=P + 2), dict(frequency=P + 2)]),
    ("mk_logit_controls", logits, UNSUPPORTED, [
        dict(dtype=3), dict(max_history=1 << 20, history_stride=1 << 20), dict(n_biases=2048, bias_stride=2048),
        dict(max_history=-1)]),
]


@pytest.mark.parametrize("name, make, code, change", [(n, m, c, k) for n, m, c, ks in REFUSALS for k in ks])
def test_refusals(lib, name, make, code, change):
    assert getattr(lib, name)(C.byref(make(**change)), 0, None) == code


@pytest.mark.parametrize("name, make", [("mk_page_tables", tables), ("mk_qk_norm_rope", qk),
                                        ("mk_paged_attention", attention), ("mk_logit_controls", logits)])
def test_null_arguments_and_devices(lib, name, make):
    fn = getattr(lib, name)
    assert fn(None, 0, None) == BAD
    assert fn(C.byref(make()), -1, None) == BAD
    assert fn(C.byref(make()), 64, None) == BAD


def test_nothing_to_do(lib):
    """Calls without rows succeed and touch nothing (no device is needed)."""
    assert lib.mk_qk_norm_rope(C.byref(qk(n_tokens=0)), 0, None) == 0
    assert lib.mk_paged_attention(C.byref(attention(batch=0)), 0, None) == 0
    assert lib.mk_logit_controls(C.byref(logits(rows=0)), 0, None) == 0


def test_workspace_refusals(lib):
    n = C.c_uint64(0)
    fn = lib.mk_logit_controls_workspace
    assert fn(None, 0, C.byref(n)) == BAD
    assert fn(C.byref(logits()), 0, None) == BAD
    assert fn(C.byref(logits(dtype=3)), 0, C.byref(n)) == UNSUPPORTED
    assert fn(C.byref(logits()), -1, C.byref(n)) == BAD
    fn = lib.mk_paged_attention_workspace
    assert fn(None, 0, C.byref(n)) == BAD
    assert fn(C.byref(attention()), 0, None) == BAD
    assert fn(C.byref(attention(head_dim=100)), 0, C.byref(n)) == UNSUPPORTED
    assert fn(C.byref(attention()), 64, C.byref(n)) == BAD


def test_struct_layouts_match_the_header():
    structs = {"mk_page_tables_args": binding.PageTablesArgs, "mk_qk_norm_rope_args": binding.QkNormRopeArgs,
               "mk_paged_attention_args": binding.PagedAttentionArgs, "mk_logit_controls_args": binding.LogitControlsArgs}
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


def test_packed_arguments_are_the_structs():
    """The bytes the wrappers build are what the ctypes structure with the same values holds."""
    a = attention(k_scale=5, v_scale=6, lse=7, status=8, dtype=1, cache_dtype=3)
    vals = []
    for f, _ in a._fields_:
        v = getattr(a, f)
        vals += list(v) if hasattr(v, "__len__") else [v or 0]
    assert serving._pack_attention(*vals) == bytes(a)


def test_controls_that_do_not_fit_are_refused_before_the_step():
    """A step cannot be taken back, so nothing of it is enqueued when its controls are wrong."""
    class Lib:
        def mk_decode_step(self, *args):
            raise AssertionError("the step ran")

    m = binding.Megakernel.__new__(binding.Megakernel)
    m.lib, m.device, m.h = Lib(), -1, None
    m.cfg = type("Cfg", (), {"vocab": 8})
    tok = torch.zeros(2, 1, dtype=torch.int32)
    for z in (None, torch.zeros(3, 8), torch.zeros(2, 8)):  # none, another number of rows, not on a GPU
        with pytest.raises(ValueError):
            m.step(tok, tok[:, 0], z, controls=dict(bias_ids=tok))


@pytest.mark.parametrize("code, change", [(c, k) for n, m, c, ks in REFUSALS if n == "mk_logit_controls" for k in ks])
def test_logit_controls_check_refuses_what_the_call_refuses(lib, code, change):
    assert lib.mk_logit_controls_check(C.byref(logits(**change)), 0) == code


def test_logit_controls_check_without_rows_arguments_or_a_device(lib):
    fn = lib.mk_logit_controls_check
    assert fn(None, 0) == BAD and fn(C.byref(logits()), -1) == BAD and fn(C.byref(logits()), 64) == BAD
    assert fn(C.byref(logits(rows=0)), 0) == 0


def test_wrappers_refuse_cpu_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mk.page_tables(torch.zeros(2, 4, dtype=torch.int32), i, i, i, i, i, 16, 2, slots=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        mk.qk_norm_rope(x, x, i, None, x)
    with pytest.raises(ValueError):
        mk.paged_attention(x[:, None], x[None], x[None], i[:, None], i, x[:, None])
    with pytest.raises(ValueError):
        mk.logit_controls(torch.zeros(2, 8), torch.zeros(2, 8))
