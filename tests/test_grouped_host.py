"""Host-side refusals of the rotary calls and of grouped and differential attention: wrong sizes, types,
strides and pointers return a status before any CUDA call (nothing here needs a GPU)."""
import ctypes
import math
import os
import subprocess
from fractions import Fraction

import numpy as np
import pytest
import torch

from mla_decode_speculative_gb300 import build, mla, runner

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mla_gb300.h")
VP = ctypes.c_void_p
INVALID, UNSUPPORTED, WORKSPACE = mla.MLA_ERR_INVALID_ARG, mla.MLA_ERR_UNSUPPORTED, mla.MLA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    build.build()
    return mla.lib()


def _heads(count, change, src, dst, dim=64):
    h = mla.Heads(count, dim, src, count * dim, dim, dst, count * dim, dim)
    for k, v in dict(change).items():
        setattr(h, k, v)
    return h


def _rotary(q=(), k=(), v=None, **kw):
    a = mla.RotaryArgs(num_rows=4, num_axes=1, rot_dim=64, neighbours=0, positions=256, axis_stride=4, turns=256,
                       q=_heads(8, q, 256, 256), k=_heads(2, k, 512, 1024), slot_map=256,
                       num_cache_rows=64)
    if v is not None:
        a.v = _heads(2, v, 512, 4096)
    for key, value in kw.items():
        setattr(a, key, value)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(num_rows=-1), INVALID), (dict(num_axes=0), INVALID), (dict(axis_stride=-1), INVALID),
    (dict(rot_dim=0), UNSUPPORTED), (dict(rot_dim=63), UNSUPPORTED), (dict(rot_dim=514), UNSUPPORTED),
    (dict(positions=None), INVALID), (dict(turns=None), INVALID), (dict(q=dict(heads=-1)), INVALID),
    (dict(q=dict(dim=62)), INVALID), (dict(q=dict(dim=1 << 17)), INVALID), (dict(q=dict(src=None)), INVALID),
    (dict(q=dict(dst=None)), INVALID), (dict(q=dict(src_row=-1)), INVALID), (dict(q=dict(dst_head=32)), INVALID),
    (dict(q=dict(dst_row=32)), INVALID), (dict(q=dict(dst_row=256)), INVALID), (dict(q=dict(src_row=1024)), INVALID),
    (dict(q=dict(src=257)), INVALID), (dict(k=dict(dst_row=64)), INVALID), (dict(v={}), INVALID)])
def test_rotary_refusals(L, change, status):
    assert L.mla_rotary(ctypes.byref(_rotary(**change)), None) == status
    assert b"mla_rotary" in L.mla_last_error_string()


@pytest.mark.parametrize("change,status", [
    (dict(v=dict(heads=0)), INVALID), (dict(k=dict(heads=0)), INVALID), (dict(v=dict(dim=0)), INVALID),
    (dict(v=dict(dst=None)), INVALID), (dict(v=dict(dst_row=100)), INVALID), (dict(slot_map=None), INVALID),
    (dict(num_cache_rows=0), INVALID), (dict(num_cache_rows=1 << 31), INVALID), (dict(rot_dim=66), INVALID)])
def test_rotary_write_refusals(L, change, status):
    a = _rotary(**{"v": {}, **change})
    assert L.mla_rotary_write(ctypes.byref(a), None) == status
    assert b"mla_rotary_write" in L.mla_last_error_string()


@pytest.mark.parametrize("heads,dim,src", [(65536, 65536, 514), (65536, 65536, 512), (65535, 65535, 514), (40000, 60001, 514)])
def test_rows_wider_than_an_int_are_refused(L, heads, dim, src):
    """2^32 values a row, one at a time: refused before anything is divided by their number as an int, which is 0."""
    a = _rotary(v={})
    a.v = mla.Heads(heads, dim, src, heads * dim, dim, 4096, heads * dim, dim)
    assert L.mla_rotary_write(ctypes.byref(a), None) == UNSUPPORTED
    assert b"too many" in L.mla_last_error_string()


def test_null_structs_and_nothing_to_do(L):
    assert L.mla_rotary(None, None) == INVALID and L.mla_rotary_write(None, None) == INVALID
    assert L.mla_decode_grouped(None, VP(256), 1 << 20, None) == INVALID
    assert L.mla_decode_differential(None, VP(256), None, 0.0, VP(256), 1 << 20, None) == INVALID
    assert L.mla_decode_grouped_workspace(None, 0) == 0
    assert L.mla_rotary(ctypes.byref(_rotary(num_rows=0)), None) == 0
    assert L.mla_rotary(ctypes.byref(_rotary(q=dict(heads=0), k=dict(heads=0))), None) == 0


def _grouped(**kw):
    a = mla.GroupedArgs(num_reqs=1, num_rows=4, num_heads=8, num_kv_heads=2, max_qlen=4, head_dim=64, window=0,
                        sm_scale=0.1, q=256, q_row=1024, k_cache=256, k_row=256, v_cache=256, v_row=256, num_cache_rows=64,
                        qo_indptr=256, row_len=256, subpage_table=256, subpage_stride=4, page_size=16, out=256, lse=256)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(num_reqs=0), INVALID), (dict(num_rows=0), INVALID), (dict(num_heads=0), INVALID), (dict(num_kv_heads=3), INVALID),
    (dict(num_kv_heads=0), INVALID), (dict(max_qlen=0), INVALID), (dict(max_qlen=5), INVALID),
    (dict(head_dim=80), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED), (dict(head_dim=512), UNSUPPORTED),
    (dict(page_size=4), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
    (dict(subpage_stride=0), INVALID), (dict(subpage_stride=1 << 28, page_size=8), INVALID),
    (dict(num_cache_rows=0), INVALID), (dict(num_cache_rows=60), INVALID), (dict(num_cache_rows=1 << 31), INVALID),
    (dict(num_rows=1 << 29), INVALID), (dict(window=-1), INVALID), (dict(wait_cycles=-1), INVALID),
    (dict(sm_scale=0.0), INVALID), (dict(sm_scale=float("nan")), INVALID), (dict(sm_scale=float("inf")), INVALID),
    (dict(q=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID), (dict(out=None), INVALID),
    (dict(lse=None), INVALID), (dict(row_len=None), INVALID), (dict(qo_indptr=None), INVALID),
    (dict(subpage_table=None), INVALID), (dict(q=264), INVALID), (dict(k_cache=258), INVALID), (dict(v_cache=264), INVALID),
    (dict(out=264), INVALID), (dict(q_row=1028), INVALID), (dict(k_row=260), INVALID), (dict(v_row=252), INVALID),
    (dict(q_row=504), INVALID), (dict(k_row=120), INVALID), (dict(v_row=1 << 40), INVALID)])
def test_grouped_refusals(L, change, status):
    a = _grouped(**change)
    assert L.mla_decode_grouped(ctypes.byref(a), VP(256), 1 << 40, None) == status
    assert b"mla_decode_grouped" in L.mla_last_error_string()


def test_differential_refusals(L):
    call = lambda a, lam=VP(256), gain=None, eps=0.0: L.mla_decode_differential(  # noqa: E731
        ctypes.byref(a), lam, gain, eps, VP(256), 1 << 40, None)
    assert call(_grouped(head_dim=256, q_row=8192, k_row=2048, v_row=2048)) == UNSUPPORTED
    assert call(_grouped(), lam=None) == INVALID and b"lambda" in L.mla_last_error_string()
    assert call(_grouped(), gain=VP(256), eps=-1.0) == INVALID
    assert call(_grouped(), gain=VP(256), eps=float("nan")) == INVALID
    assert call(_grouped(q_row=1016)) == INVALID      # two maps of 8 heads of 64 need 1024
    assert call(_grouped(k_row=248)) == INVALID


@pytest.mark.parametrize("differential", [0, 1])
def test_workspace_refusals(L, differential):
    a = _grouped()
    need = L.mla_decode_grouped_workspace(ctypes.byref(a), differential)
    assert need > 0
    call = L.mla_decode_grouped if not differential else \
        lambda a, w, n, s: L.mla_decode_differential(a, VP(256), None, 0.0, w, n, s)
    for ws, n in ((None, need), (VP(256), need - 1), (VP(264), need)):
        assert call(ctypes.byref(a), ws, n, None) == WORKSPACE
    assert L.mla_decode_grouped_workspace(ctypes.byref(_grouped(head_dim=96)), differential) == 0


@pytest.mark.parametrize("differential", [0, 1])
def test_single_row_has_no_stride(L, differential):
    """One row of queries: the distance to a next one is not looked at (what follows is the workspace's check)."""
    for q_row in (0, 64, 513, -8, 1 << 40):
        a = _grouped(num_rows=1, max_qlen=1, q_row=q_row)
        status = L.mla_decode_differential(ctypes.byref(a), VP(256), None, 0.0, None, 0, None) if differential else \
            L.mla_decode_grouped(ctypes.byref(a), None, 0, None)
        assert status == WORKSPACE, L.mla_last_error_string()


def test_structs_match_the_header(tmp_path):
    structs = {"mla_heads": mla.Heads, "mla_rotary_args": mla.RotaryArgs, "mla_grouped_args": mla.GroupedArgs}
    src = tmp_path / "t.c"
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "mla_gb300.h"', "int main(void) {"]
    want = []
    for name, cls in structs.items():
        lines.append(f'  printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append(f'  printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(cls, f).offset)
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    assert [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()] == want


def test_turns_are_the_frequencies_to_half_a_unit():
    """|turns / 2^64 - freq / (2 pi)| <= 2^-65 modulo 1, against a longer pi (to 60 digits)."""
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)
    f = [1.0, 0.9, 1e-4, 10000.0 ** -0.37, 3.0, -0.25, 0.0, 1e5, 1e-300, -4e9]
    got = mla.rotary_turns(f, device="cpu")
    assert got.dtype == torch.int64 and got.shape == (len(f),)
    for x, t in zip(f, got.tolist()):
        off = Fraction(t, 2 ** 64) - Fraction(x) / (2 * pi)
        off -= round(off)
        assert abs(off) <= Fraction(1, 2 ** 65) * Fraction(1001, 1000)
    for bad in ([[1.0]], [math.inf], [math.nan], [2.0 ** 32], [-1e300]):
        with pytest.raises(ValueError):
            mla.rotary_turns(bad, device="cpu")


def test_wrapper_refusals_on_the_host():
    """Shapes and strides that the binding itself refuses, before it looks at devices."""
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    for src, dst in ((x[0], x), (x, x[:, :, :32]), (x, x[:, :1]), (x[:3], x), (x, x[:3]), (x, x[0]), (x, x[:, :, ::2])):
        with pytest.raises(ValueError):
            mla._heads(src, dst, 4, -1, "q")
    with pytest.raises(ValueError, match="contiguous"):
        mla._heads(x.transpose(1, 2), None, 4, -1, "q")
    with pytest.raises(TypeError):
        mla._heads(x.float(), None, 4, -1, "q")
    with pytest.raises(ValueError, match="device"):
        mla._heads(x, None, 4, 0, "q")
    assert mla._heads(x, None, 4, -1, "q")[:2] == (2, 64) and mla._heads(x, x[..., :], 4, -1, "q")[6:] == (128, 64)
    pos, turns = torch.zeros((3, 4), dtype=torch.int32), mla.rotary_turns([1.0, 0.5], device="cpu")
    for bad in ((pos.long(), turns, None), (pos.T, turns, None), (pos[None], turns, None), (pos, turns, torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            mla._angles(*bad, False, -1)
    ind, lens, sub = torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.zeros((1, 4), dtype=torch.int32)
    cache = torch.zeros((64, 2, 64), dtype=torch.bfloat16)
    call = lambda q, k, v, lens=lens, maps=1: mla._grouped(q, k, v, ind, lens, sub, 16, 4, 0.1, 0, None, None, 0, -1, maps)  # noqa: E731
    for bad in ((x, cache, cache[:, :1]), (x, cache[:, :, :32], cache), (x[:, :, :32], cache, cache), (x, cache, cache[:32])):
        with pytest.raises(ValueError):
            call(*bad)
    with pytest.raises(ValueError):
        call(x, cache, cache, lens[:3])
    with pytest.raises(ValueError):
        call(x, cache, cache, maps=2)
    with pytest.raises(ValueError, match="contiguous"):
        call(x, cache.transpose(0, 1).contiguous().transpose(0, 1), cache)
    with pytest.raises(ValueError, match="contiguous"):
        call(torch.zeros((4, 4, 2, 64), dtype=torch.bfloat16)[:, ::2], cache.unflatten(1, (2, 1)).expand(-1, -1, 2, -1),
             torch.zeros((64, 2, 128), dtype=torch.bfloat16), maps=2)


def test_packed_arguments_are_the_structures_bytes():
    """The bytes that the binding packs are those of the ctypes structure with the same fields."""
    values = list(range(1, 8)) + [0.5] + list(range(9, 24))
    assert mla._pack_grouped(*values) == bytes(mla.GroupedArgs(*values))
    heads = [mla.Heads(*range(8 * i, 8 * i + 8)) for i in (1, 2, 3)]
    a = mla.RotaryArgs(1, 2, 3, 4, 5, 6, 7, 8, *heads, 9, 10)
    assert mla._pack_rotary(1, 2, 3, 4, 5, 6, 7, 8, *range(8, 32), 9, 10) == bytes(a)


def test_step_and_cache_refusals():
    cache = runner.PagedKVCache(num_reqs=1, num_rows=4, num_blocks=4, block_size=16, max_kv_len=64, num_kv_heads=2,
                                head_dim=64, device="cpu")
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    for q, k, v in ((x[:3], x, x), (x, x[:3], x), (x, x, x[:3])):
        with pytest.raises(ValueError, match="num_rows"):
            cache.append(q, k, v, None, None, cache.lens, None)
    step = runner.GroupedStep(num_reqs=1, num_rows=4, num_heads=2, num_kv_heads=2, head_dim=64, max_qlen=4, block_size=16,
                              num_blocks=4, max_kv_len=64, device="cpu")
    with pytest.raises(ValueError, match="lam"):
        step(x, cache.k, cache.v, None, None, None, 0.1, lam=torch.ones(2))
    assert cache.k.shape == (64, 2, 64) and np.prod(cache.v.shape) == 64 * 2 * 64


@pytest.mark.parametrize("change", [
    dict(head_dim=80), dict(head_dim=256, differential=True), dict(num_heads=3), dict(num_kv_heads=0), dict(max_qlen=0),
    dict(block_size=4), dict(block_size=12), dict(block_size=0), dict(max_qlen=5), dict(window=-1)])
def test_step_that_no_call_could_take_is_not_made(change):
    """Sizes that the attention refuses are refused where the step is made, not at its first call."""
    sizes = dict(num_reqs=1, num_rows=4, num_heads=4, num_kv_heads=2, head_dim=64, max_qlen=4, block_size=16, num_blocks=4,
                 max_kv_len=64, device="cpu")
    for D, bs, differential in ((64, 8, False), (128, 24, True), (256, 256, False)):
        assert runner.GroupedStep(**{**sizes, "head_dim": D, "block_size": bs}, differential=differential).workspace.numel() > 1
    with pytest.raises((ValueError, mla.MLAError)):
        runner.GroupedStep(**{**sizes, **change})
