"""Host-side refusals of the paged 8-bit cache's entry points: wrong sizes, types and pointers
return a status before any CUDA call (nothing here needs a GPU)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import scaled_reference as ref
from mla_decode_speculative_gb300 import build, mla, runner

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mla_gb300.h")
VP = ctypes.c_void_p
INVALID, UNSUPPORTED, WORKSPACE = mla.MLA_ERR_INVALID_ARG, mla.MLA_ERR_UNSUPPORTED, mla.MLA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    build.build()
    return mla.lib()


def _tables(**kw):
    a = mla.TableArgs(num_reqs=2, num_rows=4, prev_lens=256, seq_lens=256, qo_indptr=256, world_size=1, rank=0,
                      interleave=1, block_size=16, num_blocks=8, block_table=256, block_table_stride=4, free_ring=256,
                      ring_in=256, ring_out=512, slot_map=256)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(num_reqs=-1), INVALID), (dict(num_rows=-1), INVALID), (dict(world_size=0), INVALID),
    (dict(rank=1), INVALID), (dict(rank=-1), INVALID), (dict(interleave=0), INVALID),
    (dict(world_size=1 << 20, interleave=1 << 20), INVALID), (dict(block_size=0), INVALID),
    (dict(num_blocks=0), INVALID), (dict(num_blocks=1 << 27, block_size=32), INVALID),
    (dict(block_table_stride=0), INVALID), (dict(num_reqs=1 << 14, block_table_stride=1 << 18), INVALID),
    (dict(prev_lens=None), INVALID), (dict(seq_lens=None), INVALID), (dict(qo_indptr=None), INVALID),
    (dict(block_table=None), INVALID), (dict(free_ring=None), INVALID), (dict(ring_in=None), INVALID),
    (dict(ring_out=None), INVALID), (dict(ring_out=256), INVALID), (dict(ring_out=252), INVALID),
    (dict(ring_out=260), INVALID), (dict(slot_map=None), INVALID),
    (dict(num_reqs=16385), UNSUPPORTED)])
def test_table_refusals(L, change, status):
    assert L.mla_update_block_tables(ctypes.byref(_tables(**change)), None) == status
    assert b"mla_update_block_tables" in L.mla_last_error_string()


@pytest.mark.parametrize("lens_out", [None, 256, 260, 252, 1024, 1028])
def test_table_lens_out_refusals(L, lens_out):
    """Null, or overlapping prev_lens (at 256) or seq_lens (at 1024), two requests each."""
    a = _tables(seq_lens=1024)
    assert L.mla_update_block_tables_lens(ctypes.byref(a), VP(lens_out) if lens_out else None, None) == INVALID
    assert b"lens_out" in L.mla_last_error_string()
    assert L.mla_update_block_tables_lens(None, VP(4096), None) == INVALID
    assert L.mla_update_block_tables_lens(ctypes.byref(_tables(seq_lens=1024, rank=1)), VP(4096), None) == INVALID


def test_null_structs(L):
    assert L.mla_update_block_tables(None, None) == INVALID
    assert L.mla_decode_verify_scaled(None, VP(256), 16, VP(256), 1 << 20, None) == INVALID


@pytest.mark.parametrize("args,status", [
    ((-1, 256, 256, 256, 256, 16, 64), INVALID), ((4, None, 256, 256, 256, 16, 64), INVALID),
    ((4, 256, None, 256, 256, 16, 64), INVALID), ((4, 256, 256, None, 256, 16, 64), INVALID),
    ((4, 256, 256, 256, None, 16, 64), INVALID), ((4, 256, 256, 256, 256, 0, 64), UNSUPPORTED),
    ((4, 256, 256, 256, 256, 3, 63), UNSUPPORTED), ((4, 256, 256, 256, 256, 128, 256), UNSUPPORTED),
    ((4, 256, 256, 256, 256, 16, 40), INVALID), ((4, 256, 256, 256, 256, 16, 0), INVALID),
    ((4, 256, 256, 256, 256, 16, 1 << 31), INVALID), ((4, 264, 256, 256, 256, 16, 64), INVALID),
    ((4, 256, 256, 264, 256, 16, 64), INVALID)])
def test_write_refusals(L, args, status):
    T, x, slots, cache, scales, G, rows = args
    vp = [VP(p) if p else None for p in (x, slots, cache, scales)]
    assert L.mla_write_kv_scaled(T, *vp, G, rows, None) == status
    assert b"mla_write_kv_scaled" in L.mla_last_error_string()


def _decode(**kw):
    a = mla.DecodeArgs()
    a.num_reqs, a.num_rows, a.num_heads, a.max_qlen = 1, 1, 16, 1
    a.kv_dtype, a.sm_scale, a.kv_scale = mla.MLA_KV_FP8_E4M3, 0.07, 0.0   # kv_scale is not looked at
    a.q = a.kv_cache = a.qo_indptr = a.row_len = a.subpage_table = a.out = a.lse = 256
    a.num_cache_rows, a.subpage_stride, a.page_size, a.num_segments = 64, 4, 16, 4
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,G,status", [
    (dict(kv_dtype=mla.MLA_KV_BF16), 16, UNSUPPORTED), (dict(flags=mla.MLA_DECODE_FUSED_MERGE), 16, UNSUPPORTED),
    (dict(flags=mla.MLA_DECODE_UNIFORM_SEGMENTS), 16, UNSUPPORTED),
    (dict(flags=mla.MLA_DECODE_SKIP_MERGE), 16, UNSUPPORTED), (dict(flags=8), 16, INVALID),
    (dict(), 0, UNSUPPORTED), (dict(), 12, UNSUPPORTED), (dict(), 32, UNSUPPORTED),
    (dict(page_size=128, num_cache_rows=128), 128, UNSUPPORTED), (dict(num_cache_rows=72), 16, INVALID),
    (dict(page_size=4), 4, UNSUPPORTED), (dict(num_segments=1025), 16, UNSUPPORTED), (dict(q=264), 16, INVALID),
    (dict(subpage_stride=(1 << 28) - 1, page_size=8), 8, UNSUPPORTED),
    (dict(wait_cycles=-1), 16, INVALID), (dict(sm_scale=0.0), 16, INVALID), (dict(), 16, WORKSPACE)])
def test_decode_refusals(L, change, G, status):
    a = _decode(**change)
    assert L.mla_decode_verify_scaled(ctypes.byref(a), VP(256), G, None, 0, None) == status
    assert L.mla_decode_verify_scaled(ctypes.byref(_decode()), None, 16, VP(256), 1 << 30, None) == INVALID


def test_table_struct_matches_the_header(tmp_path):
    fields = [f for f, _ in mla.TableArgs._fields_]
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mla_gb300.h"\nint main(void) {\n'
                   + '  printf("%zu\\n", sizeof(mla_table_args));\n'
                   + "".join(f'  printf("%zu\\n", offsetof(mla_table_args, {f}));\n' for f in fields)
                   + "  return 0;\n}\n")
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(mla.TableArgs)] + [getattr(mla.TableArgs, f).offset for f in fields]


def test_wrapper_refusals_on_the_host():
    """Shapes that the binding itself refuses, before it looks at devices."""
    cache, scales = torch.zeros((64, 576), dtype=torch.uint8), torch.ones(4)
    for bad in ((cache[:, :512], scales, 16), (cache.float(), scales, 16), (cache, scales, 8), (cache, scales, 0)):
        with pytest.raises(ValueError):
            mla._check_scaled(*bad)
    mla._check_scaled(cache, scales, 16)


@pytest.mark.parametrize("scale_block,block_size", [(0, 16), (3, 48), (128, 128), (16, 24), (32, 16)])
def test_cache_refuses_scale_blocks(scale_block, block_size):
    with pytest.raises(ValueError, match="scale_block"):
        runner.PagedLatentCache(num_reqs=1, num_rows=1, num_blocks=1, block_size=block_size, max_kv_len=48,
                                scale_block=scale_block, device="cpu")


def test_reference_encoder_is_the_oracles():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(400) * 2.0 ** rng.integers(-12, 10, 400), ref.CODE_VALUE[:127],
                        (ref.CODE_VALUE[:126] + ref.CODE_VALUE[1:127]) / 2, [0.0, -0.0, 448.0, 500.0, -1e9]])
    x = x.astype(np.float32)
    assert [int(c) for c in ref.encode(x)] == [oracle_code(v) for v in x]
    assert ref.encode(np.array([np.nan]))[0] == 127 and ref.encode(np.array([-np.inf]))[0] == 0xFE


def oracle_code(v):
    import oracle
    return oracle.e4m3_encode(float(v))
