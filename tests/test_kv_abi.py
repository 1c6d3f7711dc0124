"""Host-side checks of the key/value cache's C ABI (include/qlora_kv.h): every
declared entry point is exported and bound, and bad arguments are refused
before any launch (fake device addresses, no GPU needed); the code search's
bucket table, compiled for the host."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest

from bit_nf4_quantized_quant_amd import _lib
from bit_nf4_quantized_quant_amd.kv import _CacheStruct

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qlora_kv.h")
CSRC = os.path.join(ROOT, "bit_nf4_quantized_quant_amd", "csrc")
A, MIS = 0x10000, 0x10004
OK, EINVAL, ESHAPE = _lib.QLORA_OK, _lib.QLORA_EINVAL, _lib.QLORA_ESHAPE

needs_lib = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libqlora.so not built")


def cache(k=A, ks=A, v=A, vs=A, pages=4, heads=2, page=16, dim=128, table=0):
    return ctypes.byref(_CacheStruct(k, ks, v, vs, pages, heads, page, dim, table))


@needs_lib
def test_declarations_are_exported_and_bound():
    names = set(re.findall(r"\b(qlora_kv_[a-z_]+)\s*\(", open(HEADER).read()))
    assert names == set(_lib.KV_SIGNATURES)
    for n in names:
        assert hasattr(_lib.lib(), n), n


BAD_CACHES = [(dict(dim=96), ESHAPE), (dict(dim=512), ESHAPE), (dict(dim=-128), EINVAL), (dict(page=24), ESHAPE),
              (dict(page=0), ESHAPE), (dict(page=-16), EINVAL), (dict(pages=0), ESHAPE), (dict(heads=0), ESHAPE),
              (dict(heads=1 << 17), ESHAPE), (dict(pages=1 << 31), ESHAPE), (dict(pages=1 << 26), ESHAPE),
              (dict(page=1 << 40), ESHAPE), (dict(table=3), EINVAL), (dict(table=-1), EINVAL)]
BAD_POINTERS = [dict(k=0), dict(ks=0), dict(v=0), dict(vs=0), dict(k=MIS), dict(ks=MIS), dict(v=MIS), dict(vs=MIS)]


def write(c="good", k=A, v=A, dtype=0, tokens=4, strides=(256, 128, 256, 128), slots=A):
    s = None if strides is None else (ctypes.c_int64 * 4)(*strides)
    return _lib.lib().qlora_kv_write(cache() if c == "good" else c, k, v, dtype, tokens, s, slots, None)


def read(c="good", slots=A, tokens=4, dtype=0, k=A, v=A):
    return _lib.lib().qlora_kv_read(cache() if c == "good" else c, slots, tokens, dtype, k, v, None)


def attend(c="good", q=A, strides=(512, 128), tokens=4, heads=4, bt=A, width=2, lengths=A, starts=None, seqs=4, max_q=1,
           max_len=32, window=0, out=A, lse=None, ws=A, ws_bytes=1 << 30, scale=0.1):
    s = None if strides is None else (ctypes.c_int64 * 2)(*strides)
    return _lib.lib().qlora_kv_attention(cache() if c == "good" else c, q, s, tokens, heads, bt, width, lengths, starts, seqs, max_q,
                                         max_len, scale, 1, window, out, lse, ws, ws_bytes, None)


@needs_lib
def test_caches_refused():
    for call in (write, read, attend):
        assert call(None) == EINVAL
        for kw, status in BAD_CACHES:
            assert call(cache(**kw)) == status, (call.__name__, kw)
        for kw in BAD_POINTERS:
            assert call(cache(**kw)) == EINVAL, (call.__name__, kw)


@needs_lib
def test_write_refusals():
    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(strides=None), dict(k=MIS), dict(v=MIS),
               dict(slots=A + 2), dict(dtype=2), dict(dtype=-1), dict(tokens=-1), dict(strides=(-256, 128, 256, 128))):
        assert write(**kw) == EINVAL, kw
    for kw in (dict(strides=(257, 128, 256, 128)), dict(strides=(256, 128, 256, 4)), dict(tokens=1 << 31),
               dict(strides=(1 << 40, 128, 256, 128)), dict(dtype=1, strides=(256, 130, 256, 128))):
        assert write(**kw) == ESHAPE, kw
    assert write(tokens=0, k=None, v=None, slots=None) == OK


@needs_lib
def test_read_refusals():
    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(k=MIS), dict(v=MIS), dict(slots=A + 2),
               dict(dtype=2), dict(tokens=-4)):
        assert read(**kw) == EINVAL, kw
    assert read(tokens=1 << 31) == ESHAPE
    assert read(tokens=0, k=None, v=None, slots=None) == OK


@needs_lib
def test_attention_refusals():
    for kw in (dict(q=None), dict(q=MIS), dict(strides=None), dict(bt=None), dict(bt=A + 2), dict(lengths=None),
               dict(lengths=A + 1), dict(starts=A + 2), dict(out=None), dict(out=MIS), dict(lse=A + 2),
               dict(tokens=-1), dict(heads=-4), dict(seqs=-1), dict(max_q=-1), dict(max_len=-1), dict(window=-1),
               dict(width=-1), dict(strides=(-512, 128)), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert attend(**kw) == EINVAL, kw
    for kw in (dict(heads=3), dict(heads=0), dict(heads=1 << 17), dict(strides=(516, 128)), dict(strides=(512, 1 << 40)),
               dict(tokens=5), dict(max_q=2), dict(max_q=0), dict(seqs=1 << 16, tokens=1 << 16), dict(max_len=1 << 31),
               dict(starts=A, max_q=1 << 30), dict(width=1 << 28)):
        assert attend(**kw) == ESHAPE, kw
    assert attend(tokens=0, seqs=0, q=None, lengths=None, out=None) == OK


@needs_lib
def test_attention_workspace_is_asked_for():
    L = _lib.lib()
    size = L.qlora_kv_attention_workspace
    assert size(cache(), 3, 4, 4, 1, 32, 0) == 0 and size(cache(dim=96), 4, 4, 4, 1, 32, 0) == 0
    assert size(cache(), 4, 0, 4, 1, 32, 0) == size(cache(), 4, 4, 0, 1, 32, 0) == size(cache(), 4, 4, 4, 0, 32, 0) == 0
    long = dict(tokens=1, seqs=1, max_len=1 << 20, width=1 << 16)
    need = size(cache(), 4, 1, 1, 1, 1 << 20, 0)
    if need:
        assert attend(ws=None, ws_bytes=need, **long) == EINVAL
        assert attend(ws=A + 16, ws_bytes=need, **long) == EINVAL
        assert attend(ws_bytes=need - 1, **long) == EINVAL


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_code_search_buckets(tmp_path):
    exe = str(tmp_path / "kv_table_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-I", CSRC, os.path.join(ROOT, "tests", "host", "kv_table_check.cpp"),
                    os.path.join(CSRC, "nf4_table.cpp"), "-o", exe, "-lpthread"],
                   check=True, capture_output=True, text=True)
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip().endswith("OK"), run.stdout[-3000:] + run.stderr[-3000:]
