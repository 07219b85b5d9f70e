"""What the paged calls refuse before anything is launched (no GPU needed: no pointer is followed)."""
import ctypes
import os
import subprocess
import sys

import pytest

from learned_kv_cache_gb300 import _lib
from learned_kv_cache_gb300.paged import _Desc


@pytest.fixture(scope="module")
def lib():
    from learned_kv_cache_gb300 import build
    build.build()
    return _lib.load()


GOOD = dict(k_pool=4096, v_pool=8192, page_stride=0, token_stride=0, table=4096, lens=4096, refs=4096, free_mask=4096,
            score=None, pos=None, dtype=1, head_dim=128, page_size=64, n_pages=100, n_rows=8, max_pages=10)
P = 4096


def desc(**kw):
    return ctypes.byref(_Desc(**{**GOOD, **kw}))


def decode(lib, c, q=P, q_stride=0, h_q=8, h_kv=2, scale=0.1, out=P, out_dtype=0, lse=None, add=0, ws=P, ws_bytes=1 << 40):
    return lib.kvp_paged_decode_attn(q, q_stride, c, h_q, h_kv, scale, out, out_dtype, lse, add, ws, ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(k_pool=None), -1), (dict(table=None), -1), (dict(lens=None), -1), (dict(refs=None), -1),
    (dict(free_mask=None), -1), (dict(v_pool=8200), -1), (dict(dtype=5), -2), (dict(head_dim=96), -2),
    (dict(page_size=8), -2), (dict(page_size=48), -2), (dict(page_size=2048), -2), (dict(n_pages=0), -1),
    (dict(n_rows=0), -1), (dict(max_pages=0), -1), (dict(max_pages=1 << 25), -1),
    (dict(n_rows=1 << 24, max_pages=1 << 10), -1), (dict(token_stride=64), -1), (dict(token_stride=132), -1),
    (dict(page_stride=64 * 128 - 8), -1), (dict(page_stride=-8), -1), (dict(page_stride=1 << 40), -1),
])
def test_a_bad_cache_is_refused_by_every_call(lib, change, code):
    c = desc(**change)
    assert lib.kvp_paged_init(c, None) == code
    assert lib.kvp_paged_append(c, P, P, None, None, 2, 1, None, None, P, 1 << 40, None) == code
    assert lib.kvp_paged_fork(c, P, 0, None, 0, None) == code
    assert lib.kvp_paged_compact(c, P, P, 4, P, 1 << 40, None) == code
    assert lib.kvp_paged_free(c, None, None) == code
    assert decode(lib, c) == code
    assert lib.kvp_last_error() != b""
    assert lib.kvp_paged_decode_attn_workspace_size(c, 8, 2, 0) == 0
    assert lib.kvp_paged_append_workspace_size(c, 1) == 0


def test_null_cache(lib):
    assert lib.kvp_paged_init(None, None) == -1
    assert lib.kvp_paged_free(None, None, None) == -1


def test_append_refusals(lib):
    c = desc()

    def app(k=P, v=P, ks=None, vs=None, h_kv=2, n_new=1, counts=None, pos=None, ws=P, ws_bytes=1 << 40, c=c):
        st = [None if s is None else (ctypes.c_int64 * 3)(*s) for s in (ks, vs)]
        return lib.kvp_paged_append(c, k, v, st[0], st[1], h_kv, n_new, counts, pos, ws, ws_bytes, None)

    assert app(k=None) == -1 and app(v=None) == -1 and app(k=P + 2) == -1
    assert app(n_new=0) == -1 and app(n_new=641) == -1          # a row holds 640 slots
    assert app(h_kv=3) == -1 and app(h_kv=0) == -1
    assert app(ks=(1024, 4, 128), n_new=2) == -1 and app(vs=(1024, -128, 128), n_new=2) == -1
    assert app(pos=P) == -1                                      # the cache keeps no positions
    # a decode step's append may need no workspace, a prefill's does
    assert lib.kvp_paged_append_workspace_size(c, 640) > lib.kvp_paged_append_workspace_size(c, 1) >= 0
    assert app(n_new=640, ws=None) == -5 and app(n_new=640, ws_bytes=16) == -5 and app(n_new=640, ws=P + 16) == -1


def test_fork_and_compact_refusals(lib):
    c = desc()
    assert lib.kvp_paged_fork(c, None, 0, None, 0, None) == -1
    assert lib.kvp_paged_fork(c, P, 2, None, 0, None) == -1
    assert lib.kvp_paged_fork(c, P, 1, None, 0, None) == -5
    assert lib.kvp_paged_compact(c, None, P, 4, P, 1 << 40, None) == -1
    assert lib.kvp_paged_compact(c, P, None, 4, P, 1 << 40, None) == -1
    assert lib.kvp_paged_compact(c, P, P, 0, P, 1 << 40, None) == -1
    assert lib.kvp_paged_compact(c, P, P, 4, None, 0, None) == -5


def test_decode_refusals(lib):
    c = desc()
    assert decode(lib, c, q=None) == -1 and decode(lib, c, out=None) == -1 and decode(lib, c, q=P + 4) == -1
    assert decode(lib, c, h_q=7) == -1 and decode(lib, c, h_kv=3, h_q=6) == -1 and decode(lib, c, h_q=0) == -1
    assert decode(lib, c, h_q=34) == -2                          # 17 query heads on a KV head
    assert decode(lib, c, q_stride=512) == -1 and decode(lib, c, q_stride=1025) == -1
    assert decode(lib, c, out_dtype=2) == -2 and decode(lib, c, scale=float("nan")) == -1
    assert decode(lib, c, add=1) == -1 and decode(lib, c, add=2) == -1
    assert decode(lib, c, ws=None) == -5 and decode(lib, c, ws_bytes=64) == -5 and decode(lib, c, ws=P + 8) == -1


def test_workspaces_grow_with_the_work(lib):
    c = desc(score=P)
    plain, scored = (lib.kvp_paged_decode_attn_workspace_size(c, 8, 2, s) for s in (0, 1))
    assert plain > 0 and scored >= plain + 8 * 640 * 8 * 4       # a logit per slot and padded head
    assert lib.kvp_paged_fork_workspace_size(c, 0) == 0 and lib.kvp_paged_fork_workspace_size(c, 1) > 0
    assert lib.kvp_paged_append_workspace_size(c, 0) == 0
    assert lib.kvp_paged_decode_attn_workspace_size(c, 34, 2, 0) == 0


def test_more_rows_than_a_launch_counts_are_refused(lib):
    """A compaction launches up to 4 blocks a row (8 of few), an append sums up to n_new / 16 + 2 pages a row: both in 32 bits."""
    for n_rows in ((1 << 28) + 1, 1 << 29, 1 << 30, (1 << 31) - 1):
        test_a_bad_cache_is_refused_by_every_call(lib, dict(n_rows=n_rows, max_pages=1, page_size=16), -1)
    c = desc(n_rows=1 << 28, max_pages=1, page_size=16)
    assert lib.kvp_paged_compact_workspace_size(c, 16) >= 4 << 28


@pytest.mark.parametrize("scale", [1e300, -1e300, 3e38, float("inf")])
def test_a_scale_that_is_no_float_is_refused(lib, scale):
    """The kernels multiply by sm_scale * log2(e) in 32 bits; an infinite one would make every row NaN."""
    assert decode(lib, desc(), scale=scale) == -1
    assert b"sm_scale" in lib.kvp_last_error()


FAKE_RUNTIME = """
typedef struct { int on; int fits[4]; } state;
state fake;
int cudaGetDevice(int* d) { *d = fake.on; return 0; }
int cudaGetLastError(void) { return 0; }
int cudaFuncSetAttribute(const void* f, int a, int v) { return 0; }
int cudaOccupancyMaxActiveClusters(int* n, const void* f, const void* c) { *n = fake.fits[fake.on]; return 0; }
"""

FAKE_USE = """
import ctypes, sys
lib, fake = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2])
state = (ctypes.c_int * 5).in_dll(fake, "fake")
desc = ctypes.create_string_buffer(bytes.fromhex(sys.argv[3]))
lib.kvp_paged_append_workspace_size.restype = ctypes.c_size_t
state[1:] = [9, 0, 9, 0]
for device in (0, 1, 2, 3, 1, 0):
    state[0] = device
    print(device, lib.kvp_paged_append_workspace_size(desc, 1) == 0)
"""


def test_every_device_is_asked_for_its_clusters(lib, tmp_path):
    """A step's append runs in one cluster of 16 where the current device holds one, not where the first device asked did
    (the CUDA runtime's answers come from a stand-in)."""
    fake = tmp_path / "fake.so"
    (tmp_path / "fake.c").write_text(FAKE_RUNTIME)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(fake), str(tmp_path / "fake.c")], check=True)
    d = bytes(_Desc(**GOOD)).hex()
    out = subprocess.run([sys.executable, "-c", FAKE_USE, _lib.LIB_PATH, str(fake), d], check=True, capture_output=True, text=True,
                         env={**os.environ, "LD_PRELOAD": str(fake)}).stdout.split()
    assert out == "0 True 1 False 2 True 3 False 1 False 0 True".split()
