"""What shared-prefix decode refuses before anything is launched (no GPU needed: no pointer is followed)."""
import math

import pytest

from tests.test_paged_host import P, desc, lib  # noqa: F401


def prefix(lib, c, q=P, q_stride=0, lead=P, h_q=8, h_kv=2, scale=0.1, out=P, lse=None, ws=P, ws_bytes=1 << 40):
    return lib.kvp_paged_prefix_decode_attn(q, q_stride, c, lead, h_q, h_kv, scale, out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), -1), (dict(out=None), -1), (dict(lead=None), -1), (dict(q=4104), -1), (dict(out=4104), -1), (dict(h_q=0), -1),
    (dict(h_kv=0), -1), (dict(h_q=7), -1), (dict(h_kv=3, h_q=9), -1), (dict(h_q=34), -2), (dict(q_stride=4), -1),
    (dict(q_stride=1028), -1), (dict(q_stride=1 << 40), -1), (dict(scale=math.nan), -1), (dict(scale=math.inf), -1),
    (dict(scale=3e38), -1), (dict(ws=None), -5), (dict(ws_bytes=100), -5), (dict(ws=P + 16), -1),
])
def test_refusals(lib, change, code):  # noqa: F811
    assert prefix(lib, desc(), **change) == code
    assert lib.kvp_last_error() != b""


def test_caches(lib):  # noqa: F811
    assert prefix(lib, desc(page_size=48)) == -2 and prefix(lib, None) == -1
    assert prefix(lib, desc(n_rows=2 * 16385)) == -2
    size = lib.kvp_paged_prefix_decode_attn_workspace_size
    assert size(desc(), 8, 2) > 0 and size(desc(n_rows=2 * 16384), 8, 2) > size(desc(), 8, 2)
    assert size(desc(n_rows=2 * 16385), 8, 2) == 0 and size(desc(), 7, 2) == 0 and size(desc(), 34, 2) == 0
    assert size(desc(dtype=9), 8, 2) == 0
