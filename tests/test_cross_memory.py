"""Dense attention whose arguments share memory: refused on the host before any launch (CPU only). The addresses are
never used; every call here has to be refused."""
import ctypes

import pytest

from block_sparse_spherical_b200 import abi, build
from test_cross import cross_cfg, prefix_cfg


@pytest.fixture(scope="module")
def lib():
    build.build()
    return abi.load()


M = 1 << 27          # from one tensor's stand-in address to the next's


def meeting(call, names, written, sizes):
    """call(addresses) has to refuse (1) each written tensor moved onto the first and onto the last bytes of every other."""
    base = {x: (i + 1) * M for i, x in enumerate(names)}
    for w in written:
        for other in names:
            if other == w:
                continue
            tail = -(-sizes[other] // 256) * 256 - 256                 # keeps every alignment
            for at in (base[other] + tail, base[other] - (-(-sizes[w] // 256) * 256 - 256)):
                assert at % 256 == 0
                if at + sizes[w] > base[other] and at < base[other] + sizes[other]:
                    assert call({**base, w: at}) == 1, (w, other)


def test_cross_memory_that_meets_is_refused(lib):
    cfg = cross_cfg(batch=1, n_k=100000, n_q=33)
    c, n = ctypes.byref(cfg), ctypes.c_size_t(0)
    assert lib.bsa_cross_workspace_size(c, ctypes.byref(n)) == 0
    need, rows, keys = n.value, 8 * 33 * 64 * 2, 4 * 100000 * 64 * 2
    sizes = dict(q=rows, k=keys, v=keys, key_len=4, out=rows, lse=8 * 33 * 4, low=rows, ws=need, status=4)
    call = lambda a: lib.bsa_cross_attention(c, a["q"], a["k"], a["v"], a["key_len"], a["out"], a["lse"], a["low"],
                                             a["ws"], need, a["status"], None)
    meeting(call, list(sizes), ["out", "lse", "low", "ws"], sizes)
    assert lib.bsa_cross_backward_workspace_size(c, ctypes.byref(n)) == 0
    need = n.value
    sizes = dict(q=rows, k=keys, v=keys, key_len=4, out=rows, lse=8 * 33 * 4, low=rows, dout=rows, dq=rows, dk=keys,
                 dv=keys, ws=need, status=4)
    call = lambda a: lib.bsa_cross_attention_backward(
        c, a["q"], a["k"], a["v"], a["key_len"], a["out"], a["lse"], a["low"], a["dout"], a["dq"], a["dk"], a["dv"],
        a["ws"], need, a["status"], None)
    meeting(call, list(sizes), ["dq", "dk", "dv", "ws"], sizes)


def test_prefix_memory_that_meets_is_refused(lib):
    cfg = prefix_cfg(n_prefix=50000)
    c, n = ctypes.byref(cfg), ctypes.c_size_t(0)
    assert lib.bsa_prefix_workspace_size(c, ctypes.byref(n)) == 0
    need, rows = n.value, 6 * 8 * 3 * 64 * 2
    shared, own = 2 * 4 * 50000 * 64 * 2, 6 * 4 * 40 * 64 * 2
    sizes = dict(q=rows, kp=shared, vp=shared, pl=8, ko=own, vo=own, ol=24, out=rows, ws=need, status=4)
    call = lambda a: lib.bsa_prefix_attention(c, a["q"], a["kp"], a["vp"], a["pl"], a["ko"], a["vo"], a["ol"], a["out"],
                                              a["ws"], need, a["status"], None)
    meeting(call, list(sizes), ["out", "ws"], sizes)
