"""What the 16-bit cache's entry points refuse, on the host, before anything is launched."""

import ctypes

import pytest

import speculative_decoding_verification_72_gb300 as sv
from speculative_decoding_verification_72_gb300 import kv_q8 as Q
from speculative_decoding_verification_72_gb300 import paged as G

OK, INVALID, DTYPE, WORKSPACE = 0, 1, 2, 3
FAKE = 0x10000          # a stand-in for a device pointer; never dereferenced
I64x3 = ctypes.c_int64 * 3


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(sv.library_path()):
        from speculative_decoding_verification_72_gb300 import build
        build.build()
    return sv.load_library()


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, ks=(16 * 256, 256, 128), vs=(16 * 256, 256, 128), page_table=FAKE, num_pages=8, Hkv=2, page_size=16, D=128,
             max_pages=4)
    a.update(kw)
    return G._PagedStruct(a["k"], a["v"], I64x3(*a["ks"]), I64x3(*a["vs"]), a["page_table"], a["num_pages"], a["Hkv"], a["page_size"],
                          a["D"], a["max_pages"])


def rows(**kw):
    a = dict(data=FAKE, stride_b=1024, stride_n=256, stride_h=128)
    a.update(kw)
    return Q._RowsStruct(*a.values())


BAD_CACHES = [dict(k=None), dict(v=None), dict(page_table=None), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(num_pages=0), dict(Hkv=0),
              dict(page_size=8), dict(page_size=24), dict(page_size=256), dict(D=96), dict(D=256), dict(max_pages=0),
              dict(max_pages=1 << 28), dict(ks=(4096, 0, 128)), dict(ks=(4096, 252, 128)), dict(vs=(0, 256, 128)),
              dict(vs=(4096, 256, 64)), dict(ks=(-4096, 256, 128)), dict(vs=(1 << 40, 256, 128))]
BAD_ROWS = [dict(data=None), dict(data=FAKE + 4), dict(stride_n=132), dict(stride_h=1)]


def append(lib, c=None, k=None, v=None, q=None, **kw):
    a = dict(dtype=1, B=2, N=3, Hq=0, base=FAKE, par=None, nn=None, freq=FAKE, rot=128, inter=0, oq=None, out=FAKE, st=FAKE)
    a.update(kw)
    return lib.spec_kv_append_rope(c or cache(), a["dtype"], k or rows(), v or rows(), q, a["B"], a["N"], a["Hq"], a["base"], a["par"],
                                   a["nn"], a["freq"], a["rot"], a["inter"], a["oq"], a["out"], a["st"], None)


def test_append(lib):
    for bad in BAD_CACHES:
        assert append(lib, cache(**bad)) == INVALID, bad
    for bad in BAD_ROWS:
        assert append(lib, None, rows(**bad)) == INVALID and append(lib, None, None, rows(**bad)) == INVALID, bad
        assert append(lib, None, None, None, rows(**bad), Hq=4, oq=FAKE) == INVALID, bad
    assert append(lib, dtype=0) == DTYPE and append(lib, dtype=3) == DTYPE
    for bad in (dict(B=-1), dict(N=0), dict(base=None), dict(base=FAKE + 2), dict(out=None), dict(out=FAKE + 1), dict(st=FAKE + 1),
                dict(freq=None), dict(freq=FAKE + 2), dict(rot=0), dict(rot=8), dict(rot=20), dict(rot=144), dict(Hq=4), dict(Hq=-1),
                dict(par=FAKE, N=1025), dict(par=FAKE + 1), dict(nn=FAKE + 2), dict(nn=FAKE, out=FAKE), dict(base=FAKE, out=FAKE)):
        a = dict(out=FAKE + 64)
        a.update(bad)
        assert append(lib, **a) == INVALID, bad
    assert append(lib, q=rows(), Hq=0, oq=FAKE, out=FAKE + 64) == INVALID
    assert append(lib, q=rows(), Hq=4, oq=None, out=FAKE + 64) == INVALID
    assert append(lib, q=rows(), Hq=4, oq=FAKE + 8, out=FAKE + 64) == INVALID
    assert append(lib, q=rows(), Hq=16384, oq=FAKE, out=FAKE + 64) == INVALID
    assert append(lib, B=1 << 30, N=1 << 20, out=FAKE + 64) == INVALID
    assert append(lib, B=0) == OK


def attention(lib, c=None, q=None, **kw):
    a = dict(dtype=1, B=2, N=3, Hq=8, base=FAKE, par=None, nn=None, sm=0.1, cap=0.0, win=0, sl=None, out=FAKE, lse=FAKE, st=FAKE, ws=FAKE,
             wsb=1 << 40)
    a.update(kw)
    return lib.spec_attention(q or rows(), a["dtype"], c or cache(), a["B"], a["N"], a["Hq"], a["base"], a["par"], a["nn"], a["sm"],
                              a["cap"], a["win"], a["sl"], a["out"], a["lse"], a["st"], a["ws"], a["wsb"], None)


def test_attention(lib):
    for bad in BAD_CACHES:
        assert attention(lib, cache(**bad)) == INVALID, bad
    for bad in BAD_ROWS:
        assert attention(lib, None, rows(**bad)) == INVALID, bad
    assert attention(lib, dtype=0) == DTYPE and attention(lib, dtype=5) == DTYPE
    nan, inf = float("nan"), float("inf")
    for bad in (dict(B=-1), dict(N=0), dict(N=1025, par=FAKE), dict(Hq=7), dict(Hq=0), dict(base=None), dict(out=None),
                dict(out=FAKE + 8), dict(ws=None), dict(ws=FAKE + 8), dict(sm=nan), dict(sm=inf), dict(cap=-1.0), dict(cap=nan),
                dict(cap=inf), dict(cap=1e-38, sm=1e30), dict(win=-1), dict(par=FAKE + 2), dict(nn=FAKE + 1), dict(lse=FAKE + 2),
                dict(sl=FAKE + 2), dict(N=(1 << 24) + 1), dict(N=1 << 30), dict(B=1 << 28, N=1024)):
        assert attention(lib, **bad) == INVALID, bad
    assert attention(lib, cache(max_pages=(1 << 27) - 17), N=64) == INVALID      # positions and rows past 2^31 - 256
    assert attention(lib, cache(max_pages=1 << 22), B=1 << 14) == INVALID        # work past 2^31
    assert attention(lib, wsb=1024) == WORKSPACE
    assert attention(lib, B=0) == OK
    size = lib.spec_attention_workspace_size
    assert size(4, 6, 32, 8, 128) > 0 and size(4, 6, 32, 8, 128) % 256 == 0 and size(4, 5000, 32, 8, 64) > 0
    for bad in ((-1, 6, 32, 8, 128), (4, 0, 32, 8, 128), (4, 6, 33, 8, 128), (4, 6, 32, 8, 96), (4, 6, 4, 8, 64), (4, 1 << 30, 8, 8, 64)):
        assert size(*bad) == 0


def test_new_caches():
    import torch
    for bad in (dict(page_size=20), dict(head_dim=96), dict(pages=0), dict(kv_heads=0), dict(dtype=torch.float32)):
        with pytest.raises(sv.SpecVerifyError):
            sv.paged_cache(**{**dict(pages=2, kv_heads=1, page_size=16, head_dim=64, device="cpu"), **bad})
