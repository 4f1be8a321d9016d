"""What the cache's and the log-probs' entry points refuse, on the host, before anything is launched."""

import ctypes

import pytest
import torch

import speculative_decoding_verification_72_gb300 as sv
from speculative_decoding_verification_72_gb300 import kv_q8 as Q

OK, INVALID, DTYPE, WORKSPACE = 0, 1, 2, 3
FAKE = 0x10000          # a stand-in for a device pointer; never dereferenced


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(sv.library_path()):
        from speculative_decoding_verification_72_gb300 import build
        build.build()
    return sv.load_library()


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, page_table=FAKE, num_pages=8, Hkv=2, page_size=16, D=128, max_pages=4)
    a.update(kw)
    return Q._CacheStruct(*a.values())


def rows(**kw):
    a = dict(data=FAKE, stride_b=1024, stride_n=256, stride_h=128)
    a.update(kw)
    return Q._RowsStruct(*a.values())


BAD_CACHES = [dict(k=None), dict(v_scale=None), dict(page_table=None), dict(k=FAKE + 8), dict(num_pages=0), dict(Hkv=0),
              dict(page_size=8), dict(page_size=24), dict(page_size=256), dict(D=96), dict(D=256), dict(max_pages=0),
              dict(max_pages=1 << 28)]
BAD_ROWS = [dict(data=None), dict(data=FAKE + 4), dict(stride_n=132), dict(stride_h=1)]


def append(lib, c=None, k=None, v=None, **kw):
    a = dict(dtype=1, B=2, N=3, base=FAKE, path=None, cols=0, n=None, out=FAKE, st=FAKE)
    a.update(kw)
    return lib.spec_kv_append_q8(c or cache(), k or rows(), v or rows(), a["dtype"], a["B"], a["N"], a["base"], a["path"],
                                 a["cols"], a["n"], a["out"], a["st"], None)


def test_append(lib):
    for bad in BAD_CACHES:
        assert append(lib, cache(**bad)) == INVALID, bad
    for bad in BAD_ROWS:
        assert append(lib, None, rows(**bad)) == INVALID and append(lib, None, None, rows(**bad)) == INVALID, bad
    assert append(lib, dtype=3) == DTYPE
    for bad in (dict(B=-1), dict(N=0), dict(base=None), dict(base=FAKE + 2), dict(out=None), dict(st=FAKE + 1),
                dict(path=FAKE, cols=0, n=FAKE), dict(path=FAKE, cols=3), dict(B=1 << 30, N=1 << 20)):
        assert append(lib, **bad) == INVALID, bad
    assert append(lib, B=0) == OK


def attention(lib, c=None, q=None, **kw):
    a = dict(dtype=1, B=2, N=3, Hq=8, base=FAKE, par=None, nn=None, sm=0.1, out=FAKE, lse=FAKE, st=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return lib.spec_attention_q8(q or rows(), a["dtype"], c or cache(), a["B"], a["N"], a["Hq"], a["base"], a["par"], a["nn"],
                                 a["sm"], a["out"], a["lse"], a["st"], a["ws"], a["wsb"], None)


def test_attention(lib):
    for bad in BAD_CACHES:
        assert attention(lib, cache(**bad)) == INVALID, bad
    for bad in BAD_ROWS:
        assert attention(lib, None, rows(**bad)) == INVALID, bad
    assert attention(lib, dtype=0) == DTYPE and attention(lib, dtype=5) == DTYPE
    for bad in (dict(B=-1), dict(N=0), dict(N=1025), dict(Hq=7), dict(Hq=0), dict(base=None), dict(out=None), dict(out=FAKE + 8),
                dict(ws=None), dict(ws=FAKE + 8), dict(sm=float("nan")), dict(sm=float("inf")), dict(par=FAKE + 2),
                dict(nn=FAKE + 1), dict(lse=FAKE + 2)):
        assert attention(lib, **bad) == INVALID, bad
    assert attention(lib, wsb=1024) == WORKSPACE
    assert attention(lib, B=0) == OK
    size = lib.spec_attention_q8_workspace_size
    assert size(4, 6, 32, 8, 128) > 0 and size(4, 6, 32, 8, 128) % 256 == 0
    for bad in ((-1, 6, 32, 8, 128), (4, 0, 32, 8, 128), (4, 1025, 32, 8, 128), (4, 6, 33, 8, 128), (4, 6, 32, 8, 96)):
        assert size(*bad) == 0


def weights(lib, c=None, q=None, **kw):
    a = dict(dtype=1, lse=FAKE, B=2, N=3, Hq=8, base=FAKE, path=None, cols=0, n=None, sm=0.1, decay=1.0, s=FAKE, out=FAKE, S=64,
             st=FAKE)
    a.update(kw)
    return lib.spec_attention_weights_q8(q or rows(), a["dtype"], a["lse"], c or cache(), a["B"], a["N"], a["Hq"], a["base"],
                                         a["path"], a["cols"], a["n"], a["sm"], a["decay"], a["s"], a["out"], a["S"], a["st"],
                                         None)


def test_weights(lib):
    for bad in BAD_CACHES:
        assert weights(lib, cache(**bad)) == INVALID, bad
    assert weights(lib, dtype=0) == DTYPE
    for bad in (dict(B=-1), dict(N=0), dict(Hq=5), dict(lse=None), dict(s=None), dict(out=None), dict(S=0),
                dict(decay=float("nan")), dict(path=FAKE, cols=3), dict(path=FAKE, n=FAKE), dict(out=FAKE + 2)):
        assert weights(lib, **bad) == INVALID, bad
    assert weights(lib, B=0) == OK


def evict(lib, c=None, **kw):
    a = dict(B=2, n=FAKE, s=FAKE, p=FAKE, S=64, keep=32, sinks=0, pf=None, os=FAKE, op=FAKE, out=FAKE, st=FAKE, ws=FAKE,
             wsb=1 << 30)
    a.update(kw)
    return lib.spec_kv_evict_q8(c or cache(), a["B"], a["n"], a["s"], a["p"], a["S"], a["keep"], a["sinks"], a["pf"], a["os"],
                                a["op"], a["out"], a["st"], a["ws"], a["wsb"], None)


def test_evict(lib):
    for bad in BAD_CACHES:
        assert evict(lib, cache(**bad)) == INVALID, bad
    for bad in (dict(B=-1), dict(S=0), dict(keep=0), dict(keep=17), dict(keep=80), dict(keep=80, S=100), dict(n=None),
                dict(s=None), dict(p=None), dict(os=None), dict(op=None), dict(out=None), dict(ws=None), dict(pf=FAKE + 1)):
        assert evict(lib, **bad) == INVALID, bad
    assert evict(lib, wsb=64) == WORKSPACE
    assert evict(lib, B=0) == OK


def logprobs(lib, **kw):
    a = dict(x=FAKE, dtype=1, stride=100, tok=FAKE, rows=4, V=100, T=1.0, n=5, lp=FAKE, ent=FAKE, lse=FAKE, saved=FAKE, tt=FAKE,
             tl=FAKE, st=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return lib.spec_token_logprobs(*a.values(), None)


def test_logprobs(lib):
    assert logprobs(lib, dtype=2) == DTYPE and logprobs(lib, dtype=9) == DTYPE
    for bad in (dict(x=None), dict(x=FAKE + 1), dict(stride=99), dict(tok=None), dict(rows=-1), dict(V=0), dict(T=0.0),
                dict(T=float("inf")), dict(n=-1), dict(n=33), dict(lp=None), dict(tt=None), dict(tl=None), dict(saved=FAKE + 8),
                dict(ws=None), dict(ws=FAKE + 4)):
        assert logprobs(lib, **bad) == INVALID, bad
    assert logprobs(lib, wsb=16) == WORKSPACE
    assert logprobs(lib, rows=0) == OK
    size = lib.spec_token_logprobs_workspace_size
    assert size(4, 100, 1, 5) > 0 and size(4, 0, 1, 5) == 0 and size(4, 100, 2, 5) == 0 and size(4, 100, 1, 33) == 0


def backward(lib, **kw):
    a = dict(x=FAKE, dtype=1, stride=100, tok=FAKE, saved=FAKE, g=FAKE, h=None, rows=4, V=100, T=1.0, d=2 * FAKE, ds=100)
    a.update(kw)
    return lib.spec_token_logprobs_backward(*a.values(), None)


def test_backward(lib):
    assert backward(lib, dtype=2) == DTYPE
    for bad in (dict(x=None), dict(stride=99), dict(ds=99), dict(tok=None), dict(saved=None), dict(saved=FAKE + 4), dict(g=None),
                dict(d=None), dict(d=FAKE, ds=101), dict(T=float("nan")), dict(rows=-1), dict(d=FAKE + 1)):
        assert backward(lib, **bad) == INVALID, bad
    assert backward(lib, rows=0) == OK


def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    z = torch.zeros((2, 1, 16, 64), dtype=torch.float8_e4m3fn)
    c = sv.Q8Cache(z, z, torch.ones((2, 1)), torch.ones((2, 1)))
    q, t, b = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16), torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_attention_q8(q, c, t, b)
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_kv_append_q8(c, q, q, t, b)
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_token_logprobs(torch.zeros((1, 1, 8)), torch.zeros((1, 1), dtype=torch.int32))
    with pytest.raises(sv.SpecVerifyError):
        sv.q8_cache(4, 2, 24, 64)


def test_rows_whose_node_is_not_exact(lib):
    """A row's node is a product with 2^32 / G rounded up, which is exact for few enough rows: 131071 heads on one kv head
    were taken, and the last row of node 0 went to node 1."""
    g = 131071
    assert (g - 1) * -(-(1 << 32) // g) >> 32 == 1
    one = cache(Hkv=1)
    for n, heads in ((8, g), (1, g), (8, 30011), (1, 1 << 21)):
        assert attention(lib, one, N=n, Hq=heads) == INVALID, (n, heads)
        assert weights(lib, one, N=n, Hq=heads) == INVALID, (n, heads)


def test_positions_whose_tiles_end_past_32_bits(lib):
    """A length of 2^31 - 100 is 2^24 tiles of 128, the last of which ends past 2^31: counted in 32 bits it came out as one."""
    for page, most in ((16, (1 << 31) // 16 - 16), (128, (1 << 31) // 128 - 2)):
        for pages in (most + 1, (1 << 31) // page - 1):
            c = cache(page_size=page, max_pages=pages, Hkv=1)
            assert append(lib, c) == attention(lib, c) == weights(lib, c) == evict(lib, c) == INVALID, (page, pages)


def test_lengths_in_place(lib):
    """out_len is written by a request's first CTA while others may still have to read the length."""
    other = 2 * FAKE
    assert append(lib, base=FAKE, out=FAKE) == append(lib, base=other, path=FAKE, cols=3, n=FAKE, out=FAKE) == INVALID
    assert evict(lib, n=FAKE, out=FAKE) == evict(lib, n=other, pf=FAKE, out=FAKE) == INVALID
