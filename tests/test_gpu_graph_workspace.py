"""Calls captured in a CUDA graph without a workspace: their replays write to no memory but the graph's and the outputs."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_72_gb300 as sv
from q8_utils import DEV, host_cache, i32, rows, table, to_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    sv.load_library()


def attention(large):
    rng = np.random.default_rng(1)
    base, N, G = [300, 40], (40 if large else 2), 4
    t = table(rng, [b + N for b in base], 16, 64)
    c = to_gpu(host_cache(rng, 64, 2, 16, 64))
    q, _ = rows(rng, (2, N, 2 * G, 64), BF)
    t, base = i32(t), i32(base)
    lib = sv.load_library()
    return (lambda: sv.spec_attention_q8(q, c, t, base)), lib.spec_attention_q8_workspace_size(2, N, 2 * G, 2, 64)


def evict(large):
    rng = np.random.default_rng(2)
    B, P, keep, n = (40 if large else 2), 16, (1024 if large else 256), (1040 if large else 300)
    S = -(-n // P) * P
    c = sv.q8_cache(B * S // P, 2, P, 64)
    t, lens = i32(np.arange(B * S // P).reshape(B, -1)), i32([n] * B)
    s = torch.rand((B, 2, S), generator=torch.Generator().manual_seed(1)).to(DEV)
    pos = torch.arange(S, dtype=torch.int32, device=DEV).expand(B, 2, S).contiguous()
    lib = sv.load_library()
    return (lambda: sv.spec_kv_evict_q8(c, t, lens, s, pos, keep)), lib.spec_kv_evict_q8_workspace_size(B, 2, keep)


def logprobs(large):
    R, V = (64, 60000) if large else (2, 9000)
    x = torch.randn((2, R, V), generator=torch.Generator().manual_seed(2)).to(BF).to(DEV)
    tok = torch.zeros((2, R), dtype=torch.int32, device=DEV)
    lib = sv.load_library()
    return (lambda: sv.spec_token_logprobs(x, tok, n_top=8)), lib.spec_token_logprobs_workspace_size(2 * R, V, 1, 8)


def greedy(large):
    B, K, V = (64, 5, 60000) if large else (2, 5, 9000)
    x = torch.randn((B, K + 1, V), generator=torch.Generator().manual_seed(3)).to(BF).to(DEV)
    d = x[:, :K].argmax(-1).int()
    d[0, 2] = 0
    lib = sv.load_library()
    return (lambda: sv.spec_verify_greedy(x, d)), lib.spec_verify_greedy_workspace_size(B, K, V, 1)


def tree_build(large):
    B, V = (16, 60000) if large else (2, 9000)
    x = torch.randn((B, 9, V), generator=torch.Generator().manual_seed(4)).to(BF).to(DEV)
    lib = sv.load_library()
    return (lambda: sv.spec_tree_build(x, 3, 4, 16)), lib.spec_tree_build_workspace_size(B, 3, 4, V)


CALLS = [attention, evict, logprobs, greedy, tree_build]


@pytest.mark.parametrize("warm", [True, False])
@pytest.mark.parametrize("make", CALLS)
def test_replays_keep_to_the_graphs_memory(make, warm):
    small, need = make(False)
    large, need_large = make(True)
    assert need_large > need
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        want = {k: v.clone() for k, v in small().items()} if warm else None
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            out = small()
        large_want = {k: v.clone() for k, v in large().items()}     # a kept workspace is replaced by a larger one here
        others = [torch.full((need,), 0x5a, dtype=torch.uint8, device=DEV) for _ in range(16)]   # and its memory taken
        for _ in range(3):
            g.replay()
        got = large()
        stream.synchronize()
        assert all(bool((t == 0x5a).all()) for t in others)
        assert all(torch.equal(got[k], v) for k, v in large_want.items())
        if want is None:
            want = small()
        assert all(torch.equal(out[k], v) for k, v in want.items())
