"""The example that decodes on the 8-bit cache: drafts change how many passes it takes, not what comes out."""

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_drafts_do_not_change_what_is_decoded():
    import q8_verify_step as E
    model = E.Model()
    prompt = torch.randint(0, model.vocab, (3, 90), generator=torch.Generator().manual_seed(5), dtype=torch.int32).cuda()
    steps = [[], []]
    plain, lp0, _ = E.decode(model, prompt, 24, report=lambda d, c, lp: steps[0].append(lp))
    spec, lp1, d = E.decode(model, prompt, 24, guesses=plain.int(), report=lambda d, c, lp: steps[1].append(lp))
    assert len(steps[1]) < len(steps[0])
    assert d.seen.tolist() == d.length.tolist()
    for b in range(3):
        # Rows of a page are kept under the largest scale it ever had and sums run in another order, so a
        # near tie may fall the other way; nothing else may.
        miss = (plain[b] != spec[b]).nonzero()
        if len(miss):
            i = int(miss[0])
            assert abs(float(lp0[b, i] - lp1[b, i])) < 0.25
            n = i
        else:
            n = 24
        assert n >= 8
        assert (lp0[b, :n] - lp1[b, :n]).abs().max() < 0.5


def test_a_budget_bounds_the_cache():
    import q8_verify_step as E
    model = E.Model()
    prompt = torch.randint(0, model.vocab, (3, 90), generator=torch.Generator().manual_seed(6), dtype=torch.int32).cuda()
    longest = []

    def report(d, count, lp):
        longest.append(int(d.length.max()))
        assert int(lp["status"].max()) == 0
        for b in range(3):
            n = int(d.length[b])
            for h in range(model.kv_heads):
                pos = d.positions[b, h, :n]
                assert (pos >= 0).all() and len(pos.unique()) == n
                assert set(range(4)) <= set(pos.tolist())                     # sinks stay
                assert set(range(int(d.seen[b]) - 8, int(d.seen[b]))) <= set(pos.tolist())
            assert (d.positions[b, :, n:] == -1).all()

    E.decode(model, prompt, 20, budget=96, report=report)
    assert max(longest) <= 96


def test_requests_that_accept_unequally():
    """One request's drafts are all right, the other's none: the first runs far ahead and stays within its pages."""
    import q8_verify_step as E
    model = E.Model()
    prompt = torch.randint(0, model.vocab, (2, 30), generator=torch.Generator().manual_seed(7), dtype=torch.int32).cuda()
    plain, _, _ = E.decode(model, prompt, 280)
    guesses = plain.int()
    guesses[1] = -1
    tokens, _, d = E.decode(model, prompt, 70, guesses=guesses)
    assert int(d.seen[0]) > 30 + 2 * 70 + 72
    assert d.seen.tolist() == d.length.tolist() and tokens.shape == (2, 70)
