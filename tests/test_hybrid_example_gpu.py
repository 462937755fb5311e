"""The example program, with its own check: hidden states served through page steps, cache
writes, paged attention and SSD decode steps against a recomputation from scratch in fp64.
The two round the same values to bf16 (or 8 bits) in each layer, some of them to different
neighbours; the bound is the suite's for bf16 inputs with fp32 state."""
import os
import sys

import pytest

from helpers import TOL_BF16, report

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "f8"])
def test_hybrid_decode(cuda_device, cache):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import hybrid_decode
    worst = hybrid_decode.main(["--check", "--steps", "9", "--cache", cache])
    report("hybrid example " + cache, hidden=worst)
    assert 0.0 < worst <= TOL_BF16


def _example():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import hybrid_decode
    return hybrid_decode


class _Loop:
    """A server and what each of its requests was given and answered."""

    def __init__(self, device, batch, pages, cache):
        self.ex = _example()
        self.sv = self.ex.Server(batch, n_pages=pages, cache=cache)
        self.said, self.hidden = [[] for _ in range(batch)], [[] for _ in range(batch)]

    def step(self, new, end=()):
        """Offers each request its new tokens; returns which of them were refused."""
        import torch
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=self.sv.dev)  # noqa: E731
        hold = [0 if r in end else len(s) + len(n) for r, (s, n) in enumerate(zip(self.said, new))]
        x, m = self.sv.step(i32(hold), torch.tensor([t for n in new for t in n], device=self.sv.dev),
                            one_each=all(len(n) == 1 for n in new))
        held = self.sv.held.tolist()
        for r, part in enumerate(x.split([len(n) for n in new])):
            if r in end:
                self.said[r], self.hidden[r] = [], []
            elif held[r] == hold[r]:
                self.said[r], self.hidden[r] = self.said[r] + new[r], self.hidden[r] + [part]
        refused = [r for r in range(len(new)) if held[r] != hold[r]]
        assert len(refused) == int(m["denied"])
        return refused

    def states(self, r):
        return [s[r].clone() for s in self.sv.layers[::2]]

    def far(self, r):
        import torch
        got = torch.cat(self.hidden[r]).double()
        want = self.ex.recompute(self.sv.w, torch.tensor(self.said[r], device=self.sv.dev), self.sv.cache_scale if self.sv.f8 else None)
        return float((got - want).norm() / want.norm())


@pytest.mark.parametrize("cache", ["bf16", "f8"])
def test_a_refused_prompt_waits(cuda_device, cache):
    lp = _Loop(cuda_device, 2, 3, cache)
    a, b = list(range(30)), list(range(100, 120))          # 2 pages each, of 3
    assert lp.step([a, b]) == [1]
    assert all((s == 0).all() for s in lp.states(1))
    for t in (7, 8, 9):                                    # the last of these takes the third page
        assert lp.step([[t], b]) == [1]
    assert all((s == 0).all() for s in lp.states(1))
    far = lp.far(0)
    assert lp.step([[], b], end=[0]) == [1]                # pages given back are there in the next step
    assert lp.step([[], b], end=[0]) == []
    report("hybrid example, refused prompt " + cache, other=far, own=lp.far(1))
    assert 0.0 < max(far, lp.far(1)) <= TOL_BF16


@pytest.mark.parametrize("cache", ["bf16", "f8"])
def test_a_refused_token_waits(cuda_device, cache):
    lp = _Loop(cuda_device, 2, 3, cache)
    assert lp.step([list(range(16)), list(range(50, 80))]) == []        # 1 and 2 pages, of 3
    before = lp.states(0)
    for t in (5, 6):
        assert lp.step([[3], [t]]) == [0]                  # a step of one token each
        assert all((s == b).all() for s, b in zip(lp.states(0), before))
    far = lp.far(1)
    assert lp.step([[3], []], end=[1]) == [0]
    assert all((s == b).all() for s, b in zip(lp.states(0), before))
    assert lp.step([[3], [11]]) == []                      # and the other place has a new request of one token
    report("hybrid example, refused token " + cache, other=far, own=lp.far(0), new=lp.far(1))
    assert 0.0 < max(far, lp.far(0), lp.far(1)) <= TOL_BF16


def test_the_program_with_too_few_pages(cuda_device, capsys):
    worst = _example().main(["--check", "--steps", "9", "--pages", "7"])
    said = [line for line in capsys.readouterr().out.splitlines() if "refused" in line]
    assert any(not line.endswith("refused 0") for line in said) and 0.0 < worst <= TOL_BF16
