"""ssm_kv_pages_step on the GPU against the oracle's lists: whole numbers, so every
output has to be equal."""
import numpy as np
import pytest

from helpers import lib
from oracle import paged

pytestmark = pytest.mark.gpu


def _step(device, held, hold, table, place, ring, ps, n_tokens):
    import torch
    i32 = lambda a: torch.tensor(np.ascontiguousarray(a), dtype=torch.int32, device=device)  # noqa: E731
    t, f = i32(table), i32(place)
    got = lib().ssm_kv_pages_step(i32(held), i32(hold), t, f, i32(ring), page_size=ps, n_tokens=n_tokens)
    torch.cuda.synchronize()
    got = dict(got, block_table=t, free_ring=f)
    return {k: v.cpu().numpy().astype(np.int64) for k, v in got.items()}


def _same(got, want):
    assert set(got) == set(want)
    for k in want:
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)


def _start(rng, batch, cols, ps, top, free, head):
    """Requests of 0..top tokens, their pages, and `free` more pages in a ring from `head`."""
    held = rng.integers(0, top + 1, batch)
    have = -(-held // ps)
    total = int(have.sum()) + free
    order = rng.permutation(total)
    table = np.full((batch, cols), -1)
    table[np.arange(cols)[None] < have[:, None]] = order[:have.sum()]
    place = np.full(total, -1)
    place[(head + np.arange(free)) % total] = order[have.sum():]
    return held, table, place, [head % total, free]


CASES = [  # batch, page, cols, longest, growth, free pages, tokens asked for beyond the new ones
    (1, 16, 4, 0, 1, 1, 0),
    (1, 1, 3, 2, 1, 5, 3),
    (5, 16, 8, 100, 1, 9, 2),
    (64, 24, 10, 200, 40, 60, 1),
    (513, 8, 12, 70, 20, 500, 7),       # more requests than a block has threads
    (300, 16, 40, 300, 300, 900, -500),  # fewer pages than needed; the maps cut short
    (200, 256, 3, 600, 500, 10000, 0),  # requests over the table's row
    (4096, 64, 2, 128, 1, 4096, 5),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "b%d-p%d-c%d" % c[:3])
def test_pages_against_lists(cuda_device, case):
    batch, ps, cols, top, grow, free, extra = case
    rng = np.random.default_rng(batch + ps)
    held, table, place, ring = _start(rng, batch, cols, ps, top, free, int(rng.integers(1 << 20)))
    hold = held + rng.integers(0, grow + 1, batch)
    hold[rng.random(batch) < 0.15] = 0
    hold[rng.random(batch) < 0.1] -= 1          # shrink by one (or to -1, which counts as 0)
    n_tokens = max(0, int(np.maximum(hold - held, 0).sum()) + extra)
    _same(_step(cuda_device, held, hold, table, place, ring, ps, n_tokens),
          paged.pages_step(held, hold, table, place, ring, ps, n_tokens))


def test_pages_no_tokens_and_nothing_to_do(cuda_device):
    held, table, place, ring = [16, 0], np.array([[1], [-1]]), np.array([0, 2]), [0, 2]
    _same(_step(cuda_device, held, held, table, place, ring, 16, 0), paged.pages_step(held, held, table, place, ring, 16, 0))


def test_pages_a_strided_table(cuda_device):
    import torch
    big = torch.full((3, 9), -7, dtype=torch.int32, device=cuda_device)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=cuda_device)  # noqa: E731
    got = lib().ssm_kv_pages_step(i32([0, 0, 0]), i32([3, 5, 1]), big[:, 2:6], i32([4, 5, 6, 7]), i32([1, 4]),
                                  page_size=4, n_tokens=9)
    assert big[:, 2:6].cpu().tolist() == [[5, -7, -7, -7], [6, 7, -7, -7], [4, -7, -7, -7]]
    assert (big[:, :2] == -7).all() and (big[:, 6:] == -7).all()
    assert got["slots"].cpu().tolist() == [20, 21, 22, 24, 25, 26, 27, 28, 16]


def test_pages_many_steps_as_a_program_runs_them(cuda_device):
    """len and ring of one step go into the next, without a copy to the host between."""
    import torch
    rng = np.random.default_rng(11)
    batch, ps, cols = 9, 4, 6
    held, table, place, ring = _start(rng, batch, cols, ps, 10, 20, 13)
    i32 = lambda a: torch.tensor(np.ascontiguousarray(a), dtype=torch.int32, device=cuda_device)  # noqa: E731
    g_held, g_table, g_place, g_ring = i32(held), i32(table), i32(place), i32(ring)
    m = lib()
    for step in range(20):
        more = rng.integers(0, 3, batch)
        done = rng.random(batch) < 0.15
        want = paged.pages_step(held, np.where(done, 0, held + more), table, place, ring, ps, 30)
        hold = torch.where(torch.tensor(done, device=cuda_device), 0, g_held + i32(more)).to(torch.int32)
        got = m.ssm_kv_pages_step(g_held, hold, g_table, g_place, g_ring, page_size=ps, n_tokens=30)
        g_held, g_ring = got["len"], got["ring"]
        _same({k: v.cpu().numpy().astype(np.int64) for k, v in dict(got, block_table=g_table, free_ring=g_place).items()}, want)
        held, table, place, ring = want["len"], want["block_table"], want["free_ring"], want["ring"]


def test_what_goes_on_to_the_next_step_holds_little_memory(cuda_device):
    """len, ring, starts and denied of a step with a million new tokens (16 MB of maps) share their memory with
    each other at most, and with no more than 4 MiB of maps where those are smaller."""
    import torch
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=cuda_device)  # noqa: E731
    for n in (1 << 20, 1 << 12):
        pages = n // 256 + 2
        got = lib().ssm_kv_pages_step(i32([0, 3]), i32([n, 4]), torch.zeros((2, pages), dtype=torch.int32, device=cuda_device),
                                      torch.arange(pages, dtype=torch.int32, device=cuda_device), i32([0, pages]), page_size=256, n_tokens=n + 1)
        assert got["len"].tolist() == [n, 4] and got["starts"].tolist() == [0, n, n + 1] and got["denied"].tolist() == [0]
        assert got["positions"][[0, n - 1, n]].tolist() == [0, n - 1, 3] and got["request"][[0, n]].tolist() == [0, 1]
        for k in ("len", "ring", "starts", "denied"):
            assert got[k].untyped_storage().nbytes() <= (4096 if n == 1 << 20 else (4 << 20) + 4096), (n, k)
