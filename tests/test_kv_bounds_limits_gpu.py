"""ssm_kv_page_bounds_update at the limit of its count of pages."""
import pytest

from helpers import lib

pytestmark = pytest.mark.gpu


def test_as_many_pages_as_are_counted(cuda_device):
    """Two requests of 2^30 - 1 pages of one token each, 2^31 - 2 in all, none of them in the cache but the first and the
    last: those two get their bounds."""
    import torch
    n = (1 << 30) - 1
    k = torch.randn((3, 1, 1, 16), device=cuda_device).to(torch.bfloat16)
    bounds = torch.full((3, 1, 2, 16), 7.0, device=cuda_device, dtype=torch.bfloat16)
    table = torch.full((2, n), -1, dtype=torch.int32, device=cuda_device)
    table[0, 0], table[1, n - 1] = 0, 2
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=cuda_device)  # noqa: E731
    lib().ssm_kv_page_bounds_update(k, bounds, table, i32(0, 0), i32(n, n))
    torch.cuda.synchronize()
    for p in (0, 2):
        assert torch.equal(bounds[p, 0, 0], k[p, 0, 0]) and torch.equal(bounds[p, 0, 1], k[p, 0, 0])
    assert (bounds[1] == 7.0).all()
