"""Failure detection of the 8-bit cache's kernels on the GPU, without a GPU fault.

A planted fault (ds_plant_wait_fault) skips one arrival of the first CTA, so that the
waits behind it run out after a short limit.  The kernel records DS_ERR_TIMEOUT, lets what
is in flight land and returns within a few limits; the next call is whole again.
"""

import time

import pytest
import torch

import sparse_attention_top_ds_b200 as ds

pytestmark = pytest.mark.gpu

LIMIT_NS = 1_000_000  # 1 ms


@pytest.fixture
def short_waits(cuda_device):
    ds.ds_set_wait_limit(LIMIT_NS)
    ds.ds_get_device_status()
    yield
    ds.ds_plant_wait_fault(0)
    ds.ds_set_wait_limit(0)
    ds.ds_get_device_status()


def planted(call):
    """Run a call with a planted fault; its waits must run out, once each at most."""
    torch.cuda.synchronize()
    ds.ds_plant_wait_fault(1)
    t0 = time.perf_counter()
    r = call()
    status = ds.ds_get_device_status()
    elapsed = time.perf_counter() - t0
    assert status == ds.DS_ERR_TIMEOUT, ds.strerror(status)
    assert elapsed < 0.1, f"the planted call took {elapsed:.3f} s"
    return r


@pytest.mark.parametrize("budget,width", [(2, 512), (5, 1024), (600, 512)])
def test_move_by_copies_gives_up_and_recovers(short_waits, budget, width):
    # (2 and 5 entries: a piece or two to a CTA; 600: more pieces than a CTA has stages)
    B, block, nb = 2, 64, max(8, budget + 5)
    g = torch.Generator("cuda").manual_seed(budget)
    src = torch.randint(1, 256, (B, nb * block, width), device="cuda", dtype=torch.uint8, generator=g)
    small = torch.randint(1, 2 ** 31 - 1, (B, nb * block), device="cuda", dtype=torch.int32, generator=g)
    kept = torch.stack([torch.randperm(nb, device="cuda", generator=g)[:budget].sort().values for _ in range(B)]).int()
    at = (kept.long()[:, :, None] * block + torch.arange(block, device="cuda")).view(B, -1)
    want = src[torch.arange(B, device="cuda")[:, None], at]

    def move():
        dst, to = torch.zeros_like(want), torch.zeros(B, budget * block, dtype=torch.int32, device="cuda")
        ds.ds_cache_compact(kept, block=block, rows=[(src, dst), (small, to)])
        return dst, to

    dst, to = planted(move)
    lost = dst != want
    assert lost.any() and not dst[lost].any(), "what was not moved must be as it was"
    assert torch.equal(to, small[torch.arange(B, device="cuda")[:, None], at])
    dst, to = move()
    assert ds.ds_get_device_status() == ds.DS_OK and torch.equal(dst, want)
