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


def cache(g, fmt, *shape):
    return torch.randint(-100, 101, shape, device="cuda", dtype=torch.int8, generator=g) if fmt == "int8" else \
        torch.randn(*shape, device="cuda", generator=g).to(torch.float8_e4m3fn)


@pytest.mark.parametrize("B,H,K,d,k,W,fmt", [
    (1, 16, 1, 64, 10, 0, "int8"),          # one CTA, one chunk
    (8, 128, 1, 512, 1024, 128, "e4m3"),    # clusters that share a tile, several chunks to a CTA
    (2, 40, 8, 192, 333, 77, "int8"),
    (160, 128, 1, 512, 2048, 64, "e4m3"),   # one CTA to a tile, all chunks
    (200, 64, 1, 320, 50, 9, "int8"),
    (1, 64, 1, 128, 0, 700, "e4m3"),
], ids=str)
def test_attention_gives_up_and_recovers(short_waits, B, H, K, d, k, W, fmt):
    T = 2500
    g = torch.Generator("cuda").manual_seed(B + d)
    q = torch.randn(B, H, d, device="cuda", generator=g).bfloat16()
    codes, scales = cache(g, fmt, T, K, d), torch.full((-(-T // 16), K), 0.01, device="cuda")
    idx = torch.rand(B, T, device="cuda", generator=g).topk(k, dim=1).indices.int() if k else None
    win = torch.randn(B, W, K, d, device="cuda", generator=g).bfloat16() if W else None

    def attend():
        return ds.ds_sparse_attention_q8(q, codes, scales, idx, 16, win=win, return_lse=True)

    out, lse = attend()
    assert ds.ds_get_device_status() == ds.DS_OK
    planted(attend)
    for _ in range(2):
        o2, l2 = attend()
        assert ds.ds_get_device_status() == ds.DS_OK and torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("B,H,K,d,k,fmt", [
    (1, 16, 1, 64, 10, "int8"),
    (8, 128, 1, 512, 1024, "e4m3"),
    (2, 48, 12, 64, 200, "bf16"),           # several tiles to a CTA, other rows for each
    (1, 640, 1, 192, 70, "int8"),           # several tiles to a CTA of the same rows
], ids=str)
def test_account_gives_up_and_recovers(short_waits, B, H, K, d, k, fmt):
    T = 2500
    g = torch.Generator("cuda").manual_seed(B + d)
    q = torch.randn(B, H, d, device="cuda", generator=g).bfloat16()
    idx = torch.rand(B, T, device="cuda", generator=g).topk(k, dim=1).indices.int()
    lse = torch.full((B, H), 5.0, device="cuda")
    if fmt == "bf16":
        kv, kw = torch.randn(B, T, K, d, device="cuda", generator=g).bfloat16(), {}
    else:
        kv, kw = cache(g, fmt, T, K, d), dict(scales=torch.full((-(-T // 16), K), 0.01, device="cuda"), block=16)

    def account():
        return ds.ds_attention_mass(q, kv, idx, lse, torch.ones(B, T, device="cuda"), **kw)

    want = account()
    assert ds.ds_get_device_status() == ds.DS_OK
    got = planted(account)
    assert torch.all(got >= 1.0) and torch.all(got <= want) and not torch.equal(got, want), "the first CTA's weights are missing"
    for _ in range(2):
        assert torch.equal(account(), want) and ds.ds_get_device_status() == ds.DS_OK
