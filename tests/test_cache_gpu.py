"""GPU parity of the 8-bit cache (ds_cache_quantize, ds_sparse_attention_q8,
ds_attention_mass, ds_cache_evict, ds_cache_compact) with the float64 oracle.

Bounds.  Codes, scales, lists and moved bytes are equal.  For the attention, with
z a score and row its row:

* a score is a sum of d products, each addition off by at most 2^-23 of the
  magnitudes added (rounded or cut off), and is then multiplied by a row's factor
  of three roundings: |dz| <= (d + 8) 2^-23 * reach, reach the largest
  scale * sum_c |q_c row_c| of an attended row;
* lse is off by at most the largest |dz|, n additions of positive terms
  (n 2^-24), and the roundings of the exponentials, the logarithm and lse itself:
  2^-20 (1 + |lse|) + the rounding of log2 scores, 2^-22 |z| <= 2^-22 reach;
* a weight p of out is rounded once to bfloat16 (half a step, 2^-8, of p, or of p
  times the row's scale), so a component is off by (2^-8 + 2 dz + n 2^-23) spread,
  spread = sum_r p_r |row_r|, and by the rounding of out, 2^-8 |out|;
* an account gains sum_h p_h with |dp_h| <= (dz + the roundings of lse and z in
  log2 units, 2^-21 (1 + |lse| + reach)) p_h, and H additions.
"""

import math

import numpy as np
import pytest
import torch

import sparse_attention_top_ds_b200 as ds
from oracle import cache as oracle
from sparse_attention_top_ds_b200 import inputs

from gpu_util import bf16_to_device, bits_of, f32_to_device, i32_to_device

pytestmark = pytest.mark.gpu

TORCH = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def codes_to_device(codes, fmt, dev="cuda"):
    return torch.from_numpy(np.ascontiguousarray(codes)).to(dev).view(TORCH[fmt])


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def dec(bits):
    return inputs.bf16_bits_to_f32(bits).astype(np.float64)


def ok_status(skipped=False):
    """No error on the device; ``skipped``: slots outside [0, T) or rows past a cache's end were given, which the
    debug build records."""
    torch.cuda.synchronize()
    assert ds.ds_get_device_status() in ((ds.DS_OK, ds.DS_ERR_RANGE) if skipped and ds.ds_debug_build() else (ds.DS_OK,))


def quantized(rows, block, fmt):
    """Oracle codes [B, n, heads, d] and scales of whole rows."""
    B, n, K, d = rows.shape
    x = inputs.bf16_bits_to_f32(rows)
    codes, scales = np.zeros(rows.shape, np.uint8), np.zeros((B, -(-n // block), K), np.float32)
    for b in range(B):
        for m in range(scales.shape[1]):
            for g in range(K):
                s = slice(m * block, (m + 1) * block)
                codes[b, s, g], scales[b, m, g] = oracle.quantize_block(x[b, s, g], fmt)
    return codes, scales


# ---------------------------------------------------------------- writing

WRITE = [
    # B, n, K, d, T, block, fmt, pos, len
    (1, 1, 1, 64, 1, 1, "e4m3", None, None),
    (8, 1, 1, 512, 40, 1, "e4m3", [0, 1, 5, 39, 7, 20, 33, 2], None),
    (2, 1, 3, 192, 9, 1, "int8", [8, 0], [1, 0]),
    (3, 37, 2, 128, 64, 16, "int8", [0, 16, 16], [37, 20, 0]),
    (2, 100, 1, 64, 200, 128, "e4m3", [128, 0], None),
    (1, 257, 1, 512, 300, 128, "e4m3", None, None),
    (2, 33, 8, 192, 48, 32, "e4m3", None, [33, 32]),
    (1, 70, 1, 448, 100, 64, "int8", [0], [65]),
    (2, 5, 1, 320, 8, 2, "e4m3", [2, 4], None),
    (1, 9, 5, 64, 16, 4, "int8", [4], [9]),
    (1, 130, 1, 384, 256, 8, "e4m3", [96], None),
]


@pytest.mark.parametrize("case", WRITE, ids=lambda c: "x".join(map(str, c[:7])))
def test_quantize_matches_the_oracle(cuda_device, case):
    B, n, K, d, T, block, fmt, pos, length = case
    rows = inputs.cache_rows(100 + n, B, n, K, d)
    codes = np.full((B, T, K, d), 0x2A, np.uint8)
    scales = np.full((B, -(-T // block), K), -3.0, np.float32)
    gc, gs = codes_to_device(codes, fmt), f32_to_device(scales)
    p = None if pos is None else i32_to_device(np.array(pos))
    ln = None if length is None else i32_to_device(np.array(length))
    r = ds.ds_cache_quantize(bf16_to_device(rows), gc, gs, block, pos=p, length=ln)
    assert r[0] is gc and r[1] is gs
    ok_status(skipped=T < n + max(pos or [0]))  # rows past the cache's end are cut
    for b in range(B):
        m = n if length is None else length[b]
        at = 0 if pos is None else pos[b]
        m = min(m, T - at)  # rows past the cache's end are not written, nor part of a scale
        if m:
            c, s = quantized(rows[b:b + 1, :m], block, fmt)
            codes[b, at:at + m], scales[b, at // block:at // block + s.shape[1]] = c[0], s[0]
    assert np.array_equal(codes_of(gc), codes)
    assert np.array_equal(bits_of(gs), scales.view(np.uint32))


def test_quantize_every_bfloat16_value(cuda_device):
    # all finite patterns, as the 64 values of one row each with a largest one beside them
    bits = np.arange(65536, dtype=np.uint16)
    bits = bits[(bits & 0x7f80) != 0x7f80].reshape(-1, 1, 64)
    rows = np.ascontiguousarray(bits[None])
    for fmt in ("e4m3", "int8"):
        c, s = quantized(rows, 1, fmt)
        gc, gs = torch.zeros(rows.shape, dtype=TORCH[fmt], device="cuda"), torch.zeros(s.shape, device="cuda")
        ds.ds_cache_quantize(bf16_to_device(rows), gc, gs, 1)
        ok_status()
        assert np.array_equal(codes_of(gc), c) and np.array_equal(bits_of(gs), s.view(np.uint32))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_quantize_marks_blocks_that_are_not_finite(cuda_device, fmt, bad):
    x = inputs.bf16_bits_to_f32(inputs.cache_rows(4, 1, 20, 2, 128))
    x[0, 9, 1, 77] = bad
    rows = inputs.f32_to_bf16_bits(x) if np.isfinite(bad) else (np.ascontiguousarray(x).view(np.uint32) >> 16).astype(np.uint16)
    gc, gs = torch.full((1, 20, 2, 128), 1, dtype=torch.int8, device="cuda").view(TORCH[fmt]), torch.zeros(1, 3, 2, device="cuda")
    ds.ds_cache_quantize(bf16_to_device(rows), gc, gs, 8)
    ok_status()
    c, s = quantized(rows, 8, fmt)
    assert np.isnan(gs.cpu().numpy()[0, 1, 1]) and np.isnan(gs.cpu().numpy()).sum() == 1
    assert np.array_equal(codes_of(gc), c) and not codes_of(gc)[0, 8:16, 1].any()


def test_quantize_skips_bad_positions_and_clips_lengths(cuda_device):
    # positions that are no multiple of the block, negative or past the cache leave the batch row alone; lengths are cut
    # to [0, n] and to the cache's end
    rows = inputs.cache_rows(5, 7, 10, 1, 64)
    pos, length = np.array([2, -4, 44, 40, 36, 0, 0]), np.array([10, 10, 10, 10, 99, -3, 4])
    gc, gs = torch.full((7, 40, 1, 64), 9, dtype=torch.int8, device="cuda"), torch.full((7, 10, 1), 5.0, device="cuda")
    ds.ds_cache_quantize(bf16_to_device(rows), gc, gs, 4, pos=i32_to_device(pos), length=i32_to_device(length))
    torch.cuda.synchronize()
    assert ds.ds_get_device_status() == (ds.DS_ERR_RANGE if ds.ds_debug_build() else ds.DS_OK)
    want, wants = np.full((7, 40, 1, 64), 9, np.uint8), np.full((7, 10, 1), 5.0, np.float32)
    for b, at, n in ((4, 36, 4), (6, 0, 4)):
        c, s = quantized(rows[b:b + 1, :n], 4, "int8")
        want[b, at:at + n], wants[b, at // 4:at // 4 + 1] = c[0], s[0]
    assert np.array_equal(codes_of(gc), want) and np.array_equal(gs.cpu().numpy(), wants)


def test_quantize_strided_rows_and_caches(cuda_device):
    # rows out of a wider tensor, caches that are slices of larger ones, one row given to every batch row
    wide = inputs.cache_rows(6, 3, 2 * 12, 3, 128)
    gw = bf16_to_device(wide)
    big, bigs = torch.zeros(3, 30, 2, 128, dtype=torch.int8, device="cuda"), torch.zeros(3, 9, 2, device="cuda")
    view = gw[:, ::2, :2]
    assert not view.is_contiguous()
    ds.ds_cache_quantize(view, big[:, 4:24], bigs[:, 2:7], 4)
    c, s = quantized(np.ascontiguousarray(wide[:, ::2, :2]), 4, "int8")
    ok_status()
    want, wants = np.zeros((3, 30, 2, 128), np.uint8), np.zeros((3, 9, 2), np.float32)
    want[:, 4:16], wants[:, 2:5] = c, s
    assert np.array_equal(codes_of(big), want) and np.array_equal(bigs.cpu().numpy(), wants)
    same = gw[:1, :12, :2].expand(3, 12, 2, 128)
    ds.ds_cache_quantize(same, big[:, 4:24], bigs[:, 2:7], 4)
    ok_status()
    c, s = quantized(np.ascontiguousarray(wide[:1, :12, :2]), 4, "int8")
    assert all(np.array_equal(codes_of(big)[b, 4:16], c[0]) for b in range(3))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("block", [1, 4, 64, 128])
def test_quantize_many_rows_matches_the_formula(cuda_device, fmt, block):
    # the same float32 operations in torch on 4 x 3000 rows: a product and a rounding per value
    torch.manual_seed(7)
    x = torch.randn(4, 3000, 2, 192, device="cuda").to(torch.bfloat16)
    nb = -(-3000 // block)
    gc, gs = torch.zeros(4, 3000, 2, 192, dtype=TORCH[fmt], device="cuda"), torch.zeros(4, nb, 2, device="cuda")
    ds.ds_cache_quantize(x, gc, gs, block)
    ok_status()
    pad = torch.zeros(4, nb * block, 2, 192, device="cuda")
    pad[:, :3000] = x.float()
    y = pad.view(4, nb, block, 2, 192)
    a = y.abs().amax(dim=(2, 4))
    top = torch.full_like(a, oracle.TOP[fmt])
    v = y * torch.div(top, a)[:, :, None, :, None]
    want = (v.round() if fmt == "int8" else v).to(TORCH[fmt]).view(4, nb * block, 2, 192)[:, :3000]
    assert torch.equal(gs, torch.div(a, top))
    assert torch.equal(gc.view(torch.uint8), want.contiguous().view(torch.uint8))


# ---------------------------------------------------------------- attention

ATTEND = [
    # B, H, K, d, T, k, W, block, fmt, shared, sink, holes, win_len
    (1, 1, 1, 64, 1, 1, 0, 1, "e4m3", False, False, 0.0, None),
    (1, 16, 1, 128, 500, 64, 0, 16, "e4m3", False, False, 0.0, None),
    (2, 128, 1, 512, 600, 200, 33, 64, "e4m3", False, True, 0.0, None),
    (3, 128, 1, 512, 300, 129, 128, 64, "int8", True, True, 0.1, [0, 77, 128]),
    (2, 40, 8, 192, 500, 333, 77, 32, "int8", False, True, 0.2, [10, 77]),
    (1, 64, 1, 512, 900, 700, 0, 128, "e4m3", True, False, 0.0, None),
    (2, 65, 1, 256, 200, 100, 5, 8, "int8", False, False, 0.0, None),
    (1, 200, 2, 320, 100, 64, 3, 2, "e4m3", False, True, 0.0, None),
    (5, 17, 1, 448, 60, 60, 1, 4, "int8", False, False, 0.5, [1, 0, 1, 1, 0]),
    (2, 8, 8, 64, 50, 13, 2, 1, "e4m3", False, True, 0.0, None),
    (2, 33, 1, 384, 40, 0, 19, 16, "e4m3", False, True, 0.0, [19, 0]),
    (1, 3, 1, 64, 9, 20, 0, 128, "int8", False, False, 0.0, None),
    (2, 130, 1, 128, 2500, 2048, 0, 64, "e4m3", True, True, 0.0, None),
    (1, 32, 1, 576 - 64, 400, 300, 300, 1, "int8", False, False, 0.0, None),
    (9, 24, 4, 64, 300, 160, 40, 16, "e4m3", True, True, 0.3, None),
]


def attend_inputs(case, seed=200):
    B, H, K, d, T, k, W, block, fmt, shared, sink, holes, wl = case
    rows = inputs.cache_rows(seed, 1 if shared else B, T, K, d)
    codes, scales = quantized(rows, block, fmt)
    g = inputs.rng(seed + 1)
    return dict(q=inputs.f32_to_bf16_bits(g.standard_normal((B, H, d))), codes=codes, scales=scales,
                idx=inputs.cache_slots(seed + 2, B, T, k, holes), win=inputs.cache_rows(seed + 3, B, W, K, d) if W else None,
                win_len=None if wl is None else np.array(wl, np.int32), sink=g.standard_normal(H).astype(np.float32) if sink else None,
                scale=1.0 / math.sqrt(d))


def attend(case, a, **kw):
    B, H, K, d, T, k, W, block, fmt, shared = case[:10]
    codes, scales = codes_to_device(a["codes"], fmt), f32_to_device(a["scales"])
    t = dict(q=bf16_to_device(a["q"]), codes=codes[0] if shared else codes, scales=scales[0] if shared else scales,
             idx=i32_to_device(a["idx"]) if k else None, win=None if a["win"] is None else bf16_to_device(a["win"]),
             win_len=None if a["win_len"] is None else i32_to_device(a["win_len"]),
             sink=None if a["sink"] is None else f32_to_device(a["sink"]))
    return ds.ds_sparse_attention_q8(t["q"], t["codes"], t["scales"], t["idx"], block, win=t["win"], win_len=t["win_len"],
                                     sink=t["sink"], return_lse=True, **kw), t


def check_attention(case, a, out, lse, scale=None):
    B, H, K, d, T, k, W, block, fmt, shared = case[:10]
    wide = (np.broadcast_to(a["codes"], (B,) + a["codes"].shape[1:]), np.broadcast_to(a["scales"], (B,) + a["scales"].shape[1:]))
    ref, ref_lse, spread, reach = oracle.attention_q8(a["q"], *wide, a["idx"], block, fmt, a["scale"] if scale is None else scale,
                                                      win=a["win"], win_len=a["win_len"], sink=a["sink"])
    out, lse = dec(bits_of(out)), lse.cpu().numpy().astype(np.float64)
    n = k + W
    dz = (d + 8) * 2.0 ** -23 * reach
    none = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(lse), none) and np.all(out[none] == 0.0)
    tol = dz + n * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(np.where(none, 0.0, ref_lse))) + 2.0 ** -22 * reach
    assert np.all(np.abs(lse - ref_lse)[~none] <= tol[~none]), np.max((np.abs(lse - ref_lse) / tol)[~none])
    tol = (2.0 ** -8 + 2 * dz + n * 2.0 ** -23 + 2.0 ** -20)[..., None] * spread + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(out - ref) <= tol), np.max(np.abs(out - ref) / np.maximum(tol, 1e-300))


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "x".join(map(str, c[:10])))
def test_attention_matches_the_oracle(cuda_device, case):
    a = attend_inputs(case)
    (out, lse), _ = attend(case, a)
    ok_status(skipped=case[11] > 0)
    check_attention(case, a, out, lse)


# B, H, K, d, T, k, W, block, fmt, shared, sink, holes, win_len: at most 32 query heads to a KV head, or at most 64 rows
FEW = [
    (3, 1, 1, 64, 50, 1, 0, 1, "e4m3", False, False, 0.0, None),
    (6, 16, 2, 512, 90, 2, 0, 4, "int8", False, False, 0.0, None),
    (5, 32, 1, 192, 200, 3, 0, 1, "e4m3", False, True, 0.0, None),
    (4, 64, 2, 320, 120, 7, 2, 1, "int8", True, False, 0.0, [2, 0, 1, 2]),
    (3, 24, 1, 448, 300, 40, 9, 8, "e4m3", False, True, 0.2, [9, 1, 4]),
    (2, 32, 1, 512, 600, 150, 70, 2, "e4m3", False, False, 0.0, None),
    (160, 128, 1, 128, 80, 2, 0, 1, "int8", True, False, 0.0, None),
    (80, 100, 1, 256, 90, 33, 31, 1, "e4m3", True, True, 0.0, None),
    (300, 128, 1, 64, 90, 20, 5, 2, "e4m3", True, False, 0.1, None),
    (250, 33, 1, 512, 70, 64, 0, 1, "int8", True, False, 0.0, None),
]


@pytest.mark.parametrize("case", FEW, ids=lambda c: "x".join(map(str, c[:10])))
def test_attention_over_few_rows_is_rounded_once(cuda_device, case):
    """A weight of out is the sum of two bfloat16 numbers, the second rounded from what the first lost: off by at most
    2^-8 * 2^-8 of it.  So out before its rounding is off by t = (2^-16 + 2 dz + n 2^-23 + 2^-20) spread (the terms of
    the file's bounds with 2^-16 for the weights' 2^-8), and out by t and half a step at |ref| + t: a bfloat16 number has 8
    bits, so half a step at y is 2^(floor(log2 y) - 8)."""
    a = attend_inputs(case)
    (out, lse), _ = attend(case, a)
    ok_status(skipped=case[11] > 0)
    B, H, K, d, T, k, W, block, fmt, shared = case[:10]
    wide = (np.broadcast_to(a["codes"], (B,) + a["codes"].shape[1:]), np.broadcast_to(a["scales"], (B,) + a["scales"].shape[1:]))
    ref, ref_lse, spread, reach = oracle.attention_q8(a["q"], *wide, a["idx"], block, fmt, a["scale"], win=a["win"], win_len=a["win_len"],
                                                sink=a["sink"])
    t = (2.0 ** -16 + 2 * (d + 8) * 2.0 ** -23 * reach + (k + W) * 2.0 ** -23 + 2.0 ** -20)[..., None] * spread
    half = np.exp2(np.floor(np.log2(np.maximum(np.abs(ref) + t, 1e-30))) - 8)
    err = np.abs(dec(bits_of(out)) - ref)
    assert np.all(err <= t + half), (np.max(err / (t + half)), np.mean(err > t + half))
    none = np.isneginf(ref_lse)  # no row and no sink
    assert np.array_equal(np.isneginf(lse.cpu().numpy()), none)
    tol = ((d + 8) * 2.0 ** -23 + 2.0 ** -22) * reach + (k + W) * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(np.where(none, 0.0, ref_lse)))
    assert np.all(np.abs(lse.cpu().numpy() - ref_lse)[~none] <= tol[~none])


def test_attention_skips_everything(cuda_device):
    case = (2, 20, 1, 64, 30, 9, 4, 4, "int8", False, False, 0.0, [0, 0])
    a = attend_inputs(case)
    a["idx"][:] = np.array([-1, 30, 31, -1, 2 ** 31 - 1, -1, -1, 40, -1])
    (out, lse), _ = attend(case, a)
    torch.cuda.synchronize()
    assert np.all(dec(bits_of(out)) == 0.0) and np.all(np.isneginf(lse.cpu().numpy()))
    a["sink"] = np.linspace(-5, 80, 20).astype(np.float32)
    (out, lse), _ = attend(case, a)
    torch.cuda.synchronize()
    ds.ds_get_device_status()  # the debug build records the slots out of range
    assert np.all(dec(bits_of(out)) == 0.0)
    assert np.allclose(lse.cpu().numpy(), np.tile(a["sink"], (2, 1)), rtol=2.0 ** -22, atol=2.0 ** -22)


def test_attention_repeated_and_out_of_order_slots(cuda_device):
    case = (2, 12, 2, 128, 40, 150, 0, 8, "e4m3", False, False, 0.0, None)
    a = attend_inputs(case)
    a["idx"] = np.random.default_rng(3).integers(0, 40, size=(2, 150)).astype(np.int32)
    (out, lse), _ = attend(case, a)
    ok_status()
    check_attention(case, a, out, lse)


def test_attention_large_scores(cuda_device):
    # scores of hundreds: one row takes nearly all of the weight, far ones underflow; ascending over the slots, so that
    # every piece of the rows brings a new maximum
    case = (1, 70, 1, 128, 512, 512, 64, 16, "e4m3", False, True, 0.0, None)
    a = attend_inputs(case)
    a["idx"][0] = np.arange(512)
    a["codes"] = np.broadcast_to(a["codes"][:, :1], a["codes"].shape).copy()
    a["scales"] = (a["scales"][:, :1] * (np.arange(32)[None, :, None] + 1)).astype(np.float32)
    (out, lse), _ = attend(case, a)
    ok_status()
    check_attention(case, a, out, lse)
    for order in (np.arange(511, -1, -1), np.random.default_rng(5).permutation(512)):
        a["idx"][0] = order
        (out, lse), _ = attend(case, a, scale=0.5)
        ok_status()
        check_attention(case, a, out, lse, scale=0.5)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_attention_scale(cuda_device, scale):
    case = (2, 18, 1, 64, 90, 70, 9, 2, "int8", False, True, 0.1, [9, 3])
    a = attend_inputs(case)
    (out, lse), _ = attend(case, a, scale=scale)
    torch.cuda.synchronize()
    ds.ds_get_device_status()
    check_attention(case, a, out, lse, scale=scale)


def test_attention_reads_only_what_is_selected(cuda_device):
    # NaN scales, NaN codes and NaN window rows where nothing points: the results do not change by a bit
    case = (3, 24, 2, 128, 200, 40, 20, 4, "e4m3", False, True, 0.3, [20, 5, 0])
    a = attend_inputs(case)
    (out, lse), _ = attend(case, a)
    for b in range(3):
        used = {int(r) for r in a["idx"][b] if 0 <= r < 200}
        for r in range(200):
            if r not in used:
                a["codes"][b, r] = 0x7F
        for n in range(50):
            if not used & set(range(4 * n, 4 * n + 4)):
                a["scales"][b, n] = np.nan
        a["win"][b, a["win_len"][b]:] = 0x7FC0
    (out2, lse2), _ = attend(case, a)
    torch.cuda.synchronize()
    ds.ds_get_device_status()
    assert np.array_equal(bits_of(out), bits_of(out2)) and np.array_equal(bits_of(lse), bits_of(lse2))


def test_attention_over_a_block_that_is_not_finite_is_nan(cuda_device):
    case = (2, 8, 2, 64, 64, 20, 0, 4, "int8", False, False, 0.0, None)
    a = attend_inputs(case)
    a["scales"][1, a["idx"][1, 3] // 4, 1] = np.nan
    (out, lse), _ = attend(case, a)
    ok_status()
    o = dec(bits_of(out))
    assert np.isnan(o[1, 4:]).all() and np.isfinite(o[0]).all() and np.isfinite(o[1, :4]).all()
    assert np.isnan(lse.cpu().numpy()[1, 4:]).all() and np.isfinite(lse.cpu().numpy()[0]).all()


@pytest.mark.parametrize("heads", [(8, 2), (20, 1), (130, 2)], ids=str)
@pytest.mark.parametrize("code,channel", [(0x7F, 0), (0xFF, 129), (0x7F, 191), (0xFF, 62)])
def test_attention_over_a_nan_code_is_nan(cuda_device, heads, code, channel):
    H, K = heads
    case = (2, H, K, 192, 700, 600, 30, 4, "e4m3", False, False, 0.0, None)
    a = attend_inputs(case)
    (out, lse), _ = attend(case, a)
    a["codes"][1, a["idx"][1, 301], K - 1, channel] = code
    (out2, lse2), _ = attend(case, a)
    ok_status()
    hit = np.zeros((2, H), bool)
    hit[1, H - H // K:] = True  # the heads of the last KV head of batch row 1
    assert np.isnan(dec(bits_of(out2))[hit]).all() and np.isnan(lse2.cpu().numpy()[hit]).all()
    assert np.array_equal(bits_of(out)[~hit], bits_of(out2)[~hit]) and np.array_equal(bits_of(lse)[~hit], bits_of(lse2)[~hit])


def test_attention_every_code(cuda_device):
    # one-hot queries on a single row read the row itself: all finite codes of both formats come back exactly
    for fmt in ("e4m3", "int8"):
        codes = np.arange(256, dtype=np.uint8)
        if fmt == "e4m3":
            codes[[0x7F, 0xFF]] = 0
        codes = codes.reshape(1, 1, 1, 256)
        q = np.zeros((1, 1, 256), np.uint16)
        out = ds.ds_sparse_attention_q8(bf16_to_device(q), codes_to_device(codes, fmt), torch.ones(1, 1, 1, device="cuda"),
                                        i32_to_device(np.zeros((1, 1))), 1)
        ok_status()
        assert np.array_equal(dec(bits_of(out))[0, 0], oracle.decode(codes[0, 0, 0], fmt))


def test_attention_strided_batches_and_broadcast_caches(cuda_device):
    case = (3, 16, 1, 128, 100, 50, 0, 8, "int8", False, False, 0.0, None)
    a = attend_inputs(case)
    (out, lse), t = attend(case, a)
    big = torch.zeros(3, 140, 1, 128, dtype=torch.int8, device="cuda")
    bigs = torch.zeros(3, 20, 1, device="cuda")
    big[:, 40:], bigs[:, 4:17] = t["codes"], t["scales"]
    o2, l2 = ds.ds_sparse_attention_q8(t["q"], big[:, 40:], bigs[:, 4:17], t["idx"], 8, return_lse=True)
    one = ds.ds_sparse_attention_q8(t["q"], t["codes"][0], t["scales"][0], t["idx"], 8)
    exp = ds.ds_sparse_attention_q8(t["q"], t["codes"][:1].expand(3, 100, 1, 128), t["scales"][:1].expand(3, 13, 1), t["idx"], 8)
    ok_status()
    assert torch.equal(out, o2) and torch.equal(lse, l2) and torch.equal(one, exp)
    buf, bl = torch.zeros_like(out), torch.zeros_like(lse)
    r = ds.ds_sparse_attention_q8(t["q"], t["codes"], t["scales"], t["idx"], 8, out=buf, lse=bl, return_lse=True)
    assert r[0] is buf and r[1] is bl and torch.equal(buf, out) and torch.equal(bl, lse)


def test_attention_far_rows_of_a_long_cache(cuda_device):
    # rows behind the 2^32nd byte of one cache, and a batch stride past it
    T, d = 9_000_000, 512
    codes = torch.zeros(T, 1, d, dtype=torch.int8, device="cuda")
    scales = torch.full((-(-T // 64), 1), 0.03125, device="cuda")
    g = np.random.default_rng(11)
    idx = np.sort(g.choice(T, size=(2, 30), replace=False), axis=1).astype(np.int32)
    idx[0, -1] = T - 1
    idx[1, -3:] = (T - 5, 8_388_608, 8_388_607)
    vals = g.integers(-90, 91, size=(60, d)).astype(np.int8)
    for i, r in enumerate(idx.ravel()):
        codes[int(r), 0] = torch.from_numpy(vals[i]).cuda()
    q = inputs.f32_to_bf16_bits(g.standard_normal((2, 16, d)))
    out, lse = ds.ds_sparse_attention_q8(bf16_to_device(q), codes, scales, i32_to_device(idx), 64, return_lse=True)
    mass = ds.ds_attention_mass(bf16_to_device(q), codes, i32_to_device(idx), lse, torch.zeros(2, T, device="cuda"), scales=scales,
                                block=64)
    ok_status()
    small = dict(q=q, codes=vals.reshape(2, 30, 1, d).view(np.uint8), scales=np.full((2, 30, 1), 0.03125, np.float32),
                 idx=np.tile(np.arange(30, dtype=np.int32), (2, 1)), win=None, win_len=None, sink=None, scale=1 / math.sqrt(d))
    check_attention((2, 16, 1, d, 30, 30, 0, 1, "int8", False), small, out, lse)
    got = mass.cpu().numpy()
    assert np.allclose(got.sum(1, dtype=np.float64), 16.0, rtol=1e-5)
    assert all((got[b] != 0).sum() == 30 and np.all(got[b, idx[b]] > 0) for b in range(2))


# ---------------------------------------------------------------- the account

MASS = [
    # B, H, K, d, T, k, block, fmt, shared, holes
    (1, 1, 1, 64, 1, 1, 1, "e4m3", False, 0.0),
    (2, 128, 1, 512, 600, 200, 64, "e4m3", False, 0.0),
    (3, 128, 1, 512, 300, 129, 64, "int8", True, 0.2),
    (5, 40, 8, 192, 200, 133, 1, "bf16", False, 0.2),
    (2, 130, 1, 256, 300, 257, 8, "int8", False, 0.0),
    (1, 200, 2, 320, 100, 64, 2, "e4m3", False, 0.0),
    (2, 9, 1, 448, 60, 60, 1, "bf16", False, 0.5),
    (2, 33, 3, 64, 40, 33, 1, "e4m3", True, 0.0),
    (4, 128, 1, 128, 700, 640, 1, "bf16", True, 0.0),
    (2, 48, 12, 64, 50, 20, 4, "int8", False, 0.1),     # more KV heads than a cluster has CTAs
    (1, 640, 1, 192, 90, 70, 8, "e4m3", False, 0.0),    # more head tiles than that
]


def mass_inputs(case, seed=300):
    B, H, K, d, T, k, block, fmt, shared, holes = case
    rows = inputs.cache_rows(seed, 1 if shared else B, T, K, d)
    codes, scales = (rows, None) if fmt == "bf16" else quantized(rows, block, fmt)
    g = inputs.rng(seed + 1)
    return dict(q=inputs.f32_to_bf16_bits(g.standard_normal((B, H, d))), codes=codes, scales=scales,
                idx=inputs.cache_slots(seed + 2, B, T, k, holes), mass=inputs.accounts(seed + 3, B, T),
                lse=(math.log(k) + 0.5 + 0.3 * g.standard_normal((B, H))).astype(np.float32), scale=1.0 / math.sqrt(d))


def account(case, a, mass=None, **kw):
    B, H, K, d, T, k, block, fmt, shared, holes = case
    if fmt == "bf16":
        c, s = bf16_to_device(a["codes"]), None
        c = c.expand(B, T, K, d) if shared else c
        c = (c[0, :, 0] if shared else c[:, :, 0]) if K == 1 else c
    else:
        c, s = codes_to_device(a["codes"], fmt), f32_to_device(a["scales"])
        c, s = (c[0], s[0]) if shared else (c, s)
    mass = f32_to_device(a["mass"]) if mass is None else mass
    r = ds.ds_attention_mass(bf16_to_device(a["q"]), c, i32_to_device(a["idx"]), f32_to_device(a["lse"]), mass, scales=s, block=block,
                             **kw)
    assert r is mass
    return mass


def check_mass(case, a, mass, times=1):
    B, H, K, d, T, k, block, fmt, shared, holes = case
    wide = np.broadcast_to(a["codes"], (B,) + a["codes"].shape[1:])
    sc = None if a["scales"] is None else np.broadcast_to(a["scales"], (B,) + a["scales"].shape[1:])
    ref, added, reach = oracle.attention_mass(a["q"], wide, sc, a["idx"], block, fmt, a["scale"], a["lse"], a["mass"])
    ref = a["mass"] + times * added
    big = np.where(np.isinf(a["lse"]), 0, np.abs(a["lse"])) + reach
    rel = ((d + 8) * 2.0 ** -23 * reach + 2.0 ** -21 * (1 + big)).max(1) + (H + 2) * 2.0 ** -23
    tol = times * (added * rel[:, None] + 2.0 ** -23 * np.abs(ref))
    err = np.abs(mass.cpu().numpy().astype(np.float64) - ref)
    assert np.all(err <= tol), np.max(err / np.maximum(tol, 1e-300))
    assert np.array_equal(bits_of(mass)[added == 0], a["mass"].view(np.uint32)[added == 0])


@pytest.mark.parametrize("case", MASS, ids=lambda c: "x".join(map(str, c)))
def test_mass_matches_the_oracle(cuda_device, case):
    a = mass_inputs(case)
    mass = account(case, a)
    ok_status(skipped=case[9] > 0)
    check_mass(case, a, mass)
    check_mass(case, a, account(case, a, mass=mass), times=2)
    again = account(case, a)
    assert np.array_equal(bits_of(again), bits_of(account(case, a)))
    ok_status(skipped=case[9] > 0)


def test_mass_heads_without_a_softmax_add_nothing(cuda_device):
    case = (2, 70, 1, 64, 50, 20, 4, "int8", False, 0.0)
    a = mass_inputs(case)
    a["lse"][0, :] = -np.inf
    a["lse"][1, 3:66] = -np.inf
    check_mass(case, a, account(case, a))
    ok_status()


@pytest.mark.parametrize("code,channel", [(0x7F, 0), (0xFF, 129), (0x7F, 191), (0xFF, 62)])
def test_mass_of_a_row_with_a_nan_code_is_nan(cuda_device, code, channel):
    case = (2, 24, 2, 192, 300, 200, 4, "e4m3", False, 0.0)
    a = mass_inputs(case)
    mass, row = account(case, a), a["idx"][1, 77]
    a["codes"][1, row, 1, channel] = code
    got = account(case, a)
    ok_status()
    assert torch.isnan(got[1, row])
    got[1, row] = mass[1, row]
    assert np.array_equal(bits_of(mass), bits_of(got))


def test_mass_strided_accounts_repeated_slots_and_no_slots(cuda_device):
    case = (3, 20, 1, 128, 30, 24, 1, "bf16", False, 0.0)
    a = mass_inputs(case)
    a["idx"] = np.random.default_rng(1).integers(0, 30, size=(3, 24)).astype(np.int32)
    big = torch.full((3, 50), -1.0, device="cuda")
    big[:, 10:40] = f32_to_device(a["mass"])
    mass = account(case, a, mass=big[:, 10:40])
    ok_status()
    # at most 24 additions to one account, in any order
    ref, added, reach = oracle.attention_mass(a["q"], a["codes"], None, a["idx"], 1, "bf16", a["scale"], a["lse"], a["mass"])
    tol = added * (136 * 2.0 ** -23 * reach.max() + 2.0 ** -21 * (10 + reach.max()) + 22 * 2.0 ** -23) + 24 * 2.0 ** -23 * ref
    assert np.all(np.abs(mass.cpu().numpy() - ref) <= tol)
    assert torch.all(big[:, :10] == -1.0) and torch.all(big[:, 40:] == -1.0)
    a["idx"] = np.zeros((3, 0), np.int32)
    before = big.clone()
    account(case, a, mass=big[:, 10:40])
    ok_status()
    assert torch.equal(big, before)


# ---------------------------------------------------------------- eviction

EVICT = [
    # B, T, block, budget, first, last, lengths
    (1, 1, 1, 1, 0, 0, None),
    (1, 1, 128, 1, 1, 0, None),
    (2, 100, 1, 37, 4, 10, None),
    (3, 100, 16, 4, 1, 2, [100, 33, 0]),
    (2, 5000, 1, 4096, 0, 0, [5000, 4097]),
    (4, 3001, 8, 100, 0, 1, [3001, 1, 799, 2999]),
    (1, 40000, 1, 20000, 16, 512, None),
    (2, 33000, 64, 16, 1, 2, [33000, 1025]),
    (1, 70000, 2, 1, 0, 0, None),
    (2, 9999, 128, 78, 10, 68, [9999, 9985]),
    (3, 2048, 4, 511, 0, 0, [2048, 2047, 2045]),
]


def evict(mass, case, length=None, **kw):
    B, T, block, budget, first, last, lengths = case
    ln = lengths if length is None else length
    r = ds.ds_cache_evict(mass, budget, block=block, length=None if ln is None else i32_to_device(np.array(ln)), keep_first=first,
                          keep_last=last, **kw)
    ok_status()
    return r[0].cpu().numpy(), r[1].cpu().numpy()


@pytest.mark.parametrize("T,block,budget", [(500_000, 1, 300_000), (3_000_000, 2, 1_000_000), (3_000_000, 128, 20_000)])
def test_evict_long_rows(cuda_device, T, block, budget):
    # more blocks to a CTA than it holds keys of; whole-number accounts, so that there are ties and sums are exact
    m = torch.randint(0, 1000, (2, T), device="cuda", generator=torch.Generator("cuda").manual_seed(5)).float()
    kept, n = ds.ds_cache_evict(m, budget, block=block, keep_first=3, keep_last=5)
    ok_status()
    nb = -(-T // block)
    key = torch.nn.functional.pad(m, (0, nb * block - T)).view(2, nb, block).sum(-1)
    key[:, :3], key[:, nb - 5:] = 1e9, 1e9
    want = key.sort(dim=1, descending=True, stable=True).indices[:, :budget].sort(dim=1).values
    assert torch.equal(kept.long(), want) and n.tolist() == [budget * block - (nb * block - T)] * 2


@pytest.mark.parametrize("block", [4, 8, 16, 32])
def test_evict_keys_of_equal_blocks_are_equal_wherever_they_are(cuda_device, block):
    # More blocks to a CTA than it holds keys of, made of a few patterns of accounts that cancel, so that a sum in another
    # order is another: blocks of one pattern have one key, and the lower ones stay.  The keys: halves of a block added row
    # by row, then halves of that.
    nb = 8 * 48 * 1024 + 90_001
    g = torch.Generator("cuda").manual_seed(block)
    pool = torch.rand(8, block, device="cuda", generator=g) + 0.5
    for i, at in enumerate((0, 0, 1, 1, 0, 1, 0, 1)):  # a large term that cancels some rows later
        pool[i, at], pool[i, block // 2 + (i * 5 + at) % (block // 2)] = 1e25, -1e25
    pick = torch.randint(0, 8, (1, nb), device="cuda", generator=g)
    m = pool[pick].view(1, nb * block)
    x = pool.double()
    while x.shape[1] > 1:
        x = x[:, :x.shape[1] // 2] + x[:, x.shape[1] // 2:]
    key = x[:, 0].float()[pick]
    budget = nb // 3
    kept, n = ds.ds_cache_evict(m, budget, block=block, keep_last=0)
    ok_status()
    want = key.sort(dim=1, descending=True, stable=True).indices[:, :budget].sort(dim=1).values
    assert torch.equal(kept.long(), want) and n.tolist() == [budget * block]


@pytest.mark.parametrize("kind", ["tail", "ties", "zeros", "special"])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: "x".join(map(str, c[:6])))
def test_evict_matches_the_oracle(cuda_device, case, kind):
    B, T, block, budget, first, last, lengths = case
    g = np.random.default_rng(T + budget)
    if kind == "tail":
        m = inputs.accounts(400 + T, B, T)
    elif kind == "ties":
        m = g.integers(0, 3, size=(B, T)).astype(np.float32)
    elif kind == "zeros":
        m = np.where(g.random((B, T)) < 0.5, 0.0, -0.0).astype(np.float32)
    else:
        m = g.standard_normal((B, T)).astype(np.float32)
        hit = g.random((B, T))
        m[hit < 0.02], m[(hit >= 0.02) & (hit < 0.03)], m[(hit >= 0.03) & (hit < 0.04)] = np.inf, -np.inf, np.nan
        m[(hit >= 0.04) & (hit < 0.05)] = 3e38
    kept, n = evict(f32_to_device(m), case)
    want, want_n = oracle.evict(m, lengths, block, budget, first, last)
    assert np.array_equal(kept, want) and np.array_equal(n, want_n)


def test_evict_sums_decide_in_64_bits(cuda_device):
    # a block whose float32 sum in order would lose the small values: 2^24 + 64 x 1 against 2^24 + 63
    m = np.zeros((1, 4 * 128), np.float32)
    m[0, 0], m[0, 1:65] = 2.0 ** 24, 1.0
    m[0, 128], m[0, 129] = 2.0 ** 24, 62.0
    m[0, 256], m[0, 257] = 2.0 ** 24, 66.0
    kept, _ = evict(f32_to_device(m), (1, 512, 128, 2, 0, 0, None))
    assert list(kept[0]) == [0, 2]


def test_evict_strided_accounts_and_given_outputs(cuda_device):
    m = inputs.accounts(9, 3, 64)
    big = f32_to_device(np.concatenate([m, np.full((3, 9), 1e9, np.float32)], 1))
    case = (3, 64, 4, 6, 1, 1, None)
    kept, new = torch.full((3, 6), -9, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    got = evict(big[:, :64], case, kept=kept, new_length=new)
    want = oracle.evict(m, None, 4, 6, 1, 1)
    assert np.array_equal(kept.cpu().numpy(), want[0]) and np.array_equal(new.cpu().numpy(), want[1])
    one = ds.ds_cache_evict(big[:1, :64].expand(3, 64), 6, block=4, keep_first=1)[0].cpu().numpy()
    assert all(np.array_equal(one[b], want[0][0]) for b in range(3))


def test_evict_clips_lengths(cuda_device):
    m = inputs.accounts(10, 3, 50)
    kept, new = ds.ds_cache_evict(f32_to_device(m), 3, block=4, length=i32_to_device(np.array([99, -5, 7])))
    torch.cuda.synchronize()
    assert ds.ds_get_device_status() == (ds.DS_ERR_RANGE if ds.ds_debug_build() else ds.DS_OK)
    want, n = oracle.evict(m, [50, 0, 7], 4, 3, 0, 1)
    assert np.array_equal(kept.cpu().numpy(), want) and np.array_equal(new.cpu().numpy(), n)


@pytest.mark.parametrize("case", EVICT, ids=lambda c: "x".join(map(str, c[:6])))
def test_compact_moves_every_array(cuda_device, case):
    B, T, block, budget, first, last, lengths = case
    g = np.random.default_rng(T)
    m = inputs.accounts(500 + T, B, T)
    ln = [T] * B if lengths is None else lengths
    kept, _ = oracle.evict(m, ln, block, budget, first, last)
    nb, cap = -(-T // block), min(T, budget * block)
    arrays = [(g.integers(0, 256, size=(B, T, 2, 64)).astype(np.uint8), cap, 0), (m, cap, 0),
              (g.integers(0, 256, size=(B, T, 3)).astype(np.uint8), cap, 0),
              (g.standard_normal((B, nb, 2)).astype(np.float32), budget, 1)]
    src = [torch.from_numpy(s).cuda() for s, _, _ in arrays]
    dst = [torch.full((B, c) + s.shape[2:], 77, dtype=s.dtype, device="cuda") for s, (_, c, _) in zip(src, arrays)]
    ds.ds_cache_compact(i32_to_device(kept), block=block, length=None if lengths is None else i32_to_device(np.array(ln)),
                        rows=list(zip(src[:3], dst[:3])), blocks=[(src[3], dst[3])])
    ok_status()
    for s, d, (raw, c, per_block) in zip(src, dst, arrays):
        want = oracle.compact(raw, np.full((B, c) + raw.shape[2:], 77, raw.dtype), kept, ln, block, per_block)
        assert np.array_equal(d.cpu().numpy(), want)


@pytest.mark.parametrize("block,width,budget", [(16, 256, 3000), (64, 1040, 500), (4, 4096, 2000), (1, 16, 9000)])
def test_compact_many_blocks(cuda_device, block, width, budget):
    # many more pieces than a CTA has stages, two large arrays and two small ones, a short last block
    T, B = 60_001 if block > 1 else 10_001, 2
    g = torch.Generator("cuda").manual_seed(block)
    nb = -(-T // block)
    src = [torch.randint(0, 256, (B, T, width), device="cuda", dtype=torch.uint8, generator=g),
           torch.randint(0, 2 ** 31 - 1, (B, T), device="cuda", dtype=torch.int32, generator=g),
           torch.randint(0, 256, (B, T, width // 2), device="cuda", dtype=torch.uint8, generator=g)]
    scales = torch.rand(B, nb, 3, device="cuda", generator=g)
    kept = torch.stack([torch.randperm(nb, device="cuda", generator=g)[:budget].sort().values for _ in range(B)]).int()
    kept[1, -1] = nb - 1
    m = min(T, budget * block)
    dst = [torch.zeros((B, m) + s.shape[2:], dtype=s.dtype, device="cuda") for s in src]
    to = torch.zeros(B, budget, 3, device="cuda")
    ds.ds_cache_compact(kept, block=block, rows=list(zip(src, dst)), blocks=[(scales, to)])
    ok_status()
    at = (kept.long()[:, :, None] * block + torch.arange(block, device="cuda")).view(B, -1)[:, :m]
    b = torch.arange(B, device="cuda")[:, None]
    for s, d in zip(src, dst):
        there = (at < T).view((B, m) + (1,) * (s.dim() - 2))
        assert torch.equal(d, torch.where(there, s[b, at.clamp_max(T - 1)], torch.zeros_like(d)))
    assert torch.equal(to, scales[b, kept.long()])


def test_compact_any_list_stays_inside(cuda_device):
    # lists that ds_cache_evict would not give: out of order, repeated, out of range.  Rows behind dst are not touched
    T, block = 10, 4
    src = torch.arange(10, dtype=torch.int32, device="cuda")[None].contiguous()
    back = torch.full((1, 16), -5, dtype=torch.int32, device="cuda")
    ds.ds_cache_compact(i32_to_device(np.array([[2, 9, 0]])), block=block, rows=[(src, back[:, :10])])
    torch.cuda.synchronize()
    assert ds.ds_get_device_status() == (ds.DS_ERR_RANGE if ds.ds_debug_build() else ds.DS_OK)
    assert back[0].tolist() == [8, 9, -5, -5, -5, -5, -5, -5, 0, 1] + [-5] * 6
    ds.ds_cache_compact(i32_to_device(np.array([[1, 1, -1]])), block=block, rows=[(src, back[:, :10])])
    ok_status()
    assert back[0].tolist() == [4, 5, 6, 7, 4, 5, 6, 7, 0, 1] + [-5] * 6


@pytest.mark.parametrize("block,width", [(4, 64), (64, 512)])
def test_compact_from_one_half_of_a_buffer_to_the_other(cuda_device, block, width):
    # src and dst by turns in one buffer [batch, 2, ...]: they share no byte, although their ranges of addresses meet.
    # Blocks of 256 bytes move by threads, of 32 KiB by bulk copies
    B, nb = 3, 7
    T = nb * block - 1
    g = np.random.default_rng(block)
    x = g.integers(0, 256, size=(B, 2, T, width)).astype(np.uint8)
    m = inputs.accounts(600 + block, B, T)
    kept, _ = oracle.evict(m, [T] * B, block, 4, 1, 1)
    for way in (0, 1):
        buf = torch.from_numpy(x).cuda()
        ds.ds_cache_compact(i32_to_device(kept), block=block, rows=[(buf[:, way], buf[:, 1 - way])])
        ok_status()
        want = x.copy()
        want[:, 1 - way] = oracle.compact(x[:, way], x[:, 1 - way], kept, [T] * B, block, 0)
        assert np.array_equal(buf.cpu().numpy(), want)


# ---------------------------------------------------------------- refusals of the front end

def test_front_end_refusals(cuda_device):
    B, T, K, d, H, block = 2, 32, 1, 64, 4, 8
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8, device="cuda")
    f = lambda *s: torch.zeros(*s, device="cuda")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    q, codes, scales, idx, rows = bf(B, H, d), i8(B, T, K, d), f(B, 4, K), i32(B, 5), bf(B, 8, K, d)
    wrong = [
        lambda: ds.ds_sparse_attention_q8(f(B, H, d), codes, scales, idx, block),
        lambda: ds.ds_sparse_attention_q8(q, bf(B, T, K, d), scales, idx, block),
        lambda: ds.ds_sparse_attention_q8(q, codes, None, idx, block),
        lambda: ds.ds_sparse_attention_q8(q, codes, f(B, 5, K), idx, block),
        lambda: ds.ds_sparse_attention_q8(q, codes, scales.double(), idx, block),
        lambda: ds.ds_sparse_attention_q8(q, codes[0], scales, idx, block),
        lambda: ds.ds_sparse_attention_q8(q, codes[:1], scales[:1], idx, block),
        lambda: ds.ds_sparse_attention_q8(q, codes, scales, idx.long(), block),
        lambda: ds.ds_sparse_attention_q8(q, codes, scales, idx[:1], block),
        lambda: ds.ds_sparse_attention_q8(q, codes, scales, idx.cpu(), block),
        lambda: ds.ds_sparse_attention_q8(q, codes, scales, i32(5, B).t(), block),
        lambda: ds.ds_sparse_attention_q8(q[:, :, :32], codes, scales, idx, block),
        lambda: ds.ds_sparse_attention_q8(q, i8(B, T, d, 2).transpose(2, 3), f(B, 4, 2), idx, block),
        lambda: ds.ds_sparse_attention_q8(q, codes, scales, idx, 12),
        lambda: ds.ds_sparse_attention_q8(q, codes, scales, idx, 0),
        lambda: ds.ds_sparse_attention_q8(q, codes, scales, idx, block, win=bf(B, 3, d)),
        lambda: ds.ds_sparse_attention_q8(q, codes, scales, idx, block, sink=f(H + 1)),
        lambda: ds.ds_sparse_attention_q8(q, codes, scales, idx, block, scale=float("nan")),
        lambda: ds.ds_sparse_attention_q8(q, codes, scales, idx, block, out=bf(B, H, d + 64)),
        lambda: ds.ds_sparse_attention_q8(bf(B, 3, d), i8(B, T, 2, d), f(B, 4, 2), idx, block),
        lambda: ds.ds_cache_quantize(rows, codes, scales, 3),
        lambda: ds.ds_cache_quantize(rows, codes[0], scales[0], block),
        lambda: ds.ds_cache_quantize(bf(B, 8, 2, d), codes, scales, block),
        lambda: ds.ds_cache_quantize(rows, codes, scales, block, pos=i32(3)),
        lambda: ds.ds_cache_quantize(rows, codes, scales, block, length=f(B)),
        lambda: ds.ds_cache_quantize(rows[:, :0], codes, scales, block),
        lambda: ds.ds_cache_quantize(rows, codes[:1].expand(B, T, K, d), scales, block),
        lambda: ds.ds_attention_mass(q, codes, idx, f(B, H), f(B, T), block=block),
        lambda: ds.ds_attention_mass(q, codes, idx, f(B, H + 1), f(B, T), scales=scales, block=block),
        lambda: ds.ds_attention_mass(q, codes, idx, f(B, H), f(B, T - 1), scales=scales, block=block),
        lambda: ds.ds_attention_mass(q, codes, idx, f(B, H), f(1, T).expand(B, T), scales=scales, block=block),
        lambda: ds.ds_attention_mass(q, codes, idx, f(B, H), None, scales=scales, block=block),
        lambda: ds.ds_cache_evict(f(B, T), 5, block=8),
        lambda: ds.ds_cache_evict(f(B, T), 0, block=8),
        lambda: ds.ds_cache_evict(f(B, T), 4, block=8, keep_first=3, keep_last=2),
        lambda: ds.ds_cache_evict(f(T, B).t(), 4),
        lambda: ds.ds_cache_evict(f(B, T).half(), 4),
        lambda: ds.ds_cache_compact(i32(B, 2), block=8),
        lambda: ds.ds_cache_compact(i32(B, 2), block=8, rows=[(codes, i8(B, 15, K, d))]),
        lambda: ds.ds_cache_compact(i32(B, 2), block=8, rows=[(codes, f(B, 16, K, d))]),
        lambda: ds.ds_cache_compact(i32(B, 2), block=8, rows=[(codes, codes[:, 8:24])]),
        lambda: ds.ds_cache_compact(i32(B, 2), block=8, rows=[(codes, i8(B, 16, K, d))], blocks=[(f(B, 5, K), f(B, 2, K))]),
        lambda: ds.ds_cache_compact(i32(B, 2), block=8, rows=[(codes, i8(B, 16, K, d))] * 9),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises((ValueError, TypeError, ds.DsError)):
            call()
            pytest.fail(f"call {i} was not refused")
    ok_status()


def test_quantize_says_which_strides_it_takes(cuda_device):
    codes, scales = torch.zeros(2, 8, 1, 64, dtype=torch.int8, device="cuda"), torch.zeros(2, 2, 1, device="cuda")
    wide = torch.zeros(2, 8, 1, 100, dtype=torch.bfloat16, device="cuda")
    odd = torch.zeros(2 * 600, dtype=torch.bfloat16, device="cuda").as_strided((2, 8, 1, 64), (516, 64, 64, 1))
    for rows in (wide[..., :64],                                            # a row stride of 100
                 odd,                                                       # a batch stride of 516
                 wide[:, :1, :, :64].expand(2, 8, 1, 64),                   # one row eight times
                 torch.zeros(900, dtype=torch.bfloat16, device="cuda").as_strided((2, 8, 1, 64), (512, 32, 64, 1))):
        with pytest.raises(ValueError, match="strides must be multiples of 8"):
            ds.ds_cache_quantize(rows, codes, scales, 4)
    ok_status()


# ---------------------------------------------------------------- together, as they would be used

def serve(q, rows, win, sink, block, budget, fmt, steps):
    """Prompt rows written, then decode steps: select, attend, account; then evict, compact and attend again."""
    B, n, K, d = rows.shape
    nb = -(-n // block)
    codes, scales = torch.zeros(B, n, K, d, dtype=TORCH[fmt], device="cuda"), torch.zeros(B, nb, K, device="cuda")
    mass = torch.zeros(B, n, device="cuda")
    ds.ds_cache_quantize(rows, codes, scales, block)
    outs = []
    for s in range(steps):
        score = torch.matmul(rows[:, :, 0].float(), q[s][:, 0, :, None].float())[..., 0].contiguous()
        idx, _ = ds.ds_topk(score, 48, return_value=False, sorted_index=True)
        out, lse = ds.ds_sparse_attention_q8(q[s], codes, scales, idx, block, win=win, sink=sink, return_lse=True)
        ds.ds_attention_mass(q[s], codes, idx, lse, mass, scales=scales, block=block)
        outs += [out, lse]
    kept, length = ds.ds_cache_evict(mass, budget, block=block, keep_first=1, keep_last=1)
    m = min(n, budget * block)
    to = torch.zeros(B, m, K, d, dtype=TORCH[fmt], device="cuda"), torch.zeros(B, budget, K, device="cuda"), torch.zeros(B, m, device="cuda")
    ds.ds_cache_compact(kept, block=block, rows=[(codes, to[0]), (mass, to[2])], blocks=[(scales, to[1])])
    # attend over everything that stays
    r = torch.arange(m, dtype=torch.int32, device="cuda")
    idx = torch.where(r < length[:, None], r, -1).to(torch.int32)
    out, lse = ds.ds_sparse_attention_q8(q[0], to[0], to[1], idx, block, win=win, sink=sink, return_lse=True)
    return outs + [mass, kept, length, *to, out, lse]


def serve_inputs(seed, fmt="e4m3"):
    g = inputs.rng(seed)
    B, n, K, d, H = 2, 150, 2, 128, 8
    q = [bf16_to_device(inputs.f32_to_bf16_bits(g.standard_normal((B, H, d)))) for _ in range(3)]
    return q, bf16_to_device(inputs.cache_rows(seed, B, n, K, d)), bf16_to_device(inputs.cache_rows(seed + 1, B, 6, K, d)), \
        f32_to_device(g.standard_normal(H).astype(np.float32)), 16, 4, fmt, 3


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_a_run_of_all_of_them(cuda_device, fmt):
    a = serve_inputs(20, fmt)
    r = serve(*a)
    ok_status()
    q, rows, win, sink, block, budget, _, steps = a
    mass, kept, length, codes, scales, moved, out, lse = r[2 * steps:]
    want, wscales = quantized(bits_of(rows), block, fmt)
    # the window and the sink take their shares: an account holds the rest of one softmax per head and step
    total = mass.cpu().numpy().sum(1, dtype=np.float64)
    assert np.all(total < 8 * steps) and np.all(total > 8)
    m = mass.cpu().numpy()
    wkept, wlen = oracle.evict(m, None, block, budget, 1, 1)
    assert np.array_equal(kept.cpu().numpy(), wkept) and np.array_equal(length.cpu().numpy(), wlen)
    zero = np.zeros(tuple(codes.shape), np.uint8)
    wc, ws = oracle.compact(want, zero, wkept, [150, 150], block, 0), oracle.compact(wscales, np.zeros(tuple(scales.shape), np.float32), wkept, [150, 150], block, 1)
    assert np.array_equal(codes_of(codes), wc) and np.array_equal(scales.cpu().numpy(), ws)
    assert np.array_equal(moved.cpu().numpy(), oracle.compact(m, np.zeros(tuple(moved.shape), np.float32), wkept, [150, 150], block, 0))
    idx = np.where(np.arange(64) < wlen[:, None], np.arange(64), -1).astype(np.int32)
    x = dict(q=bits_of(q[0]), codes=wc, scales=ws, idx=idx, win=bits_of(win), win_len=None, sink=sink.cpu().numpy(), scale=1 / math.sqrt(128))
    check_attention((2, 8, 2, 128, 64, 64, 6, block, fmt, False), x, out, lse)


def test_two_runs_give_the_same_bits(cuda_device):
    a = serve_inputs(21)
    for x, y in zip(serve(*a), serve(*a)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_runs_on_two_streams_at_once(cuda_device):
    a, b = serve_inputs(22), serve_inputs(23)
    want = [serve(*a), serve(*b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s, x in zip(streams, (a, b)):
        with torch.cuda.stream(s):
            got.append([serve(*x) for _ in range(3)])
    ok_status()
    for rounds, w in zip(got, want):
        for r in rounds:
            assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(r, w))


def test_a_stream_argument_other_than_the_current_one(cuda_device):
    a = attend_inputs(ATTEND[4])
    (out, lse), t = attend(ATTEND[4], a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, l2 = ds.ds_sparse_attention_q8(t["q"], t["codes"], t["scales"], t["idx"], 32, win=t["win"], win_len=t["win_len"], sink=t["sink"],
                                       return_lse=True, stream=s)
    kept, _ = ds.ds_cache_evict(f32_to_device(inputs.accounts(1, 2, 50)), 7, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    ds.ds_get_device_status()
    assert torch.equal(out, o2) and torch.equal(lse, l2) and kept.shape == (2, 7)


def test_both_ways_of_marshalling_agree(cuda_device, monkeypatch):
    # the extension takes these calls, and the binding's own marshalling gives the same bits
    from sparse_attention_top_ds_b200 import _native
    a = serve_inputs(26)
    taken = {}

    class Spy:
        def __getattr__(self, name):
            def call(*args):
                r = getattr(front, name)(*args)
                taken.setdefault(name, []).append(r is not None)
                return r
            return call

    front = _native._front or _native._load_front()
    monkeypatch.setattr(_native, "_front", Spy())
    by_front = serve(*a)
    assert {k: all(v) for k, v in taken.items()} == dict.fromkeys(("quantize", "attention", "mass", "evict", "compact"), True)

    class Off:
        def __getattr__(self, name):
            return lambda *args: None

    monkeypatch.setattr(_native, "_front", Off())
    for x, y in zip(by_front, serve(*a)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    test_front_end_refusals(cuda_device)


def test_captured_runs_replay_on_new_inputs_side_by_side(cuda_device):
    # two graphs of the whole run, replayed at once on two streams with inputs changed in place
    a, b = serve_inputs(24), serve_inputs(25)
    want_a, want_b = serve(*b), serve(*a)
    graphs = []
    for x in (a, b):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            serve(*x)
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                r = serve(*x)
        graphs.append((g, s, r))
    torch.cuda.synchronize()
    for x, y in zip([*a[0], *a[1:4]], [*b[0], *b[1:4]]):  # swap the two runs' inputs
        z = x.clone()
        x.copy_(y)
        y.copy_(z)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
    ok_status()
    for (_, _, r), w in zip(graphs, (want_a, want_b)):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(r, w))


@pytest.mark.parametrize("case", [(200, 64, 1, 256, 400, 150, 0, 16, "e4m3", True, False, 0.0, None),
                                  (200, 64, 1, 256, 400, 150, 0, 16, "int8", True, False, 0.0, None),
                                  (160, 20, 1, 448, 600, 300, 130, 4, "int8", True, True, 0.1, None),
                                  (300, 40, 2, 64, 700, 513, 3, 1, "e4m3", True, False, 0.3, None),
                                  (150, 128, 1, 512, 900, 400, 65, 64, "e4m3", True, True, 0.0, None),
                                  (33, 33, 1, 384, 300, 257, 0, 8, "int8", True, True, 0.0, None)],
                         ids=lambda c: "x".join(map(str, c[:10])))
def test_attention_on_many_batch_rows(cuda_device, case):
    # as many batch rows as fill the GPU, so that a CTA passes through all chunks of its rows: the first and last of them
    a = attend_inputs(case)
    (out, lse), t = attend(case, a)
    ok_status(skipped=case[11] > 0)
    for s in (slice(0, 2), slice(case[0] - 2, case[0])):
        few = dict(a, q=a["q"][s], idx=a["idx"][s], win=None if a["win"] is None else a["win"][s])
        check_attention((2,) + case[1:], few, out[s], lse[s])
