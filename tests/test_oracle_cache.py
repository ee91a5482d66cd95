"""Pins for the oracle of the 8-bit cache (CPU only): the formats against a
library's decoding and hand-worked codes, the attention against the 16-bit
attention's oracle on rows that 8 bits hold exactly, the account against the
softmax's weights, the eviction against hand-worked lists."""

import math

import numpy as np
import pytest
import torch

from oracle import cache, sparse_attention
from sparse_attention_top_ds_b200 import inputs


def bf16(a):
    return inputs.f32_to_bf16_bits(np.asarray(a, dtype=np.float32))


def test_e4m3_decoding_matches_a_library():
    lib = torch.arange(256, dtype=torch.int64).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(lib), np.isnan(cache.E4M3))
    ok = ~np.isnan(lib)
    assert np.array_equal(lib[ok], cache.E4M3[ok])
    assert np.array_equal(np.signbit(lib[ok]), np.signbit(cache.E4M3[ok]))


def test_e4m3_rounding_scalar_array_and_library_agree():
    g = np.random.default_rng(1)
    v = np.concatenate([g.uniform(-448, 448, 500), g.standard_normal(500), g.standard_normal(500) * 2.0 ** -8,
                        (cache.E4M3[:126] + cache.E4M3[1:127]) / 2, -(cache.E4M3[:126] + cache.E4M3[1:127]) / 2, [0.0, -0.0]])
    v = v.astype(np.float32)
    arr = cache.round_e4m3(v)
    assert np.array_equal(arr, np.array([cache.nearest_e4m3(t) for t in v], dtype=np.uint8))
    assert np.array_equal(arr, torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_quantized_block_by_hand():
    codes, s = cache.quantize_block(np.array([[127.0, -127.0, 1.0, 0.5, -0.5, 1.5, 2.5, 0.0]]), "int8")
    assert s == 1.0 and list(codes.view(np.int8)[0]) == [127, -127, 1, 0, 0, 2, 2, 0]
    codes, s = cache.quantize_block(np.array([[448.0, -1.0, 17.0, 19.0, 0.0]]), "e4m3")
    assert s == 1.0 and list(cache.decode(codes, "e4m3")[0]) == [448.0, -1.0, 16.0, 20.0, 0.0]


@pytest.mark.parametrize("fmt,half", [("e4m3", 2.0 ** -4), ("int8", None)])
def test_quantization_error_is_half_a_step(fmt, half):
    x = inputs.bf16_bits_to_f32(inputs.cache_rows(3, 1, 16, 1, 64))[0, :, 0].astype(np.float64)
    codes, s = cache.quantize_block(x, fmt)
    y = cache.decode(codes, fmt) * float(s)
    top = np.abs(x).max()
    # e4m3: half a step is 2^-4 of the value, and half a subnormal step 2^-10 scales below 2^-6 scales;
    # int8: half a scale; the float32 quotients and product add 2^-22
    bound = np.maximum(half * np.abs(x), 2.0 ** -10 * float(s)) if half else 0.5 * top / 127
    assert np.all(np.abs(y - x) <= bound + 2.0 ** -22 * top)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_blocks_of_zeros_tiny_and_not_finite_values(fmt):
    codes, s = cache.quantize_block(np.zeros((2, 64)), fmt)
    assert not codes.any() and 0.0 < s < 2.0 ** -100
    codes, s = cache.quantize_block(np.full((1, 64), 1e-40), fmt)
    assert not codes.any() and np.isfinite(s)
    for bad in (np.inf, -np.inf, np.nan):
        x = np.ones((2, 64))
        x[1, 3] = bad
        codes, s = cache.quantize_block(x, fmt)
        assert not codes.any() and np.isnan(s)


def test_attention_equals_the_16_bit_one_on_rows_that_8_bits_hold():
    g = np.random.default_rng(5)
    B, H, d, T, k, W, block = 3, 4, 8, 20, 7, 3, 4
    ints = g.integers(-20, 21, size=(B, T, 1, d)).astype(np.int8)
    scales = (2.0 ** g.integers(-4, 2, size=(B, 5, 1))).astype(np.float32)
    rows = ints.astype(np.float32) * np.repeat(scales, block, axis=1)[..., None]
    q, win = bf16(g.standard_normal((B, H, d))), bf16(g.standard_normal((B, W, 1, d)))
    idx, sink = inputs.cache_slots(6, B, T, k, holes=0.3), g.standard_normal(H).astype(np.float32)
    wl = np.array([0, 2, 3], dtype=np.int32)
    out, lse, spread, reach = cache.attention_q8(q, ints.view(np.uint8), scales, idx, block, "int8", 0.3, win=win, win_len=wl, sink=sink)
    ref, ref_lse = sparse_attention(q, bf16(rows[:, :, 0]), idx, 0.3, win=win[:, :, 0], win_len=wl, sink=sink)
    assert np.allclose(out, ref, rtol=0, atol=1e-12) and np.allclose(lse, ref_lse, rtol=0, atol=1e-12)
    assert np.all(np.abs(out) <= spread + 1e-12)
    assert np.all(reach >= 0)


def test_attention_heads_read_their_own_kv_head():
    g = np.random.default_rng(7)
    B, H, K, d, T = 2, 6, 3, 8, 9
    codes = g.integers(0, 256, size=(B, T, K, d)).astype(np.uint8)
    codes[(codes & 127) == 127] = 0
    scales = g.uniform(0.01, 0.02, size=(B, T, K)).astype(np.float32)
    q, idx = bf16(g.standard_normal((B, H, d))), inputs.cache_slots(8, B, T, 5)
    out, lse, _, _ = cache.attention_q8(q, codes, scales, idx, 1, "e4m3", 0.1)
    for n in range(K):
        one, one_lse, _, _ = cache.attention_q8(q[:, 2 * n:2 * n + 2], codes[:, :, n:n + 1], scales[:, :, n:n + 1], idx, 1, "e4m3", 0.1)
        assert np.array_equal(out[:, 2 * n:2 * n + 2], one) and np.array_equal(lse[:, 2 * n:2 * n + 2], one_lse)


def test_masses_of_a_softmax_sum_to_the_heads():
    g = np.random.default_rng(9)
    B, H, d, T, k = 2, 5, 8, 30, 11
    rows = inputs.cache_rows(10, B, T, 1, d)
    q, idx = bf16(g.standard_normal((B, H, d))), inputs.cache_slots(11, B, T, k)
    out, lse, _, _ = cache.attention_q8(q, rows, None, idx, 1, "bf16", 0.3)
    total, added, _ = cache.attention_mass(q, rows, None, idx, 1, "bf16", 0.3, lse, np.ones((B, T), dtype=np.float32))
    assert np.allclose(added.sum(1), H, rtol=1e-12) and np.allclose(total, added + 1.0)
    assert all(added[b, r] == 0.0 for b in range(B) for r in range(T) if r not in idx[b])


def test_evicted_blocks_by_hand():
    m = np.array([[5, 1, 2, 2, 9, 0, 3, 3, 1, 1, 7]], dtype=np.float32)       # blocks of 2: 6 4 9 6 2 (7)
    kept, n = cache.evict(m, None, 2, 3, 0, 0)
    assert list(kept[0]) == [0, 2, 5] and n[0] == 5                           # 9, 7, then 6 at the lower block
    kept, n = cache.evict(m, None, 2, 3, 0, 1)
    assert list(kept[0]) == [0, 2, 5] and n[0] == 5
    kept, n = cache.evict(m, None, 2, 3, 2, 1)
    assert list(kept[0]) == [0, 1, 5] and n[0] == 5
    kept, n = cache.evict(m, np.array([7], dtype=np.int32), 2, 3, 0, 0)       # 6 4 9 (3)
    assert list(kept[0]) == [0, 1, 2] and n[0] == 6
    kept, n = cache.evict(m, np.array([3], dtype=np.int32), 2, 3, 0, 0)       # fewer blocks than the budget
    assert list(kept[0]) == [0, 1, -1] and n[0] == 3
    kept, n = cache.evict(m, np.array([0], dtype=np.int32), 2, 3, 1, 1)
    assert list(kept[0]) == [-1, -1, -1] and n[0] == 0
    nan = np.array([[1, np.inf, np.nan, 2, -0.0, 0.0]], dtype=np.float32)
    assert list(cache.evict(nan, None, 1, 2, 0, 0)[0][0]) == [1, 2]
    assert list(cache.evict(nan, None, 1, 5, 0, 0)[0][0]) == [0, 1, 2, 3, 4]  # -0.0 and 0.0 are equal: the lower one


def test_compaction_by_hand():
    src = np.arange(11, dtype=np.int32)[None]
    dst = np.full((1, 7), -5, dtype=np.int32)
    kept = np.array([[0, 2, 5]], dtype=np.int32)
    assert list(cache.compact(src, dst, kept, [11], 2, False)[0]) == [0, 1, 4, 5, 10, -5, -5]
    assert list(cache.compact(src[:, :6], dst, kept, [11], 2, True)[0]) == [0, 2, 5, -5, -5, -5, -5]
