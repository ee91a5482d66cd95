"""The C entry points of the 8-bit cache answer bad arguments on the host, and the
Python front end refuses tensors that are not on a GPU (CPU only)."""

import ctypes
import struct

import pytest
import torch

import sparse_attention_top_ds_b200 as ds
from sparse_attention_top_ds_b200 import _native

A = ctypes.c_void_p(0x100000)


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_top_ds_b200 import build
    build.build()
    return ds.load()


def odd(n):
    return ctypes.c_void_p(0x100000 + n)


def test_quantize_arguments(lib):
    def call(rows=A, bs=0, rs=512, batch=2, n=10, heads=1, d=512, dtype=2, block=16, pos=None, length=None, codes=A, cs=100,
             scales=A, ss=7, T=100):
        return lib.ds_cache_quantize(rows, bs, rs, batch, n, heads, d, dtype, block, pos, length, codes, cs, scales, ss, T, None)

    for bad in (dict(rows=None), dict(codes=None), dict(scales=None), dict(batch=0), dict(batch=65536), dict(n=0), dict(T=0),
                dict(heads=0), dict(heads=4097, rs=4097 * 512), dict(d=0), dict(d=100), dict(d=576), dict(dtype=0), dict(dtype=1),
                dict(dtype=4), dict(block=0), dict(block=3), dict(block=256), dict(block=-1), dict(rs=511), dict(rs=516),
                dict(bs=-8), dict(bs=4), dict(cs=99), dict(ss=6), dict(rows=odd(8)), dict(codes=odd(4)), dict(scales=odd(2)),
                dict(pos=odd(1)), dict(length=odd(2)), dict(batch=65535, n=2 ** 31 - 1, block=1)):
        assert call(**bad) == ds.DS_ERR_ARG, bad


def test_attention_arguments(lib):
    def call(q=A, codes=A, cs=0, scales=A, ss=0, dtype=2, block=16, T=100, idx=A, k=10, win=None, W=0, wl=None, sink=None, batch=2,
             heads=128, kv=1, d=512, scale=0.04, out=A, lse=None):
        return lib.ds_sparse_attention_q8(q, codes, cs, scales, ss, dtype, block, T, idx, k, win, W, wl, sink, batch, heads, kv, d,
                                          scale, out, lse, None)

    for bad in (dict(q=None), dict(codes=None), dict(scales=None), dict(out=None), dict(cs=-1), dict(ss=-1), dict(dtype=1),
                dict(dtype=1, scales=None), dict(dtype=0), dict(block=0), dict(block=12), dict(block=256), dict(T=0), dict(idx=None),
                dict(k=-1), dict(k=2049), dict(W=-1), dict(W=8), dict(W=4097, win=A), dict(batch=0), dict(batch=65536), dict(heads=0),
                dict(heads=4097), dict(kv=0), dict(kv=3), dict(kv=256), dict(d=32), dict(d=100), dict(d=576),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(q=odd(8)), dict(codes=odd(8)), dict(scales=odd(1)),
                dict(idx=odd(2)), dict(win=odd(8), W=4), dict(wl=odd(2)), dict(sink=odd(2)), dict(out=odd(8)), dict(lse=odd(2))):
        assert call(**bad) == ds.DS_ERR_ARG, bad


def test_mass_arguments(lib):
    def call(q=A, cache=A, cs=0, scales=A, ss=0, dtype=2, block=16, T=100, idx=A, k=10, lse=A, batch=2, heads=128, kv=1, d=512,
             scale=0.04, mass=A, ms=100):
        return lib.ds_attention_mass(q, cache, cs, scales, ss, dtype, block, T, idx, k, lse, batch, heads, kv, d, scale, mass, ms,
                                     None)

    for bad in (dict(lse=None), dict(mass=None), dict(ms=99), dict(ms=0), dict(lse=odd(2)), dict(mass=odd(1)), dict(q=None),
                dict(cache=None), dict(scales=None), dict(dtype=1), dict(dtype=0, scales=None), dict(block=5), dict(k=2049),
                dict(idx=None), dict(kv=7), dict(d=72), dict(T=0), dict(batch=0), dict(cs=-1), dict(scale=float("inf"))):
        assert call(**bad) == ds.DS_ERR_ARG, bad


def test_evict_arguments(lib):
    def call(mass=A, ms=100, batch=2, T=100, length=None, block=16, budget=4, first=1, last=1, kept=A, new_len=A):
        return lib.ds_cache_evict(mass, ms, batch, T, length, block, budget, first, last, kept, new_len, None)

    for bad in (dict(mass=None), dict(kept=None), dict(new_len=None), dict(ms=-1), dict(batch=0), dict(batch=65536), dict(T=0),
                dict(T=(1 << 24) + 1), dict(block=0), dict(block=24), dict(block=256), dict(budget=0), dict(budget=8),
                dict(first=-1), dict(last=-1), dict(first=5, last=0), dict(first=2, last=3), dict(first=2 ** 31 - 1, last=2 ** 31 - 1),
                dict(mass=odd(2)), dict(length=odd(2)), dict(kept=odd(1)), dict(new_len=odd(2))):
        assert call(**bad) == ds.DS_ERR_ARG, bad


def test_compact_arguments(lib):
    def call(n=1, kept=A, budget=4, length=None, batch=2, T=100, block=16, arrays=True, **a):
        f = dict(src=0x100000, dst=0x900000, src_batch_stride=102400, dst_batch_stride=65536, item_bytes=1024, per_block=0)
        f.update(a)
        arr = struct.pack(_native._CACHE_ARRAY, *(f[i] or 0 for i in f)) * max(1, min(n, 9))
        return lib.ds_cache_compact(arr if arrays else None, n, kept, budget, length, batch, T, block, None)

    for bad in (dict(arrays=False), dict(n=0), dict(n=9), dict(kept=None), dict(budget=0), dict(budget=8), dict(batch=0),
                dict(batch=65536), dict(T=0), dict(T=(1 << 24) + 1), dict(block=3), dict(kept=odd(2)), dict(length=odd(1)),
                dict(src=None), dict(dst=None), dict(item_bytes=0), dict(item_bytes=(1 << 24) + 1), dict(per_block=2),
                dict(src_batch_stride=102399), dict(dst_batch_stride=65535),
                dict(dst=0x100000), dict(dst=0x100000 + 102400 + 102399), dict(src=0x900000 + 65536 + 65535)):  # overlaps
        assert call(**bad) == ds.DS_ERR_ARG, bad


def test_compact_refuses_an_array_written_where_another_is_read(lib):
    def call(*arrays):
        arr = b"".join(struct.pack(_native._CACHE_ARRAY, src, dst, 102400, 65536, 1024, 0) for src, dst in arrays)
        return lib.ds_cache_compact(arr, len(arrays), A, 4, None, 2, 100, 16, None)

    first = (0x100000, 0x900000)
    for second in ((0x900000, 0x1100000), (0x900000 + 65536 + 65535, 0x1100000), (0x1100000, 0x100000),
                   (0x1100000, 0x100000 + 204799)):
        assert call(first, second) == call(second, first) == ds.DS_ERR_ARG, second


def compact_two_rows(lib, src, dst, src_step, dst_step, batch=2):
    """Two batch rows (or more) of 100 items of 1024 bytes, 4 blocks of 16 kept."""
    arr = struct.pack(_native._CACHE_ARRAY, src, dst, src_step, dst_step, 1024, 0)
    return lib.ds_cache_compact(arr, 1, A, 4, None, batch, 100, 16, None)


SRC, DST = 100 * 1024, 64 * 1024  # bytes of a batch row that are read, and written


@pytest.mark.skipif(torch.cuda.is_available(), reason="an accepted call would run on addresses that are none")
@pytest.mark.parametrize("at,src_step,dst_step", [
    (SRC, 2 * SRC, 2 * SRC),                 # two halves of a buffer [batch, 2, ...]
    (-DST, SRC + DST, SRC + DST),            # dst in front of src in each batch row
    (SRC, SRC + DST, SRC + DST),             # no byte between them
    (SRC + 16, 5 * SRC, 3 * SRC),            # different strides that never meet
    (3 * SRC, 2 * SRC, 2 * SRC),             # dst of batch row 0 behind src of batch row 1
])
def test_compact_takes_a_dst_in_the_gaps_of_a_src(lib, at, src_step, dst_step):
    # without a GPU, a call whose arguments are accepted ends at the device
    assert compact_two_rows(lib, 0x4000000, 0x4000000 + at, src_step, dst_step) not in (ds.DS_ERR_ARG, ds.DS_OK)


@pytest.mark.parametrize("at,src_step,dst_step,batch", [
    (SRC - 1024, 2 * SRC, 2 * SRC, 2),       # two halves, dst one item early
    (2 * SRC - DST + 1024, 2 * SRC, 2 * SRC, 2),  # and so late that it reaches the next batch row
    (SRC, SRC + DST - 16, SRC + DST - 16, 2),
    (SRC, 4 * SRC, 3 * SRC, 3),              # meets in the last batch row only
    (-DST, 2 * SRC, SRC, 2),                 # dst of batch row 1 within src of batch row 0
])
def test_compact_refuses_a_dst_that_meets_a_src_in_some_batch_row(lib, at, src_step, dst_step, batch):
    assert compact_two_rows(lib, 0x4000000, 0x4000000 + at, src_step, dst_step, batch) == ds.DS_ERR_ARG


def compact_two_arrays(lib, a, b, batch=2):
    """Arrays (src, dst, their batch strides, bytes of an item, per_block) of 100 rows in blocks of 16, 4 of them kept."""
    arr = struct.pack(_native._CACHE_ARRAY * 2, *a, *b)
    return lib.ds_cache_compact(arr, 2, A, 4, None, batch, 100, 16, None)


@pytest.mark.parametrize("dst,step,item,per_block", [
    (0x8000000, 2 * DST, 1024, 0),           # the same
    (0x8000000 + DST - 1024, 2 * DST, 1024, 0),
    (0x8000000 - 4 + 1, 4, 1, 1),            # four bytes a batch row, of the first array's only the first
    (0x8000000 + 3 * DST - 1, DST, 1, 1),    # of its batch row 1 only
])
def test_compact_refuses_two_arrays_written_to_one_place(lib, dst, step, item, per_block):
    first = (0x4000000, 0x8000000, SRC, 2 * DST, 1024, 0)
    second = (0x1000000, dst, SRC, step, item, per_block)
    assert compact_two_arrays(lib, first, second) == compact_two_arrays(lib, second, first) == ds.DS_ERR_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="an accepted call would run on addresses that are none")
def test_compact_takes_two_arrays_written_side_by_side(lib):
    first = (0x4000000, 0x8000000, SRC, 2 * DST, 1024, 0)
    for second in ((0x1000000, 0x8000000 + DST, SRC, 2 * DST, 1024, 0), (0x1000000, 0x8000000 + 3 * DST, SRC, 4, 1, 1),
                   (0x4000000, 0x9000000, SRC, DST, 1024, 0)):  # one array, to two places
        for arrays in ((first, second), (second, first)):
            assert compact_two_arrays(lib, *arrays) not in (ds.DS_ERR_ARG, ds.DS_OK), second


def test_build_makes_the_front_extension(lib):
    from sparse_attention_top_ds_b200 import build
    assert not build.front_stale()
    front = _native._load_front()
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: front.quantize(q, q, q, 1, None, None), lambda: front.attention(q, q, q, q, 1, None, None, None, None, True),
                 lambda: front.mass(q, q, q, q, q, None, 1, None), lambda: front.evict(q, 1, 1, None, 0, 1),
                 lambda: front.compact(q, 1, None, [], []), lambda: front.quantize(), lambda: front.attention(None, 1, "x"),
                 lambda: front.evict(3, "x", None, q, -1, 2 ** 70)):
        assert call() is None            # nothing that is not the usual call is taken
    with pytest.raises(TypeError):
        front.bind(1, 2)


def test_front_end_refuses_tensors_off_the_gpu():
    x = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    codes, scales = torch.zeros(2, 8, 1, 64, dtype=torch.int8), torch.zeros(2, 8, 1)
    q, idx, lse = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 4)
    for f in (lambda: ds.ds_cache_quantize(x, codes, scales, 1), lambda: ds.ds_sparse_attention_q8(q, codes, scales, idx, 1),
              lambda: ds.ds_attention_mass(q, codes, idx, lse, torch.zeros(2, 8), scales=scales),
              lambda: ds.ds_cache_evict(torch.zeros(2, 8), 4), lambda: ds.ds_cache_compact(idx)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        ds.ds_cache_evict(None, 4)
