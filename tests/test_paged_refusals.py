"""Refusals of the paged cache's calls: every bad argument is an error before anything is launched (no GPU)."""
import ctypes

import pytest
import torch

from top_cache_gb300 import kvo as K

A = 1 << 20  # an aligned address that no refused call may touch


@pytest.fixture(scope="module")
def L():
    from top_cache_gb300 import build
    build.build()
    return K.lib()


PLAN = dict(lengths=A, new_tokens=A, n_requests=4, block_tokens=16, max_blocks=8, window=0, sinks=0, block_table=A, ring=A,
            ring_size=8, ring_in=A, ring_out=A, lengths_out=A, kv_lens=A, cu_new=A, slots=A, n_slots=4, status=A, stream=None)
ROWS = dict(rows=A, slots=A, n_rows=4, pool=A, n_blocks=4, block_tokens=16, format=0, stream=None)
ATTEND = dict(pool=A, n_blocks=4, block_tokens=16, format=0, block_table=A, max_blocks=8, kv_lens=A, cu_tokens=A, n_requests=2,
              queries=A, n_tokens=2, n_heads=16, scale=0.1, window=0, sinks=0, out=A, lse=A, workspace=A,
              workspace_bytes=1 << 40, status=A, stream=None)

SHAPES = [dict(block_tokens=0), dict(block_tokens=12), dict(block_tokens=65544), dict(block_tokens=-8)]
CACHE = SHAPES + [dict(format=2), dict(format=-1), dict(n_blocks=0), dict(n_blocks=1 << 27), dict(pool=None), dict(pool=A + 8)]


@pytest.mark.parametrize("over", SHAPES + [dict([(k, None)]) for k in (
    "lengths", "new_tokens", "block_table", "ring", "ring_in", "ring_out", "lengths_out", "kv_lens", "cu_new", "slots", "status")] + [
    dict(n_requests=0), dict(n_requests=4097), dict(max_blocks=0), dict(max_blocks=1 << 27), dict(ring_size=0), dict(n_slots=-1),
    dict(window=-1), dict(sinks=-1), dict(ring_in=A + 4), dict(ring_out=A + 4), dict(lengths=A + 2), dict(slots=A + 1)])
def test_plan(L, over):
    assert L.kvo_paged_plan(*{**PLAN, **over}.values()) == K.KVO_EINVAL
    assert L.kvo_last_error()


@pytest.mark.parametrize("over", CACHE + [dict(rows=None), dict(slots=None), dict(n_rows=-1), dict(n_rows=1 << 31),
                                          dict(rows=A + 2), dict(slots=A + 2)])
def test_rows(L, over):
    a = {**ROWS, **over}
    assert L.kvo_paged_write(*a.values()) == K.KVO_EINVAL
    assert L.kvo_paged_read(a["pool"], a["n_blocks"], a["block_tokens"], a["format"], a["slots"], a["n_rows"], a["rows"],
                            None) == K.KVO_EINVAL


@pytest.mark.parametrize("over", CACHE + [dict([(k, None)]) for k in ("block_table", "kv_lens", "cu_tokens", "queries", "out",
                                                                      "workspace")] + [
    dict(n_requests=0), dict(n_requests=4097), dict(max_blocks=0), dict(max_blocks=1 << 27), dict(n_heads=0), dict(n_heads=8193),
    dict(n_tokens=-1), dict(n_tokens=1 << 26), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1),
    dict(sinks=-1), dict(queries=A + 8), dict(out=A + 2), dict(lse=A + 2), dict(workspace=A + 128), dict(cu_tokens=A + 1)])
def test_attend(L, over):
    a = {**ATTEND, **over}
    a["scale"] = ctypes.c_float(a["scale"])
    assert L.kvo_paged_attend(*a.values()) == K.KVO_EINVAL


def test_sizes(L):
    for b in (8, 24, 64, 65536):
        assert L.kvo_paged_block_bytes(K.KVO_CACHE_BF16, b) == K.kvo_paged_block_bytes(K.KVO_CACHE_BF16, b) == b * 1152
        assert L.kvo_paged_block_bytes(K.KVO_CACHE_Q4, b) == K.kvo_paged_block_bytes(K.KVO_CACHE_Q4, b) == b * 324
    for fmt, b in ((2, 64), (0, 0), (0, 4), (1, 65544)):
        assert L.kvo_paged_block_bytes(fmt, b) == 0
    for r, t, h in ((0, 1, 16), (4097, 1, 16), (1, -1, 16), (1, 1, 0), (1, 1, 8193)):
        assert L.kvo_paged_attend_workspace_size(r, t, h, 0) == 0


def test_binding_refuses_host_tensors():
    i, x = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 576, dtype=torch.bfloat16)
    two = torch.zeros(2, dtype=torch.int64)
    pool = torch.zeros(4, 324 * 16, dtype=torch.uint8)
    calls = [lambda: K.kvo_paged_plan(i, i, 16, i.view(4, 1), i, two, two, i, i, torch.zeros(5, dtype=torch.int32), i, i),
             lambda: K.kvo_paged_write(x, i, pool, 4, 16, K.KVO_CACHE_Q4),
             lambda: K.kvo_paged_read(pool, 4, 16, K.KVO_CACHE_Q4, i, x),
             lambda: K.kvo_paged_attend(pool, 4, 16, K.KVO_CACHE_Q4, i.view(4, 1), i, torch.zeros(5, dtype=torch.int32),
                                        torch.zeros(4, 2, 576, dtype=torch.bfloat16), 0.1,
                                        torch.zeros(4, 2, 512, dtype=torch.bfloat16))]
    for call in calls:
        with pytest.raises(K.KvoError) as e:
            call()
        assert e.value.code == K.KVO_EINVAL
    with pytest.raises(K.KvoError):
        K.kvo_paged_block_bytes(7, 16)


@pytest.mark.parametrize("block", [8, 24, 40, 65528, 65536])
@pytest.mark.parametrize("fmt", [K.KVO_CACHE_BF16, K.KVO_CACHE_Q4])
def test_largest_pool(L, block, fmt):
    # n_blocks * block_tokens below 2^31, to the last block (calls of no rows touch nothing)
    most = (2 ** 31 - 1) // block
    for n, want in ((1, K.KVO_OK), (most, K.KVO_OK), (most + 1, K.KVO_EINVAL), (2 ** 62, K.KVO_EINVAL)):
        assert L.kvo_paged_write(A, A, 0, A, n, block, fmt, None) == want, n
        assert L.kvo_paged_read(A, n, block, fmt, A, 0, A, None) == want, n


@pytest.mark.parametrize("scale", [2.4e38, 3e38, -2.4e38, -float("inf")])
def test_scales_that_are_not_finite_in_log2_units(L, scale):
    # the kernel works in units of log2 e: 2.36e38 is the largest scale that stays finite there
    a = {**ATTEND, "scale": ctypes.c_float(scale)}
    assert L.kvo_paged_attend(*a.values()) == K.KVO_EINVAL and b"scale" in L.kvo_last_error()


def test_binding_refuses_sizes_past_32_bits():
    # ctypes would pass their low bits: a window of 2^32 + 5 tokens as one of 5
    i, x = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 576, dtype=torch.bfloat16)
    two, five = torch.zeros(2, dtype=torch.int64), torch.zeros(5, dtype=torch.int32)
    pool = torch.zeros(4, 324 * 16, dtype=torch.uint8)
    q, o = torch.zeros(4, 2, 576, dtype=torch.bfloat16), torch.zeros(4, 2, 512, dtype=torch.bfloat16)
    plan = lambda block=16, **k: K.kvo_paged_plan(i, i, block, i.view(4, 1), i, two, two, i, i, five, i, i, **k)  # noqa: E731
    attend = lambda n=4, **k: K.kvo_paged_attend(pool, n, 16, K.KVO_CACHE_Q4, i.view(4, 1), i, five, q, 0.1, o, **k)  # noqa: E731
    calls = [("block_tokens", lambda n: plan(n)), ("window", lambda n: plan(window=n)), ("sinks", lambda n: plan(sinks=n)),
             ("window", lambda n: attend(window=n)), ("sinks", lambda n: attend(sinks=n)), ("n_blocks", lambda n: attend(n)),
             ("n_blocks", lambda n: K.kvo_paged_write(x, i, pool, n, 16, K.KVO_CACHE_Q4)),
             ("n_blocks", lambda n: K.kvo_paged_read(pool, n, 16, K.KVO_CACHE_Q4, i, x)),
             ("n_tokens", lambda n: K.kvo_paged_attend_workspace_size(1, n, 16)),
             ("n_heads", lambda n: K.kvo_paged_attend_workspace_size(1, 1, n))]
    for name, call in calls:
        for n in (2 ** 31, 2 ** 32 + 5, 2 ** 64 + 4, -2 ** 31 - 1, -2 ** 64 + 4):
            with pytest.raises(K.KvoError) as e:
                call(n)
            assert e.value.code == K.KVO_EINVAL and name in str(e.value)
