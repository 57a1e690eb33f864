"""Refusals of the calls on draft trees and of the 8-bit cache's shapes: an error before anything is launched (no GPU)."""
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


MASKS = dict(parents=A, cu_tokens=A, n_requests=2, n_tokens=4, masks=A, mask_words=1, depths=A, status=A, stream=None)
ACCEPT = dict(parents=A, drafted=A, chosen=A, cu_tokens=A, kv_lens=A, n_requests=2, n_tokens=4, path=A, accepted=A, next_tokens=A,
              stream=None)
COMMIT = dict(lengths=A, kv_lens=A, cu_tokens=A, accepted=A, n_requests=2, block_tokens=16, max_blocks=8, window=0, sinks=0,
              block_table=A, ring=A, ring_size=8, ring_in=A, ring_out=A, lengths_out=A, stream=None)
MOVE = dict(pools=A, pool_stride=4 * 16 * 580, n_pools=2, n_blocks=4, block_tokens=16, format=8, block_table=A, max_blocks=8,
            kv_lens=A, cu_tokens=A, n_requests=2, path=A, n_tokens=4, accepted=A, stream=None)
ATTEND = dict(pool=A, n_blocks=4, block_tokens=16, format=8, block_table=A, max_blocks=8, kv_lens=A, cu_tokens=A, n_requests=2,
              masks=A, mask_words=1, depths=A, queries=A, n_tokens=2, n_heads=16, scale=0.1, window=0, sinks=0, out=A, lse=A,
              workspace=A, workspace_bytes=1 << 40, status=A, stream=None)
CACHE = [dict(block_tokens=12), dict(block_tokens=0), dict(format=2), dict(format=7), dict(format=9), dict(n_blocks=0),
         dict(n_blocks=1 << 27), dict([("max_blocks", 0)]), dict(max_blocks=1 << 27)]


def _none(*names):
    return [dict([(k, None)]) for k in names]


@pytest.mark.parametrize("over", _none("parents", "cu_tokens", "masks") + [
    dict(n_requests=0), dict(n_requests=4097), dict(n_tokens=-1), dict(n_tokens=1 << 30), dict(mask_words=0), dict(mask_words=33),
    dict(parents=A + 2), dict(masks=A + 1), dict(depths=A + 2), dict(status=A + 2)])
def test_masks(L, over):
    assert L.kvo_tree_masks(*{**MASKS, **over}.values()) == K.KVO_EINVAL and L.kvo_last_error()


@pytest.mark.parametrize("over", _none("parents", "drafted", "chosen", "cu_tokens", "kv_lens", "path", "accepted") + [
    dict(n_requests=0), dict(n_requests=4097), dict(n_tokens=-1), dict(chosen=A + 2), dict(next_tokens=A + 1)])
def test_accept(L, over):
    assert L.kvo_tree_accept(*{**ACCEPT, **over}.values()) == K.KVO_EINVAL


@pytest.mark.parametrize("over", _none("lengths", "kv_lens", "cu_tokens", "accepted", "block_table", "ring", "ring_in", "ring_out",
                                       "lengths_out") + [
    dict(n_requests=0), dict(n_requests=4097), dict(block_tokens=12), dict(max_blocks=0), dict(max_blocks=1 << 27), dict(ring_size=0),
    dict(window=-1), dict(sinks=-1), dict(ring_in=A + 4), dict(ring_out=A + 4), dict(lengths=A + 2)])
def test_commit(L, over):
    assert L.kvo_paged_commit(*{**COMMIT, **over}.values()) == K.KVO_EINVAL


@pytest.mark.parametrize("over", CACHE + _none("pools", "block_table", "kv_lens", "cu_tokens", "path", "accepted") + [
    dict(pools=A + 8), dict(n_pools=0), dict(n_pools=65536), dict(pool_stride=4 * 16 * 580 - 16), dict(pool_stride=4 * 16 * 580 + 8),
    dict(n_requests=0), dict(n_tokens=-1), dict(path=A + 2)])
def test_move(L, over):
    assert L.kvo_paged_move(*{**MOVE, **over}.values()) == K.KVO_EINVAL


@pytest.mark.parametrize("over", CACHE + _none("pool", "block_table", "kv_lens", "cu_tokens", "masks", "queries", "out", "workspace") + [
    dict(mask_words=0), dict(mask_words=33), dict(window=5, depths=None), dict(masks=A + 2), dict(depths=A + 1), dict(n_heads=0),
    dict(n_tokens=-1), dict(scale=float("nan")), dict(window=-1), dict(sinks=-1), dict(workspace=A + 128)])
def test_attend_tree(L, over):
    a = {**ATTEND, **over}
    a["scale"] = ctypes.c_float(a["scale"])
    assert L.kvo_paged_attend_tree(*a.values()) == K.KVO_EINVAL


@pytest.mark.parametrize("block", [8, 24, 40, 65528, 65536])
def test_8_bit_blocks(L, block):
    assert L.kvo_paged_block_bytes(K.KVO_CACHE_F8, block) == K.kvo_paged_block_bytes(K.KVO_CACHE_F8, block) == 580 * block
    most = (2 ** 31 - 1) // block
    for n, want in ((1, K.KVO_OK), (most, K.KVO_OK), (most + 1, K.KVO_EINVAL)):  # (calls of no rows touch nothing)
        assert L.kvo_paged_write(A, A, 0, A, n, block, K.KVO_CACHE_F8, None) == want
        assert L.kvo_paged_read(A, n, block, K.KVO_CACHE_F8, A, 0, A, None) == want


def test_binding_refuses_host_tensors_and_far_sizes():
    i, two, five = torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.int64), torch.zeros(5, dtype=torch.int32)
    pool = torch.zeros(4, 580 * 16, dtype=torch.uint8)
    q, o = torch.zeros(4, 2, 576, dtype=torch.bfloat16), torch.zeros(4, 2, 512, dtype=torch.bfloat16)
    m = i.view(4, 1)
    attend = lambda **k: K.kvo_paged_attend_tree(pool, 4, 16, K.KVO_CACHE_F8, m, i, five, m, q, 0.1, o, **k)  # noqa: E731
    commit = lambda block=16, **k: K.kvo_paged_commit(i, i, five, i, block, m, i, two, two, i, **k)  # noqa: E731
    move = lambda **k: K.kvo_paged_move(pool, 4, 16, K.KVO_CACHE_F8, m, i, five, i, i, **k)  # noqa: E731
    for call in (attend, commit, move, lambda: K.kvo_tree_masks(i, five, m), lambda: K.kvo_tree_accept(i, i, i, five, i, i, i),
                 lambda: move(n_pools=0)):
        with pytest.raises(K.KvoError) as e:
            call()
        assert e.value.code == K.KVO_EINVAL
    for name, call in (("window", lambda n: attend(window=n)), ("sinks", lambda n: attend(sinks=n)), ("window", lambda n: commit(window=n)),
                       ("block_tokens", lambda n: commit(n)), ("sinks", lambda n: commit(sinks=n)), ("n_pools", lambda n: move(n_pools=n))):
        for n in (2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1):
            with pytest.raises(K.KvoError) as e:
                call(n)
            assert e.value.code == K.KVO_EINVAL and name in str(e.value)
