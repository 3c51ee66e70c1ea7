"""Attention over the 4-bit cache where a row's weights favour tokens whose values are many orders of
magnitude smaller than the others': P s is held in fp16, so the power of two that goes with it has to
follow the row's own largest P s, not the largest s of the cache. References in fp64."""
import numpy as np
import pytest
import torch

import stream_ref as ref
from test_gpu_kv4_paths import _i32, _randn, attend, check

import exact_attention_138_b200 as ea


def _small(order, n, rng):
    """Which tokens hold the small values."""
    j = np.arange(n)
    return {"first": j < n // 2, "last": j >= n // 2, "alternating": j % 2 == 0, "few": j % 97 == 5,
            "random": rng.random(n) < 0.5}[order]


@pytest.mark.gpu
@pytest.mark.parametrize("H,nq,d", [(1, 1, 64), (4, 1, 128), (4, 1, 32), (8, 2, 64), (4, 5, 128)])
@pytest.mark.parametrize("order", ["first", "last", "alternating", "few", "random"])
@pytest.mark.parametrize("ratio", [3e3, 1e8, 1e20])
def test_small_values_keep_their_weight(cuda_device, H, nq, d, order, ratio):
    # keys are +a or -a along the ones, queries +1 or -1 along them: heads of one sign see the small values
    # with scores 2 a sqrt(d) = 62 above the others', heads of the other sign the large ones
    n, page = 700, 16
    rng = np.random.default_rng(3)
    small = torch.from_numpy(_small(order, n, rng))
    k = 0.05 * _randn((1, 1, n, d), 4).float() + torch.where(small, 31 * d ** -0.5, -31 * d ** -0.5)[:, None]
    v = _randn((1, 1, n, d), 5).float() * torch.where(small, 1.0, ratio)[:, None]
    q = 0.1 * _randn((1, H, nq, d), 6).float() + torch.tensor([1.0, 1.0, -1.0, 1.0])[torch.arange(H) % 4][:, None, None]
    k, v, q = (x.bfloat16() for x in (k, v, q))
    table = rng.permutation(44).astype(np.int32)[None]
    pool = ea.kv4_pool(44, 1, page, d)
    ea.kv4_append(pool, _i32(table), _i32([0]), k.cuda(), v.cuda())
    got = ea.kv4_attend(q.cuda(), pool, _i32(table), _i32([n]))
    assert ea.device_status() == ea.ATTN_OK
    check(got, attend(ref.f64(q), pool.cpu().numpy(), table, [n], [0], -1, 0, 0))


@pytest.mark.gpu
@pytest.mark.parametrize("down", [False, True])
def test_values_that_grow_or_fall_against_their_weights(cuda_device, down):
    # values of 1e-20 to 1e10 along the keys, scores that fall (or rise) as fast: every token counts
    n, d = 600, 32
    size = torch.logspace(-20, 10, n)
    k = (-size.log() / d ** 0.5)[None, None, :, None].expand(1, 1, n, d)
    v = _randn((1, 1, n, d), 9).float() * size[:, None]
    q = torch.ones((1, 2, 1, d)) + 0.002 * _randn((1, 2, 1, d), 7).float()
    if down:
        k, v = k.flip(2), v.flip(2)
    k, v, q = (x.bfloat16().contiguous() for x in (k, v, q))
    table = np.arange(38, dtype=np.int32)[None]
    pool = ea.kv4_pool(38, 1, 16, d)
    ea.kv4_append(pool, _i32(table), _i32([0]), k.cuda(), v.cuda())
    got = ea.kv4_attend(q.cuda(), pool, _i32(table), _i32([n]))
    assert ea.device_status() == ea.ATTN_OK
    check(got, attend(ref.f64(q), pool.cpu().numpy(), table, [n], [0], -1, 0, 0))
