"""Infinities, NaN and negative zeros in channels that a rotation does not turn.

A channel from rotary_dim on keeps its value (rounded once to the output type)
whatever the other channels hold, so everything here is compared bit for bit.
"""
import pytest
import torch

import nvfp4_quantized_paged_nvfp4kv_gb300 as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"
ODD = [float("inf"), -float("inf"), float("nan"), -0.0]
ROTATIONS = [(None, False), (0, False), (0, True), (32, False), (64, False), (96, False), (32, True), (64, True), (96, True)]


def rope_of(rot, inter):
    return None if rot is None else nv.Rope([10000.0 ** (-2.0 * i / max(rot, 1)) for i in range(rot // 2)], inter)


def rows(T, H, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn((T, H, 128), generator=g, device=DEV).to(dtype)


def with_odd_values(x, first):
    """A copy of x with each of ODD in every eighth row or so, at changing
    channels from `first` on; never two in one row."""
    y = x.clone()
    flat = y.view(-1, 128)
    for i in range(flat.shape[0]):
        if i % 2 == 0:
            flat[i, first + (7 * i + i // 5) % (128 - first)] = ODD[i // 2 % len(ODD)]
    return y


def same(a, b):
    """Bit for bit, any NaN like any other."""
    ints = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(1.5, float("inf"), -float("inf")).view(ints),
                                                             b.nan_to_num(1.5, float("inf"), -float("inf")).view(ints))


@pytest.mark.parametrize("rot,inter", ROTATIONS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_channels_that_are_not_turned_keep_their_values(rot, inter, dtype):
    T, hq, hkv = 37, 9, 3
    first = rot or 0
    plain = rows(T, hq, dtype, 1), rows(T, hkv, dtype, 2)
    odd = tuple(with_odd_values(x, first) for x in plain)
    pos = torch.arange(5, 5 + T, dtype=torch.int32, device=DEV)
    rope = rope_of(rot, inter)

    def call(q, k):
        qo, ko = torch.empty((T, hq, 128), dtype=torch.bfloat16, device=DEV), torch.empty_like(k)
        nv.nvfp4kv_qk_norm_rope(q, k, pos, qo, ko, rope)
        return qo, ko
    for x, base, got in zip(odd, call(*plain), call(*odd)):
        assert same(got[..., first:], x[..., first:].to(got.dtype))          # kept
        assert same(got[..., :first], base[..., :first])                     # turned: as without the odd values


@pytest.mark.parametrize("inter", [False, True])
def test_a_turned_pair_stays_by_itself(inter):
    """An infinity in a turned channel reaches its partner and nothing else."""
    rot, T, H = 96, 16, 4
    x = rows(T, H, torch.float32, 3)
    pos = torch.arange(3, 3 + T, dtype=torch.int32, device=DEV)
    rope = rope_of(rot, inter)

    def call(k):
        qo, ko = torch.empty((T, H, 128), dtype=torch.bfloat16, device=DEV), torch.empty_like(k)
        nv.nvfp4kv_qk_norm_rope(k, k, pos, qo, ko, rope)
        return ko
    base, y = call(x), x.clone()
    reached = torch.zeros(x.shape, dtype=torch.bool, device=DEV)
    for t in range(T):
        for h in range(H):
            c = (11 * t + 29 * h) % rot
            mate = c ^ 1 if inter else (c + rot // 2) % rot
            y[t, h, c] = ODD[(t + h) % 3]
            reached[t, h, c] = reached[t, h, mate] = True
    got = call(y)
    assert not got[reached].isfinite().any()
    assert torch.equal(got[~reached], base[~reached])


@pytest.mark.parametrize("rot,inter", ROTATIONS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_cache_write_of_odd_values(rot, inter, dtype):
    """The fused write leaves the bytes that appending the finished keys leaves."""
    T, hq, hkv = 29, 5, 2
    first = rot or 0
    q, v = rows(T, hq, dtype, 4), rows(T, hkv, dtype, 5)
    plain = rows(T, hkv, dtype, 6)
    k = with_odd_values(plain, first)
    pos = torch.arange(9, 9 + T, dtype=torch.int32, device=DEV)
    slots = torch.arange(3, 3 + T, dtype=torch.int32, device=DEV)
    rope = rope_of(rot, inter)
    qo, finished = torch.empty((T, hq, 128), dtype=torch.bfloat16, device=DEV), torch.empty_like(k)
    nv.nvfp4kv_qk_norm_rope(q, plain, pos, qo, finished, rope)
    finished[..., first:] = k[..., first:]
    want, got = (nv.NVFP4Cache.allocate(2, hkv, device=DEV) for _ in range(2))
    nv.nvfp4kv_quantize_append(want, finished, v, slots)
    nv.nvfp4kv_qk_norm_rope_append(got, q, k, v, pos, slots, qo, rope)
    assert torch.equal(got.pool, want.pool)
