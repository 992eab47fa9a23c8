"""Mixture-of-experts operators at their edges: calls that give up, depths and scales that end inside a tile, far values,
arguments that do not fit together.  The references and tolerances are those of test_moe.py unless a test derives its own.
"""
import math

import numpy as np
import pytest
import torch

from test_moe import call, make_weights, make_x, product_ref, wq  # noqa: F401  (wq: the fixture)

gpu = pytest.mark.gpu


def offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------ expired waits
@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_few_rows_under_a_tiny_limit_leave_the_device_as_it_was(wq, kind):
    """7 to 22 rows per INT4 expert, a CTA per tile: calls whose waits may run out while half a pack's stores to tensor
    memory are under way end, and the next calls give the results of the first."""
    N, K, counts = 9472, 8192, [16]
    wa, _ = make_weights(kind, 1, N, K, 128, 2)
    xa, _ = make_x(kind, sum(counts), K, 2)
    off = offsets(counts)
    good = call(wq, kind, xa, wa, off, None, 128, False)
    assert wq.device_status() == 0
    try:
        wq.set_wait_limit(1)
        for _ in range(5):
            call(wq, kind, xa, wa, off, None, 128, False)
        assert wq.device_status() in (wq.WQ_OK, wq.WQ_ERR_TIMEOUT)
    finally:
        wq.set_wait_limit(0)
    for _ in range(3):
        assert torch.equal(call(wq, kind, xa, wa, off, None, 128, False), good)
    assert wq.device_status() == 0


# ------------------------------------------------------------------------------------------------ CTAs that share a tile
@gpu
@pytest.mark.parametrize("kind,counts,N,K,group", [
    ("w8a8", [300, 0, 129, 70], 700, 4112, 32), ("fp8", [300, 0, 129, 70], 700, 4112, 32),
    ("fp16", [300, 0, 129, 70], 700, 4160, 32), ("bf16", [300, 0, 129, 70], 700, 4160, 32),       # pairs
    ("fp16", [20, 9, 0, 14], 200, 4160, 32), ("bf16", [20, 9, 0, 14], 200, 4224, 128)])           # a depth that is shared
@pytest.mark.parametrize("swiglu", [False, True])
def test_shared_tiles_always_give_the_same(wq, kind, counts, N, K, group, swiglu):
    """What one CTA of a cluster hands to another arrives whole: the same call gives the same bits every time, beside
    other work on the device too."""
    wa, _ = make_weights(kind, len(counts), N, K, group, 11)
    xa, _ = make_x(kind, 50, K, 11)
    off = offsets(counts)
    R = sum(counts)
    rows = torch.randint(0, 50, (R,), device="cuda", dtype=torch.int32)
    in_order = tuple(t[rows.long()].contiguous() for t in xa)
    good = call(wq, kind, xa, wa, off, rows, group, swiglu)
    other, noise = torch.cuda.Stream(), torch.empty(1 << 26, device="cuda")
    for i in range(60):
        if i % 3 == 0:
            with torch.cuda.stream(other):
                noise.mul_(1.5)
        assert torch.equal(call(wq, kind, xa, wa, off, rows, group, swiglu), good)
        assert torch.equal(call(wq, kind, in_order, wa, off, None, group, swiglu), good)
    torch.cuda.synchronize()
    assert wq.device_status() == 0


# ------------------------------------------------------------------------------------------------ arguments
@pytest.mark.parametrize("top_k", [2 - 2 ** 32, 2 ** 32 + 2, 2 ** 31, -2 ** 31 - 1, 2 ** 64 + 2])
def test_a_top_k_past_32_bits_is_refused(wq, top_k):
    """It would reach the C entry point as another number, one that the outputs have no room for."""
    with pytest.raises(ValueError, match="top_k"):
        wq.moe_route(torch.zeros(4, 8), top_k)
    with pytest.raises(ValueError, match="32 bits"):
        wq.moe_route_workspace_bytes(top_k, 8)


@gpu
def test_a_top_k_that_the_router_does_not_take(wq):
    logits = torch.zeros(4, 8, device="cuda")
    for top_k in (0, -1, 9, 2 ** 31 - 1, -2 ** 31):
        with pytest.raises(wq.WQError):
            wq.moe_route(logits, top_k)


@gpu
def test_sizes_past_32_bits_are_refused(wq):
    """A size of 2^32 + n would arrive as n, and all but n rows of the result stay as they were."""
    many = 2 ** 32 + 32
    with pytest.raises(ValueError, match="32 bits"):
        wq.moe_combine(torch.empty(many, 1, dtype=torch.float16, device="cuda"), torch.ones(1, 1, device="cuda"),
                       torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="32 bits"):
        wq.moe_route(torch.empty(many, 1, dtype=torch.float16, device="cuda"), 1)
    rows = torch.empty(many, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="32 bits"):
        wq.grouped_gemm_w8a8(torch.empty(4, 16, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda"),
                             torch.empty(1, 2, 16, dtype=torch.int8, device="cuda"), torch.ones(1, 2, device="cuda"),
                             torch.zeros(2, dtype=torch.int32, device="cuda"), rows)


# ------------------------------------------------------------------------------------------------ depth and scales
def pack(codes):
    """[..., n] 4-bit codes -> int32 words of eight, lowest bits first."""
    c = torch.nn.functional.pad(codes, (0, -codes.shape[-1] % 8)).unflatten(-1, (-1, 8)).long()
    v = (c << torch.arange(0, 32, 4, device="cuda")).sum(-1)
    return torch.where(v >= 2 ** 31, v - 2 ** 32, v).to(torch.int32)


INT4_COUNTS = [[2, 1], [12, 9], [70, 50], [300, 41]]    # below 7, below 22 and more rows per expert, one tile and several


@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("counts", INT4_COUNTS)
@pytest.mark.parametrize("group,K", [(32, 160), (32, 96), (64, 192), (64, 64), (128, 384)])
@pytest.mark.parametrize("gather", [True, False])
def test_a_large_last_scale_at_a_depth_that_ends_inside_a_tile(wq, kind, counts, group, K, gather):
    """Scale 6000, zero point 15, codes 8 .. 15 in the last group: every weight is finite (at most 42000 in size), though
    6000 * (0 - 15) would not be in fp16.  The tolerance is that of the other INT4 products."""
    N, T = 72, sum(counts)
    g = torch.Generator(device="cuda").manual_seed(K)
    codes = torch.randint(0, 16, (2, N, K), device="cuda", generator=g)
    zeros = torch.randint(0, 16, (2, N, K // group), device="cuda", generator=g)
    scales = (torch.rand(2, N, K // group, device="cuda", generator=g) * 0.01).half()
    codes[..., -group:] |= 8
    zeros[..., -1], scales[..., -1] = 15, 6000.0
    w = ((codes - zeros.repeat_interleave(group, -1)).double() * scales.double().repeat_interleave(group, -1))
    x = torch.randn(T, K, device="cuda", generator=g)
    x[:, -group:] *= 2.0 ** -12
    x = x.to(torch.float16 if kind == "fp16" else torch.bfloat16)
    off = offsets(counts)
    rows = torch.randperm(T, device="cuda", generator=g).to(torch.int32) if gather else None
    y = wq.grouped_gemm_w4a16(x, pack(codes), scales, pack(zeros), off, rows, group)
    ref, tol, _ = product_ref(kind, x.double(), w, rows, off.cpu(), T, K, False)
    assert ((y.double() - ref).abs() <= tol).all()


@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("counts", INT4_COUNTS)
@pytest.mark.parametrize("group,K", [(32, 160), (64, 192), (128, 384), (128, 256), (256, 256)])
def test_an_infinite_last_scale_gives_infinities(wq, kind, counts, group, K):
    """All products of the last group have one sign, so that the sum is that infinity whichever kernel takes the rows."""
    N, T = 40, sum(counts)
    (q, s, z), _ = make_weights(kind, 2, N, K, group, 4)
    g = torch.Generator(device="cuda").manual_seed(5)
    codes = torch.randint(0, 16, (2, N, K), device="cuda", generator=g)
    codes[..., -group:] = torch.randint(0, 7, (2, N, group), device="cuda", generator=g)
    zeros = torch.randint(0, 16, (2, N, K // group), device="cuda", generator=g)
    zeros[..., -1] = 7
    s = s.clone()
    s[:, ::2, -1] = math.inf
    (x,), _ = make_x(kind, T, K, 4)
    x = x.abs() + 0.125
    y = wq.grouped_gemm_w4a16(x, pack(codes), s, pack(zeros), offsets(counts), group_size=group)
    assert (y[:, ::2] == -math.inf).all()
    assert torch.isfinite(y[:, 1::2]).all()
