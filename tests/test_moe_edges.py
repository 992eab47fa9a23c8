"""Mixture-of-experts operators at their edges: calls that give up, depths and scales that end inside a tile, far values,
arguments that do not fit together.  The references and tolerances are those of test_moe.py unless a test derives its own.
"""
import ctypes
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


@gpu
@pytest.mark.parametrize("kind", ["w8a8", "fp8", "fp16", "bf16"])
def test_pairs_under_a_tiny_limit_leave_the_device_as_it_was(wq, kind):
    """Neither CTA of a pair leaves while something of the other's is on its way to it: after calls that may have given
    up, kernels that use the same shared memory otherwise get their results, and so do the pairs."""
    N, K, counts = 1024, 4096, [200, 90]
    wa, _ = make_weights(kind, 2, N, K, 128, 2)
    xa, _ = make_x(kind, sum(counts), K, 2)
    one, _ = make_x(kind, 3, K, 3)
    off, few = offsets(counts), offsets([1, 2])
    good, other = call(wq, kind, xa, wa, off, None, 128, False), call(wq, kind, one, wa, few, None, 128, False)
    assert wq.device_status() == 0
    for _ in range(5):
        try:
            wq.set_wait_limit(1)
            call(wq, kind, xa, wa, off, None, 128, False)
        finally:
            wq.set_wait_limit(0)
        assert torch.equal(call(wq, kind, one, wa, few, None, 128, False), other)
        assert wq.device_status() in (wq.WQ_OK, wq.WQ_ERR_TIMEOUT)
        assert torch.equal(call(wq, kind, xa, wa, off, None, 128, False), good)
        assert wq.device_status() == 0


@gpu
@pytest.mark.parametrize("kind,counts", [
    ("w8a8", [200, 90]), ("fp8", [200, 90]), ("fp16", [200, 90]), ("bf16", [200, 90]),      # pairs
    ("w8a8", [9, 14]), ("fp8", [9, 14])])                                                   # single CTAs
def test_waits_that_ran_out_are_reported(wq, kind, counts):
    """Tiles of a third of a millisecond, for which the epilogue waits longer than a wait lasts under a tiny limit (about
    0.15 ms): the calls end and say so, and the next ones are right.  (Neither of the other INT4 kernels has such a wait.)"""
    N, K, T = 9472, 131056 if kind == "w8a8" else 131072, sum(counts)
    g = torch.Generator(device="cuda").manual_seed(1)
    if kind in ("fp16", "bf16"):
        w = torch.randint(-2 ** 31, 2 ** 31, (2, N, K // 8), dtype=torch.int32, device="cuda", generator=g)
        wa = (w, torch.full((2, N, K // 128), 2.0 ** -9, dtype=torch.float16, device="cuda"),
              torch.full((2, N, K // 1024), 0x77777777, dtype=torch.int32, device="cuda"))
    else:
        w = torch.randint(0, 127, (2, N, K), dtype=torch.int8, device="cuda", generator=g)
        wa = (w if kind == "w8a8" else w.view(torch.uint8), torch.full((2, N), 2.0 ** -20, device="cuda"))
    xa, _ = make_x(kind, T, K, 2)
    off, rows = offsets(counts), torch.randperm(T, device="cuda").to(torch.int32)
    for r, swiglu in ((rows, False), (None, True)):
        good = call(wq, kind, xa, wa, off, r, 128, swiglu)
        assert wq.device_status() == 0
        for _ in range(3):
            try:
                wq.set_wait_limit(1)
                call(wq, kind, xa, wa, off, r, 128, swiglu)
                assert wq.device_status() == wq.WQ_ERR_TIMEOUT
            finally:
                wq.set_wait_limit(0)
            again = call(wq, kind, xa, wa, off, r, 128, swiglu)
            assert torch.equal(again.view(torch.int16), good.view(torch.int16))
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


@gpu
@pytest.mark.parametrize("kind", ["w8a8", "fp16", "bf16"])
def test_a_layer_whose_logits_are_of_other_tokens_is_refused(wq, kind):
    """More logits than rows of x would give zeros for the rest, fewer would leave rows of x out."""
    E, K, I, N, T = 4, 64, 32, 48, 6
    up, _ = make_weights(kind, E, 2 * I, K, 32, 1)
    down, _ = make_weights(kind, E, N, I, 32, 2)
    dt = torch.bfloat16 if kind == "bf16" else torch.float16

    def layer(x, logits):
        return wq.moe_mlp_w8a8(x, logits, up, down, 2) if kind == "w8a8" else wq.moe_mlp_w4a16(x, logits, up, down, 2, 32)

    x = torch.randn(T, K, device="cuda").to(dt)
    assert layer(x, torch.randn(T, E, device="cuda")).shape == (T, N)
    for tokens in (T - 1, T + 1):
        with pytest.raises(ValueError, match="tokens"):
            layer(x, torch.randn(tokens, E, device="cuda"))
    for bad in (torch.randn(T, E), torch.randn(T, E, device="cuda").double(), torch.randn(T, 2 * E, device="cuda")[:, ::2],
                torch.randn(T, E + 1, device="cuda"), None):
        with pytest.raises((ValueError, TypeError)):
            layer(x, bad)
    for bad in (x.cpu(), x.float(), x.t(), x[0], None):
        with pytest.raises((ValueError, TypeError)):
            layer(bad, torch.randn(T, E, device="cuda"))


@gpu
def test_arguments_that_are_no_tensors_are_refused_as_such(wq):
    """As everywhere in the binding: TypeError, with the argument's name."""
    T, E, N, K = 4, 2, 16, 32
    x = torch.zeros(T, K, dtype=torch.uint8, device="cuda")
    w = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    sx, sw, off = torch.ones(T, device="cuda"), torch.ones(E, N, device="cuda"), offsets([1, 3])
    rows = torch.zeros(T, dtype=torch.int32, device="cuda")
    good = [x, sx, w, sw, off, rows]
    wq.grouped_gemm_fp8(*good)
    for n, name in enumerate(("xq", "sx", "wq", "sw", "offsets", "rows")):
        for bad in ([0, 1], 0.5, np.zeros(4, np.int32)):
            args = list(good)
            args[n] = bad
            with pytest.raises(TypeError, match=name):
                wq.grouped_gemm_fp8(*args)
    with pytest.raises(ValueError, match="rows"):
        wq.grouped_gemm_fp8(*good[:5], rows.view(2, 2))


@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("dtype", [0, 2])
def test_router_arguments_that_overlap_are_refused(wq, T, dtype):
    """Each pair of the logits, the five outputs and the workspace, at the first, the last and the bytes before."""
    E, k = 24, 3
    ws = wq.moe_route_workspace_bytes(T, E)
    size = [T * E * (2 if dtype else 4), T * k * 4, T * k * 4, (E + 1) * 4, T * k * 4, T * k * 4, ws]
    for i in range(7):
        for j in range(7):
            if i == j or not (size[i] and size[j]):
                continue
            base = 0x1000000
            for at in (0, (size[i] - 1) // 16 * 16, 16 - (size[j] + 15) // 16 * 16):
                if at < 0 and at + size[j] <= 0:
                    continue
                p = [ctypes.c_void_p((n + 2) << 32) for n in range(7)]
                p[i], p[j] = ctypes.c_void_p(base), ctypes.c_void_p(base + at)
                status = wq.lib.wq_moe_route(p[0], dtype, T, E, k, 1, *p[1:], None)
                assert status == wq.WQ_ERR_INVALID_ARG and b"overlaps" in wq.lib.wq_last_error(), (i, j, at)


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


# ------------------------------------------------------------------------------------------------ SwiGLU far from zero
FAR_GATES = [-89.5, -88.5, -88.0, -87.5, -87.0, -80.0, -30.0, -1.0, 0.5, 30.0, 88.5, 1000.0]


def check_far(y, gates, up, u):
    """y against silu(gates) up in fp64: u for the type of y; 2 + 1.2 |g| units (2^-23) for the exponential, which turns
    subnormal below g = -87.3 (a unit of 2^-149 of it), two for the division and half of one each for the other three
    operations."""
    g = torch.tensor(gates, dtype=torch.float64, device="cuda")
    ref = g * torch.sigmoid(g) * up
    e = torch.exp(-g.abs())
    rel = u + (6 + 1.2 * g.abs()) * 2.0 ** -23 + torch.where(g < 0, 2.0 ** -149 / e, 0.0)
    err = (y.double() - ref).abs()
    assert (err <= ref.abs() * rel * 1.001 + 2.0 ** -25 * (y.dtype is torch.float16)).all(), (err / ref.abs()).tolist()


@gpu
@pytest.mark.parametrize("rows_per_expert", [1, 12, 64])
def test_swiglu_of_far_gates_int4(wq, rows_per_expert):
    """bf16, 128 depths of which the first is the gate's and the second the up's: silu(g) 2^100 is an ordinary value where
    exp(-g) is close to the end of fp32 and beyond."""
    K, I = 128, 24
    codes = torch.zeros(1, 2 * I, K, dtype=torch.int64, device="cuda")
    codes[0, :I, 0] = codes[0, I:, 1] = 1
    scales = torch.ones(1, 2 * I, 1, dtype=torch.float16, device="cuda")
    zeros = torch.zeros(1, 2 * I, 1, dtype=torch.int64, device="cuda")
    T = rows_per_expert
    gates = [FAR_GATES[i % len(FAR_GATES)] for i in range(max(T, len(FAR_GATES)))]
    for start in range(0, len(gates), T):
        part = gates[start:start + T] + [0.5] * (start + T - min(start + T, len(gates)))
        x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
        x[:, 0], x[:, 1] = torch.tensor(part, device="cuda").bfloat16(), 2.0 ** 100
        assert x[:, 0].tolist() == part
        y = wq.grouped_gemm_w4a16(x, pack(codes), scales, pack(zeros), offsets([T]), None, K, swiglu=True)
        for col in (0, I - 1):
            check_far(y[:, col], part, 2.0 ** 100, 2.0 ** -8)


@gpu
@pytest.mark.parametrize("T", [12, 200])
@pytest.mark.parametrize("fp8", [False, True])
def test_swiglu_of_far_gates_8_bits(wq, T, fp8):
    K, I = 64, 40
    one = 0x38 if fp8 else 1                                # E4M3's 1.0
    gates = (FAR_GATES * 20)[:T]
    dt = torch.uint8 if fp8 else torch.int8
    q = torch.zeros(1, 2 * I, K, dtype=dt, device="cuda")
    q[0, :I, 0] = q[0, I:, 1] = one
    sw = torch.ones(1, 2 * I, device="cuda")
    sw[0, I:] = 2.0 ** 104                                  # codes are +-1: the gate is +-sx, the up value sx 2^104
    g = torch.tensor(gates, device="cuda")
    xq = torch.zeros(T, K, dtype=dt, device="cuda")
    xq[:, 0] = torch.where(g < 0, 0xB8 if fp8 else -1, one).to(dt)
    xq[:, 1] = one
    sx = g.abs()
    fn = wq.grouped_gemm_fp8 if fp8 else wq.grouped_gemm_w8a8
    y = fn(xq, sx, q, sw, offsets([T]), swiglu=True)
    far = [i for i, v in enumerate(gates) if v < -86]
    for col in (0, I - 1):
        for i in far:
            check_far(y[i:i + 1, col], [gates[i]], 2.0 ** 104 * abs(gates[i]), 2.0 ** -11)


# ------------------------------------------------------------------------------------------------ offsets, NaN in large batches
SENTINEL = 77.0


@gpu
@pytest.mark.parametrize("kind", ["w8a8", "fp8", "fp16", "bf16"])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("swiglu", [True, False])
def test_bad_offsets_of_large_batches_stay_in_bounds(wq, kind, gather, swiglu):
    """Pairs of CTAs: offsets out of range or decreasing are clamped to [0, R] and made non-decreasing, with rows that
    repeat and lie outside x; guard rows around y stay as they are."""
    R, E, N, K = 700, 4, 136, 160
    wa, w = make_weights(kind, E, N, K, 32, 3)
    xa, x = make_x(kind, R, K, 3)
    g = torch.Generator(device="cuda").manual_seed(8)
    rows = torch.randint(-2, R + 2, (R,), device="cuda", generator=g).to(torch.int32) if gather else None
    dt = torch.bfloat16 if kind == "bf16" else torch.float16
    for raw in ([-7, 400, 5, 2000, 300], [800, 900, 701, 0, 90], [0, -1, -2, -3, 2 ** 31 - 1],
                [-2 ** 31, 2 ** 31 - 1, 0, 0, 0], [3, 260, 260, 517, 690]):
        fixed = np.maximum.accumulate(np.clip(raw, 0, R))
        off = torch.tensor(raw, dtype=torch.int32, device="cuda")
        cols = N // 2 if swiglu else N
        guarded = torch.full((R + 32, cols), SENTINEL, dtype=dt, device="cuda")
        out = guarded[16:-16]
        call(wq, kind, xa, wa, off, rows, 32, swiglu, out)
        y, tol, written = product_ref(kind, x, w, rows, fixed, R, K, swiglu)
        assert ((out.double() - y).abs() <= tol)[written].all()
        assert (out[~written] == SENTINEL).all()
        assert (guarded[:16] == SENTINEL).all() and (guarded[-16:] == SENTINEL).all()
    assert wq.device_status() == 0


@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp8"])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("swiglu", [True, False])
def test_nan_and_inf_stay_in_their_row_of_a_large_batch(wq, kind, gather, swiglu):
    """Pairs of CTAs, both halves of a tile, rows next to padding: a dirty row changes its own outputs only."""
    counts, N, K = [90, 300, 41], 136, 288
    T = sum(counts)
    wa, _ = make_weights(kind, 3, N, K, 32, 9)
    xa, _ = make_x(kind, T, K, 9)
    dirty = xa[0].clone()
    where = [0, 3, 89, 90, 245, 389, 390, T - 1]
    for n, p in enumerate(where):
        if kind == "fp8":
            dirty[p, (37 * n) % K] = 0x7F if n % 2 else 0xFF
        else:
            dirty[p, (37 * n) % K] = math.nan if n % 2 else math.inf
    off = offsets(counts)
    rows = torch.arange(T, device="cuda", dtype=torch.int32).flip(0) if gather else None
    clean_y = call(wq, kind, xa, wa, off, rows, 32, swiglu)
    y = call(wq, kind, (dirty, *xa[1:]), wa, off, rows, 32, swiglu)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[T - 1 - p for p in where] if gather else where] = False
    assert torch.equal(y[keep], clean_y[keep])
    bad = y[~keep].float()
    if kind == "fp8":
        assert torch.isnan(bad).all()
    elif not swiglu:
        assert not torch.isfinite(bad).any()


# ------------------------------------------------------------------------------------------------ rows that nothing wrote
@gpu
@pytest.mark.parametrize("K", [16, 320, 4112, 8208, 16400])
def test_the_token_quantizer_takes_any_bits_row_by_row(wq, K):
    """Rows of any bits, NaN and infinities among them, change nothing in the other rows, whichever kernel takes the
    depth (the last two: two CTAs a row, and two passes)."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(70, K, device="cuda", generator=g).half()
    q, s = wq.quantize_int8_per_token(x)
    dirty = torch.arange(70, device="cuda") % 3 == 1
    x.view(torch.int16)[dirty] = torch.randint(-2 ** 15, 2 ** 15, (int(dirty.sum()), K), device="cuda", generator=g).short()
    x[1], x[4] = math.nan, math.inf
    q2, s2 = wq.quantize_int8_per_token(x)
    assert torch.equal(q2[~dirty], q[~dirty]) and torch.equal(s2[~dirty], s[~dirty])


@gpu
@pytest.mark.parametrize("kind", ["w8a8", "fp16", "bf16"])
@pytest.mark.parametrize("T", [9, 300])
@pytest.mark.parametrize("bits", [0x7FFF, 0x7C00, 0xFFFF])
def test_a_layer_does_not_see_what_its_memory_held(wq, kind, T, bits):
    """Padded tokens leave rows of the products unwritten: with every byte of the allocator's cache NaN or infinity, the
    layer's result is the same, finite, and zero for those tokens."""
    E, k, K, I, N = 6, 2, 128, 512, 160
    g = torch.Generator(device="cuda").manual_seed(T)
    up, _ = make_weights(kind, E, 2 * I, K, 64, 1)
    down, _ = make_weights(kind, E, N, I, 64, 2)
    x = torch.randn(T, K, device="cuda", generator=g).to(torch.bfloat16 if kind == "bf16" else torch.float16)
    logits = torch.randn(T, E, device="cuda", generator=g)
    logits[1::2] = -math.inf

    def layer(fill):
        sizes = [T * k * I * 2, T * k * N * 2, T * N * 2, T * k * I, T * K, T * k * 4, T * 4, 1 << 12, 1 << 16]
        held = [torch.full((n // 2 + 256,), fill, dtype=torch.int16, device="cuda") for n in sizes for _ in range(4)]
        torch.cuda.synchronize()
        del held
        if kind == "w8a8":
            return wq.moe_mlp_w8a8(x, logits, up, down, k)
        return wq.moe_mlp_w4a16(x, logits, up, down, k, 64)

    clean = layer(0)
    assert torch.isfinite(clean).all() and (clean[1::2] == 0).all() and float(clean[::2].abs().max()) > 0
    assert torch.equal(layer(bits - (1 << 16) if bits >= 1 << 15 else bits), clean)


# ------------------------------------------------------------------------------------------------ rounding of INT4 weights
def to_bits(w, bits):
    """fp64 values rounded to `bits` significant bits, ties to even."""
    m, e = torch.frexp(w)
    return torch.ldexp(torch.round(m * 2.0 ** bits), e - bits)


@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("counts,rounded", [([3, 8], False), ([12, 30], False), ([23, 21], True), ([300, 90], True)])
@pytest.mark.parametrize("group", [32, 128])
def test_int4_weights_are_rounded_where_the_header_says(wq, kind, counts, rounded, group):
    """From 22 rows per expert on, y is the product of s (q - z) rounded to x's type; below, of s (q - z) itself.  bf16
    takes s in two parts there, (q - z) hi + round((q - z) lo), rounded once more.
    A row of x has eight entries of +-1, so that the fp32 sums are off by at most 8 2^-23 S and what is left is the
    output's rounding u |y|.  Where the terms cancel (|y| below a tenth of one, about 3% of the outputs) the weights'
    roundings, u / 2 of a term at most each, are far larger: no output may be outside for the one form, some are for the
    other."""
    N, K, T = 128, 2048, sum(counts)
    g = torch.Generator(device="cuda").manual_seed(group)
    codes = torch.randint(0, 16, (2, N, K), device="cuda", generator=g)
    zeros = torch.randint(0, 16, (2, N, K // group), device="cuda", generator=g)
    scales = torch.exp(torch.randn(2, N, K // group, device="cuda", generator=g) * 0.5 - 5).half()
    d = (codes - zeros.repeat_interleave(group, -1)).double()
    s = scales.double().repeat_interleave(group, -1)
    exact = d * s
    if kind == "fp16":
        coarse = to_bits(exact, 11)
    else:
        hi = to_bits(s, 8)
        coarse = to_bits(d * hi + to_bits(d * (s - hi), 8), 8)
    x = torch.zeros(T, K, dtype=torch.float16 if kind == "fp16" else torch.bfloat16, device="cuda")
    where = torch.rand(T, K, device="cuda", generator=g).topk(8, dim=1).indices
    x.scatter_(1, where, torch.randint(0, 2, (T, 8), device="cuda", generator=g).to(x.dtype) * 2 - 1)
    y = wq.grouped_gemm_w4a16(x, pack(codes), scales, pack(zeros), offsets(counts), group_size=group).double()
    u, outside = 2.0 ** -11 if kind == "fp16" else 2.0 ** -8, {}
    for name, w in (("exact", exact), ("rounded", coarse)):
        at, outside[name] = 0, 0
        for e, n in enumerate(counts):
            xe = x[at:at + n].double()
            ref, size = xe @ w[e].T, xe.abs() @ w[e].abs().T
            tol = 8 * 2.0 ** -23 * size * (1 + u) + ref.abs() * u + 2.0 ** -25
            outside[name] += int(((y[at:at + n] - ref).abs() > tol).sum())
            at += n
    assert outside["rounded" if rounded else "exact"] == 0, outside
    assert outside["exact" if rounded else "rounded"] > 0, outside


# ------------------------------------------------------------------------------------------------ streams, graphs, sizes
@gpu
@pytest.mark.parametrize("T", [40, 300, 5000])
def test_routers_on_two_streams_and_in_two_graphs(wq, T):
    """Calls that overlap share nothing; two graphs of the router, one after the other, may share a workspace, and follow
    the logits in memory."""
    E, k = 48, 5
    g = torch.Generator(device="cuda").manual_seed(T)
    logits = [torch.randn(T, E, device="cuda", generator=g) for _ in range(2)]
    good = [wq.moe_route(x, k) for x in logits]
    y = torch.randn(T * k, 72, device="cuda", generator=g).half()
    sums = [wq.moe_combine(y, w, slots) for _, w, _, _, slots in good]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(30):
        got = []
        for x, st in zip(logits, streams):
            r = wq.moe_route(x, k, stream=st)
            got.append((r, wq.moe_combine(y, r[1], r[4], stream=st)))
        torch.cuda.synchronize()
        for (r, out), want, total in zip(got, good, sums):
            assert all(torch.equal(a, b) for a, b in zip(r, want)) and torch.equal(out, total)
    workspace = torch.empty(max(16, wq.moe_route_workspace_bytes(T, E)), dtype=torch.uint8, device="cuda")
    held, graphs, out = torch.empty_like(logits[0]), [], []
    for renormalize in (True, False):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            out.append(wq.moe_route(held, k, renormalize, workspace=workspace))
    for x in (*logits, logits[0].neg()):
        held.copy_(x)
        workspace.fill_(0xA5)
        for graph in graphs:
            graph.replay()
        for renormalize, got in zip((True, False), out):
            assert all(torch.equal(a, b) for a, b in zip(got, wq.moe_route(x, k, renormalize)))


@gpu
def test_the_router_at_its_most_tokens(wq):
    """2^23 tokens, logits past 2^31 elements: a known choice for each token."""
    T, E = 1 << 23, 300
    token = torch.arange(T, device="cuda")
    want = (token * 7919 + (token >> 11)) % E
    logits = torch.zeros(T, E, dtype=torch.float16, device="cuda")
    logits.scatter_(1, want[:, None], 4.0)
    ids, weights, off, rows, slots = wq.moe_route(logits, 1, renormalize=False)
    assert torch.equal(ids[:, 0].long(), want)
    p = math.exp(4.0) / (math.exp(4.0) + E - 1)
    assert float((weights.double() - p).abs().max()) <= 2.0 ** -15 * p
    assert torch.equal(off.long(), torch.cat([token.new_zeros(1), torch.bincount(want, minlength=E).cumsum(0)]))
    order = torch.sort(want, stable=True).indices
    assert torch.equal(rows.long(), order)
    assert torch.equal(slots[order, 0].long(), token)


@gpu
@pytest.mark.parametrize("N", [16400, 16401])
def test_a_combine_past_32_bit_offsets(wq, N):
    """Rows of y and of the result past 2^31 elements."""
    T, R = 140000, 140001
    y = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    y.copy_((torch.arange(R, device="cuda") % 251)[:, None] + (torch.arange(N, device="cuda") % 3))
    slots = torch.arange(T, device="cuda").flip(0).to(torch.int32)[:, None] + 1
    weights = torch.full((T, 1), 0.5, device="cuda")
    out = wq.moe_combine(y, weights, slots)
    for t in (0, 1, 69999, 131071, 131072, T - 1):
        assert torch.equal(out[t], y[T - t] * 0.5)
    assert torch.equal(out[:, N - 1], y[1:, N - 1].flip(0) * 0.5)


@gpu
@pytest.mark.parametrize("kind,R", [("fp16", 140000), ("bf16", 140000), ("w8a8", 3000), ("fp16", 3000), ("fp16", 9000)])
def test_products_past_32_bit_offsets(wq, kind, R):
    """y past 2^31 elements: pairs of CTAs in order and gathered, single CTAs (6 rows per expert) and both other INT4
    kernels (6 and 18 rows per expert), whose outputs are as many by their width."""
    E, K = (3, 32) if R == 140000 else (500, 32)
    N = 16400 if R == 140000 else (1 << 31) // R + 1000
    g = torch.Generator(device="cuda").manual_seed(3)
    counts = [70001, 69989, 10] if R == 140000 else [R // E] * E
    off = offsets(counts)
    if kind == "w8a8":
        wa = (torch.randint(-128, 128, (E, N, K), device="cuda", dtype=torch.int8, generator=g), torch.ones(E, N, device="cuda"))
        xa = (torch.randint(-128, 128, (R, K), device="cuda", dtype=torch.int8, generator=g), torch.full((R,), 2.0 ** -6, device="cuda"))
    else:
        wa = (torch.randint(-2 ** 31, 2 ** 31, (E, N, K // 8), device="cuda", dtype=torch.int32, generator=g),
              torch.full((E, N, 1), 2.0 ** -6, dtype=torch.float16, device="cuda"),
              torch.full((E, N, 1), 7, dtype=torch.int32, device="cuda"))
        xa = (torch.randn(R, K, device="cuda", generator=g).to(torch.bfloat16 if kind == "bf16" else torch.float16),)
    rows = torch.arange(R, device="cuda", dtype=torch.int32).flip(0)
    nibbles = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    u = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
    for r in (None, rows):
        y = call(wq, kind, xa, wa, off, r, 32, False)
        for p in (0, 1, R // 2, (1 << 31) // N, (1 << 31) // N + 1, R - 2, R - 1):
            e = int(torch.searchsorted(off.long(), torch.tensor(p, device="cuda"), right=True)) - 1
            t = R - 1 - p if r is not None else p
            x = xa[0][t].double()
            if kind == "w8a8":
                ref = (wa[0][e].double() @ x) * 2.0 ** -6
                tol = ref.abs() * (u + 2.0 ** -22) + 2.0 ** -25
            else:
                w = (((wa[0][e].unsqueeze(-1) >> nibbles) & 15).view(N, K).double() - 7) * 2.0 ** -6   # exact in 8 bits
                ref = w @ x
                tol = K * 2.0 ** -23 * (w.abs() @ x.abs()) * (1 + u) + ref.abs() * u + 2.0 ** -25
            assert ((y[p].double() - ref).abs() <= tol).all(), p
        del y
    assert wq.device_status() == 0
