"""Mixture-of-experts operators: router, quantized expert products, combine, and the layer made of them.

Every result is compared with the definition computed in fp64 (integers exactly).  Tolerances, with u the half step of
the output type (fp16 2^-11, bf16 2^-8) and S = sum_k |w x| of an element:
  w8a8    the accumulator is exact; its conversion and two fp32 products round by 2^-24 each: u + 2^-22 relative,
          and half an fp16 subnormal step (2^-25)
  fp8     products of codes are exact, K fp32 additions round (or truncate) by at most 2^-23 of a partial sum <= S
  w4a16   each weight is rounded to the activations' type: (u + K 2^-23) S, and u of the result; fp16 weights may be
          subnormal: 2^-25 sum |x|
  SwiGLU  errors dg, du of the two products give 1.1 dg |u| + |silu(g)| du + 1.1 dg du (|silu'| < 1.1), the fp32
          exponential and division (2 + 1.2 |g| + 4) 2^-23 relative
"""
import ctypes
import math

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def wq():
    import bit_gemv_gemm_group_b200 as m
    return m


# ------------------------------------------------------------------------------------------------ refusals (CPU)
FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


def _route(wq, logits=FAKE, dtype=0, T=4, E=8, k=2, ws=FAKE, slots=FAKE):
    return wq.lib.wq_moe_route(logits, dtype, T, E, k, 1, FAKE, FAKE, FAKE, FAKE, slots, ws, None)


def test_route_refusals(wq):
    inv, una, mis = wq.WQ_ERR_INVALID_ARG, wq.WQ_ERR_UNSUPPORTED, wq.WQ_ERR_ALIGNMENT
    assert _route(wq, logits=None) == inv
    assert _route(wq, slots=ODD) == mis
    assert _route(wq, T=0) == inv and _route(wq, E=0) == inv and _route(wq, k=0) == inv
    assert _route(wq, dtype=5) == inv
    assert _route(wq, k=9) == inv                      # top_k > E
    assert _route(wq, E=513) == una and _route(wq, E=64, k=33) == una
    assert _route(wq, T=(1 << 23) + 1, k=1) == una and _route(wq, T=1 << 23, E=512, k=32, ws=None) == inv
    assert _route(wq, T=129, ws=None) == inv           # needs a workspace


def test_route_workspace(wq):
    assert wq.moe_route_workspace_bytes(64, 64) == 0 and wq.moe_route_workspace_bytes(0, 64) == 0
    # 16-bit counts of every block (16 tokens each, doubled until 256 blocks cover T), experts padded to 8
    assert wq.moe_route_workspace_bytes(129, 64) == 9 * 64 * 2
    assert wq.moe_route_workspace_bytes(130, 9) == 9 * 16 * 2
    assert wq.moe_route_workspace_bytes(16 * 256, 8) == 256 * 8 * 2
    assert wq.moe_route_workspace_bytes(16 * 256 + 1, 8) == 129 * 8 * 2


def _w4(wq, x=FAKE, T=4, rows=FAKE, off=FAKE, R=8, E=2, N=64, K=256, g=128, sw=0, y=FAKE, bf=False):
    fn = wq.lib.wq_grouped_gemm_w4a16_bf16 if bf else wq.lib.wq_grouped_gemm_w4a16
    return fn(x, T, rows, off, R, FAKE, FAKE, FAKE, E, N, K, g, sw, y, None)


def _w8(wq, xq=FAKE, T=4, rows=FAKE, off=FAKE, R=8, E=2, N=64, K=256, sw=0, y=FAKE, fp8=False):
    if fp8:
        return wq.lib.wq_grouped_gemm_fp8(xq, FAKE, 1, T, rows, off, R, FAKE, FAKE, 1, E, N, K, sw, y, None)
    return wq.lib.wq_grouped_gemm_w8a8(xq, FAKE, T, rows, off, R, FAKE, FAKE, E, N, K, sw, y, None)


@pytest.mark.parametrize("bf", [False, True])
def test_w4_refusals(wq, bf):
    inv, una, mis = wq.WQ_ERR_INVALID_ARG, wq.WQ_ERR_UNSUPPORTED, wq.WQ_ERR_ALIGNMENT
    call = lambda **k: _w4(wq, bf=bf, **k)  # noqa: E731
    assert call(x=None) == inv and call(off=None) == inv and call(y=ODD) == mis and call(rows=ODD) == mis
    for k in ("T", "R", "E", "N", "K"):
        assert call(**{k: 0}) == inv
    assert call(g=96) == una and call(K=192) == inv and call(E=513) == una
    assert call(rows=None) == inv                      # R != T without rows
    assert call(N=63, sw=1) == inv
    assert call(E=512, N=1 << 23) == una and call(K=1 << 30) == una and call(R=(1 << 29) + 1) == una


@pytest.mark.parametrize("fp8", [False, True])
def test_w8_refusals(wq, fp8):
    inv, una, mis = wq.WQ_ERR_INVALID_ARG, wq.WQ_ERR_UNSUPPORTED, wq.WQ_ERR_ALIGNMENT
    call = lambda **k: _w8(wq, fp8=fp8, **k)  # noqa: E731
    assert call(xq=None) == inv and call(off=ODD) == mis and call(y=None) == inv
    for k in ("T", "R", "E", "N", "K"):
        assert call(**{k: 0}) == inv
    assert call(K=24) == una and call(E=513) == una and call(rows=None) == inv and call(N=63, sw=1) == inv
    if not fp8:
        assert call(K=131072) == una


def test_combine_refusals(wq):
    inv, mis = wq.WQ_ERR_INVALID_ARG, wq.WQ_ERR_ALIGNMENT
    call = lambda y=FAKE, dt=1, R=8, T=4, k=2, N=64, out=FAKE: wq.lib.wq_moe_combine(  # noqa: E731
        y, dt, R, FAKE, FAKE, T, k, N, out, None)
    assert call(y=None) == inv and call(out=ODD) == mis and call(dt=0) == inv
    assert call(R=0) == inv and call(T=0) == inv and call(k=0) == inv and call(N=0) == inv


def test_outputs_that_overlap_inputs_are_refused(wq):
    """The sizes are known, so an output inside, across the start or across the end of an input is an error."""
    at = lambda o: ctypes.c_void_p(0x1000000 + o)  # noqa: E731
    far = [ctypes.c_void_p((i + 2) << 32) for i in range(8)]
    inv = wq.WQ_ERR_INVALID_ARG
    T, R, E, N, K = 4, 8, 2, 64, 256
    x4, w4, x8, w8, out = T * K * 2, E * N * K // 2, T * K, E * N * K, R * N * 2
    for sizes, call in (
            ((x4, 32, 12, w4, E * N * 4, E * N * 4), lambda y, p: wq.lib.wq_grouped_gemm_w4a16(
                p[0], T, p[1], p[2], R, p[3], p[4], p[5], E, N, K, 128, 0, y, None)),
            ((x8, 32, 12, w8, T * 4, E * N * 4), lambda y, p: wq.lib.wq_grouped_gemm_w8a8(
                p[0], p[4], T, p[1], p[2], R, p[3], p[5], E, N, K, 0, y, None)),
            ((x8, 32, 12, w8, 4, E * 4), lambda y, p: wq.lib.wq_grouped_gemm_fp8(
                p[0], p[4], 0, T, p[1], p[2], R, p[3], p[5], 0, E, N, K, 0, y, None)),
            ((R * N * 2, T * 2 * 4, T * 2 * 4), lambda y, p: wq.lib.wq_moe_combine(p[0], 1, R, p[1], p[2], T, 2, N, y, None))):
        for i, size in enumerate(sizes):
            p = list(far)
            p[i] = at(0)
            last = (size - 1) // 16 * 16
            y_bytes = out if len(sizes) == 6 else T * N * 2
            for o in (0, last, 16 - y_bytes):
                assert call(at(o), p) == inv, (i, o)
                assert b"overlaps" in wq.lib.wq_last_error()


# ------------------------------------------------------------------------------------------------ router
def route_ref(logits, k, renorm):
    x = logits.double().cpu().numpy()
    T, E = x.shape
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        ok = np.where(~np.isnan(x[t]) & (x[t] > -np.inf))[0]
        order = ok[np.argsort(-x[t][ok], kind="stable")]
        m = min(k, len(order))
        if m == 0:
            continue
        ids[t, :m] = order[:m]
        top = x[t][order[0]]
        with np.errstate(invalid="ignore"):
            e = np.where(x[t][order] == top, 1.0, np.exp(x[t][order] - top))
        w[t, :m] = e[:m] / (e[:m].sum() if renorm else e.sum())
    flat = ids.reshape(-1)
    pairs = np.concatenate([np.where(flat == e)[0] for e in range(E)]).astype(np.int64)
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])]).astype(np.int32)
    rows = np.full(T * k, -1, np.int32)
    slots = np.full(T * k, -1, np.int32)
    rows[:len(pairs)] = pairs // k
    slots[pairs] = np.arange(len(pairs))
    return ids, w, offsets, rows, slots.reshape(T, k)


def check_route(got, logits, k, renorm):
    ref = route_ref(logits, k, renorm)
    for i, name in ((0, "ids"), (2, "offsets"), (3, "rows"), (4, "slots")):
        assert np.array_equal(got[i].cpu().numpy(), ref[i]), name
    # expf is within 2 units (2^-22), the argument's subtraction rounds by 2^-24 |l - top| (at most 2^-24 * 200
    # before the term underflows), sums of at most 512 terms and a division: 2^-15 covers all of it
    err = np.abs(got[1].cpu().numpy().astype(np.float64) - ref[1])
    assert np.all(err <= 2.0 ** -15 * ref[1] + 1e-37)


@gpu
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (32, 64, 8), (64, 128, 8), (65, 128, 8), (128, 128, 8), (129, 128, 8),
                                   (700, 33, 3), (1000, 512, 32), (257, 500, 7), (4096, 130, 4), (16 * 256 + 5, 64, 8),
                                   (128 * 256 + 77, 16, 2), (200000, 24, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_route(wq, T, E, k, dtype):
    g = torch.Generator().manual_seed(T * 1000 + E)
    logits = (torch.randn(T, E, generator=g) * 2).to(dtype).cuda()
    for renorm in (True, False):
        check_route(wq.moe_route(logits, k, renormalize=renorm), logits, k, renorm)


@gpu
@pytest.mark.parametrize("T", [40, 300])
def test_route_masked_and_special(wq, T):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, 24, generator=g)
    x[:, 5] = -math.inf
    x[0] = -math.inf                                   # nothing selectable
    x[1] = math.nan
    x[2, 3:] = -math.inf                               # fewer than k
    x[3] = torch.finfo(torch.float32).min              # the lowest finite value is selectable
    x[4, 2] = math.nan
    x[5, 7], x[5, 9] = math.inf, math.inf
    x[6] = 0.0
    x[6, ::2] = -0.0                                   # equal: the lowest index first
    x[7, 3] = math.inf
    x[8] = 1e30
    x[9, 0] = -1e38
    x[10:20] = -math.inf
    for k in (1, 4, 24):
        for renorm in (True, False):
            check_route(wq.moe_route(x.cuda(), k, renormalize=renorm), x, k, renorm)
    everything = torch.full((T, 24), -math.inf)
    check_route(wq.moe_route(everything.cuda(), 3), everything, 3, True)
    same = torch.zeros(T, 24)                          # every token to the same experts
    check_route(wq.moe_route(same.cuda(), 3), same, 3, True)


# ------------------------------------------------------------------------------------------------ expert products
FORMATS = ["w8a8", "fp8", "fp16", "bf16"]
SENTINEL = 77.0


def make_weights(kind, E, N, K, group, seed):
    """(arguments of the call after x, fp64 weights [E, N, K])."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind in ("fp16", "bf16"):
        G = K // group
        codes = torch.randint(0, 16, (E, N, K), device="cuda", generator=g)
        zeros = torch.randint(0, 16, (E, N, G), device="cuda", generator=g)
        scales = torch.exp(torch.randn(E, N, G, device="cuda", generator=g) * 0.5 - 5).half()

        def pack(c):
            pad = (-c.shape[-1]) % 8
            c = torch.nn.functional.pad(c, (0, pad)).view(*c.shape[:-1], -1, 8).long()
            v = (c << torch.arange(0, 32, 4, device="cuda")).sum(-1)
            return torch.where(v >= 2 ** 31, v - 2 ** 32, v).to(torch.int32)

        w = (codes.double() - zeros.double().repeat_interleave(group, -1)) * scales.double().repeat_interleave(group, -1)
        return (pack(codes), scales, pack(zeros)), w
    sw = torch.exp(torch.randn(E, N, device="cuda", generator=g) * 0.5 - 5)
    if kind == "w8a8":
        q = torch.randint(-128, 128, (E, N, K), device="cuda", generator=g).to(torch.int8)
        return (q, sw * 2.0 ** -6), q.double() * (sw * 2.0 ** -6).double()[..., None]
    q = (torch.randn(E, N, K, device="cuda", generator=g) * 40).clamp(-448, 448).to(torch.float8_e4m3fn)
    return (q.view(torch.uint8), sw), q.double() * sw.double()[..., None]


def make_x(kind, T, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    if kind in ("fp16", "bf16"):
        x = torch.randn(T, K, device="cuda", generator=g).to(torch.float16 if kind == "fp16" else torch.bfloat16)
        return (x,), x.double()
    sx = torch.exp(torch.randn(T, device="cuda", generator=g) * 0.3 - 3)
    if kind == "w8a8":
        q = torch.randint(-128, 128, (T, K), device="cuda", generator=g).to(torch.int8)
        return (q, sx), q.double() * sx.double()[:, None]
    q = torch.randn(T, K, device="cuda", generator=g).to(torch.float8_e4m3fn)
    return (q.view(torch.uint8), sx), q.double() * sx.double()[:, None]


def product_ref(kind, x, w, rows, off, R, K, swiglu):
    """(y, tolerance, written) in fp64 for the sorted rows; x [T, K] and w [E, N, K] in fp64."""
    E, N, _ = w.shape
    y = torch.zeros(R, N // 2 if swiglu else N, dtype=torch.float64, device="cuda")
    tol, written = torch.zeros_like(y), torch.zeros(R, dtype=torch.bool, device="cuda")
    u = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi <= lo:
            continue
        src = rows[lo:hi].long() if rows is not None else torch.arange(lo, hi, device="cuda")
        good = (src >= 0) & (src < x.shape[0])
        xe = torch.where(good[:, None], x[src.clamp(0, x.shape[0] - 1)], 0.0)
        d, s = xe @ w[e].T, xe.abs() @ w[e].abs().T
        if kind == "w8a8":
            dd = d.abs() * 2.0 ** -22
        elif kind == "fp8":
            dd = d.abs() * 2.0 ** -22 + K * 2.0 ** -23 * s
        else:
            dd = (u + K * 2.0 ** -23) * s + (2.0 ** -25 * xe.abs().sum(1, keepdim=True) if kind == "fp16" else 0)
        if swiglu:
            g, l, dg, dl = d[:, :N // 2], d[:, N // 2:], dd[:, :N // 2], dd[:, N // 2:]
            sg = g * torch.sigmoid(g)
            v = sg * l
            t = 1.1 * dg * l.abs() + sg.abs() * dl + 1.1 * dg * dl + (6 + 1.2 * g.abs()) * 2.0 ** -23 * v.abs()
        else:
            v, t = d, dd
        y[lo:hi], written[lo:hi] = v, True
        tol[lo:hi] = t + (v.abs() + t) * u + 2.0 ** -25
    return y, tol, written


def call(wq, kind, xa, wa, off, rows, group, swiglu, out=None, stream=None):
    if kind in ("fp16", "bf16"):
        return wq.grouped_gemm_w4a16(*xa, *wa, off, rows, group, swiglu, out, stream)
    fn = wq.grouped_gemm_w8a8 if kind == "w8a8" else wq.grouped_gemm_fp8
    return fn(*xa, *wa, off, rows, swiglu, out, stream)


def check_product(wq, kind, counts, T, N, K, group=32, swiglu=False, gather=True, start=0, spare=0, seed=0, bad=False,
                  extremes=False):
    E = len(counts)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + start, dtype=torch.int32, device="cuda")
    R = int(off[-1]) + spare
    if not gather:
        T = R
    wa, w = make_weights(kind, E, N, K, group, seed)
    xa, x = make_x(kind, T, K, seed)
    rows = None
    if gather:
        g = torch.Generator(device="cuda").manual_seed(seed + 2)
        rows = torch.randint(0, T, (R,), device="cuda", generator=g).to(torch.int32)  # the same token many times
        if bad:
            rows[::5] = torch.tensor([-1, T, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32,
                                     device="cuda").repeat(R)[:rows[::5].numel()]
    dt = torch.bfloat16 if kind == "bf16" else torch.float16
    out = torch.full((R, N // 2 if swiglu else N), SENTINEL, dtype=dt, device="cuda")
    got = call(wq, kind, xa, wa, off, rows, group, swiglu, out)
    assert got.data_ptr() == out.data_ptr()
    assert wq.device_status() == 0
    y, tol, written = product_ref(kind, x, w, rows, off.cpu(), R, K, swiglu)
    err = (got.double() - y).abs()
    over = (err > tol) & written[:, None]
    assert not over.any(), (f"{int(over.sum())} of {int(written.sum()) * y.shape[1]} outside; worst "
                            f"{float((err / tol)[over].max()):.3g} of the tolerance at {over.nonzero()[:4].tolist()}")
    assert torch.equal(got[~written], torch.full_like(got[~written], SENTINEL)), "a row outside the experts was written"
    again = call(wq, kind, xa, wa, off, rows, group, swiglu, out.clone())
    assert torch.equal(again[written], got[written]), "not repeatable"
    return got


@gpu
@pytest.mark.parametrize("kind", FORMATS)
@pytest.mark.parametrize("counts,N,K", [
    ([1], 1, 32), ([3], 128, 128), ([0, 0, 5, 0], 130, 160), ([15, 16, 17, 1, 0, 33], 256, 512),
    ([255, 0, 256, 257], 100, 288), ([600, 1], 384, 1024), ([2] * 70, 66, 96)])
@pytest.mark.parametrize("gather", [True, False])
def test_products(wq, kind, counts, N, K, gather):
    check_product(wq, kind, counts, T=37, N=N, K=K, gather=gather)


@gpu
@pytest.mark.parametrize("kind", FORMATS)
@pytest.mark.parametrize("counts,N,K", [([1, 2], 2, 64), ([9, 0, 40], 128, 256), ([300, 7], 258, 480), ([5] * 20, 100, 96)])
@pytest.mark.parametrize("gather", [True, False])
def test_products_swiglu(wq, kind, counts, N, K, gather):
    check_product(wq, kind, counts, T=50, N=N, K=K, swiglu=True, gather=gather)


@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("K", [256, 1280, 2304])
def test_products_group_sizes(wq, kind, group, K):
    check_product(wq, kind, [4, 0, 70, 129], T=64, N=200, K=K, group=group)
    check_product(wq, kind, [4, 0, 3, 1], T=64, N=200, K=K, group=group, swiglu=True)


@gpu
@pytest.mark.parametrize("kind", ["w8a8", "fp8"])
@pytest.mark.parametrize("K", [16, 48, 1360, 4112])
def test_products_odd_depth(wq, kind, K):
    check_product(wq, kind, [7, 100, 0, 2], T=64, N=150, K=K, swiglu=True)


@gpu
@pytest.mark.parametrize("kind", FORMATS)
@pytest.mark.parametrize("counts", [[3, 0, 4], [90, 200]])
def test_rows_outside_are_left_and_bad_rows_are_zero(wq, kind, counts):
    check_product(wq, kind, counts, T=40, N=72, K=128, start=5, spare=9)
    got = check_product(wq, kind, counts, T=40, N=72, K=128, bad=True)
    assert float(got[0].float().abs().max()) == 0.0     # rows[0] is -1
    check_product(wq, kind, counts, T=40, N=72, K=128, bad=True, swiglu=True)


@gpu
@pytest.mark.parametrize("kind", FORMATS)
def test_bad_offsets_stay_in_bounds(wq, kind):
    """Offsets out of range or decreasing are clamped to [0, R] and made non-decreasing."""
    R, N, K = 40, 64, 128
    wa, w = make_weights(kind, 4, N, K, 32, 3)
    xa, x = make_x(kind, R, K, 3)
    for raw in ([-7, 10, 5, 2000, 30], [50, 60, 70, 80, 90], [0, -1, -2, -3, 2 ** 31 - 1]):
        fixed = np.maximum.accumulate(np.clip(raw, 0, R))
        off = torch.tensor(raw, dtype=torch.int32, device="cuda")
        dt = torch.bfloat16 if kind == "bf16" else torch.float16
        out = torch.full((R, N), SENTINEL, dtype=dt, device="cuda")
        call(wq, kind, xa, wa, off, None, 32, False, out)
        y, tol, written = product_ref(kind, x, w, None, fixed, R, K, False)
        assert ((out.double() - y).abs() <= tol)[written].all()
        assert (out[~written] == SENTINEL).all()


@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp8"])
def test_nan_and_inf_stay_in_their_row(wq, kind):
    counts, T, N, K = [5, 30], 35, 96, 256
    wa, w = make_weights(kind, 2, N, K, 32, 9)
    xa, x = make_x(kind, T, K, 9)
    dirty = xa[0].clone()
    if kind == "fp8":
        dirty[3, 10] = 0x7F
        dirty[20] = 0xFF
    else:
        dirty[3, 10] = math.nan
        dirty[20, 0] = math.inf
    off = torch.tensor([0, 5, 35], dtype=torch.int32, device="cuda")
    clean_y = call(wq, kind, xa, wa, off, None, 32, False)
    y = call(wq, kind, (dirty, *xa[1:]), wa, off, None, 32, False)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[3] = keep[20] = False
    assert torch.equal(y[keep], clean_y[keep])
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[20]).any()


@gpu
def test_fp8_scalar_scales(wq):
    """sx [1] and sw [E]: per tensor and per expert."""
    E, N, K, T = 3, 80, 256, 30
    (q, _), _ = make_weights("fp8", E, N, K, 32, 4)
    (xq, _), _ = make_x("fp8", T, K, 4)
    sx, sw = torch.tensor([0.03], device="cuda"), torch.tensor([0.01, 0.02, 0.005], device="cuda")
    off = torch.tensor([0, 11, 11, 30], dtype=torch.int32, device="cuda")
    for swiglu in (False, True):
        y = wq.grouped_gemm_fp8(xq, sx, q, sw, off, swiglu=swiglu)
        full = wq.grouped_gemm_fp8(xq, sx.expand(T).contiguous(), q, sw[:, None].expand(E, N).contiguous(), off,
                                   swiglu=swiglu)
        assert torch.equal(y, full)
        x64 = xq.view(torch.float8_e4m3fn).double() * sx.double()
        w64 = q.view(torch.float8_e4m3fn).double() * sw.double()[:, None, None]
        ref, tol, written = product_ref("fp8", x64, w64, None, off.cpu(), T, K, swiglu)
        assert ((y.double() - ref).abs() <= tol)[written].all()


# INT4 by rows per expert: fewer than 7 on average, and below 22.  N for E experts such that there are tiles enough for
# each of the shapes that the first of them takes.
HANDFUL = [1, 8, 0, 9, 3, 2, 17, 1]
FEW = [9, 0, 40, 7]


@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("group,K", [(32, 32), (32, 416), (64, 1088), (128, 128), (128, 1152), (256, 1280), (256, 2304)])
@pytest.mark.parametrize("N,swiglu", [(70, False), (62, True), (1250, False), (1262, True), (4757, False), (4802, True)])
def test_products_of_a_handful_of_rows(wq, kind, group, K, N, swiglu):
    check_product(wq, kind, HANDFUL, T=40, N=N, K=K, group=group, swiglu=swiglu)


@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("N", [70, 1250, 4757])
def test_a_handful_of_rows_in_order_and_bad_ones(wq, kind, N):
    check_product(wq, kind, HANDFUL, T=40, N=N, K=480, gather=False)
    check_product(wq, kind, HANDFUL, T=40, N=N, K=480, start=2, spare=3)
    check_product(wq, kind, HANDFUL, T=40, N=N, K=480, bad=True)
    check_product(wq, kind, HANDFUL, T=1, N=N + N % 2, K=480, bad=True, swiglu=True)
    check_product(wq, kind, [0] * 300 + [1] + [0] * 211, T=3, N=N, K=64)        # the most experts


@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("group,K", [(32, 416), (64, 1088), (128, 2304), (256, 1280)])
@pytest.mark.parametrize("N,swiglu", [(200, False), (200, True)])
def test_products_of_few_rows(wq, kind, group, K, N, swiglu):
    check_product(wq, kind, FEW, T=40, N=N, K=K, group=group, swiglu=swiglu)
    check_product(wq, kind, FEW, T=40, N=N, K=K, group=group, swiglu=swiglu, bad=True, spare=3)


@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_a_handful_of_rows_with_bad_offsets(wq, kind):
    R, E, N, K = 40, 8, 64, 128
    wa, w = make_weights(kind, E, N, K, 32, 3)
    xa, x = make_x(kind, R, K, 3)
    for raw in ([-7, 10, 5, 2000, 30, 1, 2, 3, 4], [50, 60, 70, 80, 90, 1, 1, 1, 1], [0, -1, -2, -3, 9, 9, 8, 7, 2 ** 31 - 1]):
        fixed = np.maximum.accumulate(np.clip(raw, 0, R))
        off = torch.tensor(raw, dtype=torch.int32, device="cuda")
        out = torch.full((R, N), SENTINEL, dtype=xa[0].dtype, device="cuda")
        call(wq, kind, xa, wa, off, None, 32, False, out)
        y, tol, written = product_ref(kind, x, w, None, fixed, R, K, False)
        assert ((out.double() - y).abs() <= tol)[written].all()
        assert (out[~written] == SENTINEL).all()


@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("counts", [[5, 1, 3, 0], [20, 2, 9, 0]])
def test_nan_and_inf_beside_few_rows(wq, kind, counts):
    """A row's NaN or infinity stays in its sums, also when it is row 0 and other indices lie outside x."""
    N, K, T = 96, 256, 12
    wa, w = make_weights(kind, 4, N, K, 64, 9)
    (x,), _ = make_x(kind, T, K, 9)
    dirty = x.clone()
    dirty[0, 3] = math.nan
    dirty[5, 0] = math.inf
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    R = sum(counts)
    rows = (torch.arange(R, device="cuda") % T).to(torch.int32)
    rows[3], rows[R - 1] = -1, T
    clean_y = call(wq, kind, (x,), wa, off, rows, 64, False)
    y = call(wq, kind, (dirty,), wa, off, rows, 64, False)
    keep = (rows != 0) & (rows != 5)
    assert torch.equal(y[keep], clean_y[keep])
    assert torch.isnan(y[rows == 0]).all() and not torch.isfinite(y[rows == 5]).any()
    assert (y[3] == 0).all() and (y[R - 1] == 0).all()
    # One infinity: each sum has the sign of its weight, or is NaN where the weight is zero.
    expert = torch.searchsorted(off.long(), torch.arange(R, device="cuda"), right=True) - 1
    for p in (rows == 5).nonzero().flatten().tolist():
        s = torch.sign(w[expert[p], :, 0])
        assert torch.equal(torch.nan_to_num(torch.sign(y[p].double()), 0.0), s)


@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("counts", [[2, 1], [12, 9]])
@pytest.mark.parametrize("group,K", [(32, 160), (64, 192), (128, 384)])
def test_infinite_scales_beside_the_end_of_few_rows(wq, kind, counts, group, K):
    """The last group's scale is infinite: sums get its sign, also where the depth ends inside a step of the kernel."""
    N, T = 40, sum(counts)
    (q, s, z), _ = make_weights(kind, 2, N, K, group, 4)
    (x,), x64 = make_x(kind, T, K, 4)
    s = s.clone()
    s[:, ::2, -1] = math.inf
    off = torch.tensor([0, counts[0], T], dtype=torch.int32, device="cuda")
    y = wq.grouped_gemm_w4a16(x, q, s, z, off, group_size=group)
    nibbles = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    codes = ((q.unsqueeze(-1) >> nibbles) & 15).view(2, N, K).double()
    zeros = ((z.unsqueeze(-1) >> nibbles) & 15).view(2, N, -1)[..., :K // group].double()
    last = codes[..., -group:] - zeros[..., -1:]
    for p in range(T):
        d = last[0 if p < counts[0] else 1] @ x64[p, -group:]
        assert torch.equal(y[p, ::2].double(), torch.sign(d[::2]) * math.inf)
        assert torch.isfinite(y[p, 1::2]).all()


@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("R,K,N", [(20, 512, 136), (20, 512, 2000), (20, 512, 9500), (60, 512, 136), (60, 4096, 136)])
def test_few_rows_graph_replay_with_new_routing(wq, kind, R, K, N):
    T, E = 60, 5
    wa, w = make_weights(kind, E, N, K, 128, 8)
    xa, x = make_x(kind, T, K, 8)
    off = torch.tensor([0, 2, 2, 9, 10, R], dtype=torch.int32, device="cuda")
    rows = torch.randint(0, T, (R,), device="cuda", dtype=torch.int32)
    out = torch.full((R, N), SENTINEL, dtype=xa[0].dtype, device="cuda")
    call(wq, kind, xa, wa, off, rows, 128, False, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(wq, kind, xa, wa, off, rows, 128, False, out)
    for new in ([0, R, R, R, R, R], [0, 1, 2, 3, 4, 5], [10, 10, 10, 10, 10, 10], [0, 4, 8, 12, 16, R - 1]):
        off.copy_(torch.tensor(new, dtype=torch.int32))
        rows.copy_(torch.randint(0, T, (R,), dtype=torch.int32))
        out.fill_(SENTINEL)
        graph.replay()
        y, tol, written = product_ref(kind, x, w, rows, off.cpu(), R, K, False)
        assert ((out.double() - y).abs() <= tol)[written].all()
        assert (out[~written] == SENTINEL).all()


@gpu
@pytest.mark.parametrize("counts,N", [(HANDFUL, 70), (HANDFUL, 1250), (HANDFUL, 4757), (FEW, 200)])
def test_few_rows_on_two_streams(wq, counts, N):
    """Two calls of one kernel that overlap on the GPU share nothing."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    R, cases = int(off[-1]), []
    for i in range(2):
        wa, _ = make_weights("fp16", len(counts), N, 2304, 128, i)
        xa, _ = make_x("fp16", 30, 2304, i)
        rows = torch.randint(0, 30, (R,), device="cuda", dtype=torch.int32)
        cases.append((xa, wa, rows, call(wq, "fp16", xa, wa, off, rows, 128, False)))
    torch.cuda.synchronize()
    for _ in range(20):
        got = [call(wq, "fp16", xa, wa, off, rows, 128, False, stream=st) for (xa, wa, rows, _), st in zip(cases, streams)]
        torch.cuda.synchronize()
        for y, c in zip(got, cases):
            assert torch.equal(y, c[3])


@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_few_rows_waits_that_run_out(wq, kind):
    """As above, for INT4 experts with 7 to 22 rows."""
    N, K, counts = 640, 2048, [30, 9, 0, 5]
    wa, _ = make_weights(kind, 4, N, K, 128, 2)
    T = sum(counts)
    xa, _ = make_x(kind, T, K, 2)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    good = call(wq, kind, xa, wa, off, None, 128, False)
    try:
        wq.set_wait_limit(1)
        for _ in range(3):
            call(wq, kind, xa, wa, off, None, 128, False)
        assert wq.device_status() in (wq.WQ_OK, wq.WQ_ERR_TIMEOUT)
    finally:
        wq.set_wait_limit(0)
    assert torch.equal(call(wq, kind, xa, wa, off, None, 128, False), good)
    assert wq.device_status() == 0


@gpu
@pytest.mark.parametrize("kind", FORMATS)
def test_one_expert_equals_the_dense_product(wq, kind):
    """E = 1 with every row is the dense matmul the library offers already."""
    T, N, K = 64, 256, 512
    wa, _ = make_weights(kind, 1, N, K, 128, 5)
    xa, _ = make_x(kind, T, K, 5)
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    y = call(wq, kind, xa, wa, off, None, 128, False)
    dense = [t[0].contiguous() for t in wa]
    if kind == "w8a8":
        assert torch.equal(y, wq.gemm_w8a8(*xa, *dense))
    elif kind == "fp8":
        d = wq.gemm_fp8(*xa, *dense)
        assert torch.allclose(y.float(), d.float(), rtol=2.0 ** -9, atol=1e-3)
    else:
        d = wq.gemm_w4a16(*xa, *dense, 128) if kind == "fp16" else wq.gemm_w4a16_bf16(*xa, *dense, 128)
        u = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
        x64, q, s, z = xa[0].double(), *dense
        codes = ((q.view(N, -1, 1) >> torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)) & 15).view(N, K)
        zer = ((z.view(N, -1, 1) >> torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)) & 15).view(N, -1)[:, :K // 128]
        w = (codes.double() - zer.double().repeat_interleave(128, 1)) * s.double().repeat_interleave(128, 1)
        bound = x64.abs() @ w.abs().T
        assert ((y.double() - d.double()).abs() <= 4 * u * bound + 2.0 ** -24).all()


@gpu
@pytest.mark.parametrize("kind", FORMATS)
def test_products_graph_replay_with_new_routing(wq, kind):
    """A captured call follows the offsets and rows in memory at replay."""
    N, K, T, R, E = 136, 256, 60, 120, 5
    wa, w = make_weights(kind, E, N, K, 32, 8)
    xa, x = make_x(kind, T, K, 8)
    off = torch.tensor([0, 20, 20, 90, 100, 120], dtype=torch.int32, device="cuda")
    rows = torch.randint(0, T, (R,), device="cuda", dtype=torch.int32)
    dt = torch.bfloat16 if kind == "bf16" else torch.float16
    out = torch.full((R, N), SENTINEL, dtype=dt, device="cuda")
    call(wq, kind, xa, wa, off, rows, 32, False, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(wq, kind, xa, wa, off, rows, 32, False, out)
    for new in ([0, 120, 120, 120, 120, 120], [0, 1, 2, 3, 4, 5], [10, 10, 10, 10, 10, 10], [0, 24, 48, 72, 96, 119]):
        off.copy_(torch.tensor(new, dtype=torch.int32))
        rows.copy_(torch.randint(0, T, (R,), dtype=torch.int32))
        out.fill_(SENTINEL)
        graph.replay()
        y, tol, written = product_ref(kind, x, w, rows, off.cpu(), R, K, False)
        assert ((out.double() - y).abs() <= tol)[written].all()
        assert (out[~written] == SENTINEL).all()


@gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("counts", [[3, 9], [70, 50]])
def test_products_tiny_and_mixed_values(wq, kind, counts):
    """Subnormal activations and scales, and values near the largest, keep their precision."""
    N, K, group = 96, 512, 64
    (q, s, z), _ = make_weights(kind, 2, N, K, group, 6)
    T = sum(counts)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, K, device="cuda", generator=g)
    x[: T // 2] *= 2.0 ** -18                            # fp16 subnormals
    x[T // 2:, ::7] *= 1000.0
    x = x.to(torch.float16 if kind == "fp16" else torch.bfloat16)
    s = s.clone()
    s[0, ::3] = 2.0 ** -20                               # a subnormal fp16 scale
    codes = ((q.unsqueeze(-1) >> torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)) & 15).view(2, N, K).double()
    zeros = ((z.unsqueeze(-1) >> torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)) & 15).view(2, N, -1)
    zeros = zeros[..., :K // group].double().repeat_interleave(group, -1)
    w = (codes - zeros) * s.double().repeat_interleave(group, -1)
    off = torch.tensor([0, counts[0], T], dtype=torch.int32, device="cuda")
    y = wq.grouped_gemm_w4a16(x, q, s, z, off, group_size=group)
    ref, tol, written = product_ref(kind, x.double(), w, None, off.cpu(), T, K, False)
    assert ((y.double() - ref).abs() <= tol)[written].all()


@gpu
@pytest.mark.parametrize("kind", FORMATS)
@pytest.mark.parametrize("counts", [[3, 9, 0, 5], [300, 40, 0, 180]])
def test_waits_that_run_out_leave_the_context_usable(wq, kind, counts):
    """Under a limit of a nanosecond the kernels finish or give up; afterwards the same call gives the same result."""
    N, K = 640, 2048
    wa, _ = make_weights(kind, 4, N, K, 128, 2)
    T = sum(counts)
    xa, _ = make_x(kind, T, K, 2)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    rows = torch.randperm(T, device="cuda").to(torch.int32)
    good = [call(wq, kind, xa, wa, off, r, 128, False) for r in (rows, None)]
    assert wq.device_status() == 0
    try:
        wq.set_wait_limit(1)
        for _ in range(3):
            for r in (rows, None):
                call(wq, kind, xa, wa, off, r, 128, False)
        assert wq.device_status() in (wq.WQ_OK, wq.WQ_ERR_TIMEOUT)
    finally:
        wq.set_wait_limit(0)
    for r, y in zip((rows, None), good):
        assert torch.equal(call(wq, kind, xa, wa, off, r, 128, False), y)
    assert wq.device_status() == 0


@gpu
def test_calls_on_two_streams(wq):
    """Calls that overlap on the GPU share nothing."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    cases = []
    for i, kind in enumerate(["w8a8", "fp16"]):
        wa, _ = make_weights(kind, 8, 512, 1024, 128, i)
        xa, _ = make_x(kind, 100, 1024, i)
        off = torch.tensor([0, 3, 50, 50, 120, 130, 260, 280, 300], dtype=torch.int32, device="cuda")
        rows = torch.randint(0, 100, (300,), device="cuda", dtype=torch.int32)
        cases.append((kind, xa, wa, off, rows, call(wq, kind, xa, wa, off, rows, 128, False)))
    torch.cuda.synchronize()
    for _ in range(20):
        got = [call(wq, k, xa, wa, off, rows, 128, False, stream=s) for (k, xa, wa, off, rows, _), s in zip(cases, streams)]
        torch.cuda.synchronize()
        for y, c in zip(got, cases):
            assert torch.equal(y, c[5])


@gpu
def test_output_past_32_bit_offsets(wq):
    """R * N over 2^31: the last rows land where they belong."""
    R, N, K, E = 140000, 16400, 16, 3
    (q, sw), w = make_weights("w8a8", E, N, K, 32, 1)
    xq = torch.randint(-128, 128, (R, K), device="cuda", dtype=torch.int8)
    sx = torch.full((R,), 0.01, device="cuda")
    off = torch.tensor([0, 70001, 139990, R], dtype=torch.int32, device="cuda")
    y = wq.grouped_gemm_w8a8(xq, sx, q, sw, off)
    for p, e in ((0, 0), (70000, 0), (70001, 1), (131071, 1), (139989, 1), (139990, 2), (R - 1, 2)):
        ref = (xq[p].double() * sx[p].double()) @ w[e].T
        assert ((y[p].double() - ref).abs() <= ref.abs() * (2.0 ** -11 + 2.0 ** -22) + 2.0 ** -25).all()


@gpu
@pytest.mark.parametrize("R", [2, 300, 900])
def test_int4_weights_past_32_bit_offsets(wq, R):
    """4.7 GB of codes: the last expert's rows, by each of the INT4 kernels (below 7, below 22 and more rows per expert)."""
    E, N, K, group = 40, 28672, 8192, 128
    g = torch.Generator(device="cuda").manual_seed(R)
    q = torch.randint(-2 ** 31, 2 ** 31, (E, N, K // 8), device="cuda", dtype=torch.int32, generator=g)
    s = torch.full((E, N, K // group), 2.0 ** -6, dtype=torch.float16, device="cuda")
    s[-1] = (torch.rand(N, K // group, device="cuda", generator=g) * 2.0 ** -6).half()
    z = torch.randint(-2 ** 31, 2 ** 31, (E, N, K // group // 8), device="cuda", dtype=torch.int32, generator=g)
    x = torch.randn(R, K, device="cuda", generator=g).half()
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = R
    y = wq.grouped_gemm_w4a16(x, q, s, z, off, group_size=group)
    at = torch.tensor([0, 1, 63, 64, 14335, 28671], device="cuda")
    nibbles = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    codes = ((q[-1, at].unsqueeze(-1) >> nibbles) & 15).view(len(at), K).double()
    zeros = ((z[-1, at].unsqueeze(-1) >> nibbles) & 15).view(len(at), -1).double()
    w = (codes - zeros.repeat_interleave(group, 1)) * s[-1, at].double().repeat_interleave(group, 1)
    ref, size = x.double() @ w.T, x.double().abs() @ w.abs().T
    u = 2.0 ** -11
    tol = (u + K * 2.0 ** -23) * size + 2.0 ** -25 * x.double().abs().sum(1, keepdim=True)
    assert ((y[:, at].double() - ref).abs() <= tol + (ref.abs() + tol) * u + 2.0 ** -25).all()


@gpu
@pytest.mark.parametrize("R", [5, 900])
def test_int8_weights_past_32_bit_offsets(wq, R):
    E, N, K = 20, 28672, 8192
    g = torch.Generator(device="cuda").manual_seed(R)
    q = torch.randint(-128, 128, (E, N, K), device="cuda", dtype=torch.int8, generator=g)
    sw = torch.rand(E, N, device="cuda", generator=g) * 2.0 ** -10
    x = torch.randint(-128, 128, (R, K), device="cuda", dtype=torch.int8, generator=g)
    sx = torch.full((R,), 2.0 ** -6, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = R
    y = wq.grouped_gemm_w8a8(x, sx, q, sw, off)
    at = torch.tensor([0, 127, 128, 28671], device="cuda")
    ref = (x.double() @ q[-1, at].double().T) * 2.0 ** -6 * sw[-1, at].double()
    assert ((y[:, at].double() - ref).abs() <= ref.abs() * (2.0 ** -11 + 2.0 ** -22) + 2.0 ** -25).all()


@gpu
def test_binding_checks(wq):
    wa, _ = make_weights("w8a8", 2, 64, 128, 32, 0)
    xa, _ = make_x("w8a8", 6, 128, 0)
    off = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        wq.grouped_gemm_w8a8(*xa, *wa, off[:2].contiguous())
    with pytest.raises(TypeError):
        wq.grouped_gemm_w8a8(*xa, *wa, off.long())
    with pytest.raises(ValueError):
        wq.grouped_gemm_w8a8(*xa, *wa, off, out=torch.empty(6, 63, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        wq.grouped_gemm_w8a8(xa[0][:, :64].contiguous(), xa[1], *wa, off)
    with pytest.raises(ValueError):
        wq.grouped_gemm_w8a8(*xa, *wa, off.cpu())
    with pytest.raises(ValueError):
        wq.moe_combine(torch.zeros(4, 8, dtype=torch.float16, device="cuda"), torch.zeros(2, 3, device="cuda"),
                       torch.zeros(2, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(wq.WQError):
        wq.moe_route(torch.zeros(4, 8, device="cuda"), 9)


# ------------------------------------------------------------------------------------------------ combine, layer
@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (7, 2, 8), (5, 3, 1030), (33, 8, 4096), (4, 9, 131), (2, 32, 12), (300, 4, 70)])
def test_combine(wq, dtype, T, k, N):
    g = torch.Generator(device="cuda").manual_seed(N)
    R = T * k + 3
    y = torch.randn(R, N, device="cuda", generator=g).to(dtype)
    weights = torch.randn(T, k, device="cuda", generator=g)
    slots = torch.randint(-1, R, (T, k), device="cuda", generator=g).to(torch.int32)
    slots[0, 0] = 2 ** 31 - 1                          # outside: adds nothing
    if T > 1:
        slots[1] = -1
    got = wq.moe_combine(y, weights, slots)
    inside = ((slots >= 0) & (slots < R))[..., None]
    rows = torch.where(inside, y.double()[slots.long().clamp(0, R - 1)], 0.0)
    terms = rows * weights.double()[..., None]
    ref, s = terms.sum(1), terms.abs().sum(1)
    u = torch.finfo(dtype).eps / 2
    tol = ref.abs() * u + (1 + u) * k * 2.0 ** -24 * s + 2.0 ** -25
    assert ((got.double() - ref).abs() <= tol).all()
    if T > 1:
        assert float(got[1].float().abs().max()) == 0.0


@gpu
@pytest.mark.parametrize("kind", ["w8a8", "fp16", "bf16"])
@pytest.mark.parametrize("T", [1, 5, 200])
def test_layer(wq, kind, T):
    """Router, products and combine as a model runs them, with padded tokens, eager and as one graph."""
    E, k, K, I, N = 12, 3, 256, 320, 192
    g = torch.Generator(device="cuda").manual_seed(T)
    logits = torch.randn(T, E, device="cuda", generator=g)
    if T > 4:
        logits[1] = -math.inf                          # a padded token: zeros
        logits[2, 2:] = -math.inf                      # fewer experts than k
    group = 64
    up, w1 = make_weights(kind, E, 2 * I, K, group, 1)
    down, w2 = make_weights(kind, E, N, I, group, 2)
    dt = torch.bfloat16 if kind == "bf16" else torch.float16
    x = torch.randn(T, K, device="cuda", generator=g).to(dt)
    if kind == "w8a8":
        run = lambda: wq.moe_mlp_w8a8(x, logits, up, down, k)  # noqa: E731
    else:
        run = lambda: wq.moe_mlp_w4a16(x, logits, up, down, k, group)  # noqa: E731
    got = run()
    ids, weights, _, _, _ = route_ref(logits.cpu(), k, True)
    ref = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e < 0:
                continue
            d = w1[e] @ x[t].double()
            h = d[:I] * torch.sigmoid(d[:I]) * d[I:]
            ref[t] += weights[t, j] * (w2[e] @ h)
    # The rounding between the products dominates: INT8 per token is off by at most half a step of max|h| / 127, rms
    # max|h| / (127 sqrt(12)), 0.03 of h at max|h| = 13 rms (SwiGLU has long tails); bf16 2^-8 and fp16 2^-11 a step,
    # weights, h, y and out each: four of them, and the gate's slope near 1.
    rel = float((got.double() - ref).norm() / ref.norm())
    assert rel < (0.05 if kind == "w8a8" else 0.02 if kind == "bf16" else 0.003)
    if T > 4:
        assert float(got[1].float().abs().max()) == 0.0
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    graph.replay()
    assert torch.equal(out, got)
    assert wq.device_status() == 0
