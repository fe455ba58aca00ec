"""Microscaled 4-bit tensors on the GPU: quantisation and dequantisation bit
for bit against the format in 64-bit NumPy (tests/_mx.py), the product within
the bound of its fp32 sums.

Product's bound.  Every product of two E2M1 values under their block scales is
exact, so the error is that of adding K terms in fp32 in some order: at most K
additions, each off by less than one step (2^-23 relative to the partial sum's
magnitude, whether the adder rounds or cuts), so |Y - exact| <= K 2^-23 S with
S = sum |x w|.  The terms of one K = 64 step are added inside the tensor core,
which leaves K / 64 additions of partial sums and 6 levels inside a step; the
bound used is (K / 64 + 8) 2^-23 S, and half a step of bf16 (2^-8 relative)
where the output is bf16.
"""
import numpy as np
import pytest
import torch

import _mx
from activation_aware_codebook_b200 import binding as bb
from activation_aware_codebook_b200 import synth

pytestmark = pytest.mark.gpu

FMTS = [bb.MX_E8M0, bb.MX_E4M3]


def f64(t):
    return t.detach().cpu().double().numpy()


def activations(rows, K, seed, dtype=torch.bfloat16):
    x = synth.make_activations(max(rows, 1), K, seed, True)[:rows]
    if dtype == torch.float32:  # bits below bf16's
        x = x.float() * (1.0 + 0.003 * torch.sin(torch.arange(K)))
    return x


def starts_of(rows, groups, offsets):
    return list(range(0, rows + 1, rows // groups)) if offsets is None else list(offsets)


def check_packed(q, x, starts):
    """q's codes, scales and row scales against the reference for the rows of its groups."""
    code, byte, g = _mx.quantize(x, q.fmt)
    at = _mx.scale_index(q.rows, byte.shape[1], starts)
    rows = np.arange(starts[0], starts[-1])
    assert np.array_equal(q.codes.cpu().numpy()[rows], _mx.pack(code)[rows])
    assert np.array_equal(q.scales.cpu().numpy()[at[rows]], byte[rows])
    if q.fmt == bb.MX_E4M3:
        assert np.array_equal(q.row_scale.cpu().numpy()[rows].astype(np.float64), g[rows],
                              equal_nan=True)


def values_of(q, starts):
    code = _mx.unpack(q.codes.cpu().numpy())
    at = _mx.scale_index(q.rows, q.K // _mx.BLOCK[q.fmt], starts)
    g = q.row_scale.cpu().double().numpy() if q.fmt == bb.MX_E4M3 else None
    return _mx.values(code, q.scales.cpu().numpy()[at], g, q.fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (130, 96), (257, 544), (5, 4096),
                                    (2, 16448), (2, 32768), (1, 33024), (2, 65568)])
def test_quantize_bit_exact(fmt, dtype, rows, K):
    """Rows that fit one, two and more runs a thread, K of half a scale tile."""
    x = activations(rows, K, rows + K, dtype)
    q = bb.mx_quantize(x.cuda(), fmt)
    check_packed(q, f64(x), [0, rows])
    # the padding of the last tile along K is zero
    words = -(-K // (4 * _mx.BLOCK[fmt]))
    blocks = K // _mx.BLOCK[fmt]
    last = q.scales.view(-1, words, 32, 4, 4)[:, -1, 0, 0].cpu().numpy()
    if blocks % 4:
        assert not last[0, blocks % 4:].any()


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_borders_and_extremes(fmt):
    """Every border between codes and its neighbours under every scale, zeros,
    subnormals, the largest numbers, and rows of one value."""
    rows = []
    s = 2.0 ** np.arange(-3, 5) if fmt == bb.MX_E8M0 else _mx.E4M3_VALUES[1:]
    borders = np.concatenate([_mx.BORDERS, _mx.LEVELS[1:]])
    for v in s:
        cand = torch.tensor(borders * v, dtype=torch.float64).to(torch.bfloat16)
        near = cand.view(torch.int16)
        row = torch.zeros(64, dtype=torch.bfloat16)
        row[:14] = cand
        row[14:28] = (near + 1).view(torch.bfloat16)
        row[28:42] = -(near - 1).view(torch.bfloat16)
        rows.append(row)
        row = row.clone()
        row[32] = 2688.0  # the row's largest, in another block
        rows.append(row)
    tiny = torch.finfo(torch.bfloat16).tiny
    for v in (0.0, -0.0, tiny, tiny / 64, 3e38, -3.3e38, 1e-30, 6.0, 7.5, 2688.0, 2720.0):
        row = torch.zeros(64)
        row[5] = v
        row[40] = -v / 3
        rows.append(row.to(torch.bfloat16))
        rows.append(torch.full((64,), v).to(torch.bfloat16))
    x = torch.stack(rows)
    q = bb.mx_quantize(x.cuda(), fmt)
    check_packed(q, f64(x), [0, x.shape[0]])
    q = bb.mx_quantize(x.float().cuda(), fmt)
    check_packed(q, f64(x), [0, x.shape[0]])


@pytest.mark.parametrize("fmt", FMTS)
def test_nan_and_infinity_reach_the_output(fmt):
    x = activations(6, 128, 3)
    x[1, 40] = float("nan")
    x[3, 7] = float("inf")
    x[4, 127] = -float("inf")
    q = bb.mx_quantize(x.cuda(), fmt)
    check_packed(q, f64(x), [0, 6])
    v = bb.mx_dequant(q, torch.float32)
    ref = values_of(q, [0, 6])
    assert np.array_equal(f64(v), ref, equal_nan=True)
    W = bb.mx_quantize(activations(130, 128, 4).cuda(), fmt)
    Y = bb.mx_linear(q, W).cpu()
    assert torch.isnan(Y[[1, 3, 4]]).all() and torch.isfinite(Y[[0, 2, 5]]).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_swiglu(fmt, dtype):
    """The same bits as quantising silu(a) * b computed in fp32 by torch, and
    within one rounding of its 64-bit value (codes near a border may differ)."""
    x = torch.cat([activations(67, 4640, 1, dtype), activations(67, 4640, 2, dtype)], 1)
    x[3, :40] = torch.linspace(-120, 120, 40).to(dtype)
    xg = x.cuda()
    a, b = xg.float().chunk(2, 1)
    h = a / (1.0 + torch.exp(-a)) * b
    q, r = bb.mx_quantize(xg, fmt, swiglu=True), bb.mx_quantize(h, fmt)
    assert torch.equal(q.codes, r.codes)
    assert torch.equal(bb.mx_dequant(q), bb.mx_dequant(r))
    a, b = f64(x)[:, :4640], f64(x)[:, 4640:]
    with np.errstate(over="ignore"):
        h64 = a / (1.0 + np.exp(-a)) * b
    # exp, +, / and * in fp32: exp is within 2 steps, each other step half of
    # one; above 88.73 fp32's exp(-a) is infinite, where the value is below
    # 88.73 exp(-88.72) |b| < 3e-37 |b|
    ok = np.abs(f64(h) - h64) <= 4 * 2.0 ** -23 * np.abs(h64) + 3e-37 * (1 + np.abs(b))
    assert ok.all()


# gates where exp(-a) nears fp32's end (at 88.72) and passes it
FAR_GATES = [-86.0, -86.5, -86.75, -87.0, -87.25, -87.5, -88.0, -88.5, -88.7, -88.75, -89.0,
             -95.0, -104.0, -200.0, -608.0, -1e4, -1e6, -1e30, -1e38, -3e38]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_swiglu_of_far_gates(fmt, dtype):
    """Rows and blocks whose gates all lie around or below -87, under small and large b:
    the bits of the documented form in fp32 (0 where exp(-a) is infinite), by
    the quantisation and by the product that quantises its rows itself."""
    K = 160
    b = torch.cat([torch.logspace(-30, 38, K // 2), -torch.logspace(-30, 38, K // 2)]).float()
    b = b[torch.arange(K) * 37 % K]  # 37 and 160 have no common factor
    one = torch.linspace(0.5, 1.5, K)
    rows = [(torch.full((K,), a), v) for a in FAR_GATES for v in (one, -one, b)]
    # a block of far gates beside ordinary ones; NaN and infinities among far gates
    mixed = torch.full((K,), -1e30)
    mixed[32:64] = torch.linspace(-3, 3, 32)
    rows += [(mixed, one), (mixed, b)]
    for at, (ga, up) in enumerate([(float("nan"), 1.0), (-float("inf"), 1.0), (-1e30, float("inf")),
                                   (-88.5, float("nan"))]):
        a, v = torch.full((K,), -200.0), one.clone()
        a[33 + at], v[33 + at] = ga, up
        rows.append((a, v))
    x = torch.stack([torch.cat(r) for r in rows]).to(dtype).cuda()
    a, u = x.float().chunk(2, 1)
    h = a / (1.0 + torch.exp(-a)) * u
    q, r = bb.mx_quantize(x, fmt, swiglu=True), bb.mx_quantize(h, fmt)
    assert torch.equal(q.codes, r.codes)
    starts = [0, x.shape[0]]
    assert np.array_equal(values_of(q, starts), values_of(r, starts), equal_nan=True)
    # the rows of the largest gates are zeros, whatever b
    last = slice(3 * FAR_GATES.index(-200.0), 3 * len(FAR_GATES))
    assert not values_of(q, starts)[last].any()
    W = bb.mx_quantize(synth.make_weight(130, K, 3).cuda(), fmt)
    for i in range(0, x.shape[0], 2):
        part = x[i:i + 2]
        if fmt == bb.MX_E8M0:  # (bf16 and fp32 rows by the product's own kernel)
            assert bb.mx_workspace_size(fmt, part.shape[0], K, 1, True) == 0
        y, z = bb.mx_linear(part, W, swiglu=True), bb.mx_linear(bb.mx_quantize(h[i:i + 2], fmt), W)
        assert torch.equal(y.isnan(), z.isnan()) and torch.equal(y.nan_to_num(7.0), z.nan_to_num(7.0))


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_gather_groups_and_strides(fmt):
    """Ragged groups (empty, one row, across tile bands), gathered rows with
    padding and out-of-range indices, a strided source, and rows of no group
    left as they were."""
    K, n = 160, 90
    offsets = [3, 3, 4, 140, 140, 270, 399, 400]
    R = 404
    src = activations(n, K + 24, 9)
    x = src.cuda()[:, 8:8 + K]  # ldx = K + 24, rows 16-byte aligned
    index = (torch.arange(R) * 7 % n).to(torch.int32)
    index[10], index[200], index[300] = -1, n, 2 ** 31 - 1
    ref = f64(src)[:, 8:8 + K][np.clip(index.numpy(), 0, n - 1)]
    ref[[10, 200, 300]] = 0.0
    out = bb.MxTensor.empty(fmt, R, K, len(offsets) - 1,
                            torch.tensor(offsets, dtype=torch.int32).cuda())
    out.codes.fill_(0x5A)
    out.scales.fill_(0x5A)
    if fmt == bb.MX_E4M3:
        out.row_scale.fill_(-7.0)
    bb.mx_quantize(x, fmt, rows=index.cuda(), out=out)
    check_packed(out, ref, offsets)
    outside = [0, 1, 2, 400, 401, 402, 403]
    assert (out.codes[outside] == 0x5A).all()
    if fmt == bb.MX_E4M3:
        assert (out.row_scale[outside] == -7.0).all()
    words = -(-K // (4 * _mx.BLOCK[fmt]))
    at = _mx.scale_index(R, words * 4, offsets)
    free = np.ones(out.scales.numel(), dtype=bool)
    free[at[at >= 0]] = False
    assert (out.scales.cpu().numpy()[free] == 0x5A).all()
    # and back: rows of no group are not written either
    back = torch.full((R, K), 11.0, dtype=torch.float32, device="cuda")
    bb.mx_dequant(out, out=back)
    code = _mx.unpack(out.codes.cpu().numpy())
    g = out.row_scale.cpu().double().numpy() if fmt == bb.MX_E4M3 else None
    at = _mx.scale_index(R, K // _mx.BLOCK[fmt], offsets)
    v = _mx.values(code, out.scales.cpu().numpy()[np.maximum(at, 0)], g, fmt)
    inside = np.arange(offsets[0], offsets[-1])
    assert np.array_equal(f64(back)[inside], v[inside])
    assert (back[outside] == 11.0).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,K", [(1, 32), (129, 416), (300, 2080)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dequant_exact(fmt, rows, K, dtype):
    """Any codes and scales, not only those that quantisation makes; a strided output."""
    r = np.random.RandomState(rows + K)
    q = bb.MxTensor.empty(fmt, rows, K)
    q.codes.copy_(torch.from_numpy(r.randint(0, 256, (rows, K // 2)).astype(np.uint8)))
    lo, hi = (90, 160) if fmt == bb.MX_E8M0 else (0, 127)
    q.scales.copy_(torch.from_numpy(r.randint(lo, hi, q.scales.numel()).astype(np.uint8)))
    if fmt == bb.MX_E4M3:
        q.row_scale.copy_(torch.from_numpy(2.0 ** r.randint(-30, 30, rows)).float())
    out = torch.zeros(rows, K + 8, dtype=dtype, device="cuda")
    bb.mx_dequant(q, out=out[:, :K])
    assert np.array_equal(f64(out)[:, :K], values_of(q, [0, rows]))
    assert not out[:, K:].any()


def check_product(Y, X, W, x_starts, groups, y0=None):
    """Y against the 64-bit product of the values that X and W stand for."""
    xv = values_of(X, x_starts)
    N = W.rows // groups
    wv = values_of(W, list(range(0, W.rows + 1, N)))
    Yh = f64(Y)
    K = X.K
    for e in range(groups):
        a, b = x_starts[e], x_starts[e + 1]
        w = wv[e * N:(e + 1) * N]
        ref = xv[a:b] @ w.T
        bound = (K / 64 + 8) * 2.0 ** -23 * (np.abs(xv[a:b]) @ np.abs(w).T) + 1e-35
        if Y.dtype == torch.bfloat16:
            bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
        err = np.abs(Yh[a:b] - ref)
        assert np.all(err <= bound), (e, float((err / bound).max()))
    if y0 is not None:
        outside = list(range(0, x_starts[0])) + list(range(x_starts[-1], Y.shape[0]))
        assert (Yh[outside] == y0).all()
    assert bb.device_timeouts() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [32, 64, 96, 256, 288, 1056])
def test_linear_one_tile(fmt, K):
    """K inside one MMA step, one stage, and a last stage that is partly filled."""
    X = bb.mx_quantize(activations(32, K, K).cuda(), fmt)
    W = bb.mx_quantize(activations(128, K, K + 1).cuda(), fmt)
    Y = bb.mx_linear(X, W)
    torch.cuda.synchronize()
    check_product(Y, X, W, [0, 32], 1)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 2, 17, 33, 64, 65, 100, 128, 129, 200, 256, 300, 700])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_linear_tokens(fmt, M, out_dtype):
    """Every token tile, partial tiles of both operands, split and unsplit K."""
    N, K = 330, 2144
    x = activations(M, K, M + 5)
    X = bb.mx_quantize(x.cuda(), fmt)
    W = bb.mx_quantize(synth.make_weight(N, K, 6).cuda(), fmt)
    Y = bb.mx_linear(X, W, out_dtype=out_dtype)
    torch.cuda.synchronize()
    check_product(Y, X, W, [0, M], 1)
    # the one-call form: the same bits, twice
    for _ in range(2):
        assert torch.equal(bb.mx_linear(x.cuda(), W, out_dtype=out_dtype), Y)


@pytest.mark.parametrize("M,N,K", [(1, 200, 4096), (8, 200, 512), (17, 200, 2080), (160, 130, 288),
                                   (100, 128 * 150, 96), (520, 128 * 80, 96)])
@pytest.mark.parametrize("x_top,w_top", [(3e38, 1e-30), (1e-30, 3e38), (1e31, 1e-10), (1e-37, 1e36),
                                         (1e-36, 1e-3), (1e-20, 1e-22), (1e18, 1e18)])
def test_linear_range_of_row_scales(M, N, K, x_top, w_top):
    """E4M3 row scales far from 1: where the product is in range, so is Y, by
    split, walking and paired CTAs and by the product's own quantisation.
    Row scales are powers of two, exact beside the sum but for subnormal Y
    (half a step of 2^-149 for each of two roundings)."""
    g = torch.Generator().manual_seed(K)
    x = (torch.rand(M, K, generator=g) * 2 - 1) * x_top
    w = (torch.rand(N, K, generator=g) * 2 - 1) * w_top
    X, W = bb.mx_quantize(x.cuda(), bb.MX_E4M3), bb.mx_quantize(w.cuda(), bb.MX_E4M3)
    xv, wv = values_of(X, [0, M]), values_of(W, [0, N])
    ref = xv @ wv.T
    bound = (K / 64 + 8) * 2.0 ** -23 * (np.abs(xv) @ np.abs(wv).T) + 2.0 ** -149
    for Y in (bb.mx_linear(X, W), bb.mx_linear(x.cuda(), W)):
        assert torch.isfinite(Y).all()
        assert (np.abs(f64(Y) - ref) <= bound).all()
    # a row of zeros stays one beside the largest scales
    x[0] = 0.0
    assert not bb.mx_linear(x.cuda(), W)[0].any()


@pytest.mark.parametrize("fmt", FMTS)
def test_linear_many_tiles(fmt):
    """More tiles than SMs: persistent CTAs over several tiles, an accumulator reused."""
    for M, N, K in ((30, 128 * 151, 320), (515, 128 * 100 + 7, 320), (1300, 3700, 544)):
        X = bb.mx_quantize(activations(M, K, M).cuda(), fmt)
        W = bb.mx_quantize(synth.make_weight(N, K, N).cuda(), fmt)
        Y = bb.mx_linear(X, W)
        torch.cuda.synchronize()
        check_product(Y, X, W, [0, M], 1)


@pytest.mark.parametrize("fmt", FMTS)
def test_linear_into_slices(fmt):
    """Outputs side by side in one matrix, at odd columns, and fp32 activations."""
    K, M, widths = 512, 50, (70, 33, 129)
    x = activations(M, K, 2, torch.float32).cuda()
    Ws = [bb.mx_quantize(synth.make_weight(n, K, n).cuda(), fmt) for n in widths]
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((M, sum(widths) + 3), 5.0, dtype=dtype, device="cuda")
        at = 1
        for n, W in zip(widths, Ws):
            bb.mx_linear(x, W, out=y[:, at:at + n])
            at += n
        X = bb.mx_quantize(x, fmt)
        at = 1
        for n, W in zip(widths, Ws):
            check_product(y[:, at:at + n], X, W, [0, M], 1)
            at += n
        assert (y[:, 0] == 5.0).all() and (y[:, at:] == 5.0).all()


GROUPS = [
    [0, 5],                                # one group, ragged by offsets
    [2, 2, 3, 40, 40, 41, 200],            # empty and single rows, rows of no group in front
    [0, 0, 0, 0],                          # nothing at all
    [0, 300, 300, 301, 700],               # tiles that start inside a scale band
    [0] + [7 * i for i in range(1, 41)],   # many small groups
    [0, 20, 20, 60, 61, 61, 61, 61, 61],   # few rows a group on average, one of 40
    [0] * 30 + [150],                      # one group with all the rows
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", range(len(GROUPS)))
@pytest.mark.parametrize("K", [96, 1184])
def test_linear_grouped(fmt, case, K):
    offsets = GROUPS[case]
    E, N = len(offsets) - 1, 150
    R = offsets[-1] + 3
    x = activations(R, K, case + K)
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    X = bb.mx_quantize(x.cuda(), fmt, groups=E, offsets=off)
    W = bb.mx_quantize(synth.make_weight(E * N, K, E).cuda(), fmt, groups=E)
    for dtype in (torch.float32, torch.bfloat16):
        Y = torch.full((R, N), 3.0, dtype=dtype, device="cuda")
        bb.mx_linear(X, W, out=Y)
        torch.cuda.synchronize()
        check_product(Y, X, W, offsets, E, y0=3.0)
        Y2 = torch.full((R, N), 3.0, dtype=dtype, device="cuda")
        bb.mx_linear(x.cuda(), W, out=Y2, offsets=off)
        assert torch.equal(Y, Y2)


@pytest.mark.parametrize("fmt", FMTS)
def test_linear_equal_groups(fmt):
    """Groups of equal size without offsets; expert weights of whole and partial tiles."""
    for E, per, N in ((4, 35, 256), (3, 130, 100)):
        K = 320
        X = bb.mx_quantize(activations(E * per, K, E).cuda(), fmt, groups=E)
        W = bb.mx_quantize(synth.make_weight(E * N, K, 8).cuda(), fmt, groups=E)
        Y = bb.mx_linear(X, W)
        torch.cuda.synchronize()
        check_product(Y, X, W, [e * per for e in range(E + 1)], E)


@pytest.mark.parametrize("fmt", FMTS)
def test_group_rows_do_not_depend_on_their_batch(fmt):
    """A token's output is the same alone, in a batch and next to other experts'
    rows: the same quantisation, and the same order of the sum where the plan
    does not split K (many tiles)."""
    K, N, E = 352, 128 * 40, 4
    x = activations(64, K, 1).cuda()
    W = bb.mx_quantize(synth.make_weight(E * N, K, 2).cuda(), fmt, groups=E)
    off = torch.tensor([0, 16, 16, 40, 64], dtype=torch.int32).cuda()
    Y = bb.mx_linear(x, W, offsets=off)
    perm = torch.cat([torch.arange(16), torch.arange(16, 40).flip(0), torch.arange(40, 64)])
    Z = bb.mx_linear(x, W, rows=perm.to(torch.int32).cuda(), offsets=off)
    assert torch.equal(Z, Y[perm.cuda()])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("rows,K,N", [(1, 32, 130), (1, 4096, 300), (2, 2080, 70), (3, 544, 128),
                                      (5, 1056, 200), (8, 288, 129), (16, 2048, 260),
                                      (4, 96, 128 * 151), (1, 32768, 128), (7, 1152, 128 * 150),
                                      (4, 2336, 128 * 149)])
def test_few_rows_are_quantised_by_the_product(fmt, dtype, swiglu, rows, K, N):
    """A few rows are quantised by the product itself: the same bits as
    quantisation and product, for K split over CTAs, whole, and for CTAs with
    several tiles; rows picked by an index with padding."""
    if rows <= 4:
        assert (bb.mx_workspace_size(fmt, rows, K, 1, swiglu) == 0) == (
            fmt == bb.MX_E8M0 or (not swiglu and rows * K <= 8192))
    x = activations(rows + 2, (2 if swiglu else 1) * K, rows + K, dtype).cuda()
    W = bb.mx_quantize(synth.make_weight(N, K, 3).cuda(), fmt)
    index = torch.arange(rows, dtype=torch.int32).flip(0)
    if rows > 1:
        index[rows // 2] = -1
    for rows_arg in (None, index.cuda()):
        src = x[:rows] if rows_arg is None else x
        X = bb.mx_quantize(src, fmt, rows=rows_arg, swiglu=swiglu)
        for out_dtype in (torch.float32, torch.bfloat16):
            Y = bb.mx_linear(X, W, out_dtype=out_dtype)
            Z = bb.mx_linear(src, W, rows=rows_arg, swiglu=swiglu, out_dtype=out_dtype)
            assert torch.equal(Y, Z)
    torch.cuda.synchronize()
    check_product(Y, X, W, [0, rows], 1)


@pytest.mark.parametrize("fmt", FMTS)
def test_few_rows_of_one_ragged_group(fmt):
    """Rows outside the one group are left as they were; a NaN stays in its row."""
    K, N, R = 608, 200, 12
    x = activations(R, K, 5)
    x[6, 100] = float("nan")
    W = bb.mx_quantize(synth.make_weight(N, K, 3).cuda(), fmt)
    for lo, hi in ((0, 12), (3, 9), (5, 5), (11, 12)):
        off = torch.tensor([lo, hi], dtype=torch.int32).cuda()
        Y = torch.full((R, N), 2.5, device="cuda")
        bb.mx_linear(x.cuda(), W, out=Y, offsets=off)
        X = bb.mx_quantize(x.cuda(), fmt, offsets=off)
        Z = torch.full((R, N), 2.5, device="cuda")
        bb.mx_linear(X, W, out=Z)
        assert torch.equal(Y.nan_to_num(7.0), Z.nan_to_num(7.0))
        assert torch.isnan(Y).any(1).cpu().tolist() == [lo <= r < hi and r == 6 for r in range(R)]
        assert (Y[:lo] == 2.5).all() and (Y[hi:] == 2.5).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(160, 128 * 80, 288), (1100, 5100, 544), (2300, 2600, 320)])
def test_linear_wide_tiles(fmt, M, N, K):
    """Tiles of 192 and 256 tokens, by single CTAs and by pairs, with last tiles
    of few rows and weight rows that end inside a tile."""
    X = bb.mx_quantize(activations(M, K, M).cuda(), fmt)
    W = bb.mx_quantize(synth.make_weight(N, K, N).cuda(), fmt)
    for dtype in (torch.float32, torch.bfloat16):
        Y = bb.mx_linear(X, W, out_dtype=dtype)
        torch.cuda.synchronize()
        check_product(Y, X, W, [0, M], 1)


@pytest.mark.parametrize("fmt", FMTS)
def test_linear_grouped_wide_tiles(fmt):
    """Ragged groups large enough for pairs of CTAs: tiles that start at any row."""
    offsets = [5, 5, 700, 701, 1500, 1900, 2611]
    E, N, K = 6, 2600, 352
    x = activations(2620, K, 4).cuda()
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    X = bb.mx_quantize(x, fmt, groups=E, offsets=off)
    W = bb.mx_quantize(synth.make_weight(E * N, K, E).cuda(), fmt, groups=E)
    assert bb.mx_launch_plan(E, 2620, N, K)["rows"] == 256
    Y = torch.full((2620, N), 3.0, device="cuda")
    bb.mx_linear(X, W, out=Y)
    torch.cuda.synchronize()
    check_product(Y, X, W, offsets, E, y0=3.0)
    Z = torch.full((2620, N), 3.0, device="cuda")
    bb.mx_linear(x, W, out=Z, offsets=off)
    assert torch.equal(Y, Z)


def test_empty_calls():
    for fmt in FMTS:
        W = bb.mx_quantize(synth.make_weight(40, 64, 1).cuda(), fmt)
        x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
        X = bb.mx_quantize(x, fmt)
        assert bb.mx_dequant(X).shape == (0, 64)
        assert bb.mx_linear(X, W).shape == (0, 40) and bb.mx_linear(x, W).shape == (0, 40)
        # rows that all come from padding
        none = torch.full((5,), -1, dtype=torch.int32, device="cuda")
        assert not bb.mx_linear(x, W, rows=none).any()


@pytest.mark.parametrize("fmt", FMTS)
def test_mixture_of_experts_block(fmt):
    """The calls together, as a mixture-of-experts MLP uses them: rows gathered
    by expert into the gate and up halves, SwiGLU and quantisation in one, the
    down projection, and the weighted sum back to the tokens; each stage
    against 64 bits on the values it was given."""
    T, H, F, E, top = 45, 256, 224, 6, 2
    g = torch.Generator().manual_seed(5)
    x = activations(T, H, 3)
    scores = torch.randn(T, E, generator=g)
    scores[:, 4] = -9.0  # an expert that nobody picks
    weight, pick = torch.softmax(scores, 1).topk(top, dim=1)
    flat = pick.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    rows = (order // top).to(torch.int32).cuda()
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    off = offsets.to(torch.int32).cuda()
    up = bb.mx_quantize(synth.make_weight(E * 2 * F, H, 6).cuda(), fmt, groups=E)
    down = bb.mx_quantize(synth.make_weight(E * H, F, 7).cuda(), fmt, groups=E)
    hidden = bb.mx_linear(x.cuda(), up, rows=rows, offsets=off)
    y = bb.mx_linear(hidden, down, offsets=off, swiglu=True)
    out = torch.zeros(T, H, device="cuda").index_add_(
        0, rows.long(), y * weight.reshape(-1)[order].cuda()[:, None])
    torch.cuda.synchronize()
    starts = offsets.tolist()
    X = bb.mx_quantize(x.cuda(), fmt, rows=rows, groups=E, offsets=off)
    check_product(hidden, X, up, starts, E)
    Hq = bb.mx_quantize(hidden, fmt, swiglu=True, groups=E, offsets=off)
    check_product(y, Hq, down, starts, E)
    ref = np.zeros((T, H))
    np.add.at(ref, rows.cpu().numpy(), f64(y) * f64(weight.reshape(-1)[order])[:, None])
    # `top` products and sums in fp32
    assert np.abs(f64(out) - ref).max() <= (top + 1) * 2.0 ** -23 * np.abs(f64(y)).max()


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_beyond_32_bits(fmt):
    """2.3e9 values: codes past 2^30 bytes, activations past 2^32; the last rows
    are those of the same rows alone, through every call."""
    rows, K, N, tail = 70000, 32768, 40, 3
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    last = activations(tail, K, 8).cuda()
    x[-tail:] = last
    q, small = bb.mx_quantize(x, fmt), bb.mx_quantize(last, fmt)
    assert torch.equal(q.codes[-tail:], small.codes)
    W = bb.mx_quantize(synth.make_weight(N, K, 3).cuda(), fmt)
    Y = bb.mx_linear(q, W)
    assert not Y[:-tail].any()
    check_product(bb.mx_linear(small, W), small, W, [0, tail], 1)
    # the same products in another order of K may differ in their last bits
    ref = bb.mx_linear(small, W)
    S = bb.mx_linear(bb.mx_quantize(last.abs(), fmt),
                     bb.mx_quantize(bb.mx_dequant(W).abs(), fmt))
    assert (Y[-tail:] - ref).abs().le(2 * (K / 64 + 8) * 2.0 ** -23 * S + 1e-35).all()
    del Y
    back = bb.mx_dequant(q, out=x)
    assert torch.equal(back[-tail:], bb.mx_dequant(small)) and not back[:100].any()


def test_smallest_and_most_groups():
    for fmt in FMTS:
        x = activations(3, 32, 1).cuda()
        W = bb.mx_quantize(activations(1, 32, 2).cuda(), fmt)
        X = bb.mx_quantize(x, fmt)
        check_product(bb.mx_linear(X, W), X, W, [0, 3], 1)
        E, N, K, R = 1024, 3, 64, 300
        W = bb.mx_quantize(synth.make_weight(E * N, K, 4).cuda(), fmt, groups=E)
        cut = torch.sort(torch.randint(0, R + 1, (E + 1,), generator=torch.Generator().manual_seed(1))).values
        off = cut.to(torch.int32).cuda()
        x = activations(R, K, 5).cuda()
        X = bb.mx_quantize(x, fmt, groups=E, offsets=off)
        Y = torch.full((R, N), 4.0, device="cuda")
        bb.mx_linear(X, W, out=Y)
        torch.cuda.synchronize()
        check_product(Y, X, W, cut.tolist(), E, y0=4.0)


def test_offsets_that_are_not_sound_stay_inside():
    """Offsets out of range or descending give unspecified rows; rows that other
    tensors own are not touched."""
    for fmt in FMTS:
        E, N, K, R = 3, 70, 96, 50
        W = bb.mx_quantize(synth.make_weight(E * N, K, 4).cuda(), fmt, groups=E)
        for offsets in ([-5, 10, 20, 99], [40, 10, 30, 50], [60, 70, 80, 90], [0, 50, 0, 50]):
            off = torch.tensor(offsets, dtype=torch.int32).cuda()
            whole = torch.full((R + 20, N), 6.0, device="cuda")
            bb.mx_linear(activations(R, K, 3).cuda(), W, out=whole[10:10 + R], offsets=off)
            X = bb.mx_quantize(activations(R, K, 3).cuda(), fmt, groups=E, offsets=off)
            bb.mx_dequant(X)
            torch.cuda.synchronize()
            assert (whole[:10] == 6.0).all() and (whole[10 + R:] == 6.0).all()
    assert bb.device_timeouts() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_that_name_every_row_in_every_group(fmt):
    """1024 groups, every other one of all rows: the tiles beyond the plan's
    bound are left out, nothing around the output is touched, and the call after
    it is right."""
    E, N, K, R = 1024, 40, 96, 3000
    W = bb.mx_quantize(synth.make_weight(E * N, K, 4).cuda(), fmt, groups=E)
    x = activations(R, K, 3).cuda()
    wild = torch.tensor([0, R] * (E // 2) + [0], dtype=torch.int32).cuda()
    whole = torch.full((R + 2, N), 6.0, device="cuda")
    bb.mx_linear(x, W, out=whole[1:-1], offsets=wild)
    torch.cuda.synchronize()
    assert (whole[[0, -1]] == 6.0).all() and bb.device_timeouts() == 0
    sound = [0] * 512 + [R] * 513
    off = torch.tensor(sound, dtype=torch.int32).cuda()
    X = bb.mx_quantize(x, fmt, groups=E, offsets=off)
    check_product(bb.mx_linear(X, W), X, W, sound, E)


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    W = bb.mx_quantize(x, bb.MX_E4M3)
    W8 = bb.mx_quantize(x, bb.MX_E8M0)
    i32 = dict(dtype=torch.int32, device="cuda")
    bad = [lambda: bb.mx_quantize(x.half(), bb.MX_E4M3),
           lambda: bb.mx_quantize(x[0], bb.MX_E4M3),
           lambda: bb.mx_quantize(x.cpu(), bb.MX_E4M3),
           lambda: bb.mx_quantize(x, bb.MX_E4M3, rows=torch.zeros(4, device="cuda")),
           lambda: bb.mx_quantize(x, bb.MX_E4M3, groups=2, offsets=torch.zeros(2, **i32)),
           lambda: bb.mx_quantize(x, bb.MX_E4M3, out=W8),
           lambda: bb.mx_quantize(x, bb.MX_E4M3, out=W, groups=2),
           lambda: bb.mx_quantize(x, bb.MX_E4M3, out=W, offsets=torch.zeros(2, **i32)),
           lambda: bb.mx_linear(W, W, rows=torch.zeros(4, **i32)),
           lambda: bb.mx_linear(W, W, out=torch.zeros(4, 5, device="cuda")),
           lambda: bb.mx_linear(W, W, out=torch.zeros(4, 4, dtype=torch.int32, device="cuda")),
           lambda: bb.mx_linear(x[:, :32], W),
           lambda: bb.mx_linear(x, W, rows=torch.zeros(4, dtype=torch.int32)),
           lambda: bb.MxTensor(W.codes, W.scales[:-1], W.row_scale, bb.MX_E4M3),
           lambda: bb.MxTensor(W.codes, W.scales, None, bb.MX_E4M3),
           lambda: bb.MxTensor(W.codes.t(), W.scales, W.row_scale, bb.MX_E4M3)]
    for f in bad:
        with pytest.raises((ValueError, TypeError)):
            f()
    for f in (lambda: bb.mx_quantize(torch.zeros(4, 40, dtype=torch.bfloat16, device="cuda"), 0),
              lambda: bb.mx_quantize(x, 2), lambda: bb.mx_linear(W8, W),
              lambda: bb.mx_quantize(x, bb.MX_E4M3, groups=3)):
        with pytest.raises(bb.AaacError):
            f()


@pytest.mark.parametrize("fmt", FMTS)
def test_captured_on_forked_streams(fmt):
    """A capture that forks: one quantised input, three products on streams of
    their own, joined again; replayed on new inputs."""
    K, M = 384, 33
    Ws = [bb.mx_quantize(synth.make_weight(n, K, n).cuda(), fmt) for n in (200, 64, 129)]
    x = activations(M, K, 1).cuda()
    X = bb.MxTensor.empty(fmt, M, K)
    ys = [torch.zeros(M, W.rows, device="cuda") for W in Ws]
    streams = [torch.cuda.Stream() for _ in range(4)]

    def step():
        main = torch.cuda.current_stream()
        bb.mx_quantize(x, fmt, out=X)
        for s, W, y in zip(streams, Ws, ys):
            s.wait_stream(main)
            bb.mx_linear(X, W, out=y, stream=s)
        for s in streams[:3]:
            main.wait_stream(s)

    with torch.cuda.stream(streams[3]):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[3]):
        step()
    for seed in (2, 3):
        new = activations(M, K, seed).cuda()
        x.copy_(new)
        for y in ys:
            y.zero_()
        g.replay()
        torch.cuda.synchronize()
        for y, W in zip(ys, Ws):
            assert torch.equal(y, bb.mx_linear(bb.mx_quantize(new, fmt), W))


@pytest.mark.parametrize("fmt", FMTS)
def test_streams_and_graphs(fmt):
    """Two streams with a workspace each, and a captured call replayed on new
    inputs and new expert counts."""
    K, N, E, R = 512, 300, 3, 60
    W = bb.mx_quantize(synth.make_weight(E * N, K, 2).cuda(), fmt, groups=E)
    xs = [activations(R, K, s).cuda() for s in (1, 2)]
    offs = [torch.tensor(o, dtype=torch.int32).cuda() for o in ([0, 20, 20, 60], [0, 1, 50, 58])]
    want = [torch.zeros(R, N, device="cuda") for _ in xs]
    for x, o, y in zip(xs, offs, want):
        bb.mx_linear(x, W, offsets=o, out=y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [torch.zeros(R, N, device="cuda") for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x, o, y in zip(streams, xs, offs, got):
            bb.mx_linear(x, W, offsets=o, out=y, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x, o, y = xs[0].clone(), offs[0].clone(), torch.zeros(R, N, device="cuda")
    ws = torch.empty(bb.mx_workspace_size(fmt, R, K, E), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bb.mx_linear(x, W, offsets=o, out=y, ws=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        bb.mx_linear(x, W, offsets=o, out=y, ws=ws)
    launches = bb.kernel_launches()
    for i in (1, 0, 1):
        x.copy_(xs[i])
        o.copy_(offs[i])
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
    assert bb.kernel_launches() == launches
