"""The microscaled product under every kind of plan: each case names the plan
that mx_launch_plan gives it (token columns of a tile, CTAs that share a tile's
K, weight rows of a tile), so that no compiled form of the kernel goes
unchecked.  References in 64 bits from the values of the quantised operands
(mx_dequant to fp32 is exact; test_gpu_mx.py holds it to the format)."""
import pytest
import torch

from activation_aware_codebook_b200 import binding as bb
from activation_aware_codebook_b200 import synth

pytestmark = pytest.mark.gpu

FMTS = [bb.MX_E8M0, bb.MX_E4M3]


def product_error(Y, X, W, starts):
    """The largest |Y - exact| over its bound, over the rows of the groups.

    K / 64 additions of a step's sum to an fp32 sum and 6 levels inside a step,
    each off by less than a step of 2^-23 of the magnitudes' sum S.  Split K
    has K / 64 / split of them in a CTA and split - 1 <= 7 between CTAs, fewer
    in all at the K used here.  Half a step of bf16 (2^-8) where Y is bf16."""
    x, w = (bb.mx_dequant(t, torch.float32).double() for t in (X, W))
    groups = len(starts) - 1
    N, K = W.rows // groups, X.K
    worst = 0.0
    for e in range(groups):
        a, b = starts[e], starts[e + 1]
        if a == b:
            continue
        we = w[e * N:(e + 1) * N]
        ref = x[a:b] @ we.t()
        bound = (K / 64 + 8) * 2.0 ** -23 * (x[a:b].abs() @ we.abs().t()) + 1e-35
        if Y.dtype == torch.bfloat16:
            bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
        ratio = (Y[a:b].double() - ref).abs() / bound
        assert not ratio.isnan().any()
        worst = max(worst, float(ratio.max()))
    return worst


# rows, N, K, (columns, split, weight rows).  The stages of K never divide by
# the split, K ends inside a stage, and N and the rows end inside a tile.
DENSE = [
    (1, 6453, 5696, (32, 2, 128)),
    (1, 4782, 4128, (32, 3, 128)),
    (3, 2759, 3456, (32, 5, 128)),
    (19, 17, 3808, (32, 8, 128)),
    (39, 6464, 5728, (64, 2, 128)),
    (1328, 129, 4640, (64, 3, 128)),
    (1355, 21, 4704, (64, 5, 128)),
    (38, 21, 3136, (64, 7, 128)),
    (70, 6772, 8256, (128, 2, 128)),
    (132, 2911, 4928, (128, 3, 128)),
    (1166, 282, 5440, (128, 4, 128)),
    (132, 1102, 5824, (128, 8, 128)),
    (452, 2521, 9312, (192, 2, 128)),
    (133, 3128, 5920, (192, 5, 128)),
    (262, 1238, 6208, (192, 7, 128)),
    (597, 1851, 7200, (256, 3, 128)),
    (841, 733, 10464, (256, 6, 128)),
    (199, 1804, 17600, (256, 8, 128)),
    # persistent CTAs over one tile and over several
    (131, 6792, 32, (128, 1, 128)),
    (270, 9873, 320, (128, 1, 128)),
    (1514, 4651, 320, (192, 1, 128)),
    (387, 6719, 32, (256, 1, 128)),
    (1341, 6219, 2432, (256, 1, 128)),
    (1042, 7651, 2400, (192, 1, 256)),
    (583, 16182, 2496, (256, 1, 256)),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,N,K,plan", DENSE)
def test_plans(fmt, rows, N, K, plan):
    p = bb.mx_launch_plan(1, rows, N, K)
    assert (p["columns"], p["split"], p["rows"]) == plan
    assert p["split"] == 1 or p["stages"] % p["split"]
    x = synth.make_activations(rows, K, rows, True, device="cuda")
    X = bb.mx_quantize(x, fmt)
    W = bb.mx_quantize(synth.make_weight(N, K, N, device="cuda"), fmt)
    for dtype in (torch.float32, torch.bfloat16):
        whole = torch.full((rows + 2, N + 3), 3.0, dtype=dtype, device="cuda")
        Y = whole[1:-1, 2:-1]
        bb.mx_linear(X, W, out=Y)
        assert product_error(Y, X, W, [0, rows]) <= 1.0
        assert (whole[[0, -1]] == 3.0).all()
        assert (whole[:, :2] == 3.0).all() and (whole[:, -1] == 3.0).all()
        # rows of 16 bytes, and the one-call form: the same bits
        assert torch.equal(bb.mx_linear(x, W, out_dtype=dtype), Y)
    assert bb.device_timeouts() == 0


# groups, rows, N, K, (columns, split, weight rows)
RAGGED = [
    (2, 17, 17, 4224, (64, 6, 128)),
    (6, 7, 1035, 5824, (64, 2, 128)),
    (8, 1185, 16, 3488, (64, 5, 128)),
    (8, 568, 546, 5056, (128, 3, 128)),
    (6, 2205, 19, 5056, (128, 7, 128)),
    (6, 1018, 522, 7296, (192, 3, 128)),
    (8, 1129, 136, 8576, (192, 7, 128)),
    (2, 697, 940, 7808, (256, 4, 128)),
    (8, 2098, 130, 7392, (256, 6, 128)),
    (8, 133, 2271, 2400, (64, 1, 128)),
    (8, 778, 1547, 288, (128, 1, 128)),
    (8, 1939, 1176, 2400, (192, 1, 128)),
    (8, 1629, 1560, 2464, (256, 1, 128)),
    (6, 880, 4358, 2400, (192, 1, 256)),
    (6, 1165, 4413, 2432, (256, 1, 256)),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("skew", ["spread", "crowded"])
@pytest.mark.parametrize("groups,rows,N,K,plan", RAGGED)
def test_ragged_plans(fmt, skew, groups, rows, N, K, plan):
    """Groups that are empty, of one row and of several tiles; rows of no group
    in front and behind stay as they were; one group with nearly all rows."""
    p = bb.mx_launch_plan(groups, rows, N, K)
    assert (p["columns"], p["split"], p["rows"]) == plan
    g = torch.Generator().manual_seed(rows)
    if skew == "spread":
        cut = torch.sort(torch.randint(1, rows, (groups - 1,), generator=g)).values.tolist()
        if groups > 3:
            cut[1] = cut[0]      # an empty group
            cut[2] = cut[1] + 1  # and one of a single row
            cut.sort()
        starts = [1] + cut + [max(rows - 2, cut[-1])]
    else:
        starts = [0] * (groups // 2) + [1] + [rows] * (groups - groups // 2)
    assert len(starts) == groups + 1
    off = torch.tensor(starts, dtype=torch.int32).cuda()
    x = synth.make_activations(rows, K, rows, True, device="cuda")
    X = bb.mx_quantize(x, fmt, groups=groups, offsets=off)
    W = bb.mx_quantize(synth.make_weight(groups * N, K, N, device="cuda"), fmt, groups=groups)
    outside = list(range(starts[0])) + list(range(starts[-1], rows))
    for dtype in (torch.float32, torch.bfloat16):
        Y = torch.full((rows, N), 3.0, dtype=dtype, device="cuda")
        bb.mx_linear(X, W, out=Y)
        assert product_error(Y, X, W, starts) <= 1.0
        assert (Y[outside] == 3.0).all()
        Z = torch.full((rows, N), 3.0, dtype=dtype, device="cuda")
        bb.mx_linear(x, W, out=Z, offsets=off)
        assert torch.equal(Y, Z)
    assert bb.device_timeouts() == 0
