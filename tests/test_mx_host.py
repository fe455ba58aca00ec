"""Host-side checks of the microscaled calls (no GPU): sizes, plans, and the
refusals, which all come before anything is launched."""
import ctypes
import subprocess
import types

import numpy as np
import pytest

import _mx
from activation_aware_codebook_b200 import binding as bb
from activation_aware_codebook_b200.csrc import build as cbuild

OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 6
FAKE = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return bb.load()


def tensor(**kw):
    d = dict(fmt=bb.MX_E4M3, groups=1, rows=64, K=256, codes=FAKE, scales=FAKE, row_scale=FAKE,
             offsets=None)
    d.update(kw)
    return bb.CMxTensor(**d)


def source(**kw):
    d = dict(X=FAKE, type=0, flags=0, rows=64, ldx=256, index=None)
    d.update(kw)
    return bb.CMxSource(**d)


def ref(x):
    return ctypes.byref(x) if x is not None else None


def test_struct_layouts():
    assert ctypes.sizeof(bb.CMxTensor) == 56
    assert ctypes.sizeof(bb.CMxSource) == 40


@pytest.mark.parametrize("fmt", [bb.MX_E8M0, bb.MX_E4M3])
@pytest.mark.parametrize("rows,K,groups", [(0, 32, 1), (1, 32, 1), (127, 96, 3), (128, 4096, 1),
                                           (1000, 160, 64)])
def test_sizes(lib, fmt, rows, K, groups):
    n = bb.mx_scale_bytes(fmt, rows, K, groups)
    assert n == _mx.scale_bytes(rows, K, fmt, groups)
    # every scale of any split into groups has a place of its own inside
    r = np.random.RandomState(rows + K)
    for _ in range(5):
        starts = np.sort(r.randint(0, rows + 1, groups + 1)).tolist()
        at = _mx.scale_index(rows, K // _mx.BLOCK[fmt], starts)
        used = at[at >= 0]
        assert len(np.unique(used)) == len(used) and (len(used) == 0 or used.max() < n)
    for swiglu in (False, True):
        ws = bb.mx_workspace_size(fmt, rows, K, groups, swiglu)
        # 0 only for the few rows of one group that the product quantises itself
        assert ws >= rows * K // 2 + n + 4 * rows or (ws == 0 and groups == 1 and rows <= 8)


def test_sizes_of_invalid_shapes(lib):
    for args in ((2, 4, 64, 1), (0, -1, 64, 1), (0, 1 << 31, 64, 1), (0, 4, 48, 1), (0, 4, 0, 1),
                 (0, 4, 64, 0), (0, 4, 64, 1025), (0, 4, 1 << 25, 1)):
        assert bb.mx_scale_bytes(*args) == 0 and bb.mx_workspace_size(*args) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=2), UNSUPPORTED), (dict(rows=-1), SHAPE), (dict(K=272), SHAPE), (dict(K=0), SHAPE),
    (dict(groups=0), SHAPE), (dict(groups=1025), SHAPE), (dict(groups=3), SHAPE),
    (dict(codes=None), INVALID), (dict(codes=FAKE + 8), ALIGN), (dict(scales=None), INVALID),
    (dict(scales=FAKE + 4), ALIGN), (dict(row_scale=None), INVALID),
    (dict(row_scale=FAKE + 2), ALIGN), (dict(offsets=FAKE + 1), ALIGN)])
def test_bad_tensors_are_refused(lib, kw, status):
    t, good, src = tensor(**kw), tensor(), source()
    assert lib.aaac_mx_quantize(ref(src), ref(t), None) == status
    assert lib.aaac_last_error()
    assert lib.aaac_mx_dequant(ref(t), FAKE, 1, 256, None) == status
    assert lib.aaac_mx_linear(ref(t), ref(good), FAKE, 1, 64, None) == status
    assert lib.aaac_mx_linear(ref(good), ref(t), FAKE, 1, 1 << 20, None) == status
    assert lib.aaac_mx_linear_ws(ref(src), 64, None, ref(t), FAKE, 1, 1 << 20, FAKE, 1 << 40,
                                 None) == status


def test_null_tensors_are_refused(lib):
    t, src = tensor(), source()
    assert lib.aaac_mx_quantize(None, ref(t), None) == INVALID
    assert lib.aaac_mx_quantize(ref(src), None, None) == INVALID
    assert lib.aaac_mx_dequant(None, FAKE, 1, 256, None) == INVALID
    assert lib.aaac_mx_linear(None, ref(t), FAKE, 1, 64, None) == INVALID
    assert lib.aaac_mx_linear(ref(t), None, FAKE, 1, 64, None) == INVALID
    assert lib.aaac_mx_linear_ws(None, 64, None, ref(t), FAKE, 1, 64, FAKE, 1 << 40, None) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), INVALID), (dict(X=FAKE + 8), ALIGN), (dict(type=2), UNSUPPORTED),
    (dict(flags=2), INVALID), (dict(rows=63), SHAPE), (dict(rows=-1), SHAPE),
    (dict(ldx=255), SHAPE), (dict(ldx=260), ALIGN), (dict(type=1, ldx=258), ALIGN),
    (dict(flags=1), SHAPE), (dict(flags=1, ldx=511), SHAPE), (dict(index=FAKE + 2), ALIGN),
    (dict(ldx=(1 << 31) + 8), SHAPE)])
def test_bad_sources_are_refused(lib, kw, status):
    src, t = source(**kw), tensor()
    assert lib.aaac_mx_quantize(ref(src), ref(t), None) == status
    assert lib.aaac_mx_linear_ws(ref(src), 64, None, ref(t), FAKE, 1, 64, FAKE, 1 << 40,
                                 None) == status


def test_bad_products_are_refused(lib):
    x, w = tensor(), tensor(rows=128)
    f = lib.aaac_mx_linear
    assert f(ref(tensor(fmt=bb.MX_E8M0)), ref(w), FAKE, 1, 128, None) == INVALID     # formats
    assert f(ref(tensor(K=288)), ref(w), FAKE, 1, 128, None) == SHAPE                # K
    assert f(ref(tensor(groups=2)), ref(w), FAKE, 1, 128, None) == SHAPE             # groups
    assert f(ref(x), ref(tensor(offsets=FAKE)), FAKE, 1, 128, None) == INVALID       # ragged w
    assert f(ref(x), ref(tensor(rows=0)), FAKE, 1, 128, None) == SHAPE               # no weights
    assert f(ref(x), ref(w), None, 1, 128, None) == INVALID                          # output
    assert f(ref(x), ref(w), FAKE + 2, 1, 128, None) == ALIGN
    assert f(ref(x), ref(w), FAKE + 1, 0, 128, None) == ALIGN
    assert f(ref(x), ref(w), FAKE, 2, 128, None) == UNSUPPORTED
    assert f(ref(x), ref(w), FAKE, 1, 127, None) == SHAPE
    big = tensor(rows=(1 << 31) - 1)
    assert f(ref(big), ref(big), FAKE, 1, 1 << 31, None) == SHAPE                    # tiles
    g = lib.aaac_mx_linear_ws
    need = bb.mx_workspace_size(bb.MX_E4M3, 64, 256, 1)
    src = source()
    assert g(ref(src), 64, None, ref(w), FAKE, 1, 128, None, need, None) == WORKSPACE
    assert g(ref(src), 64, None, ref(w), FAKE, 1, 128, FAKE, need - 1, None) == WORKSPACE
    assert g(ref(src), 64, None, ref(w), FAKE, 1, 128, FAKE + 8, need, None) == ALIGN
    assert g(ref(src), -1, None, ref(w), FAKE, 1, 128, FAKE, need, None) == SHAPE
    assert g(ref(src), 64, FAKE + 2, ref(w), FAKE, 1, 128, FAKE, need, None) == ALIGN
    w3 = tensor(rows=129, groups=3)
    assert g(ref(src), 64, None, ref(w3), FAKE, 1, 128, FAKE, 1 << 40, None) == SHAPE
    assert lib.aaac_mx_dequant(ref(x), FAKE + 8, 1, 256, None) == ALIGN
    assert lib.aaac_mx_dequant(ref(x), FAKE, 0, 260, None) == ALIGN
    assert lib.aaac_mx_dequant(ref(x), FAKE, 0, 255, None) == SHAPE


def test_no_rows_is_no_work(lib):
    x, w, src = tensor(rows=0, codes=None, scales=None, row_scale=None), tensor(), source(rows=0, X=None)
    before = bb.kernel_launches()
    assert lib.aaac_mx_quantize(ref(src), ref(x), None) == OK
    assert lib.aaac_mx_dequant(ref(x), None, 1, 256, None) == OK
    assert lib.aaac_mx_linear(ref(x), ref(w), None, 1, 64, None) == OK
    assert lib.aaac_mx_linear_ws(ref(src), 0, None, ref(w), None, 1, 64, None, 0, None) == OK
    assert bb.kernel_launches() == before


def test_armed_fault_stops_every_call(lib):
    x, w, src = tensor(), tensor(), source()
    for call in (lambda: lib.aaac_mx_quantize(ref(src), ref(x), None),
                 lambda: lib.aaac_mx_dequant(ref(x), FAKE, 1, 256, None),
                 lambda: lib.aaac_mx_linear(ref(x), ref(w), FAKE, 1, 64, None),
                 lambda: lib.aaac_mx_linear_ws(ref(src), 64, None, ref(w), FAKE, 1, 64, FAKE,
                                               1 << 40, None)):
        before = bb.kernel_launches()
        bb.inject_fault("launch")
        assert call() == 5
        assert bb.kernel_launches() == before


@pytest.mark.parametrize("groups,rows", [(1, 1), (1, 32), (1, 33), (1, 64), (1, 128), (1, 129),
                                         (1, 8192), (8, 3), (64, 128), (16, 8200), (1024, 5)])
@pytest.mark.parametrize("N,K", [(1, 32), (1024, 4096), (4096, 4096), (14336, 4096),
                                 (5120, 27648), (100, 4096)])
def test_plan_covers_every_split_of_the_rows(lib, groups, rows, N, K):
    p = bb.mx_launch_plan(groups, rows, N, K)
    assert p["stages"] == -(-K // 256)
    assert 1 <= p["split"] <= min(8, p["stages"])
    assert p["rows"] in (128, 256) and (p["rows"] == 128 or p["split"] == 1)
    n_tiles = -(-N // p["rows"])
    assert p["columns"] in (32, 64, 128, 192, 256)
    # a 32-token tile may not start inside a scale band: one such tile a group
    assert p["columns"] > 32 or (groups == 1 and rows <= 32)
    r = np.random.RandomState(groups + rows)
    for k in range(20):
        cut = np.sort(r.randint(0, rows + 1, groups - 1))
        if k == 0:
            cut[:] = rows
        counts = np.diff(np.concatenate([[0], cut, [rows]]))
        tiles = int(sum(-(-c // p["columns"]) for c in counts)) * n_tiles
        assert tiles <= p["tiles"]
    if p["split"] > 1:  # a cluster a tile, within a grid's limits
        assert p["ctas"] == p["tiles"] * p["split"] and p["tiles"] <= 65535


_TILES = r"""
#include <cstdio>
#include "mx.cuh"
// lines of: width most groups offsets[groups + 1] -> the running sums of the tiles
int main() {
  int width, most, groups, rows;
  while (scanf("%d %d %d %d", &width, &most, &groups, &rows) == 4) {
    (void)rows;
    int sum = 0, from, to;
    if (scanf("%d", &from) != 1) return 1;
    for (int e = 0; e < groups; e++, from = to) {
      if (scanf("%d", &to) != 1) return 1;
      const int last = to < from ? from : to;  // as the kernels read a group
      sum = aaac::mx_add_tiles(sum, aaac::mx_group_tiles(last - from, width, most), most);
      printf("%d ", sum);
    }
    printf("\n");
  }
}
"""


def test_tile_sums_hold_for_any_offsets(lib, tmp_path):
    """The kernel's tile counts on the host: exact for sound offsets, and for
    descending ones inside the plan's bound, whose product with the weight tiles
    stays inside 32 bits (512 groups of 2^24 rows alone make 2^26 tiles of 128
    rows, 2^32 with 64 weight tiles); a group of 2^31 - 1 rows is counted whole."""
    (tmp_path / "tiles.cu").write_text(_TILES)
    subprocess.run([cbuild.NVCC, "-std=c++17", *cbuild.ARCH, "-I", cbuild.HERE, "-o",
                    str(tmp_path / "tiles"), str(tmp_path / "tiles.cu")], check=True)
    cases, text = [], ""
    r = np.random.RandomState(7)
    for groups, rows, N in ((1, (1 << 31) - 1, 1), (1024, 1 << 24, 8192), (1024, 17000000, 8192),
                            (1024, 300, 150), (6, 2620, 2600), (33, 70000, 1000)):
        p = bb.mx_launch_plan(groups, rows, N, 64)
        n_tiles = -(-N // p["rows"])
        most = p["tiles"] // n_tiles
        assert p["tiles"] == most * n_tiles < 1 << 31
        sound = np.concatenate([[0], np.sort(r.randint(0, rows, groups - 1)), [rows]])
        wild = np.where(np.arange(groups + 1) % 2, rows, 0)
        for offsets in (sound, wild, sound[::-1]):
            cases.append((p["columns"], most, rows, offsets.tolist(), offsets is sound))
            text += f"{p['columns']} {most} {groups} {rows} " + " ".join(map(str, offsets)) + "\n"
    out = subprocess.run([str(tmp_path / "tiles")], input=text, capture_output=True, text=True,
                         check=True).stdout.splitlines()
    assert len(out) == len(cases)
    for line, (width, most, rows, offsets, sound) in zip(out, cases):
        got = list(map(int, line.split()))
        exact = np.cumsum([max(-(-(b - a) // width), 0) for a, b in zip(offsets, offsets[1:])])
        assert got == np.minimum(exact, most).tolist()
        if sound:
            assert got == exact.tolist()


def test_plan_refusals(lib):
    out = (ctypes.c_int32 * 6)()
    assert lib.aaac_mx_launch_plan(1, 4, 4, 64, None) == INVALID
    for args in ((0, 4, 4, 64), (1, 0, 4, 64), (1, 4, 0, 64), (1, 4, 4, 48),
                 (1, (1 << 31) - 1, (1 << 31) - 1, 64)):
        assert lib.aaac_mx_launch_plan(*args, out) == SHAPE


def test_binding_refuses_without_cuda(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    with pytest.raises(RuntimeError):
        bb.mx_quantize(torch.zeros(8, 64, dtype=torch.bfloat16), bb.MX_E4M3)


def test_swiglu_needs_two_halves():
    """An odd width has no halves: 65 columns of a padded buffer are not 2 x 32."""
    import torch
    x = torch.zeros(4, 72, dtype=torch.bfloat16)[:, :65]
    with pytest.raises(ValueError, match="halves"):
        bb.mx_quantize(x, bb.MX_E4M3, swiglu=True)
    with pytest.raises(ValueError, match="halves"):
        bb.mx_linear(x, types.SimpleNamespace(K=32), swiglu=True)


def test_output_types_are_refused_by_name():
    import torch
    for dtype in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(ValueError, match="bfloat16 or float32"):
            bb._mx_out(None, 4, 4, dtype, "cpu")
    y, kind, ld = bb._mx_out(None, 4, 5, torch.bfloat16, "cpu")
    assert y.shape == (4, 5) and y.dtype == torch.bfloat16 and (kind, ld) == (0, 5)


def test_workspace_of_fewer_bytes_than_elements_is_refused():
    """numel() of an expanded or strided tensor says nothing about its bytes."""
    import torch
    x, W = torch.zeros(40, 64, dtype=torch.bfloat16), types.SimpleNamespace(K=64)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20),
               torch.zeros(1 << 20, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            bb.mx_linear(x, W, ws=ws)


def test_launches_that_fail_are_not_counted(lib):
    """kernel_launches counts kernels that were launched."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    x, w = tensor(), tensor()
    few = source(rows=4)
    before = bb.kernel_launches()
    assert lib.aaac_mx_quantize(ref(source()), ref(x), None) == 5  # AAAC_ERR_CUDA
    assert lib.aaac_mx_dequant(ref(x), FAKE, 1, 256, None) == 5
    assert lib.aaac_mx_linear(ref(x), ref(w), FAKE, 1, 64, None) == 5
    assert lib.aaac_mx_linear_ws(ref(source()), 64, None, ref(w), FAKE, 1, 64, FAKE, 1 << 40,
                                 None) == 5
    assert lib.aaac_mx_linear_ws(ref(few), 4, None, ref(w), FAKE, 1, 64, None, 0, None) == 5
    assert bb.kernel_launches() == before
