"""The debugging build with device-side index checks (build.py --checks).

On the CPU: the normal library reports that it is not a checked build and its
check flag reads 0 without touching a device.  On the GPU: the checked library
runs whole layers of both formats and several group sizes in a
child process, gives the same tables as the normal library, and every check
holds (flag 0).
"""
import ctypes
import os
import subprocess
import sys

import pytest

from activation_aware_codebook_b200 import binding as bb
from activation_aware_codebook_b200.csrc import build as cbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_normal_build_reports_no_checks():
    cbuild.build()
    lib = bb.load()
    assert lib.aaac_checked_build() == 0
    v = ctypes.c_uint32(7)
    assert lib.aaac_device_checks(ctypes.byref(v)) == 0
    assert v.value == 0
    assert lib.aaac_device_checks(None) == 1  # AAAC_ERR_INVALID_ARG


_CHILD = r"""
import sys, torch
from activation_aware_codebook_b200 import binding as bb, synth
assert bb.load().aaac_checked_build() == 1, "not the checked build"
dev = torch.device("cuda", 0)
out = []
for (N, K, fmt, g, S, it, seed) in [(256, 512, bb.INT4, 128, 16, 6, 1),
                                     (384, 1024, bb.NVFP4, 16, 16, 6, 2),
                                     (200, 2048, bb.NVFP4, 16, 8, 4, 3),
                                     (130, 768, bb.INT4, 128, 128, 5, 4)]:
    W = synth.make_weight(N, K, seed, "normal" if seed % 2 else "student_t4", device=dev)
    X = synth.make_activations(512, K, seed + 100, bool(seed % 2), device=dev)
    r = bb.run_layer(W, X, bb.Config(fmt, g, S, it))
    torch.cuda.synchronize()
    out.append(r["T"].view(torch.int32).cpu())
torch.save(out, sys.argv[1])
print("CHECKS", bb.device_checks())
"""


@pytest.mark.gpu
def test_checked_build_runs_clean_and_agrees(tmp_path):
    cbuild.build(checks=True)
    env = dict(os.environ, AAAC_CHECKED="1", PYTHONPATH=ROOT)
    res = subprocess.run([sys.executable, "-c", _CHILD, str(tmp_path / "checked.pt")], env=env,
                         cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stderr[-3000:]
    assert "CHECKS 0" in res.stdout, res.stdout
    env["AAAC_CHECKED"] = "0"
    res2 = subprocess.run([sys.executable, "-c", _CHILD.replace(
        'assert bb.load().aaac_checked_build() == 1, "not the checked build"', ""),
        str(tmp_path / "plain.pt")], env=env, cwd=ROOT, capture_output=True, text=True,
        timeout=600)
    assert res2.returncode == 0, res2.stderr[-3000:]
    import torch
    a = torch.load(tmp_path / "checked.pt")
    b = torch.load(tmp_path / "plain.pt")
    assert all(torch.equal(x, y) for x, y in zip(a, b))


_WAIT_CHILD = r"""
import sys, torch
from activation_aware_codebook_b200 import binding as bb, synth
assert bb.load().aaac_checked_build() == 1, "not the checked build"
dev = "cuda"
# rows, N, K, groups: persistent CTAs, pairs of CTAs, ragged groups; four tiles a CTA or more
cases = [(100, 128 * 600 + 5, 288, 1, 128), (1100, 128 * 120, 288, 1, 256),
         (130, 128 * 60 + 5, 288, 8, 128)]
for fmt in (bb.MX_E8M0, bb.MX_E4M3):
    for M, N, K, E, rows in cases:
        p = bb.mx_launch_plan(E, M, N, K)
        assert p["rows"] == rows and p["split"] == 1 and p["tiles"] * rows >= 4 * 148 * 128, p
        off = (None if E == 1 else
               torch.arange(E + 1, dtype=torch.int32, device=dev) * (M // E) + 2)
        X = bb.mx_quantize(synth.make_activations(M, K, M, True, device=dev), fmt, groups=E, offsets=off)
        W = bb.mx_quantize(synth.make_weight(E * N, K, 3, device=dev), fmt, groups=E)
        want = torch.full((M, N), 3.0, device=dev)
        bb.mx_linear(X, W, out=want)
        assert torch.isfinite(want).all()
        got = torch.full((M, N), 5.0, device=dev)
        bb.inject_fault("wait")
        bb.mx_linear(X, W, out=got)
        torch.cuda.synchronize()
        bb.inject_fault(None)
        nan = got.isnan()
        inside = slice(0, M) if E == 1 else slice(2, int(off[-1]))
        rest = torch.ones(M, dtype=torch.bool, device=dev)
        rest[inside] = False
        assert (got[rest] == 5.0).all()
        # every tile was written: the first ones of each CTA, and NaN
        print("CASE", fmt, M, N, E, int(nan.sum()), int((got[inside] == 5.0).sum()),
              bool((nan | (got == want))[inside].all()))
        assert 0 < int(nan.sum()) < nan.numel()
        assert (nan | (got == want))[inside].all(), "tiles keep what was there"
        bb.mx_linear(X, W, out=got)
        assert torch.equal(got[inside], want[inside])
assert bb.device_timeouts() == 1
print("WAITS OK")
"""

_WAIT_LINEAR_CHILD = r"""
import torch
from activation_aware_codebook_b200 import binding as bb, synth
assert bb.load().aaac_checked_build() == 1, "not the checked build"
M, N, K = 1100, 128 * 120 + 5, 256  # 605 tiles of 128 x 256: four a CTA
cfg = bb.Config(bb.INT4, 128, 16, 1)
packed = bb.run_layer(synth.make_weight(N, K, 3, device="cuda"),
                      synth.make_activations(64, K, 4, True, device="cuda"), cfg)
x = synth.make_activations(M, K, 5, True, device="cuda")
ws = torch.empty(bb.linear_workspace_size(cfg, M, N, K), dtype=torch.uint8, device="cuda")
assert ws.numel() > 0
want = bb.linear(x, packed, cfg, N, K, ws=ws)
assert torch.isfinite(want).all()
got = torch.full((M, N), 5.0, device="cuda")
bb.inject_fault("wait")
bb.linear(x, packed, cfg, N, K, ws=ws, out=got)
torch.cuda.synchronize()
bb.inject_fault(None)
nan = got.isnan()
print("CASE", int(nan.sum()), int((got == 5.0).sum()), nan.numel())
assert 0 < int(nan.sum()) < nan.numel()
assert (nan | (got == want)).all(), "tiles keep what was there"
assert bb.device_timeouts() == 1
assert torch.equal(bb.linear(x, packed, cfg, N, K, ws=ws), want)
print("WAITS OK")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("child", [_WAIT_CHILD, _WAIT_LINEAR_CHILD], ids=["mx_linear", "linear"])
def test_a_product_whose_wait_runs_out_writes_nan_everywhere(child):
    """The epilogue gives up after a CTA's first tile: every later tile of the
    CTA is NaN, not what the buffer held; the status says so, and the next
    product on the same context is right."""
    cbuild.build(checks=True)
    env = dict(os.environ, AAAC_CHECKED="1", PYTHONPATH=ROOT)
    res = subprocess.run([sys.executable, "-c", child], env=env, cwd=ROOT, capture_output=True,
                         text=True, timeout=300)
    assert res.returncode == 0 and "WAITS OK" in res.stdout, res.stdout + res.stderr[-3000:]


def test_waits_run_out_in_checked_builds_only():
    cbuild.build()
    assert bb.load().aaac_inject_fault(b"wait") == 4  # AAAC_ERR_UNSUPPORTED
