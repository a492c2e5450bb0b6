"""Which tile of the MXFP4 projection a product of many rows takes, and how many of them follow one another in a workgroup: what
the GPU tests of those paths rely on."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# m, n, k, codes in, f32 out, the tile's features and rows, tiles in turn of a workgroup. n of whole 16-byte stores and not, k of less
# than a slice, of a few and of more than the ring's stages, whole slices and not.
TILE_CASES = [
    (5300, 5000, 160, True, False, 256, 256, 2), (5300, 5001, 352, False, False, 256, 256, 2), (7400, 6600, 96, False, False, 256, 256, 3),
    (7400, 6603, 736, True, False, 256, 256, 3), (5376, 5120, 128, True, False, 256, 256, 2),
    (3000, 3000, 160, True, True, 128, 128, 2), (2999, 3001, 288, False, True, 128, 128, 2), (3000, 3000, 96, False, False, 128, 128, 2),
    (3001, 3003, 416, True, False, 128, 128, 2), (4200, 4200, 32, True, True, 128, 128, 3), (4200, 4200, 544, True, False, 128, 128, 3),
    (1000, 4100, 672, True, False, 128, 64, 1), (1000, 4101, 160, False, True, 128, 64, 1), (477, 2688, 544, True, True, 64, 64, 1),
    (90, 1001, 288, False, False, 64, 64, 1),
]


def test_tiles(tmp_path):
    hipcc = next((c for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")) if c and os.path.exists(c)), None)
    if not hipcc:
        pytest.skip("hipcc not found")
    exe = str(tmp_path / "mx_tiles")
    cmd = [hipcc, "-std=c++17", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I",
           os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "c", "mx_tiles.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    args = [str(int(v)) for m, n, _, _, f32, *_ in TILE_CASES for v in (m, n, f32)]
    r = subprocess.run([exe, *args], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    for case, line in zip(TILE_CASES, r.stdout.splitlines(), strict=False):
        m, n, tn, tm, turns = *case[:2], *case[5:]
        got = tuple(int(v) for v in line.split())
        tiles = -(-n // tn) * -(-m // tm)
        assert got[:2] == (tn, tm) and -(-tiles // (256 * got[2])) == turns, (case, got, tiles)
    assert len(r.stdout.splitlines()) == len(TILE_CASES)


def test_more_features_than_a_launch_holds():
    """Up to 64 rows a workgroup of 512 threads takes 16 features, and a launch holds fewer than 2^32 threads: 2^27 - 15 features, whose
    codes are still below 2 GiB, are refused on the host."""
    import ctypes as C

    import fp8_w8a8_linear_amd as nhm
    n, k = (1 << 27) - 15, 32
    assert n * k // 2 < 1 << 31
    for m in (1, 4, 5, 64):
        need = nhm.mxfp4_linear_workspace_bytes(m, n, k, nhm.NHM_BF16)
        w = nhm._Mxfp4Weight(0x10000, 0x20000, n, k, None)
        status = nhm.lib.nhm_mxfp4_linear(0x30000, nhm.NHM_BF16, None, m, k, C.byref(w), 0x40000, nhm.NHM_BF16, n, 0x50000, need, None)
        assert status == 4, (m, status, nhm.lib.nhm_last_error())
