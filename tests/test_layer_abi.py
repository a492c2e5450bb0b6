"""CPU tests of the layer operators' C ABI (include/nhm_layer.h): every declared symbol is exported, and bad arguments are
refused on the host before anything is enqueued; once more in a host build under AddressSanitizer and
UndefinedBehaviorSanitizer."""
import ctypes as C
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def nhm():
    import fp8_w8a8_linear_amd as m
    return m


def check(nhm, call, cases):
    for over, status in cases:
        st = call(**over)
        assert st == status, (over, st, nhm.lib.nhm_last_error())
        assert nhm.lib.nhm_last_error() != b""


def test_every_declared_symbol_is_exported(nhm):
    txt = open(os.path.join(ROOT, "include", "nhm_layer.h")).read()
    names = sorted(set(re.findall(r"NHM_API\s+[\w\s\*]+?\b(nhm_\w+)\s*\(", txt)))
    assert len(names) == 13 and all(n in nhm._SIGS and hasattr(nhm.lib, n) for n in names), names


def test_mxfp4_refusals(nhm):
    X, Q, S = 0x10000, 0x20000, 0x30000

    def quant(x=X, t=nhm.NHM_BF16, rows=4, cols=64, ldx=64, q=Q, ldq=32, s=S, lds=2):
        return nhm.lib.nhm_mxfp4_quantize(x, t, rows, cols, ldx, q, ldq, s, lds, None)

    assert quant(rows=0, x=None, q=None, s=None) == 0 and quant(cols=0, ldx=0, ldq=0, lds=0) == 0
    check(nhm, quant, [(dict(x=None), 1), (dict(q=None), 1), (dict(s=None), 1), (dict(t=1), 4), (dict(t=3), 4), (dict(rows=-1), 2),
                       (dict(cols=48), 2), (dict(ldx=56), 2), (dict(ldq=28), 2), (dict(lds=1), 2), (dict(x=X + 2), 3),
                       (dict(ldx=68), 3), (dict(t=2, ldx=66), 3), (dict(q=Q + 2), 3), (dict(ldq=33), 3)])

    def dequant(q=Q, ldq=32, s=S, lds=2, rows=4, cols=64, o=X, ldo=64):
        return nhm.lib.nhm_mxfp4_dequantize(q, ldq, s, lds, rows, cols, o, ldo, None)

    assert dequant(rows=0, q=None, s=None, o=None) == 0
    check(nhm, dequant, [(dict(q=None), 1), (dict(s=None), 1), (dict(o=None), 1), (dict(rows=-1), 2), (dict(cols=33), 2),
                         (dict(ldq=31), 2), (dict(lds=1), 2), (dict(ldo=63), 2), (dict(o=X + 8), 3), (dict(ldo=65), 3),
                         (dict(q=Q + 1), 3), (dict(ldq=34), 3)])


def test_mxfp4_linear_refusals(nhm):
    A, AS, W, S, O, WS = [0x10000 * i for i in range(1, 7)]
    need = nhm.mxfp4_linear_workspace_bytes(32, 64, 128, nhm.NHM_BF16)
    assert need >= 32 * 64 + 32 * 4 and need % 256 == 0
    assert nhm.mxfp4_linear_workspace_bytes(32, 64, 128, nhm.NHM_MXFP4) % 256 == 0
    assert nhm.mxfp4_linear_workspace_bytes(0, 64, 128, nhm.NHM_BF16) == 0

    def call(a=A, t=nhm.NHM_BF16, sa=None, m=32, lda=128, w=W, s=S, n=64, k=128, o=O, ot=nhm.NHM_BF16, ldo=64, ws=WS, wsb=need, p=None):
        wt = nhm._Mxfp4Weight(w, s, n, k, p)
        return nhm.lib.nhm_mxfp4_linear(a, t, sa, m, lda, C.byref(wt), o, ot, ldo, ws, wsb, None)

    assert call(m=0) == 0 and call(m=0, a=None, o=None, ws=None, wsb=0) == 0
    codes = dict(t=nhm.NHM_MXFP4, sa=AS, lda=64)
    check(nhm, call, [(dict(a=None), 1), (dict(o=None), 1), (dict(w=None), 1), (dict(s=None), 1), (dict(codes, sa=None), 1),
                      (dict(t=1), 4), (dict(t=2), 4), (dict(ot=1), 4), (dict(ot=3), 4), (dict(m=-1), 2), (dict(n=0), 2), (dict(k=0), 2),
                      (dict(k=112), 2), (dict(lda=120), 2), (dict(codes, lda=63), 2), (dict(ldo=63), 2), (dict(a=A + 8), 3),
                      (dict(lda=132), 3), (dict(codes, lda=72), 3), (dict(w=W + 8), 3), (dict(o=O + 1), 3),
                      (dict(ot=nhm.NHM_F32, o=O + 2), 3), (dict(ws=WS + 16), 3), (dict(ws=None), 5), (dict(wsb=need - 1), 5), (dict(p=S + 2), 3),
                      (dict(n=1 << 20, k=4096, lda=4096, ldo=1 << 20, wsb=1 << 60), 4),
                      (dict(codes, m=1 << 20, lda=4096, wsb=1 << 60), 4)])
    assert nhm.lib.nhm_mxfp4_linear(A, 0, None, 4, 64, None, O, 0, 64, WS, need, None) == 1
    size = nhm.lib.nhm_mxfp4_packed_scale_bytes
    assert size(10, 128) == 40 and size(10, 160) == 80 and size(10, 100) == 0 and size(0, 128) == 0

    def pack(s=S, n=10, k=160, p=W):
        return nhm.lib.nhm_mxfp4_pack_scales(s, n, k, p, None)

    assert pack(n=0, s=None, p=None) == 0
    check(nhm, pack, [(dict(s=None), 1), (dict(p=None), 1), (dict(n=-1), 2), (dict(k=100), 2), (dict(p=W + 2), 3),
                      (dict(n=1 << 30, k=128), 4)])


def test_conv_refusals(nhm):
    X, W, B, SL, CP, O, CU, HI = [0x10000 * i for i in range(1, 9)]

    def dec(x=X, ldx=64, w=W, b=B, dim=64, width=4, batch=4, sl=SL, cp=CP, slots=8, o=O, ldo=64):
        return nhm.lib.nhm_causal_conv_decode(x, ldx, w, b, dim, width, 1, batch, sl, cp, slots, o, ldo, None)

    def pre(x=X, ldx=64, T=40, w=W, b=B, dim=64, width=4, cu=CU, n=3, sl=SL, hi=HI, cp=CP, slots=8, o=O, ldo=64):
        return nhm.lib.nhm_causal_conv_prefill(x, ldx, T, w, b, dim, width, 1, cu, n, sl, hi, cp, slots, o, ldo, None)

    assert dec(batch=0) == 0 and dec(batch=0, x=None, o=None) == 0 and pre(T=0, n=0, x=None, o=None, cu=None, sl=None, hi=None) == 0
    both = [(dict(x=None), 1), (dict(w=None), 1), (dict(sl=None), 1), (dict(cp=None), 1), (dict(o=None), 1), (dict(dim=0), 2),
            (dict(slots=0), 2), (dict(ldx=56), 2), (dict(ldo=56), 2), (dict(width=1), 4), (dict(width=5), 4),
            (dict(dim=60), 4), (dict(x=X + 2), 3), (dict(ldx=66), 3), (dict(w=W + 8), 3), (dict(b=B + 2), 3), (dict(cp=CP + 4), 3),
            (dict(o=O + 8), 3), (dict(ldo=68), 3), (dict(sl=SL + 2), 3)]
    check(nhm, dec, both + [(dict(batch=-1), 2)])
    check(nhm, pre, both + [(dict(T=-1), 2), (dict(n=-1), 2), (dict(cu=None), 1), (dict(hi=None), 1), (dict(cu=CU + 2), 3),
                            (dict(hi=HI + 1), 3)])


def test_scan_refusals(nhm):
    U, DT, B, CC, Z, SL, SP, O, CU, HI, WS, A, D, BI = [0x10000 * i for i in range(1, 15)]

    def args(u=U, ldu=64, dt=DT, lddt=64, b=B, ldb=16, c=CC, ldc=16, z=Z, ldz=64):
        return u, ldu, dt, lddt, b, ldb, c, ldc, z, ldz

    def par(a=A, d=D, bi=BI, dim=64, n=16):
        return nhm._ScanParams(a, d, bi, dim, n)

    def split(kw):
        pk = {k: kw.pop(k) for k in ("a", "d", "bi", "dim", "n") if k in kw}
        ak = {k: kw.pop(k) for k in ("u", "ldu", "dt", "lddt", "b", "ldb", "c", "ldc", "z", "ldz") if k in kw}
        return par(**pk), args(**ak), kw

    def dec(**kw):
        p, a, kw = split(kw)
        d = dict(batch=4, sl=SL, sp=SP, t=nhm.NHM_F32, slots=8, o=O, ldo=64)
        d.update(kw)
        return nhm.lib.nhm_selective_scan_decode(C.byref(p), *a, d["batch"], d["sl"], d["sp"], d["t"], d["slots"], d["o"], d["ldo"], None)

    def pre(**kw):
        p, a, kw = split(kw)
        need = nhm.selective_scan_prefill_workspace_bytes(64, 16, 40, 3)
        d = dict(T=40, cu=CU, ns=3, sl=SL, hi=HI, sp=SP, t=nhm.NHM_F32, slots=8, o=O, ldo=64, ws=WS, wsb=need)
        d.update(kw)
        return nhm.lib.nhm_selective_scan_prefill(C.byref(p), *a, d["T"], d["cu"], d["ns"], d["sl"], d["hi"], d["sp"], d["t"],
                                                  d["slots"], d["o"], d["ldo"], d["ws"], d["wsb"], None)

    assert dec(batch=0) == 0 and dec(batch=0, u=None, dt=None, b=None, c=None, z=None, o=None) == 0
    assert pre(T=0, ns=0, u=None, dt=None, b=None, c=None, z=None, o=None, cu=None, sl=None, hi=None) == 0
    both = [(dict(a=None), 1), (dict(u=None), 1), (dict(dt=None), 1), (dict(b=None), 1), (dict(c=None), 1), (dict(sl=None), 1),
            (dict(sp=None), 1), (dict(o=None), 1), (dict(dim=0), 2), (dict(n=0), 2), (dict(slots=0), 2), (dict(ldu=63), 2),
            (dict(lddt=63), 2), (dict(ldb=15), 2), (dict(ldc=15), 2), (dict(ldz=63), 2), (dict(ldo=63), 2), (dict(dim=60), 4),
            (dict(n=6), 4), (dict(n=68, ldb=68, ldc=68), 4), (dict(ldu=(1 << 23) + 1), 4), (dict(t=1), 4), (dict(t=9), 4), (dict(a=A + 4), 3), (dict(sp=SP + 8), 3),
            (dict(d=D + 2), 3), (dict(bi=BI + 1), 3), (dict(u=U + 1), 3), (dict(z=Z + 1), 3), (dict(sl=SL + 2), 3), (dict(o=O + 1), 3)]
    check(nhm, dec, both + [(dict(batch=-1), 2)])
    check(nhm, pre, both + [(dict(T=-1), 2), (dict(ns=-1), 2), (dict(cu=None), 1), (dict(hi=None), 1), (dict(cu=CU + 2), 3)])
    assert nhm.lib.nhm_selective_scan_decode(None, *args(), 4, SL, SP, 2, 8, O, 64, None) == 1
    # a workspace that is needed: too short, missing, not aligned
    dim, T = 64, 1 << 16
    need = nhm.selective_scan_prefill_workspace_bytes(dim, 16, T, 1)
    if need:
        check(nhm, pre, [(dict(T=T, ns=1, wsb=need - 1), 5), (dict(T=T, ns=1, ws=None, wsb=need), 5),
                         (dict(T=T, ns=1, ws=WS + 128, wsb=need), 3)])


def test_logprob_refusals(nhm):
    X, T, LP, R, H, TL, TT, WS = [0x10000 * i for i in range(1, 9)]
    need = nhm.token_logprobs_workspace_bytes(4, 1000, 8)
    assert need > 0 and need % 256 == 0

    def call(x=X, t=nhm.NHM_F32, ld=1000, rows=4, vocab=1000, tok=T, n=8, lp=LP, r=R, h=H, tl=TL, tt=TT, ws=WS, wsb=need):
        return nhm.lib.nhm_token_logprobs(x, t, ld, rows, vocab, tok, n, lp, r, h, tl, tt, ws, wsb, None)

    assert call(rows=0, x=None, tl=None, tt=None, ws=None, wsb=0) == 0
    check(nhm, call, [(dict(x=None), 1), (dict(tl=None), 1), (dict(tt=None), 1), (dict(t=1), 4), (dict(t=3), 4), (dict(rows=-1), 2),
                      (dict(vocab=0), 2), (dict(n=-1), 2), (dict(ld=999), 2), (dict(n=65), 4),
                      (dict(vocab=(1 << 24) + 1, ld=1 << 25), 4), (dict(rows=1 << 24), 4), (dict(x=X + 2), 3), (dict(tok=T + 1), 3),
                      (dict(lp=LP + 2), 3), (dict(r=R + 1), 3), (dict(h=H + 2), 3), (dict(tl=TL + 2), 3), (dict(tt=TT + 2), 3),
                      (dict(ws=WS + 128), 3), (dict(ws=None), 5), (dict(wsb=need - 1), 5)])
    size = nhm.token_logprobs_workspace_bytes
    assert size(1 << 24, 10, 0) == 0 and size((1 << 24) - 1, 10, 0) > 0 and size(1, (1 << 24) + 1, 0) == 0 and size(1, 10, 65) == 0


def test_binding_refusals(nhm):
    """The binding refuses host tensors before a library call."""
    import torch
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    i32 = lambda *s: z(*s, dtype=torch.int32)  # noqa: E731
    for f in [lambda: nhm.mxfp4_quantize(z(4, 64)), lambda: nhm.mxfp4_dequantize(z(4, 32, dtype=torch.uint8), z(4, 2, dtype=torch.uint8)),
              lambda: nhm.Mxfp4Weight(z(4, 32, dtype=torch.uint8), z(4, 2, dtype=torch.uint8)),
              lambda: nhm.causal_conv_decode(z(4, 64), z(64, 4), None, i32(4), z(8, 3, 64)),
              lambda: nhm.causal_conv_prefill(z(4, 64), z(64, 4), None, i32(2), i32(1), i32(1), z(8, 3, 64)),
              lambda: nhm.ScanParams(z(64, 16, dtype=torch.float32)), lambda: nhm.token_logprobs(z(4, 100), i32(4))]:
        with pytest.raises(TypeError):
            f()


def test_validation_under_asan_ubsan(tmp_path):
    hipcc = next((c for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")) if c and os.path.exists(c)),
                 None)
    if not hipcc:
        pytest.skip("hipcc not found")
    exe = str(tmp_path / "layer_validation")
    # the sanitizer flags apply to the host pass only
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    cmd = [hipcc, "-std=c++17", "-O1", "-g", "--offload-arch=gfx950", *san, "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "fp8_w8a8_linear_amd", "csrc", "layer.hip"),
           os.path.join(ROOT, "tests", "c", "layer_validation.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0 and "layer validation ok" in r.stdout, r.stdout + r.stderr
