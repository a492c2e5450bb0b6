"""CPU tests of the serving operators' C ABI (include/nhm_serving.h): every declared symbol is exported, and bad
arguments are refused on the host before anything is enqueued. The same calls run once more in a host build under
AddressSanitizer and UndefinedBehaviorSanitizer."""
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


def test_every_declared_symbol_is_exported(nhm):
    txt = open(os.path.join(ROOT, "include", "nhm_serving.h")).read()
    names = sorted(set(re.findall(r"NHM_API\s+[\w\s\*]+?\b(nhm_\w+)\s*\(", txt)))
    assert names and all(n in nhm._SIGS and hasattr(nhm.lib, n) for n in names), names


def test_lora_refusals(nhm):
    A, W, S, LA, LB, LS, ID, O, WS = [0x10000 * i for i in range(1, 10)]
    need = nhm.fp8_linear_lora_workspace_bytes(32, 64, 128, nhm.NHM_BF16, 16)
    assert need >= 32 * 128 and need % 256 == 0
    assert nhm.fp8_linear_lora_workspace_bytes(0, 64, 128, nhm.NHM_BF16, 16) == 0
    assert nhm.fp8_linear_lora_workspace_bytes(32, 64, 128, nhm.NHM_BF16, 12) == 0

    def call(a=A, t=nhm.NHM_BF16, m=32, lda=128, w=W, ws=S, sa=S, n=64, k=128, la=LA, lb=LB, ls=LS, e=4, rank=16, ids=ID,
             out=O, ot=nhm.NHM_BF16, ldo=64, wsp=WS, wsb=need, per_tensor=0):
        wt, lo = nhm._Fp8Weight(w, ws, sa, n, k, per_tensor), nhm._Lora(la, lb, ls, e, rank)
        return nhm.lib.nhm_fp8_linear_lora(a, t, m, lda, C.byref(wt), C.byref(lo), ids, out, ot, ldo, 0, wsp, wsb, None)

    assert call(m=0) == 0 and call(m=0, a=None, out=None, ids=None, wsp=None, wsb=0) == 0
    for over, status in [(dict(a=None), 1), (dict(out=None), 1), (dict(w=0), 1), (dict(la=0), 1), (dict(lb=0), 1),
                         (dict(ids=None), 1), (dict(e=0), 2), (dict(e=-3), 2), (dict(m=-1), 2), (dict(lda=120), 2),
                         (dict(ldo=63), 2), (dict(k=100), 2), (dict(n=0), 2), (dict(rank=0), 4), (dict(rank=4), 4),
                         (dict(rank=12), 4), (dict(rank=136), 4), (dict(rank=-8), 4), (dict(t=2), 4), (dict(t=9), 4),
                         (dict(ot=1), 4), (dict(per_tensor=3), 4), (dict(a=A + 2), 3), (dict(lda=132), 3),
                         (dict(la=LA + 8), 3), (dict(lb=LB + 2), 3), (dict(ls=LS + 2), 3), (dict(ids=ID + 1), 3),
                         (dict(out=O + 1), 3), (dict(ot=nhm.NHM_F32, out=O + 2), 3), (dict(wsp=WS + 16), 3),
                         (dict(wsp=None), 5), (dict(wsb=need - 1), 5)]:
        st = call(**over)
        assert st == status, (over, st, nhm.lib.nhm_last_error())
        assert nhm.lib.nhm_last_error() != b""
    lo = nhm._Lora(LA, LB, LS, 4, 16)
    wt = nhm._Fp8Weight(W, S, S, 64, 128, 0)
    assert nhm.lib.nhm_fp8_linear_lora(A, 0, 32, 128, None, C.byref(lo), ID, O, 0, 64, 0, WS, need, None) == 1
    assert nhm.lib.nhm_fp8_linear_lora(A, 0, 32, 128, C.byref(wt), None, ID, O, 0, 64, 0, WS, need, None) == 1
    big = nhm._Fp8Weight(W, S, S, 1 << 19, 4096, 0)                   # a weight of 2 GiB
    assert nhm.lib.nhm_fp8_linear_lora(A, 0, 8, 4096, C.byref(big), C.byref(lo), ID, O, 0, 1 << 19, 0, WS, 1 << 62, None) == 4


def _mixer_args(nhm):
    g = nhm.Geometry(**nhm.GEOMETRY)
    w = lambda n, k: nhm._Fp8Weight(0x1000, 0x2000, 0x3000, n, k, 0)  # noqa: E731
    return nhm._MixerParams(g, w(10304, 2688), w(2688, 4096), 0x5000, 0x6000, 0x7000, 0x8000, 0x9000, 0xA000)


def test_mixer_lora_refusals(nhm):
    """The mixer calls with adapters: their checks of the adapter sets, then those of the calls without."""
    H, SL, SP, CP, O, WS, ID, CU, HI = [0x100000 * i for i in range(1, 10)]
    p = _mixer_args(nhm)
    ok = nhm._Lora(0x10000, 0x20000, 0x30000, 4, 16)
    big = nhm._Lora(0x10000, 0x20000, None, 4, 64)

    def dec(li=ok, lo=big, ids=ID, hidden=H, batch=8, wsb=None, ws=WS, pp=p):
        ref = lambda l: None if l is None else C.byref(l)  # noqa: E731
        wsb = nhm.decode_lora_ws_layout(8, 64)["total"] if wsb is None else wsb
        return nhm.lib.nhm_mixer_decode_lora(None if pp is None else C.byref(pp), ref(li), ref(lo), ids, hidden, batch, SL, SP,
                                             nhm.NHM_F32, CP, 64, O, ws, wsb, None)

    def pre(li=ok, lo=big, ids=ID, hidden=H, T=40, n=2, wsb=None):
        ref = lambda l: None if l is None else C.byref(l)  # noqa: E731
        wsb = nhm.prefill_lora_ws_layout(40, 2, 64)["total"] if wsb is None else wsb
        return nhm.lib.nhm_mixer_prefill_lora(C.byref(p), ref(li), ref(lo), ids, hidden, T, CU, n, SL, HI, 128, SP, nhm.NHM_F32,
                                              CP, 64, O, WS, wsb, None)

    assert dec(batch=0) == 0 and dec(batch=0, ids=None) == 0 and pre(T=0, n=0) == 0
    assert dec(pp=None) == 1
    for call, need in ((dec, nhm.decode_lora_ws_layout(8, 64)["total"]), (pre, nhm.prefill_lora_ws_layout(40, 2, 64)["total"])):
        for over, status in [(dict(ids=None), 1), (dict(ids=ID + 2), 3), (dict(hidden=None), 1), (dict(hidden=H + 8), 3),
                             (dict(wsb=need - 1), 5), (dict(li=nhm._Lora(0, 0x20000, None, 4, 16)), 1),
                             (dict(lo=nhm._Lora(0x10000, 0x20008, None, 4, 16)), 3),
                             (dict(li=nhm._Lora(0x10000, 0x20000, None, 0, 16)), 2),
                             (dict(lo=nhm._Lora(0x10000, 0x20000, None, 4, 20)), 4)]:
            st = call(**over)
            assert st == status, (call, over, st, nhm.lib.nhm_last_error())
    assert pre(T=-1) == 2 and pre(T=1 << 31) == 2 and dec(batch=-1) == 2
    base = nhm.decode_ws_layout(8)
    lay = nhm.decode_lora_ws_layout(8, 64)
    assert lay["total"] > base["total"] and all(lay[k] == base[k] for k in base if k != "total")
    assert nhm.prefill_lora_ws_layout(512, 2, 8)["total"] > nhm.prefill_ws_layout(512, 2)["total"]
    for bad in (0, 4, 12, 136):
        with pytest.raises(nhm.NhmError):
            nhm.decode_lora_ws_layout(8, bad)
        with pytest.raises(nhm.NhmError):
            nhm.prefill_lora_ws_layout(512, 2, bad)


def test_beam_select_refusals(nhm):
    X, CU, FI, SC, PA, TO, WS = [0x10000 * i for i in range(1, 8)]
    need = nhm.beam_select_workspace_bytes(2, 4, 1000, 8)
    assert need > 0 and need % 256 == 0
    for bad in [(0, 4, 1000, 8), (2, 0, 1000, 8), (2, 33, 1000, 8), (2, 4, 0, 8), (2, 4, (1 << 24) + 1, 8),
                (2, 4, 1000, 0), (2, 4, 1000, 65), (1 << 24, 4, 1000, 8), (-1, 4, 1000, 8)]:
        assert nhm.beam_select_workspace_bytes(*bad) == 0

    def call(x=X, t=nhm.NHM_F32, ld=1000, G=2, K=4, V=1000, cum=CU, fin=None, eos=0, n=8, sc=SC, pa=PA, to=TO, ws=WS,
             wsb=need):
        return nhm.lib.nhm_beam_select(x, t, ld, G, K, V, cum, fin, eos, n, sc, pa, to, ws, wsb, None)

    assert call(G=0) == 0 and call(G=0, x=None, cum=None, ws=None, wsb=0) == 0
    for over, status in [(dict(x=None), 1), (dict(cum=None), 1), (dict(sc=None), 1), (dict(pa=None), 1), (dict(to=None), 1),
                         (dict(G=-1), 2), (dict(K=0), 2), (dict(V=0, ld=0), 2), (dict(n=0), 2), (dict(ld=999), 2),
                         (dict(fin=FI, eos=-1), 2), (dict(fin=FI, eos=1000), 2), (dict(t=nhm.NHM_E4M3), 4), (dict(t=-7), 4),
                         (dict(K=33), 4), (dict(n=65), 4), (dict(V=(1 << 24) + 1, ld=1 << 25), 4), (dict(G=1 << 23), 4),
                         (dict(x=X + 2), 3), (dict(t=nhm.NHM_BF16, x=X + 1), 3), (dict(cum=CU + 1), 3),
                         (dict(fin=FI + 2), 3), (dict(sc=SC + 2), 3), (dict(pa=PA + 1), 3), (dict(to=TO + 3), 3),
                         (dict(ws=WS + 8), 3), (dict(ws=None), 5), (dict(wsb=need - 1), 5)]:
        st = call(**over)
        assert st == status, (over, st, nhm.lib.nhm_last_error())


def test_beam_reorder_refusals(nhm):
    PA, SL, NW, SP, CP = [0x10000 * i for i in range(1, 6)]

    def call(g=None, pa=PA, sl=SL, G=2, K=4, layers=2, sp=SP, cp=CP, t=nhm.NHM_F32, S=16, nw=NW, arr=True):
        geo = nhm.Geometry(**dict(nhm.GEOMETRY, **(g or {})))
        a = (nhm._StatePool * max(layers, 1))(*[(sp, cp)] * max(layers, 1))
        return nhm.lib.nhm_beam_reorder(C.byref(geo), pa, sl, G, K, a if arr else None, layers, t, S, nw, None)

    assert call(G=0) == 0
    for over, status in [(dict(pa=None), 1), (dict(sl=None), 1), (dict(nw=None), 1), (dict(arr=False), 1), (dict(sp=None), 1),
                         (dict(cp=None), 1), (dict(G=-1), 2), (dict(K=0), 2), (dict(layers=0), 2), (dict(S=0), 2),
                         (dict(K=33), 4), (dict(layers=65), 4), (dict(G=1 << 23), 4), (dict(t=nhm.NHM_E4M3), 4),
                         (dict(g=dict(d_state=64)), 4), (dict(nw=SL), 4), (dict(nw=PA + 16), 4), (dict(pa=PA + 2), 3),
                         (dict(sl=SL + 1), 3), (dict(nw=NW + 2), 3), (dict(sp=SP + 8), 3), (dict(cp=CP + 4), 3)]:
        st = call(**over)
        assert st == status, (over, st, nhm.lib.nhm_last_error())
    assert nhm.lib.nhm_beam_reorder(None, PA, SL, 2, 4, None, 1, 2, 16, NW, None) == 1


def test_batch_plan_refusals(nhm):
    L, P, A, CU, HI, TS, TP, TA = [0x10000 * i for i in range(1, 9)]

    def call(ln=L, past=P, ad=A, n=4, T=100, cu=CU, hi=HI, ts=TS, tp=TP, ta=TA):
        return nhm.lib.nhm_batch_plan(ln, past, ad, n, T, cu, hi, ts, tp, ta, None)

    for over, status in [(dict(ln=None), 1), (dict(cu=None), 1), (dict(hi=None), 1), (dict(n=-1), 2), (dict(T=-1), 2),
                         (dict(T=1 << 31), 2), (dict(n=8193), 4), (dict(ln=L + 2), 3), (dict(past=P + 1), 3),
                         (dict(ad=A + 2), 3), (dict(cu=CU + 2), 3), (dict(hi=HI + 2), 3), (dict(ts=TS + 1), 3),
                         (dict(tp=TP + 2), 3), (dict(ta=TA + 3), 3)]:
        st = call(**over)
        assert st == status, (over, st, nhm.lib.nhm_last_error())


def test_binding_refuses_host_tensors(nhm):
    """The binding checks what it passes on: device, dtype, shape, layout."""
    import torch
    with pytest.raises(TypeError):
        nhm.Lora(torch.zeros(2, 8, 16, dtype=torch.bfloat16), torch.zeros(2, 4, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        nhm.Lora(torch.zeros(2, 8, 16, dtype=torch.bfloat16), torch.zeros(3, 4, 8, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        nhm.beam_select(torch.zeros(4, 10), torch.zeros(2, 2), 3)
    with pytest.raises(ValueError):
        nhm.beam_select(torch.zeros(4, 10), torch.zeros(3, 2), 3)
    with pytest.raises(ValueError):
        nhm.beam_reorder(torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32), [], [])


def test_validation_under_asan_ubsan(tmp_path):
    hipcc = next((c for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")) if c and os.path.exists(c)),
                 None)
    if not hipcc:
        pytest.skip("hipcc not found")
    exe = str(tmp_path / "serving_validation")
    csrc = os.path.join(ROOT, "fp8_w8a8_linear_amd", "csrc")
    # the sanitizer flags apply to the host pass only
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    cmd = [hipcc, "-std=c++17", "-O1", "-g", "--offload-arch=gfx950", *san, "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), os.path.join(csrc, "api.hip"),
           os.path.join(csrc, "serving.hip"), os.path.join(ROOT, "tests", "c", "serving_validation.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0 and "serving validation ok" in r.stdout, r.stdout + r.stderr


def test_limits_are_the_documented_ones(nhm):
    """n_groups * n_beams below 2^24 for a selection, up to 2^24 for a reorder."""
    size = nhm.lib.nhm_beam_select_workspace_bytes
    assert size(1 << 24, 1, 10, 1) == 0 and size((1 << 24) - 1, 1, 10, 1) > 0
    assert size(1 << 22, 4, 10, 1) == 0 and size((1 << 22) - 1, 4, 10, 1) > 0
    assert size(1 << 19, 32, 10, 1) == 0 and size(((1 << 24) - 1) // 32, 32, 10, 1) > 0
    X, CU, SC, PA, TO, WS = [0x10000 * i for i in range(1, 7)]
    for G, K in [(1 << 24, 1), (1 << 22, 4), (1 << 19, 32)]:
        st = nhm.lib.nhm_beam_select(X, nhm.NHM_F32, 10, G, K, 10, CU, None, 0, 1, SC, PA, TO, WS, 1 << 60, None)
        assert st == 4, (G, K, nhm.lib.nhm_last_error())
    geo = nhm.Geometry(**nhm.GEOMETRY)
    pool = (nhm._StatePool * 1)((X, X))
    for G, K in [((1 << 24) + 1, 1), ((1 << 22) + 1, 4)]:
        assert nhm.lib.nhm_beam_reorder(C.byref(geo), PA, SC, G, K, pool, 1, nhm.NHM_F32, 16, TO, None) == 4
