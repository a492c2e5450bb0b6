"""The serving operators on the GPU against the float64 oracle: adapters beside a projection, beam
selection, state reorder, batch plan, each at the sizes, masks and orders where it can go wrong."""
import ctypes as C

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import serving_oracle as so  # noqa: E402


@pytest.fixture(scope="module")
def nhm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_w8a8_linear_amd as m
    return m


def bits(a):
    from workloads import bf16_bits
    return bf16_bits(np.asarray(a, np.float32))


def widen(t, f32):
    from oracle import bf16_to_f64
    from tests.gpu_util import host
    return t.cpu().numpy().astype(np.float64) if f32 else bf16_to_f64(host(t))


# ---------------------------------------------------------------- adapters beside a projection

def lora_inputs(m, n, k, rank, adapters, seed, order="mixed", bare=0.15, codes=False, scaled=True):
    from oracle import quantize_static
    from workloads import linear_case
    r = np.random.default_rng(seed)
    a, w, ws, sa = linear_case(m, n, k, extra=seed)
    if codes:
        a = quantize_static(a, sa)
    la = bits(r.standard_normal((adapters, rank, k), dtype=np.float32) / np.sqrt(k))
    lb = bits(r.standard_normal((adapters, n, rank), dtype=np.float32) * 0.02)
    ls = r.choice([0.25, -1.0, 2.0], adapters).astype(np.float32) if scaled else None
    ids = r.integers(0, adapters, m).astype(np.int32)
    ids[r.random(m) < bare] = -1
    if order == "runs":
        ids = np.sort(ids)[::-1].copy()
    return a, w, ws, sa, la, lb, ls, ids


def lora_device(nhm, inp):
    from tests.gpu_util import dev
    a, w, ws, sa, la, lb, ls, ids = inp
    W = nhm.Fp8Weight(dev(w), dev(ws), dev(sa))
    L = nhm.Lora(dev(la), dev(lb), None if ls is None else dev(ls))
    return dev(a), W, L, dev(ids)


LORA_CASES = [
    # m, n, k, rank, adapters, order, codes, f32, exact
    (1, 10304, 2688, 16, 3, "mixed", False, False, False),
    (1, 37, 16, 8, 1, "mixed", False, True, True),
    (2, 100, 2960, 24, 5, "mixed", True, False, False),
    (8, 10304, 2688, 64, 16, "mixed", False, False, False),
    (16, 2688, 4096, 128, 40, "mixed", False, True, True),
    (16, 4099, 9008, 40, 16, "mixed", True, True, True),
    (17, 2688, 4096, 8, 4, "mixed", True, False, True),
    (33, 77, 48, 128, 33, "mixed", False, True, True),
    (61, 2688, 4096, 32, 32, "mixed", True, True, True),
    (61, 1001, 2688, 72, 7, "runs", False, False, False),
    (130, 10304, 528, 64, 9, "mixed", False, False, True),
    (257, 10304, 2688, 16, 4, "runs", False, False, True),
    (300, 10307, 272, 120, 64, "mixed", False, True, True),
    (641, 1000, 1040, 32, 5, "runs", False, False, False),
    (641, 1003, 176, 56, 5, "mixed", False, True, True),
    (700, 10304, 336, 64, 3, "runs", True, False, False),
    (3000, 4100, 144, 48, 6, "runs", False, False, True),
    (3000, 4101, 144, 128, 200, "mixed", False, True, True),
    (5, 70, 16400, 16, 4, "mixed", False, True, True),           # k past the GEMV's: a tile of five rows
    (9, 130, 16448, 24, 9, "mixed", True, False, False),
    (9000, 300, 272, 40, 7, "runs", False, False, True),         # many rows: their low-rank kernel
    (8193, 77, 176, 128, 300, "mixed", True, True, True),
    (8200, 260, 48, 8, 12, "mixed", False, False, True),
    (15000, 64, 16, 64, 5, "runs", False, True, True),
    (50, 8001, 272, 40, 20, "mixed", False, False, False),       # 32 and 48 features to a workgroup, rows past 64
    (64, 10304, 336, 128, 70, "mixed", True, True, True),
    (45, 10300, 144, 64, 3, "mixed", False, False, True),
    (199, 2690, 1040, 16, 90, "mixed", True, False, False),
    (640, 513, 528, 32, 300, "mixed", False, True, True),
    (64, 20000, 272, 48, 30, "mixed", False, False, False),      # past it: the panel kernel
]


@pytest.mark.parametrize("m,n,k,rank,adapters,order,codes,f32,exact", LORA_CASES)
def test_lora_linear(nhm, m, n, k, rank, adapters, order, codes, f32, exact):
    print(f"lora m={m} n={n} k={k} rank={rank} adapters={adapters} {order} codes={codes} f32={f32} exact={exact}", flush=True)
    inp = lora_inputs(m, n, k, rank, adapters, seed=m + rank, order=order, codes=codes, scaled=rank != 24)
    x, W, L, ids = lora_device(nhm, inp)
    o = nhm.fp8_linear_lora(x, W, L, ids, out_type=nhm.NHM_F32 if f32 else nhm.NHM_BF16, exact=exact)
    again = nhm.fp8_linear_lora(x, W, L, ids, out_type=nhm.NHM_F32 if f32 else nhm.NHM_BF16, exact=exact)
    torch.cuda.synchronize()
    assert torch.equal(o, again)
    got = widen(o, f32)
    ref = so.fp8_linear_lora(*inp, codes=codes)
    tol = so.lora_bound(*inp, ref, codes=codes, exact=exact or m <= 16, f32=f32)
    err = np.abs(got - ref)
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert np.all(err <= tol), f"at {worst}: got {got[worst]} ref {ref[worst]} tol {tol[worst]}"
    print(f"  worst err/tol {np.max(err / tol):.3f}")


@pytest.mark.parametrize("m,n,k,exact,f32", [(3, 10304, 2688, False, False), (8, 2688, 4096, False, True),
                                             (61, 2688, 4096, True, False), (61, 2688, 4096, False, False),
                                             (257, 10304, 2688, True, False), (257, 10304, 2688, False, True),
                                             (700, 10304, 336, True, False), (700, 10304, 336, False, False),
                                             (641, 1000, 1040, False, True), (50, 10304, 336, True, False),
                                             (64, 8001, 528, False, True), (300, 2690, 272, False, False),
                                             (64, 20000, 272, False, False)])
def test_lora_rows_without_adapter(nhm, m, n, k, exact, f32):
    """Rows without an adapter (negative or past the set) hold the projection alone, bit for bit, whatever rows with
    one share their tiles."""
    inp = list(lora_inputs(m, n, k, 16, 3, seed=5))
    ids = np.full(m, -1, np.int32)
    ids[1::3] = 3
    ids[2::3] = 2 ** 31 - 1
    ids[5::7] = 1
    inp[7] = ids
    x, W, L, idd = lora_device(nhm, inp)
    t = nhm.NHM_F32 if f32 else nhm.NHM_BF16
    got = nhm.fp8_linear_lora(x, W, L, idd, out_type=t, exact=exact)
    codes_only = torch.zeros((m * k + 255) // 256 * 256, dtype=torch.uint8, device="cuda")   # no split over k
    base = nhm.fp8_linear(x, W, ws=codes_only, out_type=t, exact=exact)
    torch.cuda.synchronize()
    bare = torch.from_numpy((ids < 0) | (ids >= 3)).cuda()
    assert torch.equal(got[bare], base[bare])
    assert not torch.equal(got[~bare], base[~bare]) or not bool((~bare).any())


@pytest.mark.parametrize("m,n,k", [(7, 300, 272), (50, 300, 272), (64, 20000, 272), (257, 10304, 272), (641, 1000, 1040),
                                   (700, 10304, 336)])
def test_lora_rows_without_adapter_keep_the_sign_of_zero(nhm, m, n, k):
    """A zero row without an adapter under negative weight scales is -0 with and without its neighbours' adapters."""
    inp = list(lora_inputs(m, n, k, 16, 3, seed=15))
    inp[0][::2] = 0
    inp[2] = -np.abs(inp[2])
    inp[7] = np.where(np.arange(m) % 2 == 0, -1, 1).astype(np.int32)
    x, W, L, idd = lora_device(nhm, inp)
    for t in (nhm.NHM_BF16, nhm.NHM_F32):
        got = nhm.fp8_linear_lora(x, W, L, idd, out_type=t)
        base = nhm.fp8_linear(x, W, out_type=t)
        torch.cuda.synchronize()
        bits_of = lambda o: o[::2].view(torch.int32 if t == nhm.NHM_F32 else torch.int16)  # noqa: E731
        assert torch.equal(bits_of(got), bits_of(base))
        assert bool((bits_of(base) < 0).all())


@pytest.mark.parametrize("m,n,k", [(8, 2688, 4096), (61, 2688, 4096), (257, 10304, 272), (700, 10304, 336),
                                   (641, 1000, 1040), (50, 10304, 336), (64, 8001, 528), (300, 2690, 272),
                                   (64, 20000, 272)])
def test_lora_rows_keep_to_their_adapter(nhm, m, n, k):
    """NaN and infinities in other adapters, and in other rows, do not reach a row."""
    inp = list(lora_inputs(m, n, k, 24, 4, seed=9, bare=0.2))
    a, _, _, _, la, lb, _, ids = inp
    ids[0], ids[1], ids[2] = 0, 3, -1
    x, W, L, idd = lora_device(nhm, inp)
    clean = nhm.fp8_linear_lora(x, W, L, idd)
    la2, lb2, a2 = la.copy(), lb.copy(), a.copy()
    la2[3, :, ::5] = 0x7FC0                  # NaN
    lb2[3, ::3] = 0x7F80                     # +inf
    lb2[3, 1::3] = 0xFF80
    a2[1, 7] = 0x7FC0
    inp2 = [a2, inp[1], inp[2], inp[3], la2, lb2, inp[6], ids]
    x2, W2, L2, idd2 = lora_device(nhm, inp2)
    got = nhm.fp8_linear_lora(x2, W2, L2, idd2)
    torch.cuda.synchronize()
    keep = torch.from_numpy((ids != 3) & (np.arange(m) != 1)).cuda()
    assert torch.equal(got[keep], clean[keep])
    assert bool(torch.isnan(got.view(torch.bfloat16)[1].float()).any())


@pytest.mark.parametrize("m,n,k", [(7, 2690, 4096), (61, 2688, 4096), (60, 9999, 272), (64, 20000, 528), (257, 10304, 272), (700, 10304, 336), (641, 1000, 1040)])
def test_lora_per_tensor_weight_scale(nhm, m, n, k):
    """One weight scale for the whole projection gives what the same value in every channel gives, bit for bit."""
    from tests.gpu_util import dev
    from workloads import linear_case
    inp = list(lora_inputs(m, n, k, 16, 3, seed=31))
    _, w, ws, _ = linear_case(m, n, k, extra=77, per_tensor=True)
    inp[1], inp[2] = w, ws
    x, W, L, ids = lora_device(nhm, inp)
    W1 = nhm.Fp8Weight(dev(w), dev(ws[:1].copy()), dev(inp[3]))
    assert W1.per_tensor
    a = nhm.fp8_linear_lora(x, W, L, ids)
    b = nhm.fp8_linear_lora(x, W1, L, ids)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_lora_strides_through_the_abi(nhm):
    """Row strides above k and n; the padding is not touched."""
    from tests.gpu_util import dev, host
    from oracle import bf16_to_f64
    for m, n, k, lda, ldo in [(5, 100, 272, 320, 104), (5, 101, 272, 280, 103), (50, 2690, 528, 544, 2693),
                              (300, 10304, 272, 288, 10312), (700, 10304, 272, 280, 10305)]:
        inp = lora_inputs(m, n, k, 16, 3, seed=21)
        a, w, ws, sa, la, lb, ls, ids = inp
        ap = np.zeros((m, lda), np.uint16)
        ap[:, :k] = a
        ap[:, k:] = 0x7FC0
        x = dev(ap)
        _, W, L, idd = lora_device(nhm, inp)
        out = torch.full((m, ldo), 0x1234, dtype=torch.int16, device="cuda")
        need = nhm.fp8_linear_lora_workspace_bytes(m, n, k, nhm.NHM_BF16, 16)
        wsb = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
        st = nhm.lib.nhm_fp8_linear_lora(x.data_ptr(), nhm.NHM_BF16, m, lda, C.byref(W.struct), C.byref(L.struct),
                                         idd.data_ptr(), out.data_ptr(), nhm.NHM_BF16, ldo, 1, wsb.data_ptr(), need,
                                         torch.cuda.current_stream().cuda_stream)
        assert st == 0, nhm.lib.nhm_last_error()
        torch.cuda.synchronize()
        o = host(out)
        ref = so.fp8_linear_lora(*inp)
        assert np.all(np.abs(bf16_to_f64(o[:, :n]) - ref) <= so.lora_bound(*inp, ref, f32=False))
        assert np.all(o[:, n:] == 0x1234)
        assert bool((wsb[need:] == 0x5A).all())


def test_lora_captured_and_on_a_stream(nhm):
    """A captured call, replayed with new adapters per row between eager calls, and a call on a side stream."""
    inp = lora_inputs(8, 10304, 2688, 32, 6, seed=3)
    x, W, L, ids = lora_device(nhm, inp)
    ws = torch.empty(nhm.fp8_linear_lora_workspace_bytes(8, 10304, 2688, nhm.NHM_BF16, 32), dtype=torch.uint8, device="cuda")
    out = torch.empty((8, 10304), dtype=torch.int16, device="cuda")
    nhm.fp8_linear_lora(x, W, L, ids, out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nhm.fp8_linear_lora(x, W, L, ids, out=out, ws=ws)
    for shift in range(4):
        ids.copy_((ids + shift) % 6)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = nhm.fp8_linear_lora(x, W, L, ids)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), shift
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2 = nhm.fp8_linear_lora(x, W, L, ids, out=torch.empty_like(out), stream=side,
                             ws=torch.empty_like(ws))
    side.synchronize()
    assert torch.equal(o2, eager)


def test_lora_zero_rows(nhm):
    inp = lora_inputs(1, 64, 128, 8, 2, seed=1)
    x, W, L, ids = lora_device(nhm, inp)
    out = nhm.fp8_linear_lora(x[:0], W, L, ids[:0])
    assert out.shape == (0, 64)


# ---------------------------------------------------------------- beam selection

# A score's error: its f32 rounding, 2^-24 |score|, and the error of log(sum): each f32 exponential is off
# by |d| 2^-24 (its scaled argument) + 2^-22 (the instruction) of itself, and |d| e^-|d| <= 0.37; the f32
# partial sums of at most 64 terms add 64 2^-24. Together under 72 2^-24 of the sum, absolute in the log.
def score_tol(ref):
    return 2.0 ** -24 * np.abs(ref) + 72 * 2.0 ** -24


def check_select(nhm, x, cum, n_cand, finished=None, eos=0, f32=True, dev_logits=None, ld=None):
    from oracle import bf16_to_f64
    from tests.gpu_util import dev
    G, K, V = x.shape
    if f32:
        xs = x.astype(np.float32)
        ref_x = xs.astype(np.float64)
    else:
        xs = bits(x)
        ref_x = bf16_to_f64(xs)
    s, p, t, gap = so.beam_select(ref_x, cum, n_cand, finished, eos)
    assert gap > 1e-5, "the inputs leave the order to rounding"
    got = nhm.beam_select(dev(xs.reshape(G * K, V)), dev(cum.astype(np.float32)), n_cand,
                          finished=None if finished is None else dev(finished.astype(np.int32)), eos=eos)
    torch.cuda.synchronize()
    gs, gp, gt = (v.cpu().numpy() for v in got)
    assert np.array_equal(gp, p) and np.array_equal(gt, t), (gp, p, gt, t)
    none = p < 0
    assert np.all(gs[none] == -np.inf)
    with np.errstate(invalid="ignore"):
        assert np.all((np.abs(gs - s) <= score_tol(s))[~none] | (gs == s)[~none])


@pytest.mark.parametrize("G,K,V,n,f32", [
    (1, 1, 1, 1, True), (1, 1, 7, 7, False), (1, 1, 7, 16, True), (2, 3, 5, 64, True), (1, 4, 32000, 8, False),
    (3, 5, 50257, 10, True), (2, 32, 2047, 64, True), (2, 32, 2048, 64, False), (5, 2, 2049, 33, True),
    (1, 8, 131072, 16, False), (2, 2, 131073, 1, False), (4, 16, 1000, 64, False), (70, 1, 513, 2, True),
    (1, 32, 20000, 64, True), (1, 3, 1 << 20, 5, False)])
def test_beam_select(nhm, G, K, V, n, f32):
    print(f"select G={G} K={K} V={V} n={n} f32={f32}", flush=True)
    r = np.random.default_rng(G * 1000 + V)
    check_select(nhm, r.standard_normal((G, K, V)) * 3, (-10 * r.random((G, K))).astype(np.float32), n, f32=f32)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("kind", ["constant", "ascending", "descending", "few_values", "one_hot", "huge", "late_peaks"])
def test_beam_select_shapes_of_rows(nhm, kind, f32):
    """Ties, sorted rows (each element beats the ones before it), one dominant logit, large magnitudes."""
    G, K, V, n = 2, 3, 9001, 40
    r = np.random.default_rng(4)
    base = np.arange(V, dtype=np.float64)
    x = {"constant": np.full((G, K, V), 1.5), "ascending": np.broadcast_to(base / 64, (G, K, V)),
         "descending": np.broadcast_to(-base / 64, (G, K, V)), "few_values": r.integers(0, 4, (G, K, V)) * 2.0,
         "one_hot": np.where(base == 4444, 50.0, -50.0) + np.zeros((G, K, V)),
         "huge": r.integers(-3, 4, (G, K, V)) * 1e30,
         "late_peaks": np.where(base >= V - 50, base, 0.0) / 16 + np.zeros((G, K, V))}[kind]
    cum = np.array([[0.0, -1.25, -2.5], [-0.75, -0.5, -3.25]], np.float32)
    check_select(nhm, np.ascontiguousarray(x), cum, n, f32=f32)


def test_beam_select_equal_beams(nhm):
    """Beams with the same row and score: the order is by beam, then token."""
    r = np.random.default_rng(8)
    row = r.standard_normal(5000) * 2
    x = np.broadcast_to(row, (1, 6, 5000)).copy()
    check_select(nhm, x, np.zeros((1, 6), np.float32), 30)


@pytest.mark.parametrize("f32", [True, False])
def test_beam_select_masks(nhm, f32):
    """NaN, infinities, rows with nothing left, unused and finished beams, and too few continuations."""
    r = np.random.default_rng(6)
    G, K, V, n = 3, 4, 3001, 24
    x = r.standard_normal((G, K, V)) * 3
    x[0, 0] = -np.inf                                # nothing left
    x[0, 1, ::2] = np.nan
    x[0, 2, 5:] = -np.inf                            # five left
    x[1] = -np.inf                                   # a group with a few only
    x[1, 3, [7, 2999]] = [1.0, 2.0]
    x[2, 1, [10, 20]] = np.inf                       # share the probability
    x[2, 2] = np.finfo(np.float32).min if f32 else -3.3895313892515355e38   # the type's lowest value: an even row
    cum = (-3 * r.random((G, K))).astype(np.float32)
    cum[0, 3] = -np.inf                              # unused
    cum[2, 3] = np.nan
    check_select(nhm, x, cum, n, f32=f32)
    fin = np.zeros((G, K), np.int32)
    fin[0, 2], fin[1, 0], fin[1, 3], fin[2, 0] = 1, 7, -1, 1
    check_select(nhm, x, cum, n, finished=fin, eos=V - 1, f32=f32)
    check_select(nhm, x, cum, 1, finished=np.ones((G, K), np.int32), eos=0, f32=f32)
    check_select(nhm, np.full((G, K, V), -np.inf), cum, n, f32=f32)


def test_beam_select_strides_and_alignment(nhm):
    """Rows at every alignment: a row stride above the vocabulary and a base off the 16-byte grid."""
    from oracle import bf16_to_f64
    r = np.random.default_rng(12)
    G, K, V, n = 2, 3, 4099, 12
    cum = (-2 * r.random((G, K))).astype(np.float32)
    cumd = torch.from_numpy(cum).cuda()
    for f32 in (True, False):
        for ld, off in [(V, 1), (V + 1, 3), (V + 5, 0), (V + 8, 7)]:
            buf = np.full(off + G * K * ld + 16, 1e4, np.float32)      # the padding would win if it were read
            x = (r.standard_normal((G * K, V)) * 3).astype(np.float32)
            for i in range(G * K):
                buf[off + i * ld:off + i * ld + V] = x[i]
            if f32:
                d, ref_x = torch.from_numpy(buf).cuda(), x.astype(np.float64)
            else:
                b = bits(buf)
                d, ref_x = torch.from_numpy(b.view(np.int16)).cuda(), bf16_to_f64(bits(x))
            s, p, t, gap = so.beam_select(ref_x.reshape(G, K, V), cum, n)
            assert gap > 1e-5
            gs = torch.empty((G, n), device="cuda")
            gp, gt = (torch.empty((G, n), dtype=torch.int32, device="cuda") for _ in range(2))
            need = nhm.beam_select_workspace_bytes(G, K, V, n)
            ws = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
            st = nhm.lib.nhm_beam_select(d.data_ptr() + off * (4 if f32 else 2), nhm.NHM_F32 if f32 else nhm.NHM_BF16, ld, G,
                                         K, V, cumd.data_ptr(), None, 0, n, gs.data_ptr(), gp.data_ptr(), gt.data_ptr(),
                                         ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
            assert st == 0, nhm.lib.nhm_last_error()
            torch.cuda.synchronize()
            assert np.array_equal(gp.cpu().numpy(), p) and np.array_equal(gt.cpu().numpy(), t)
            assert np.all(np.abs(gs.cpu().numpy() - s) <= score_tol(s))
            assert bool((ws[need:] == 0x5A).all())


def test_beam_select_captured(nhm):
    r = np.random.default_rng(2)
    G, K, V, n = 4, 4, 32000, 8
    x = torch.from_numpy((r.standard_normal((G * K, V)) * 3).astype(np.float32)).cuda()
    cum = torch.from_numpy((-r.random((G, K))).astype(np.float32)).cuda()
    out = nhm.beam_select(x, cum, n)
    ws = torch.empty(nhm.beam_select_workspace_bytes(G, K, V, n), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nhm.beam_select(x, cum, n, scores=out[0], parents=out[1], tokens=out[2], ws=ws)
    for i in range(4):
        x.copy_(torch.roll(x, 17 * (i + 1), dims=1))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        eager = nhm.beam_select(x, cum, n)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), i


# ---------------------------------------------------------------- state reorder

SMALL = dict(hidden=256, n_heads=8, head_dim=64, d_state=128, n_groups=2, conv_width=4, rms_eps=1e-5)


def pools(layers, S, f32, seed, g=SMALL):
    r = np.random.default_rng(seed)
    conv_dim = g["n_heads"] * 64 + 2 * g["n_groups"] * 128
    ssm = [r.integers(0, 1 << 15, (S, g["n_heads"], 64, 128)).astype(np.float32 if f32 else np.uint16) for _ in range(layers)]
    conv = [r.integers(0, 1 << 15, (S, 3, conv_dim)).astype(np.uint16) for _ in range(layers)]
    return ssm, conv


@pytest.mark.parametrize("G,K,layers,f32,seed", [(1, 1, 1, True, 0), (2, 4, 3, True, 1), (3, 5, 2, False, 2),
                                                 (1, 32, 1, False, 3), (4, 2, 64, False, 4), (5, 8, 1, True, 5)])
def test_beam_reorder(nhm, G, K, layers, f32, seed):
    from tests.gpu_util import dev, host
    print(f"reorder G={G} K={K} layers={layers} f32={f32}", flush=True)
    r = np.random.default_rng(seed)
    S = G * K + 3
    for case in range(4):
        ssm, conv = pools(layers, S, f32, seed)
        slots = r.permutation(S)[:G * K].reshape(G, K).astype(np.int32)
        parents = r.integers(0, K, (G, K)).astype(np.int32)
        if case == 1:
            parents[:] = K - 1                                      # one parent for all
        if case == 2:
            parents[r.random((G, K)) < 0.4] = -1                    # beams without a parent
            parents[0, -1] = K + 5
        if case == 3:
            slots[0, 0] = -1                                        # absent rows
            slots[-1, -1] = S + 2
        sd, cd = [dev(p) for p in ssm], [dev(p) for p in conv]
        new = nhm.beam_reorder(dev(parents), dev(slots), sd, cd, g=SMALL)
        torch.cuda.synchronize()
        want = so.beam_reorder(parents, slots, ssm + conv)
        assert np.array_equal(new.cpu().numpy(), want)
        for got, ref in zip(sd + cd, ssm + conv):
            assert np.array_equal(host(got), ref), case


def test_beam_reorder_full_geometry_captured(nhm):
    """The mixer's own geometry; a captured call replayed with other parents, slots handed on in turn."""
    from tests.gpu_util import dev, host
    r = np.random.default_rng(7)
    G, K, S = 2, 3, 7
    ssm, conv = pools(2, S, True, 11, g=nhm.GEOMETRY)
    slots = r.permutation(S)[:G * K].reshape(G, K).astype(np.int32)
    sd, cd = [dev(p) for p in ssm], [dev(p) for p in conv]
    cur, new, par = dev(slots), dev(slots.copy()), dev(np.zeros((G, K), np.int32))
    nhm.beam_reorder(dev(np.broadcast_to(np.arange(K, dtype=np.int32), (G, K)).copy()), cur, sd, cd, new_slots=new)
    torch.cuda.synchronize()
    assert torch.equal(new, cur)                                    # every beam goes on from itself
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nhm.beam_reorder(par, cur, sd, cd, new_slots=new)
        cur.copy_(new)
    for i in range(4):
        p = r.integers(0, K, (G, K)).astype(np.int32)
        par.copy_(torch.from_numpy(p))
        graph.replay()
        torch.cuda.synchronize()
        slots = so.beam_reorder(p, slots, ssm + conv)
        assert np.array_equal(cur.cpu().numpy(), slots), i
        for got, ref in zip(sd + cd, ssm + conv):
            assert np.array_equal(host(got), ref), i


# ---------------------------------------------------------------- batch plan

@pytest.mark.parametrize("n,T", [(0, 0), (0, 9), (1, 0), (1, 1), (3, 7), (17, 512), (64, 4096), (1023, 5000), (1024, 5000),
                                 (1025, 300000), (8192, 100001)])
@pytest.mark.parametrize("kind", ["short", "over", "plain"])
def test_batch_plan(nhm, n, T, kind):
    from tests.gpu_util import dev
    r = np.random.default_rng(n + T)
    mean = T / max(n, 1) * (2.0 if kind == "over" else 0.7)
    lengths = r.poisson(mean, n).astype(np.int32)
    lengths[r.random(n) < 0.2] = 0
    if n > 2:
        lengths[2] = -5
    past = np.where(r.random(n) < 0.5, 0, r.integers(-3, 1 << 30, n)).astype(np.int32)
    ad = r.integers(-2, 99, n).astype(np.int32)
    plan = nhm.BatchPlan(n, T)
    for t in (plan.cu_seqlens, plan.has_initial, plan.token_seq, plan.token_pos, plan.token_adapter):
        t.fill_(123456)
    opt = kind != "plain"
    nhm.batch_plan(dev(lengths), plan, past=dev(past) if opt else None, adapters=dev(ad) if opt else None)
    torch.cuda.synchronize()
    want = so.batch_plan(lengths, T, past if opt else None, ad if opt else None)
    for name, ref in want.items():
        assert np.array_equal(getattr(plan, name).cpu().numpy(), ref), name


def test_batch_plan_saturates(nhm):
    """Lengths whose sum passes 2^31, and a call without the per-token outputs."""
    from tests.gpu_util import dev
    lengths = np.full(4000, 2 ** 31 - 1, np.int32)
    plan = nhm.BatchPlan(4000, 1000)
    nhm.batch_plan(dev(lengths), plan)
    torch.cuda.synchronize()
    want = so.batch_plan(lengths, 1000)
    assert np.array_equal(plan.cu_seqlens.cpu().numpy(), want["cu_seqlens"])
    assert np.array_equal(plan.token_seq.cpu().numpy(), want["token_seq"])
    cu, has = (torch.empty(4001, dtype=torch.int32, device="cuda") for _ in range(2))
    ln = dev(lengths)
    st = nhm.lib.nhm_batch_plan(ln.data_ptr(), None, None, 4000, 2 ** 31 - 1, cu.data_ptr(), has.data_ptr(), None, None,
                                None, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert int(cu[1]) == 2 ** 31 - 1 and int(cu[4000]) == 2 ** 31 - 1 and int(has[:4000].sum()) == 0


# ---------------------------------------------------------------- the binding's refusals


def refused(error, f, *a, **kw):
    with pytest.raises(error):
        f(*a, **kw)


def test_binding_refuses_other_tensors(nhm):
    """Wrong shapes, types, orders and devices are errors ahead of any launch, and leave the outputs as they were."""
    x, W, L, ids = lora_device(nhm, lora_inputs(5, 64, 48, 8, 2, seed=1))
    out = torch.full((5, 64), 7, dtype=torch.int16, device="cuda")
    call = nhm.fp8_linear_lora
    refused(TypeError, call, x.cpu(), W, L, ids)
    refused(TypeError, call, x, W, L, ids.long(), out=out)
    refused(TypeError, call, x, W, L, ids.cpu(), out=out)
    refused(ValueError, call, x, W, L, ids[:4], out=out)
    refused(ValueError, call, x[:, :32].contiguous(), W, L, ids, out=out)
    refused(ValueError, call, x, W, L, ids, out=out[:, :32])
    refused(ValueError, call, x, W, L, ids, out=out.t().contiguous().t())
    refused(TypeError, call, x, W, L, ids, out=out, out_type=nhm.NHM_F32)
    refused(nhm.NhmError, call, x, W, L, ids, out=out, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    refused(ValueError, nhm.Lora, L.a, L.b[:1], None)
    refused(ValueError, nhm.Lora, L.a, L.b, torch.ones(3, device="cuda"))
    refused(ValueError, call, x, W, nhm.Lora(L.a, L.b[:, :32].contiguous()), ids)

    logits, cum = torch.zeros((6, 100), device="cuda"), torch.zeros((2, 3), device="cuda")
    refused(ValueError, nhm.beam_select, logits, cum[0], 4)
    refused(ValueError, nhm.beam_select, logits[:5], cum, 4)
    refused(TypeError, nhm.beam_select, logits.double(), cum, 4)
    refused(ValueError, nhm.beam_select, logits, cum, 4, scores=torch.zeros((2, 3), device="cuda"))
    refused(nhm.NhmError, nhm.beam_select, logits, cum, 65)
    refused(nhm.NhmError, nhm.beam_select, logits, cum, 4, finished=torch.zeros((2, 3), dtype=torch.int32, device="cuda"), eos=100)

    g = dict(hidden=256, n_heads=8, head_dim=64, d_state=128, n_groups=2, conv_width=4, rms_eps=1e-5)
    ssm = torch.zeros((6, 8, 64, 128), device="cuda")
    conv = torch.zeros((6, 3, 8 * 64 + 2 * 2 * 128), dtype=torch.int16, device="cuda")
    par = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    slots = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    refused(ValueError, nhm.beam_reorder, par, slots, [ssm], [conv[:5]], g=g)
    refused(ValueError, nhm.beam_reorder, par, slots, [ssm, ssm[:5]], [conv, conv[:5]], g=g)
    refused(ValueError, nhm.beam_reorder, par, slots, [ssm], [], g=g)
    refused(TypeError, nhm.beam_reorder, par, slots, [ssm, ssm.to(torch.bfloat16)], [conv, conv], g=g)
    refused(nhm.NhmError, nhm.beam_reorder, par, slots, [ssm], [conv], new_slots=slots, g=g)

    n = torch.ones(4, dtype=torch.int32, device="cuda")
    refused(ValueError, nhm.batch_plan, n, nhm.BatchPlan(5, 8))
    refused(TypeError, nhm.batch_plan, n.long(), nhm.BatchPlan(4, 8))
    torch.cuda.synchronize()
    assert bool((out == 7).all()) and bool((ssm == 0).all())
