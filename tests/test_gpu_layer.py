"""The layer operators (include/nhm_layer.h) against plain 64-bit forms: MXFP4 quantisation and projections, the causal
convolution and the selective scan for prompts and single tokens, and the scoring of tokens."""
import numpy as np
import pytest

from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def nhm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_w8a8_linear_amd as m
    return m


def bf16(a):
    """numpy float -> a bfloat16 tensor on the GPU."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16).cuda()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def u8(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.uint8)).cuda()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def wider(t, left, right):
    """The same rows as a slice of wider ones, whose other columns are NaN."""
    w = torch.full((t.shape[0], left + t.shape[1] + right), float("nan"), dtype=t.dtype, device=t.device)
    w[:, left:left + t.shape[1]] = t
    return w[:, left:left + t.shape[1]]


def within(got, ref, tol, what):
    got, ref = np.asarray(got), np.asarray(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    ok = (np.abs(got - ref) <= tol) | (got == ref) | np.isnan(ref)
    if not ok.all():
        at = np.unravel_index(np.argmax(np.where(ok, 0, np.abs(got - ref))), got.shape)
        raise AssertionError(f"{what}: {(~ok).sum()} of {ok.size} outside, at {at}: {got[at]} for {ref[at]}, {np.broadcast_to(tol, ref.shape)[at]} allowed")


# ---------------------------------------------------------------- MXFP4

def unpack(b):
    b = b.cpu().numpy()
    return np.stack([b & 15, b >> 4], axis=2).reshape(b.shape[0], -1)


def check_quant(nhm, x, what):
    codes, scales = nhm.mxfp4_quantize(x)
    want_c, want_s = lo.mxfp4_quantize(f64(x))
    assert np.array_equal(scales.cpu().numpy(), want_s), what
    assert np.array_equal(unpack(codes), want_c), what
    got = f64(nhm.mxfp4_dequantize(codes, scales).view(torch.bfloat16))
    within(got, lo.mxfp4_values(want_c, want_s), 0.0, what)


def test_mxfp4_every_bf16_pattern(nhm):
    """All 65,536 bf16 patterns, each in a block of its neighbours and in blocks whose largest value is 1 to 2^9 times its own;
    infinities, NaN and zeros among them."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    check_quant(nhm, bits.view(-1, 256).cuda(), "patterns in order")
    finite = torch.where(torch.isfinite(bits), bits, torch.zeros_like(bits))
    x = finite.view(-1, 1).repeat(1, 32)
    for j in range(10):
        y = x.clone()
        y[:, 1:] = torch.where((x[:, 1:].float() * 2.0 ** j).isfinite(), x[:, 1:].float() * 2.0 ** j, x[:, 1:].float()).to(torch.bfloat16) * 0.4375
        y[:, 0] = (x[:, 0].float() * 2.0 ** j).to(torch.bfloat16)
        y[:, 31] = x[:, 31]
        check_quant(nhm, y.cuda(), f"beside 2^{j} times the value")


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (61, 2688), (17, 4128), (1000, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_mxfp4_quantize(nhm, rows, cols, dtype):
    r = np.random.default_rng(rows * cols)
    x = r.normal(size=(rows, cols)) * np.exp2(r.integers(-130, 120, (rows, 1)).astype(float))
    x[r.random(x.shape) < 0.05] = 0.0
    x[-1, :32] = 0.0
    if rows > 2:
        x[1, 5], x[2, 40 % cols] = np.nan, -np.inf
    x = x.astype(np.float32)
    t = bf16(x) if dtype == "bf16" else torch.from_numpy(x).cuda()
    check_quant(nhm, t, "contiguous")
    check_quant(nhm, wider(t, 8, 16), "rows of wider ones")


def test_mxfp4_dequantize_every_code(nhm):
    codes = np.tile(np.arange(32) % 16, (256, 1)).astype(np.uint8)
    got = f64(nhm.mxfp4_dequantize(u8(lo.mxfp4_pack(codes)), u8(np.arange(256)[:, None])).view(torch.bfloat16))
    want = lo.mxfp4_values(codes, np.arange(256)[:, None].astype(np.uint8))
    want = np.where(np.abs(want) >= 2.0 ** 128, np.sign(want) * np.inf, want)
    within(got, want, 0.0, "values")
    assert np.array_equal(np.signbit(got[:255]), np.signbit(want[:255]))


def linear_case(nhm, m, n, k, codes, f32, seed, pad=0, lo_scale=110, hi_scale=135):
    r = np.random.default_rng(seed)
    w, ws = r.integers(0, 16, (n, k)).astype(np.uint8), r.integers(lo_scale, hi_scale, (n, k // 32)).astype(np.uint8)
    weight = nhm.Mxfp4Weight(u8(lo.mxfp4_pack(w)), u8(ws))
    wv = lo.mxfp4_values(w, ws)
    if codes:
        a, s = r.integers(0, 16, (m, k)).astype(np.uint8), r.integers(lo_scale, hi_scale, (m, k // 32)).astype(np.uint8)
        x, xs = u8(lo.mxfp4_pack(a)), u8(s)
        av = lo.mxfp4_values(a, s)
        if pad:
            big = torch.full((m, k // 2 + 2 * pad), 0xff, dtype=torch.uint8, device="cuda")
            big[:, pad:pad + k // 2] = x
            x = big[:, pad:pad + k // 2]
    else:
        x, xs = bf16(r.normal(size=(m, k)) * np.exp2(r.integers(-8, 8, (m, 1)).astype(float))), None
        av = lo.mxfp4_values(*lo.mxfp4_quantize(f64(x)))
        if pad:
            x = wider(x, pad, pad)
    dt = torch.float32 if f32 else torch.bfloat16
    out = torch.full((m + 2, n + 2 * pad + 3 * (pad > 0)), 7.0, dtype=dt, device="cuda")
    view = out[1:m + 1, pad:pad + n]
    nhm.mxfp4_linear(x, weight, a_scale=xs, out=view)
    ref, tol = lo.mxfp4_linear(av, wv)
    within(f64(view), ref, tol * (1 + 2.0 ** -8) + lo.half_step(ref, not f32), f"m {m} n {n} k {k}")
    rest = out.clone()
    rest[1:m + 1, pad:pad + n] = 7.0
    assert bool((rest == 7.0).all()), "stores outside the output"
    return x, weight, xs, view


SHAPES = [(1, 16, 32), (1, 10304, 2688), (2, 33, 64), (5, 130, 96), (8, 2688, 4096), (13, 100, 544), (16, 257, 2688), (17, 64, 128),
          (31, 130, 160), (33, 515, 288), (61, 2688, 4096), (64, 96, 2720), (65, 130, 256), (100, 257, 416), (128, 128, 128),
          (129, 300, 1056), (200, 1000, 512), (477, 2688, 4096), (513, 770, 96), (640, 1030, 2688), (1000, 4096, 320),
          (1025, 515, 800), (2049, 2690, 1024)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_mxfp4_linear(nhm, m, n, k):
    """Either input type with either output type, rows of wider ones and odd offsets among them."""
    print(m, n, k, flush=True)
    linear_case(nhm, m, n, k, codes=True, f32=True, seed=1)
    linear_case(nhm, m, n, k, codes=False, f32=False, seed=2)
    linear_case(nhm, m, n, k, codes=True, f32=False, seed=3, pad=16)
    if m < 600:
        linear_case(nhm, m, n, k, codes=False, f32=True, seed=4, pad=8)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_mxfp4_linear_wide_scales(nhm, m):
    """Scales from 2^-60 to 2^60 within a row: what is small beside the rest is summed all the same."""
    linear_case(nhm, m, 70, 1056, codes=True, f32=True, seed=5, lo_scale=67, hi_scale=187)


@pytest.mark.parametrize("m", [3, 40, 300])
def test_mxfp4_linear_nan_scales(nhm, m):
    """A NaN scale makes its own row (of the activations) or feature NaN and no other; so does a NaN or infinite bf16 input."""
    r = np.random.default_rng(6)
    n, k = 150, 352
    w, ws = r.integers(0, 16, (n, k)).astype(np.uint8), r.integers(120, 130, (n, k // 32)).astype(np.uint8)
    ws[100, 10] = 255
    w[100, 320:] = 0
    weight = nhm.Mxfp4Weight(u8(lo.mxfp4_pack(w)), u8(ws))
    a, s = r.integers(0, 16, (m, k)).astype(np.uint8), r.integers(120, 130, (m, k // 32)).astype(np.uint8)
    s[1, 3] = 255
    got = f64(nhm.mxfp4_linear(u8(lo.mxfp4_pack(a)), weight, a_scale=u8(s), out_type=nhm.NHM_F32))
    ref, tol = lo.mxfp4_linear(lo.mxfp4_values(a, s), lo.mxfp4_values(w, ws))
    within(got, ref, tol, "NaN scales")
    x = r.normal(size=(m, k))
    x[0, 351], x[2, 0] = np.inf, np.nan
    got = f64(nhm.mxfp4_linear(bf16(x), weight, out_type=nhm.NHM_F32))
    assert np.isnan(got[[0, 2]]).all() and np.isnan(got[:, 100]).all()
    assert np.isfinite(np.delete(np.delete(got, 100, axis=1), [0, 2], axis=0)).all()


def test_mxfp4_linear_rows_alone(nhm):
    """Twice the same call gives the same bits, and so do other values in the other rows; no rows are a valid call."""
    x, weight, xs, out = linear_case(nhm, 300, 200, 512, codes=True, f32=True, seed=7)
    assert torch.equal(nhm.mxfp4_linear(x, weight, a_scale=xs, out_type=nhm.NHM_F32), out)
    y, ys = x.clone(), xs.clone()
    y[7], ys[7] = 0x77, 200
    other = nhm.mxfp4_linear(y, weight, a_scale=ys, out_type=nhm.NHM_F32)
    keep = torch.arange(300, device="cuda") != 7
    assert torch.equal(other[keep], out[keep])
    assert nhm.mxfp4_linear(x[:0], weight, a_scale=xs[:0]).shape == (0, 200)


@pytest.mark.parametrize("k", [32, 288, 4096, 15360, 15616, 40960])
def test_mxfp4_linear_quantises_alike(nhm, k):
    """bf16 rows and their codes give the same bits, whether or not the quantisation is a launch of its own (up to four rows
    whose codes fit LDS are quantised beside the product); infinities and NaN, and rows of a wider tensor, among them."""
    r = np.random.default_rng(k)
    w = nhm.Mxfp4Weight(u8(r.integers(0, 256, (50, k // 2))), u8(r.integers(118, 130, (50, k // 32))))
    for m in (1, 2, 3, 4, 5, 70):
        x = r.normal(size=(m, k)) * np.exp2(r.integers(-140, 100, (m, 1)).astype(float))
        x[m - 1, k - 1] = np.nan if m % 2 else np.inf
        x = wider(bf16(x), 8, 16)
        codes, scales = nhm.mxfp4_quantize(x)
        for t in (nhm.NHM_F32, nhm.NHM_BF16):
            want, got = nhm.mxfp4_linear(codes, w, a_scale=scales, out_type=t), nhm.mxfp4_linear(x, w, out_type=t)
            bits = torch.int32 if t == nhm.NHM_F32 else torch.int16
            assert torch.equal(got.view(bits), want.view(bits)), (m, t)
            assert bool(torch.isnan(got.view(torch.float32 if t == nhm.NHM_F32 else torch.bfloat16)[m - 1]).all())


@pytest.mark.parametrize("m", [3, 20, 70])
def test_mxfp4_linear_rows_far_apart(nhm, m):
    """Rows of codes so far apart that the operand fills its 2 GiB."""
    r = np.random.default_rng(14)
    n, k = 130, 544
    ld = ((1 << 31) // m - 64) // 16 * 16
    x = torch.empty(m * ld, dtype=torch.uint8, device="cuda").as_strided((m, k // 2), (ld, 1))
    x.copy_(u8(r.integers(0, 256, (m, k // 2))))
    s = u8(r.integers(118, 130, (m, k // 32)))
    w = nhm.Mxfp4Weight(u8(r.integers(0, 256, (n, k // 2))), u8(r.integers(118, 130, (n, k // 32))))
    assert torch.equal(nhm.mxfp4_linear(x, w, a_scale=s), nhm.mxfp4_linear(x.contiguous(), w, a_scale=s))


def test_mxfp4_linear_packed_scales(nhm):
    """A weight without packed scale codes gives the same bits; with them, new scale codes count from pack() on."""
    import ctypes as C
    r = np.random.default_rng(8)
    m, n, k = 100, 70, 416
    weight = nhm.Mxfp4Weight(u8(r.integers(0, 256, (n, k // 2))), u8(r.integers(118, 130, (n, k // 32))))
    x = bf16(r.normal(size=(m, k)))
    codes, scales = nhm.mxfp4_quantize(x)

    def bare(a, t, s):
        wt = nhm._Mxfp4Weight(weight.w.data_ptr(), weight.scale.data_ptr(), n, k, None)
        size = nhm.mxfp4_linear_workspace_bytes(m, n, k, t)
        ws, out = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.empty(m, n, dtype=torch.float32, device="cuda")
        st = torch.cuda.current_stream().cuda_stream
        assert nhm.lib.nhm_mxfp4_linear(a.data_ptr(), t, s, m, a.shape[1], C.byref(wt), out.data_ptr(), nhm.NHM_F32, n, ws.data_ptr(), size, st) == 0
        return out

    for _ in range(2):
        want = nhm.mxfp4_linear(x, weight, out_type=nhm.NHM_F32)
        assert torch.equal(bare(x, nhm.NHM_BF16, None), want) and torch.equal(bare(codes, nhm.NHM_MXFP4, scales.data_ptr()), want)
        weight.scale.copy_(u8(r.integers(118, 130, (n, k // 32))))
        weight.pack()


# ---------------------------------------------------------------- batches

BATCHES = [[1], [2, 3], [0], [5, 130, 1, 0, 260, 128], [0, 0, 7, 0], [8, 8, 8], [1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1], [64, 16, 63, 65],
           [517], [3, 0, 2, 1, 9, 2, 2, 0]]


def batch(lengths, tail, r, slots_more=3):
    """(cu, slots, has_initial, tokens, pool rows): distinct slots, every third sequence (from the second) without one."""
    n = len(lengths)
    slots = r.permutation(n + slots_more)[:n]
    if n > 2:
        slots[2::5] = [-1 - i if i % 2 else n + slots_more + i for i in range(len(slots[2::5]))]
    return np.concatenate([[0], np.cumsum(lengths)]), slots, (r.random(n) < 0.6).astype(int), sum(lengths) + tail, n + slots_more


# ---------------------------------------------------------------- convolution

@pytest.mark.parametrize("lengths", BATCHES, ids=str)
@pytest.mark.parametrize("width,dim,silu,bias,strided", [(4, 64, True, True, False), (4, 520, True, True, True), (3, 1032, False, True, True),
                                                         (2, 8, True, False, False)])
def test_conv_prefill(nhm, lengths, width, dim, silu, bias, strided):
    r = np.random.default_rng(len(lengths) + dim)
    cu, slots, init, tokens, S = batch(lengths, 5 if strided else 0, r)
    x, w, b = bf16(r.normal(size=(tokens, dim))), bf16(r.normal(size=(dim, width)) * 0.5), bf16(r.normal(size=dim)) if bias else None
    pool = bf16(r.normal(size=(S, width - 1, dim)))
    if sum(lengths) < tokens:
        x[sum(lengths):] = float("nan")          # rows behind the last sequence reach nothing
    before = f64(pool)
    out = torch.full((tokens, dim + 24), 3.0, dtype=torch.bfloat16, device="cuda")[:, 8:8 + dim] if strided else \
        torch.full((tokens, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    nhm.causal_conv_prefill(wider(x, 16, 8) if strided else x, w, b, i32(cu), i32(slots), i32(init), pool, out=out, silu=silu)
    want_pool, X, W, B = before.copy(), f64(x), f64(w), f64(b) if bias else np.zeros(dim)
    got = f64(out)
    for i, (s, h) in enumerate(zip(slots, init)):
        held = 0 <= s < S
        win = before[s] if held and h else np.zeros((width - 1, dim))
        rows = np.concatenate([win, X[cu[i]:cu[i + 1]]])
        ref, tol = lo.causal_conv(rows, W, B, silu)
        within(got[cu[i]:cu[i + 1]], ref, tol * (1 + 2.0 ** -8) + lo.half_step(ref, True), f"sequence {i}")
        if held:
            want_pool[s] = rows[len(rows) - (width - 1):]
    assert np.array_equal(f64(pool), want_pool)
    assert not got[cu[-1]:].any()


@pytest.mark.parametrize("width,dim,batch_size,strided", [(4, 4096, 8, False), (4, 520, 33, True), (3, 8, 1, False), (2, 72, 70, True)])
def test_conv_decode(nhm, width, dim, batch_size, strided):
    r = np.random.default_rng(dim)
    S = batch_size + 2
    slots = r.permutation(S)[:batch_size]
    slots[3::7] = -1
    slots[5::11] = S
    x, w, b = bf16(r.normal(size=(batch_size, dim))), bf16(r.normal(size=(dim, width))), bf16(r.normal(size=dim))
    pool = bf16(r.normal(size=(S, width - 1, dim)))
    before = f64(pool)
    out = nhm.causal_conv_decode(wider(x, 8, 8) if strided else x, w, b, i32(slots), pool).view(torch.bfloat16)
    want, got = before.copy(), f64(out)
    for i, s in enumerate(slots):
        if not 0 <= s < S:
            assert not got[i].any()
            continue
        rows = np.concatenate([before[s], f64(x[i:i + 1])])
        ref, tol = lo.causal_conv(rows, f64(w), f64(b), True)
        within(got[i:i + 1], ref, tol * (1 + 2.0 ** -8) + lo.half_step(ref, True), f"row {i}")
        want[s] = rows[1:]
    assert np.array_equal(f64(pool), want)


# ---------------------------------------------------------------- scan

class Layer:
    def __init__(self, nhm, r, dim, n, D=True, bias=True):
        self.A_log = np.log(np.arange(1, n + 1) * np.exp(0.3 * r.normal(size=(dim, n)))).astype(np.float32)
        self.D = r.normal(size=dim).astype(np.float32) if D else None
        d = np.exp(r.uniform(np.log(1e-3), np.log(1e-1), dim))
        self.bias = np.log(np.expm1(d)).astype(np.float32) if bias else None
        up = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
        self.params = nhm.ScanParams(up(self.A_log), up(self.D), up(self.bias))

    def ref(self, u, dt, B, C, h, z):
        dim = u.shape[1]
        zero = np.zeros(dim)
        return lo.selective_scan(u, dt, B, C, self.A_log.astype(float), zero if self.D is None else self.D.astype(float),
                                 zero if self.bias is None else self.bias.astype(float), h, z)


def scan_inputs(r, t, dim, n, z):
    proj = bf16(r.normal(size=(t, 2 * n + 5)))                # B and C of odd offsets in one projection's rows
    return (bf16(r.normal(size=(t, dim))), bf16(r.normal(size=(t, dim)) * 1.5), proj[:, 5:5 + n], proj[:, 5 + n:],
            bf16(r.normal(size=(t, dim)) * 2) if z else None)


def check_state(got, ref, err, bf):
    within(got, ref, err + (lo.half_step(ref, True) + err * 2.0 ** -8 if bf else 0), "state")


@pytest.mark.parametrize("lengths", BATCHES, ids=str)
@pytest.mark.parametrize("dim,n,bf,z,strided", [(64, 16, False, True, False), (88, 16, True, True, True), (8, 4, False, False, True),
                                                (40, 32, False, True, False), (24, 64, True, False, False), (136, 12, False, True, True),
                                                (72, 44, False, True, False)])
def test_scan_prefill(nhm, lengths, dim, n, bf, z, strided):
    r = np.random.default_rng(len(lengths) * 100 + dim)
    cu, slots, init, tokens, S = batch(lengths, 4 if strided else 0, r)
    lay = Layer(nhm, r, dim, n, D=dim != 40, bias=dim != 24)
    u, dt, B, C, zt = scan_inputs(r, tokens, dim, n, z)
    for t in (u, dt, B, C) + ((zt,) if z else ()):
        t[sum(lengths):] = float("nan")
    pool = bf16(r.normal(size=(S, dim, n))) if bf else torch.from_numpy(r.normal(size=(S, dim, n)).astype(np.float32)).cuda()
    before = f64(pool)
    wide = (lambda t: None if t is None else wider(t, 3, 2)) if strided else (lambda t: t)
    out = wide(torch.full((tokens, dim), 3.0, dtype=torch.bfloat16, device="cuda"))
    nhm.selective_scan_prefill(lay.params, wide(u), wide(dt), B, C, i32(cu), i32(slots), i32(init), pool, z=wide(zt), out=out)
    after, got = f64(pool), f64(out)
    U, DT, BB, CC, Z = f64(u), f64(dt), f64(B), f64(C), f64(zt) if z else None
    touched = np.zeros(S, bool)
    for i, (s, h0) in enumerate(zip(slots, init)):
        held, e = 0 <= s < S, slice(cu[i], cu[i + 1])
        h = before[s] if held and h0 else np.zeros((dim, n))
        ref, tol, h, err = lay.ref(U[e], DT[e], BB[e], CC[e], h, Z[e] if z else None)
        within(got[e], ref, tol * (1 + 2.0 ** -8) + lo.half_step(ref, True), f"sequence {i}")
        if held:
            touched[s] = True
            check_state(after[s], h, err, bf)
    assert np.array_equal(after[~touched], before[~touched])
    assert not got[cu[-1]:].any()


@pytest.mark.parametrize("dim,n,bf,lengths", [(64, 16, False, [3000]), (8, 16, True, [5000, 0, 300]), (64, 32, False, [1500, 700]),
                                              (24, 64, False, [1100]), (512, 16, False, [900, 100, 1300]), (200, 8, True, [2049])])
def test_scan_prefill_long(nhm, dim, n, bf, lengths):
    """Few long sequences: cut into chunks that run side by side. A channel that hardly forgets keeps its state from end to end."""
    r = np.random.default_rng(dim + n)
    cu, slots, init, tokens, S = batch(lengths, 0, r)
    slots = np.where((slots < 0) | (slots >= S), [i for i in range(S) if i not in slots][0], slots)
    lay = Layer(nhm, r, dim, n)
    lay.A_log[0] = np.log(1e-4)
    lay.params.A_log[0] = float(np.log(np.float32(1e-4)))
    u, dt, B, C, z = scan_inputs(r, tokens, dim, n, True)
    pool = bf16(r.normal(size=(S, dim, n))) if bf else torch.from_numpy(r.normal(size=(S, dim, n)).astype(np.float32)).cuda()
    before = f64(pool)
    out = nhm.selective_scan_prefill(lay.params, u, dt, B, C, i32(cu), i32(slots), i32(init), pool, z=z).view(torch.bfloat16)
    after, got = f64(pool), f64(out)
    U, DT, BB, CC, Z = f64(u), f64(dt), f64(B), f64(C), f64(z)
    lay.A_log[0] = f64(lay.params.A_log[0])
    for i, (s, h0) in enumerate(zip(slots, init)):
        e = slice(cu[i], cu[i + 1])
        ref, tol, h, err = lay.ref(U[e], DT[e], BB[e], CC[e], before[s] if h0 else np.zeros((dim, n)), Z[e])
        within(got[e], ref, tol * (1 + 2.0 ** -8) + lo.half_step(ref, True), f"sequence {i}")
        check_state(after[s], h, err, bf)


@pytest.mark.parametrize("dim,n,bf,z,batch_size", [(4096, 16, False, True, 8), (72, 16, True, True, 33), (8, 4, False, False, 1), (40, 32, False, True, 5),
                                                   (24, 64, True, True, 6), (136, 12, True, False, 9), (64, 8, False, True, 3)])
def test_scan_decode(nhm, dim, n, bf, z, batch_size):
    r = np.random.default_rng(dim * n)
    S = batch_size + 2
    slots = r.permutation(S)[:batch_size]
    slots[3::7] = -1
    slots[4::9] = S
    lay = Layer(nhm, r, dim, n)
    u, dt, B, C, zt = scan_inputs(r, batch_size, dim, n, z)
    pool = bf16(r.normal(size=(S, dim, n))) if bf else torch.from_numpy(r.normal(size=(S, dim, n)).astype(np.float32)).cuda()
    before = f64(pool)
    out = nhm.selective_scan_decode(lay.params, wider(u, 1, 2), dt, B, C, i32(slots), pool, z=zt).view(torch.bfloat16)
    after, got = f64(pool), f64(out)
    touched = np.zeros(S, bool)
    for i, s in enumerate(slots):
        if not 0 <= s < S:
            assert not got[i].any()
            continue
        touched[s], e = True, slice(i, i + 1)
        ref, tol, h, err = lay.ref(f64(u)[e], f64(dt)[e], f64(B)[e], f64(C)[e], before[s], f64(zt)[e] if z else None)
        within(got[e], ref, tol * (1 + 2.0 ** -8) + lo.half_step(ref, True), f"row {i}")
        check_state(after[s], h, err, bf)
    assert np.array_equal(after[~touched], before[~touched])


def test_scan_extremes(nhm):
    """Steps of 0 and of 30 (softplus at both ends), A from 1e-6 to 1e4: states kept and states forgotten at once; a NaN input
    stays in its own sequence and channel."""
    r = np.random.default_rng(9)
    dim, n, lengths = 16, 16, [40, 40]
    lay = Layer(nhm, r, dim, n, bias=False)
    a = np.log(np.exp(r.uniform(np.log(1e-6), np.log(1e4), (dim, n)))).astype(np.float32)
    lay.A_log[:] = a
    lay.params.A_log.copy_(torch.from_numpy(a))
    u, dt, B, C, z = scan_inputs(r, 80, dim, n, True)
    dt[:, :4] = -100.0
    dt[:, 4:8] = 30.0
    dt[::3, 8:12] = 25.0
    u[50, 3], u[45, 9] = float("nan"), float("inf")
    pool = torch.zeros(2, dim, n, device="cuda")
    args = (i32([0, 40, 80]), i32([0, 1]), i32([0, 0]), pool)
    got = f64(nhm.selective_scan_prefill(lay.params, u, dt, B, C, *args, z=z).view(torch.bfloat16))
    clean = u.clone()
    clean[50, 3] = clean[45, 9] = 0.0
    bad = np.zeros((80, dim), bool)
    bad[50:, 3], bad[45:, 9] = True, True
    for e in (slice(0, 40), slice(40, 80)):
        ref, tol, _, _ = lay.ref(f64(clean)[e], f64(dt)[e], f64(B)[e], f64(C)[e], np.zeros((dim, n)), f64(z)[e])
        keep = ~bad[e]
        within(np.where(keep, got[e], 0), np.where(keep, ref, 0), tol * (1 + 2.0 ** -8) + lo.half_step(ref, True), "finite channels")
    assert np.isnan(got[50:, 3]).all() and not np.isfinite(got[45:, 9]).any()


def test_scan_infinite_decay(nhm):
    """A = -inf (A_log past 88.7) forgets a state within a step and leaves it alone where there is none: past a sequence's end,
    whether it ends inside a block of tokens or its last chunk, and as a single token."""
    r = np.random.default_rng(13)
    dim, n = 16, 16
    for lengths in ([5, 40], [1500]):
        lay = Layer(nhm, r, dim, n)
        lay.params.A_log[:, 3], lay.params.A_log[2] = 100.0, float("inf")
        t, S = sum(lengths), len(lengths)
        u, dt, B, C, z = scan_inputs(r, t, dim, n, True)
        pool = torch.from_numpy(r.normal(size=(S, dim, n)).astype(np.float32)).cuda()
        cu = np.concatenate([[0], np.cumsum(lengths)])
        out = nhm.selective_scan_prefill(lay.params, u, dt, B, C, i32(cu), i32(np.arange(S)), i32(np.ones(S)), pool, z=z)
        last = cu[1:] - 1
        gone = f64(lay.params.A_log) > 88.7
        delta = lo.softplus(f64(dt)[last] + f64(lay.params.dt_bias))
        want = (delta * f64(u)[last])[:, :, None] * f64(B)[last][:, None, :]
        assert np.isfinite(f64(out.view(torch.bfloat16))).all() and np.isfinite(f64(pool)).all()
        within(f64(pool)[:, gone], want[:, gone], np.abs(want[:, gone]) * 20 * lo.U, "states forgotten")   # softplus 16 U and two products
        one = nhm.selective_scan_decode(lay.params, u[:S], dt[:S], B[:S], C[:S], i32(np.arange(S)), pool, z=z[:S])
        want = (lo.softplus(f64(dt)[:S] + f64(lay.params.dt_bias)) * f64(u)[:S])[:, :, None] * f64(B)[:S][:, None, :]
        assert np.isfinite(f64(one.view(torch.bfloat16))).all()
        within(f64(pool)[:, gone], want[:, gone], np.abs(want[:, gone]) * 20 * lo.U, "states forgotten in a step")


@pytest.mark.parametrize("n", [4, 8, 16, 20, 64])
def test_scan_values_that_are_not_finite(nhm, n):
    """Infinities and NaN stay in their channel and sequence, also beside the lanes of no state; the others' bits stay."""
    r = np.random.default_rng(n)
    dim, t = 40, 150
    lay = Layer(nhm, r, dim, n)
    u, dt, B, C, z = scan_inputs(r, t, dim, n, True)
    where = (i32([0, 100, t]), i32([0, 1]), i32([0, 0]))
    run = lambda u, dt, p: f64(nhm.selective_scan_prefill(lay.params, u, dt, B, C, *where, p, z=z).view(torch.bfloat16))  # noqa: E731
    pools = torch.zeros(2, dim, n, device="cuda"), torch.zeros(2, dim, n, device="cuda")
    clean = run(u, dt, pools[0])
    bu, bdt = u.clone(), dt.clone()
    bu[20, 5], bu[90, 9], bdt[33, 13], bdt[110, 17] = float("inf"), float("nan"), float("nan"), float("inf")
    got = run(bu, bdt, pools[1])
    bad = np.zeros((t, dim), bool)
    bad[20:100, 5] = bad[90:100, 9] = bad[33:100, 13] = bad[110:, 17] = True
    assert np.array_equal(got[~bad], clean[~bad]) and not np.isfinite(got[bad]).any()
    kept = np.ones((2, dim), bool)
    kept[0, [5, 9, 13]] = kept[1, 17] = False
    assert np.array_equal(f64(pools[1])[kept], f64(pools[0])[kept])


def test_decode_is_a_prefill_of_one(nhm):
    """Prompts, then tokens one by one, against the whole as one prompt: the same recurrence, within its roundings."""
    r = np.random.default_rng(10)
    dim, n, t = 64, 16, 12
    lay = Layer(nhm, r, dim, n)
    u, dt, B, C, z = scan_inputs(r, t, dim, n, True)
    w, b = bf16(r.normal(size=(dim, 4))), bf16(r.normal(size=dim))
    whole, parts = torch.zeros(2, dim, n, device="cuda"), torch.zeros(2, dim, n, device="cuda")
    cw, cp = torch.zeros(2, 3, dim, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 3, dim, dtype=torch.bfloat16, device="cuda")
    one = i32([1])
    full = nhm.selective_scan_prefill(lay.params, u, dt, B, C, i32([0, t]), one, i32([0]), whole, z=z)
    conv = nhm.causal_conv_prefill(u, w, b, i32([0, t]), one, i32([0]), cw)
    got = [nhm.selective_scan_prefill(lay.params, u[:5], dt[:5], B[:5], C[:5], i32([0, 5]), one, i32([0]), parts, z=z[:5])]
    cgot = [nhm.causal_conv_prefill(u[:5], w, b, i32([0, 5]), one, i32([0]), cp)]
    for i in range(5, t):
        e = slice(i, i + 1)
        got.append(nhm.selective_scan_decode(lay.params, u[e], dt[e], B[e], C[e], one, parts, z=z[e]))
        cgot.append(nhm.causal_conv_decode(u[e], w, b, one, cp))
    assert torch.equal(conv, torch.cat(cgot)) and torch.equal(cw, cp)
    ref, tol, h, err = lay.ref(f64(u), f64(dt), f64(B), f64(C), np.zeros((dim, n)), f64(z))
    for o in (full, torch.cat(got)):
        within(f64(o.view(torch.bfloat16)), ref, tol * (1 + 2.0 ** -8) + lo.half_step(ref, True), "outputs")
    check_state(f64(parts[1]), h, err, False)
    assert not parts[0].any()


# ---------------------------------------------------------------- scoring of tokens

def check_scores(nhm, x, tokens, n_top, logits=None):
    lp, rank, ent, tl, tt = nhm.token_logprobs(x if logits is None else logits, i32(tokens), n_top=n_top)
    X = f64(x)
    for i in range(X.shape[0]):
        w_lp, w_rank, w_ent, w_tl, w_tt = lo.token_logprobs(X[i], tokens[i], n_top)
        within(f64(lp)[i], w_lp, lo.logprob_tolerance(w_lp), f"row {i}: log probability")
        assert int(rank[i]) == w_rank, f"row {i}: rank {int(rank[i])} for {w_rank}"
        within(f64(ent)[i], w_ent, 2 * lo.logprob_tolerance(w_ent), f"row {i}: entropy")
        assert tt[i].tolist() == w_tt.tolist(), f"row {i}: alternatives"
        within(f64(tl)[i], w_tl, lo.logprob_tolerance(w_tl), f"row {i}: alternatives' log probabilities")


@pytest.mark.parametrize("rows,vocab,n_top", [(1, 1, 1), (2, 7, 10), (3, 1000, 0), (1, 131072, 20), (5, 50257, 64), (40, 2049, 5), (300, 333, 3),
                                              (17, 32000, 1), (9, 4096, 33)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs(nhm, rows, vocab, n_top, dtype):
    r = np.random.default_rng(vocab + n_top)
    x = r.normal(size=(rows, vocab)) * r.choice([0.5, 3.0, 30.0], (rows, 1))
    x = bf16(x) if dtype == "bf16" else torch.from_numpy(x.astype(np.float32)).cuda()
    tokens = r.integers(0, vocab, rows)
    tokens[::2] = x.argmax(dim=1).cpu().numpy()[::2]
    check_scores(nhm, x, tokens, n_top)
    if vocab > 100:
        check_scores(nhm, x, tokens, n_top, wider(x, 3, 5))       # rows of odd offsets


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs_special_values(nhm, dtype):
    """Rows of equal logits, of few levels, masked ones, NaN, infinities, one of nothing; tokens among them and outside."""
    r = np.random.default_rng(11)
    V = 5000
    x = r.normal(size=(16, V)) * 4
    x[0] = 1.25
    x[1] = np.round(x[1] / 4)
    x[2, r.random(V) < 0.9] = -np.inf
    x[3] = -np.inf
    x[4, r.random(V) < 0.3] = np.nan
    x[5, [7, 4000, 4999]] = np.inf
    x[6] = -np.inf
    x[6, 4321] = -3.0
    x[7, 17] = 1e30 if dtype == "f32" else 2.0 ** 100
    x[8] = np.where(r.random(V) < 0.5, 0.0, -0.0)
    x[9] = np.nan
    x[10, 100:] = x[10, :100].min() - 200.0
    x[11] = -x[11].max() - 1e5
    x[12, [1, 2]] = -np.inf
    t = bf16(x) if dtype == "bf16" else torch.from_numpy(x.astype(np.float32)).cuda()
    if dtype == "f32":
        t.view(torch.int32)[13, 50] = 0x7f800001                  # a signalling NaN
        t.view(torch.int32)[13, 51] = -0x7fffff
        t.view(torch.int32)[13, 60:70] = 1                         # subnormals: apart from zero and each other
        t.view(torch.int32)[13, 65] = 2
    else:
        t.view(torch.int16)[13, 50] = 0x7f81
    tokens = np.array([2500, 4000, int(np.flatnonzero(x[2] == -np.inf)[40]), 10, int(np.flatnonzero(np.isnan(x[4]))[3]), 4000, 4321, 3, 4998, 0, 99,
                       4999, 2, 65, -1, V])
    check_scores(nhm, t, tokens, 12)
    check_scores(nhm, t, np.roll(tokens, 1) % V, 0)
    lp, rank, ent, _, _ = nhm.token_logprobs(t, None)
    assert not lp.any() and not rank.any()
    within(f64(ent), [lo.token_logprobs(row, 0, 0)[2] for row in f64(t)], 2.0 ** -17, "entropy without tokens")


def test_logprobs_are_the_beams(nhm):
    """The alternatives of a row are the continuations beam selection takes from it."""
    r = np.random.default_rng(12)
    x = bf16(r.normal(size=(6, 40000)) * 3)
    _, _, _, tl, tt = nhm.token_logprobs(x, None, n_top=8)
    scores, _, tokens = nhm.beam_select(x, torch.zeros(6, 1, device="cuda"), 8)
    assert torch.equal(tt, tokens) and torch.allclose(tl, scores, rtol=0, atol=2.0 ** -18)


def test_logprobs_row_past_two_gib(nhm):
    """Rows whose offsets pass 32 bits."""
    rows, vocab = 17, 1 << 24
    x = torch.full((rows, vocab), -1e4, dtype=torch.float32, device="cuda")[:, :vocab - 1]
    x[:, 5], x[rows - 1, vocab - 2] = 1.0, 2.0
    lp, rank, ent, tl, tt = nhm.token_logprobs(x, i32([vocab - 2] * rows), n_top=2)
    assert rank.tolist() == [vocab - 1] * (rows - 1) + [1] and tt[rows - 1].tolist() == [vocab - 2, 5] and tt[0].tolist() == [5, 0]
    within(f64(lp)[-1], -np.log1p(np.exp(-1.0)), 2.0 ** -19, "log probability")


# ---------------------------------------------------------------- offsets past 32 bits

def far(t, ld, at=0):
    """The same rows ld elements apart, in memory that is not initialised."""
    v = torch.empty(t.shape[0] * ld, dtype=t.dtype, device="cuda").as_strided(t.shape, (ld, 1), at)
    v.copy_(t)
    return v


def test_rows_far_apart(nhm):
    """Rows of which the last lie more than 2^32 bytes, and 2^31 elements, from the first: the same bits as close together."""
    r = np.random.default_rng(15)
    t, ld, dim, n = 36000, 65536, 64, 16
    x, dt, z, B, C = (bf16(r.normal(size=(t, c))) for c in (dim, dim, dim, n, n))
    fx, fz = far(x, ld, 8), far(z, ld, 3)
    assert all(torch.equal(a, b) for a, b in zip(nhm.mxfp4_quantize(fx), nhm.mxfp4_quantize(x)))
    where = (i32([0, 20000, t - 5]), i32([1, 0]), i32([1, 0]))
    w, b, lay = bf16(r.normal(size=(dim, 4))), bf16(r.normal(size=dim)), Layer(nhm, r, dim, n)
    windows = bf16(r.normal(size=(2, 3, dim)))
    cp = [windows.clone() for _ in range(2)]
    out = far(torch.full_like(x, 3.0), ld, 16)
    nhm.causal_conv_prefill(fx, w, b, *where, cp[0], out=out)
    assert torch.equal(out.view(torch.int16), nhm.causal_conv_prefill(x, w, b, *where, cp[1])) and torch.equal(*cp)
    states = torch.from_numpy(r.normal(size=(2, dim, n)).astype(np.float32)).cuda()
    sp = [states.clone() for _ in range(2)]
    out = far(torch.full_like(x, 3.0), ld, 5)
    nhm.selective_scan_prefill(lay.params, fx, far(dt, ld, 1), far(B, ld), far(C, ld, 7), *where, sp[0], z=fz, out=out)
    want = nhm.selective_scan_prefill(lay.params, x, dt, B, C, *where, sp[1], z=z)
    assert torch.equal(out.view(torch.int16), want) and torch.equal(*sp)
    slots = i32(np.where(np.arange(t) == t - 1, 0, -1))
    for fs in (nhm.causal_conv_decode(fx, w, b, slots, cp[0]), nhm.causal_conv_decode(x, w, b, slots, cp[1])), (
            nhm.selective_scan_decode(lay.params, fx, dt, B, C, slots, sp[0], z=fz),
            nhm.selective_scan_decode(lay.params, x, dt, B, C, slots, sp[1], z=z)):
        assert torch.equal(*fs) and bool(fs[0][-1].any()) and not fs[0][:-1].any()
    assert torch.equal(*cp) and torch.equal(*sp)


@pytest.mark.parametrize("m,ld", [(3, 1 << 30), (40, 1 << 26), (70, 1 << 25), (300, 1 << 23), (300, (1 << 23) + 1)])
def test_mxfp4_linear_outputs_far_apart(nhm, m, ld):
    r = np.random.default_rng(m)
    n, k = 136, 256
    w = nhm.Mxfp4Weight(u8(r.integers(0, 256, (n, k // 2))), u8(r.integers(118, 130, (n, k // 32))))
    x = bf16(r.normal(size=(m, k)))
    out = torch.empty(m * ld, dtype=torch.float32, device="cuda").as_strided((m, n), (ld, 1))
    nhm.mxfp4_linear(x, w, out=out)
    assert torch.equal(out, nhm.mxfp4_linear(x, w, out_type=nhm.NHM_F32))


# ---------------------------------------------------------------- streams and graphs

def everything(nhm, s, stream=None):
    """One pass of every operator over s; the outputs."""
    kw = dict(stream=stream)
    codes, scales = nhm.mxfp4_quantize(s["x"], **kw)
    y = nhm.mxfp4_linear(codes, s["w"], a_scale=scales, ws=s["ws"][0], **kw)
    y2 = nhm.mxfp4_linear(s["x"], s["w"], out_type=nhm.NHM_F32, ws=s["ws"][1], **kw)
    c = nhm.causal_conv_prefill(s["x"], s["cw"], s["cb"], s["cu"], s["slots"], s["init"], s["cp"], **kw)
    c1 = nhm.causal_conv_decode(s["x"][:3], s["cw"], s["cb"], s["slots"], s["cp"], **kw)
    h = nhm.selective_scan_prefill(s["p"], s["x"], s["dt"], s["B"], s["C"], s["cu"], s["slots"], s["init"], s["sp"], z=s["x"],
                                   ws=s["ws"][2], **kw)
    h1 = nhm.selective_scan_decode(s["p"], s["x"][:3], s["dt"][:3], s["B"][:3], s["C"][:3], s["slots"], s["sp"], **kw)
    scores = nhm.token_logprobs(s["logits"], s["tokens"], n_top=6, ws=s["ws"][3], **kw)
    return [codes, scales, nhm.mxfp4_dequantize(codes, scales, **kw), y, y2, c, c1, h, h1, *scores]


def everything_inputs(nhm, seed):
    r = np.random.default_rng(seed)
    dim, n, t = 64, 16, 700
    s = dict(x=bf16(r.normal(size=(t, dim))), dt=bf16(r.normal(size=(t, dim))), B=bf16(r.normal(size=(t, n))), C=bf16(r.normal(size=(t, n))),
             cw=bf16(r.normal(size=(dim, 4))), cb=bf16(r.normal(size=dim)), cu=i32([0, 300, 301, 690]), slots=i32([2, 0, 3]), init=i32([1, 0, 1]),
             cp=bf16(r.normal(size=(4, 3, dim))), sp=torch.from_numpy(r.normal(size=(4, dim, n)).astype(np.float32)).cuda(),
             p=Layer(nhm, r, dim, n).params, logits=bf16(r.normal(size=(9, 20000))), tokens=i32(r.integers(0, 20000, 9)),
             w=nhm.Mxfp4Weight(u8(r.integers(0, 256, (200, dim // 2))), u8(r.integers(110, 130, (200, dim // 32)))))
    sizes = [nhm.mxfp4_linear_workspace_bytes(t, 200, dim, nhm.NHM_MXFP4), nhm.mxfp4_linear_workspace_bytes(t, 200, dim, nhm.NHM_BF16),
             nhm.selective_scan_prefill_workspace_bytes(dim, n, t, 3), nhm.token_logprobs_workspace_bytes(9, 20000, 6)]
    s["ws"] = [torch.empty(max(v, 1), dtype=torch.uint8, device="cuda") for v in sizes]
    return s


def same(a, b):
    return all(torch.equal(x.view(torch.uint8) if x.dtype != torch.float32 else x, y.view(torch.uint8) if y.dtype != torch.float32 else y)
               for x, y in zip(a, b))


def test_another_stream(nhm):
    s = everything_inputs(nhm, 1)
    pools = s["cp"].clone(), s["sp"].clone()
    want = everything(nhm, s)
    torch.cuda.synchronize()
    s["cp"].copy_(pools[0])
    s["sp"].copy_(pools[1])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = everything(nhm, s, stream=st)
    st.synchronize()
    assert same(got, want)


def test_two_graphs_replayed_at_once(nhm):
    """Two captured passes with workspaces of their own, replayed several times on two streams, with eager work between."""
    sides = []
    for seed in (2, 3):
        s = everything_inputs(nhm, seed)
        pools = s["cp"].clone(), s["sp"].clone()

        def reset(s=s, pools=pools):
            s["cp"].copy_(pools[0])
            s["sp"].copy_(pools[1])

        want = [o.clone() for o in everything(nhm, s)]
        torch.cuda.synchronize()
        reset()
        torch.cuda.synchronize()
        g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=st):
            out = everything(nhm, s)
        sides.append((g, st, out, want, reset))
    for _ in range(4):
        for g, st, out, want, reset in sides:
            reset()
            for o in out:
                o.zero_()
        torch.cuda.synchronize()
        for g, st, *_ in sides:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for g, st, out, want, reset in sides:
            assert same(out, want)


def test_binding_refusals_on_the_gpu(nhm):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = nhm.Mxfp4Weight(u8(np.zeros((8, 32))), u8(np.zeros((8, 2))))
    z = torch.zeros(4, 32, dtype=torch.uint8, device="cuda")
    p = nhm.ScanParams(torch.zeros(64, 16, device="cuda"))
    b = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    pool, cp = torch.zeros(8, 64, 16, device="cuda"), torch.zeros(8, 3, 64, dtype=torch.bfloat16, device="cuda")
    cw, sl = torch.zeros(64, 4, dtype=torch.bfloat16, device="cuda"), i32(np.zeros(4))
    wrong = [lambda: nhm.mxfp4_linear(z, w), lambda: nhm.mxfp4_linear(x, w, a_scale=z[:, :2]), lambda: nhm.mxfp4_linear(x.t(), w),
             lambda: nhm.mxfp4_linear(x.float(), w), lambda: nhm.mxfp4_linear(x[:, :32], w),
             lambda: nhm.mxfp4_linear(x, w, out=torch.zeros(4, 9, device="cuda")), lambda: nhm.mxfp4_quantize(x[:, ::2]),
             lambda: nhm.Mxfp4Weight(z, z), lambda: nhm.selective_scan_decode(p, x, x, b, b[:, :8], sl, pool),
             lambda: nhm.selective_scan_decode(p, x, x, b, b, sl[:2], pool), lambda: nhm.selective_scan_decode(p, x, x, b, b, sl, pool[:, :8]),
             lambda: nhm.selective_scan_decode(p, x, x.float(), b, b, sl, pool), lambda: nhm.causal_conv_decode(x, cw, None, sl, cp[:, :2]),
             lambda: nhm.causal_conv_decode(x, cw, None, sl.long(), cp), lambda: nhm.causal_conv_decode(x, cw[:32], None, sl, cp),
             lambda: nhm.causal_conv_prefill(x, cw, None, sl, sl, sl, cp), lambda: nhm.token_logprobs(x, sl[:2]),
             lambda: nhm.token_logprobs(x, sl, n_top=2, top_tokens=i32(np.zeros((4, 3)))), lambda: nhm.token_logprobs(x[0], sl),
             lambda: nhm.token_logprobs(x, sl.cpu())]
    for i, f in enumerate(wrong):
        with pytest.raises((ValueError, TypeError)):
            f()
            print("not refused:", i)
    for f in [lambda: nhm.token_logprobs(x, sl, n_top=65), lambda: nhm.mxfp4_quantize(x[:, :16]),
              lambda: nhm.mxfp4_linear(x.repeat(2, 1), w, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))]:
        with pytest.raises(nhm.NhmError):
            f()
