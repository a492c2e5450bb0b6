"""The layer operators (include/nhm_layer.h) on the paths that depend on a batch's shape, and on values in places where a
kernel's own layout counts, against plain 64-bit forms."""
import numpy as np
import pytest

from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_gpu_layer import Layer, bf16, check_scores, check_state, f64, i32, nhm, scan_inputs, u8, within  # noqa: E402,F401
from tests.test_layer_tiles import TILE_CASES  # noqa: E402


# ---------------------------------------------------------------- MXFP4 projection: the tiles of many rows

@pytest.mark.parametrize("m,n,k,codes,f32,tn,tm,turns", TILE_CASES)
def test_mxfp4_linear_tiles(nhm, m, n, k, codes, f32, tn, tm, turns):
    """Every tile, one and several in turn of a workgroup, stores of whole 16 bytes and single ones, ragged edges on both sides; whole
    outputs against products in 64 bits, and nothing stored beside them."""
    print(m, n, k, tn, tm, turns, flush=True)
    r = np.random.default_rng(m + n + k)
    w, ws = r.integers(0, 16, (n, k)).astype(np.uint8), r.integers(110, 135, (n, k // 32)).astype(np.uint8)
    weight = nhm.Mxfp4Weight(u8(lo.mxfp4_pack(w)), u8(ws))
    if codes:
        a, s = r.integers(0, 16, (m, k)).astype(np.uint8), r.integers(110, 135, (m, k // 32)).astype(np.uint8)
        x, xs = u8(lo.mxfp4_pack(a)), u8(s)
    else:
        x, xs = bf16(r.normal(size=(m, k)) * np.exp2(r.integers(-8, 8, (m, 1)).astype(float))), None
        a, s = lo.mxfp4_quantize(f64(x))
    right = 0 if n % 8 == 0 else 5               # rows of whole 16 bytes behind their like, odd ones behind odd ones
    out = torch.full((m + 2, n + right), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    nhm.mxfp4_linear(x, weight, a_scale=xs, out=out[1:m + 1, :n])
    av, wv = (torch.from_numpy(v).cuda() for v in (lo.mxfp4_values(a, s), lo.mxfp4_values(w, ws).T.copy()))
    ref, tol = av @ wv, lo.U * (k / 128 + 18) * (av.abs() @ wv.abs())          # as the oracle's
    tol = tol * (1 + 2.0 ** -8) + ref.abs() * (lo.U if f32 else 2.0 ** -8)
    wrong = ~((out[1:m + 1, :n].double() - ref).abs() <= tol)
    assert not bool(wrong.any()), f"{int(wrong.sum())} outside, first at {wrong.nonzero()[0].tolist()}"
    out[1:m + 1, :n] = 7.0
    assert bool((out == 7.0).all()), "stores outside the output"


# ---------------------------------------------------------------- scoring of tokens

def to_logits(x, dtype):
    return bf16(x) if dtype == "bf16" else torch.from_numpy(x.astype(np.float32)).cuda()


def put_signalling_nan(t, row, at):
    if t.dtype == torch.float32:
        t.view(torch.int32)[row, at] = 0x7f800001
    else:
        t.view(torch.int16)[row, at] = 0x7f81


def lane_place(i, lane, dtype):
    """The place in a piece of 2,048 logits of the i-th of a lane's 32."""
    E = 4 if dtype == "f32" else 8
    return ((i // E) * 64 + lane) * E + i % E


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["best", "infinite", "far above"])
def test_logprobs_signalling_nan_behind(nhm, dtype, kind):
    """A signalling NaN counts as -inf also behind what decides its lane: the row's best logit, a +inf, and a logit 200 above the
    rest, at every two neighbouring places of a lane's 32, in the first and in a later piece."""
    r = np.random.default_rng(21)
    V = 5000
    x = r.normal(size=(62, V)) * 3
    tokens, nans = np.zeros(62, int), []
    for row in range(62):
        i, lane, piece = 1 + row % 31, int(r.integers(0, 64)), row // 31
        at, nan = (piece * 2048 + lane_place(j, lane, dtype) for j in (i - 1, i))
        x[row, at] = {"best": 20.0, "infinite": np.inf, "far above": 200.0}[kind]
        tokens[row] = at if row % 3 else r.integers(0, V)
        nans.append((row, nan))
    t = to_logits(x, dtype)
    for row, nan in nans:
        put_signalling_nan(t, row, nan)
    check_scores(nhm, t, tokens, 5)
    check_scores(nhm, t, tokens, 0)


def test_logprobs_of_many_rows(nhm):
    """More than 2^22 rows, the last of them among them, against torch's log softmax in 64 bits."""
    rows, V = (1 << 22) + 5, 7
    g = torch.Generator(device="cuda")
    g.manual_seed(22)
    x = (torch.randn(rows, V, generator=g, device="cuda") * 2).to(torch.bfloat16)
    tokens = torch.randint(-1, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
    lp, rank, ent, tl, tt = nhm.token_logprobs(x, tokens, n_top=2)
    want, t = torch.log_softmax(x.double(), dim=1), tokens.long().clamp(min=0)[:, None]
    none = tokens < 0
    own, at = x.gather(1, t), torch.arange(V, device="cuda")
    place = 1 + ((x > own) | ((x == own) & (at < t))).sum(dim=1)
    tol = 2.0 ** -19 + 2.0 ** -24 * 64          # as the oracle's; no log probability is below -64
    assert bool(((lp - want.gather(1, t)[:, 0]).abs() <= tol)[~none].all()) and not lp[none].any()
    assert torch.equal(rank.long(), torch.where(none, 0, place))
    assert bool(((ent + (want.exp() * want).sum(dim=1)).abs() <= 2 * tol).all())
    order = torch.sort(x.float(), dim=1, descending=True, stable=True)[1][:, :2]
    assert torch.equal(tt.long(), order) and bool(((tl - want.gather(1, order)).abs() <= tol).all())


def strip_tolerance(x, pieces):
    """(of the log of the sum, of the entropy) of a row that waves walk in strips of up to `pieces` pieces. D: an entry's distance from
    the row's largest logit in log2, p its probability. A term and its rescalings, at most `pieces` of them, each an exp2 (2 U) of an
    argument of three roundings: 2 U (1 + pieces) + 3 ln2 U D; seven sums in f32 to a piece's term. The moment's terms are D times that,
    with D's own three roundings and 32 sums."""
    x = np.where(np.isnan(x), -np.inf, x)
    if not np.isfinite(x.max()):
        return 2.0 ** -23, 2.0 ** -23           # counts, exact, and a logarithm
    D = (x.max() - x) / np.log(2)
    p = np.exp2(-D) / np.exp2(-D).sum()
    D, p = D[p > 0], p[p > 0]
    each = 2 * (1 + pieces) + 2.1 * D
    s = lo.U * (p * (each + 7)).sum()
    return s, s + np.log(2) * (lo.U * (p * D * (each + 35)).sum() + (p * D).sum() * s)


@pytest.mark.parametrize("rows,V,pieces", [(1400, 40000, 7), (4100, 20001, 10)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs_over_many_pieces(nhm, rows, V, pieces, dtype):
    """Strips of several pieces and of more than one span of eight: maxima that rise and fall along the row, infinities, NaN and masked
    runs in its later pieces, tokens and alternatives anywhere."""
    strips = -(-(-(-V // 2048)) // pieces)
    assert nhm.token_logprobs_workspace_bytes(rows, V, 0) == -(-rows * strips * 24 // 256) * 256, "other strips: choose other sizes"
    r = np.random.default_rng(V)
    special = r.normal(size=(18, V)) * 3
    special[0] = np.sort(special[0] * 2)
    special[1] = np.sort(special[1] * 2)[::-1]
    special[2, V - 3] = 120.0
    special[3, :V * 3 // 5] = -np.inf
    special[4, 6 * 2048 + lane_place(7, 33, dtype)] = np.inf
    special[5, V // 2:][r.random(V - V // 2) < 0.3] = np.nan
    special[6] += np.arange(V) // 2048 * 8.0
    special[7] = -np.inf
    special[7, V - 1] = -3.0
    special[8] = -np.inf
    special[9] = 1.25
    special[10] = np.round(special[10] / 3)
    special[11, V - 100:] += 30.0
    special[12, 17::2048] = 40.0
    special[13, [3, V - 2]] = np.inf
    special[14] -= np.arange(V) // 2048 * 8.0
    special[15, 8 * 2048 + lane_place(20, 5, dtype)] = 150.0
    special[16, :2048] = np.nan
    special[16, 9 * 2048:] = -np.inf
    special[17] = np.where(np.arange(V) < V - 4096, -1e30, special[17])
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    t = (torch.randn(rows, V, generator=g, device="cuda") * 3).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    at = np.r_[r.permutation(np.arange(1, rows - 1))[:17], rows - 1]
    t[torch.from_numpy(at).cuda()] = to_logits(special, dtype)
    put_signalling_nan(t, int(at[4]), 6 * 2048 + lane_place(8, 33, dtype))
    put_signalling_nan(t, int(at[15]), 8 * 2048 + lane_place(21, 5, dtype))
    look = np.r_[at, 0, r.integers(0, rows, 6)]
    X = f64(t[torch.from_numpy(look).cuda()])
    tolerance = [strip_tolerance(x, pieces) for x in X]
    for call, n_top in enumerate((20, 64, 0)):
        tokens = r.integers(0, V, rows)
        tokens[look] = r.integers([0, V // 3, V - 2048][call], [2048, V * 2 // 3, V][call], len(look))
        if call == 1:
            tokens[look] = np.nanargmax(np.where(np.isnan(X), -np.inf, X), axis=1)
        lp, rank, ent, tl, tt = nhm.token_logprobs(t, i32(tokens), n_top=n_top)
        lp, ent, tl = f64(lp), f64(ent), f64(tl)
        for i, x, (tol, tol_h) in zip(look, X, tolerance):
            w_lp, w_rank, w_ent, w_tl, w_tt = lo.token_logprobs(x, tokens[i], n_top)
            what = f"row {i}, place {np.flatnonzero(look == i)}, call {call}"
            within(lp[i], w_lp, tol + lo.half_step(np.nan_to_num(w_lp, neginf=0), False), what + ": log probability")
            assert int(rank[i]) == w_rank, f"{what}: rank {int(rank[i])} for {w_rank}"
            within(ent[i], w_ent, tol_h + lo.half_step(w_ent, False), what + ": entropy")
            assert tt[i].tolist() == w_tt.tolist(), what + ": alternatives"
            within(tl[i], w_tl, tol + lo.half_step(np.nan_to_num(w_tl, neginf=0), False), what + ": alternatives' log probabilities")


# ---------------------------------------------------------------- scan: values that are not finite

@pytest.mark.parametrize("n", [4, 16, 20, 64])
@pytest.mark.parametrize("first", [150, 2600])
def test_scan_not_finite_in_every_form(nhm, n, first):
    """u of infinity or NaN and dt of NaN or +inf keep to their channel and sequence, in the sequence's first tokens, its middle and its
    last ones, whether it is scanned whole or in chunks; dt of -inf, once or at every token, is a step of 0."""
    r = np.random.default_rng(n + first)
    dim, t = 40, first + 200
    assert (nhm.selective_scan_prefill_workspace_bytes(dim, n, t, 2) > 0) == (first > 1000)
    lay = Layer(nhm, r, dim, n)
    u, dt, B, C, z = scan_inputs(r, t, dim, n, True)
    states = torch.from_numpy(r.normal(size=(2, dim, n)).astype(np.float32)).cuda()
    where = (i32([0, first, t]), i32([0, 1]), i32([1, 1]))
    run = lambda u, dt, p: f64(nhm.selective_scan_prefill(lay.params, u, dt, B, C, *where, p, z=z).view(torch.bfloat16))  # noqa: E731
    pools = states.clone(), states.clone()
    clean = run(u, dt, pools[0])
    bu, bdt, bad = u.clone(), dt.clone(), np.zeros((t, dim), bool)
    inf, nan, mid, last = float("inf"), float("nan"), first // 2, first - 3
    for x, at, ch, v in [(bu, 20, 5, inf), (bu, 0, 6, nan), (bdt, 3, 7, inf), (bdt, mid, 13, nan), (bdt, mid + 1, 14, inf), (bu, mid + 2, 15, -inf),
                         (bu, last, 9, nan), (bdt, last, 10, inf), (bu, last + 2, 11, inf), (bdt, first + 10, 17, inf), (bu, first, 18, nan)]:
        x[at, ch] = v
        bad[at:first if at < first else t, ch] = True
    still = [21, 25, 39]
    bdt[mid, 21], bdt[:, 25], bdt[[0, last, first, t - 1], 39] = -inf, -inf, -inf
    got = run(bu, bdt, pools[1])
    same = ~bad
    same[:, still] = False
    assert np.array_equal(got[same], clean[same]) and not np.isfinite(got[bad]).any()
    kept = np.ones((2, dim), bool)
    kept[0, [5, 6, 7, 13, 14, 15, 9, 10, 11]] = kept[1, [17, 18]] = kept[:, still] = False
    assert np.array_equal(f64(pools[1])[kept], f64(pools[0])[kept])
    for i, e in enumerate((slice(0, first), slice(first, t))):
        ref, tol, h, err = lay.ref(f64(u)[e], f64(bdt)[e], f64(B)[e], f64(C)[e], f64(states)[i], f64(z)[e])
        within(got[e][:, still], ref[:, still], (tol * (1 + 2.0 ** -8) + lo.half_step(ref, True))[:, still], "steps of 0")
        check_state(f64(pools[1])[i, still], h[still], err[still], False)
    assert torch.equal(pools[1][:, 25], states[:, 25])


@pytest.mark.parametrize("n", [4, 16, 20, 64])
def test_scan_decode_not_finite(nhm, n):
    """The same for single tokens: a step of 0 leaves the state's bits alone."""
    r = np.random.default_rng(n)
    dim = 40
    lay = Layer(nhm, r, dim, n)
    u, dt, B, C, z = scan_inputs(r, 3, dim, n, True)
    states = torch.from_numpy(r.normal(size=(3, dim, n)).astype(np.float32)).cuda()
    run = lambda u, dt, p: f64(nhm.selective_scan_decode(lay.params, u, dt, B, C, i32([2, 0, 1]), p, z=z).view(torch.bfloat16))  # noqa: E731
    pools = states.clone(), states.clone()
    clean = run(u, dt, pools[0])
    inf, nan = float("inf"), float("nan")
    bu, bdt, bad = u.clone(), dt.clone(), np.zeros((3, dim), bool)
    for x, at, ch, v in [(bu, 0, 0, inf), (bu, 1, 5, nan), (bdt, 2, 7, inf), (bdt, 0, 39, nan)]:
        x[at, ch] = v
        bad[at, ch] = True
    bdt[:, 21] = -inf
    got = run(bu, bdt, pools[1])
    same = ~bad
    same[:, 21] = False
    assert np.array_equal(got[same], clean[same]) and not np.isfinite(got[bad]).any()
    assert torch.equal(pools[1][:, 21], states[:, 21])
    for i, s in enumerate([2, 0, 1]):
        ref, tol, _, _ = lay.ref(f64(u)[i:i + 1], f64(bdt)[i:i + 1], f64(B)[i:i + 1], f64(C)[i:i + 1], f64(states)[s], f64(z)[i:i + 1])
        within(got[i, 21], ref[0, 21], (tol * (1 + 2.0 ** -8) + lo.half_step(ref, True))[0, 21], "a step of 0")


# ---------------------------------------------------------------- single tokens of many sequences

def test_decode_of_many_rows(nhm):
    """More rows than a launch's y extent, of more than 2^32 threads together: the rows with a slot as in a call of their own, padding zero."""
    rows, dim, n = 65535 + 5, 4104, 64
    r = np.random.default_rng(24)
    lay = Layer(nhm, r, dim, n)
    g = torch.Generator(device="cuda")
    g.manual_seed(24)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    u, dt, B, C, z = rand(rows, dim), rand(rows, dim), rand(rows, n), rand(rows, n), rand(rows, dim)
    w, b = bf16(r.normal(size=(dim, 4))), bf16(r.normal(size=dim))
    at = torch.tensor([0, 65534, 65535, rows - 1], device="cuda")
    slots = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    slots[at] = i32([3, 0, 2, 1])
    states, windows = torch.randn(4, dim, n, generator=g, device="cuda"), rand(4, 3, dim)
    pools = states.clone(), states.clone()
    out = nhm.selective_scan_decode(lay.params, u, dt, B, C, slots, pools[0], z=z)
    want = nhm.selective_scan_decode(lay.params, u[at], dt[at], B[at], C[at], i32([3, 0, 2, 1]), pools[1], z=z[at])
    assert torch.equal(out[at], want) and torch.equal(*pools) and not torch.equal(pools[0], states)
    out[at] = 0
    assert not out.any()
    pools = windows.clone(), windows.clone()
    out = nhm.causal_conv_decode(u, w, b, slots, pools[0])
    assert torch.equal(out[at], nhm.causal_conv_decode(u[at], w, b, i32([3, 0, 2, 1]), pools[1])) and torch.equal(*pools)
    out[at] = 0
    assert not out.any()


# ---------------------------------------------------------------- batches of padding alone

@pytest.mark.parametrize("tokens", [0, 7, 2000])
def test_no_sequences(nhm, tokens):
    """A batch without sequences: every row is behind the last one and zero, the pools stay."""
    dim, n = 72, 16
    r = np.random.default_rng(25)
    lay = Layer(nhm, r, dim, n)
    u, dt, B, C, z = (torch.full((tokens, c), float("nan"), dtype=torch.bfloat16, device="cuda") for c in (dim, dim, n, n, dim))
    none, states, windows = i32([]), torch.randn(2, dim, n, device="cuda"), bf16(r.normal(size=(2, 3, dim)))
    pools = states.clone(), windows.clone()
    out = torch.full((tokens, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    nhm.selective_scan_prefill(lay.params, u, dt, B, C, i32([0]), none, none, pools[0], z=z, out=out)
    assert not out.any()
    out.fill_(3.0)
    nhm.causal_conv_prefill(u, bf16(r.normal(size=(dim, 4))), None, i32([0]), none, none, pools[1], out=out)
    assert not out.any() and torch.equal(pools[0], states) and torch.equal(pools[1], windows)
