"""The serving operators at the ends of their documented limits."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def nhm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_w8a8_linear_amd as m
    return m


@pytest.mark.parametrize("G,f32", [((1 << 22) + 3, False), ((1 << 23) + 5, True), ((1 << 24) - 1, False)])
def test_beam_select_many_groups(nhm, G, f32):
    """One beam in each of more groups than one launch of 512 threads a group can hold."""
    print(f"select G={G} f32={f32}", flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(G)
    x = torch.randint(-8, 9, (G, 3), generator=g, device="cuda").float() / 4     # ties go to the lowest token
    cum = torch.randint(-64, 1, (G, 1), generator=g, device="cuda").float() / 8
    s, p, t = nhm.beam_select(x if f32 else x.bfloat16(), cum, 1)
    torch.cuda.synchronize()
    top, lse = x.double().amax(dim=1), torch.logsumexp(x.double(), dim=1)
    first = torch.where(x == top[:, None].float(), torch.arange(3, device="cuda"), 3).amin(dim=1)
    assert torch.equal(t.view(-1).long(), first) and not bool(p.any())
    want = cum.view(-1).double() + top - lse
    # 2^-24 of the score, and three f32 terms of the sum: |d| 2^-24 + 2^-22 each, two additions, |d| <= 4
    assert bool(((s.view(-1).double() - want).abs() <= 2.0 ** -24 * want.abs() + 40 * 2.0 ** -24).all())


LONG_KINDS = ["normal", "constant", "ascending", "descending", "few_values", "one_hot", "huge", "late_peaks", "span_peaks",
              "equal_peaks", "masked"]
LONG_GROUPS, LONG_V = (0, 700, 1365), 40000         # 1,366 groups of 3 beams: one strip to a row, of 20 pieces


def long_rows(kind):
    """float64 [3, 3, LONG_V] of the groups that are looked at: what a strip has kept from one span meets the next one's."""
    r = np.random.default_rng(len(kind))
    base = np.arange(LONG_V, dtype=np.float64)
    x = r.standard_normal((3, 3, LONG_V)) * 3
    if kind == "constant":
        x[:] = 1.5
    elif kind == "ascending":
        x[:] = base / 64
    elif kind == "descending":
        x[:] = -base / 64
    elif kind == "few_values":
        x = r.integers(0, 4, x.shape) * 2.0
    elif kind == "one_hot":
        x[:] = np.where(base == 33333, 50.0, -50.0)
    elif kind == "huge":
        x = r.integers(-3, 4, x.shape) * 1e30
    elif kind == "late_peaks":
        x[:] = np.where(base >= LONG_V - 50, base - LONG_V, -700.0) / 16
    elif kind == "span_peaks":                       # each span of 16,384 logits has better ones than the one before
        x = r.integers(0, 8, x.shape) / 4.0 + 4.0 * (base // 16384)
    elif kind == "equal_peaks":                      # each span as many of the same best value, fewer than are asked for
        x = np.where((base % 16384) % 1024 == 7, 9.0, -r.integers(0, 64, x.shape) / 8.0)
    elif kind == "masked":
        x[:, 0, :20000] = -np.inf                    # nothing in the first span
        x[:, 1, 16000:] = np.nan                     # nothing after it
        x[0, 2] = -np.inf
        x[1, 2, [3, 39999]] = np.inf
        x[2, 2, 100:] = -np.inf
    return x


def long_reference(kind, f32, n_cand):
    from oracle import bf16_to_f64, serving_oracle as so
    from workloads import bf16_bits
    x = long_rows(kind).astype(np.float32)
    with np.errstate(invalid="ignore"):
        xs = x if f32 else bf16_bits(x)
    cum = np.array([[0.0, -1.25, -2.5], [-0.75, -0.5, -3.25], [-2.0, -0.125, -1.0]], np.float32)
    return xs, cum, so.beam_select(xs.astype(np.float64) if f32 else bf16_to_f64(xs), cum, n_cand)


# The error of log(sum), in 2^-24: that of the terms and of the f32 partial sums, 72 (each exponential |d| + 4 of itself, |d| e^-|d|
# <= 0.37, and 64 additions); at each of at most 19 changes of a lane's maximum between pieces the sum so far is scaled by an
# exponential off by 3 |d| + 2 of itself, of which a part w <= 1 is in the final sum, and once more at the join of the lanes: 2 each,
# and 3 sum(|d| w) <= 3 (1 + ln 640) = 23, since w <= 640 e^-(sum of the later |d|).
LONG_TOL = (72 + 2 * 20 + 2 * 23) * 2.0 ** -24


@pytest.mark.parametrize("n", [1, 40, 64])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("kind", LONG_KINDS)
def test_beam_select_long_strips(nhm, kind, f32, n):
    """Strips of three spans of eight pieces (the last a short one), as with thousands of rows. The other groups' beams are
    finished, so that their logits count for nothing."""
    G, V = 1366, LONG_V
    xs, cum, (s, p, t, gap) = long_reference(kind, f32, n)
    print(f"select long strips {kind} f32={f32} n={n} gap={gap:.2e}", flush=True)
    assert gap > 2 * LONG_TOL, "the inputs leave the order to rounding"
    logits = torch.full((G * 3, V), 1e4, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    d = torch.from_numpy(xs if f32 else xs.view(np.int16)).cuda()
    cums = torch.zeros((G, 3), device="cuda")
    fin = torch.ones((G, 3), dtype=torch.int32, device="cuda")
    for i, g in enumerate(LONG_GROUPS):
        logits[3 * g:3 * g + 3] = d[i] if f32 else d[i].view(torch.bfloat16)
        cums[g] = torch.from_numpy(cum[i]).cuda()
        fin[g] = 0
    gs, gp, gt = (v.cpu().numpy() for v in nhm.beam_select(logits, cums, n, finished=fin, eos=V - 1))
    at = list(LONG_GROUPS)
    assert np.array_equal(gp[at], p) and np.array_equal(gt[at], t)
    none = p < 0
    assert np.all(gs[at][none] == -np.inf)
    with np.errstate(invalid="ignore"):
        assert np.all((np.abs(gs[at] - s) <= 2.0 ** -24 * np.abs(s) + LONG_TOL)[~none] | (gs[at] == s)[~none])
    rest = np.setdiff1d(np.arange(G), at)
    k = min(n, 3)
    assert np.all(gs[rest, :k] == 0) and np.all(gp[rest, :k] == np.arange(k)) and np.all(gt[rest, :k] == V - 1)
    assert np.all(gp[rest, 3:] == -1) and np.all(gs[rest, 3:] == -np.inf)
