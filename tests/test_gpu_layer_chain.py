"""The layer operators together, as a server runs them: a batch of prompts from its plan through one selective scan layer
with MXFP4 projections and the scoring of its logits, then single tokens, each stage against its plain 64-bit form of what
the stage before it left, and the same steps from a captured graph."""
import numpy as np
import pytest

from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_gpu_layer import Layer, bf16, check_state, f64, i32, u8, within  # noqa: E402


@pytest.fixture(scope="module")
def nhm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_w8a8_linear_amd as m
    return m


HIDDEN, DIM, N, VOCAB, TOP = 96, 160, 16, 1500, 4


class Block:
    def __init__(self, nhm, seed):
        r = np.random.default_rng(seed)
        self.layer = Layer(nhm, r, DIM, N)
        self.values, self.weights = {}, {}
        for name, n, k, gain in [("in", 2 * DIM, HIDDEN, 1.5), ("x", DIM + 2 * N, DIM, 1.0), ("out", HIDDEN, DIM, 1.0), ("head", VOCAB, HIDDEN, 3.0)]:
            codes, scales = lo.mxfp4_quantize(r.normal(size=(n, k)) * gain / np.sqrt(k))
            self.values[name] = lo.mxfp4_values(codes, scales)
            self.weights[name] = nhm.Mxfp4Weight(u8(lo.mxfp4_pack(codes)), u8(scales))
        self.cw, self.cb = bf16(r.normal(size=(DIM, 4)) / 2), bf16(r.normal(size=DIM) / 4)

    def run(self, nhm, x, tokens, conv, scan, codes):
        """The layer's stages on x; conv(x) and scan(u, dt, B, C, z) are the calls for prompts or for single tokens."""
        bf = lambda t: t.view(torch.bfloat16)  # noqa: E731
        o = dict(x=x)
        o["xz"] = bf(nhm.mxfp4_linear(x, self.weights["in"]))
        o["u"] = bf(conv(o["xz"][:, :DIM]))
        if codes:       # quantised once, as where several projections read the same activation
            c, s = nhm.mxfp4_quantize(o["u"])
            o["proj"] = bf(nhm.mxfp4_linear(c, self.weights["x"], a_scale=s))
        else:
            o["proj"] = bf(nhm.mxfp4_linear(o["u"], self.weights["x"]))
        p = o["proj"]
        o["y"] = bf(scan(o["u"], p[:, :DIM], p[:, DIM:DIM + N], p[:, DIM + N:], o["xz"][:, DIM:]))
        o["out"] = bf(nhm.mxfp4_linear(o["y"], self.weights["out"]))
        o["logits"] = nhm.mxfp4_linear(o["out"], self.weights["head"], out_type=nhm.NHM_F32)
        o["scores"] = nhm.token_logprobs(o["logits"], tokens, n_top=TOP)
        return o

    def check_linear(self, o, a, name, to, f32=False):
        av = lo.mxfp4_values(*lo.mxfp4_quantize(f64(o[a])))
        ref, tol = lo.mxfp4_linear(av, self.values[name])
        within(f64(o[to]), ref, tol * (1 + 2.0 ** -8) + lo.half_step(ref, not f32), to)

    def check(self, o, tokens, spans, slots, init, windows, states):
        """spans: the rows of each sequence; windows and states by slot as they were. Returns them as they should be, the
        states' tolerances with them."""
        self.check_linear(o, "x", "in", "xz")
        self.check_linear(o, "u", "x", "proj")
        self.check_linear(o, "y", "out", "out")
        self.check_linear(o, "out", "head", "logits", f32=True)
        W, b = f64(self.cw), f64(self.cb)
        xz, u, y, p = f64(o["xz"]), f64(o["u"]), f64(o["y"]), f64(o["proj"])
        windows, states, errs = windows.copy(), states.copy(), np.zeros_like(states)
        for e, s, h0 in zip(spans, slots, init):
            rows = np.concatenate([windows[s] * (h0 != 0), xz[e, :DIM]])
            ref, tol = lo.causal_conv(rows, W, b, True)
            within(u[e], ref, tol * (1 + 2.0 ** -8) + lo.half_step(ref, True), "conv")
            windows[s] = rows[len(rows) - 3:]
            ref, tol, states[s], errs[s] = self.layer.ref(u[e], p[e, :DIM], p[e, DIM:DIM + N], p[e, DIM + N:], states[s] * (h0 != 0), xz[e, DIM:])
            within(y[e], ref, tol * (1 + 2.0 ** -8) + lo.half_step(ref, True), "scan")
        lp, rank, ent, tl, tt = o["scores"]
        for i, row in enumerate(f64(o["logits"])):
            w_lp, w_rank, w_ent, w_tl, w_tt = lo.token_logprobs(row, int(tokens[i]), TOP)
            within(f64(lp)[i], w_lp, lo.logprob_tolerance(w_lp), "log probability")
            within(f64(ent)[i], w_ent, 2 * lo.logprob_tolerance(w_ent), "entropy")
            within(f64(tl)[i], w_tl, lo.logprob_tolerance(w_tl), "alternatives' log probabilities")
            assert int(rank[i]) == w_rank and tt[i].tolist() == w_tt.tolist(), f"row {i}"
        return windows, states, errs


@pytest.mark.parametrize("lengths,tail,codes", [([70, 1, 33, 0, 5], 11, False), ([2, 0, 1], 0, True), ([900], 0, False), ([17, 300, 40], 1, True)])
def test_prompts_then_tokens(nhm, lengths, tail, codes):
    r = np.random.default_rng(sum(lengths))
    block, S, n = Block(nhm, 5), len(lengths) + 2, len(lengths)
    slots, past = r.permutation(S)[:n], np.where(r.random(n) < 0.5, 12, 0)
    cp = bf16(r.normal(size=(S, 3, DIM)))
    sp = torch.from_numpy(r.normal(size=(S, DIM, N)).astype(np.float32)).cuda()
    windows, states = f64(cp), f64(sp)
    T = sum(lengths) + tail
    plan = nhm.batch_plan(i32(lengths), nhm.BatchPlan(n, T), past=i32(past))
    x, tokens, sl = bf16(r.normal(size=(T, HIDDEN))), r.integers(0, VOCAB, T), i32(slots)
    where = (plan.cu_seqlens, sl, plan.has_initial)
    o = block.run(nhm, x, i32(tokens), lambda v: nhm.causal_conv_prefill(v, block.cw, block.cb, *where, cp),
                  lambda u, dt, B, C, z: nhm.selective_scan_prefill(block.layer.params, u, dt, B, C, *where, sp, z=z), codes)
    cu = np.concatenate([[0], np.cumsum(lengths)])
    windows, states, errs = block.check(o, tokens, [slice(cu[i], cu[i + 1]) for i in range(n)], slots, past, windows, states)
    assert np.array_equal(f64(cp), windows)
    check_state(f64(sp), states, errs, False)
    assert not o["u"][cu[-1]:].any() and not o["y"][cu[-1]:].any()
    # single tokens, from the states as the device holds them
    for _ in range(3):
        states = f64(sp)
        x, tokens = bf16(r.normal(size=(n, HIDDEN))), r.integers(0, VOCAB, n)
        o = block.run(nhm, x, i32(tokens), lambda v: nhm.causal_conv_decode(v, block.cw, block.cb, sl, cp),
                      lambda u, dt, B, C, z: nhm.selective_scan_decode(block.layer.params, u, dt, B, C, sl, sp, z=z), codes)
        windows, states, errs = block.check(o, tokens, [slice(i, i + 1) for i in range(n)], slots, np.ones(n), windows, states)
        assert np.array_equal(f64(cp), windows)
        check_state(f64(sp), states, errs, False)


@pytest.mark.parametrize("rows", [1, 6, 70])
def test_captured_steps(nhm, rows):
    """Steps of single tokens from a graph, eager work between the replays: bit for bit the eager steps."""
    r = np.random.default_rng(rows)
    block = Block(nhm, 6)
    sl = i32(r.permutation(rows + 1)[:rows])
    start = bf16(r.normal(size=(rows + 1, 3, DIM))), torch.from_numpy(r.normal(size=(rows + 1, DIM, N)).astype(np.float32)).cuda()
    steps = [(bf16(r.normal(size=(rows, HIDDEN))), i32(r.integers(0, VOCAB, rows))) for _ in range(4)]

    def step(x, tokens, cp, sp):
        return block.run(nhm, x, tokens, lambda v: nhm.causal_conv_decode(v, block.cw, block.cb, sl, cp),
                         lambda u, dt, B, C, z: nhm.selective_scan_decode(block.layer.params, u, dt, B, C, sl, sp, z=z), False)

    pools, x, tokens = [t.clone() for t in start], steps[0][0].clone(), steps[0][1].clone()
    step(x, tokens, *pools)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = step(x, tokens, *pools)
    for p, s in zip(pools, start):
        p.copy_(s)
    eager = [t.clone() for t in start]
    for sx, st in steps:
        x.copy_(sx)
        tokens.copy_(st)
        g.replay()
        torch.cuda.synchronize()
        want = step(sx, st, *eager)
        assert torch.equal(o["logits"], want["logits"]) and all(torch.equal(a, b) for a, b in zip(o["scores"], want["scores"]))
        assert torch.equal(pools[0], eager[0]) and torch.equal(pools[1], eager[1])
