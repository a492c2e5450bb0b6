"""The mixer calls with adapters on the GPU at the full geometry in larger batches, on bf16 state pools, and captured into
graphs together with the plan, the selection and the reorder."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import serving_oracle as so  # noqa: E402
from tests.test_gpu_serving_chain import SMALL, adapters, block, flip_tol, lora, nhm  # noqa: E402,F401

# Two f32 states within the bar of 1e-3 of each other round to bf16 values a step (2^-7 of the value at most) apart on about
# 1e-3 / 2^-8 of the elements: an RMS of sqrt(1e-3 2^-8) = 2e-3; twice that, as for the mixer without adapters.
STATE_TOL = {True: 1e-3, False: 4e-3}


def pool(sp, f32):
    from workloads import bf16_bits
    return sp.copy() if f32 else bf16_bits(sp)


def wide(sp, f32):
    from oracle import bf16_to_f64
    return sp.astype(np.float32) if f32 else bf16_to_f64(sp).astype(np.float32)


def check_projections(p, ai, ao, ids, h, zx, norm, out, exact_out):
    """Both projections with their adapters, every row, each from the call's own input of it."""
    from oracle import bf16_to_f64
    for x, w, ad, got, exact in ((h, "in", ai, zx, True), (norm, "out", ao, out, exact_out)):
        args = (x, p[w + "_w"], p[w + "_w_scale"], p[w + "_a_scale"], *ad, ids)
        ref = so.fp8_linear_lora(*args)
        err = np.abs(bf16_to_f64(got) - ref)
        assert np.all(err <= so.lora_bound(*args, ref, exact=exact, f32=False)), w


def check_state(got, ref, f32):
    from oracle import bf16_from_f64, bf16_to_f64
    from tests.gpu_util import rel_l2
    if f32:
        assert rel_l2(got, ref) <= STATE_TOL[True]
    elif not np.any(ref):
        assert not np.any(got)
    else:
        assert rel_l2(bf16_to_f64(got), bf16_to_f64(bf16_from_f64(ref.astype(np.float64)))) <= STATE_TOL[False]


@pytest.mark.parametrize("B,f32", [(3, False), (24, False), (40, True), (61, False), (130, True)])
def test_decode_full_geometry(nhm, B, f32):
    from oracle import bf16_to_f64
    from tests.gpu_util import dev, host, rel_max, ws_region, zeros_ws
    g, S = nhm.GEOMETRY, B + 3
    print(f"decode with adapters B={B} f32 state={f32}", flush=True)
    p, pd, ai, ao, h, sp, cp = block(nhm, g, 200 + B, S, B, e=9)
    r = np.random.default_rng(B)
    slots = r.permutation(S)[:B].astype(np.int32)
    ids = r.integers(-1, 9, B).astype(np.int32)
    slots[1], ids[1] = -1, 2                              # a padded row, with an adapter
    sp = pool(sp, f32)
    spd, cpd = dev(sp), dev(cp)
    out = torch.full((B, g["hidden"]), 0x5555, dtype=torch.int16, device="cuda")
    lay = nhm.decode_lora_ws_layout(B, 24, g)
    ws = zeros_ws(lay["total"])
    nhm.mixer_decode_lora(pd, lora(nhm, ai), lora(nhm, ao), dev(ids), dev(h), dev(slots), spd, cpd, out, ws)
    torch.cuda.synchronize()
    got, sg, cg = host(out), host(spd), host(cpd)
    n_in = p["in_w"].shape[0]
    zx = ws_region(ws, lay["zxbcdt"], B * n_in, np.uint16).reshape(B, n_in)
    norm = ws_region(ws, lay["norm"], B * 4096, np.uint16).reshape(B, 4096)
    live = slots >= 0
    assert np.all(got[1] == 0)
    check_projections(p, ai, ao, ids[live], h[live], zx[live], norm[live], got[live], exact_out=B <= 32)
    rest = np.setdiff1d(np.arange(S), slots)
    assert np.array_equal(sg[rest], sp[rest]) and np.array_equal(cg[rest], cp[rest])
    for b in sorted({0, 2, B // 2, B - 2, B - 1} - {1}):
        s = slots[b]
        o, win, st = so.mixer_sequence_lora(p, ai, ao, ids[b:b + 1], h[b:b + 1], cp[s], wide(sp[s], f32), g)
        assert rel_max(bf16_to_f64(got[b]), o[0]) <= flip_tol(g), b
        check_state(sg[s], st, f32)
        assert np.array_equal(cg[s][:2], cp[s][1:]), b


@pytest.mark.parametrize("lengths,f32", [([70, 1, 0, 230], False), ([300, 129, 271], True), ([40, 33], False)])
def test_prefill_full_geometry(nhm, lengths, f32):
    from oracle import bf16_to_f64
    from tests.gpu_util import dev, host, rel_l2, ws_region, zeros_ws
    g, n, T = nhm.GEOMETRY, len(lengths), sum(lengths)
    print(f"prefill with adapters {lengths} f32 state={f32}", flush=True)
    p, pd, ai, ao, h, sp, cp = block(nhm, g, 300 + T, n + 1, T)
    seq_ad = (np.arange(n, dtype=np.int32) * 2) % 5 - 1
    past = np.arange(n, dtype=np.int32) % 2
    slots = np.arange(n, dtype=np.int32)[::-1].copy()
    sp = pool(sp, f32)
    spd, cpd = dev(sp), dev(cp)
    plan = nhm.batch_plan(dev(np.array(lengths, np.int32)), nhm.BatchPlan(n, T), past=dev(past), adapters=dev(seq_ad))
    out = torch.empty((T, g["hidden"]), dtype=torch.int16, device="cuda")
    lay = nhm.prefill_lora_ws_layout(T, n, 24, g=g)
    ws = zeros_ws(lay["total"])
    nhm.mixer_prefill_lora(pd, lora(nhm, ai), lora(nhm, ao), plan.token_adapter, dev(h), plan.cu_seqlens, dev(slots),
                           plan.has_initial, spd, cpd, out, ws)
    torch.cuda.synchronize()
    got, sg = host(out), host(spd)
    n_in = p["in_w"].shape[0]
    zx = ws_region(ws, lay["zxbcdt"], T * n_in, np.uint16).reshape(T, n_in)
    norm = ws_region(ws, lay["norm"], T * 4096, np.uint16).reshape(T, 4096)
    check_projections(p, ai, ao, np.repeat(seq_ad, lengths), h, zx, norm, got, exact_out=False)
    t0 = 0
    for i, ln in enumerate(lengths):
        s = slots[i]
        win, st = (cp[s], wide(sp[s], f32)) if past[i] else (np.zeros_like(cp[s]), np.zeros(sp[s].shape, np.float32))
        if ln:
            ref, _, st = so.mixer_sequence_lora(p, ai, ao, np.full(ln, seq_ad[i]), h[t0:t0 + ln], win, st, g)
            assert rel_l2(bf16_to_f64(got[t0:t0 + ln]), ref) <= 2e-2, i
        check_state(sg[s], st, f32)
        t0 += ln
    assert np.array_equal(sg[n], sp[n])


@pytest.mark.parametrize("lengths,T,with_lora", [([9, 0, 23], 40, True), ([70, 1, 130], 260, True), ([0, 0], 5, True),
                                                 ([9, 0, 23], 33, False), ([300, 400], 777, False), ([5], 6, True)])
def test_prefill_of_a_padded_batch(nhm, lengths, T, with_lora):
    """Rows behind the last sequence, as a plan of fewer tokens than its buffer leaves them: zero outputs whatever hidden and
    the workspace hold there, and the sequences as without them."""
    from oracle import bf16_to_f64
    from tests.gpu_util import dev, host, rel_l2, zeros_ws
    g, n, used = SMALL, len(lengths), sum(lengths)
    print(f"padded prefill {lengths} in {T}, adapters {with_lora}", flush=True)
    p, pd, ai, ao, h, sp, cp = block(nhm, g, 400 + T, n, T)
    seq_ad = np.arange(n, dtype=np.int32)
    slots = np.arange(n, dtype=np.int32)
    plan = nhm.batch_plan(dev(np.array(lengths, np.int32)), nhm.BatchPlan(n, T), adapters=dev(seq_ad))
    lay = nhm.prefill_lora_ws_layout(T, n, 24, g=g)
    h[used:] = 0
    noise = h.copy()
    noise[used:] = 0x7FC0                                 # NaN
    got = []
    for hidden, fill in ((h, 0), (noise, 0xFF)):
        ws = zeros_ws(lay["total"]).fill_(fill)
        spd, cpd = dev(sp), dev(cp)
        out = torch.full((T, g["hidden"]), 0x5555, dtype=torch.int16, device="cuda")
        args = (dev(hidden), plan.cu_seqlens, dev(slots), plan.has_initial, spd, cpd, out, ws)
        if with_lora:
            nhm.mixer_prefill_lora(pd, lora(nhm, ai), lora(nhm, ao), plan.token_adapter, *args)
        else:
            nhm.mixer_prefill(pd, *args)
        torch.cuda.synchronize()
        got.append((host(out), host(spd), host(cpd)))
        assert np.all(bf16_to_f64(got[-1][0][used:]) == 0)
    assert all(np.array_equal(a, b) for a, b in zip(*got))
    none = tuple(np.zeros_like(v) for v in ai[:2]) + (None,), tuple(np.zeros_like(v) for v in ao[:2]) + (None,)
    t0 = 0
    for i, ln in enumerate(lengths):
        if ln:
            ref, _, st = so.mixer_sequence_lora(p, *((ai, ao) if with_lora else none), np.full(ln, seq_ad[i]), h[t0:t0 + ln],
                                                np.zeros_like(cp[i]), np.zeros_like(sp[i]), g)
            assert rel_l2(bf16_to_f64(got[1][0][t0:t0 + ln]), ref) <= 2e-2, i
            check_state(got[1][1][i], st, True)
        else:
            assert not np.any(got[1][1][i])
        t0 += ln


def test_captured_plan_prefill_and_steps(nhm):
    """A plan and a prefill of two layers in one graph, a step of decode, logits, selection and reorder in another: each
    replayed several times with other inputs, eager work in between, every output and state as the eager calls leave it."""
    from tests.gpu_util import dev, upload_params, zeros_ws
    from workloads import bf16_bits, e4m3_weight
    import workloads.synthetic as w
    g, R, K, V, T = SMALL, 3, 4, 1000, 64
    r = np.random.default_rng(1)
    S = R * K + 1
    layers = []
    for i in range(2):
        p = w.block_params(5, i, g)
        n_in = p["in_w"].shape[0]
        layers.append(dict(pd=upload_params(p, g), li=lora(nhm, adapters(r, 3, n_in, 256, 16)),
                           lo=lora(nhm, adapters(r, 3, 256, 512, 8)), sp=dev(w.ssm_pool(5, i, S, g=g)),
                           cp=dev(w.conv_pool(5, i, S, g=g)), out=torch.empty((T, 256), dtype=torch.int16, device="cuda"),
                           step=torch.empty((R * K, 256), dtype=torch.int16, device="cuda")))
    head_w, head_s = e4m3_weight(r, V, 256, std=0.1)
    head = nhm.Fp8Weight(dev(head_w), dev(head_s), dev(np.array([4 / 448], np.float32)))
    table = dev(bf16_bits(r.standard_normal((V, 256), dtype=np.float32)))
    ws = zeros_ws(max(nhm.prefill_lora_ws_layout(T, R, 16, g=g)["total"], nhm.decode_lora_ws_layout(R * K, 16, g)["total"]))
    head_ws = zeros_ws(nhm.fp8_linear_workspace_bytes(R * K, V, 256, nhm.NHM_BF16))
    pick_ws = zeros_ws(nhm.beam_select_workspace_bytes(R, K, V, K))
    lengths, past, req_ad = (torch.zeros(R, dtype=torch.int32, device="cuda") for _ in range(3))
    hidden = torch.zeros((T, 256), dtype=torch.int16, device="cuda")
    plan = nhm.BatchPlan(R, T)
    slots = dev(r.permutation(S)[:R * K].reshape(R, K).astype(np.int32))
    first = slots[:, 0].contiguous()
    rows = dev(bf16_bits(r.standard_normal((R * K, 256), dtype=np.float32)))
    cum = torch.zeros((R, K), device="cuda")
    logits = torch.empty((R * K, V), device="cuda")
    scores, parents = torch.empty((R, K), device="cuda"), torch.empty((R, K), dtype=torch.int32, device="cuda")
    tokens, new_slots = torch.empty_like(parents), torch.empty_like(parents)
    beam_ad = torch.zeros(R * K, dtype=torch.int32, device="cuda")

    def prefill():
        nhm.batch_plan(lengths, plan, past=past, adapters=req_ad)
        x = hidden
        for ly in layers:
            nhm.mixer_prefill_lora(ly["pd"], ly["li"], ly["lo"], plan.token_adapter, x, plan.cu_seqlens, first,
                                   plan.has_initial, ly["sp"], ly["cp"], ly["out"], ws)
            x = ly["out"]

    def step():
        nhm.fp8_linear(rows, head, out=logits, ws=head_ws, exact=True)
        nhm.beam_select(logits, cum, K, scores=scores, parents=parents, tokens=tokens, ws=pick_ws)
        nhm.beam_reorder(parents, slots, [ly["sp"] for ly in layers], [ly["cp"] for ly in layers], new_slots=new_slots, g=g)
        x = table[tokens.view(-1).long()]
        for ly in layers:
            nhm.mixer_decode_lora(ly["pd"], ly["li"], ly["lo"], beam_ad, x, new_slots.view(-1), ly["sp"], ly["cp"],
                                  ly["step"], ws)
            x = ly["step"]
        rows.copy_(x)
        slots.copy_(new_slots)
        cum.copy_(scores)

    state = [rows, slots, cum] + [ly[k] for ly in layers for k in ("sp", "cp")]
    results = state + [plan.cu_seqlens, plan.has_initial, plan.token_seq, plan.token_pos, plan.token_adapter, logits, scores,
                       parents, tokens, new_slots] + [ly[k] for ly in layers for k in ("out", "step")]
    graphs = []
    for f in (prefill, step):
        f()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f()
        graphs.append((f, graph))
    for turn in range(4):
        lengths.copy_(torch.from_numpy(r.integers(0, T // R + 1, R).astype(np.int32)))
        past.copy_(torch.from_numpy(r.integers(0, 2, R).astype(np.int32)))
        req_ad.copy_(torch.from_numpy(r.integers(-1, 3, R).astype(np.int32)))
        beam_ad.copy_(req_ad.repeat_interleave(K))
        hidden.copy_(dev(bf16_bits(r.standard_normal((T, 256), dtype=np.float32))))
        for f, graph in graphs:
            before = [t.clone() for t in state]
            f()
            torch.cuda.synchronize()
            want = [t.clone() for t in results]
            for t, b in zip(state, before):
                t.copy_(b)
            for t in results[len(state):]:
                t.fill_(1)
            ws.fill_(0xA5)
            graph.replay()
            torch.cuda.synchronize()
            for i in range(len(results)):
                if touched(f is step, i, len(state)):
                    assert torch.equal(results[i], want[i]), (turn, f.__name__, i)


def touched(is_step, i, states):
    """Whether a graph writes result i: the states, then the plan's five (prefill), the step's five, and each layer's
    prefill and step outputs in turn."""
    if i < states:
        return True
    i -= states
    if i < 10:
        return (i >= 5) == is_step
    return ((i - 10) % 2 == 1) == is_step
