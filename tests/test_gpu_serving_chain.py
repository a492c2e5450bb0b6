"""The serving operators together on the GPU, as a server runs them: the mixer with adapters against the oracle, and
one batch of requests from its plan through prefill, beam search steps and state reorders."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import serving_oracle as so  # noqa: E402

SMALL = dict(hidden=256, n_heads=8, head_dim=64, d_state=128, n_groups=2, conv_width=4, rms_eps=1e-5)


@pytest.fixture(scope="module")
def nhm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_w8a8_linear_amd as m
    return m


def adapters(r, e, n, k, rank, scaled=True):
    from workloads import bf16_bits
    a = bf16_bits(r.standard_normal((e, rank, k), dtype=np.float32) / np.sqrt(k))
    b = bf16_bits(r.standard_normal((e, n, rank), dtype=np.float32) * 0.05)
    return a, b, r.choice([0.5, 1.0], e).astype(np.float32) if scaled else None


def lora(nhm, ad):
    from tests.gpu_util import dev
    return nhm.Lora(dev(ad[0]), dev(ad[1]), None if ad[2] is None else dev(ad[2]))


def block(nhm, g, seed, S, T, e=5, rank=(24, 8)):
    """(oracle parameters, device parameters, adapters of both projections, hidden, pools)."""
    import workloads.synthetic as w
    from tests.gpu_util import upload_params
    r = np.random.default_rng(seed)
    p = w.block_params(4, seed, g)
    n_in, inner = p["in_w"].shape[0], p["out_w"].shape[1]
    ai = adapters(r, e, n_in, g["hidden"], rank[0])
    ao = adapters(r, e, g["hidden"], inner, rank[1], scaled=False)
    return p, upload_params(p, g), ai, ao, w.hidden(4, T, g, extra=seed), w.ssm_pool(4, seed, S, g=g), w.conv_pool(4, seed, S, g=g)


def flip_tol(g):
    """The block tolerance, max |d| <= 2e-2 RMS, is what one code of the norm output on the other side of a step moves a
    row of the 4,096-channel geometry by: a step of 32 a_scale = 0.29 times the largest |W w_scale| against an
    output RMS that grows with the square root of the channels summed (the weights' spread is the same). With 512
    channels the same flip is sqrt(4096 / 512) = 2.83 times as much of the RMS."""
    return 2e-2 * np.sqrt(4096 / (g["n_heads"] * g["head_dim"]))


def check_block(nhm, g, got_bits, ref, p, ao, ids, norm_bits, exact=True):
    """The output against the oracle's block, and, with no flips in the way, against the oracle's out_proj with adapters
    of the norm output that the call left in its workspace."""
    from oracle import bf16_to_f64
    from tests.gpu_util import rel_max
    got = bf16_to_f64(got_bits)
    err = rel_max(got, ref)
    assert err <= flip_tol(g), err
    own = so.fp8_linear_lora(norm_bits, p["out_w"], p["out_w_scale"], p["out_a_scale"], *ao, ids)
    tol = so.lora_bound(norm_bits, p["out_w"], p["out_w_scale"], p["out_a_scale"], *ao, ids, own, exact=exact, f32=False)
    assert np.all(np.abs(got - own) <= tol)
    return err


@pytest.mark.parametrize("B,geom", [(1, "full"), (5, "full"), (20, "small"), (33, "small"), (70, "small")])
def test_decode_with_adapters(nhm, B, geom):
    from tests.gpu_util import dev, host, rel_l2, ws_region, zeros_ws
    g = nhm.GEOMETRY if geom == "full" else SMALL
    S = B + 2
    print(f"decode with adapters B={B} {geom}", flush=True)
    p, pd, ai, ao, h, sp, cp = block(nhm, g, B, S, B)
    r = np.random.default_rng(B)
    slots = r.permutation(S)[:B].astype(np.int32)
    ids = r.integers(-1, 5, B).astype(np.int32)
    if B > 2:
        slots[1] = -1                                    # a padded row, with an adapter
        ids[1] = 2
    spd, cpd = dev(sp), dev(cp)
    out = torch.full((B, g["hidden"]), 0x5555, dtype=torch.int16, device="cuda")
    lay = nhm.decode_lora_ws_layout(B, 24, g)
    ws = zeros_ws(lay["total"])
    nhm.mixer_decode_lora(pd, lora(nhm, ai), lora(nhm, ao), dev(ids), dev(h), dev(slots), spd, cpd, out, ws)
    torch.cuda.synchronize()
    ref = np.zeros((B, g["hidden"]))
    for b in range(B):
        s = slots[b]
        if s >= 0:
            o, cp[s], sp[s] = so.mixer_sequence_lora(p, ai, ao, ids[b:b + 1], h[b:b + 1], cp[s], sp[s], g)
            ref[b] = o[0]
    got = host(out)
    if B > 2:
        assert np.all(got[1] == 0)
    inner = g["n_heads"] * 64
    norm = ws_region(ws, lay["norm"], B * inner, np.uint16).reshape(B, inner)
    err = check_block(nhm, g, got, ref, p, ao, ids, norm, exact=B <= 32)
    assert np.all(rel_l2(host(spd, np.float32), sp) <= 1e-3)
    assert rel_l2(host(cpd).astype(np.float64), cp.astype(np.float64)) <= 1e-2
    print(f"  end to end {err:.4f}")


def test_decode_adapters_on_one_projection_or_none(nhm):
    """NULL sets: the projections as without; rows without an adapter: the block's own output, bit for bit."""
    from tests.gpu_util import dev, host, zeros_ws
    B, S = 6, 8
    p, pd, ai, ao, h, sp, cp = block(nhm, nhm.GEOMETRY, 3, S, B)
    slots = dev(np.arange(1, B + 1, dtype=np.int32))
    hd = dev(h)

    def run(li, lo, ids):
        spd, cpd = dev(sp), dev(cp)
        out = torch.empty((B, 2688), dtype=torch.int16, device="cuda")
        ws = zeros_ws(nhm.decode_lora_ws_layout(B, 24)["total"])
        if li is None and lo is None and ids is None:
            nhm.mixer_decode(pd, hd, slots, spd, cpd, out, ws)
        else:
            nhm.mixer_decode_lora(pd, li, lo, ids, hd, slots, spd, cpd, out, ws)
        torch.cuda.synchronize()
        return host(out), host(spd, np.float32), host(cpd)

    base = run(None, None, None)
    li, lo = lora(nhm, ai), lora(nhm, ao)
    none = dev(np.full(B, -1, np.int32))
    for got in (run(li, lo, none), run(None, None, none), run(li, None, none), run(None, lo, none)):
        assert all(np.array_equal(a, b) for a, b in zip(got, base))
    ids = np.array([-1, 0, -1, 3, -1, -1], np.int32)
    got = run(li, lo, dev(ids))
    assert np.array_equal(got[0][ids < 0], base[0][ids < 0]) and not np.array_equal(got[0][ids >= 0], base[0][ids >= 0])
    only_out = run(None, lo, dev(ids))
    assert np.array_equal(only_out[1], base[1]) and not np.array_equal(only_out[0], base[0])   # in_proj untouched


@pytest.mark.parametrize("lengths,geom", [([5, 40, 1, 0, 17], "small"), ([130, 3, 97], "small"), ([19], "full")])
def test_prefill_with_adapters(nhm, lengths, geom):
    from tests.gpu_util import dev, host, rel_l2, rel_max, ws_region, zeros_ws
    from oracle import bf16_to_f64
    g = nhm.GEOMETRY if geom == "full" else SMALL
    n, T = len(lengths), sum(lengths)
    print(f"prefill with adapters {lengths} {geom}", flush=True)
    p, pd, ai, ao, h, sp, cp = block(nhm, g, 50 + T, n + 1, T)
    seq_ad = np.arange(n, dtype=np.int32) - 1
    past = np.arange(n, dtype=np.int32) % 2
    slots = np.arange(n, dtype=np.int32)[::-1].copy()
    plan = nhm.batch_plan(dev(np.array(lengths, np.int32)), nhm.BatchPlan(n, T), past=dev(past), adapters=dev(seq_ad))
    spd, cpd = dev(sp), dev(cp)
    out = torch.empty((T, g["hidden"]), dtype=torch.int16, device="cuda")
    lay = nhm.prefill_lora_ws_layout(T, n, 24, g=g)
    ws = zeros_ws(lay["total"])
    nhm.mixer_prefill_lora(pd, lora(nhm, ai), lora(nhm, ao), plan.token_adapter, dev(h), plan.cu_seqlens, dev(slots),
                           plan.has_initial, spd, cpd, out, ws)
    torch.cuda.synchronize()
    ref = np.zeros((T, g["hidden"]))
    t0 = 0
    for i, ln in enumerate(lengths):
        s = slots[i]
        win, st = (cp[s], sp[s]) if past[i] else (np.zeros_like(cp[s]), np.zeros_like(sp[s]))
        if ln:
            ref[t0:t0 + ln], cp[s], sp[s] = so.mixer_sequence_lora(p, ai, ao, np.full(ln, seq_ad[i]), h[t0:t0 + ln], win, st, g)
        else:
            cp[s], sp[s] = win, st
        t0 += ln
    got = bf16_to_f64(host(out))
    inner = g["n_heads"] * 64
    norm = ws_region(ws, lay["norm"], T * inner, np.uint16).reshape(T, inner)
    check_block(nhm, g, host(out), ref, p, ao, np.repeat(seq_ad, lengths), norm, exact=T <= 16)
    assert rel_l2(got, ref) <= 2e-2
    assert rel_l2(host(spd, np.float32), sp) <= 1e-3
    print(f"  end to end {rel_max(got, ref):.4f}, rel l2 {rel_l2(got, ref):.5f}")


def test_requests_from_plan_to_beams(nhm):
    """Two requests with an adapter each: plan, prefill, then three steps of four beams each: logits from the block
    output by an f32 projection, selection, reorder of two layers' states, the next token's input, decode. Every step's
    selection is checked against the oracle's on the same logits, and the states and outputs against
    sequences that are followed one by one."""
    from oracle import bf16_to_f64
    from tests.gpu_util import dev, host, rel_l2, upload_params, zeros_ws
    from workloads import bf16_bits, e4m3_weight
    import workloads.synthetic as w
    g, R, K, V, e = SMALL, 2, 4, 1000, 3
    r = np.random.default_rng(0)
    lengths, req_ad = np.array([9, 23], np.int32), np.array([2, -1], np.int32)
    T, S = int(lengths.sum()), R * K + 1
    layers = []
    for i in range(2):
        p = w.block_params(5, i, g)
        ad = (adapters(r, e, p["in_w"].shape[0], 256, 16), adapters(r, e, 256, 512, 8))
        layers.append(dict(p=p, pd=upload_params(p, g), ad=ad, li=lora(nhm, ad[0]), lo=lora(nhm, ad[1]),
                           sp=w.ssm_pool(5, i, S, g=g), cp=w.conv_pool(5, i, S, g=g)))
    for ly in layers:
        ly["spd"], ly["cpd"] = dev(ly["sp"]), dev(ly["cp"])
    head_w, head_s = e4m3_weight(r, V, 256, std=0.1)
    head = nhm.Fp8Weight(dev(head_w), dev(head_s), dev(np.array([4 / 448], np.float32)))
    table = bf16_bits(r.standard_normal((V, 256), dtype=np.float32))
    table_d = dev(table)
    prompt = r.integers(0, V, T)
    lora_ws = zeros_ws(max(nhm.prefill_lora_ws_layout(T, R, 16, g=g)["total"], nhm.decode_lora_ws_layout(R * K, 16, g)["total"]))

    # prefill, into each request's first slot
    plan = nhm.batch_plan(dev(lengths), nhm.BatchPlan(R, T), adapters=dev(req_ad))
    slots = r.permutation(S)[:R * K].reshape(R, K).astype(np.int32)
    first = dev(np.ascontiguousarray(slots[:, 0]))
    x = table_d[torch.from_numpy(prompt).cuda()]
    for ly in layers:
        out = torch.empty((T, 256), dtype=torch.int16, device="cuda")
        nhm.mixer_prefill_lora(ly["pd"], ly["li"], ly["lo"], plan.token_adapter, x, plan.cu_seqlens, first, plan.has_initial,
                               ly["spd"], ly["cpd"], out, lora_ws)
        x = out
    last = x[(plan.cu_seqlens[1:] - 1).long()].contiguous()

    # the oracle follows each beam as a sequence of its own: (windows and states per layer)
    def follow(tokens, state, ad):
        hcur = table[np.array(tokens)]
        new = []
        for ly, (win, st) in zip(layers, state):
            o, win, st = so.mixer_sequence_lora(ly["p"], *ly["ad"], np.full(len(tokens), ad), hcur, win, st, g)
            hcur = bf16_bits(o)
            new.append((win, st))
        return hcur[-1], new

    zero = [(np.zeros_like(ly["cp"][0]), np.zeros_like(ly["sp"][0])) for ly in layers]
    t0, beams, outs = 0, [], []
    for i, ln in enumerate(lengths):
        o, st = follow(prompt[t0:t0 + ln], zero, req_ad[i])
        beams.append([st] * K)
        outs.append(o)
        t0 += ln
    assert rel_l2(bf16_to_f64(host(last)), bf16_to_f64(np.stack(outs))) <= 2e-2

    cum = torch.full((R, K), float("-inf"), device="cuda")
    cum[:, 0] = 0.0                                       # one beam each at first
    slots_d = dev(slots)
    rows = torch.zeros((R * K, 256), dtype=torch.int16, device="cuda")
    rows[::K] = last
    beam_ad = dev(np.repeat(req_ad, K).astype(np.int32))
    for step in range(3):
        logits = nhm.fp8_linear(rows, head, out_type=nhm.NHM_F32, exact=True)
        scores, parents, tokens = nhm.beam_select(logits, cum, K)
        new_slots = nhm.beam_reorder(parents, slots_d, [ly["spd"] for ly in layers], [ly["cpd"] for ly in layers], g=g)
        x = table_d[tokens.view(-1).long()]
        for ly in layers:
            out = torch.empty((R * K, 256), dtype=torch.int16, device="cuda")
            nhm.mixer_decode_lora(ly["pd"], ly["li"], ly["lo"], beam_ad, x, new_slots.view(-1), ly["spd"], ly["cpd"], out, lora_ws)
            x = out
        torch.cuda.synchronize()
        lg = logits.cpu().numpy().astype(np.float64).reshape(R, K, V)
        s, pr, tk, gap = so.beam_select(lg, cum.cpu().numpy(), K)
        assert gap > 1e-6 and np.array_equal(parents.cpu().numpy(), pr) and np.array_equal(tokens.cpu().numpy(), tk), step
        ns = new_slots.cpu().numpy()
        assert np.array_equal(np.sort(ns, axis=1), np.sort(slots, axis=1)), step
        got = bf16_to_f64(host(x)).reshape(R, K, 256)
        new_beams = []
        for i in range(R):
            row = []
            for j in range(K):
                o, st = follow([tk[i, j]], beams[i][pr[i, j]], req_ad[i])
                row.append(st)
                ref = bf16_to_f64(o)
                assert rel_l2(got[i, j], ref) <= 2e-2, (step, i, j)
                for ly, (_, sr) in zip(layers, st):
                    assert rel_l2(ly["spd"][int(ns[i, j])].cpu().numpy(), sr) <= 5e-3, (step, i, j)
            new_beams.append(row)
        beams, slots, slots_d, cum, rows = new_beams, ns, new_slots, scores, x


def test_mixer_binding_refuses_other_tensors(nhm):
    """The mixer calls with adapters check their tensors ahead of any launch."""
    from tests.gpu_util import dev
    p, P, ai, ao, h, ssm, conv = block(nhm, SMALL, 3, 4, 4)
    li, lo = lora(nhm, ai), lora(nhm, ao)
    x, ssm, conv = dev(h), dev(ssm), dev(conv)
    ids, slots = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.arange(4, dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 7)
    ws = torch.empty(nhm.decode_lora_ws_layout(4, 24, SMALL)["total"], dtype=torch.uint8, device="cuda")
    good = dict(lora_in=li, lora_out=lo, row_adapter=ids, hidden=x, slot_idx=slots, ssm_pool=ssm, conv_pool=conv, out=out, ws=ws)
    for bad, error in [(dict(lora_in=lo), ValueError), (dict(lora_out=li), ValueError), (dict(row_adapter=ids[:3]), ValueError),
                       (dict(row_adapter=ids.long()), TypeError), (dict(slot_idx=slots[:3]), ValueError),
                       (dict(conv_pool=conv[:3]), ValueError), (dict(ssm_pool=ssm.double()), TypeError),
                       (dict(out=out[:3]), ValueError), (dict(hidden=x[:, :128].contiguous()), ValueError),
                       (dict(hidden=x.cpu()), TypeError), (dict(ws=ws[:1024]), nhm.NhmError),
                       (dict(row_adapter=None), nhm.NhmError)]:
        with pytest.raises(error):
            nhm.mixer_decode_lora(P, **{**good, **bad})
    torch.cuda.synchronize()
    assert bool((out == 7).all())
    nhm.mixer_decode_lora(P, **good)
    torch.cuda.synchronize()
