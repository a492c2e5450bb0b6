"""The serving operators beside the mixer, as cases to time and to compare.

Four operators of one batch of requests over a state pool:

* ``lora``: an FP8 W8A8 projection with the low-rank adapters of many requests beside it;
* ``select``: beam search's selection over beams and vocabulary;
* ``reorder``: the recurrent states of the selected beams moved to their slots;
* ``plan``: the prefill's index tensors and the per-token adapter map from request lengths.

``run`` computes a case in its plain form (elementary torch operations) or, with ``own`` set,
through the framework's calls.
"""
import math

import numpy as np
import torch

own = False

# the mixer's projections and the square control of the linear sweep, [n, k]
IN_PROJ, OUT_PROJ, SQUARE = (10304, 2688), (2688, 4096), (4096, 4096)
LAYERS = 23


def listed():
    return [
        # one decode token of one adapted request: launch latency and the weight stream
        dict(name="lora_one_token", op="lora", m=1, n=IN_PROJ[0], k=IN_PROJ[1], rank=16, adapters=4, order="mixed",
             bare=0.0, codes=False, f32=False, exact=False),
        # a decode batch whose rows all have another adapter, the mixer's input projection
        dict(name="lora_decode_8", op="lora", m=8, n=IN_PROJ[0], k=IN_PROJ[1], rank=64, adapters=64, order="mixed",
             bare=0.1, codes=False, f32=False, exact=False),
        # a larger decode batch through the output projection, codes in and f32 out
        dict(name="lora_decode_61", op="lora", m=61, n=OUT_PROJ[0], k=OUT_PROJ[1], rank=32, adapters=32, order="mixed",
             bare=0.2, codes=True, f32=True, exact=True),
        # a short prefill: a few requests' tokens one after another, products summed in f32
        dict(name="lora_prefill_477", op="lora", m=477, n=IN_PROJ[0], k=IN_PROJ[1], rank=24, adapters=8, order="runs",
             bare=0.1, codes=False, f32=False, exact=True),
        # a long prefill of a few requests
        dict(name="lora_prefill_15360", op="lora", m=15360, n=IN_PROJ[0], k=IN_PROJ[1], rank=64, adapters=8,
             order="runs", bare=0.0, codes=False, f32=False, exact=False),
        # one request's beams
        dict(name="select_one", op="select", groups=1, beams=4, vocab=32000, cand=8, f32=False, finished=False,
             masked=False),
        # several requests, odd vocabulary, some beams finished, a mask over the vocabulary
        dict(name="select_odd", op="select", groups=8, beams=5, vocab=50257, cand=10, f32=True, finished=True,
             masked=True),
        # many requests, a large vocabulary
        dict(name="select_many", op="select", groups=64, beams=8, vocab=131072, cand=16, f32=False, finished=False,
             masked=False),
        # the states of a few beams of one layer, stored in bf16
        dict(name="reorder_one_layer", op="reorder", groups=2, beams=4, layers=1, heads=64, f32=False, copies=1),
        # every layer's f32 states of a batch of beams
        dict(name="reorder_all_layers", op="reorder", groups=6, beams=5, layers=LAYERS, heads=64, f32=True, copies=2),
        # a decode-like batch of short requests
        dict(name="plan_short", op="plan", seqs=17, tokens=512, past=True),
        # a packed batch of many requests
        dict(name="plan_long", op="plan", seqs=1021, tokens=131072, past=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["lora", "lora", "select", "reorder", "plan"])
    if op == "lora":
        if rng.random() < 0.6:
            n, k = rng.choice([IN_PROJ, OUT_PROJ, SQUARE])
        else:                              # other projections: any number of outputs
            n, k = log(64, 12000), 16 * log(16, 256)
        m = log(1, 15360)
        m = max(1, min(m, 15360 * IN_PROJ[0] * IN_PROJ[1] // (n * k)))
        rank = 8 * rng.choice([1, 2, 3, 4, 5, 8] if m > 2048 else [1, 2, 3, 4, 5, 8, 16])
        f32 = rng.random() < 0.3           # f32 outputs are for sums in f32
        return dict(op=op, m=m, n=n, k=k, rank=rank, adapters=log(1, 64),
                    order=rng.choice(["runs", "mixed"]) if m <= 512 else "runs", bare=rng.choice([0.0, 0.2]),
                    codes=rng.random() < 0.3, f32=f32, exact=f32 or rng.random() < 0.5)
    if op == "select":
        f32 = rng.random() < 0.4
        beams, vocab = rng.randint(1, 16), log(1000, 152000)
        most = 64 * 8 * 131072 // (2 if f32 else 1)
        groups = max(1, min(log(1, 64), most // (beams * vocab)))
        return dict(op=op, groups=groups, beams=beams, vocab=vocab, cand=log(1, 64), f32=f32,
                    finished=rng.random() < 0.3, masked=rng.random() < 0.3)
    if op == "reorder":
        beams, heads = rng.randint(2, 8), rng.choice([8, 64])
        groups, layers = rng.randint(1, 6), log(1, LAYERS)
        copies = rng.randint(0, beams - 1)
        while groups * copies > 12:
            copies -= 1
        return dict(op=op, groups=groups, beams=beams, layers=layers, heads=heads, f32=rng.random() < 0.5,
                    copies=copies)
    return dict(op=op, seqs=log(1, 1021), tokens=log(64, 131072), past=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _gens(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g, np.random.default_rng(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prepare_lora(c, seed):
    g, r = _gens(seed)
    m, n, k, rank, na = c["m"], c["n"], c["k"], c["rank"], c["adapters"]
    w = _randn(g, n, k) * 0.02
    w_scale = (w.abs().amax(dim=1) / 448.0).contiguous()
    wq = (w / w_scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    a_scale = torch.full((1,), 4.0 / 448.0, device="cuda")
    x = _randn(g, m, k).to(torch.bfloat16)
    if c["codes"]:
        x = (x.float() / a_scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    a = (_randn(g, na, rank, k) / math.sqrt(k)).to(torch.bfloat16)
    b = (_randn(g, na, n, rank) * 0.02).to(torch.bfloat16)
    scale = torch.from_numpy(r.choice([0.5, 1.0, 2.0], na).astype(np.float32)).cuda()
    if c["order"] == "mixed":
        ids = r.permutation(na)[np.arange(m) % na] if na >= m else r.integers(0, na, m)
        ids = np.where(r.random(m) < c["bare"], -1, ids)
    else:                                  # runs of tokens, one request after another
        parts = min(m, 1 + int(r.integers(2, 6)))
        cuts = np.sort(r.choice(np.arange(1, m), parts - 1, replace=False)) if parts > 1 else np.zeros(0, np.int64)
        who = np.where(r.random(parts) < c["bare"], -1, r.integers(0, na, parts))
        ids = np.repeat(who, np.diff(np.concatenate([[0], cuts, [m]])))
    ids = ids.astype(np.int32)
    s = dict(case=c, x=x, wq=wq, w_scale=w_scale, a_scale=a_scale, a=a, b=b, scale=scale,
             row_adapter=torch.from_numpy(ids).cuda(),
             rows={int(e): torch.from_numpy(np.nonzero(ids == e)[0]).cuda() for e in np.unique(ids) if e >= 0})
    if own:
        import fp8_w8a8_linear_amd as nhm
        s["weight"] = nhm.Fp8Weight(wq, w_scale, a_scale)
        s["lora"] = nhm.Lora(a, b, scale)
        s["out"] = torch.empty((m, n), dtype=torch.float32 if c["f32"] else torch.bfloat16, device="cuda")
        t = nhm.NHM_E4M3 if c["codes"] else nhm.NHM_BF16
        s["ws"] = torch.empty(nhm.fp8_linear_lora_workspace_bytes(m, n, k, t, rank), dtype=torch.uint8, device="cuda")
    return s


def _prepare_select(c, seed):
    g, r = _gens(seed)
    G, K, V = c["groups"], c["beams"], c["vocab"]
    logits = _randn(g, G * K, V) * 3.0
    if c["masked"]:                        # a constrained step: most of the vocabulary is not allowed
        logits.masked_fill_(torch.rand(G * K, V, generator=g, device="cuda") < 0.7, -math.inf)
        logits[G * K // 2] = -math.inf     # and one beam has nothing left
    logits = logits.to(torch.float32 if c["f32"] else torch.bfloat16)
    cum = torch.from_numpy((-20.0 * r.random((G, K))).astype(np.float32)).cuda()
    finished = torch.from_numpy((r.random((G, K)) < 0.25).astype(np.int32)).cuda() if c["finished"] else None
    s = dict(case=c, logits=logits, cum=cum, finished=finished, eos=int(r.integers(0, V)))
    if own:
        import fp8_w8a8_linear_amd as nhm
        n = c["cand"]
        s["scores"] = torch.empty((G, n), dtype=torch.float32, device="cuda")
        s["parents"] = torch.empty((G, n), dtype=torch.int32, device="cuda")
        s["tokens"] = torch.empty((G, n), dtype=torch.int32, device="cuda")
        s["ws"] = torch.empty(nhm.beam_select_workspace_bytes(G, K, V, n), dtype=torch.uint8, device="cuda")
    return s


def _geometry(c):
    groups = 8 if c["heads"] == 64 else 2
    return dict(hidden=2688 if c["heads"] == 64 else 256, n_heads=c["heads"], head_dim=64, d_state=128,
                n_groups=groups, conv_width=4, rms_eps=1e-5)


def _prepare_reorder(c, seed):
    g, r = _gens(seed)
    G, K, geo = c["groups"], c["beams"], _geometry(c)
    slots_total = G * K + 2
    conv_dim = geo["n_heads"] * 64 + 2 * geo["n_groups"] * 128
    dt = torch.float32 if c["f32"] else torch.bfloat16
    ssm = [(_randn(g, slots_total, geo["n_heads"], 64, 128) * 0.1).to(dt) for _ in range(c["layers"])]
    conv = [_randn(g, slots_total, 3, conv_dim).to(torch.bfloat16) for _ in range(c["layers"])]
    slots = r.permutation(slots_total)[:G * K].reshape(G, K).astype(np.int32)
    parents = np.empty((G, K), np.int32)
    for i in range(G):                     # `copies` beams share a parent with an earlier one
        kept = r.permutation(K)[:K - c["copies"]]
        parents[i] = r.permutation(np.concatenate([kept, r.choice(kept, c["copies"])]))
    s = dict(case=c, ssm=ssm, conv=conv, slots=torch.from_numpy(slots).cuda(),
             parents=torch.from_numpy(parents).cuda())
    if own:
        s["new_slots"] = torch.empty((G, K), dtype=torch.int32, device="cuda")
        s["geometry"] = geo
    return s


def _prepare_plan(c, seed):
    _, r = _gens(seed)
    n, T = c["seqs"], c["tokens"]
    used = T - T // 16                     # the batch's token buffer is a little larger than the batch
    cuts = np.sort(r.integers(0, used + 1, n - 1))
    lengths = np.diff(np.concatenate([[0], cuts, [used]])).astype(np.int32)
    past = np.where(r.random(n) < 0.5, r.integers(1, 100000, n), 0).astype(np.int32)
    adapters = r.integers(-1, 64, n).astype(np.int32)
    s = dict(case=c, lengths=torch.from_numpy(lengths).cuda(), adapters=torch.from_numpy(adapters).cuda(),
             past=torch.from_numpy(past).cuda() if c["past"] else None)
    if own:
        import fp8_w8a8_linear_amd as nhm
        s["plan"] = nhm.BatchPlan(n, T, device="cuda")
    return s


def prepare(case, seed):
    return {"lora": _prepare_lora, "select": _prepare_select, "reorder": _prepare_reorder,
            "plan": _prepare_plan}[case["op"]](case, seed)


# ---------------------------------------------------------------- the plain forms and the calls

def _plain_lora(s):
    c = s["case"]
    if c["codes"]:
        q = s["x"].view(torch.float8_e4m3fn).float()
        x = q * s["a_scale"]
    else:
        x = s["x"].float()
        q = (x / s["a_scale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    out = (q @ s["wq"].view(torch.float8_e4m3fn).float().T) * s["a_scale"] * s["w_scale"]
    for e, rows in s["rows"].items():
        t = (x[rows] @ s["a"][e].float().T) * s["scale"][e]
        out[rows] += t @ s["b"][e].float().T
    return out if c["f32"] else out.to(torch.bfloat16)


def _plain_select(s):
    c = s["case"]
    G, K, V, n = c["groups"], c["beams"], c["vocab"], c["cand"]
    x = s["logits"].double()               # scores of different beams lie close together
    x = torch.where(torch.isnan(x), -math.inf, x)
    top = x.amax(dim=1, keepdim=True)
    d = torch.where(x == top, 0.0, x - top)
    logp = d - d.exp().sum(dim=1, keepdim=True).log()
    logp = torch.where(x == -math.inf, -math.inf, logp).view(G, K, V)
    if s["finished"] is not None:          # a finished beam goes on as it is, by its end token alone
        stop = torch.full((V,), -math.inf, dtype=torch.float64, device=x.device)
        stop[s["eos"]] = 0.0
        logp = torch.where((s["finished"] != 0)[:, :, None], stop, logp)
    score = (s["cum"].double()[:, :, None] + logp).view(G, K * V)
    best, flat = torch.sort(score, dim=1, descending=True, stable=True)
    best, flat = best[:, :n], flat[:, :n]
    if n > K * V:
        raise ValueError("more candidates than beams x vocabulary")
    none = best == -math.inf
    parents = torch.where(none, -1, flat // V).to(torch.int32)
    tokens = torch.where(none, -1, flat % V).to(torch.int32)
    return dict(scores=best.float(), parents=parents, tokens=tokens)


def _plain_reorder(s):
    parents, slots = s["parents"].long(), s["slots"].long()
    K = parents.shape[1]
    j = torch.arange(K, device=parents.device)
    has = parents >= 0
    same = (parents[:, :, None] == parents[:, None, :]) & (j[None, :] < j[:, None])
    first = has & ~same.any(dim=2)
    used = (parents[:, :, None] == j).any(dim=1)
    free = torch.argsort(used.to(torch.int32), dim=1, stable=True)      # beams without a child first
    rank = (torch.cumsum((~first).long(), dim=1) - 1).clamp(min=0)
    src = slots.gather(1, parents.clamp(min=0))
    new = torch.where(first, src, slots.gather(1, free.gather(1, rank)))
    src = torch.where(has, src, new).view(-1)
    for pool in s["ssm"] + s["conv"]:
        pool[new.view(-1)] = pool[src]
    return dict(new_slots=new.to(torch.int32), ssm=s["ssm"], conv=s["conv"])


def _plain_plan(s):
    T = s["case"]["tokens"]
    lengths, n = s["lengths"], s["lengths"].shape[0]
    cu = torch.zeros(n + 1, dtype=torch.int64, device=lengths.device)
    cu[1:] = torch.cumsum(lengths.long(), dim=0)
    t = torch.arange(T, device=lengths.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    real = seq < n
    at = seq.clamp(max=n - 1)
    past = s["past"] if s["past"] is not None else torch.zeros_like(lengths)
    pos = torch.where(real, past[at] + t - cu[at], -1)
    return dict(cu_seqlens=cu.to(torch.int32), has_initial=(past > 0).to(torch.int32),
                token_seq=torch.where(real, seq, -1).to(torch.int32), token_pos=pos.to(torch.int32),
                token_adapter=torch.where(real, s["adapters"][at], -1).to(torch.int32))


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"lora": _plain_lora, "select": _plain_select, "reorder": _plain_reorder,
                "plan": _plain_plan}[c["op"]](s)
    import fp8_w8a8_linear_amd as nhm
    if c["op"] == "lora":
        return nhm.fp8_linear_lora(s["x"], s["weight"], s["lora"], s["row_adapter"], out=s["out"], ws=s["ws"],
                                   exact=c["exact"])
    if c["op"] == "select":
        nhm.beam_select(s["logits"], s["cum"], c["cand"], finished=s["finished"], eos=s["eos"], scores=s["scores"],
                        parents=s["parents"], tokens=s["tokens"], ws=s["ws"])
        return dict(scores=s["scores"], parents=s["parents"], tokens=s["tokens"])
    if c["op"] == "reorder":
        nhm.beam_reorder(s["parents"], s["slots"], s["ssm"], s["conv"], new_slots=s["new_slots"], g=s["geometry"])
        return dict(new_slots=s["new_slots"], ssm=s["ssm"], conv=s["conv"])
    p = nhm.batch_plan(s["lengths"], s["plan"], past=s["past"], adapters=s["adapters"])
    return dict(cu_seqlens=p.cu_seqlens, has_initial=p.has_initial, token_seq=p.token_seq, token_pos=p.token_pos,
                token_adapter=p.token_adapter)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "lora":
        m, n, k, r = c["m"], c["n"], c["k"], c["rank"]
        used = min(m, c["adapters"]) if c["order"] == "mixed" else min(m, c["adapters"], 4)
        b = (m * k * (1 if c["codes"] else 2) + n * k + 4 * n + 4 * m + used * r * (n + k) * 2
             + m * n * (4 if c["f32"] else 2))
        return {"bytes": b, "flops": 2 * m * n * k + 2 * m * r * (n + k)}
    if c["op"] == "select":
        e = c["groups"] * c["beams"] * c["vocab"]
        return {"bytes": e * (4 if c["f32"] else 2) + c["groups"] * (8 * c["beams"] + 12 * c["cand"]), "flops": 4 * e}
    if c["op"] == "reorder":
        geo = _geometry(c)
        row = geo["n_heads"] * 64 * 128 * (4 if c["f32"] else 2) + 3 * (geo["n_heads"] * 64 + geo["n_groups"] * 256) * 2
        return {"bytes": 2 * c["groups"] * c["copies"] * c["layers"] * row + 12 * c["groups"] * c["beams"], "flops": 0}
    return {"bytes": 20 * c["seqs"] + 12 * c["tokens"], "flops": 2 * c["tokens"]}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_lora(c, s):
    f8 = torch.float8_e4m3fn
    sa = s["a_scale"].double()
    if c["codes"]:
        q = s["x"].view(f8).to(torch.float64)
        x = q * sa
    else:
        x = s["x"].to(torch.float64)
        # the code is defined on the f32 quotient
        q = torch.clamp(s["x"].float() / s["a_scale"], -448.0, 448.0).to(f8).to(torch.float64)
    y = torch.matmul(q, s["wq"].view(f8).to(torch.float64).t().contiguous()).mul_(sa * s["w_scale"].double())
    ids = s["row_adapter"].cpu().numpy()
    for e in range(c["adapters"]):
        rows = np.flatnonzero(ids == e)
        if rows.size == 0:
            continue
        rows = torch.from_numpy(rows).cuda()
        low = torch.matmul(x[rows], s["a"][e].double().t().contiguous())
        y[rows] = y[rows] + torch.matmul(low, s["b"][e].double().t().contiguous()) * s["scale"][e].double()
    return y


def _exact_select(c, s):
    G, K, V, n = c["groups"], c["beams"], c["vocab"], c["cand"]
    cum = s["cum"].double().cpu().numpy()
    fin = np.zeros((G, K), bool) if s["finished"] is None else s["finished"].cpu().numpy() != 0
    scores = np.full((G, n), -np.inf)
    parents = np.full((G, n), -1, np.int32)
    tokens = np.full((G, n), -1, np.int32)
    for g in range(G):
        rows = s["logits"][g * K:(g + 1) * K].float().cpu().numpy()
        cand = []
        for b in range(K):
            if fin[g, b]:
                cand.append((cum[g, b], b, s["eos"]))
                continue
            v = np.flatnonzero(rows[b] > -np.inf)
            if v.size == 0:
                continue
            x = rows[b][v].astype(np.float64)
            hi = x.max()
            lse = hi + np.log(np.exp(x - hi).sum())
            if v.size > n:                 # the row's own best, every tie of the last one among them
                last = -np.partition(-x, n - 1)[n - 1]
                at = np.flatnonzero(x >= last)
                v, x = v[at], x[at]
            cand += [(cum[g, b] + (xi - lse), b, int(vi)) for xi, vi in zip(x, v)]
        cand.sort(key=lambda t: (-t[0], t[1], t[2]))
        for i, (sc, b, v) in enumerate([t for t in cand if t[0] > -np.inf][:n]):
            scores[g, i], parents[g, i], tokens[g, i] = sc, b, v
    return dict(scores=torch.from_numpy(scores), parents=torch.from_numpy(parents), tokens=torch.from_numpy(tokens))


def _exact_reorder(c, s):
    slots, parents = s["slots"].cpu().numpy(), s["parents"].cpu().numpy()
    new = np.empty_like(slots)
    moves = []
    for g in range(c["groups"]):
        taken, later = set(), []
        for j, p in enumerate(parents[g]):
            if p >= 0 and p not in taken:
                taken.add(p)
                new[g, j] = slots[g, p]
            else:
                later.append(j)
        free = [slots[g, b] for b in range(c["beams"]) if b not in taken]
        for j, to in zip(later, free):
            new[g, j] = to
            if parents[g, j] >= 0:
                moves.append((int(slots[g, parents[g, j]]), int(to)))
    for pool in s["ssm"] + s["conv"]:
        for src, to in moves:
            pool[to] = pool[src]
    return dict(new_slots=torch.from_numpy(new), ssm=s["ssm"], conv=s["conv"])


def _exact_plan(c, s):
    lengths, adapters = s["lengths"].cpu().numpy(), s["adapters"].cpu().numpy()
    past = s["past"].cpu().numpy() if s["past"] is not None else np.zeros(c["seqs"], np.int32)
    T = c["tokens"]
    cu = np.zeros(c["seqs"] + 1, np.int32)
    seq, pos, ad = (np.full(T, -1, np.int32) for _ in range(3))
    for i, ln in enumerate(lengths):
        cu[i + 1] = cu[i] + ln
        seq[cu[i]:cu[i + 1]] = i
        pos[cu[i]:cu[i + 1]] = past[i] + np.arange(ln)
        ad[cu[i]:cu[i + 1]] = adapters[i]
    out = dict(cu_seqlens=cu, has_initial=(past > 0).astype(np.int32), token_seq=seq, token_pos=pos, token_adapter=ad)
    return {k: torch.from_numpy(v) for k, v in out.items()}


def exact(case, seed):
    f = {"lora": _exact_lora, "select": _exact_select, "reorder": _exact_reorder, "plan": _exact_plan}[case["op"]]
    return f(case, prepare(case, seed))
