"""Plain CPU oracle of the serving operators: adapters beside a W8A8 projection, beam selection,
state reorder, batch plan (test infrastructure only; float64 throughout).

The definitions are those of include/nhm_serving.h, evaluated in the plainest way: one row, one
candidate, one beam or one token at a time where that is fast enough."""
from __future__ import annotations

import numpy as np

from .nhm_oracle import (GEOMETRY, bf16_from_f64, bf16_to_f64, causal_conv1d_silu, dt_and_decay, e4m3_decode, fp8_linear,
                         gated_group_rmsnorm, layout, quantize_static, ssm_scan_sequential)

__all__ = ["fp8_linear_lora", "lora_bound", "mixer_sequence_lora", "beam_select", "beam_reorder", "batch_plan"]


def _lora_input(a, a_scale, codes):
    """(the codes the projection reads, the values the adapters read)."""
    if codes:
        return a, e4m3_decode(a) * np.float64(a_scale[0])
    return quantize_static(a, a_scale), bf16_to_f64(a)


def fp8_linear_lora(a, w_codes, w_scale, a_scale, lora_a, lora_b, lora_scale, row_adapter, codes=False):
    """float64 [m, n]: the projection of a (bf16 bits, or e4m3 codes) plus each row's adapter (bf16 bits
    [e, rank, k], [e, n, rank]; scale f32 [e] or None)."""
    q, x = _lora_input(a, a_scale, codes)
    out = fp8_linear(q, w_codes, w_scale, a_scale)
    for e in range(lora_a.shape[0]):
        rows = np.flatnonzero(row_adapter == e)
        if rows.size:
            s = 1.0 if lora_scale is None else np.float64(lora_scale[e])
            out[rows] += (x[rows] @ bf16_to_f64(lora_a[e]).T) @ bf16_to_f64(lora_b[e]).T * s
    return out


def lora_bound(a, w_codes, w_scale, a_scale, lora_a, lora_b, lora_scale, row_adapter, ref, codes=False, exact=True,
               f32=True):
    """The largest error the stated arithmetic allows, [m, n]:
    - the projection's sum: 2^-22 of the sum of |a w| where every product is summed in f32, 2^-16 on
      the e4m3 matrix instructions (the bars of the projection alone);
    - t = x A^T in f32: k / 32 + 64 additions and roundings of at most 2^-24 of the sum of |x A| each
      (a dot of 32 products per matrix instruction, then the partial sums), carried through |B|;
    - t as bf16 parts: 2^-25 of |t| for three (f32 output), 2^-17 for two, carried through |B|;
    - t B^T in f32: rank + 8 additions of at most 2^-24 of the sum of |t B|;
    - the sum of both and its scales: 2^-22 of the result, and half a bf16 step, 2^-8, for bf16."""
    q, x = _lora_input(a, a_scale, codes)
    k, rank = x.shape[1], lora_a.shape[1]
    S = np.abs(e4m3_decode(q)) @ np.abs(e4m3_decode(w_codes)).T * np.float64(a_scale[0])
    S *= np.asarray(w_scale, np.float64)[None, :]
    tol = (2.0 ** -22 if exact else 2.0 ** -16) * S + (2.0 ** -22 + (0 if f32 else 2.0 ** -8)) * np.abs(ref)
    for e in range(lora_a.shape[0]):
        rows = np.flatnonzero(row_adapter == e)
        if rows.size == 0:
            continue
        s = 1.0 if lora_scale is None else abs(np.float64(lora_scale[e]))
        A, B = bf16_to_f64(lora_a[e]), np.abs(bf16_to_f64(lora_b[e]))
        t_abs = np.abs(x[rows] @ A.T) * s
        t_sum = (np.abs(x[rows]) @ np.abs(A).T) * s
        tol[rows] += (k / 32 + 64) * 2.0 ** -24 * (t_sum @ B.T)
        tol[rows] += ((2.0 ** -25 if f32 else 2.0 ** -17) + (rank + 8) * 2.0 ** -24) * (t_abs @ B.T)
        tol[rows] += 2.0 ** -22 * (t_abs @ B.T)
    return tol


def mixer_sequence_lora(p, lora_in, lora_out, adapter, hidden, window, state, g=GEOMETRY):
    """One mixer block over one sequence, from a carried window and state, with adapters beside both
    projections (lora_*: (a, b, scale) or None; adapter int [T]): the stages of mixer_sequence with the adapters'
    part added to a projection before its one rounding to bf16. Without adapters it is mixer_sequence."""
    lay = layout(g)
    H, P, N, G = g["n_heads"], g["head_dim"], g["d_state"], g["n_groups"]
    T = hidden.shape[0]

    def project(x, w, ws, sa, lora):
        if lora is None:
            return fp8_linear(quantize_static(x, sa), w, ws, sa)
        return fp8_linear_lora(x, w, ws, sa, *lora, adapter)

    zx = bf16_from_f64(project(hidden, p["in_w"], p["in_w_scale"], p["in_a_scale"], lora_in))
    z = zx[:, lay["z_off"]:lay["z_off"] + lay["z_width"]]
    xbc = zx[:, lay["xbc_off"]:lay["xbc_off"] + lay["xbc_width"]]
    _, conv, new_window = causal_conv1d_silu(xbc, window, p["conv_w"], p["conv_b"])
    part = lambda o, n: bf16_to_f64(conv[:, lay[o]:lay[o] + lay[n]])  # noqa: E731
    dt, dA = dt_and_decay(zx[:, lay["dt_off"]:lay["dt_off"] + lay["dt_width"]], p["dt_bias"], p["A_log"])
    y, h = ssm_scan_sequential(part("x_off", "x_width").reshape(T, H, P), part("b_off", "b_width").reshape(T, G, N),
                               part("c_off", "c_width").reshape(T, G, N), dt, dA, p["D"],
                               np.asarray(state, np.float32).astype(np.float64))
    _, norm = gated_group_rmsnorm(bf16_from_f64(y.reshape(T, H * P)), z, p["norm_w"], G, g["rms_eps"])
    out = project(norm, p["out_w"], p["out_w_scale"], p["out_a_scale"], lora_out)
    return out, new_window, h.astype(np.float32)


def beam_select(logits, cum, n_cand, finished=None, eos=0):
    """(scores float64, parents int32, tokens int32, gap): logits float64 [groups, beams, vocab]. gap is the
    smallest difference between neighbouring scores of different beams among the candidates and the first one
    left out (0 differences, exact ties, aside): how far the order is from depending on rounding."""
    G, K, V = logits.shape
    scores = np.full((G, n_cand), -np.inf)
    parents = np.full((G, n_cand), -1, np.int32)
    tokens = np.full((G, n_cand), -1, np.int32)
    gap = np.inf
    for g in range(G):
        flat = np.full((K, V), -np.inf)
        for b in range(K):
            c = np.float64(cum[g, b])
            if finished is not None and finished[g, b]:
                flat[b, eos] = c
                continue
            x = np.where(np.isnan(logits[g, b]), -np.inf, logits[g, b])
            top = x.max()
            if top == -np.inf:
                continue
            d = np.full(V, -np.inf)
            d[x == top] = 0.0
            if top < np.inf:
                d = x - top
            with np.errstate(invalid="ignore"):
                flat[b] = c + (d - np.log(np.exp(d).sum()))
        f = flat.reshape(-1)
        f[np.isnan(f)] = -np.inf
        order = np.argsort(-f, kind="stable")
        order = order[f[order] > -np.inf]
        near = order[:n_cand + 1]
        for p, r in zip(near[:-1], near[1:]):
            if p // V != r // V and f[p] != f[r]:
                gap = min(gap, abs(f[p] - f[r]))
        for i, o in enumerate(order[:n_cand]):
            scores[g, i], parents[g, i], tokens[g, i] = f[o], o // V, o % V
    return scores, parents, tokens, gap


def beam_reorder(parents, slots, pools):
    """new_slots int32; pools (a list of arrays [n_slots, ...]) are updated in place."""
    G, K = parents.shape
    new = np.empty_like(slots)
    before = [p.copy() for p in pools]
    S = pools[0].shape[0]
    for g in range(G):
        par = [p if 0 <= p < K else -1 for p in parents[g].tolist()]
        firsts = {}
        for j, p in enumerate(par):
            if p >= 0 and p not in firsts:
                firsts[p] = j
        free = [slots[g, b] for b in range(K) if b not in firsts]
        for j, p in enumerate(par):
            if p >= 0 and firsts[p] == j:
                new[g, j] = slots[g, p]
                continue
            new[g, j] = free.pop(0)
            if p >= 0 and 0 <= slots[g, p] < S and 0 <= new[g, j] < S:
                for pool, old in zip(pools, before):
                    pool[new[g, j]] = old[slots[g, p]]
    return new


def batch_plan(lengths, n_tokens, past=None, adapters=None):
    n = len(lengths)
    cu = np.zeros(n + 1, np.int32)
    seq, pos, ad = (np.full(n_tokens, -1, np.int32) for _ in range(3))
    for i in range(n):
        cu[i + 1] = min(int(cu[i]) + max(int(lengths[i]), 0), n_tokens)
        r = np.arange(cu[i], cu[i + 1])
        seq[r] = i
        pos[r] = (0 if past is None else past[i]) + r - cu[i]
        ad[r] = -1 if adapters is None else adapters[i]
    has = np.zeros(n, np.int32) if past is None else (np.asarray(past) > 0).astype(np.int32)
    return dict(cu_seqlens=cu, has_initial=has, token_seq=seq, token_pos=pos, token_adapter=ad)
