"""CPU pins of oracle/layer_oracle.py against forms that are not the oracle's."""
import numpy as np
import torch

from oracle import layer_oracle as lo


def test_mxfp4_codes_by_thresholds():
    """Codes against comparisons with the midpoints, on magnitudes that hit them all; scales against the definition."""
    r = np.random.default_rng(0)
    x = r.normal(size=(64, 96)) * np.exp2(r.integers(-40, 40, (64, 1)))
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x[0, :7], x[0, 7], x[0, 8:32] = mids, 4.0, 0.0                       # amax 5: scale 1
    x[1, :7], x[1, 7], x[1, 8:32] = -mids * 2.0 ** -30, 7.9 * 2.0 ** -30, 0.0
    code, scale = lo.mxfp4_quantize(x)
    assert scale[0, 0] == 127 and scale[1, 0] == 97
    assert code[0, :8].tolist() == [0, 2, 2, 4, 4, 6, 6, 6] and code[1, :8].tolist() == [8, 10, 10, 12, 12, 14, 14, 7]
    v = np.abs(x) / np.repeat(2.0 ** (scale.astype(float) - 127), 32, axis=1)
    want = sum(((v > m) if i % 2 == 0 else (v >= m)).astype(int) for i, m in enumerate(mids))
    assert np.array_equal(code & 7, want)
    amax = np.abs(x).reshape(64, 3, 32).max(axis=2)
    s = 2.0 ** (scale.astype(float) - 127)
    assert np.all((amax >= 4 * s) & (amax < 8 * s))


def test_mxfp4_special_blocks():
    x = np.zeros((1, 160))
    x[0, 1] = -0.0
    x[0, 40], x[0, 70], x[0, 100] = np.nan, np.inf, 2.0 ** -140
    x[0, 128] = 3.3e38
    code, scale = lo.mxfp4_quantize(x)
    assert scale[0].tolist() == [0, 255, 255, 0, 252] and code[0, 1] == 8
    v = lo.mxfp4_values(code, scale)
    assert np.isnan(v[0, 32:96]).all() and v[0, 100] == 0.0 and v[0, 128] == 6 * 2.0 ** 125      # 7.8 saturates


def test_conv_is_torch_conv1d():
    r = np.random.default_rng(1)
    for width in (2, 3, 4):
        rows, w, b = r.normal(size=(width - 1 + 9, 5)), r.normal(size=(5, width)), r.normal(size=5)
        want = torch.nn.functional.conv1d(torch.from_numpy(rows.T[None]), torch.from_numpy(w[:, None]), torch.from_numpy(b),
                                          groups=5)[0].T
        assert np.allclose(lo.causal_conv(rows, w, b, False)[0], want.numpy(), rtol=1e-13)
        assert np.allclose(lo.causal_conv(rows, w, b, True)[0], torch.nn.functional.silu(want).numpy(), rtol=1e-13)


def test_scan_closed_form():
    """y_t = sum_{s <= t} C_t . B_s exp(A sum dt) dt_s u_s, written out; and a sequence in two parts."""
    r = np.random.default_rng(2)
    t, dim, n = 7, 3, 4
    u, dt, B, C = r.normal(size=(t, dim)), r.normal(size=(t, dim)), r.normal(size=(t, n)), r.normal(size=(t, n))
    A_log, D, bias, h0, z = r.normal(size=(dim, n)), r.normal(size=dim), r.normal(size=dim), r.normal(size=(dim, n)), r.normal(size=(t, dim))
    out, _, h, _ = lo.selective_scan(u, dt, B, C, A_log, D, bias, h0, z)
    d = torch.nn.functional.softplus(torch.from_numpy(dt + bias), threshold=100).numpy()
    A, cs = -np.exp(A_log), np.concatenate([np.zeros((1, dim)), np.cumsum(d, axis=0)])
    for i in range(t):
        y = (C[i] * np.exp(A * cs[i + 1][:, None]) * h0).sum(axis=1) + D * u[i]
        for s in range(i + 1):
            y += (C[i] * B[s] * np.exp(A * (cs[i + 1] - cs[s + 1])[:, None])).sum(axis=1) * d[s] * u[s]
        assert np.allclose(out[i], y * z[i] / (1 + np.exp(-z[i])), rtol=1e-11, atol=1e-13)
    a, _, mid, _ = lo.selective_scan(u[:3], dt[:3], B[:3], C[:3], A_log, D, bias, h0, z[:3])
    b, _, end, _ = lo.selective_scan(u[3:], dt[3:], B[3:], C[3:], A_log, D, bias, mid, z[3:])
    assert np.allclose(np.concatenate([a, b]), out) and np.allclose(end, h)


def test_logprobs_are_log_softmax():
    r = np.random.default_rng(3)
    x = np.round(r.normal(size=50) * 3, 1)                                # with ties
    x[7] = np.nan
    clean = torch.from_numpy(np.where(np.isnan(x), -np.inf, x))
    want = torch.log_softmax(clean, 0)
    lp, rank, h, tl, tt = lo.token_logprobs(x, 11, 6)
    assert np.isclose(lp, want[11]) and np.isclose(h, torch.distributions.Categorical(logits=clean).entropy())
    order = sorted((v for v in range(50) if v != 7), key=lambda v: (-x[v], v))
    assert rank == order.index(11) + 1 and tt.tolist() == order[:6] and np.allclose(tl, want[order[:6]])
    assert lo.token_logprobs(x, 7, 0)[:2] == (-np.inf, 50)
    x[3] = x[30] = np.inf
    lp, rank, h, tl, tt = lo.token_logprobs(x, 30, 4)
    assert np.isclose(lp, -np.log(2)) and rank == 2 and np.isclose(h, np.log(2)) and tt.tolist() == [3, 30, -1, -1]
    assert lo.token_logprobs(np.full(4, -np.inf), 2, 2)[:3] == (-np.inf, 3, 0.0)
