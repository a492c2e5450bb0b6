"""Pins of the serving operators' oracle against torch and hand-made values (CPU)."""
import numpy as np
import torch

from oracle import serving_oracle as so
from workloads import bf16_bits, linear_case


def test_lora_against_torch_and_merged_weights():
    """A row's adapter is the projection with scale B A added to the weight; rows without one are the projection."""
    from oracle import bf16_to_f64, fp8_linear, quantize_static
    r = np.random.default_rng(0)
    a, w, ws, sa = linear_case(6, 20, 32, extra=1)
    la, lb = bf16_bits(r.standard_normal((3, 8, 32))), bf16_bits(r.standard_normal((3, 20, 8)))
    ls = np.array([0.5, 2.0, -1.0], np.float32)
    ids = np.array([0, -1, 2, 2, 7, 1], np.int32)
    got = so.fp8_linear_lora(a, w, ws, sa, la, lb, ls, ids)
    base = fp8_linear(quantize_static(a, sa), w, ws, sa)
    x = torch.from_numpy(bf16_to_f64(a))
    for i, e in enumerate(ids):
        want = torch.from_numpy(base[i])
        if 0 <= e < 3:
            delta = ls[e] * torch.from_numpy(bf16_to_f64(lb[e])) @ torch.from_numpy(bf16_to_f64(la[e]))
            want = want + delta @ x[i]
        assert np.allclose(got[i], want.numpy(), rtol=1e-12, atol=1e-12)
    assert np.array_equal(got[1], base[1]) and np.array_equal(got[4], base[4])


def test_beam_select_against_torch():
    r = np.random.default_rng(1)
    x, cum = r.standard_normal((3, 4, 50)), -r.random((3, 4)).astype(np.float32)
    s, p, t, gap = so.beam_select(x, cum, 9)
    ref = torch.from_numpy(cum).double()[:, :, None] + torch.log_softmax(torch.from_numpy(x), dim=2)
    v, at = torch.topk(ref.reshape(3, -1), 9, dim=1)
    assert np.allclose(s, v.numpy(), atol=1e-12) and np.array_equal(p * 50 + t, at.numpy()) and gap > 0


def test_beam_select_by_hand():
    x = np.full((1, 2, 3), -np.inf)
    x[0, 0] = [0.0, 0.0, np.nan]
    x[0, 1, 2] = np.inf
    s, p, t, _ = so.beam_select(x, np.array([[-1.0, -2.0]]), 4)
    assert np.allclose(s[0, :3], [-1 - np.log(2), -1 - np.log(2), -2.0]) and s[0, 3] == -np.inf
    assert p[0].tolist() == [0, 0, 1, -1] and t[0].tolist() == [0, 1, 2, -1]
    s, p, t, _ = so.beam_select(x, np.array([[-1.0, -0.5]]), 2, finished=np.array([[1, 0]]), eos=1)
    assert s[0].tolist() == [-0.5, -1.0] and p[0].tolist() == [1, 0] and t[0].tolist() == [2, 1]


def test_beam_reorder_by_hand():
    pool = np.arange(6.0)[:, None].repeat(2, axis=1)
    new = so.beam_reorder(np.array([[2, 2, 0, -1]]), np.array([[5, 1, 3, 0]], np.int32), [pool])
    # beam 0 keeps parent 2's slot 3, beam 2 parent 0's slot 5; beams 1 and 3 get the slots of beams 1 and 3
    assert new[0].tolist() == [3, 1, 5, 0]
    assert pool[:, 0].tolist() == [0.0, 3.0, 2.0, 3.0, 4.0, 5.0]


def test_batch_plan_by_hand():
    p = so.batch_plan([2, 0, 3], 7, past=[0, 4, 9], adapters=[5, 6, -1])
    assert p["cu_seqlens"].tolist() == [0, 2, 2, 5] and p["has_initial"].tolist() == [0, 1, 1]
    assert p["token_seq"].tolist() == [0, 0, 2, 2, 2, -1, -1]
    assert p["token_pos"].tolist() == [0, 1, 9, 10, 11, -1, -1]
    assert p["token_adapter"].tolist() == [5, 5, -1, -1, -1, -1, -1]


def test_mixer_without_adapters_is_the_mixer():
    from oracle import mixer_sequence
    g = dict(hidden=256, n_heads=8, head_dim=64, d_state=128, n_groups=2, conv_width=4, rms_eps=1e-5)
    import workloads.synthetic as w
    p = w.block_params(3, 0, g)
    h, win, st = w.hidden(3, 4, g), w.conv_pool(3, 0, 1, g=g)[0], w.ssm_pool(3, 0, 1, g=g)[0]
    ref = mixer_sequence(p, h, win, st, g)
    lay_n, inner = p["in_w"].shape[0], p["out_w"].shape[1]
    zero_in = (np.zeros((1, 8, 256), np.uint16), np.zeros((1, lay_n, 8), np.uint16), None)
    zero_out = (np.zeros((1, 8, inner), np.uint16), np.zeros((1, 256, 8), np.uint16), None)
    for li, lo in ((None, None), (zero_in, zero_out)):
        out, window, state = so.mixer_sequence_lora(p, li, lo, np.zeros(4, np.int32), h, win, st, g)
        assert np.array_equal(out, ref["out"]) and np.array_equal(window, ref["window"])
        assert np.array_equal(state, ref["state"])
