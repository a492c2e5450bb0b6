"""The layer operators (include/nhm_layer.h) on the paths that depend on a batch's shape, and on values in places where a
kernel's own layout counts, against plain 64-bit forms."""
import numpy as np
import pytest

from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_gpu_layer import bf16, check_scores, nhm  # noqa: E402,F401


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
