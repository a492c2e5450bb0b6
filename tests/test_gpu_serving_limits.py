"""The serving operators at the ends of their documented limits."""
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
