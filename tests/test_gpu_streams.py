"""Calls on a stream that is not the current one: memory that a call takes for itself belongs to its stream."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

SMALL = dict(hidden=256, n_heads=8, head_dim=64, d_state=128, n_groups=2, conv_width=4, rms_eps=1e-5)


@pytest.fixture(scope="module")
def nhm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_w8a8_linear_amd as m
    return m


def inputs(nhm, m=40, n=512, k=1024):
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    W = nhm.Fp8Weight((rand(n, k) * 50).to(torch.float8_e4m3fn).view(torch.uint8), torch.rand(n, generator=g, device="cuda"),
                      torch.full((1,), 0.01, device="cuda"))
    L = nhm.Lora((rand(3, 16, k) / 32).bfloat16(), rand(3, n, 16).bfloat16(), None)
    ids = torch.arange(m, dtype=torch.int32, device="cuda") % 4 - 1
    return rand(m, k).bfloat16(), W, L, ids


def calls(nhm):
    """{entry point: (a call of it without outputs or workspace, argument places of what it takes for itself)}."""
    x, W, L, ids = inputs(nhm)
    logits, cum = torch.randn(6, 5000, device="cuda"), torch.zeros(2, 3, device="cuda")
    ssm = torch.zeros((6, 8, 64, 128), device="cuda")
    conv = torch.zeros((6, 3, 8 * 64 + 2 * 2 * 128), dtype=torch.int16, device="cuda")
    par = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    slots = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    return {
        "nhm_fp8_linear_lora": (lambda st: nhm.fp8_linear_lora(x, W, L, ids, stream=st), (7, 11)),
        "nhm_beam_select": (lambda st: nhm.beam_select(logits, cum, 4, stream=st), (10, 11, 12, 13)),
        "nhm_beam_reorder": (lambda st: nhm.beam_reorder(par, slots, [ssm], [conv], g=SMALL, stream=st), (9,)),
        "nhm_fp8_linear_ex": (lambda st: nhm.fp8_linear(x, W, stream=st), (5, 8)),
        "nhm_fp8_quantize_static": (lambda st: nhm.quantize_static(x, W.a_scale, stream=st), (5,)),
        "nhm_fp8_dequant_channel_bf16": (lambda st: nhm.fp8_dequant_channel_bf16(W.w, W.w_scale, stream=st), (5,)),
    }


@pytest.mark.parametrize("name", ["nhm_fp8_linear_lora", "nhm_beam_select", "nhm_beam_reorder", "nhm_fp8_linear_ex",
                                  "nhm_fp8_quantize_static", "nhm_fp8_dequant_channel_bf16"])
def test_memory_of_a_call_belongs_to_its_stream(nhm, monkeypatch, name):
    """The library's call is replaced by one that notes its arguments and launches nothing."""
    call, places = calls(nhm)[name]
    side, seen = torch.cuda.Stream(), []
    monkeypatch.setattr(nhm.lib, name, lambda *a: seen.append(a) or 0)

    def owner(p):
        p = getattr(p, "value", p)
        return [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= p < s["address"] + s["total_size"]]

    for stream, want in ((side, side.cuda_stream), (None, torch.cuda.current_stream().cuda_stream)):
        kept = call(stream)  # noqa: F841
        assert [owner(seen[-1][i]) for i in places] == [[want]] * len(places)


def test_side_stream_without_workspace(nhm):
    """Calls queued behind other work on a side stream while the current stream takes and fills memory of their sizes."""
    x, W, L, ids = inputs(nhm)
    logits, cum = torch.randn(6, 50000, device="cuda"), torch.zeros(2, 3, device="cuda")
    want = [nhm.fp8_linear_lora(x, W, L, ids, exact=True), *nhm.beam_select(logits, cum, 4), nhm.fp8_linear(x, W, exact=True)]
    sizes = [nhm.fp8_linear_lora_workspace_bytes(40, 512, 1024, nhm.NHM_BF16, 16), nhm.beam_select_workspace_bytes(2, 3, 50000, 4),
             nhm.fp8_linear_workspace_bytes(40, 512, 1024, nhm.NHM_BF16)] + [t.numel() * t.element_size() for t in want]
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(3000000)
        got = [nhm.fp8_linear_lora(x, W, L, ids, exact=True, stream=side), *nhm.beam_select(logits, cum, 4, stream=side),
               nhm.fp8_linear(x, W, exact=True, stream=side)]
        for _ in range(2):
            noise = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del got, noise
